"""examples/transformer_layer.py step by step against plain fp64 formulas, each step on the inputs it had.

Tolerances: bf16 products of a few hundred terms (fp32 sums) rounded to bf16 2^-8 |c| plus 1e-4; fp32 results 1e-4 of
sums of magnitude about 1 (1e-3 where bf16 rows are combined); the layer operators' own as in test_gpu_layer.py."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import signal_gated_tiled_amd as sgt  # noqa: E402
from oracle import layer as O  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("transformer_layer", os.path.join(ROOT, "examples", "transformer_layer.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules[spec.name] = m   # (dataclasses look their module up)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def near(got, ref, rel, floor):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= rel * np.abs(ref) + floor)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], ref[bad][:3])


@pytest.mark.parametrize("lens", [[200, 1, 55], [37, 219]])
def test_prompt_layer(ex, lens):
    L = ex.make_layer(3)
    x, cu, partials = ex.inputs(L, lens, 4)
    with sgt.Context(0) as ctx:
        got = ex.prompt(ctx, L, x, cu, partials)
    r, T_r = L.rank, x[0].shape[0]
    near(got["normed"], O.rms_norm(f64(x[r]), None, f64(L.norm1), 1e-6)[1], 2.0 ** -8, 1e-6)
    normed = torch.empty_like(x[r])
    rows_all = []
    for p in range(L.W):
        sgt.rms_norm(x[p], L.norm1, normed)
        rows_all.append(normed.clone())
    near(got["qkv"], f64(torch.cat(rows_all)) @ f64(L.qkv), 2.0 ** -8, 1e-4)
    q, k, v = ex.split_heads(L, got["qkv"])
    off = cu.cpu().numpy()
    out, _, spread = O.packed_attention(f64(q), f64(k), f64(v), off, off, L.D ** -0.5, True)
    assert (np.abs(f64(got["attn"]) - out) <= 2.0 ** -8 * (spread + np.abs(out)) + 1e-6).all()
    block = slice(r * T_r, (r + 1) * T_r)
    ref = f64(got["attn"]).reshape(sum(lens), -1)[block] @ f64(L.o) + sum(f64(partials[p]) for p in range(L.W) if p != r)
    near(got["summed"], ref, 1e-4, 1e-4)
    s, y = O.rms_norm(f64(got["summed"]), f64(x[r]), f64(L.norm2), 1e-6)
    near(got["stream"], s, 2.0 ** -8, 1e-6)
    near(got["rows"], y, 2.0 ** -8, 1e-6)
    ids, gate = O.moe_gate(f64(got["logits"]), L.topk, score="sigmoid", bias=f64(L.bias), n_group=4, topk_group=2,
                           group_top=2, scale=2.0)
    assert np.array_equal(got["ids"].cpu().numpy(), ids)
    near(got["gate"], gate, 1e-5, 1e-7)
    rows, ref = f64(got["rows"]), np.zeros((T_r, L.hidden))
    for t in range(T_r):
        for j in range(L.topk):
            y = rows[t] @ f64(L.expert[ids[t, j]])
            ref[t] += f64(got["gate"])[t, j] * y
    # each expert's row is rounded to bf16: 2^-8 of values of magnitude up to 5, weights that sum to 2
    near(got["moe"], ref, 2.0 ** -8, 2 * 5 * 2.0 ** -8)


def test_tokens(ex):
    L, lens, steps = ex.make_layer(5), [33, 1, 160, 62], 5
    x, cu, partials = ex.inputs(L, lens, 6)
    qkv = torch.randn(sum(lens), L.qkv.shape[1], device="cuda").to(torch.bfloat16)
    one, two = (ex.Tokens(L, qkv, lens, steps + 1) for _ in range(2))
    ks = [[t for t in f64(part)] for part in ex.split_heads(L, qkv)[1:]]
    off = np.cumsum([0] + lens)
    cache = [[ks[i][off[b]:off[b + 1]] for b in range(len(lens))] for i in range(2)]
    for s in range(steps):
        row = torch.randn(len(lens), L.hidden, device="cuda").to(torch.bfloat16)
        for t in (one, two):
            t.x.copy_(row)
        before = f64(one.add)
        one.step()
        two.replay()
        torch.cuda.synchronize()
        assert torch.equal(one.out, two.out) and torch.equal(one.lse, two.lse) and torch.equal(one.lens, two.lens)
        total, normed = O.rms_norm(f64(row), before, f64(L.norm1), 1e-6)
        near(one.add, total, 2.0 ** -8, 1e-6)
        near(one.row, normed, 2.0 ** -8, 1e-6)
        near(one.qkv, f64(one.row) @ f64(L.qkv), 2.0 ** -8, 1e-4)
        q, k, v = (f64(t) for t in ex.split_heads(L, one.qkv))
        for b in range(len(lens)):
            for i, new in enumerate((k, v)):
                cache[i][b].append(new[b])
            kk, vv = np.stack(cache[0][b]), np.stack(cache[1][b])
            for h in range(L.Hq):
                hk = h // (L.Hq // L.Hkv)
                z = kk[:, hk] @ q[b, h] * L.D ** -0.5
                w = np.exp(z - z.max())
                w /= w.sum()
                bound = 2.0 ** -8 * (w @ np.abs(vv[:, hk]) + np.abs(w @ vv[:, hk])) + 1e-6
                assert (np.abs(f64(one.out)[b, h] - w @ vv[:, hk]) <= bound).all()
