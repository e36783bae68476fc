"""Arguments the transformer-layer entry points refuse: each is checked before any GPU call (no GPU here)."""
from __future__ import annotations

import os

import pytest

P = 4096  # an aligned address that is never read: every call here is refused


@pytest.fixture(scope="module")
def L():
    from signal_gated_tiled_amd import _sgt
    if not os.path.exists(_sgt.LIB_PATH):
        from signal_gated_tiled_amd import build
        build.build()
    return _sgt.lib()


EINVAL, EUNSUP = -1, -2


def norm(L, **kw):
    a = dict(x=P, x_dtype=1, x_stride=64, residual=P, sum_out=P, r_dtype=1, weight=P, w_dtype=1, out=P, out_dtype=1,
             scales=None, block=0, T=4, H=64, eps=1e-6, stream=None)
    a.update(kw)
    return L.sgt_rms_norm(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(x_dtype=2), EINVAL, "x_dtype"), (dict(r_dtype=7), EINVAL, "r_dtype"), (dict(w_dtype=-1), EINVAL, "w_dtype"),
    (dict(out_dtype=3), EINVAL, "out_dtype"), (dict(T=-1), EINVAL, "T=-1"), (dict(T=2 ** 31), EINVAL, "T="),
    (dict(H=0), EINVAL, "H=0"), (dict(H=65537, x_stride=65537), EUNSUP, "65536"), (dict(x_stride=63), EINVAL, "x_stride"),
    (dict(eps=-1.0), EINVAL, "eps"), (dict(eps=float("nan")), EINVAL, "eps"), (dict(eps=float("inf")), EINVAL, "eps"),
    (dict(out_dtype=2), EINVAL, "scales"), (dict(out_dtype=2, scales=P, block=64), EINVAL, "block"),
    (dict(scales=P), EINVAL, "8-bit"), (dict(block=128), EINVAL, "8-bit"),
    (dict(x=None), EINVAL, "NULL"), (dict(weight=None), EINVAL, "NULL"), (dict(out=None), EINVAL, "NULL"),
    (dict(x=P + 1), EINVAL, "aligned"), (dict(out_dtype=2, scales=P + 2), EINVAL, "aligned"),
])
def test_rms_norm(L, kw, status, word):
    assert norm(L, **kw) == status
    assert word in L.sgt_last_error().decode()


def gate(L, **kw):
    a = dict(logits=P, dtype=0, stride=64, bias=None, ids=P, gate=P, T=4, E=64, topk=8, score=0, n_group=1, topk_group=1,
             group_top=1, renorm=1, scale=1.0, stream=None)
    a.update(kw)
    return L.sgt_moe_gate(*a.values())


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=2), "dtype"), (dict(score=2), "score"), (dict(T=-1), "T ="), (dict(E=0, stride=0), "E ="),
    (dict(E=1025, stride=1025), "E ="), (dict(topk=0), "topk"), (dict(topk=65), "topk"), (dict(E=4, topk=5), "topk"),
    (dict(stride=63), "stride"), (dict(n_group=3), "n_group"), (dict(n_group=0), "n_group"),
    (dict(E=128, stride=128, n_group=128), "n_group"),
    (dict(n_group=8, topk_group=9), "topk_group"), (dict(n_group=8, topk_group=0), "topk_group"),
    (dict(n_group=16, topk_group=1, topk=5), "topk"), (dict(group_top=3), "group_top"),
    (dict(n_group=64, topk_group=8, group_top=2), "group_top"), (dict(scale=float("nan")), "scale"),
    (dict(logits=None), "NULL"), (dict(ids=None), "NULL"), (dict(gate=None), "NULL"), (dict(bias=P + 2), "aligned"),
])
def test_moe_gate(L, kw, word):
    assert gate(L, **kw) == EINVAL
    assert word in L.sgt_last_error().decode()


def prompt(L, **kw):
    a = dict(q=P, q_token=1024, q_head=128, k=P, k_token=256, k_head=128, v=P, v_token=256, v_head=128, out=P, lse=P,
             cu_q=P, cu_k=P, n_seqs=2, total_q=100, total_k=100, Hq=8, Hkv=2, D=128, causal=1, scale=0.1, stream=None)
    a.update(kw)
    return L.sgt_attn_prompt(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(Hq=7), EINVAL, "Hq"), (dict(Hkv=0), EINVAL, "Hkv"), (dict(Hq=1026), EINVAL, "Hq"), (dict(D=96), EUNSUP, "head"),
    (dict(n_seqs=-1), EINVAL, "n_seqs"), (dict(n_seqs=0), EINVAL, "no sequence"), (dict(total_q=-1), EINVAL, "total_q"),
    (dict(total_k=2 ** 31), EINVAL, "total_k"), (dict(scale=float("inf")), EINVAL, "scale"),
    (dict(q_token=1020), EINVAL, "stride"), (dict(v_head=-8), EINVAL, "stride"), (dict(k_token=1 << 24), EUNSUP, "stride"),
    (dict(total_q=2 ** 30, Hq=1024, Hkv=1), EINVAL, "rows"),
    (dict(q=None), EINVAL, "NULL"), (dict(k=None), EINVAL, "NULL"), (dict(out=None), EINVAL, "NULL"),
    (dict(cu_k=None), EINVAL, "NULL"), (dict(v=P + 8), EINVAL, "aligned"), (dict(lse=P + 2), EINVAL, "misaligned"),
])
def test_attn_prompt(L, kw, status, word):
    assert prompt(L, **kw) == status
    assert word in L.sgt_last_error().decode()


def decode(L, **kw):
    a = dict(q=P, q_stride=1024, k=P, v=P, page=4096, slot=256, head=128, n_pages=9, page_size=16, table=P, table_stride=4,
             max_pages=4, lens=P, out=P, out_dtype=1, lse=P, workspace=P, bytes=1 << 40, B=3, Hq=8, Hkv=2, D=128, scale=0.1,
             stream=None)
    a.update(kw)
    return L.sgt_attn_decode(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(Hq=9), EINVAL, "Hq"), (dict(D=32), EUNSUP, "head"), (dict(B=-1), EINVAL, "B ="), (dict(out_dtype=2), EINVAL, "out"),
    (dict(page_size=0), EINVAL, "page_size"), (dict(n_pages=-1), EINVAL, "n_pages"), (dict(max_pages=-1), EINVAL, "max_pages"),
    (dict(table_stride=3), EINVAL, "table_stride"),
    (dict(max_pages=1 << 20, table_stride=1 << 20, page_size=1 << 12), EUNSUP, "tokens"),
    (dict(q_stride=1020), EINVAL, "stride"), (dict(slot=-8), EINVAL, "stride"), (dict(scale=float("nan")), EINVAL, "scale"),
    (dict(q=None), EINVAL, "NULL"), (dict(v=None), EINVAL, "NULL"), (dict(table=None), EINVAL, "NULL"),
    (dict(lens=None), EINVAL, "NULL"), (dict(workspace=None), EINVAL, "NULL"), (dict(k=P + 8), EINVAL, "aligned"),
    (dict(workspace=P + 8), EINVAL, "aligned"), (dict(lens=P + 2), EINVAL, "misaligned"), (dict(bytes=0), EINVAL, "needed"),
])
def test_attn_decode(L, kw, status, word):
    assert decode(L, **kw) == status
    assert word in L.sgt_last_error().decode()


def test_nothing_to_do_is_no_error(L):
    assert norm(L, T=0, x=None, out=None) == 0
    assert gate(L, T=0, logits=None) == 0
    assert prompt(L, total_q=0, q=None, n_seqs=0) == 0
    assert decode(L, B=0, q=None) == 0


def test_workspace_query():
    import signal_gated_tiled_amd as sgt
    assert sgt.attn_decode_workspace(3, 8, 2, 128) > 0
    for bad in ((-1, 8, 2, 128), (3, 8, 3, 128), (3, 8, 2, 100), (1 << 24, 8, 2, 128)):
        with pytest.raises(sgt.SgtError):
            sgt.attn_decode_workspace(*bad)


def test_binding_refuses_tensors_of_the_host():
    torch = pytest.importorskip("torch")
    import signal_gated_tiled_amd as sgt
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 8, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        sgt.rms_norm(x, x[0], x)
    with pytest.raises(ValueError, match="GPU tensor"):
        sgt.moe_gate(x, i, i.float())
    h = x.view(2, 1, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        sgt.attn_prompt(h, h, h, h, i[0], i[0])
    with pytest.raises(ValueError, match="GPU tensor"):
        sgt.attn_decode(h, h, h, i, i[:, 0], h, x)
