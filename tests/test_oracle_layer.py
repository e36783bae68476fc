"""Pins of the fp64 definitions of the transformer-layer operators (CPU): closed forms, brute force and invariants."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import layer as L


def test_rms_norm_closed_form():
    s, y = L.rms_norm([[3.0, 4.0]], [[0.0, 0.0]], [2.0, 1.0], 0.0)
    assert np.allclose(s, [[3, 4]]) and np.allclose(y, [[6 / math.sqrt(12.5), 4 / math.sqrt(12.5)]])
    s, y = L.rms_norm([[1.0, -1.0]], [[1.0, 1.0]], [1.0, 1.0], 1e-6)
    assert np.allclose(s, [[2, 0]]) and np.allclose(y, [[2 / math.sqrt(2 + 1e-6), 0]])


def test_f8_scales_cover_ragged_blocks():
    y = np.array([[448.0, 1.0, -896.0]])
    assert np.allclose(L.f8_scales(y, 0), [[2.0]])
    assert np.allclose(L.f8_scales(y, 2), [[1.0, 2.0]])
    assert L.f8_scales(np.zeros((1, 4)), 0)[0, 0] == 2.0 ** -126


def test_gate_order_ties_and_sums():
    ids, gate = L.moe_gate([[0.0, 1.0, 1.0, 0.0]], 3)
    assert ids.tolist() == [[1, 2, 0]]
    assert np.allclose(gate.sum(), 1.0) and np.allclose(gate[0, 0] / gate[0, 2], math.e)
    ids, gate = L.moe_gate([[0.0, 1.0, 1.0, 0.0]], 2, score="sigmoid", bias=[0.6, 0, 0, 0], renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(gate, [[1.0, 2 / (1 + math.exp(-1))]])


def test_gate_groups_limit_the_choice():
    x = [[9.0, 0.0, 5.0, 5.0, 1.0, 1.0]]
    assert L.moe_gate(x, 2, score="sigmoid", n_group=3, topk_group=1, group_top=2)[0].tolist() == [[2, 3]]
    assert L.moe_gate(x, 2, score="sigmoid", n_group=3, topk_group=1, group_top=1)[0].tolist() == [[0, 1]]
    assert L.moe_gate([[-np.inf, np.nan, 3.0]], 3)[0].tolist() == [[2, 0, 1]]


@pytest.mark.parametrize("lq,lk", [(3, 3), (2, 5), (4, 2), (1, 0)])
def test_attention_is_the_definition(lq, lk):
    rng = np.random.default_rng(lq * 10 + lk)
    q, k, v = rng.standard_normal((lq, 2, 4)), rng.standard_normal((lk, 1, 4)), rng.standard_normal((lk, 1, 4))
    out, lse, mag = L.attention(q, k, v, 0.5, True)
    for i in range(lq):
        for h in range(2):
            seen = [j for j in range(lk) if j <= i + lk - lq]
            w = [math.exp(0.5 * float(q[i, h] @ k[j, 0])) for j in seen]
            if not seen:
                assert (out[i, h] == 0).all() and lse[i, h] == -np.inf
                continue
            assert math.isclose(lse[i, h], math.log(sum(w)), rel_tol=1e-12, abs_tol=1e-12)
            assert np.allclose(out[i, h], sum(a * v[j, 0] for a, j in zip(w, seen)) / sum(w))
            assert (mag[i, h] >= np.abs(out[i, h]) - 1e-12).all()


def test_paged_is_packed_over_the_same_tokens():
    rng = np.random.default_rng(0)
    cache_k, cache_v = rng.standard_normal((5, 4, 2, 8)), rng.standard_normal((5, 4, 2, 8))
    table, lens = np.array([[3, 0, 9], [1, 4, 2]]), [6, 12]
    q = rng.standard_normal((2, 4, 8))
    out, lse, _ = L.paged_attention(q, cache_k, cache_v, table, lens, 0.3)
    k = np.concatenate([cache_k[3], cache_k[0][:2]])
    v = np.concatenate([cache_v[3], cache_v[0][:2]])
    ref = L.attention(q[:1], k, v, 0.3, False)
    assert np.allclose(out[0], ref[0][0]) and np.allclose(lse[0], ref[1][0])
    # a page outside the cache is not seen
    k, v = np.concatenate([cache_k[i] for i in (1, 4, 2)]), np.concatenate([cache_v[i] for i in (1, 4, 2)])
    assert np.allclose(out[1], L.attention(q[1:], k, v, 0.3, False)[0][0])
