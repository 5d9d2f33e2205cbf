"""Pins of the 8-bit cache's oracle: hand-worked scales and codes, an append of many
parts against one, attention against a dense formulation, eviction against a sort."""

import numpy as np
import pytest
import torch

from cache_utils import PAGE, end_pos, make_pool, pages
from oracle import cache as oc


def test_block_scale_by_hand():
    assert oc.scale_of(0.0) == 0.0
    assert oc.scale_of(448.0) == 1.0 and oc.scale_of(np.nextafter(np.float32(448), np.float32(1e9))) == 2.0
    assert oc.scale_of(224.0) == 0.5 and oc.scale_of(1.75) == 2.0 ** -8 and oc.scale_of(1.0) == 2.0 ** -8
    assert oc.scale_of(1e-45) == 2.0 ** -126
    assert np.isnan(oc.scale_of(np.inf)) and np.isnan(oc.scale_of(np.nan))


def test_codes_match_torch():
    x = torch.randn(4096, generator=torch.Generator().manual_seed(0)) * 100
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(oc.encode(x.numpy()), want)


@pytest.mark.parametrize("cuts", [(0, 130), (0, 1, 130), (0, 63, 64, 65, 130), (0, 100, 130)])
def test_append_in_parts_rounds_within_half_a_step(cuts):
    """Values come back within half an E4M3 step (2^-4 relative, 2^-10 of the block's
    scale below the normal range) for each rounding: one, and one more per growth of
    the block's scale, of which every later part makes at most one."""
    rng = np.random.default_rng(3)
    H, d, n = 2, 8, 130
    k, v = rng.standard_normal((n, H, d)), rng.standard_normal((n, H, d))
    pool, table = oc.new_pool(3, H, d), np.array([[2, 0, 1]], np.int32)
    lens, pos = np.zeros(1, np.int32), np.zeros(1, np.int32)
    for lo, hi in zip(cuts[:-1], cuts[1:]):
        lens, pos = oc.append(pool, k[lo:hi], v[lo:hi], table, lens, pos, np.array([0, hi - lo]), np.arange(lo, hi), None)
    assert lens[0] == n and pos[0] == n
    parts = len(cuts) - 1
    for h in range(H):
        for name, x in (("k", k), ("v", v)):
            got = oc.tokens(pool, name, table[0], n, h)
            step = np.repeat(pool[name + "_scale"][table[0], h], PAGE)[:n, None] * 2.0 ** -10
            assert np.all(np.abs(got - x[:, h]) <= parts * np.maximum(2.0 ** -4 * np.abs(x[:, h]) * 1.07, step))
    np.testing.assert_array_equal(pool["timestamps"][table[0]].reshape(-1)[:n], np.arange(n))
    np.testing.assert_array_equal(pool["positions"][table[0]].reshape(-1)[:n], np.arange(n))


def test_attention_is_the_dense_sum():
    rng = np.random.default_rng(5)
    lens, n, H, d = [70, 0, 3], [2, 3, 1], 2, 4
    pool, table, _, _ = make_pool(rng, lens, H, d, gaps=True)
    off = np.concatenate([[0], np.cumsum(n)])
    q = rng.standard_normal((6, H, d))
    ts = 1_700_000_000 + rng.integers(0, 10 ** 6, 6)
    rp, rt = rng.standard_normal(2 * 20 + 1), rng.standard_normal(10)
    pos = end_pos(pool, table, lens)
    out, w, _ = oc.attn(pool, q, table, np.array(lens), pos, off, ts, np.array([1, 0, 1]), rp, rt, 0.25, -20, 20)
    want_w = pool["weights"].astype(np.float64).copy()
    for b in range(3):
        for i in range(n[b]):
            p_i = pos[b] + (min(i, n[b] - 1) if b != 1 else i)  # one candidate, after the history
            t_i = ts[off[b] + i]
            for h in range(H):
                o = np.zeros(d)
                for j in range(lens[b]):
                    pg, sl = table[b, j // PAGE], j % PAGE
                    kk = oc.VALUES[pool["k_codes"][pg, h, sl]] * pool["k_scale"][pg, h]
                    vv = oc.VALUES[pool["v_codes"][pg, h, :, sl]] * pool["v_scale"][pg, h]
                    dp = int(min(max(p_i - int(pool["positions"][pg, sl]), -20), 20))
                    bk = min(9, int(max(t_i - pool["timestamps"][pg, sl], 0) + 1).bit_length() - 1)
                    s = q[off[b] + i, h] @ kk + rp[dp + 20] + rt[bk]
                    P = 0.25 * s / (1 + np.exp(-s))
                    o += P * vv
                    want_w[pg, sl] += abs(P)
                np.testing.assert_allclose(out[off[b] + i, h], o, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(w, want_w, rtol=1e-12)


def test_kept_tokens_by_hand():
    w = [5, 1, 1, 9, float("nan"), 1, -float("inf"), 0]
    assert oc.kept_tokens(w, 8, 8, 1, 1) == list(range(8))
    assert oc.kept_tokens(w, 8, 3, 0, 0) == [0, 1, 3]          # ties at 1: the lowest index
    assert oc.kept_tokens(w, 8, 4, 1, 1) == [0, 1, 3, 7]
    assert oc.kept_tokens(w, 8, 2, 4, 4) == [6, 7]             # the last ones first
    assert oc.kept_tokens(w, 8, 5, 2, 2) == [0, 1, 3, 6, 7]
    assert oc.kept_tokens(w, 8, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]  # NaN below -inf


def test_evicted_values_survive():
    rng = np.random.default_rng(9)
    lens = [200, 50]
    pool, table, free, _ = make_pool(rng, lens, 2, 8, extra=pages(100), gaps=True)
    before = {h: oc.tokens(pool, "k", table[0], 200, h) for h in range(2)}
    new_pages = np.full(table.shape, -1, np.int32)
    new_pages[0, :pages(100)] = free
    nt, nl, kept = oc.evict(pool, table, np.array(lens, np.int32), new_pages, 100, 4, 16)
    assert list(nl) == [100, 50] and list(nt[1]) == list(table[1]) and list(nt[0]) == list(new_pages[0])
    assert list(kept[1]) == list(range(50)) + [-1] * 50
    for h in range(2):
        got, want = oc.tokens(pool, "k", nt[0], 100, h), before[h][kept[0]]
        step = np.repeat(pool["k_scale"][nt[0, :2], h], PAGE)[:100, None] * 2.0 ** -10
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), step))
