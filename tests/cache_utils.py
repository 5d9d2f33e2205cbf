"""Inputs and comparisons of the 8-bit cache's tests: a pool whose pages are dealt to
sequences in random order, with one page that belongs to none."""

from __future__ import annotations

import numpy as np
import torch

from hstu_sequential_transduction_b200 import ops
from oracle import cache as oc

PAGE = oc.PAGE


def pages(n):
    return -(-n // PAGE)


def make_pool(rng, lens, heads, d, extra=0, cols=None, gaps=False, std=1.0):
    """(pool, table, free pages): a pool holding `lens` random tokens per sequence, every
    byte of its other slots and pages random too (NaN codes among them)."""
    need = [pages(x) for x in lens]
    n = sum(need) + extra + 1
    order = rng.permutation(n)
    cols = cols or max([1] + need)
    pool = oc.new_pool(n, heads, d)
    for name in ("k_codes", "v_codes"):
        pool[name][:] = rng.integers(0, 256, pool[name].shape)
    for name in ("k_scale", "v_scale"):
        pool[name][:] = np.exp2(rng.integers(-9, -5, pool[name].shape)) * std
    pool["timestamps"][:] = rng.integers(-2 ** 40, 2 ** 40, pool["timestamps"].shape)
    pool["positions"][:] = rng.integers(0, 2 ** 20, pool["positions"].shape)
    pool["weights"][:] = rng.random(pool["weights"].shape)
    table = np.full((len(lens), cols), -7, np.int32)
    at = 0
    for b, L in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        ts = 1_700_000_000 + np.cumsum(rng.exponential(200.0, need[b] * PAGE)).astype(np.int64)
        for j in range(L):
            page, slot = table[b, j // PAGE], j % PAGE
            for h in range(heads):
                pool["k_codes"][page, h, slot] &= 0xBF  # at most 1.875: finite, and scores stay moderate
                pool["v_codes"][page, h, :, slot] &= 0xBF
            pool["timestamps"][page, slot] = ts[j]
            pool["positions"][page, slot] = j * 3 + j % 2 if gaps else j
    return pool, table, order[at:-1], order[-1]


def to_cache(pool, dev, weights=True):
    t = {k: torch.from_numpy(v.copy()).to(dev) for k, v in pool.items()}
    return ops.HstuCache(t["k_codes"], t["v_codes"], t["k_scale"], t["v_scale"], t["timestamps"], t["positions"],
                         t["weights"] if weights else None)


def pool_of(cache):
    names = ("k_codes", "v_codes", "k_scale", "v_scale", "timestamps", "positions", "weights")
    return {n: getattr(cache, n).cpu().numpy() for n in names if getattr(cache, n) is not None}


def assert_pool_equal(got, want):
    """Every byte, with NaN scales equal to NaN scales."""
    for name, w in want.items():
        if name in got:
            np.testing.assert_array_equal(got[name], w, err_msg=name)


def dev(a, device, dtype=None):
    return None if a is None else torch.as_tensor(np.asarray(a), dtype=dtype).to(device)


def end_pos(pool, table, lens):
    """The position after each sequence's last cached token."""
    return np.array([pool["positions"][table[b, (L - 1) // PAGE], (L - 1) % PAGE] + 1 if L else 0
                     for b, L in enumerate(lens)], np.int32)
