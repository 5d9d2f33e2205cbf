"""Blocks of the 8-bit cache that are not finite: a NaN scale, as the append writes it, and
NaN codes (0x7f, 0xff) under a finite scale, as a pool that was filled in another way may
hold them.  Attention spreads NaN exactly as far as the formula does; all else stays
within the bounds of the finite case."""

import numpy as np
import pytest
import torch

from cache_utils import PAGE, pool_of
from hstu_sequential_transduction_b200 import ops
from oracle import cache as oc
from test_gpu_cache import _attn_inputs, _check_attn, _evict_inputs, _run_attn, _run_evict, _values, _want_attn

pytestmark = pytest.mark.gpu

# (type, head width, new tokens): the float32 kernel, the one for few rows, the tensor cores'
KERNELS = [("f32", 32, 3), ("f32", 64, 20), ("bf16", 64, 1), ("bf16", 128, 30), ("bf16", 64, 65), ("bf16", 128, 140)]
LENS = [300, 70, 130]  # last pages of 44, 6 and 2 tokens


def _check_with_nan(x, out, wout):
    want, want_w, terms = _want_attn(x)
    got, got_w = _values(out), _values(wout)
    assert np.isnan(want).any()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(np.isnan(got_w), np.isnan(want_w))
    off, woff = np.isnan(want), np.isnan(want_w)
    zero = lambda a, m: np.where(m, 0.0, a)  # noqa: E731
    t = dict(out={n: zero(a, off) for n, a in terms["out"].items()}, w={n: zero(a, woff) for n, a in terms["w"].items()})
    _check_attn(x, torch.as_tensor(zero(got, off)), zero(want, off), t, torch.as_tensor(zero(got_w, woff)),
                zero(want_w, woff), np.full(want_w.shape, -5.0))


@pytest.mark.parametrize("dtype,d,new", KERNELS)
@pytest.mark.parametrize("name,page", [("k", 1), ("v", 1), ("k", 4), ("v", 4), ("k", 0), ("v", 0)])
def test_attention_of_a_block_with_a_nan_scale(dtype, d, new, name, page, cuda_device):
    """One page of one head, whole or the ragged last one, of keys or of values."""
    x = _attn_inputs((LENS, [new] * 3, None), dtype, d, 2, 71)
    x["pool"][name + "_scale"][x["table"][0, page], 1] = np.nan
    x["pool"][name + "_scale"][x["table"][2, 2], 0] = np.nan  # its last page, of two tokens
    out, wout, ws, _ = _run_attn(x, cuda_device)
    assert ops.hstu_check_device_flag(ws) == (0, 0)
    _check_with_nan(x, out, wout)


@pytest.mark.parametrize("case", [3, 4, 7])
@pytest.mark.parametrize("heads,d", [(2, 32), (2, 64), (1, 128)])
@pytest.mark.parametrize("how", ["scale", "code"])
def test_evict_blocks_that_are_not_finite(case, heads, d, how, cuda_device):
    """A kept value that is not finite makes its new block's scale NaN; every other block,
    and what is no code, is as the definition has it byte for byte."""
    x = _evict_inputs(case, heads, d, 83)
    pool, table, lens, new_pages, keep, first, recent = x
    rng = np.random.default_rng(4)
    for name in "kv":
        for b in range(len(lens)):
            j = int(rng.integers(0, int(lens[b])))
            page, slot, h, e = table[b, j // PAGE], j % PAGE, int(rng.integers(0, heads)), int(rng.integers(0, d))
            pool["weights"][page, slot] = 50.0 + b  # kept
            if how == "scale":
                pool[name + "_scale"][page, h] = np.nan
            else:
                pool[name + "_codes"][(page, h, slot, e) if name == "k" else (page, h, e, slot)] = 0x7F
    want = {n: a.copy() for n, a in pool.items()}
    w_table, w_lens, w_kept = oc.evict(want, table, lens, new_pages, keep, first, recent)
    cache, (table2, lens2, kept), flag = _run_evict(*x, cuda_device)
    assert flag == (0, 0)
    np.testing.assert_array_equal(kept.cpu().numpy(), w_kept)
    np.testing.assert_array_equal(table2.cpu().numpy(), w_table)
    np.testing.assert_array_equal(lens2.cpu().numpy(), w_lens)
    got = pool_of(cache)
    # (where all that is kept is the last tokens, these may be gone)
    assert recent >= keep or any(np.isnan(want[n + "_scale"][new_pages[new_pages >= 0]]).any() for n in "kv")
    for n in ("k_scale", "v_scale", "timestamps", "positions", "weights"):
        np.testing.assert_array_equal(got[n], want[n], err_msg=n)
    for n in "kv":
        finite = ~np.isnan(want[n + "_scale"])  # under a NaN scale every code means NaN
        np.testing.assert_array_equal(got[n + "_codes"][finite], want[n + "_codes"][finite], err_msg=n)
