"""What the 8-bit cache's attention reports when its offsets or its pipeline go wrong, and
that nothing else changes then."""

import numpy as np
import pytest
import torch

from cache_utils import assert_pool_equal, dev, make_pool, pool_of, to_cache
from hstu_sequential_transduction_b200 import ops

pytestmark = pytest.mark.gpu

# (type, head width, new tokens of a sequence): the float32 kernel, the one for few rows, the tensor cores'
KERNELS = [("f32", 32, 5), ("bf16", 64, 5), ("bf16", 128, 70)]


def _call(dtype, d, off, T, lens, device, max_seq_len, fill=None, **kw):
    """An attention over caches of `lens` tokens; (out, weights_out, flag)."""
    rng = np.random.default_rng(11)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pool, table, _, _ = make_pool(rng, lens, 2, d)
    cache = to_cache(pool, device)
    B = len(lens)
    q = torch.as_tensor(rng.standard_normal((T, 2, d)), dtype=torch.float32).to(tdt).to(device)
    args = dict(max_seq_len=max_seq_len, max_cache_len=max(list(lens) + [1]), inv_n=1 / 64, pos_lo=-32, pos_hi=32)
    rp, rt = 0.1 * torch.randn(65, device=device), 0.1 * torch.randn(16, device=device)
    t = dev(table if B else np.zeros((0, 1)), device, torch.int32)
    ws = ops.alloc_workspace(ops.hstu_cache_attn_workspace_size(q, cache, t, rp, rt, weights=True, **args), device)
    out = torch.full_like(q, 7.0)
    wout = torch.full_like(cache.weights, -5.0)
    ops.hstu_cache_attn_fwd(q, cache, t, dev(lens, device, torch.int32), None, dev(off, device, torch.int64),
                            torch.full((T,), 1_700_000_000, device=device), None, rp, rt, out=out, weights_out=wout,
                            workspace=ws, **args, **kw)
    return out, wout, ops.hstu_check_device_flag(ws)


@pytest.mark.parametrize("dtype,d,n", KERNELS)
@pytest.mark.parametrize("lens", [[90, 0, 130], [0, 0, 0]])
@pytest.mark.parametrize("front,back,bits", [(0, 0, 0), (3, 0, 1), (0, 4, 16), (2, 1, 17)])
def test_attention_reports_uncovered_rows(dtype, d, n, lens, front, back, bits, cuda_device):
    """Rows in front of the first sequence and behind the last one: flagged, left as they
    were, and the sequences between them computed as without them."""
    off = front + n * np.arange(4)
    T = int(off[-1]) + back
    out, wout, flag = _call(dtype, d, off, T, lens, cuda_device, n)
    assert flag == (5 if bits else 0, bits)
    assert bool((out[:front] == 7.0).all()) and bool((out[front + 3 * n:] == 7.0).all())
    assert not bool((out[front:front + 3 * n] == 7.0).any())


@pytest.mark.parametrize("dtype,d,n", KERNELS)
def test_attention_reports_rows_of_no_sequence(dtype, d, n, cuda_device):
    """Every sequence empty, or no sequence at all, with rows in the call."""
    out, _, flag = _call(dtype, d, np.zeros(4), n, [90, 0, 130], cuda_device, n)
    assert flag == (5, 16) and bool((out == 7.0).all())
    out, _, flag = _call(dtype, d, np.zeros(1), n, [], cuda_device, n)
    assert flag == (5, 16) and bool((out == 7.0).all())
    out, _, flag = _call(dtype, d, np.zeros(1), 0, [], cuda_device, n)
    assert flag == (0, 0)


@pytest.mark.parametrize("off,T,bits", [([0], 0, 0), ([0], 4, 16), ([4], 4, 1)])
def test_append_of_no_sequences(off, T, bits, cuda_device):
    pool, _, _, _ = make_pool(np.random.default_rng(5), [70], 2, 64)
    cache = to_cache(pool, cuda_device)
    k = torch.ones(T, 2, 64, device=cuda_device)
    none = torch.zeros(0, dtype=torch.int32, device=cuda_device)
    ws = ops.alloc_workspace(ops.hstu_cache_append_workspace_size(), cuda_device)
    ops.hstu_cache_append(k, k, cache, none.view(0, 1), none, none, dev(off, cuda_device, torch.int64),
                          torch.zeros(T, dtype=torch.int64, device=cuda_device), None, max_seq_len=4, workspace=ws)
    assert ops.hstu_check_device_flag(ws) == (5 if bits else 0, bits)
    assert_pool_equal(pool_of(cache), pool)


# ---- a wait that runs out -------------------------------------------------------------

WAITS = [(64, 1), (64, 30), (128, 8), (128, 64), (64, 65), (128, 200)]


def _withheld(monkeypatch):
    """From here on one CTA of an attention never gets its first keys."""
    def desc(*args, real=ops._cache_attn_desc):
        d = real(*args)
        d.debug_checks = ops.HSTU_DEBUG_CACHE_WAIT_TEST
        return d

    monkeypatch.setattr(ops, "_cache_attn_desc", desc)


def _wait_inputs(d, n, device):
    rng = np.random.default_rng(n)
    lens = [1100, 300, 700]
    pool, table, _, _ = make_pool(rng, lens, 2, d)
    cache = to_cache(pool, device)
    q = torch.as_tensor(rng.standard_normal((3 * n, 2, d)), dtype=torch.float32).to(torch.bfloat16).to(device)
    args = dict(max_seq_len=n, max_cache_len=max(lens), inv_n=1 / 64, pos_lo=-32, pos_hi=32)
    rp, rt = (0.1 * torch.randn(m, generator=torch.Generator().manual_seed(m)).to(device) for m in (65, 16))
    t = dev(table, device, torch.int32)
    inputs = (q, cache, t, dev(lens, device, torch.int32), None, dev(n * np.arange(4), device, torch.int64),
              1_700_000_000 + torch.arange(3 * n, device=device), None, rp, rt)
    size = ops.hstu_cache_attn_workspace_size(q, cache, t, rp, rt, weights=True, **args)
    return cache, inputs, args, size


@pytest.mark.parametrize("d,n", WAITS)
def test_bounded_waits_of_the_attention_run_out(d, n, cuda_device, monkeypatch):
    """The kernel ends and reports, and the next call on the same workspace is as any other."""
    cache, inputs, args, size = _wait_inputs(d, n, cuda_device)
    ws = ops.alloc_workspace(size, cuda_device)
    want_w = torch.zeros_like(cache.weights)
    want = ops.hstu_cache_attn_fwd(*inputs, weights_out=want_w, workspace=ws, **args)
    assert ops.hstu_check_device_flag(ws) == (0, 0)
    with monkeypatch.context() as m:
        _withheld(m)
        ops.hstu_cache_attn_fwd(*inputs, weights_out=torch.zeros_like(want_w), workspace=ws, **args)
        assert ops.hstu_check_device_flag(ws) == (5, 32)
    wout = torch.zeros_like(want_w)
    out = ops.hstu_cache_attn_fwd(*inputs, weights_out=wout, workspace=ws, **args)
    assert ops.hstu_check_device_flag(ws) == (0, 0)
    assert torch.equal(out, want) and torch.equal(wout, want_w)


@pytest.mark.parametrize("d,n", WAITS)
@pytest.mark.parametrize("same", [False, True])
def test_weights_survive_a_wait_that_runs_out(d, n, same, cuda_device, monkeypatch):
    """A flagged call adds nothing to the weights that later evictions go by."""
    cache, inputs, args, size = _wait_inputs(d, n, cuda_device)
    ws = ops.alloc_workspace(size, cuda_device)
    ws.fill_(255)  # NaN where nothing is written
    wout = cache.weights if same else torch.full_like(cache.weights, -5.0)
    before = wout.clone()
    _withheld(monkeypatch)
    ops.hstu_cache_attn_fwd(*inputs, weights_out=wout, workspace=ws, **args)
    assert ops.hstu_check_device_flag(ws) == (5, 32)
    assert torch.equal(wout, before)
