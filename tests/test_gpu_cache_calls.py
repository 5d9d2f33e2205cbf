"""Calls on the 8-bit cache that its other tests do not make: attentions that run at the
same time, and tables without a column."""

import numpy as np
import pytest
import torch

from cache_utils import dev, make_pool, to_cache
from hstu_sequential_transduction_b200 import ops

pytestmark = pytest.mark.gpu


def test_evict_with_tables_of_no_pages(cuda_device):
    """No room for a cached token: nothing moves; a length says otherwise and is flagged."""
    pool, _, _, _ = make_pool(np.random.default_rng(3), [70], 2, 64)
    cache = to_cache(pool, cuda_device)
    none = torch.zeros(2, 0, dtype=torch.int32, device=cuda_device)
    kw = dict(keep=4, max_cache_len=100)
    ws = ops.alloc_workspace(ops.hstu_cache_evict_workspace_size(cache, none, **kw), cuda_device)
    for lens, flag in (([0, 0], (0, 0)), ([0, 5], (5, 64))):
        table, new_lens, kept = ops.hstu_cache_evict(cache, none, dev(lens, cuda_device, torch.int32), none,
                                                     workspace=ws, **kw)
        assert ops.hstu_check_device_flag(ws) == flag
        assert new_lens.tolist() == lens and kept.tolist() == [[-1] * 4] * 2 and table.shape == (2, 0)


# ---- calls at the same time -----------------------------------------------------------

def _workspace(ws, size, device):
    assert ws is None or ws.numel() >= size
    return ops.alloc_workspace(size, device) if ws is None else ws


def _attention(dtype, d, n, lens, device, seed, ws=None):
    """A prepared attention: a call that repeats it, what it writes, and its workspace."""
    rng = np.random.default_rng(seed)
    pool, table, _, _ = make_pool(rng, lens, 2, d)
    cache = to_cache(pool, device)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T = n * len(lens)
    q = torch.as_tensor(rng.standard_normal((T, 2, d)), dtype=torch.float32).to(tdt).to(device)
    args = dict(max_seq_len=n, max_cache_len=max(lens), inv_n=1 / 500, pos_lo=-64, pos_hi=64)
    rp, rt = (0.1 * torch.randn(m, generator=torch.Generator().manual_seed(m)).to(device) for m in (129, 32))
    t = dev(table, device, torch.int32)
    inputs = (q, cache, t, dev(lens, device, torch.int32), None, dev(n * np.arange(len(lens) + 1), device, torch.int64),
              1_700_000_000 + 50 * torch.arange(T, device=device), None, rp, rt)
    out, wout = torch.empty_like(q), torch.zeros_like(cache.weights)
    ws = _workspace(ws, ops.hstu_cache_attn_workspace_size(q, cache, t, rp, rt, weights=True, **args), device)
    return lambda: ops.hstu_cache_attn_fwd(*inputs, out=out, weights_out=wout, workspace=ws, **args), (out, wout), ws


def _append(n, lens, device, seed, ws=None):
    """The same tokens appended again and again behind the same lengths: the same bytes."""
    rng = np.random.default_rng(seed)
    pool, table, _, _ = make_pool(rng, [x + n for x in lens], 2, 64)
    cache = to_cache(pool, device)
    T = n * len(lens)
    k, v = (torch.as_tensor(rng.standard_normal((T, 2, 64)), dtype=torch.float32).bfloat16().to(device) for _ in "kv")
    inputs = (k, v, cache, dev(table, device, torch.int32), dev(lens, device, torch.int32), None,
              dev(n * np.arange(len(lens) + 1), device, torch.int64), torch.arange(T, device=device), None)
    new = [torch.zeros(len(lens), dtype=torch.int32, device=device) for _ in range(2)]
    ws = _workspace(ws, ops.hstu_cache_append_workspace_size(), device)
    call = lambda: ops.hstu_cache_append(*inputs, max_seq_len=n, new_lens=new[0], new_pos=new[1], workspace=ws)  # noqa: E731
    return call, (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, *new), ws


def _evict(lens, keep, device, seed, ws=None):
    rng = np.random.default_rng(seed)
    cols = -(-max(lens) // 64)
    pool, table, free, _ = make_pool(rng, lens, 2, 64, extra=len(lens) * -(-keep // 64), cols=cols)
    cache = to_cache(pool, device)
    new_pages = np.full(table.shape, -1, np.int32)
    new_pages[:, :-(-keep // 64)] = free.reshape(len(lens), -1)
    t, n = dev(table, device, torch.int32), dev(new_pages, device, torch.int32)
    kw = dict(keep=keep, first=4, recent=32, max_cache_len=max(lens))
    ws = _workspace(ws, ops.hstu_cache_evict_workspace_size(cache, t, **kw), device)
    new = (torch.zeros_like(t), torch.zeros(len(lens), dtype=torch.int32, device=device),
           torch.zeros(len(lens), keep, dtype=torch.int32, device=device))
    ln = dev(lens, device, torch.int32)
    call = lambda: ops.hstu_cache_evict(cache, t, ln, n, new_table=new[0], new_lens=new[1], kept=new[2],  # noqa: E731
                                        workspace=ws, **kw)
    return call, (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, *new), ws


MAKE = {"cores": lambda *a: _attention("bf16", 128, 200, [4000, 900], *a),
        "cores64": lambda *a: _attention("bf16", 64, 70, [1500, 3000, 64], *a),
        "rows": lambda *a: _attention("bf16", 128, 9, [6000, 100, 2000], *a),
        "f32": lambda *a: _attention("f32", 32, 12, [900, 500], *a),
        "append": lambda *a: _append(300, [70, 0, 129], *a),
        "evict": lambda *a: _evict([6000, 5000], 1000, *a)}


@pytest.mark.parametrize("one,two", [("cores", "cores"), ("cores64", "rows"), ("cores", "append"), ("rows", "rows"),
                                     ("rows", "evict"), ("f32", "f32"), ("append", "evict")])
def test_calls_in_flight_together(one, two, cuda_device):
    """Everything prepared before, and both streams held until all calls are queued: what
    each call writes is, byte for byte, what it writes alone."""
    calls = [MAKE[one](cuda_device, 5), MAKE[two](cuda_device, 6)]
    want = []
    for call, outs, _ in calls:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    again = [MAKE[one](cuda_device, 5), MAKE[two](cuda_device, 6)]
    gate, streams = torch.cuda.Stream(), [torch.cuda.Stream() for _ in again]
    marks = [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in again]
    torch.cuda.synchronize()
    with torch.cuda.stream(gate):
        torch.cuda._sleep(20_000_000)  # ten milliseconds, in which the host queues the calls
        opened = gate.record_event()
    for st, mark in zip(streams, marks):
        st.wait_event(opened)
        mark[0].record(st)
    for _ in range(12):
        for st, (call, _, _) in zip(streams, again):
            with torch.cuda.stream(st):
                call()
    for st, mark in zip(streams, marks):
        mark[1].record(st)
    torch.cuda.synchronize()
    assert all(marks[i][0].elapsed_time(marks[1 - i][1]) > 0 for i in range(2))  # each began before the other ended
    for (_, outs, ws), w in zip(again, want):
        assert ops.hstu_check_device_flag(ws) == (0, 0)
        for a, b in zip(outs, w):
            assert torch.equal(a, b)


def test_captured_calls_share_a_workspace(cuda_device):
    """A graph of each kind of call, all on one workspace, replayed in turn and again."""
    kinds = list(MAKE)
    want = []
    for kind in kinds:
        call, outs, _ = MAKE[kind](cuda_device, 7)
        call()
        want.append([t.clone() for t in outs])
    ws = ops.alloc_workspace(1 << 26, cuda_device)
    ws.fill_(255)
    calls = [MAKE[kind](cuda_device, 7, ws) for kind in kinds]
    graphs = []
    torch.cuda.synchronize()
    for call, _, _ in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for order in (range(len(kinds)), reversed(range(len(kinds)))):
        for i in order:
            graphs[i].replay()
            assert ops.hstu_check_device_flag(ws) == (0, 0)
            for a, b in zip(calls[i][1], want[i]):
                assert torch.equal(a, b), kinds[i]
