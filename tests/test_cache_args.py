"""Refusals of the 8-bit cache's entry points: found on the host before anything is
launched, so they run without a GPU (addresses here are never read)."""

import ctypes
import re
import os

import pytest
import torch

from hstu_sequential_transduction_b200 import ops

A = 1 << 20  # a 256-byte aligned address
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _pool(**kw):
    f = dict(num_pages=4, num_heads=2, head_dim=64, max_pages=2, k_codes=A, v_codes=A, k_scale=A, v_scale=A,
             timestamps=A, positions=A, weights=A)
    f.update(kw)
    return ops.hstu_cache(*(f[n] for n, _ in ops.hstu_cache._fields_))


def _call(name, types_and_values):
    return getattr(ops.load_library(), name)(*types_and_values)


P, I, L, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


def _append(pool=None, **kw):
    f = dict(dtype=ops.HSTU_BF16, B=2, max_len=8, T=10, k=A, sk=128, v=A, sv=128, off=A, ts=A, nt=0, table=A, lens=A,
             pos=0, nl=2 * A, npos=0, ws=A, bytes=256)
    f.update(kw)
    return _call("hstu_cache_append", (ctypes.byref(_pool() if pool is None else pool), I(f["dtype"]), I(f["B"]),
                                       I(f["max_len"]), L(f["T"]), P(f["k"]), L(f["sk"]), P(f["v"]), L(f["sv"]),
                                       P(f["off"]), P(f["ts"]), P(f["nt"]), P(f["table"]), P(f["lens"]), P(f["pos"]),
                                       P(f["nl"]), P(f["npos"]), P(f["ws"]), Z(f["bytes"]), P(0)))


def _desc(**kw):
    f = dict(num_seqs=2, max_seq_len=8, total_tokens=10, num_heads=2, d_qk=64, d_v=64, dtype=ops.HSTU_BF16,
             inv_n=0.1, pos_lo=-4, pos_hi=4, num_time_buckets=8)
    f.update(kw)
    return ops.make_attn_desc(**f)


def _attn(pool=None, desc=None, **kw):
    f = dict(max_cache=128, q=A, sq=128, off=A, ts=A, nt=0, rp=A, rt=A, table=A, lens=A, pos=0, add=0, w=0, out=A,
             ws=A, bytes=1 << 30)
    f.update(kw)
    return _call("hstu_cache_attn_fwd", (ctypes.byref(desc or _desc()), ctypes.byref(pool or _pool()), I(f["max_cache"]),
                                         P(f["q"]), L(f["sq"]), P(f["off"]), P(f["ts"]), P(f["nt"]), P(f["rp"]),
                                         P(f["rt"]), P(f["table"]), P(f["lens"]), P(f["pos"]), P(f["add"]), P(f["w"]),
                                         P(f["out"]), P(f["ws"]), Z(f["bytes"]), P(0)))


def _evict(pool=None, **kw):
    f = dict(B=2, max_cache=128, keep=64, first=0, recent=0, table=A, lens=A, new=2 * A, nt=3 * A, nl=4 * A, kept=A,
             ws=A, bytes=1 << 30)
    f.update(kw)
    return _call("hstu_cache_evict", (ctypes.byref(pool or _pool()), I(f["B"]), I(f["max_cache"]), I(f["keep"]),
                                      I(f["first"]), I(f["recent"]), P(f["table"]), P(f["lens"]), P(f["new"]),
                                      P(f["nt"]), P(f["nl"]), P(f["kept"]), P(f["ws"]), Z(f["bytes"]), P(0)))


BAD_POOLS = [(dict(num_pages=-1), INVALID), (dict(num_heads=0), INVALID), (dict(max_pages=-1), INVALID),
             (dict(head_dim=48), UNSUPPORTED), (dict(max_pages=1 << 26), UNSUPPORTED), (dict(k_codes=0), INVALID),
             (dict(v_codes=A + 8), INVALID), (dict(k_scale=0), INVALID), (dict(positions=0), INVALID)]


@pytest.mark.parametrize("kw,status", BAD_POOLS)
@pytest.mark.parametrize("call", [_append, _attn, _evict])
def test_bad_pools(call, kw, status):
    assert call(pool=_pool(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), INVALID), (dict(B=-1), INVALID),
    (dict(T=-1), INVALID), (dict(max_len=-1), INVALID), (dict(k=0), INVALID), (dict(v=A + 2), INVALID),
    (dict(sk=120), INVALID), (dict(sv=132), INVALID), (dict(off=0), INVALID), (dict(ts=0), INVALID),
    (dict(table=0), INVALID), (dict(lens=0), INVALID), (dict(nl=0), INVALID), (dict(nl=A), INVALID),
    (dict(pos=2 * A), INVALID), (dict(npos=2 * A), INVALID), (dict(npos=A), INVALID),
    (dict(ws=0), WORKSPACE), (dict(ws=A + 16), WORKSPACE), (dict(bytes=255), WORKSPACE),
])
def test_append_refusals(kw, status):
    assert _append(**kw) == status


def test_append_types_and_widths():
    assert _append(dtype=ops.HSTU_F32, pool=_pool(head_dim=128), sk=256, sv=256) == UNSUPPORTED
    assert _append(pool=_pool(head_dim=32)) == UNSUPPORTED
    assert _append(B=1 << 30, T=1 << 40, max_len=1 << 30) == UNSUPPORTED  # more blocks than a launch has


@pytest.mark.parametrize("kw,status", [
    (dict(max_cache=-1), INVALID), (dict(max_cache=129), INVALID), (dict(q=0), INVALID), (dict(q=A + 2), INVALID),
    (dict(sq=120), INVALID), (dict(sq=130), INVALID), (dict(off=0), INVALID), (dict(ts=0), INVALID),
    (dict(rp=0), INVALID), (dict(rt=0), INVALID), (dict(table=0), INVALID), (dict(lens=0), INVALID),
    (dict(out=0), INVALID), (dict(add=A + 4), INVALID), (dict(ws=0), WORKSPACE), (dict(bytes=256), WORKSPACE),
])
def test_attention_refusals(kw, status):
    assert _attn(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(num_heads=3), INVALID), (dict(d_qk=128, d_v=128), INVALID), (dict(dtype=ops.HSTU_F32, d_qk=32, d_v=32), INVALID),
    (dict(d_v=128), UNSUPPORTED), (dict(local_window=4), UNSUPPORTED), (dict(global_window=4), UNSUPPORTED),
    (dict(inv_n=float("nan")), INVALID), (dict(num_time_buckets=0), INVALID),
])
def test_attention_descriptors(kw, status):
    assert _attn(desc=_desc(**kw)) == status
    n = ctypes.c_size_t(0)
    lib = ops.load_library()
    assert lib.hstu_cache_attn_workspace_size(ctypes.byref(_desc(**kw)), ctypes.byref(_pool()), I(128), I(1),
                                              ctypes.byref(n)) == status
    d = _desc()
    d.debug_checks = ops.HSTU_DEBUG_WAIT_TEST
    assert _attn(desc=d) == UNSUPPORTED
    assert _attn(desc=_desc(d_qk=128, d_v=128, fp8_qk=True), pool=_pool(head_dim=128), sq=256) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(max_cache=-1), INVALID), (dict(keep=0), INVALID), (dict(first=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(table=0), INVALID), (dict(lens=0), INVALID), (dict(new=0), INVALID),
    (dict(nt=0), INVALID), (dict(nl=0), INVALID), (dict(kept=0), INVALID), (dict(nl=A), INVALID),
    (dict(nt=A), INVALID), (dict(nt=2 * A), INVALID), (dict(ws=0), WORKSPACE), (dict(bytes=256), WORKSPACE),
])
def test_evict_refusals(kw, status):
    assert _evict(**kw) == status


def test_more_tokens_than_indices_reach():
    """Kernels round token indices up to whole rounds within 32 bits."""
    most = 2 ** 31 - 65536
    for cols, status in ((most // 64, WORKSPACE), (most // 64 + 1, UNSUPPORTED), (2 ** 25 - 1, UNSUPPORTED)):
        pool = _pool(max_pages=cols)
        assert _attn(pool=pool, max_cache=64 * min(cols, 2 ** 25 - 1), ws=0) == status
        assert _evict(pool=pool, ws=0) == status
    assert _evict(max_cache=most, ws=0) == WORKSPACE
    assert _evict(max_cache=most + 1, ws=0) == UNSUPPORTED


def test_evict_needs_weights():
    assert _evict(pool=_pool(weights=0)) == INVALID


def test_struct_matches_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "hstu.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} hstu_cache;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [re.sub(r".*[ *]", "", x.strip()) for part in body.split(";") for x in part.split(",") if x.strip()]
    assert names == [n for n, _ in ops.hstu_cache._fields_]
    assert re.search(r"#define HSTU_CACHE_PAGE (\d+)", text).group(1) == str(ops.HSTU_CACHE_PAGE)


def test_python_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        ops.HstuCache.empty(2, 1, 64, "cpu")
    with pytest.raises(ValueError, match="pages of 32"):
        ops.HstuCache(torch.zeros(1, 1, 32, 64), *([None] * 6))


def test_a_cache_keeps_its_tensors():
    cache = object.__new__(ops.HstuCache)
    cache._structs = {}
    with pytest.raises(AttributeError, match="keeps its tensors"):
        cache.weights = None


def test_wait_test_hook():
    """Taken by the bf16 attention over the cache and by no other call."""
    n = ctypes.c_size_t(0)
    d = _desc()
    d.debug_checks = ops.HSTU_DEBUG_CACHE_WAIT_TEST
    assert _attn(desc=d, ws=0) == WORKSPACE  # past the descriptor's checks
    f32 = _desc(dtype=ops.HSTU_F32)
    f32.debug_checks = ops.HSTU_DEBUG_CACHE_WAIT_TEST
    assert _attn(desc=f32) == UNSUPPORTED
    assert ops.load_library().hstu_attn_workspace_size(ctypes.byref(d), 0, ctypes.byref(n)) == INVALID
    d.debug_checks = 8
    assert _attn(desc=d) == INVALID
