"""The 8-bit key/value cache on the GPU against its oracle: append and eviction byte for
byte over the whole pool (slots behind a sequence's end and pages of no sequence
included), attention within derived bounds, and the three in a row with hstu_attn_fwd.

Bounds of the attention.  With u = 2^-24, a score s = q.k + bias of m = sum |q k| + |bias|
carries at most c_m m, P = SiLU(s) / N at most c_P P, and the tanh form c_h h, h = |s| / 2N:
  float32: c_m = 1.1 (d + 8) u (d products and sums; |SiLU'| <= 1.1), c_P = 2^-22 (expf to
           2 u, a division, two products);
  bf16:    c_m as float32; c_x = 1.1 2^-14 on x = max |q| sum |k|: two E4M3 parts hold a
           query element to 2^-10 of a scale whose rows' largest magnitude is above 224,
           that is 2^-17.8 of it, and a row's own largest is at least 2^-3 of that;
           c_P = 2^-8 (P to 16 bits); c_h = 2^-10 (tanh.approx: 2^-11 of tanh).
The errors of the cached tokens' terms are independent, so a sum of them stays within six
times the root of the sum of their squares; float32 sums add L u, the output's own rounding
half a step.  A token's weight sums n H terms of one sign: there the h term counts fully."""

import numpy as np
import pytest
import torch

import oracle
from cache_utils import PAGE, assert_pool_equal, dev, end_pos, make_pool, pages, pool_of, to_cache
from hstu_sequential_transduction_b200 import ops
from oracle import cache as oc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _bf16(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16)


def _values(t):
    return t.double().cpu().numpy()


# ---- append -------------------------------------------------------------------------

APPEND = [
    # cached, new, candidates
    ([0], [1], None),
    ([63], [1], None),
    ([64], [1], None),
    ([1, 0, 127, 64, 200], [64, 0, 1, 130, 63], None),
    ([5, 60], [70, 10], [3, 10]),
    ([0, 0, 0], [257, 0, 64], [0, 0, 64]),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("dtype,d,heads", [("bf16", 128, 2), ("bf16", 64, 3), ("f32", 32, 1), ("f32", 64, 2)])
@pytest.mark.parametrize("strided", [False, True])
def test_append(case, dtype, d, heads, strided, cuda_device):
    lens, new, nt = APPEND[case]
    rng = np.random.default_rng(100 + case)
    cols = pages(max(a + b for a, b in zip(lens, new))) + 1
    pool, table, free, _ = make_pool(rng, lens, heads, d, extra=sum(map(pages, new)) + len(new), cols=cols)
    at = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        lo, hi = pages(L), pages(L + n - (nt[b] if nt else 0))
        table[b, lo:hi] = free[at:at + hi - lo]
        at += hi - lo
    off = np.concatenate([[0], np.cumsum(new)])
    T = int(off[-1])
    kv = rng.standard_normal((T, 2, heads, d)) * np.exp2(rng.integers(-12, 12, (T, 1, 1, 1)))
    kv[rng.random(T) < 0.1] = 0.0
    kv = _bf16(kv) if dtype == "bf16" else torch.as_tensor(kv, dtype=torch.float32)
    k, v = kv[:, 0], kv[:, 1]
    ts = rng.integers(0, 2 ** 40, T)
    pos = np.array([2 * x for x in lens], np.int32)
    lens = np.array(lens, np.int32)
    nt = None if nt is None else np.array(nt, np.int32)
    want = {n: a.copy() for n, a in pool.items()}
    want_lens, want_pos = oc.append(want, _values(k), _values(v), table, lens, pos, off, ts, nt)
    cache = to_cache(pool, cuda_device)
    kd, vd = (x.to(cuda_device) if strided else x.contiguous().to(cuda_device) for x in (k, v))
    if strided:
        g = kv.to(cuda_device)
        kd, vd = g[:, 0], g[:, 1]
    ws = ops.alloc_workspace(ops.hstu_cache_append_workspace_size(), cuda_device)
    got = ops.hstu_cache_append(kd, vd, cache, dev(table, cuda_device), dev(lens, cuda_device), dev(pos, cuda_device),
                                dev(off, cuda_device), dev(ts, cuda_device), dev(nt, cuda_device),
                                max_seq_len=max(new), workspace=ws)
    assert ops.hstu_check_device_flag(ws) == (0, 0)
    np.testing.assert_array_equal(got[0].cpu().numpy(), want_lens)
    np.testing.assert_array_equal(got[1].cpu().numpy(), want_pos)
    assert_pool_equal(pool_of(cache), want)


def _append(cache, k, v, table, lens, off, device, **kw):
    T = k.shape[0]
    ws = ops.alloc_workspace(ops.hstu_cache_append_workspace_size(), device)
    out = ops.hstu_cache_append(k, v, cache, dev(table, device, torch.int32), dev(lens, device, torch.int32), None,
                                dev(off, device, torch.int64), torch.arange(T, device=device), None,
                                max_seq_len=max(1, T), workspace=ws, **kw)
    return out, ops.hstu_check_device_flag(ws)


def test_append_extremes(cuda_device):
    """The largest and smallest magnitudes, and blocks with a value that is not finite."""
    x = torch.zeros(4, 1, 64)
    x[0, 0, :4] = torch.tensor([3.0e38, -1.0, 448.0, 1e-38])
    x[1, 0, :3] = torch.tensor([1e-40, -1.4e-45, 0.0])
    x[2, 0, 5], x[3, 0, 6] = float("inf"), float("nan")
    for row in range(4):
        cache = ops.HstuCache.empty(1, 1, 64, cuda_device)
        k = x[row:row + 1].to(cuda_device)
        _, flag = _append(cache, k, torch.ones_like(k), [[0]], [0], [0, 1], cuda_device)
        assert flag == (0, 0)
        scale = float(cache.k_scale[0, 0])
        if row >= 2:
            assert np.isnan(scale)
        else:
            assert scale == oc.scale_of(float(x[row].abs().max()))
            np.testing.assert_array_equal(cache.k_codes[0, 0, 0].cpu().numpy(),
                                          oc.encode(x[row, 0].double().numpy() / scale))
        assert float(cache.v_scale[0, 0]) == 2.0 ** -8


def test_append_drops_what_does_not_fit(cuda_device):
    """Bad lengths, targets and pages: flagged, dropped, nothing else touched."""
    rng = np.random.default_rng(8)
    pool, table, free, _ = make_pool(rng, [60, 10, 10], 2, 64, extra=3, cols=2)
    table[0, 1], table[1, 1] = free[0], 10 ** 6
    k = _bf16(rng.standard_normal((90, 2, 64))).to(cuda_device)
    off = np.array([0, 80, 85, 90])
    cache = to_cache(pool, cuda_device)
    (nl, npos), flag = _append(cache, k, k, table, [60, 10, 10], off, cuda_device)  # 140 tokens, room for 128
    assert flag == (5, 64) and nl.tolist() == [60, 15, 15] and npos.tolist() == [60, 15, 15]
    got = pool_of(cache)
    for n in ("k_codes", "v_codes", "k_scale", "v_scale", "timestamps"):
        np.testing.assert_array_equal(got[n][table[0, 0]], pool[n][table[0, 0]])
    _, flag = _append(cache, k[:60], k[:60], table, [0, 64, 0], np.array([0, 0, 60, 60]), cuda_device)
    assert flag == (5, 128)  # the page 10^6
    (nl, _), flag = _append(cache, k, k, table, [-1, 10, 300], off, cuda_device)
    assert flag == (5, 64) and nl.tolist() == [-1, 15, 300]


# ---- attention ----------------------------------------------------------------------

ATTN = [
    # cached, new, candidates
    ([1], [1], None),
    ([64], [1], None),
    ([130], [1], None),
    ([0, 7, 65, 300], [1, 1, 1, 1], None),
    ([0, 200, 63, 1000], [3, 0, 17, 5], None),
    ([500, 129], [12, 70], [12, 64]),
    ([2000], [130], [100]),
    ([90, 0, 400], [16, 33, 300], [0, 33, 299]),
]
TYPES = [("bf16", 128, 2), ("bf16", 64, 3), ("bf16", 128, 1), ("f32", 32, 2), ("f32", 64, 1)]


def _attn_inputs(case, dtype, d, heads, seed, per_head=False, std=1.0, pos=100, nb=40):
    lens, new, nt = case
    rng = np.random.default_rng(seed)
    pool, table, _, _ = make_pool(rng, lens, heads, d, gaps=True, extra=2, std=std)
    lens = np.array(lens, np.int32)
    T = sum(new)
    q = rng.standard_normal((T, heads, d)) * np.exp2(rng.integers(-3, 2, (T, 1, 1)))
    add = rng.standard_normal((T, heads, d)) * 0.1
    q, add = (_bf16(x) if dtype == "bf16" else torch.as_tensor(x, dtype=torch.float32) for x in (q, add))
    lead = (heads,) if per_head else ()
    f = dict(dtype=torch.float32)
    return dict(pool=pool, table=table, lens=lens, seq_pos=end_pos(pool, table, lens),
                off=np.concatenate([[0], np.cumsum(new)]), ts=1_700_000_000 + rng.integers(0, 10 ** 6, T),
                nt=None if nt is None else np.array(nt, np.int32), q=q, add=add,
                rp=torch.as_tensor(0.3 * rng.standard_normal(lead + (2 * pos + 1,)), **f),
                rt=torch.as_tensor(0.3 * rng.standard_normal(lead + (nb,)), **f), pos=pos, max_new=max(new),
                max_len=int(max(lens)), inv_n=1.0 / 500)


def _run_attn(x, device, own=False, add=True, weights="other", q=None, ws=None, **kw):
    cache = to_cache(x["pool"], device, weights=weights != "none")
    g = {n: dev(x[n], device) for n in ("table", "lens", "seq_pos", "off", "ts", "nt", "rp", "rt")}
    q = x["q"].to(device) if q is None else q
    wout = {"other": lambda: torch.full_like(cache.weights, -5.0), "same": lambda: cache.weights, "off": lambda: None,
            "none": lambda: torch.full(cache.timestamps.shape, -5.0, device=device)}[weights]()
    args = dict(max_seq_len=x["max_new"], max_cache_len=x["max_len"], inv_n=x["inv_n"], pos_lo=-x["pos"],
                pos_hi=x["pos"], cand_own_index=own)
    if ws is None:
        ws = ops.alloc_workspace(ops.hstu_cache_attn_workspace_size(q, cache, g["table"], g["rp"], g["rt"],
                                                                    weights=wout is not None, **args), device)
        ws.fill_(255)  # NaN where nothing was written
    out = ops.hstu_cache_attn_fwd(q, cache, g["table"], g["lens"], g["seq_pos"], g["off"], g["ts"], g["nt"], g["rp"],
                                  g["rt"], addend=x["add"].to(device) if add else None, weights_out=wout,
                                  workspace=ws, **args, **kw)
    return out, wout, ws, cache


def _want_attn(x, own=False, add=True):
    return oc.attn(x["pool"], _values(x["q"]), x["table"], x["lens"], x["seq_pos"], x["off"], x["ts"], x["nt"],
                   x["rp"].numpy(), x["rt"].numpy(), x["inv_n"], -x["pos"], x["pos"], own=own,
                   addend=_values(x["add"]) if add else None)


def _check_attn(x, out, want, terms, wout=None, want_w=None, base=None):
    bf16 = x["q"].dtype == torch.bfloat16
    H, d = x["q"].shape[1:]
    c_m, c_x = 1.1 * (d + 8) * U, 1.1 * 2.0 ** -14 if bf16 else 0.0
    c_P, c_h = (2.0 ** -8, 2.0 ** -10) if bf16 else (2.0 ** -22, 0.0)
    L = x["max_len"]
    t = terms["out"]
    half = torch.finfo(x["q"].dtype).eps / 2
    tol = 6 * ((c_P + L * U) * t["P"] + c_h * t["h"] + c_m * t["m"] + c_x * t["x"]) * (1 + half) + half * np.abs(want) + 1e-30
    err = np.abs(_values(out) - want)
    assert np.all(err <= tol), f"output off by {np.max(err / tol):.2f} of its bound"
    if wout is None:
        return
    got = wout.double().cpu().numpy()
    mine = np.zeros(want_w.shape, bool)  # the call's cached tokens
    for b, n in enumerate(x["lens"]):
        j = np.arange(n)
        mine[x["table"][b][j // PAGE], j % PAGE] = True
    w = terms["w"]
    n = x["max_new"] * H
    c_Pw = 2.0 ** -8 if bf16 else 2.0 ** -22
    tol = 6 * (c_Pw + n * U) * w["P"] + np.sqrt(n) * c_h * w["h"] + 6 * (c_m * w["m"] + c_x * w["x"]) + 2 * U * np.abs(want_w)
    err = np.abs(got - want_w)[mine]
    assert np.all(err <= tol[mine] + 1e-30), f"weights off by {np.max(err / (tol[mine] + 1e-30)):.2f} of their bound"
    np.testing.assert_array_equal(got[~mine], base[~mine])


@pytest.mark.parametrize("case", range(len(ATTN)))
@pytest.mark.parametrize("dtype,d,heads", TYPES)
def test_attention(case, dtype, d, heads, cuda_device):
    x = _attn_inputs(ATTN[case], dtype, d, heads, 200 + case)
    out, wout, ws, _ = _run_attn(x, cuda_device)
    assert ops.hstu_check_device_flag(ws) == (0, 0)
    want, want_w, terms = _want_attn(x)
    _check_attn(x, out, want, terms, wout, want_w, np.full(want_w.shape, -5.0))


@pytest.mark.parametrize("case", [3, 5, 7])
@pytest.mark.parametrize("dtype,d,heads", [("bf16", 128, 4), ("bf16", 64, 2), ("f32", 32, 2)])
@pytest.mark.parametrize("own,per_head,add,weights", [(True, False, False, "off"), (False, True, True, "same"),
                                                      (True, True, True, "none"), (False, False, False, "off")])
def test_attention_options(case, dtype, d, heads, own, per_head, add, weights, cuda_device):
    x = _attn_inputs(ATTN[case], dtype, d, heads, 300 + case, per_head=per_head)
    out, wout, ws, cache = _run_attn(x, cuda_device, own=own, add=add, weights=weights)
    assert ops.hstu_check_device_flag(ws) == (0, 0)
    if weights == "none":
        x["pool"]["weights"][:] = 0.0
    want, want_w, terms = _want_attn(x, own=own, add=add)
    base = {"off": None, "none": np.full(want_w.shape, -5.0), "same": x["pool"]["weights"].astype(np.float64)}[weights]
    _check_attn(x, out, want, terms, wout, want_w, base)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_of_strided_queries_into_the_addend(dtype, d, new, cuda_device):
    """q as a block of a wider projection, the output written over the addend."""
    x = _attn_inputs(([300, 64], [new, new + 3], None), dtype, d, 2, 17)
    T = x["q"].shape[0]
    wide = torch.randn(T, 4, 2, d, device=cuda_device).to(x["q"].dtype)
    wide[:, 2] = x["q"].to(cuda_device)
    buf = x["add"].to(cuda_device)
    x2 = dict(x, add=buf)
    cache = to_cache(x["pool"], cuda_device)
    g = {n: dev(x[n], cuda_device) for n in ("table", "lens", "seq_pos", "off", "ts", "nt", "rp", "rt")}
    out = ops.hstu_cache_attn_fwd(wide[:, 2], cache, g["table"], g["lens"], g["seq_pos"], g["off"], g["ts"], None,
                                  g["rp"], g["rt"], addend=buf, out=buf, max_seq_len=x["max_new"],
                                  max_cache_len=x["max_len"], inv_n=x["inv_n"], pos_lo=-x["pos"], pos_hi=x["pos"])
    assert out.data_ptr() == x2["add"].data_ptr()
    want, _, terms = _want_attn(x)
    _check_attn(x, out, want, terms)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("new", [1, 150])
def test_attention_scales_far_apart(dtype, d, new, cuda_device):
    """Pages whose scales differ by up to 2^40, one of them all zero, queries whose rows do."""
    x = _attn_inputs(([700], [new], None), dtype, d, 2, 23)
    rng = np.random.default_rng(5)
    for n in ("k_scale", "v_scale"):
        x["pool"][n] *= np.exp2(rng.integers(-20, 1 if n == "k_scale" else 20, x["pool"][n].shape)).astype(np.float32)
        x["pool"][n][x["table"][0, 3]] = 0.0
    x["q"] = (x["q"].double() * torch.as_tensor(np.exp2(rng.integers(-30, 2, (new, 1, 1))))).to(x["q"].dtype)
    out, wout, ws, _ = _run_attn(x, cuda_device)
    want, want_w, terms = _want_attn(x)
    _check_attn(x, out, want, terms, wout, want_w, np.full(want_w.shape, -5.0))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("new", [1, 140])
def test_attention_of_unsorted_and_far_stamps(dtype, d, new, cuda_device):
    x = _attn_inputs(([333], [new], None), dtype, d, 2, 29, nb=50)
    rng = np.random.default_rng(6)
    x["pool"]["timestamps"][:] = rng.integers(-2 ** 45, 2 ** 45, x["pool"]["timestamps"].shape)
    x["pool"]["positions"][:] = rng.integers(0, 2 ** 20, x["pool"]["positions"].shape)
    x["ts"] = rng.integers(-2 ** 45, 2 ** 45, new)
    out, wout, ws, _ = _run_attn(x, cuda_device)
    want, want_w, terms = _want_attn(x)
    _check_attn(x, out, want, terms, wout, want_w, np.full(want_w.shape, -5.0))


@pytest.mark.parametrize("new", [1, 100])
def test_attention_drops_and_flags(new, cuda_device):
    """A sequence with a bad length is left as it was; a bad page's tokens are skipped."""
    x = _attn_inputs(([100, 200, 150], [new, new, new], None), "bf16", 64, 2, 31)
    bad = dict(x, lens=np.array([100, 5000, 150], np.int32), max_len=200)
    fill = torch.full(x["q"].shape, 7.0, dtype=torch.bfloat16, device=cuda_device)
    out, wout, ws, _ = _run_attn(bad, cuda_device, out=fill.clone())
    assert ops.hstu_check_device_flag(ws) == (5, 64)
    want, _, terms = _want_attn(x)
    rows = np.r_[0:new, 2 * new:3 * new]
    sub = {n: a[rows] for n, a in terms["out"].items()}
    _check_attn(x, out[torch.as_tensor(rows, device=cuda_device)], want[rows], {"out": sub})
    assert torch.equal(out[new:2 * new], fill[new:2 * new])
    bad = dict(x, table=x["table"].copy())
    bad["table"][1, 1] = 10 ** 6
    out, wout, ws, _ = _run_attn(bad, cuda_device)
    assert ops.hstu_check_device_flag(ws) == (5, 128)
    y = dict(x, pool={n: a.copy() for n, a in x["pool"].items()})
    y["pool"]["v_scale"][x["table"][1, 1]] = 0.0  # without the page: as if its values were zero
    want, _, terms = _want_attn(y)
    _check_attn(x, out, want, terms)


@pytest.mark.parametrize("new", [3, 66])
def test_attention_of_more_sequences_than_threads(new, cuda_device):
    """A thousand sequences, some without a cache, some without new tokens: several units a CTA."""
    rng = np.random.default_rng(3)
    n = [int(a) for a in rng.integers(0, 3, 1000) * new // 2]
    x = _attn_inputs(([int(a) for a in rng.integers(0, 70, 1000)], n, None), "bf16", 64, 1, 47)
    out, wout, ws, _ = _run_attn(x, cuda_device)
    assert ops.hstu_check_device_flag(ws) == (0, 0)
    want, want_w, terms = _want_attn(x)
    _check_attn(x, out, want, terms, wout, want_w, np.full(want_w.shape, -5.0))


@pytest.mark.parametrize("cached,new", [(5000, 300), (900, 129), (130, 500)])
@pytest.mark.parametrize("same_stamp", [True, False])
def test_attention_of_candidates(cached, new, same_stamp, cuda_device):
    """Ranking: all rows candidates, of one stamp (one bias a key) or of several, with a
    ragged last tile; rows of very different sizes in one of the sequences."""
    x = _attn_inputs(([cached, 0, cached // 2 + 1], [new, new - 1, new], [new, new - 1, new]), "bf16", 128, 2, 53)
    if same_stamp:
        x["ts"][:] = 1_700_000_000 + 10 ** 6
        x["q"][:new] = _bf16(np.random.default_rng(1).standard_normal((new, 2, 128)))
    out, wout, ws, _ = _run_attn(x, cuda_device)
    assert ops.hstu_check_device_flag(ws) == (0, 0)
    want, want_w, terms = _want_attn(x)
    _check_attn(x, out, want, terms, wout, want_w, np.full(want_w.shape, -5.0))


@pytest.mark.parametrize("new,max_cache", [(0, 100), (1, 0), (200, 0), (200, 100)])
def test_attention_of_nothing(new, max_cache, cuda_device):
    """No new tokens (weights are passed on), an empty cache (the addend or zeros)."""
    lens = [min(100, max_cache), 0]
    x = _attn_inputs((lens, [new, new], None), "bf16", 64, 2, 59)
    x["max_len"], x["max_new"] = max_cache, max(new, 1)
    if max_cache == 0:
        x["table"] = np.zeros((2, 1), np.int32)
    for add in (True, False):
        out, wout, ws, _ = _run_attn(x, cuda_device, add=add)
        assert ops.hstu_check_device_flag(ws) == (0, 0)
        want, want_w, terms = _want_attn(x, add=add)
        _check_attn(x, out, want, terms, wout, want_w, np.full(want_w.shape, -5.0))


def test_attention_of_a_page_twice(cuda_device):
    """Sequences may read the same pages where no weights are taken."""
    for new in (1, 100):
        x = _attn_inputs(([200, 200], [new, new], None), "bf16", 64, 2, 61)
        x["table"][1] = x["table"][0]
        out, _, ws, _ = _run_attn(x, cuda_device, weights="off")
        assert ops.hstu_check_device_flag(ws) == (0, 0)
        want, _, terms = _want_attn(x)
        _check_attn(x, out, want, terms)


def test_calls_on_two_streams_at_once(cuda_device):
    """Two attentions with a workspace each, in flight together, and one workspace reused
    for calls of other kinds in turn."""
    xs = [_attn_inputs(([1500, 700], [n, n], None), "bf16", 128, 2, 67 + n) for n in (150, 4)]
    alone = [_run_attn(x, cuda_device)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = []
    for _ in range(5):
        for x, st in zip(xs, streams):
            with torch.cuda.stream(st):
                outs.append(_run_attn(x, cuda_device)[0])
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, alone[i % 2])
    ws = ops.alloc_workspace(1 << 26, cuda_device)
    ws.fill_(255)
    for _ in range(2):
        for x, want in zip(xs, alone):
            assert torch.equal(_run_attn(x, cuda_device, ws=ws)[0], want)


def test_attention_repeats_itself(cuda_device):
    """The same bytes whatever ran before, on another stream and from a captured graph."""
    for new in (1, 9, 200):
        x = _attn_inputs(([900, 300], [new, new], None), "bf16", 128, 2, 37)
        out, wout, ws, _ = _run_attn(x, cuda_device)
        out2, wout2, _, _ = _run_attn(x, cuda_device)
        assert torch.equal(out, out2) and torch.equal(wout, wout2)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out3, wout3, _, _ = _run_attn(x, cuda_device)
        side.synchronize()
        assert torch.equal(out, out3) and torch.equal(wout, wout3)


# ---- eviction -----------------------------------------------------------------------

EVICT = [
    # cached, keep, first, recent
    ([2], 1, 0, 0),
    ([65], 64, 0, 0),
    ([130, 40, 0, 64], 63, 4, 16),
    ([1000, 70, 500], 100, 7, 30),
    ([300], 10, 20, 20),
    ([300, 301], 100, 64, 0),
    ([4000], 1024, 4, 256),
    ([5000, 4097], 4096, 64, 1000),
    ([40000, 16385], 300, 3, 17),
]


def _evict_inputs(case, heads, d, seed):
    lens, keep, first, recent = EVICT[case]
    rng = np.random.default_rng(seed)
    cols = max(pages(max(lens)), pages(keep))
    pool, table, free, _ = make_pool(rng, lens, heads, d, extra=pages(keep) * len(lens), cols=cols, gaps=True)
    new_pages = np.full(table.shape, -9, np.int32)
    for b in range(len(lens)):
        new_pages[b, :pages(keep)] = free[b * pages(keep):(b + 1) * pages(keep)]
    return pool, table, np.array(lens, np.int32), new_pages, keep, first, recent


def _run_evict(pool, table, lens, new_pages, keep, first, recent, device, ws=None):
    cache = to_cache(pool, device)
    kw = dict(keep=keep, first=first, recent=recent, max_cache_len=int(max(lens)))
    t = dev(table, device)
    if ws is None:
        ws = ops.alloc_workspace(ops.hstu_cache_evict_workspace_size(cache, t, **kw), device)
    got = ops.hstu_cache_evict(cache, t, dev(lens, device), dev(new_pages, device), workspace=ws, **kw)
    return cache, got, ops.hstu_check_device_flag(ws)


def _check_evict(x, cuda_device):
    pool, table, lens, new_pages, keep, first, recent = x
    want = {n: a.copy() for n, a in pool.items()}
    w_table, w_lens, w_kept = oc.evict(want, table, lens, new_pages, keep, first, recent)
    cache, (table2, lens2, kept), flag = _run_evict(*x, cuda_device)
    assert flag == (0, 0)
    np.testing.assert_array_equal(kept.cpu().numpy(), w_kept)
    np.testing.assert_array_equal(lens2.cpu().numpy(), w_lens)
    np.testing.assert_array_equal(table2.cpu().numpy(), w_table)
    assert_pool_equal(pool_of(cache), want)


@pytest.mark.parametrize("case", range(len(EVICT)))
@pytest.mark.parametrize("heads,d", [(1, 32), (3, 64), (2, 128)])
def test_evict(case, heads, d, cuda_device):
    _check_evict(_evict_inputs(case, heads, d, 400 + case), cuda_device)


@pytest.mark.parametrize("values", [[0.0], [1.0, 2.0], [0.0, -0.0], [float("nan"), 1.0], [float("nan")],
                                    [float("inf"), float("-inf"), float("nan"), 0.0, 1e-45, -1.0]])
def test_evict_ties_and_odd_weights(values, cuda_device):
    x = _evict_inputs(3, 1, 32, 77)
    rng = np.random.default_rng(7)
    x[0]["weights"][:] = rng.choice(np.array(values, np.float32), x[0]["weights"].shape)
    _check_evict(x, cuda_device)


def test_evict_scales_far_apart(cuda_device):
    x = _evict_inputs(3, 2, 64, 78)
    rng = np.random.default_rng(8)
    for n in ("k_scale", "v_scale"):
        x[0][n][:] = np.exp2(rng.integers(-60, 60, x[0][n].shape))
        x[0][n][::3] = 0.0
    _check_evict(x, cuda_device)


def test_evict_drops_and_flags(cuda_device):
    pool, table, lens, new_pages, keep, first, recent = _evict_inputs(3, 2, 64, 79)
    bad = lens.copy()
    bad[1] = 10 ** 6
    cache = to_cache(pool, cuda_device)
    t = dev(table, cuda_device)
    kw = dict(keep=keep, first=first, recent=recent, max_cache_len=1000)
    ws = ops.alloc_workspace(ops.hstu_cache_evict_workspace_size(cache, t, **kw), cuda_device)
    table2, lens2, kept = ops.hstu_cache_evict(cache, t, dev(bad, cuda_device), dev(new_pages, cuda_device),
                                               workspace=ws, **kw)
    assert ops.hstu_check_device_flag(ws) == (5, 64)
    assert lens2.tolist() == [100, 10 ** 6, 100] and kept[1].tolist() == [-1] * keep
    np.testing.assert_array_equal(table2[1].cpu().numpy(), table[1])
    wrong = new_pages.copy()
    wrong[0, 0] = -1
    _, _, flag = _run_evict(pool, table, lens, wrong, keep, first, recent, cuda_device)
    assert flag == (5, 128)
    wrong = table.copy()
    wrong[0, 2] = 10 ** 6
    _, _, flag = _run_evict(pool, wrong, lens, new_pages, keep, first, recent, cuda_device)
    assert flag == (5, 128)


# ---- the three together ---------------------------------------------------------------

@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
def test_serving_run(dtype, d, cuda_device):
    """History appended in two parts, candidates ranked (attention among the new tokens by
    hstu_attn_fwd, over the history by the cache), the cache cut, candidates ranked again;
    each step against the oracle on what the GPU's pool holds."""
    rng = np.random.default_rng(41)
    H, hist, cand, first = 2, [150, 64, 9], [33, 20, 1], [70, 64, 0]
    cut, keep = [h - f for h, f in zip(hist, first)], 100
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rows = lambda n: torch.as_tensor(rng.standard_normal((n, H, d)), dtype=torch.float32).to(tdt)  # noqa: E731
    cache = ops.HstuCache.empty(12, H, d, cuda_device)
    table = np.array([[3, 7, 1], [0, 11, 11], [5, 11, 11]], np.int32)
    lens = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    pos = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    rp, rt = (0.2 * torch.randn(n, generator=torch.Generator().manual_seed(1)) for n in (201, 32))
    kw = dict(inv_n=1 / 200, pos_lo=-100, pos_hi=100)
    base = 1_700_000_000
    for part, n in ((0, first), (1, cut)):
        off = np.concatenate([[0], np.cumsum(n)])
        ts = np.concatenate([base + 60 * (np.arange(m) + (f if part else 0)) for m, f in zip(n, first)])
        lens, pos = ops.hstu_cache_append(rows(sum(n)).to(cuda_device), rows(sum(n)).to(cuda_device), cache,
                                          dev(table, cuda_device), lens, pos, dev(off, cuda_device),
                                          dev(ts.astype(np.int64), cuda_device), None, max_seq_len=max(n))
    assert lens.tolist() == hist and pos.tolist() == hist
    off = np.concatenate([[0], np.cumsum(cand)])
    T = int(off[-1])
    q, k, v = rows(T), rows(T), rows(T)
    ts = np.concatenate([np.full(c, base + 60 * h) for c, h in zip(cand, hist)]).astype(np.int64)
    nt = np.array(cand, np.int32)
    g = [dev(a, cuda_device) for a in (off, ts, nt)]
    qkv = [a.to(cuda_device) for a in (q, k, v)]

    def rank(tab, lens):
        tab_h, lens_h = tab.cpu().numpy(), lens.cpu().numpy()
        own = ops.hstu_attn_fwd(*qkv, *g, rp.to(cuda_device), rt.to(cuda_device), max_seq_len=max(cand), **kw)
        before = pool_of(cache)
        out = ops.hstu_cache_attn_fwd(qkv[0], cache, tab, lens, pos, *g, rp.to(cuda_device), rt.to(cuda_device),
                                      addend=own, weights_out=cache.weights, max_seq_len=max(cand),
                                      max_cache_len=int(lens.max()), **kw)
        want, want_w, terms = oc.attn(before, _values(q), tab_h, lens_h, pos.cpu().numpy(), off, ts, nt, rp.numpy(),
                                      rt.numpy(), kw["inv_n"], -100, 100, addend=_values(own))
        x = dict(q=q, max_len=int(lens_h.max()), max_new=max(cand), lens=lens_h, table=tab_h)
        _check_attn(x, out, want, terms, cache.weights, want_w, before["weights"].astype(np.float64))
        # and the whole against attention over history and candidates at once, on the cached values
        for b in range(3):
            L, n = int(lens_h[b]), cand[b]
            old = {m: np.stack([oc.tokens(before, m, tab_h[b], L, h) for h in range(H)], 1) for m in "kv"}
            sl = slice(off[b], off[b + 1])
            full = [np.concatenate([old[m], _values(a)[sl]]) for m, a in (("k", k), ("v", v))]
            pj = np.concatenate([before["positions"][tab_h[b][np.arange(L) // PAGE], np.arange(L) % PAGE],
                                 np.full(n, int(pos[b]))])
            tj = np.concatenate([before["timestamps"][tab_h[b][np.arange(L) // PAGE], np.arange(L) % PAGE], ts[sl]])
            for i in (0, n - 1):
                row = off[b] + i
                see = np.r_[0:L, L + i]
                dp = np.clip(int(pos[b]) - pj[see], -100, 100) + 100
                bk = np.minimum(np.floor(np.log2(1.0 + np.maximum(ts[row] - tj[see], 0))).astype(int), 31)
                for h in range(H):
                    s = full[0][see, h] @ _values(q)[row, h] + rp.numpy()[dp] + rt.numpy()[bk]
                    o = (s / (1 + np.exp(-s)) / 200) @ full[1][see, h]
                    bound = (2e-2 if dtype == "bf16" else 1e-4) * max(1e-3, np.abs(o).max())
                    assert np.max(np.abs(_values(out)[row, h] - o)) <= bound
        return out

    t = dev(table, cuda_device)
    rank(t, lens)
    new_pages = np.array([[2, 4, 6], [8, 9, 10], [8, 9, 10]], np.int32)
    before = pool_of(cache)
    want = {n: a.copy() for n, a in before.items()}
    w_table, w_lens, w_kept = oc.evict(want, table, np.array(hist, np.int32), new_pages, keep, 4, 32)
    t2, lens2, kept = ops.hstu_cache_evict(cache, t, lens, dev(new_pages, cuda_device), keep=keep, first=4, recent=32,
                                           max_cache_len=150)
    np.testing.assert_array_equal(kept.cpu().numpy(), w_kept)
    assert_pool_equal(pool_of(cache), want)
    rank(t2, lens2)


def test_captured_serving_step(cuda_device):
    """Append and attention of one token captured into a graph: each replay moves on by one
    token, as the same calls one by one do."""
    rng = np.random.default_rng(43)
    H, d, steps = 2, 64, 70
    B = 3
    table = dev(np.array([[0, 1], [2, 3], [4, 5]]), cuda_device, torch.int32)
    off = torch.arange(B + 1, device=cuda_device)
    rp, rt = torch.randn(65, device=cuda_device) * 0.1, torch.randn(16, device=cuda_device) * 0.1
    toks = [torch.as_tensor(rng.standard_normal((3, B, H, d)), dtype=torch.float32).to(torch.bfloat16).to(cuda_device)
            for _ in range(steps)]

    def fresh():
        z = lambda: torch.zeros(B, dtype=torch.int32, device=cuda_device)  # noqa: E731
        st = dict(cache=ops.HstuCache.empty(6, H, d, cuda_device), lens=z(), pos=z(), nl=z(), np=z(),
                  qkv=torch.zeros(3, B, H, d, dtype=torch.bfloat16, device=cuda_device),
                  ts=torch.full((B,), 1000, device=cuda_device), out=torch.zeros(B, H, d, dtype=torch.bfloat16,
                                                                                  device=cuda_device))
        kw = dict(max_seq_len=1, max_cache_len=128, inv_n=1 / 64, pos_lo=-32, pos_hi=32)
        st["ws"] = [ops.alloc_workspace(256, cuda_device), ops.alloc_workspace(ops.hstu_cache_attn_workspace_size(
            st["qkv"][0], st["cache"], table, rp, rt, weights=True, **kw), cuda_device)]
        st["kw"] = kw
        return st

    def step(st):
        ops.hstu_cache_append(st["qkv"][1], st["qkv"][2], st["cache"], table, st["lens"], st["pos"], off, st["ts"],
                              None, max_seq_len=1, new_lens=st["nl"], new_pos=st["np"], workspace=st["ws"][0])
        ops.hstu_cache_attn_fwd(st["qkv"][0], st["cache"], table, st["nl"], st["pos"], off, st["ts"], None, rp, rt,
                                out=st["out"], weights_out=st["cache"].weights, workspace=st["ws"][1], **st["kw"])
        st["lens"].copy_(st["nl"])
        st["pos"].copy_(st["np"])
        st["ts"].add_(7)

    eager, replay = fresh(), fresh()
    warm = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(replay)
    for t in toks:
        eager["qkv"].copy_(t)
        step(eager)
        replay["qkv"].copy_(t)
        graph.replay()
        assert torch.equal(eager["out"], replay["out"])
    assert eager["lens"].tolist() == [steps] * B
    assert_pool_equal(pool_of(replay["cache"]), pool_of(eager["cache"]))


@pytest.mark.parametrize("raw", [False, True])
def test_what_a_call_allocates_belongs_to_its_stream(raw, cuda_device, monkeypatch):
    """Memory of another stream's could be given out again while the call still runs."""
    made = []

    def recorded(*args, real=ops._cache_empty):
        made.append(real(*args))
        return made[-1]

    monkeypatch.setattr(ops, "_cache_empty", recorded)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    x = _attn_inputs(([300, 70], [3, 3], None), "bf16", 64, 2, 91)
    cache = to_cache(x["pool"], cuda_device, weights=True)
    g = {n: dev(x[n], cuda_device) for n in ("table", "lens", "seq_pos", "off", "ts", "rp", "rt")}
    q = x["q"].to(cuda_device)
    new_pages = np.full(x["table"].shape, -1, np.int32)
    new_pages[:, 0] = np.setdiff1d(np.arange(len(x["pool"]["positions"])), x["table"])[:2]
    new_pages = dev(new_pages, cuda_device)
    args = dict(max_seq_len=3, max_cache_len=300, inv_n=1 / 64, pos_lo=-100, pos_hi=100)
    torch.cuda.synchronize()
    out = ops.hstu_cache_attn_fwd(q, cache, g["table"], g["lens"], g["seq_pos"], g["off"], g["ts"], None, g["rp"],
                                  g["rt"], stream=stream, **args)
    ops.hstu_cache_append(q, q, cache, g["table"], g["lens"], g["seq_pos"], g["off"], g["ts"], None, max_seq_len=3,
                          stream=stream)
    ops.hstu_cache_evict(cache, g["table"], g["lens"], new_pages, keep=64, max_cache_len=300, stream=stream)
    torch.cuda.synchronize()
    owners = [[seg["stream"] for seg in torch.cuda.memory_snapshot()
               if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]] for t in made]
    assert len(made) == 9 and owners == [[side.cuda_stream]] * 9
    want = ops.hstu_cache_attn_fwd(q, to_cache(x["pool"], cuda_device), g["table"], g["lens"], g["seq_pos"], g["off"],
                                   g["ts"], None, g["rp"], g["rt"], **args)
    assert torch.equal(out, want)
