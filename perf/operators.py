"""Cases of the operators on an 8-bit key/value cache, for measuring them.

A serving program keeps each user's history as E4M3 codes in pages of 64 tokens,
with one power-of-two scale per page and head for keys and one for values:

  append   writes new history tokens' keys and values into the pages
  attn     attention of new tokens or candidates over the cached history, with
           the attention weight each cached token received where it is asked for
  evict    keeps the first, the last and the heaviest tokens in new pages

`run` computes them in plain torch operations, or (own = True) through the
library's calls.  Pages are [heads, 64, d] for keys and [heads, d, 64] for values.
"""

import math

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"


# ---- cases --------------------------------------------------------------------

def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", heads=4, d=128, seqs=1, len_lo=0, len_hi=0, n_lo=1, n_hi=1,
             targets=False, weights=False, addend=False, per_head=False, gaps=False, keep=0, first=0, recent=0,
             pos=4096, buckets=128, n_scale=16384, gap_s=300.0, std=1.0)
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token over a short history: latency
        _case("attn_one_token", "attn", len_lo=2048, len_hi=2048, weights=True, pos=2560, n_scale=2560, gap_s=120.0),
        # one token each for a batch of long histories (8k to 16k tokens), with the weights eviction needs
        _case("attn_token_batch", "attn", seqs=64, len_lo=8192, len_hi=16384, weights=True),
        # ranking: 512 candidates against 2048 tokens of history for each of 16 users
        _case("attn_ranking", "attn", seqs=16, heads=2, len_lo=2048, len_hi=2048, n_lo=512, n_hi=512, targets=True,
              addend=True, pos=2560, n_scale=2560, gap_s=120.0, std=0.02),
        # candidates against long histories, some tokens evicted before, weights taken
        _case("attn_candidates_long", "attn", seqs=8, len_lo=8192, len_hi=16384, n_lo=256, n_hi=512, targets=True,
              weights=True, gaps=True),
        # a few new tokens of short histories, head width 64, a bias table per head
        _case("attn_chunk_d64", "attn", seqs=32, d=64, len_lo=64, len_hi=1024, n_lo=1, n_hi=48, per_head=True,
              addend=True, pos=1024, buckets=64, n_scale=1024),
        # the small fp32 layer's sizes
        _case("attn_f32_small", "attn", dtype="f32", heads=2, d=32, seqs=4, len_lo=16, len_hi=128, n_lo=1, n_hi=16,
              weights=True, pos=127, buckets=32, n_scale=128, gap_s=60.0),
        # one new token for each of 64 users
        _case("append_token_batch", "append", seqs=64, len_lo=64, len_hi=4096, gaps=True),
        # whole long histories at once
        _case("append_histories", "append", seqs=8, n_lo=8192, n_hi=16384),
        # short histories with a part in the cache already, head width 64
        _case("append_chunks_d64", "append", seqs=32, d=64, len_lo=0, len_hi=512, n_lo=1, n_hi=1024),
        # one user's cache cut to half
        _case("evict_one", "evict", len_lo=2048, len_hi=2048, keep=1024, first=4, recent=256),
        # a batch of long caches cut to 4096 tokens
        _case("evict_batch", "evict", seqs=32, len_lo=8192, len_hi=16384, keep=4096, first=64, recent=1024, gaps=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn", "attn", "append", "evict"))
    f32 = op == "attn" and rng.random() < 0.2
    c = _case("drawn", op, dtype="f32" if f32 else "bf16", heads=rng.choice((1, 2, 4)),
              d=rng.choice((32, 64) if f32 else (64, 128)), seqs=_log(rng, 1, 64), gaps=rng.random() < 0.5,
              pos=rng.choice((127, 1024, 2560, 4096)), buckets=rng.choice((32, 64, 128)),
              std=rng.choice((0.02, 0.5, 1.0)), gap_s=rng.choice((60.0, 120.0, 300.0)))
    hi = _log(rng, 1, 512 if f32 else 16384)
    c.update(len_lo=rng.randint(0, hi), len_hi=hi)
    if op == "attn":
        n = _log(rng, 1, 16 if f32 else 512)
        c.update(n_lo=rng.randint(1, n), n_hi=n, targets=rng.random() < 0.5, weights=rng.random() < 0.5,
                 addend=rng.random() < 0.5, per_head=rng.random() < 0.3, n_scale=rng.choice((128, 2560, 16384)))
    elif op == "append":
        n = _log(rng, 1, 8192)
        c.update(n_lo=rng.randint(1, n), n_hi=n)
    else:
        c.update(keep=_log(rng, 1, hi), first=rng.choice((0, 4, 64)), recent=rng.choice((0, 16, 1000)))
    top = {k: max(w[k] for w in (work(x) for x in listed() if x["op"] == op)) for k in ("bytes", "flops")}
    while c["seqs"] > 1 and any(work(c)[k] > top[k] for k in top):
        c["seqs"] = max(1, c["seqs"] * 2 // 3)
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return [lo + int((hi - lo) * (i + 0.5) / n) for i in range(n)]


def _lengths(case):
    """(cached tokens, new tokens) of each sequence: pairs that the case fixes, in an order of its own."""
    ns = _spread(case["n_lo"], case["n_hi"], case["seqs"])
    mixed = np.random.RandomState(1).permutation(case["seqs"])
    return _spread(case["len_lo"], case["len_hi"], case["seqs"]), [ns[i] for i in mixed]


def work(case):
    lens, ns = _lengths(case)
    H, d, e = case["heads"], case["d"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "attn":
        L, T = sum(lens), sum(ns)
        b = L * (2 * H * d + 12) + T * H * d * e * (3 if case["addend"] else 2) + T * 8
        if case["weights"]:
            b += 8 * L
        return {"bytes": float(b), "flops": 4.0 * d * H * sum(x * y for x, y in zip(lens, ns))}
    if case["op"] == "append":
        T = sum(ns)
        return {"bytes": float(T * (2 * H * d * (e + 1) + 8 + 12 + 4)), "flops": 0.0}
    kept = sum(min(x, case["keep"]) for x in lens if x > case["keep"])
    read = sum(4 * x for x in lens if x > case["keep"])
    return {"bytes": float(read + kept * 2 * (2 * H * d + 16) + 4 * kept + 16 * case["seqs"]), "flops": 0.0}


# ---- inputs -------------------------------------------------------------------

def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _pages(n):
    return -(-n // PAGE)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    lens, ns = _lengths(case)
    order = rng.permutation(case["seqs"])
    lens, ns = [lens[i] for i in order], [ns[i] for i in order]
    B, H, d, op = case["seqs"], case["heads"], case["d"], case["op"]
    after = [x + (n if op == "append" else 0) for x, n in zip(lens, ns)]
    kept = [min(x, case["keep"]) if op == "evict" else 0 for x in lens]
    need = [_pages(x) for x in after]
    new = [_pages(x) for x in kept]
    cols = max(1, max(need), max(new))
    spare = sum(need) + sum(new)  # one page that no sequence owns fills the tables' unused entries
    ids = rng.permutation(spare)
    table = np.full((B, cols), spare, np.int32)
    new_table = np.full((B, cols), spare, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
        new_table[b, :new[b]] = ids[at:at + new[b]]
        at += new[b]
    dev = lambda a, t: torch.as_tensor(np.asarray(a), dtype=t, device=DEV)  # noqa: E731
    s = {"case": case, "table": dev(table, torch.int32), "lens": dev(lens, torch.int32),
         "max_len": max(lens), "max_new": max(ns), "max_after": max(after)}
    N = spare + 1
    # positions: dense, or with the holes that earlier evictions left
    slot = torch.arange(cols * PAGE, device=DEV)
    pos = slot * 2 + slot % 3 if case["gaps"] else slot
    gaps = torch.empty((B, cols * PAGE), device=DEV).exponential_(1.0 / case["gap_s"], generator=g)
    ts = 1_700_000_000 + torch.floor(torch.cumsum(gaps.double(), 1)).long()
    cached = slot[None, :] < s["lens"][:, None]
    s["positions"] = torch.zeros((N, PAGE), dtype=torch.int32, device=DEV)
    s["timestamps"] = torch.zeros((N, PAGE), dtype=torch.int64, device=DEV)
    pg = s["table"].long()
    s["positions"][pg] = torch.where(cached, pos[None, :], 0).int().view(B, cols, PAGE)
    s["timestamps"][pg] = torch.where(cached, ts, 0).view(B, cols, PAGE)
    s["weights"] = torch.rand((N, PAGE), device=DEV, generator=g)
    end = torch.where(s["lens"] > 0, pos[(s["lens"].long() - 1).clamp(min=0)] + 1, 0)
    s["seq_pos"] = end.int()
    mine = torch.zeros(N, dtype=torch.bool, device=DEV)
    mine[pg.reshape(-1)] = True
    mine[spare] = False
    for name, shape in (("k", (N, H, PAGE, d)), ("v", (N, H, d, PAGE))):
        x = torch.randn(shape, device=DEV, generator=g) * (mine[:, None, None, None] * case["std"])
        # a page's own spread, so that scales differ
        x *= torch.exp2(torch.randint(-2, 3, (N, H, 1, 1), device=DEV, generator=g).float())
        codes, s[name + "_scale"] = _quantise(x, (2, 3))
        s[name + "_codes"] = codes.view(torch.uint8)
    if op == "evict":
        s["new_table"] = dev(new_table, torch.int32)
        return s
    off = np.concatenate([[0], np.cumsum(ns)])
    T = int(off[-1])
    s["off"] = dev(off, torch.int64)
    s["row_seq"] = dev(np.repeat(np.arange(B), ns), torch.int64)
    s["row_idx"] = dev(np.concatenate([np.arange(n) for n in ns]), torch.int64)
    s["nt"] = dev(ns if case["targets"] else [0] * B, torch.int32)
    last = torch.where(s["lens"] > 0, ts.gather(1, (s["lens"].long() - 1).clamp(min=0)[:, None])[:, 0], ts[:, 0])
    step = torch.empty((B, max(ns)), device=DEV).exponential_(1.0 / case["gap_s"], generator=g)
    later = last[:, None] + torch.floor(torch.cumsum(step.double(), 1)).long()
    if case["targets"]:  # candidates carry the last token's stamp
        later = last[:, None].expand(B, max(ns))
    s["ts"] = later[s["row_seq"], s["row_idx"]].contiguous()
    rows = lambda std: (torch.randn((T, H, d), device=DEV, generator=g) * std).to(_dtype(case))  # noqa: E731
    if op == "append":
        s["k_new"], s["v_new"] = rows(case["std"]), rows(case["std"])
        return s
    s["q"] = rows(case["std"])
    s["addend"] = rows(0.05) if case["addend"] else None
    lead = (H,) if case["per_head"] else ()
    s["rab_pos"] = 0.1 * torch.randn(lead + (2 * case["pos"] + 1,), device=DEV, generator=g)
    s["rab_time"] = 0.1 * torch.randn(lead + (case["buckets"],), device=DEV, generator=g)
    s["weights_out"] = torch.zeros_like(s["weights"]) if case["weights"] else None
    return s


# ---- the plain forms ------------------------------------------------------------

def _quantise(x, dims):
    """E4M3 codes of x with one scale per block (its two axes `dims`): the smallest
    power of two that keeps the largest magnitude within 448; 0 for a zero block."""
    amax = x.abs().amax(dims)
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), 0.0)
    return _encode(x, scale[..., None, None]), scale


def _encode(x, scale):
    return (x / torch.where(scale > 0, scale, 1.0)).to(torch.float8_e4m3fn)


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale[..., None, None]


def run(state):
    return {"attn": _attn, "append": _append, "evict": _evict}[state["case"]["op"]](state)


def _attn(s):
    if own:
        return _own_attn(s)
    c = s["case"]
    B, H, d, n = c["seqs"], c["heads"], c["d"], s["max_new"]
    P = max(1, _pages(s["max_len"]))
    pg = s["table"][:, :P].long()
    L = P * PAGE
    k = _values(s["k_codes"][pg], s["k_scale"][pg]).permute(0, 2, 1, 3, 4).reshape(B, H, L, d)
    v = _values(s["v_codes"][pg], s["v_scale"][pg]).permute(0, 2, 1, 4, 3).reshape(B, H, L, d)
    at = s["off"][:-1, None] + torch.arange(n, device=DEV)
    real = at < s["off"][1:, None]
    at = torch.where(real, at, 0)
    q = s["q"].float()[at].permute(0, 2, 1, 3)
    hist = s["off"].diff() - s["nt"]
    i = torch.arange(n, device=DEV)
    p_i = s["seq_pos"][:, None] + torch.minimum(i[None, :], hist[:, None])
    dp = p_i[:, :, None] - s["positions"][pg].view(B, 1, L)
    dp = dp.clamp(-c["pos"], c["pos"]) + c["pos"]
    dt = s["ts"][at][:, :, None] - s["timestamps"][pg].view(B, 1, L)
    bucket = torch.frexp(dt.clamp(min=0).double() + 1.0)[1] - 1
    bucket = bucket.clamp(max=c["buckets"] - 1)
    x = torch.matmul(q, k.transpose(2, 3))
    if c["per_head"]:
        x += s["rab_pos"][:, dp.long()].transpose(0, 1)
        x += s["rab_time"][:, bucket.long()].transpose(0, 1)
    else:
        x += (s["rab_pos"][dp.long()] + s["rab_time"][bucket.long()])[:, None]
    ok = (torch.arange(L, device=DEV)[None, :] < s["lens"][:, None])[:, None, None, :] & real[:, None, :, None]
    p = torch.where(ok, x / (1.0 + torch.exp(-x)), 0.0) / c["n_scale"]
    o = torch.matmul(p, v)
    out = o.permute(0, 2, 1, 3)[s["row_seq"], s["row_idx"]]
    if s["addend"] is not None:
        out = out + s["addend"].float()
    out = out.to(_dtype(c))
    if not c["weights"]:
        return {"out": out}
    w = p.abs().sum((1, 2)).view(B, P, PAGE)
    have = (torch.arange(L, device=DEV)[None, :] < s["lens"][:, None]).view(B, P, PAGE)
    s["weights_out"][pg] = torch.where(have, s["weights"][pg] + w, s["weights_out"][pg])
    return {"out": out, "weights": s["weights_out"]}


def _append(s):
    if own:
        return _own_append(s)
    c = s["case"]
    B, H, d = c["seqs"], c["heads"], c["d"]
    lens, count = s["lens"].long(), s["off"].diff()
    J = _pages(PAGE - 1 + s["max_new"])  # blocks that a sequence may touch
    blk = lens[:, None] // PAGE + torch.arange(J, device=DEV)
    slot = blk[:, :, None] * PAGE + torch.arange(PAGE, device=DEV)
    i = slot - lens[:, None, None]
    new = (i >= 0) & (i < count[:, None, None])
    touched = new.any(2)
    pg = torch.where(touched, s["table"].long().gather(1, blk.clamp(max=s["table"].shape[1] - 1)),
                     s["table"].new_full((), s["k_scale"].shape[0] - 1).long())
    old = (i < 0) & touched[:, :, None]
    row = torch.where(new, s["off"][:-1, None, None] + i, 0)
    for name, x in (("k", s["k_new"]), ("v", s["v_new"])):
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        was = codes[pg]
        have = _values(was, scale[pg])  # [B, J, H, 64, d], or [B, J, H, d, 64] for values
        y = x.float()[row]              # [B, J, 64, H, d]
        if name == "k":
            y, o, w = y.permute(0, 1, 3, 2, 4), old[:, :, None, :, None], new[:, :, None, :, None]
        else:
            y, o, w = y.permute(0, 1, 3, 4, 2), old[:, :, None, None, :], new[:, :, None, None, :]
        y = torch.where(w, y, 0.0)
        fresh = _quantise(y, (3, 4))[1]
        size = torch.where(old.any(2)[:, :, None], torch.maximum(fresh, scale[pg]), fresh)
        put = _encode(torch.where(o, have, y), size[..., None, None]).view(torch.uint8)
        codes[pg] = torch.where(o | w, put, was)
        scale[pg] = torch.where(touched[:, :, None], size, scale[pg])
    s["timestamps"][pg] = torch.where(new, s["ts"][row], s["timestamps"][pg])
    s["positions"][pg] = torch.where(new, (s["seq_pos"][:, None, None] + i).int(), s["positions"][pg])
    s["weights"][pg] = torch.where(new, 0.0, s["weights"][pg])
    return _pool(s) | {"lens": (lens + count).int(), "seq_pos": (s["seq_pos"] + count).int()}


def _evict(s):
    if own:
        return _own_evict(s)
    c = s["case"]
    B, keep = c["seqs"], c["keep"]
    P = max(1, _pages(s["max_len"]))
    J = min(_pages(keep), s["new_table"].shape[1])  # more than the table's pages: nothing is cut
    L, K = P * PAGE, J * PAGE
    pg = s["table"][:, :P].long()
    lens = s["lens"].long()
    j = torch.arange(L, device=DEV)[None, :]
    there = j < lens[:, None]
    safe = (j < c["first"]) | (j >= lens[:, None] - c["recent"])
    # the last ones first, then the first ones, where `keep` has no room for both
    rank = torch.where(j >= lens[:, None] - c["recent"], math.inf, 0.0)
    key = torch.where(safe, 3.0e38, s["weights"][pg].view(B, L))
    key = torch.where(rank > 0, rank, key)
    key = torch.where(there, key, -math.inf)
    by = torch.sort(key, dim=1, descending=True, stable=True)[1]
    # among the last ones the latest, where `keep` is less than `recent`
    late = min(keep, c["recent"])
    chosen = torch.zeros((B, L + 1), dtype=torch.bool, device=DEV)
    nth = torch.arange(L, device=DEV)[None, :]
    n_last = torch.minimum(lens, torch.full_like(lens, c["recent"]))[:, None]
    n_skip = (n_last - late).clamp(min=0)
    take = (nth >= n_skip) & (nth < n_skip + keep)
    chosen.scatter_(1, torch.where(take, by, L), True)
    chosen = chosen[:, :L] & there
    cut = lens > keep
    src = torch.sort(torch.where(chosen, j, L), dim=1)[0]
    src = torch.nn.functional.pad(src, (0, max(0, K - L)), value=L)[:, :K]
    got = (src < L) & cut[:, None]
    src = torch.where(got, src, 0)
    page, slot = pg.gather(1, src // PAGE), src % PAGE
    to = torch.where(cut[:, None], s["new_table"][:, :J].long(), s["k_scale"].shape[0] - 1)
    have = got.view(B, J, PAGE)
    kk = s["k_codes"][page, :, slot].view(torch.float8_e4m3fn).float() * s["k_scale"][page][..., None]
    vv = s["v_codes"][page, :, :, slot].view(torch.float8_e4m3fn).float() * s["v_scale"][page][..., None]
    for name, x in (("k", kk), ("v", vv)):  # [B, K, H, d]
        x = torch.where(got[:, :, None, None], x, 0.0).view(B, J, PAGE, c["heads"], c["d"])
        x = x.permute(0, 1, 3, 2, 4) if name == "k" else x.permute(0, 1, 3, 4, 2)
        codes, scale = _quantise(x, (3, 4))
        w = have[:, :, None, :, None] if name == "k" else have[:, :, None, None, :]
        s[name + "_codes"][to] = torch.where(w, codes.view(torch.uint8), s[name + "_codes"][to])
        s[name + "_scale"][to] = torch.where(cut[:, None, None], scale, s[name + "_scale"][to])
    for name in ("timestamps", "positions", "weights"):
        s[name][to] = torch.where(have, s[name][page, slot].view(B, J, PAGE), s[name][to])
    kept = torch.where(got, src, -1)[:, :keep].int()
    if kept.shape[1] < keep:
        kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[1]), value=-1)
    kept = torch.where(cut[:, None], kept, torch.where(j < lens[:, None], j, -1).int()[:, :keep] if L >= keep else
                       torch.nn.functional.pad(torch.where(j < lens[:, None], j, -1).int(), (0, keep - L), value=-1))
    return _pool(s) | {"table": torch.where(cut[:, None], s["new_table"], s["table"]),
                       "lens": lens.clamp(max=keep).int(), "kept": kept}


def _pool(s):
    f8 = torch.float8_e4m3fn
    return {"k": s["k_codes"].view(f8), "v": s["v_codes"].view(f8), "k_scale": s["k_scale"], "v_scale": s["v_scale"],
            "timestamps": s["timestamps"], "positions": s["positions"], "weights": s["weights"]}


# ---- the library's calls ----------------------------------------------------------

def _handle(s):
    """What a serving program keeps between calls: the cache's handle and a workspace."""
    if "cache" not in s:
        from hstu_sequential_transduction_b200 import ops
        s["ops"] = ops
        s["cache"] = ops.HstuCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["timestamps"],
                                   s["positions"], s["weights"])
        s["workspace"] = None
    return s["ops"], s["cache"]


def _own_attn(s):
    ops, cache = _handle(s)
    c = s["case"]
    kw = dict(max_seq_len=s["max_new"], max_cache_len=s["max_len"], inv_n=1.0 / c["n_scale"], pos_lo=-c["pos"],
              pos_hi=c["pos"])
    if s["workspace"] is None:
        s["workspace"] = ops.alloc_workspace(ops.hstu_cache_attn_workspace_size(
            s["q"], cache, s["table"], s["rab_pos"], s["rab_time"], weights=c["weights"], **kw), s["q"].device)
    out = ops.hstu_cache_attn_fwd(s["q"], cache, s["table"], s["lens"], s["seq_pos"], s["off"], s["ts"], s["nt"],
                                  s["rab_pos"], s["rab_time"], addend=s["addend"], weights_out=s["weights_out"],
                                  workspace=s["workspace"], **kw)
    return {"out": out, "weights": s["weights_out"]} if c["weights"] else {"out": out}


def _own_append(s):
    ops, cache = _handle(s)
    if s["workspace"] is None:
        s["workspace"] = ops.alloc_workspace(ops.hstu_cache_append_workspace_size(), s["k_new"].device)
    lens, pos = ops.hstu_cache_append(s["k_new"], s["v_new"], cache, s["table"], s["lens"], s["seq_pos"], s["off"],
                                      s["ts"], None, max_seq_len=s["max_new"], workspace=s["workspace"])
    return _pool(s) | {"lens": lens, "seq_pos": pos}


def _own_evict(s):
    ops, cache = _handle(s)
    c = s["case"]
    kw = dict(keep=c["keep"], first=c["first"], recent=c["recent"], max_cache_len=s["max_len"])
    if s["workspace"] is None:
        s["workspace"] = ops.alloc_workspace(ops.hstu_cache_evict_workspace_size(cache, s["table"], **kw),
                                             s["table"].device)
    table, lens, kept = ops.hstu_cache_evict(cache, s["table"], s["lens"], s["new_table"], workspace=s["workspace"],
                                             **kw)
    return _pool(s) | {"table": table, "lens": lens, "kept": kept}


# ---- the definitions in 64 bits -------------------------------------------------------

def _code_values():
    """The 256 values of E4M3: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _near(y):
    """The E4M3 value nearest to y (|y| <= 448), ties to even."""
    a = y.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(y / step) * step


def _scales(x):
    """The smallest powers of two that keep the largest magnitudes x [pages, heads] within 448."""
    e = torch.ceil(torch.log2(torch.where(x > 0, x, 1.0) / 448.0))
    e = torch.where(x > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(x <= 448.0 * torch.exp2(e - 1), e - 1, e)
    return torch.where(x > 0, torch.exp2(e), 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    val = _code_values()
    return {"attn": _exact_attn, "append": _exact_append, "evict": _exact_evict}[case["op"]](s, case, val)


def _exact_attn(s, c, val):
    lens, off, table = s["lens"].tolist(), s["off"].tolist(), s["table"].long()
    H, d = c["heads"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    w = s["weights_out"].double() if c["weights"] else None
    powers = 2 ** torch.arange(0, 62, device=DEV)
    rp, rt = s["rab_pos"].double(), s["rab_time"].double()
    if not c["per_head"]:
        rp, rt = rp.expand(H, -1), rt.expand(H, -1)
    for b, L in enumerate(lens):
        lo, hi = off[b], off[b + 1]
        if L == 0 or hi == lo:
            if L and w is not None:
                pg = table[b, :_pages(L)]
                flat = w[pg].reshape(-1)
                flat[:L] = s["weights"][pg].double().reshape(-1)[:L]
                w[pg] = flat.view(-1, PAGE)
            continue
        pg = table[b, :_pages(L)]
        k = (val[s["k_codes"][pg].long()] * s["k_scale"][pg].double()[:, :, None, None]).transpose(0, 1)
        v = (val[s["v_codes"][pg].long()] * s["v_scale"][pg].double()[:, :, None, None]).permute(1, 0, 3, 2)
        k, v = k.reshape(H, -1, d)[:, :L], v.reshape(H, -1, d)[:, :L]
        n, nt = hi - lo, int(s["nt"][b])
        i = torch.arange(n, device=DEV).clamp(max=n - nt) + s["seq_pos"][b].long()
        dp = (i[:, None] - s["positions"][pg].reshape(-1)[:L].long()).clamp(-c["pos"], c["pos"]) + c["pos"]
        dt = (s["ts"][lo:hi, None] - s["timestamps"][pg].reshape(-1)[:L]).clamp(min=0) + 1
        bk = (torch.searchsorted(powers, dt, right=True) - 1).clamp(max=c["buckets"] - 1)
        for h in range(H):
            x = s["q"][lo:hi, h].double() @ k[h].T + rp[h][dp] + rt[h][bk]
            p = x * torch.sigmoid(x) / c["n_scale"]
            out[lo:hi, h] = p @ v[h]
            if w is not None:
                if h == 0:
                    flat = w[pg].reshape(-1)
                    flat[:L] = s["weights"][pg].double().reshape(-1)[:L]
                flat[:L] += p.abs().sum(0)
        if w is not None:
            w[pg] = flat.view(-1, PAGE)
    if s["addend"] is not None:
        out += s["addend"].double()
    return {"out": out} if w is None else {"out": out, "weights": w}


def _exact_pool(s, val):
    return {"k": val[s["k_codes"].long()], "v": val[s["v_codes"].long()], "k_scale": s["k_scale"].double(),
            "v_scale": s["v_scale"].double(), "timestamps": None, "positions": None,
            "weights": s["weights"].double()}


def _exact_append(s, c, val):
    e = _exact_pool(s, val)
    lens, off, table = s["lens"].tolist(), s["off"].tolist(), s["table"].long()
    for b, L in enumerate(lens):
        n = off[b + 1] - off[b]
        if n == 0:
            continue
        lo, hi = L // PAGE, _pages(L + n)
        pg = table[b, lo:hi]
        a, z = L - lo * PAGE, L + n - lo * PAGE  # the new tokens' slots among these pages
        for name, x in (("k", s["k_new"]), ("v", s["v_new"])):
            codes = e[name][pg] if name == "k" else e[name][pg].transpose(2, 3)  # [pages, H, 64, d]
            sc = e[name + "_scale"][pg]
            t = codes.permute(0, 2, 1, 3).reshape(-1, c["heads"], c["d"]).clone()
            old = t * sc[:, None, :].expand(-1, PAGE, -1).reshape(-1, c["heads"], 1)
            y = torch.zeros_like(t)
            y[a:z] = x[off[b]:off[b + 1]].double()
            new = _scales(y.view(-1, PAGE, c["heads"], c["d"]).abs().amax((1, 3)))
            if a:
                new[0] = torch.maximum(new[0], sc[0])
                y[:a] = old[:a]
            div = torch.where(new > 0, new, 1.0)[:, None, :].expand(-1, PAGE, -1).reshape(-1, c["heads"], 1)
            t[:z] = _near(y[:z] / div[:z])
            t = t.view(-1, PAGE, c["heads"], c["d"]).permute(0, 2, 1, 3)
            e[name][pg] = t if name == "k" else t.transpose(2, 3)
            e[name + "_scale"][pg] = new
        w = e["weights"][pg].reshape(-1)
        w[a:z] = 0.0
        e["weights"][pg] = w.view(-1, PAGE)
    return e | {"lens": None, "seq_pos": None}


def _exact_evict(s, c, val):
    e = _exact_pool(s, val)
    lens, table, new_table = s["lens"].tolist(), s["table"].long(), s["new_table"].long()
    keep = c["keep"]
    for b, L in enumerate(lens):
        if L <= keep:
            continue
        w = s["weights"][table[b, :_pages(L)]].reshape(-1)[:L].cpu().numpy()
        late = min(keep, c["recent"])
        early = min(keep - late, c["first"], L - late)
        mid = np.arange(early, L - late)
        best = mid[np.argsort(-w[mid].astype(np.float64), kind="stable")[:keep - late - early]]
        kept = np.concatenate([np.arange(early), np.sort(best), np.arange(L - late, L)])
        j = torch.as_tensor(kept, device=DEV)
        page, slot = table[b][j // PAGE], j % PAGE
        to = new_table[b, :_pages(keep)]
        for name in ("k", "v"):
            x = e[name][page, :, slot] if name == "k" else e[name][page, :, :, slot]  # [keep, H, d]
            x = x * e[name + "_scale"][page][..., None]
            full = torch.zeros((len(to) * PAGE,) + x.shape[1:], dtype=torch.float64, device=DEV)
            full[:keep] = x
            sc = _scales(full.view(-1, PAGE, c["heads"], c["d"]).abs().amax((1, 3)))
            div = torch.where(sc > 0, sc, 1.0)[:, None, :].expand(-1, PAGE, -1).reshape(-1, c["heads"], 1)
            codes = e[name][to] if name == "k" else e[name][to].transpose(2, 3)
            t = codes.permute(0, 2, 1, 3).reshape(full.shape).clone()
            t[:keep] = _near(full / div)[:keep]
            t = t.view(-1, PAGE, c["heads"], c["d"]).permute(0, 2, 1, 3)
            e[name][to] = t if name == "k" else t.transpose(2, 3)
            e[name + "_scale"][to] = sc
        flat = e["weights"][to].reshape(-1)
        flat[:keep] = s["weights"][page, slot].double()
        e["weights"][to] = flat.view(-1, PAGE)
    return e | {"table": None, "lens": None, "kept": None}
