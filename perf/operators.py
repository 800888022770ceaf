"""The block-scaled 8-bit KV cache: its operators' plain forms and the
framework's calls for them, over the sizes they are meant for.

A pool holds one E4M3 code per element, [num_blocks][16][kv heads][head dim],
and each (block, kv head) of it one power-of-two scale 2^e, kept as the byte
e + 127: the cached value is code * 2^e.

write    The step's new K and V go into the cache.  A block written from its
         first slot on takes the smallest exponent e in [-56, 56] with
         amax <= 448 * 2^e over its new finite elements; a block that already
         holds earlier tokens keeps the larger of that and its own, and when
         its exponent grows the codes of its earlier tokens are re-coded.
         The pass then reads back the rows of the step (from the first block
         written on) as 16-bit values: what the cache now stands for.
read     Rows of every request's context as 16-bit values, request after
         request, without gaps.
attend   Causal grouped-query attention of the step's tokens over their
         requests' contexts, read through the block tables.

A case's lengths come from the case alone ("lens"); its values from the seed.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16
E_MIN, E_MAX, BIAS = -56, 56, 127
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
WORKSPACE_BYTES = 256 << 20   # an engine's one workspace, kept for all its steps


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _case(op, name=None, *, reqs, ctx, new=(1, 1), chunks=0, chunk_new=(0, 0), chunk_ctx=(0, 0),
          shared=0, hq=0, hkv=8, d=128, dtype="bf16", lens=0):
    """reqs requests with ctx (low, high) tokens already cached and new (low,
    high) tokens of this step, after `chunks` requests of chunk_new tokens at
    chunk_ctx; the first `shared` cached tokens of the reqs requests lie in
    common blocks."""
    c = {"op": op, "reqs": reqs, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
         "new_hi": new[1], "chunks": chunks, "chunk_lo": chunk_new[0], "chunk_hi": chunk_new[1],
         "chunk_ctx_lo": chunk_ctx[0], "chunk_ctx_hi": chunk_ctx[1], "shared": shared, "hq": hq,
         "hkv": hkv, "d": d, "dtype": dtype, "lens": lens}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # The smallest step: three requests of a few tokens; latency is all of it.
        _case("write", "write-small", reqs=3, ctx=(0, 40), new=(2, 5), hkv=2, d=64, lens=1),
        # A decode step: one token of each running request joins its last block.
        _case("write", "write-decode", reqs=256, ctx=(127, 4095), hkv=8, d=128, lens=2),
        # A prompt chunk beside decodes: the most rows a step writes.
        _case("write", "write-mixed", reqs=200, ctx=(255, 8191), chunks=1, chunk_new=(5000, 5000),
              chunk_ctx=(2048, 2048), hkv=8, d=128, lens=3),
        # A few short contexts handed on as 16-bit rows.
        _case("read", "read-short", reqs=5, ctx=(3, 333), hkv=4, d=64, dtype="fp16", lens=4),
        # Whole contexts handed to another engine or to a dense kernel.
        _case("read", "read-contexts", reqs=64, ctx=(256, 8192), hkv=8, d=128, lens=5),
        # The smallest step's attention: latency is all of it.
        _case("attend", "attend-small", reqs=3, ctx=(0, 40), new=(2, 5), hq=4, hkv=2, d=64, lens=1),
        # The decode step: every request reads its whole context for one token.
        _case("attend", "attend-decode", reqs=256, ctx=(127, 4095), hq=32, hkv=8, d=128, lens=2),
        # Few requests over long contexts that share a prompt's blocks.
        _case("attend", "attend-long", reqs=6, ctx=(30001, 32767), shared=16384, hq=32, hkv=8,
              d=128, lens=6),
        # Drafted tokens being verified: up to 8 a request, 7 heads a kv head.
        _case("attend", "attend-drafts", reqs=64, ctx=(1, 2000), new=(1, 8), hq=28, hkv=4, d=64,
              dtype="fp16", lens=7),
        # One long prompt chunk: bound by the matrix products.
        _case("attend", "attend-chunk", reqs=0, ctx=(0, 0), chunks=1, chunk_new=(5000, 5000),
              chunk_ctx=(2048, 2048), hq=32, hkv=8, d=128, lens=8),
        # Several ragged prompts from their first token on.
        _case("attend", "attend-prompts", reqs=0, ctx=(0, 0), chunks=5, chunk_new=(17, 1300),
              chunk_ctx=(0, 0), hq=16, hkv=16, d=64, dtype="fp16", lens=9),
        # A prompt chunk beside decodes in one call.
        _case("attend", "attend-mixed", reqs=100, ctx=(255, 4095), chunks=1,
              chunk_new=(2000, 2000), chunk_ctx=(501, 501), hq=40, hkv=8, d=128, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    lens = rng.randrange(1 << 20)
    hkv = rng.choice([1, 2, 3, 4, 8, 12])
    if op == "write":
        hi = _log(rng, 2, 8000)
        chunks = rng.choice([0, 0, 1, 2])
        c = _log(rng, 17, 2500)
        return _case(op, reqs=_log(rng, 1, 300), ctx=(0, hi), new=(1, rng.choice([1, 1, 4, 16])),
                     chunks=chunks, chunk_new=(max(1, c // 2), c), chunk_ctx=(0, _log(rng, 1, 2048)),
                     hkv=hkv if hkv < 12 else 8, d=d, dtype=dtype, lens=lens)
    if op == "read":
        hi = _log(rng, 1, 8192)
        return _case(op, reqs=_log(rng, 1, max(1, min(200, 200000 // hi))), ctx=(0, hi),
                     hkv=min(hkv, 8), d=d, dtype=dtype, lens=lens)
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    hkv = min(hkv, 40 // g)
    form = rng.choice(["decode", "decode", "short", "chunk", "mixed"])
    if form == "decode":
        hi = _log(rng, 1, 32768)
        shared = rng.choice([0, 0, hi // 32 * 16])
        return _case(op, reqs=_log(rng, 1, max(1, min(256, 500000 // hi))), ctx=(shared, hi),
                     shared=shared, hq=hkv * g, hkv=hkv, d=d, dtype=dtype, lens=lens)
    if form == "short":
        hi = _log(rng, 1, 4000)
        return _case(op, reqs=_log(rng, 1, max(1, min(128, 200000 // hi))), ctx=(0, hi),
                     new=(1, rng.randint(2, 16)), hq=hkv * g, hkv=hkv, d=d, dtype=dtype, lens=lens)
    n = _log(rng, 17, 2000)
    if form == "chunk":
        return _case(op, reqs=0, ctx=(0, 0), chunks=rng.randint(1, 3), chunk_new=(max(17, n // 2), n),
                     chunk_ctx=(0, _log(rng, 1, 2000)), hq=hkv * g, hkv=hkv, d=d, dtype=dtype,
                     lens=lens)
    return _case(op, reqs=_log(rng, 1, 100), ctx=(0, _log(rng, 1, 4000)), chunks=1, chunk_new=(n, n),
                 chunk_ctx=(0, _log(rng, 1, 2000)), hq=hkv * g, hkv=hkv, d=d, dtype=dtype, lens=lens)


def _lengths(case):
    """(cached tokens, new tokens) of each request."""
    rng = np.random.default_rng(case["lens"])
    span = lambda lo, hi, n: rng.integers(lo, hi, size=n, endpoint=True)  # noqa: E731
    c, r = case["chunks"], case["reqs"]
    old = np.concatenate([span(case["chunk_ctx_lo"], case["chunk_ctx_hi"], c),
                          span(case["ctx_lo"], case["ctx_hi"], r)])
    new = np.concatenate([span(case["chunk_lo"], case["chunk_hi"], c),
                          span(case["new_lo"], case["new_hi"], r)])
    return old.astype(np.int64), new.astype(np.int64)


def _read_range(case):
    """(first position, rows) that the pass reads back of each request: from
    the first block that the step writes on, or the whole context."""
    old, new = _lengths(case)
    if case["op"] == "write":
        first = old // BLOCK * BLOCK
        return first, old + new - first
    return np.zeros_like(old), old + new


# ---------------------------------------------------------------------------
# A state: what an engine holds before the call
# ---------------------------------------------------------------------------

def _pow2(e):
    """2^e in float32, exactly (e an integer tensor in [-126, 127])."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _coded(x):
    """float32 [..., 16, H, D] -> E4M3 codes and scale bytes [..., H]."""
    amax = x.abs().amax(dim=(-3, -1))
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 0.875, ex - 9, ex - 8).clamp(E_MIN, E_MAX)
    codes = (x * _pow2(-e)[..., None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return codes.to(torch.float8_e4m3fn).view(torch.uint8), (e + BIAS).to(torch.uint8)


def _pool(blocks, case, gen, spread):
    """A pool of N(0, 1) values whose size differs from block to block and
    from head to head (2^(spread * N(0, 1))), as keys and values do."""
    dev = "cuda"
    h, d = case["hkv"], case["d"]
    codes = torch.empty((blocks, BLOCK, h, d), dtype=torch.uint8, device=dev)
    scales = torch.empty((blocks, h), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // (BLOCK * h * d))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn((n, BLOCK, h, d), generator=gen, device=dev)
        x *= torch.exp2(spread * torch.randn((n, 1, h, 1), generator=gen, device=dev))
        codes[i:i + n], scales[i:i + n] = _coded(x)
    return codes, scales


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    host = np.random.default_rng(int(seed))
    old, new = _lengths(case)
    total = old + new
    r, h, d, dt = len(old), case["hkv"], case["d"], DTYPES[case["dtype"]]
    # the block tables: a random order of the pool, shared blocks first
    need = -(-total // BLOCK)
    sh = np.where(np.arange(r) >= case["chunks"], case["shared"] // BLOCK, 0)
    blocks = int((need - sh).sum()) + int(sh.max(initial=0))
    nb = blocks + max(1, blocks // 10)
    order = host.permutation(nb).astype(np.int32)
    width = int(need.max())
    table = np.full((r, width), -1, np.int32)
    common, at = order[:int(sh.max(initial=0))], int(sh.max(initial=0))
    for i in range(r):
        table[i, :sh[i]] = common[:sh[i]]
        n = int(need[i] - sh[i])
        table[i, sh[i]:need[i]] = order[at:at + n]
        at += n
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    i32 = lambda a: up(a.astype(np.int32))  # noqa: E731
    t = int(new.sum())
    s = {"case": case, "table": up(table), "tokens": t, "max_new": int(new.max()),
         "max_len": int(total.max()), "seq_lens": i32(total),
         "starts": i32(np.concatenate([[0], np.cumsum(new)])),
         "scale": 1.0 / math.sqrt(d)}
    s["k"], s["k_scales"] = _pool(nb, case, gen, 0.7)
    s["v"], s["v_scales"] = _pool(nb, case, gen, 1.0)
    if case["op"] == "write":
        # the step's own projections: one [T, ...] tensor, K and V views of it
        qkv = torch.randn((t, 4 * h, d), generator=gen, device=dev)
        qkv *= torch.exp2(torch.randn((t, 4 * h, 1), generator=gen, device=dev))
        qkv = qkv.to(dt)
        s["key"], s["value"] = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
        # request and position of each token, as the step's index build leaves them
        req = np.repeat(np.arange(r), new)
        s["req"] = i32(req)
        s["pos"] = i32(np.arange(t) - (np.cumsum(new) - new)[req] + old[req])
    if case["op"] in ("write", "read"):
        first, rows = _read_range(case)
        n = int(rows.sum())
        s["first"], s["row_starts"] = i32(first), i32(np.concatenate([[0], np.cumsum(rows)]))
        s["rows"] = n
        s["key_out"] = torch.empty((n, h, d), dtype=dt, device=dev)
        s["value_out"] = torch.empty((n, h, d), dtype=dt, device=dev)
    if case["op"] == "attend":
        s["q"] = torch.randn((t, case["hq"], d), generator=gen, device=dev).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
        # the step's plan: its prompt chunks and its other requests, apart
        chunk = new > 16
        pick = lambda m: (up(np.flatnonzero(m)), int(new[m].max(initial=0)),  # noqa: E731
                          int(total[m].max(initial=0)))
        s["long"], s["short"] = pick(chunk), pick(~chunk)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _values(codes, scale_bytes):
    """Codes [..., H, D] and scale bytes [..., H] as float32 values."""
    e = scale_bytes.to(torch.int32) - BIAS
    return codes.view(torch.float8_e4m3fn).float() * _pow2(e)[..., None]


def _plain_write_one(x, codes, scales, blk, off, first, first_blk):
    """One of K and V: x float32 [T, H, D] to block blk[t], slot off[t]; each
    request's first block first_blk holds first[r] earlier tokens."""
    nb, _, h, _ = codes.shape
    finite = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    amax = torch.zeros((nb, h), device=x.device).index_reduce_(0, blk, finite.amax(-1), "amax")
    start = torch.full((nb,), BLOCK, device=x.device).index_reduce_(0, blk, off, "amin")
    m, ex = torch.frexp(amax)
    e_new = torch.where(m <= 0.875, ex - 9, ex - 8)
    e_new = torch.where(amax > 0, e_new, torch.full_like(e_new, E_MIN)).clamp(E_MIN, E_MAX)
    e_old = (scales.to(torch.int32) - BIAS).clamp(E_MIN, E_MAX)
    e = torch.where((start == 0)[:, None], e_new, torch.maximum(e_old, e_new))
    # the earlier tokens of the requests' first blocks
    held = codes[first_blk]
    down = (e_old - e)[first_blk].clamp(max=0)
    again = held.view(torch.float8_e4m3fn).float() * _pow2(down)[:, None, :, None]
    again = again.to(torch.float8_e4m3fn).view(torch.uint8)
    live = torch.arange(BLOCK, device=x.device)[None, :] < first[:, None]
    codes[first_blk] = torch.where(live[:, :, None, None], again, held)
    new = (x * _pow2(-e)[blk][..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes[blk, off] = new.to(torch.float8_e4m3fn).view(torch.uint8)
    scales.copy_(torch.where((start < BLOCK)[:, None], (e + BIAS).to(torch.uint8), scales))


def _plain_write(s):
    pos, table = s["pos"].long(), s["table"]
    blk = table[s["req"].long(), pos // BLOCK].long()
    off = pos % BLOCK
    at = (s["seq_lens"] - (s["starts"][1:] - s["starts"][:-1])).long()   # first new position
    rows = torch.arange(table.shape[0], device=table.device)
    first_blk = table[rows, at // BLOCK].long()
    _plain_write_one(s["key"].float(), s["k"], s["k_scales"], blk, off, at % BLOCK, first_blk)
    _plain_write_one(s["value"].float(), s["v"], s["v_scales"], blk, off, at % BLOCK, first_blk)


def _plain_read(s):
    n = s["rows"]
    row = torch.arange(n, device="cuda")
    starts = s["row_starts"].long()
    req = torch.searchsorted(starts, row, right=True) - 1
    pos = s["first"].long()[req] + row - starts[req]
    blk = s["table"][req, pos // BLOCK].long()
    off = pos % BLOCK
    dt = s["key_out"].dtype
    s["key_out"].copy_(_values(s["k"][blk, off], s["k_scales"][blk]).to(dt))
    s["value_out"].copy_(_values(s["v"][blk, off], s["v_scales"][blk]).to(dt))


def _plain_attend(s, group, out):
    """The requests of `group`, padded to its longest, into out [T + 1, Hq, D]
    (row T takes what is past a request)."""
    reqs, mq, ml = group
    if not mq:
        return
    c, n_req = s["case"], reqs.shape[0]
    hq, h, d = c["hq"], c["hkv"], c["d"]
    g = hq // h
    table, pages = s["table"][reqs].clamp(min=0).long(), -(-ml // BLOCK)
    at = table[:, :pages]
    k = _values(s["k"][at], s["k_scales"][at][:, :, None]).view(n_req, pages * BLOCK, h, d)
    v = _values(s["v"][at], s["v_scales"][at][:, :, None]).view(n_req, pages * BLOCK, h, d)
    starts = s["starts"].long()
    start, n = starts[reqs], starts[reqs + 1] - starts[reqs]
    total = s["seq_lens"].long()[reqs]
    i = torch.arange(mq, device="cuda")
    tok = torch.where(i[None] < n[:, None], start[:, None] + i, s["tokens"])     # [R, mq]
    q = s["q"][tok.clamp(max=s["tokens"] - 1)].float()                           # [R, mq, Hq, D]
    q = q.view(n_req, mq, h, g, d).permute(0, 2, 1, 3, 4).reshape(n_req, h, mq * g, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                  # [R, H, mq*g, L]
    last = (total - n)[:, None] + i                                              # [R, mq]
    j = torch.arange(pages * BLOCK, device="cuda")
    hidden = j > last.clamp(min=0).repeat_interleave(g, 1)[:, :, None]           # [R, mq*g, L]
    score.masked_fill_(hidden[:, None], -math.inf)
    score -= score.amax(-1, keepdim=True)
    score.exp_()
    total_w = score.sum(-1, keepdim=True)
    # slots past a context may hold anything: no weight, no value
    v = torch.where((j < total[:, None])[:, :, None, None], v, 0.0)
    o = torch.matmul(score, v.permute(0, 2, 1, 3)) / total_w                     # [R, H, mq*g, D]
    o = o.view(n_req, h, mq, g, d).permute(0, 2, 1, 3, 4).reshape(n_req * mq, hq, d)
    out[tok.reshape(-1)] = o.to(out.dtype)


def _plain(s):
    op = s["case"]["op"]
    if op == "attend":
        out = torch.empty((s["tokens"] + 1, *s["q"].shape[1:]), dtype=s["q"].dtype, device="cuda")
        _plain_attend(s, s["short"], out)
        _plain_attend(s, s["long"], out)
        return {"out": out[:-1]}
    if op == "write":
        _plain_write(s)
    _plain_read(s)
    return {"key": s["key_out"], "value": s["value_out"]}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _calls(s):
    import paged_kv_attention_prepare_gb300 as pa

    op = s["case"]["op"]
    if op == "attend":
        pa.pa_attention_scaled(s["q"], s["k"], s["v"], s["k_scales"], s["v_scales"], s["table"],
                               s["starts"], s["seq_lens"], s["max_new"], s["max_len"], s["scale"],
                               s["out"], s["workspace"], shared_blocks=s["case"]["shared"] > 0)
        return {"out": s["out"]}
    if op == "write":
        pa.pa_cache_write_scaled(s["key"], s["value"], s["k"], s["v"], s["k_scales"], s["v_scales"],
                                 s["table"], s["starts"], s["seq_lens"])
    pa.pa_cache_read(s["k"], s["v"], s["table"], s["first"], s["row_starts"], s["key_out"],
                     s["value_out"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    return {"key": s["key_out"], "value": s["value_out"]}


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    old, new = _lengths(case)
    total = old + new
    h, d, t = case["hkv"], case["d"], int(new.sum())
    row = h * d                                   # elements of one token's K (or V)
    if case["op"] in ("write", "read"):
        _, rows = _read_range(case)
        n = int(rows.sum())
        pages = int((-(-rows // BLOCK)).sum())
        # codes and scales in, K and V rows out, twice (K and V)
        read_back = 2 * (n * row + pages * h + n * row * 2)
        if case["op"] == "read":
            return {"bytes": read_back, "flops": 0}
        # the new rows in, their codes and scales out
        return {"bytes": read_back + 2 * (t * row * 2 + t * row + pages * h), "flops": 0}
    pages = -(-total // BLOCK)
    sh = min(case["shared"] // BLOCK, int(pages.min())) if case["reqs"] else 0
    extra = max(0, case["reqs"] - 1) * sh         # shared blocks are read once
    kv = 2 * ((int(total.sum()) - extra * BLOCK) * row + (int(pages.sum()) - extra) * h)
    seen = int((old * new + new * (new + 1) // 2).sum())
    return {"bytes": kv + 2 * t * case["hq"] * d * 2, "flops": 4 * d * case["hq"] * seen}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_table():
    """The values of the codes 0x00 .. 0x7e, ascending."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def _decode64(codes):
    """E4M3 bytes as float64."""
    full = np.concatenate([_e4m3_table(), [np.nan]])
    full = torch.from_numpy(np.concatenate([full, -full])).to("cuda")
    return full[codes.long()]


def _encode64(y):
    """The nearest E4M3 values of float64 y, ties to the even code, at most
    448 in magnitude."""
    tab = torch.from_numpy(_e4m3_table()).to("cuda")
    mid = (tab[1:] + tab[:-1]) / 2
    a = y.abs()
    up = torch.searchsorted(mid, a)                # below or on the midpoint: the lower code
    tie = (up < mid.numel()) & (mid[up.clamp(max=mid.numel() - 1)] == a) & (up % 2 == 1)
    return torch.copysign(tab[up + tie.long()], y)


def _pow2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rows(case, s):
    """Each request's (K, V) of the positions read back, in float64."""
    old, new = _lengths(case)
    first, rows = _read_range(case)
    table = s["table"].cpu().numpy()
    starts = np.concatenate([[0], np.cumsum(new)])
    got = {}
    for name, x in (("k", s.get("key")), ("v", s.get("value"))):
        parts = []
        for r in range(len(old)):
            lo, hi = int(first[r]), int(first[r] + rows[r])
            pages = torch.from_numpy(table[r, lo // BLOCK:-(-hi // BLOCK)].astype(np.int64)).cuda()
            val = _decode64(s[name][pages])                          # [pages, 16, H, D]
            e = (s[name + "_scales"][pages].double() - BIAS)         # [pages, H]
            if x is not None and new[r]:
                # positions of these pages that the step writes, and their values
                pos = lo + torch.arange(pages.numel() * BLOCK, device="cuda").view(-1, BLOCK)
                mine = (pos >= int(old[r])) & (pos < hi)
                src = x[int(starts[r]):int(starts[r + 1])].double()
                fresh = torch.zeros_like(val)
                fresh[mine] = src
                amax = torch.where(torch.isfinite(fresh), fresh.abs(), 0.0).amax((1, 3))
                # smallest e with amax <= 448 * 2^e, by trial
                trial = torch.arange(E_MIN, E_MAX + 1, device="cuda", dtype=torch.float64)
                fits = amax[..., None] <= E4M3_MAX * _pow2_64(trial)
                need = (E_MIN + (~fits).sum(-1).double()).clamp(max=E_MAX)
                holds = (pos[:, :1] < int(old[r]))                   # earlier tokens in the page
                e2 = torch.where(holds, torch.maximum(e.clamp(E_MIN, E_MAX), need), need)
                kept = _encode64(val * _pow2_64(e - e2)[:, None, :, None])
                put = _encode64(fresh * _pow2_64(-e2)[:, None, :, None])
                val, e = torch.where(mine[:, :, None, None], put, kept), e2
            val = val * _pow2_64(e)[:, None, :, None]
            parts.append(val.reshape(-1, *val.shape[2:])[:hi - lo])
        got[name] = parts
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("write", "read"):
        got = _exact_rows(case, s)
        return {"key": torch.cat(got["k"]), "value": torch.cat(got["v"])}
    old, new = _lengths(case)
    got = _exact_rows({**case, "op": "read"}, s)
    h, d, g = case["hkv"], case["d"], case["hq"] // case["hkv"]
    out = torch.empty((int(new.sum()), case["hq"], d), dtype=torch.float64, device="cuda")
    at = 0
    for r in range(len(old)):
        n, k, v = int(new[r]), got["k"][r], got["v"][r]
        seen = (torch.arange(k.shape[0], device="cuda")[None, :]
                <= int(old[r]) + torch.arange(n, device="cuda")[:, None])
        q = s["q"][at:at + n].double()
        for a in range(case["hq"]):
            w = (q[:, a] @ k[:, a // g].T) / math.sqrt(d)
            w = torch.softmax(torch.where(seen, w, -math.inf), dim=-1)
            out[at:at + n, a] = w @ v[:, a // g]
        at += n
    return {"out": out}
