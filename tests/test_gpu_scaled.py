"""Block-scaled FP8 pools on the GPU against a 64-bit restatement
(scaled_ref.py): the write byte for byte with its scale bytes, the read back
bit for bit, attention within a bound derived term by term, and runs of them
together."""

import numpy as np
import pytest
import torch

import paged_kv_attention_prepare_gb300 as pa
import scaled_ref as ref
from gpu_step import to_dev

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(autouse=True)
def clean_status():
    pa.pa_get_status()
    yield


def _host(t):
    return t.detach().cpu().numpy()


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _ok():
    assert pa.pa_get_status() == (pa.PA_OK, 0)


def _flagged():
    status, detail = pa.pa_get_status()
    assert status == pa.PA_ERR_DEVICE_CHECK
    return pa.check_bits(detail)


# ---------------------------------------------------------------------------
# Write
# ---------------------------------------------------------------------------

def _write(key, value, pools, bt, qsl, lens, **kw):
    """pa_cache_write_scaled on copies of the host pools; the four arrays after."""
    dev = [to_dev(a) for a in pools]
    pa.pa_cache_write_scaled(key, value, *dev, to_dev(bt), to_dev(qsl),
                             to_dev(np.asarray(lens, np.int32)), **kw)
    torch.cuda.synchronize()
    return [_host(a) for a in dev]


def _write_ref(key, value, pools, bt, qsl, lens):
    kc, vc, ks, vs = (a.copy() for a in pools)
    ref.write_one(ref.f64(key), kc, ks, bt, qsl, lens)
    ref.write_one(ref.f64(value), vc, vs, bt, qsl, lens)
    return kc, vc, ks, vs


def _nan(codes):
    """Codes with every NaN as 0x7f: a NaN's sign is not kept."""
    return np.where(codes & 0x7F == 0x7F, 0x7F, codes)


def _same(got, want):
    for name, a, b in zip(("key_cache", "value_cache", "k_scales", "v_scales"), got, want):
        if a.ndim == 4:
            a, b = _nan(a), _nan(b)
        np.testing.assert_array_equal(a, b, err_msg=name)


def _pools(rng, nb, hkv, d, **kw):
    kc, ks = ref.make_pools(rng, nb, hkv, d, **kw)
    vc, vs = ref.make_pools(rng, nb, hkv, d, **kw)
    return kc, vc, ks, vs


def _rows(rng, t, hkv, d, dtype, spread=3.0):
    """New rows whose size differs from token to token and head to head, so
    that some blocks keep their scale and some grow."""
    x = rng.standard_normal((t, hkv, d)) * 2.0 ** (spread * rng.standard_normal((t, hkv, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 64), (8, 128), (5, 128)])
def test_write_matches_reference(dtype, hkv, d):
    # every first slot 0 .. 15, one token to several blocks, a lone first token
    rng = np.random.default_rng(hkv * d)
    new = np.array([1] * 16 + [1, 2, 15, 16, 17, 33, 40, 5, 100])
    old = np.array(list(range(16)) + [0, 31, 1, 16, 8, 0, 7, 160, 3])
    lens = old + new
    bt, nb = ref.tables(rng, lens)
    pools = _pools(rng, nb, hkv, d, spread=6)
    qsl, t = _starts(new), int(new.sum())
    key, value = (_rows(rng, t, hkv, d, dtype) for _ in range(2))
    got = _write(key, value, pools, bt, qsl, lens)
    _ok()
    want = _write_ref(key, value, pools, bt, qsl, lens)
    _same(got, want)
    # the case is not empty: some first blocks grew and some did not
    first = bt[np.arange(len(new)), old // 16]
    held = old % 16 > 0
    grew = want[2][first] != pools[2][first]
    assert grew[held].any() and not grew[held].all()


@pytest.mark.parametrize("d", [64, 128])
def test_write_takes_views_of_a_fused_projection(d):
    rng = np.random.default_rng(d)
    hq, hkv, new, old = 6, 2, np.array([20, 1, 3]), np.array([5, 15, 0])
    t = int(new.sum())
    qkv = torch.from_numpy(rng.standard_normal((t, (hq + 2 * hkv) * d)).astype(np.float32))
    qkv = qkv.to(torch.bfloat16).cuda()
    key = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    value = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
    bt, nb = ref.tables(rng, old + new)
    pools = _pools(rng, nb, hkv, d)
    got = _write(key, value, pools, bt, _starts(new), old + new)
    _ok()
    _same(got, _write_ref(key, value, pools, bt, _starts(new), old + new))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_write_values_at_the_edges(dtype):
    # rows of zeros, of infinities, of NaN, of one large value, of the type's
    # smallest and largest values, and 448 * 2^e with its neighbours: each as a
    # block of its own and as a token that joins a block
    rng = np.random.default_rng(9)
    d, dt = 64, DT[dtype]
    info = torch.finfo(dt)
    base = rng.standard_normal(d)
    rows = []
    for fill in (0.0, -0.0, float("inf"), -float("inf"), float("nan"), info.max, info.min,
                 info.tiny, info.smallest_normal * info.eps, 448.0, 448.0 * (1 + info.eps),
                 448.0 / 2 ** 7, 464.0, 1e-3):
        for where in (slice(0, 1), slice(0, d), slice(d - 1, d)):
            x = base.copy()
            x[where] = fill
            rows.append(x)
    x = torch.from_numpy(np.stack(rows)[:, None, :]).to(dt).cuda()
    n = len(rows)
    new = np.ones(n, np.int64)
    for old in (0, 9):
        lens = np.full(n, old + 1)
        bt, nb = ref.tables(rng, lens)
        pools = _pools(rng, nb, 1, d, spread=8)
        # bytes outside the range that the write leaves: read as its nearest end
        pools[2][bt[0, 0]], pools[2][bt[1, 0]], pools[3][bt[2, 0]] = 0, 255, 70
        got = _write(x, x, pools, bt, _starts(new), lens)
        _ok()
        _same(got, _write_ref(x, x, pools, bt, _starts(new), lens))


def test_write_recodes_far_and_keeps_nan():
    # a held block whose exponent grows by 1, by 3 .. 12 (into E4M3's
    # subnormals and past them) and by 112 from end to end; NaN codes stay NaN
    rng = np.random.default_rng(11)
    d, grow = 64, [0, 1, 3, 5, 8, 10, 12, 16, 30, 112]
    n = len(grow)
    lens = np.full(n, 8)
    bt, nb = ref.tables(rng, lens)
    pools = _pools(rng, nb, 1, d)
    every = np.arange(256, dtype=np.uint8)                  # all codes, NaN among them
    x = np.zeros((n, 1, d))
    for r, up in enumerate(grow):
        for codes, scales in ((pools[0], pools[2]), (pools[1], pools[3])):
            codes[bt[r, 0], :4, 0] = every.reshape(4, d)
            scales[bt[r, 0], 0] = ref.E_MIN + ref.BIAS
        x[r, 0, 0] = 448.0 * 2.0 ** (ref.E_MIN + up)
    key = torch.from_numpy(x).to(torch.bfloat16).cuda()
    got = _write(key, key, pools, bt, _starts(np.ones(n, int)), lens)
    _ok()
    _same(got, _write_ref(key, key, pools, bt, _starts(np.ones(n, int)), lens))


def test_write_leaves_everything_else_as_it_was():
    # a padded batch: requests without tokens, tokens behind the last request;
    # slots behind the last new token, other blocks and other scales stay
    rng = np.random.default_rng(12)
    hkv, d = 2, 64
    new, old = np.array([3, 0, 1, 0, 0]), np.array([2, 40, 16, 0, 7])
    lens = old + new
    bt, nb = ref.tables(rng, lens, extra_blocks=20)
    pools = _pools(rng, nb, hkv, d, garbage=True)
    key, value = (_rows(rng, 4 + 6, hkv, d, "bf16") for _ in range(2))
    got = _write(key, value, pools, bt, _starts(new), lens)
    _ok()
    want = _write_ref(key, value, pools, bt, _starts(new), lens)
    _same(got, want)
    live = bt[0, 0]                              # the one block that held tokens
    for a, b, c in zip(got[:2], want[:2], pools[:2]):
        np.testing.assert_array_equal(a[live, 5:], c[live, 5:])
        rest = np.arange(nb) != live
        np.testing.assert_array_equal(a[rest], b[rest])
    # nothing to write at all
    none = _write(key[:0], value[:0], pools, bt, _starts(np.zeros(5, int)), lens)
    _same(none, pools)


def test_write_many_requests():
    # more requests than a thread block has threads
    rng = np.random.default_rng(13)
    n = 1500
    new, old = rng.integers(0, 4, n), rng.integers(0, 50, n)
    lens = old + new
    bt, nb = ref.tables(rng, lens)
    pools = _pools(rng, nb, 1, 64)
    key, value = (_rows(rng, int(new.sum()), 1, 64, "bf16") for _ in range(2))
    got = _write(key, value, pools, bt, _starts(new), lens)
    _ok()
    _same(got, _write_ref(key, value, pools, bt, _starts(new), lens))


def test_write_more_requests_than_the_plain_shared_memory_holds():
    rng = np.random.default_rng(31)
    n = 20_000
    new = (rng.random(n) < 0.1).astype(int)
    old = rng.integers(0, 20, n)
    lens = old + new
    bt, nb = ref.tables(rng, lens)
    pools = _pools(rng, nb, 1, 64)
    key, value = (_rows(rng, int(new.sum()), 1, 64, "fp16") for _ in range(2))
    got = _write(key, value, pools, bt, _starts(new), lens)
    _ok()
    _same(got, _write_ref(key, value, pools, bt, _starts(new), lens))


def test_write_starts_that_go_back_are_flagged():
    # requests 0 and 2 both take tokens 0 .. 19, request 1 would take -20
    rng = np.random.default_rng(32)
    lens = np.array([20, 5, 33])
    bt, nb = ref.tables(rng, lens)
    pools = _pools(rng, nb, 2, 64)
    key, value = (_rows(rng, 20, 2, 64, "bf16") for _ in range(2))
    got = _write(key, value, pools, bt, np.array([0, 20, 0, 20], np.int32), lens)
    assert _flagged() == {"seq_len"}
    want = pools
    for r in (0, 2):
        want = _write_ref(key, value, want, bt[r:r + 1], np.array([0, 20]), lens[r:r + 1])
    _same(got, want)


def test_write_bad_blocks_and_lengths_are_flagged_and_skipped():
    rng = np.random.default_rng(14)
    new, old = np.array([4, 4, 4, 4, 4]), np.array([0, 14, 30, 0, 3])
    lens = old + new
    bt, nb = ref.tables(rng, lens)
    pools = _pools(rng, nb, 2, 64)
    key, value = (_rows(rng, 20, 2, 64, "bf16") for _ in range(2))
    bad = bt.copy()
    bad[1, 1] = nb          # out of the pool
    bad[3, 0] = -1
    narrow = np.ascontiguousarray(bad[:, :2])    # request 2 needs a third block
    wrong = lens.copy()
    wrong[4] = 3                                 # shorter than its new tokens
    got = _write(key, value, pools, narrow, _starts(new), wrong)
    assert _flagged() == {"block_id", "logical_block", "seq_len"}
    want = [a.copy() for a in pools]
    for r, upto in ((0, None), (1, 16), (2, 32)):    # what is left to write
        hi = int(lens[r]) if upto is None else upto
        n = hi - int(old[r])
        for x, codes, scales in ((key, want[0], want[2]), (value, want[1], want[3])):
            ref.write_one(ref.f64(x)[4 * r:4 * r + n], codes, scales, bt[r:r + 1],
                          np.array([0, n]), [hi])
    _same(got, want)


def test_one_block_in_two_requests_stays_inside_it():
    # refused by contract, bounded all the same: only that block may change
    rng = np.random.default_rng(15)
    bt = np.array([[2], [2]], np.int32)
    pools = _pools(rng, 6, 2, 64)
    key, value = (_rows(rng, 2, 2, 64, "bf16") for _ in range(2))
    got = _write(key, value, pools, bt, _starts([1, 1]), [3, 3])
    _ok()
    rest = np.arange(6) != 2
    for a, b in zip(got, pools):
        np.testing.assert_array_equal(a[rest], b[rest])


def test_tokens_one_by_one_leave_the_scale_of_their_largest():
    # a block filled one token at a time ends with the same scale as in one
    # call, and each code within one extra rounding in the subnormal range
    rng = np.random.default_rng(16)
    hkv, d, n = 2, 128, 16
    pools = _pools(rng, 4, hkv, d)
    key, value = (_rows(rng, n, hkv, d, "bf16", spread=2) for _ in range(2))
    bt = np.array([[1]], np.int32)
    whole = _write(key, value, pools, bt, _starts([n]), [n])
    step = [to_dev(a) for a in pools]
    for i in range(n):
        pa.pa_cache_write_scaled(key[i:i + 1], value[i:i + 1], *step, to_dev(bt),
                                 to_dev(_starts([1])), to_dev(np.array([i + 1], np.int32)))
    _ok()
    for a, b in zip(step[2:], whole[2:]):
        np.testing.assert_array_equal(_host(a), b)
    for a, b in zip(step[:2], whole[:2]):
        assert np.abs(ref.decode(_host(a)[1]) - ref.decode(b[1])).max() <= 2.0 ** -9


# ---------------------------------------------------------------------------
# Read
# ---------------------------------------------------------------------------

def _read(pools, bt, first, rows, dtype, out_rows=None, fill=7.0, **kw):
    n = int(np.sum(rows)) if out_rows is None else out_rows
    hkv, d = pools[0].shape[2:]
    ko = torch.full((n, hkv, d), fill, dtype=dtype, device="cuda")
    vo = torch.full_like(ko, -fill)
    pa.pa_cache_read(*pools[:2], to_dev(bt), to_dev(np.asarray(first, np.int32)),
                     to_dev(_starts(rows)), ko, vo, **kw)
    torch.cuda.synchronize()
    return ko, vo


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 64), (8, 128), (7, 128)])
def test_read_matches_reference(dtype, hkv, d):
    rng = np.random.default_rng(100 + hkv * d)
    first = np.array([0, 0, 5, 16, 31, 0, 0, 0, 100, 3])
    rows = np.array([1, 0, 11, 16, 1, 0, 0, 0, 333, 37])
    bt, nb = ref.tables(rng, first + rows)
    pools = _pools(rng, nb, hkv, d, spread=9)
    pools[2][bt[2, 0]], pools[3][bt[3, 1]] = 0, 255        # read as the ends of the range
    dev = [to_dev(a) for a in pools]
    ko, vo = _read(dev, bt, first, rows, DT[dtype], k_scales=dev[2], v_scales=dev[3])
    _ok()
    for got, codes, scales in ((ko, pools[0], pools[2]), (vo, pools[1], pools[3])):
        want = np.concatenate([ref.context(codes, scales, bt[r], first[r] + rows[r])[first[r]:]
                               for r in range(len(rows))])
        want = torch.from_numpy(want).to(DT[dtype])        # one rounding, to nearest even
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8", "fp8_unscaled"])
@pytest.mark.parametrize("hkv,d,bs", [(2, 64, 16), (3, 40, 16), (1, 8, 4), (8, 128, 32)])
def test_read_of_other_pools(kind, hkv, d, bs):
    # pools of one scale, and 16-bit pools, of any block size and head_dim
    rng = np.random.default_rng(7)
    dt = DT.get(kind, torch.bfloat16)
    first, rows = np.array([3, 0, 17]), np.array([50, 1, 6])
    need = -(-(first + rows) // bs)
    nb = int(need.sum()) + 2
    perm = rng.permutation(nb)
    bt = np.full((3, int(need.max())), -1, np.int32)
    at = 0
    for r in range(3):
        bt[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
    shape = (nb, bs, hkv, d)
    kw = {}
    if kind in DT:
        pools = [torch.from_numpy(rng.standard_normal(shape)).to(dt).cuda() for _ in range(2)]
        vals = pools
    else:
        codes = [ref.encode(rng.standard_normal(shape) * 50) for _ in range(2)]
        pools = [to_dev(c) for c in codes]
        sc = (1.0, 1.0)
        if kind == "fp8":
            sc = (0.3, 1.7)
            kw = {n: torch.tensor([s], dtype=torch.float32, device="cuda")
                  for n, s in zip(("k_scale", "v_scale"), sc)}
        vals = [(torch.from_numpy(ref.decode(c)).float() * np.float32(s)).to(dt).cuda()
                for c, s in zip(codes, sc)]
    ko, vo = _read(pools, bt, first, rows, dt, **kw)
    _ok()
    slots = np.concatenate([bt[r][p // bs] * bs + p % bs
                            for r in range(3) for p in [first[r] + np.arange(rows[r])]])
    at = to_dev(slots.astype(np.int64))
    for got, v in ((ko, vals[0]), (vo, vals[1])):
        assert torch.equal(got, v.reshape(nb * bs, hkv, d)[at])


def test_read_many_requests_and_rows_behind_them():
    # most requests ask for nothing; the outputs have room for more rows, which
    # stay as they were
    rng = np.random.default_rng(8)
    n = 3000
    rows = np.where(rng.random(n) < 0.03, rng.integers(1, 40, n), 0)
    first = rng.integers(0, 20, n)
    bt, nb = ref.tables(rng, np.where(rows > 0, first + rows, 0))
    pools = _pools(rng, nb, 2, 64)
    dev = [to_dev(a) for a in pools]
    total = int(rows.sum())
    ko, vo = _read(dev, bt, first, rows, torch.bfloat16, out_rows=total + 13,
                   k_scales=dev[2], v_scales=dev[3])
    _ok()
    want = np.concatenate([ref.context(pools[0], pools[2], bt[r], first[r] + rows[r])[first[r]:]
                           for r in range(n) if rows[r]])
    assert torch.equal(ko[:total].cpu(), torch.from_numpy(want).bfloat16())
    assert (ko[total:] == 7).all() and (vo[total:] == -7).all()


def test_read_bad_rows_are_flagged_and_left():
    rng = np.random.default_rng(9)
    first, rows = np.array([0, 0, 0, -4]), np.array([20, 20, 40, 8])
    bt, nb = ref.tables(rng, first.clip(0) + rows)
    pools = _pools(rng, nb, 1, 64)
    dev = [to_dev(a) for a in pools]
    bad = np.ascontiguousarray(bt[:, :2])                  # request 2 is wider than that
    bad[1, 0] = nb
    ko, vo = _read(dev, bad, first, rows, torch.bfloat16, k_scales=dev[2], v_scales=dev[3])
    assert _flagged() == {"block_id", "logical_block", "seq_len"}
    left = np.zeros(88, bool)
    left[20:36] = left[40 + 32:80] = left[80:84] = True
    assert (ko.cpu()[torch.from_numpy(left)] == 7).all()
    want = ref.context(pools[1], pools[3], bt[0], 20)
    assert torch.equal(vo[:20].cpu(), torch.from_numpy(want).bfloat16())
    # more rows asked for than there is room: those that fit are read
    ko, vo = _read(dev, bt, np.zeros(4, int), rows, torch.bfloat16, out_rows=25,
                   k_scales=dev[2], v_scales=dev[3])
    assert _flagged() == {"token_count"}
    want = ref.context(pools[0], pools[2], bt[0], 20)
    assert torch.equal(ko[:20].cpu(), torch.from_numpy(want).bfloat16())


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def _attend(q, pools, bt, qsl, lens, scale, workspace="full", max_q=None, max_seq=None, **kw):
    t, hq, d = q.shape
    hkv = pools[0].shape[2]
    n = np.diff(qsl)
    max_q = int(n.max(initial=1)) if max_q is None else max_q
    max_seq = int(np.max(lens, initial=1)) if max_seq is None else max_seq
    ws = None
    if workspace is not None:
        size = pa.pa_attention_workspace_size(len(lens), t, max_q, max_seq, hq, hkv, d) \
            if workspace == "full" else workspace
        # contents need no initialisation: all NaN patterns
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    pa.pa_attention_scaled(q, *pools, to_dev(bt), to_dev(np.asarray(qsl, np.int32)),
                           to_dev(np.asarray(lens, np.int32)), max_q, max_seq, scale, out, ws, **kw)
    torch.cuda.synchronize()
    return out


def _case(seed, new, old, hq, hkv, d, dtype, spread=2, v_spread=None):
    rng = np.random.default_rng(seed)
    new, old = np.asarray(new), np.asarray(old)
    lens = old + new
    bt, nb = ref.tables(rng, lens, width_extra=1)
    kc, ks = ref.make_pools(rng, nb, hkv, d, spread=spread)
    vc, vs = ref.make_pools(rng, nb, hkv, d, spread=spread if v_spread is None else v_spread)
    pools = kc, vc, ks, vs
    # blocks that no request reads, and slots behind a context, hold anything
    used = np.zeros((nb, 16), bool)
    for r, n in enumerate(lens):
        for p in range(int(n)):
            used[bt[r, p // 16], p % 16] = True
    for i in (0, 1):
        pools[i][~used] = 0x7F                                        # NaN
        pools[2 + i][~used.any(1)] = rng.integers(0, 256)
    t = int(new.sum())
    q = rng.standard_normal((t, hq, d))
    q[np.abs(q) < 2.0 ** -14] = 0        # f16 holds every q of either type exactly
    q = torch.from_numpy(q.astype(np.float32)).to(DT[dtype]).cuda()
    return q, pools, bt, _starts(new), lens


def _check(case, scale=None, **kw):
    q, pools, bt, qsl, lens = case
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out = _attend(q, [to_dev(a) for a in pools], bt, qsl, lens, scale, **kw)
    _ok()
    want = ref.attention(ref.f64(q), *pools, bt, qsl, lens, scale)
    ref.check_attention(ref.f64(out), *want, q.dtype)
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("g", [1, 3, 4, 7, 8, 12])
def test_attention_single_tokens(d, dtype, g):
    # contexts of one token, of block and partition edges, and odd ones
    old = np.array([0, 1, 14, 15, 16, 17, 63, 200, 511, 512, 1023, 1024, 1500, 2047, 2500])
    _check(_case(d + g, np.ones(len(old), int), old, 2 * g, 2, d, dtype))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("g", [1, 4, 7])
def test_attention_short_requests(d, dtype, g):
    new = np.array([2, 16, 5, 1, 8, 16, 3])
    old = np.array([0, 0, 11, 700, 1020, 1100, 30])
    _check(_case(d * g, new, old, 3 * g, 3, d, dtype))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("g", [1, 4, 5, 16])
def test_attention_chunks(d, dtype, g):
    # prompt chunks only: the tensor-core kernel, ragged last tiles
    new = np.array([17, 200, 129, 300])
    old = np.array([0, 0, 350, 77])
    _check(_case(3 * d + g, new, old, 2 * g, 2, d, dtype))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_seq", [None, 4000])
def test_attention_mixed_batch(d, max_seq):
    # chunks beside short requests and single tokens: on the tensor-core kernel
    # alone, or (contexts that may be long) on both kernels side by side
    new = np.array([1, 260, 1, 4, 40, 1, 16, 1])
    old = np.array([900, 130, 0, 15, 0, 1300, 64, 33])
    case = _case(d, new, old, 8, 2, d, "bf16")
    full = _check(case, max_seq=max_seq)
    # any workspace is right: none, the counters alone, room for few partials
    for ws in (None, 256, 4096, 200_000):
        _check(case, workspace=ws, max_seq=max_seq)
    again = _check(case, max_seq=max_seq)
    assert torch.equal(full, again)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,new", [(8, (1, 2)), (3, (4, 6)), (5, (2, 5)), (16, (1, 1))])
def test_attention_items_of_many_rows(d, g, new):
    # short requests of 9 rows and more on average: items of 16 rows, some of
    # their tiles empty, contexts of several partitions and of none
    rng = np.random.default_rng(d + g)
    old = np.array([0, 0, 3, 700, 1030, 2050, 4500, 15, 2047])
    new = rng.integers(new[0], new[1], len(old), endpoint=True)
    case = _case(d * g, new, old, 2 * g, 2, d, "bf16")
    full = _check(case)
    assert torch.equal(full, _check(case))
    for ws in (None, 256, 60_000):
        _check(case, workspace=ws)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_many_short_requests_of_many_rows(d, dtype):
    # 30 rows a request and enough requests to fill the GPU: the tensor-core
    # kernel alone, single tokens included
    rng = np.random.default_rng(d)
    r = 48
    new, old = rng.integers(1, 9, r), rng.integers(0, 300, r)
    new[:3], old[:3] = 1, [0, 500, 127]
    case = _case(d, new, old, 32, 4, d, dtype)
    _check(case)
    _check(case, workspace=None)
    # ... which then checks the lengths too
    q, pools, bt, qsl, lens = case
    bad = lens.copy()
    bad[5], bad[7] = 100_000, 0
    out = _attend(q, [to_dev(a) for a in pools], bt, qsl, bad, 0.1, max_seq=600)
    assert _flagged() == {"seq_len"}
    rows = np.ones(q.shape[0], bool)
    for i in (5, 7):
        rows[qsl[i]:qsl[i + 1]] = False
        assert torch.isnan(out[qsl[i]:qsl[i + 1]]).all()      # left as they were
    want = ref.attention(ref.f64(q), *pools, bt, qsl, lens, 0.1)
    ref.check_attention(ref.f64(out), *want, q.dtype, rows=rows)


@pytest.mark.parametrize("r", [60, 256, 257])
def test_attention_contexts_in_classes_of_length(r):
    # the tensor-core kernel takes long contexts first: lengths on both sides of
    # the classes' borders at 400 keys, and more requests than it does that for
    rng = np.random.default_rng(r)
    new = rng.integers(4, 7, r)
    lens = rng.choice([7, 96, 97, 98, 198, 199, 299, 300, 399, 400], r)
    lens[:2] = 400, 7
    out = _check(_case(35, new, lens - new, 32, 4, 64, "bf16"), max_seq=400)
    assert not torch.isnan(out).any()


def test_attention_one_workspace_for_calls_of_all_sizes():
    # calls that use the workspace's counters and calls that do not, in turn on
    # one stream, with nothing cleared between them
    cases = [_case(1, [1, 2], [3, 40], 4, 2, 64, "bf16"),
             _case(2, [1] * 40, list(range(1000, 1400, 10)), 16, 4, 64, "bf16"),
             _case(3, [200, 1], [10, 900], 8, 2, 64, "bf16"),
             _case(4, [3] * 60, [30] * 60, 32, 4, 64, "bf16")]
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for i in (0, 1, 2, 3, 0, 2, 1, 0, 3):
        q, pools, bt, qsl, lens = cases[i]
        out = torch.full_like(q, float("nan"))
        pa.pa_attention_scaled(q, *[to_dev(a) for a in pools], to_dev(bt), to_dev(qsl),
                               to_dev(lens.astype(np.int32)), int(np.diff(qsl).max()),
                               int(lens.max()), 0.125, out, ws)
        got.append((i, out))
    _ok()
    for i, out in got:
        q, pools, bt, qsl, lens = cases[i]
        want = ref.attention(ref.f64(q), *pools, bt, qsl, lens, 0.125)
        ref.check_attention(ref.f64(out), *want, q.dtype)


@pytest.mark.parametrize("g", [2, 130])
def test_attention_on_the_split_kernel_alone(g):
    # a scale that is not positive, and more heads a group than a tile's rows,
    # keep long chunks on the split-K kernel
    case = _case(g, [40, 1], [20, 300], g, 1, 64, "bf16")
    _check(case, scale=-0.125 if g == 2 else 0.125)
    _check(case, scale=0.0)


@pytest.mark.parametrize("kind", ["tokens", "chunk"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread,v_spread", [(6, 2), (1, 12), (3, 30)])
def test_attention_scales_far_apart(kind, d, spread, v_spread):
    # blocks' exponents differ by up to 2 * spread: near one-hot scores, and
    # weights times V's scales that span far more than f16
    new, old = ([1, 1, 3], [1400, 90, 640]) if kind == "tokens" else ([150, 33], [300, 0])
    _check(_case(spread + d, new, old, 4, 2, d, "bf16", spread=spread, v_spread=v_spread))


@pytest.mark.parametrize("kind", ["tokens", "chunk"])
def test_attention_v_scales_at_both_ends(kind):
    # Half of the blocks hold V near 2^56, half near 2^-56 (or zeros with the
    # smallest scale, as written); keys equal, so the weights are too
    new, old = ([1, 2], [2000, 300]) if kind == "tokens" else ([100], [400])
    q, pools, bt, qsl, lens = _case(5, new, old, 4, 2, 64, "bf16", spread=0)
    rng = np.random.default_rng(6)
    nb = pools[0].shape[0]
    pools[3][:] = np.where(rng.random((nb, 1)) < 0.5, pa.SCALE_MIN, pa.SCALE_MAX)
    zero = rng.random(nb) < 0.3
    pools[1][zero & (pools[3][:, 0] == pa.SCALE_MIN)] &= 0x80
    _check((q, pools, bt, qsl, lens))
    # one far block only: contexts whose large block weighs almost nothing
    pools[3][:] = pa.SCALE_MIN
    pools[3][bt[0, 3]] = pa.SCALE_MAX
    _check((q, pools, bt, qsl, lens))


def test_attention_shared_blocks():
    # requests that share whole partitions of blocks, with their scales
    rng = np.random.default_rng(3)
    for d in (64, 128):
        case = _case(d, np.ones(9, int), rng.integers(4200, 4400, 9), 8, 2, d, "bf16", spread=4)
        q, pools, bt, qsl, lens = case
        bt[:, :256] = bt[0, :256]                            # a common prefix of 4096 tokens
        a = _check(case, shared_blocks=True)
        b = _check(case)
        assert torch.isfinite(a).all() and torch.isfinite(b).all()


def test_attention_equals_one_scale_per_pool():
    # every byte the same: the cached values of a pool with that scale
    rng = np.random.default_rng(4)
    q, pools, bt, qsl, lens = _case(8, [1, 120, 7], [500, 60, 200], 8, 2, 128, "bf16")
    pools[2][:], pools[3][:] = 125, 121
    dev = [to_dev(a) for a in pools]
    a = _attend(q, dev, bt, qsl, lens, 0.1)
    b = torch.empty_like(a)
    one = lambda s: torch.tensor([s], dtype=torch.float32, device="cuda")  # noqa: E731
    ws = torch.empty(pa.pa_attention_workspace_size(3, q.shape[0], 120, 560, 8, 2, 128),
                     dtype=torch.uint8, device="cuda")
    pa.pa_attention(q, dev[0], dev[1], to_dev(bt), to_dev(qsl), to_dev(lens.astype(np.int32)), 120,
                    560, 0.1, b, ws, k_scale=one(2.0 ** -2), v_scale=one(2.0 ** -6))
    _ok()
    want = ref.attention(ref.f64(q), *pools, bt, qsl, lens, 0.1)
    for x in (a, b):
        ref.check_attention(ref.f64(x), *want, q.dtype)


def test_attention_padding_rows_are_left():
    q, pools, bt, qsl, lens = _case(9, [1, 30], [40, 100], 4, 2, 64, "fp16")
    t = q.shape[0]
    wide = torch.cat([q, torch.full((5, 4, 64), float("nan"), dtype=q.dtype, device="cuda")])
    qsl3 = np.concatenate([qsl, [t, t]]).astype(np.int32)       # two empty requests
    bt4 = np.concatenate([bt, np.full((2, bt.shape[1]), -1, np.int32)])
    lens4 = np.concatenate([lens, [0, 0]])
    out = _attend(wide, [to_dev(a) for a in pools], bt4, qsl3, lens4, 0.125, max_q=64, max_seq=500)
    _ok()
    assert torch.isnan(out[t:]).all()
    want = ref.attention(ref.f64(q), *pools, bt, qsl, lens, 0.125)
    ref.check_attention(ref.f64(out[:t]), *want, q.dtype)


@pytest.mark.parametrize("max_seq", [600, 8000, 20_000])
@pytest.mark.parametrize("max_q", [1, 8, 100])
def test_attention_bounds_above_what_the_batch_holds(max_q, max_seq):
    # one call laid out for more: the bounds choose the kernel, not the result
    for new, old in (([1], [500]), ([1, 1, 1], [3, 40, 515])):
        q, pools, bt, qsl, lens = _case(33, new, old, 8, 2, 64, "bf16")
        t, extra = q.shape[0], 100 - q.shape[0]
        wide = torch.cat([q, torch.full((extra, 8, 64), float("nan"), dtype=q.dtype, device="cuda")])
        out = _attend(wide, [to_dev(a) for a in pools], bt, qsl, lens, 0.125, max_q=max_q,
                      max_seq=max_seq)
        _ok()
        assert torch.isnan(out[t:]).all()
        want = ref.attention(ref.f64(q), *pools, bt, qsl, lens, 0.125)
        ref.check_attention(ref.f64(out[:t]), *want, q.dtype)


@pytest.mark.parametrize("max_seq", [4096, 4097])
def test_attention_many_rows_with_contexts_that_may_be_long(max_seq):
    # both sides of the length up to which the tensor-core kernel takes them
    rng = np.random.default_rng(34)
    new, old = rng.integers(4, 9, 48), rng.integers(0, 300, 48)
    _check(_case(34, new, old, 32, 4, 64, "bf16"), max_seq=max_seq)


def test_attention_bad_blocks_and_lengths_are_flagged():
    q, pools, bt, qsl, lens = _case(10, [1, 1, 40, 1], [40, 100, 30, 20], 4, 2, 64, "bf16")
    nb = pools[0].shape[0]
    bt = bt.copy()
    bt[1, 2], bt[2, 1] = nb + 5, -7
    long = lens.copy()
    long[3] = 10_000                                           # wider than the table
    pools = [np.where(a == 0x7F, 0, a) if a.ndim == 4 else a for a in pools]   # no NaN anywhere
    out = _attend(q, [to_dev(a) for a in pools], bt, qsl, long, 0.125, max_seq=20_000)
    assert _flagged() == {"block_id", "seq_len"}
    want = ref.attention(ref.f64(q[:1]), *pools, bt[:1], qsl[:2], lens[:1], 0.125)
    ref.check_attention(ref.f64(out[:1]), *want, q.dtype)


# ---------------------------------------------------------------------------
# Together, as an engine uses them
# ---------------------------------------------------------------------------

class _Engine:
    """Two requests stepped together over one set of pools, with a float64
    shadow of the cache."""

    def __init__(self, hq, hkv, d, dtype, nb=40):
        self.rng = np.random.default_rng(21)
        self.shape = (hq, hkv, d)
        self.dt = DT[dtype]
        self.host = list(_pools(self.rng, nb, hkv, d, garbage=True))
        self.dev = [to_dev(a) for a in self.host]
        self.bt = np.full((3, 8), -1, np.int32)
        self.perm = list(self.rng.permutation(nb))
        self.lens = np.zeros(3, np.int64)

    def step(self, new):
        new = np.asarray(new)
        hq, hkv, d = self.shape
        for r in range(3):
            while (self.bt[r] >= 0).sum() * 16 < self.lens[r] + new[r]:
                self.bt[r, (self.bt[r] >= 0).sum()] = self.perm.pop()
        self.lens += new
        t, qsl = int(new.sum()), _starts(new)
        mk = lambda h: torch.from_numpy(  # noqa: E731
            (self.rng.standard_normal((t, h, d)) * 2.0 ** self.rng.standard_normal((t, h, 1)))
            .astype(np.float32)).to(self.dt).cuda()
        q, key, value = mk(hq), mk(hkv), mk(hkv)
        bt, sl = to_dev(self.bt), to_dev(self.lens.astype(np.int32))
        pa.pa_cache_write_scaled(key, value, *self.dev, bt, to_dev(qsl), sl)
        ref.write_one(ref.f64(key), self.host[0], self.host[2], self.bt, qsl, self.lens)
        ref.write_one(ref.f64(value), self.host[1], self.host[3], self.bt, qsl, self.lens)
        out = _attend(q, self.dev, self.bt, qsl, self.lens, d ** -0.5)
        rows = self.lens
        ko, vo = _read(self.dev, self.bt, np.zeros(3), rows, self.dt, k_scales=self.dev[2],
                       v_scales=self.dev[3])
        _ok()
        for i, got in ((0, ko), (1, vo)):
            want = np.concatenate([ref.context(self.host[i], self.host[2 + i], self.bt[r], rows[r])
                                   for r in range(3)])
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(self.dt))
        want = ref.attention(ref.f64(q), *self.host, self.bt, qsl, self.lens, d ** -0.5)
        ref.check_attention(ref.f64(out), *want, self.dt)

    def fork(self, src, dst):
        """Request dst becomes a copy-on-write fork of src: whole blocks are
        shared, a partial last block is copied with its scales."""
        n = int(self.lens[src])
        self.lens[dst] = n
        self.bt[dst] = self.bt[src]
        if n % 16:
            new = int(self.perm.pop())
            old = int(self.bt[src, n // 16])
            pa.pa_copy_blocks_scaled(*self.dev, to_dev(np.array([old], np.int32)),
                                     to_dev(np.array([new], np.int32)))
            for a in self.host:
                a[new] = a[old]
            self.bt[dst, n // 16] = new


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_steps_together(d, dtype):
    e = _Engine(4, 2, d, dtype)
    e.step([37, 5, 0])       # prompts
    e.step([1, 1, 0])        # decode
    e.fork(0, 2)             # beam search: request 2 forks request 0 mid-block
    for new in ([1, 1, 1], [1, 3, 1], [1, 0, 2], [20, 1, 1], [1, 1, 30]):
        e.step(new)


def test_copy_blocks_scaled_copies_codes_and_scales():
    rng = np.random.default_rng(22)
    pools = _pools(rng, 50, 3, 64, garbage=True)
    dev = [to_dev(a) for a in pools]
    src, dst = np.array([3, 9, 3, -1, 4], np.int32), np.array([40, 41, 42, 43, 50], np.int32)
    pa.pa_copy_blocks_scaled(*dev, to_dev(src), to_dev(dst))
    assert _flagged() == {"block_id"}                          # the last two pairs
    for a, b in zip(dev, pools):
        b = b.copy()
        b[dst[:3]] = b[src[:3]]
        np.testing.assert_array_equal(_host(a), b)


def test_captured_step_replays_with_new_inputs():
    # write, attention and read back as one graph, replayed on other lengths,
    # tables and values in the same buffers; on a stream of its own
    rng = np.random.default_rng(23)
    hq, hkv, d, r, nb, mb = 8, 2, 64, 4, 120, 30
    i32 = dict(dtype=torch.int32, device="cuda")
    bt, qsl, sl = torch.zeros(r, mb, **i32), torch.zeros(r + 1, **i32), torch.zeros(r, **i32)
    first, starts = torch.zeros(r, **i32), torch.zeros(r + 1, **i32)
    tcap, ncap, bound = 90, 1500, 4000           # bound on seq_lens: both kernels side by side
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, out = torch.zeros(tcap, hq, d, **bf), torch.zeros(tcap, hq, d, **bf)
    key, value = torch.zeros(tcap, hkv, d, **bf), torch.zeros(tcap, hkv, d, **bf)
    ko, vo = torch.zeros(ncap, hkv, d, **bf), torch.zeros(ncap, hkv, d, **bf)
    pools = _pools(rng, nb, hkv, d)
    dev = [to_dev(a) for a in pools]
    ws = torch.empty(pa.pa_attention_workspace_size(r, tcap, tcap, bound, hq, hkv, d),
                     dtype=torch.uint8, device="cuda")

    def calls():
        pa.pa_cache_write_scaled(key, value, *dev, bt, qsl, sl)
        pa.pa_attention_scaled(q, *dev, bt, qsl, sl, tcap, bound, 0.125, out, ws)
        pa.pa_cache_read(dev[0], dev[1], bt, first, starts, ko, vo, k_scales=dev[2],
                         v_scales=dev[3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()                                  # nothing to do yet: no tokens, no rows
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls()
    host = [a.copy() for a in pools]
    for new, old in (([1, 1, 40, 3], [300, 15, 70, 0]), ([0, 1, 1, 1], [10, 64, 33, 400]),
                     ([17, 17, 17, 17], [0, 0, 0, 16])):
        new, old = np.array(new), np.array(old)
        lens, t = old + new, int(new.sum())
        perm = rng.permutation(nb)
        tab, at = np.full((r, mb), -1, np.int32), 0
        for i in range(r):
            n = -(-int(lens[i]) // 16)
            tab[i, :n] = perm[at:at + n]
            at += n
        qq, kk, vv = (_rows(rng, t, h, d, "bf16", 1.0) for h in (hq, hkv, hkv))
        bt.copy_(to_dev(tab))
        qsl.copy_(to_dev(_starts(new)))
        sl.copy_(to_dev(lens.astype(np.int32)))
        starts.copy_(to_dev(_starts(lens)))
        q[:t], key[:t], value[:t] = qq, kk, vv
        out.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        _ok()
        qs = _starts(new)
        ref.write_one(ref.f64(kk), host[0], host[2], tab, qs, lens)
        ref.write_one(ref.f64(vv), host[1], host[3], tab, qs, lens)
        for a, b in zip(dev, host):
            np.testing.assert_array_equal(_host(a), b)
        want = ref.attention(ref.f64(qq), *host, tab, qs, lens, 0.125)
        ref.check_attention(ref.f64(out[:t]), *want, torch.bfloat16)
        assert (out[t:] == 7).all()
        rows = np.concatenate([ref.context(host[1], host[3], tab[i], lens[i]) for i in range(r)])
        assert torch.equal(vo[:len(rows)].cpu(), torch.from_numpy(rows).bfloat16())


def test_pools_past_32_bit_offsets():
    # blocks whose codes lie past 2^31 and 2^32 bytes of a pool
    rng = np.random.default_rng(24)
    hq, hkv, d = 8, 8, 128
    nb = (1 << 32) // (16 * hkv * d) + 40
    hi = [nb - 1, nb // 2 + 3, nb - 7, 0, nb - 20, nb // 2 - 1, nb - 3, nb // 2 + 9]
    bt = np.array([hi[:4], hi[4:]], np.int32)
    new, old = np.array([1, 25]), np.array([60, 30])
    lens, qsl = old + new, _starts([1, 25])
    small = _pools(rng, 8, hkv, d)                             # block i is hi[i]
    local = np.arange(8, dtype=np.int32).reshape(2, 4)
    dev = [torch.zeros((nb, 16, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    dev += [torch.zeros((nb, hkv), dtype=torch.uint8, device="cuda") for _ in range(2)]
    at = to_dev(np.array(hi, np.int64))
    for a, b in zip(dev, small):
        a[at] = to_dev(b)
    key, value = (_rows(rng, 26, hkv, d, "bf16", 1.0) for _ in range(2))
    q = _rows(rng, 26, hq, d, "bf16", 0.5)
    pa.pa_cache_write_scaled(key, value, *dev, to_dev(bt), to_dev(qsl),
                             to_dev(lens.astype(np.int32)))
    out = _attend(q, dev, bt, qsl, lens, 0.1)
    ko, vo = _read(dev, bt, np.zeros(2), lens, torch.bfloat16, k_scales=dev[2], v_scales=dev[3])
    _ok()
    ref.write_one(ref.f64(key), small[0], small[2], local, qsl, lens)
    ref.write_one(ref.f64(value), small[1], small[3], local, qsl, lens)
    for a, b in zip(dev, small):
        np.testing.assert_array_equal(_host(a[at]), b)
    want = ref.attention(ref.f64(q), *small, local, qsl, lens, 0.1)
    ref.check_attention(ref.f64(out), *want, q.dtype)
    rows = np.concatenate([ref.context(small[0], small[2], local[i], lens[i]) for i in range(2)])
    assert torch.equal(ko.cpu(), torch.from_numpy(rows).bfloat16())
    del dev
    torch.cuda.empty_cache()


def test_calls_on_a_given_stream():
    # the stream argument: an object, a handle, and the current one
    rng = np.random.default_rng(25)
    pools = _pools(rng, 10, 2, 64)
    bt, qsl, sl = np.array([[4, 7]], np.int32), _starts([20]), np.array([20], np.int32)
    key, value, q = (_rows(rng, 20, h, 64, "bf16", 1.0) for h in (2, 2, 4))
    args = [to_dev(a) for a in (bt, qsl, sl, np.zeros(1, np.int32))]
    want = None
    for how in ("object", "handle", "current"):
        dev = [to_dev(a) for a in pools]
        out = torch.full_like(q, float("nan"))
        ko, vo = torch.empty_like(key), torch.empty_like(value)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        kw = {"stream": side if how == "object" else side.cuda_stream if how == "handle" else None}
        with torch.cuda.stream(side if how == "current" else torch.cuda.current_stream()):
            pa.pa_cache_write_scaled(key, value, *dev, *args[:3], **kw)
            pa.pa_attention_scaled(q, *dev, *args[:3], 20, 20, 0.125, out, **kw)
            pa.pa_cache_read(dev[0], dev[1], args[0], args[3], args[1], ko, vo, k_scales=dev[2],
                             v_scales=dev[3], **kw)
        side.synchronize()
        _ok()
        got = [*dev, out, ko, vo]
        if want is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = got


def test_binding_refuses_tensors_that_do_not_fit():
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    i32, bf = torch.int32, torch.bfloat16
    pools = [z(4, 16, 2, 64), z(4, 16, 2, 64), z(4, 2), z(4, 2)]
    bt, qsl, sl = z(1, 2, dt=i32), z(2, dt=i32), z(1, dt=i32)
    x, q = z(3, 2, 64, dt=bf), z(3, 4, 64, dt=bf)

    def write(**kw):
        a = dict(key=x, value=x, kc=pools[0], vc=pools[1], ks=pools[2], vs=pools[3], bt=bt, qsl=qsl,
                 sl=sl)
        a.update(kw)
        pa.pa_cache_write_scaled(*a.values())

    for kw in (dict(key=x.float()), dict(value=x.half()), dict(kc=pools[0].to(bf)),
               dict(ks=pools[2].int()), dict(bt=bt.long()), dict(qsl=qsl.long()), dict(key=None)):
        with pytest.raises(TypeError):
            write(**kw)
    for kw in (dict(key=x[:, :1]), dict(value=x[:2]), dict(key=x.transpose(0, 1)),
               dict(vc=pools[1][:3]), dict(ks=z(4, 3)), dict(vs=z(2, 2)), dict(qsl=z(3, dt=i32)),
               dict(bt=z(2, 2, dt=i32)), dict(sl=z(2, dt=i32)), dict(kc=pools[0][:, ::2]),
               dict(key=z(3, 2, 128, dt=bf)[:, :, ::2])):
        with pytest.raises(ValueError):
            write(**kw)

    def attend(**kw):
        a = dict(q=q, kc=pools[0], vc=pools[1], ks=pools[2], vs=pools[3], bt=bt, qsl=qsl, sl=sl,
                 max_q=3, max_seq=16, scale=1.0, out=torch.empty_like(q))
        a.update(kw)
        pa.pa_attention_scaled(*a.values())

    for kw in (dict(out=q.float()), dict(q=q.float(), out=q.float()), dict(max_q="3"),
               dict(scale=None), dict(kc=pools[0].to(bf), vc=pools[1].to(bf))):
        with pytest.raises(TypeError):
            attend(**kw)
    for kw in (dict(kc=q, vc=q), dict(out=q[:2]), dict(q=q[:, :, :32], out=q[:, :, :32]), dict(max_seq=1 << 40),
               dict(q=q.transpose(0, 1))):
        with pytest.raises(ValueError):
            attend(**kw)
    with pytest.raises(pa.PAError) as e:
        attend(q=z(3, 3, 64, dt=bf), out=z(3, 3, 64, dt=bf))          # 3 heads over 2
    assert e.value.status == pa.PA_ERR_UNSUPPORTED
    with pytest.raises(pa.PAError) as e:                              # tables beside a pool scale
        pa.pa_cache_read(*pools[:2], bt, sl, qsl, x, x.clone(), k_scales=pools[2],
                         v_scales=pools[3], k_scale=torch.ones(1, device="cuda"))
    assert e.value.status == pa.PA_ERR_INVALID
    with pytest.raises(TypeError):                                    # one table alone
        pa.pa_cache_read(*pools[:2], bt, sl, qsl, x, x.clone(), k_scales=pools[2])
    assert pa.pa_get_status() == (pa.PA_OK, 0)
