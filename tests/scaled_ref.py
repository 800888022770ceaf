"""Plain 64-bit restatement of the block-scaled FP8 cache, for the tests: the
write with its scales, the read back, and attention with the size of each
term that its error bound needs."""

from __future__ import annotations

import numpy as np
import torch

E_MIN, E_MAX, BIAS = -56, 56, 127
BS = 16

_c = np.arange(127)
# the values of codes 0x00 .. 0x7e, ascending
POSITIVE = np.where(_c >> 3 == 0, (_c & 7) * 2.0 ** -9,
                    (8 + (_c & 7)) * 2.0 ** ((_c >> 3) - 10.0))
_MID = (POSITIVE[1:] + POSITIVE[:-1]) / 2
TABLE = np.concatenate([POSITIVE, [np.nan], -POSITIVE, [np.nan]])


def decode(codes):
    return TABLE[np.asarray(codes, np.uint8)]


def encode(x):
    """Nearest E4M3 codes of float64 x, ties to the even code, saturating;
    NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    up = np.searchsorted(_MID, a)                     # on a midpoint: the lower code
    on = (up < _MID.size) & (_MID[np.minimum(up, _MID.size - 1)] == a)
    up = up + (on & (up % 2 == 1))
    codes = up | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7F, codes).astype(np.uint8)


def exponent(x):
    """The exponent a block of new elements x (any shape) takes."""
    a = np.abs(x[np.isfinite(x)])
    top = float(a.max(initial=0.0))
    for e in range(E_MIN, E_MAX + 1):
        if top <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def scale_exp(byte):
    """The exponent readers take from a scale byte."""
    return int(np.clip(int(byte) - BIAS, E_MIN, E_MAX))


def f64(t):
    """A torch tensor's values as a float64 array."""
    return t.detach().cpu().double().numpy()


def write_one(x, codes, scales, bt, qsl, lens):
    """One of K and V: x float64 [T, H, D] into codes uint8 [NB, 16, H, D] and
    scales uint8 [NB, H], in place."""
    for r in range(len(lens)):
        n, length = int(qsl[r + 1]) - int(qsl[r]), int(lens[r])
        for b in range((length - n) // BS, -(-length // BS) if n else 0):
            lo, hi = max(length - n, b * BS), min(length, b * BS + BS)
            phys, off, t0 = int(bt[r][b]), lo % BS, int(qsl[r]) + lo - (length - n)
            new = x[t0:t0 + hi - lo]
            for h in range(codes.shape[2]):
                e = exponent(new[:, h])
                if off:
                    e_old = scale_exp(scales[phys, h])
                    e = max(e, e_old)
                    if e > e_old:
                        codes[phys, :off, h] = encode(decode(codes[phys, :off, h]) * 2.0 ** (e_old - e))
                codes[phys, off:off + hi - lo, h] = encode(new[:, h] * 2.0 ** -e)
                scales[phys, h] = e + BIAS


def block_values(codes, scales, blocks):
    """float64 values [len(blocks) * 16, H, D] of the listed blocks."""
    e = np.vectorize(scale_exp, otypes=[np.float64])(scales[blocks])
    v = decode(codes[blocks]) * 2.0 ** e[:, None, :, None]
    return v.reshape(-1, *v.shape[2:])


def context(codes, scales, table_row, length):
    blocks = np.asarray(table_row[: -(-int(length) // BS)], np.int64)
    return block_values(codes, scales, blocks)[: int(length)]


def attention(q, kc, vc, ks, vs, bt, qsl, lens, scale):
    """float64 [T, Hq, D] q over the pools.  Returns (out, mean, size, keys,
    vmax): the result; each element's weighted mean of |v|; each (token,
    head)'s largest scale * sum |q k|; the number of keys it sees; and the
    largest |v| of its context, the last three [T, Hq]."""
    t, hq, d = q.shape
    out, mean = np.full(q.shape, np.nan), np.zeros(q.shape)
    size, keys, vmax = (np.zeros((t, hq)) for _ in range(3))
    g = hq // kc.shape[2]
    for r in range(len(lens)):
        n, length = int(qsl[r + 1]) - int(qsl[r]), int(lens[r])
        if n == 0:
            continue
        k, v = context(kc, ks, bt[r], length), context(vc, vs, bt[r], length)
        rows = slice(int(qsl[r]), int(qsl[r + 1]))
        last = length - n + np.arange(n)
        hidden = np.arange(length)[None] > last[:, None]
        for h in range(hq):
            kh, vh = k[:, h // g], v[:, h // g]
            s = np.where(hidden, -np.inf, (q[rows, h] @ kh.T) * scale)
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[rows, h] = w @ vh
            mean[rows, h] = w @ np.abs(vh)
            size[rows, h] = np.where(hidden, 0, (np.abs(q[rows, h]) @ np.abs(kh).T) * scale).max(1)
            keys[rows, h] = last + 1
            vmax[rows, h] = np.abs(vh).max()
    return out, mean, size, keys, vmax


def attention_bound(ref, mean, size, keys, vmax, dtype):
    """How far a kernel's output may be from `ref`, element by element.

    - the output's own rounding, half a step: eps / 2 * |out|, and half the
      smallest subnormal of an fp16 output (2^-25);
    - the weights in f16: 2^-11 of each, so 2^-11 * mean|v|; weights under
      f16's normal range by at most 2^-25 of the heaviest, over `keys` keys of
      at most vmax;
    - float32 scores: the D products are summed in D / 16 matrix steps that
      each align and truncate to float32 (8 steps of 2^-22 of sum |q k|), then
      two multiply-adds and 2^x (2^-22 each): a relative error of each weight
      of at most 2^-18 * size + 2^-19, in the sum of the weights too, so
      twice that of mean|v|;
    - float32 sums over keys: sequential chains of at most keys / 4 additions
      with 2^-24 each, in O and in the sum: keys * 2^-25 of mean|v|."""
    half = torch.finfo(dtype).eps / 2
    rel = 2.0 ** -11 + 2 * (2.0 ** -18 * size + 2.0 ** -19) + keys * 2.0 ** -25
    return (half * np.abs(ref) * (1 + 2.0 ** -8) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
            + mean * rel[..., None] + (keys * vmax * 2.0 ** -25)[..., None])


def check_attention(got, ref, mean, size, keys, vmax, dtype, rows=None):
    tol = attention_bound(ref, mean, size, keys, vmax, dtype)
    err = np.abs(got - ref)
    if rows is not None:
        err, tol = err[rows], tol[rows]
    assert np.isfinite(got if rows is None else got[rows]).all()
    bad = np.argwhere(err > tol)
    assert bad.size == 0, (f"{len(bad)} of {err.size} past the bound; worst "
                           f"{(err / tol).max():.2f} of it; first {tuple(bad[0])}")
    return float((err / tol).max())


def make_pools(rng, nb, hkv, d, spread=2, garbage=False):
    """Random pools: codes, and scale bytes whose exponents lie within +-spread
    of -7 (values near 1).  With ``garbage``, any byte may be anything."""
    shape = (nb, BS, hkv, d)
    if garbage:
        codes = rng.integers(0, 256, shape).astype(np.uint8)
        return codes, rng.integers(0, 256, (nb, hkv)).astype(np.uint8)
    codes = encode(rng.standard_normal(shape) * 100.0)
    e = rng.integers(-7 - spread, -7 + spread, size=(nb, hkv), endpoint=True)
    return codes, (np.clip(e, E_MIN, E_MAX) + BIAS).astype(np.uint8)


def tables(rng, lens, extra_blocks=3, width_extra=0):
    """Random disjoint block tables for contexts of the given lengths; -1
    behind each request's last block.  Returns (table, num_blocks)."""
    need = [-(-int(x) // BS) for x in lens]
    nb = sum(need) + extra_blocks
    perm = rng.permutation(nb)
    bt = np.full((len(lens), max(need + [1]) + width_extra), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        bt[r, :n] = perm[at:at + n]
        at += n
    return bt, nb
