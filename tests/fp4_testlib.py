"""The microscaled 4-bit cache in plain numpy (float64 attention): what the
tests compare the kernels with.  Shares no code with the library."""
from __future__ import annotations

import numpy as np

BS = 16
PER_TENSOR, PER_HEAD = 0, 1
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 non-negative finite E4M3 values, by code
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def bf16_to_f32(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def to_bf16(x):
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def nearest(table, a):
    """Index of the value of the ascending table nearest to a >= 0, ties to the
    even index, the last one for anything above."""
    mid = (table[1:] + table[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")    # a tie goes down ...
    hi = np.searchsorted(mid, a, side="right")   # ... or up
    return np.where(lo % 2 == 0, lo, hi)


def quantize(bits, scale):
    """bf16 rows [N][hkv][dh] -> (codes [N][hkv][dh], scale codes [N][hkv][dh/16])."""
    n, hkv, dh = bits.shape
    x = bf16_to_f32(bits).reshape(n, hkv, dh // 16, 16)
    s = np.broadcast_to(np.asarray(scale, np.float32), (hkv,)).reshape(1, hkv, 1)
    with np.errstate(all="ignore"):
        nan = np.isnan(x).any(-1)
        top = np.float32(3.3895313892515355e38)  # the largest finite bf16
        amax = np.minimum(np.where(np.isnan(x), 0, np.abs(x)).max(-1), top).astype(np.float32)
        sb = nearest(E4M3, (amax / (s * np.float32(6))).astype(np.float32))
        r = (E4M3[sb].astype(np.float32) * s).astype(np.float32)
        live = (r > 0) & ~nan
        a = (np.abs(x) / np.where(live, r, 1)[..., None]).astype(np.float32)
        c = nearest(E2M1, np.where(np.isnan(a), 0, a)) | np.where(np.signbit(x), 8, 0)
    c = np.where(live[..., None], c, 0)
    return c.reshape(n, hkv, dh).astype(np.uint8), np.where(nan, 0x7F, sb).astype(np.uint8)


def new_cache(num_blocks, hkv, dh, fill=0):
    return np.full((num_blocks, hkv, 9 * dh), fill, np.uint8)


def write(bits, slots, cache, scale):
    dh = bits.shape[-1]
    codes, sb = quantize(bits, scale)
    both = codes[..., 0::2] | (codes[..., 1::2] << 4)
    for t, slot in enumerate(slots):
        if 0 <= slot < cache.shape[0] * BS:
            b, r = divmod(int(slot), BS)
            cache[b, :, r * (dh // 2):(r + 1) * (dh // 2)] = both[t]
            o = 8 * dh + r * (dh // 16)
            cache[b, :, o:o + dh // 16] = sb[t]


def unit_values(cache):
    """code * block scale of every row, exact: [blocks][hkv][16][dh]."""
    nb, hkv, pg = cache.shape
    dh = pg // 9
    c = cache[..., :8 * dh].reshape(nb, hkv, BS, dh // 2)
    c = np.stack((c & 15, c >> 4), -1).reshape(nb, hkv, BS, dh // 16, 16)
    v = np.where(c & 8, -E2M1[c & 7], E2M1[c & 7])
    sb = cache[..., 8 * dh:].reshape(nb, hkv, BS, dh // 16)
    s = np.where((sb & 0x7F) == 0x7F, np.nan, E4M3[np.minimum(sb & 0x7F, 126)] * np.where(sb & 0x80, -1, 1))
    with np.errstate(invalid="ignore"):
        return (v * s[..., None]).reshape(nb, hkv, BS, dh)


def read(cache, scale, table, starts, cu, rows, fill=0):
    """bf16 bits of the gathered rows [rows][hkv][dh]."""
    nb, hkv, pg = cache.shape
    out = np.full((rows, hkv, pg // 9), fill, np.uint16)
    s = np.broadcast_to(np.asarray(scale, np.float32), (hkv,)).reshape(hkv, 1)
    for b in range(len(cu) - 1):
        for j in range(cu[b + 1] - cu[b]):
            pos = j + (int(starts[b]) if starts is not None else 0)
            blk = int(table[b, pos // BS]) if 0 <= pos < table.shape[1] * BS else -1
            if 0 <= blk < nb:
                u = unit_values(cache[blk:blk + 1])[0, :, pos % BS].astype(np.float32)
                out[cu[b] + j] = to_bf16((u * s).astype(np.float32))
            else:
                out[cu[b] + j] = 0
    return out


def attention(q, K, V, ks, vs, table, lens, cu_q, window, sinks):
    """Float64 attention of each sequence's last queries over the cache.  q: bf16
    bits [rows][hq][dh]; K, V: pages.  Returns (out, tol): tol bounds how far a
    kernel's bf16 output may be off,

      2^-8 |out|                   the rounding to bf16
      2^-11 A                      one f16 per probability, A = sum p |V|
      2^-32 B                      B = sum |V|: a weight 2^(x - m) reaches f16
        times 2^7, where the least step is 2^-24, so it is off by at most half of
        2^-31 when it lies below f16's normal values; m is at most the row's
        largest logit, so the weights' sum is at least 1
      (2^-17 S + 2^-16) A          S = sum |q_i K_i| / sqrt(dh) at its largest: a
        logit's binary32 sum over at most 8 matrix steps is off by at most
        2^-18 S, and enters the numerator and the denominator; the base-2
        exponentials and the running rescales add a few 2^-22 each

    NaN where a visible token's values are."""
    rows, hq, dh = q.shape
    nb, hkv, _ = K.shape
    G = hq // hkv
    Ku, Vu = unit_values(K), unit_values(V)
    ks = np.broadcast_to(np.asarray(ks, np.float64), (hkv,))
    vs = np.broadcast_to(np.asarray(vs, np.float64), (hkv,))
    out = np.zeros((rows, hq, dh))
    tol = np.zeros((rows, hq, dh))
    for b in range(len(lens)):
        n, L = int(cu_q[b + 1] - cu_q[b]), int(lens[b])
        if L < n or L > table.shape[1] * BS:
            continue
        t = np.arange(L)
        blk = table[b, t // BS].astype(np.int64)
        good = (blk >= 0) & (blk < nb)
        blk = np.where(good, blk, 0)
        qv = bf16_to_f32(q[cu_q[b]:cu_q[b + 1]]).astype(np.float64)
        for j in range(n):
            pos = L - n + j
            seen = good & (t <= pos)
            if window:
                seen &= (t > pos - window) | (t < sinks)
            if not seen.any():
                continue
            w = np.nonzero(seen)[0]
            for g in range(hkv):
                k = Ku[blk[w], g, w % BS] * ks[g]
                v = Vu[blk[w], g, w % BS] * vs[g]
                qq = qv[j, g * G:(g + 1) * G]
                x = qq @ k.T / np.sqrt(dh)
                S = (np.abs(qq) @ np.abs(k).T / np.sqrt(dh)).max(-1)
                p = np.exp(x - np.max(x, -1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o = p @ v
                A = p @ np.abs(v)
                r = slice(g * G, (g + 1) * G)
                out[cu_q[b] + j, r] = o
                tol[cu_q[b] + j, r] = 2.0 ** -8 * np.abs(o) + A * (2.0 ** -11 + 2.0 ** -17 * S[:, None] + 2.0 ** -16) \
                    + 2.0 ** -32 * np.abs(v).sum(0)
    return out, tol


def check(got, want, tol, what=""):
    """got: bf16 bits.  NaN has to meet NaN."""
    got = bf16_to_f32(got).astype(np.float64)
    assert got.shape == want.shape
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    err = np.abs(got - want)[~nan]
    bad = ~(err <= tol[~nan] + 1e-30)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} values off, worst "
                           f"{np.max(err[bad] / (tol[~nan][bad] + 1e-30)):.3g} times the tolerance, by {err[bad].max():.3g}")


class Batch:
    """A batch's tokens and pages: lens tokens per sequence, pages in a shuffled
    pool with some to spare, caches first filled with `fill` bytes (0x7F: every
    scale NaN), so that what lies behind a sequence is poison."""

    def __init__(self, seed, lens, hq, hkv, dh, per_head=True, fill=0x7F, extra=3, amp=1.0):
        r = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        self.hq, self.hkv, self.dh = hq, hkv, dh
        pages = (self.lens + BS - 1) // BS
        self.nb = int(pages.sum()) + extra
        perm = r.permutation(self.nb).astype(np.int32)
        self.table = np.full((len(lens), max(1, int(pages.max()))), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        std = amp * np.exp(r.uniform(-1, 1, hkv))
        N = int(self.lens.sum())
        self.k = to_bf16(r.standard_normal((N, hkv, dh)) * std[None, :, None])
        self.v = to_bf16(r.standard_normal((N, hkv, dh)) * std[None, ::-1, None])
        self.ks = (std * 4.5 / 2688).astype(np.float32)
        self.vs = (std[::-1] * 4.5 / 2688).astype(np.float32)
        if not per_head:
            self.ks, self.vs = self.ks.max(keepdims=True), self.vs.max(keepdims=True)
        self.gran = PER_HEAD if per_head else PER_TENSOR
        seq = np.repeat(np.arange(len(lens)), self.lens)
        pos = np.concatenate([np.arange(n) for n in self.lens]) if N else np.zeros(0, np.int64)
        self.slots = self.table[seq, pos // BS].astype(np.int64) * BS + pos % BS
        self.fill = fill
        self.rng = r

    def pages(self):
        K, V = new_cache(self.nb, self.hkv, self.dh, self.fill), new_cache(self.nb, self.hkv, self.dh, self.fill)
        write(self.k, self.slots, K, self.ks)
        write(self.v, self.slots, V, self.vs)
        return K, V

    def queries(self, counts):
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        return to_bf16(self.rng.standard_normal((int(cu[-1]), self.hq, self.dh)) * 1.5), cu
