"""A plain 64-bit implementation of the 4-bit key/value cache and its attention
(include/cider.h), by index formulas in numpy; shares nothing with the library.
Quantization decisions are in fp32, as the definition states them."""
import numpy as np

PAGE = 64


def block_bytes(D, gs):
    return 64 * D + 512 * (D // gs)


def to_f64(bits, dtype):
    """uint16 patterns of fp16 (0) / bf16 (1) as float64."""
    if dtype == 1:
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return bits.view(np.float16).astype(np.float64)


def to_bits(x, dtype):
    """float64 / float32 rounded to nearest even into uint16 patterns, through fp32."""
    f = np.asarray(x, np.float32)
    if dtype == 0:
        with np.errstate(over="ignore"):
            return f.astype(np.float16).view(np.uint16)
    u = np.ascontiguousarray(f).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(f), ((u >> 16) | 0x40).astype(np.uint16), r)


def quantize(x, gs):
    """x float64 [..., D] holding 16-bit values -> (u = code + 8 uint8 [..., D], s fp32 [..., D / gs])."""
    g = x.astype(np.float32).reshape(*x.shape[:-1], x.shape[-1] // gs, gs)
    s = np.abs(g).max(-1) / np.float32(7)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(g / s[..., None])
    q = np.where(s[..., None] == 0, 0, np.clip(q, -8, 7))
    return (q.astype(np.int64) + 8).astype(np.uint8).reshape(x.shape), s


def k_place(t, d, D):
    """(byte in the block, 0 for the low nibble) of K's element d of token t of the page."""
    j, m, e = (d // 8) % 4, d // 32, d % 8
    return 4 * ((t * 4 + j) * (D // 32) + m) + e // 2, e % 2


def v_place(t, d, D):
    B, b, j, i = t // 32, (t // 16) % 2, (t // 4) % 4, t % 4
    g, x, c = d // 64, (d // 16) % 4, d % 16
    n = 4 * b + i
    return 32 * D + 4 * ((((B * (D // 64) + g) * 4 + j) * 16 + c) * 4 + x) + n // 2, n % 2


class Cache:
    """uint8 [num_pages, kv_heads, block], the layout of include/cider.h."""

    def __init__(self, data, D, gs):
        self.data, self.D, self.gs = data, D, gs
        t, d = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
        self.places = [k_place(t, d, D), v_place(t, d, D)]

    def scales(self, which):
        """fp32 view [num_pages, kv_heads, D / gs, 64] of K's (0) or V's (1) scales."""
        n = 256 * (self.D // self.gs)
        at = 64 * self.D + which * n
        P, H, _ = self.data.shape
        return np.ascontiguousarray(self.data[:, :, at:at + n]).view(np.float32).reshape(P, H, -1, PAGE)

    def put(self, page, t, which, u, s):
        """Token t of a page: codes u [H, D], scales s [H, D / gs]."""
        byte, high = (x[t] for x in self.places[which])
        for h in range(u.shape[0]):
            for d in range(self.D):
                old = self.data[page, h, byte[d]]
                self.data[page, h, byte[d]] = ((old & 0x0F) | (u[h, d] << 4)) if high[d] else \
                    ((old & 0xF0) | u[h, d])
        n = 256 * (self.D // self.gs)
        for g in range(self.D // self.gs):
            at = 64 * self.D + which * n + 4 * (g * PAGE + t)
            self.data[page, :, at:at + 4] = np.ascontiguousarray(s[:, g:g + 1]).view(np.uint8).reshape(-1, 4)

    def values(self, which, pages):
        """float64 [H, 64 * len(pages), D] and the fp32 scales [H, 64 * len(pages), D]."""
        byte, high = self.places[which]
        u = (self.data[pages][:, :, byte] >> (4 * high)) & 15
        s = np.repeat(self.scales(which)[pages].transpose(0, 1, 3, 2), self.gs, -1).astype(np.float64)
        with np.errstate(invalid="ignore"):
            x = s * (u.astype(np.float64) - 8)
        return [y.transpose(1, 0, 2, 3).reshape(y.shape[1], -1, self.D) for y in (x, s)]


def fill(cache, pages, kv_lens, k, v):
    """Quantizes whole sequences k[b], v[b] float64 [kv, H, D] into the cache (vectorised over pages)."""
    D, gs = cache.D, cache.gs
    n = 256 * (D // gs)
    for b, kv in enumerate(kv_lens):
        for which, x in ((0, k[b]), (1, v[b])):
            u, s = quantize(x, gs)
            byte, high = cache.places[which]
            for first in range(0, kv, PAGE):
                cnt = min(PAGE, kv - first)
                page = pages[b][first // PAGE]
                for half in (0, 1):
                    mine = high[:cnt] == half
                    t, d = np.nonzero(mine)
                    vals = u[first:first + cnt].transpose(1, 0, 2)[:, t, d]
                    blk = cache.data[page]
                    keep = 0x0F if half else 0xF0
                    at = byte[t, d]
                    blk[:, at] = (blk[:, at] & keep) | (vals << 4 if half else vals)
                sc = s[first:first + cnt].transpose(1, 2, 0)  # H, groups, tokens
                for g in range(D // gs):
                    at = 64 * D + which * n + 4 * g * PAGE
                    cache.data[page, :, at:at + 4 * cnt] = np.ascontiguousarray(sc[:, g]).view(np.uint8).reshape(
                        sc.shape[0], -1)


def visible(p, have, window, sinks):
    t = np.arange(have)
    see = t <= p
    if window:
        see &= (t > p - window) | (t < sinks)
    return see


def attention(cache, pages, kv, q, G, scale, window, sinks):
    """One sequence: q float64 [n, HQ, D] -> (y, bound of the kernel's error without the output's rounding).

    The bound, with w_t = P_t / sum P and |v_t| the magnitudes of the values:
      2^-11 sum w |v|            the weights' rounding to fp16 (11 significant bits),
      2^-16 sum w 16 s_v         fp32 sums of products of codes 0 .. 15 and of the offset 8 (under 256
                                 sequential additions of 32-token products at these lengths),
      4 e sum w (|v| + 16 s_v)   scores off by e (twice: numerator and denominator, first order), where
                                 e = 2^-18 scale max_t sum |q| 16 s_k covers fp32 sums of at most 40
                                 sequential additions (2^-24 each, q's rounding far below) and exp2's 2^-22;
      2^-38 16 max s_v n / sum P fp16's smallest steps for weights under 2^-28 of the largest."""
    n, HQ, D = q.shape
    y, bound = np.zeros((n, HQ, D)), np.zeros((n, HQ, D))
    if kv == 0:
        return y, bound
    ids = list(pages[:-(-kv // PAGE)])
    (k, ks), (v, vs) = cache.values(0, ids), cache.values(1, ids)
    for i in range(n):
        see = np.nonzero(visible(kv - n + i, kv, window, sinks))[0]
        if not len(see):
            continue
        for h in range(HQ):
            kk, vv, kss, vss = (x[h // G][see] for x in (k, v, ks, vs))
            s = scale * (kk @ q[i, h])
            p = np.exp(s - s.max())
            w = p / p.sum()
            y[i, h] = w @ vv
            e = 2.0 ** -18 * scale * (kss @ np.abs(q[i, h])).max() * 16 + 2.0 ** -20
            a, a16 = w @ np.abs(vv), w @ (16 * vss)
            bound[i, h] = 2.0 ** -11 * a + 2.0 ** -16 * a16 + 4 * e * (a + a16) + \
                2.0 ** -38 * 16 * vss.max(0) * len(see) / p.sum()
    return y, bound
