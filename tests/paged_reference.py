"""The paged entry cache and its attentions in numpy, 64 bits, from the format's definition (no code of
the library): entries are encoded and decoded value by value, attention is a plain softmax.

Bounds on the library's outputs (assert_attention).  A softmax weight p is rounded to 2^-8 of itself at
most (bf16, the RoPE dims; f16, the others: 2^-11).  Small ones are rounded no finer than an absolute
step: with Vmax the largest of an entry's 448 values, 2^-17 of the largest p Vmax of 32 tokens is allowed
to each of them; a chunk of 16 tokens shares its 32 with one other, so F = 32 * (sum over chunks of
max(p Vmax)) bounds the sum of these.  (f16's step is 2^-24 of the largest p Vmax of all tokens: less than
that for up to 4096 tokens; weights below 2^-126 of the largest vanish: less than that.)  A logit is a
512-term fp32 sum, off by at most delta = 512 * 2^-24 * scale * sum|q||k|, the exponential by 2^-22, which
move every weight by that relatively, and the denominator too.  bf16 outputs add their rounding, 2^-8 of
the value.  With A = sum p |v|:
    |out - ref| <= (2^-8 + 2 delta + 2^-21) A + 2^-17 F + (2^-8 |ref| for bf16 outputs)
    |lse - ref| <= delta + 2^-20 (1 + |ref|)        (fp32 sums of at most 2^17 terms, in pieces)
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
ENTRY = {"fp8": 576, "fp4": 368}


def bf16_bits(x):
    """float64 -> bf16 bits through float32, ties to even."""
    u = np.asarray(x, np.float32).view(np.uint32)
    out = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(np.asarray(x)), np.uint16(0x7FC0), out)


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


E4M3 = np.array([(-1.0 if c & 0x80 else 1.0) * ((c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else
                                                 (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10)) for c in range(256)])
E4M3[0x7F] = E4M3[0xFF] = np.nan


def e4m3_codes(x):
    """Nearest E4M3 code, ties to the even one, saturating at 448."""
    mags = E4M3[:0x7F]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(mags, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), 0x7F, c + np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def rotate(x, pos, base):
    """RoPE dims [64] turned at pos."""
    i = np.arange(32)
    a = pos * base ** (-i / 32.0)
    out = np.empty(64)
    out[0::2] = x[0::2] * np.cos(a) - x[1::2] * np.sin(a)
    out[1::2] = x[0::2] * np.sin(a) + x[1::2] * np.cos(a)
    return out


def fp4_group(x):
    """Codes (magnitude index, sign) [32] and the exponent byte of one group."""
    if np.isnan(x).any():
        return np.zeros(32, int), np.zeros(32, int), 255
    amax = np.abs(x).max()
    e = -126
    while e < 125 and amax > 6.0 * 2.0 ** e:
        e += 1
    v = np.minimum(np.abs(x) / 2.0 ** e, 6.0)
    d = np.abs(v[:, None] - GRID)
    best = d.min(1)
    # ties to the even index
    m = np.array([min((k for k in range(8) if d[i, k] == best[i]), key=lambda k: (k % 2, k)) for i in range(32)])
    return m, np.signbit(x).astype(int), e + 127


class Cache:
    """pages [n_pages, page_size, ...] as raw bytes, a page table and lengths, all numpy."""

    def __init__(self, pages, table, seq_len, page_size, fmt):
        self.pages, self.table, self.seq_len, self.P, self.fmt = pages, table, seq_len, page_size, fmt
        self.n_pages = pages.shape[0]

    def page_of(self, b, t):
        if t // self.P >= self.table.shape[1]:
            return -1
        pg = int(self.table[b, t // self.P])
        return pg if 0 <= pg < self.n_pages else -1

    def store(self, b, t, x):
        """x: 512 float64 values (RoPE dims as they go in)."""
        pg, r = self.page_of(b, t), t % self.P
        page = self.pages[pg]
        if self.fmt == "fp8":
            e = page[r * 576:(r + 1) * 576]
            e[:448] = e4m3_codes(x[:448])
            e[448:] = bf16_bits(x[448:]).view(np.uint8)
            return
        c, k = page[(r // 16) * 5888:(r // 16 + 1) * 5888], r % 16
        ex = []
        for g in range(14):
            m, s, eb = fp4_group(x[32 * g:32 * g + 32])
            ex.append(eb)
            if eb != 255:
                for w in range(4):
                    word = 0
                    for i in range(8):
                        word |= int(m[8 * w + i]) << (4 * i)
                        word |= int(s[8 * w + i]) << (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)
                    c[g * 256 + k * 16 + 4 * w:][:4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
            c[3584 + g * 16 + k] = eb
        c[3808 + k] = max([e for e in ex if e < 255], default=1)
        c[3824 + k] = 0
        c[3840 + 128 * k:3840 + 128 * k + 128] = bf16_bits(x[448:]).view(np.uint8)

    def value(self, b, t):
        """The 512 values of token t, or None where its page is no page."""
        pg, r = self.page_of(b, t), t % self.P
        if pg < 0:
            return None
        page = self.pages[pg]
        if self.fmt == "fp8":
            e = page[r * 576:(r + 1) * 576]
            return np.concatenate([E4M3[e[:448]], bf16_values(e[448:].copy().view(np.uint16))])
        c, k = page[(r // 16) * 5888:(r // 16 + 1) * 5888], r % 16
        out = np.empty(512)
        words = c[:3584].reshape(14, 16, 16)[:, k].copy().view(np.uint32).astype(np.int64)   # [14, 4]
        for i in range(8):
            mag = GRID[(words >> (4 * i)) & 7]
            neg = (words >> (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)) & 1
            out[:448].reshape(14, 4, 8)[:, :, i] = np.where(neg == 1, -mag, mag)
        ex = c[3584:3808].reshape(14, 16)[:, k].astype(np.float64)
        out[:448] = (out[:448].reshape(14, 32) * np.where(ex == 255, np.nan, 2.0 ** (ex - 127))[:, None]).ravel()
        out[448:] = bf16_values(c[3840 + 128 * k:3840 + 128 * k + 128].copy().view(np.uint16))
        return out

    def values(self, b, tokens):
        """[len, 512] values, and which of the tokens have a page."""
        v = [self.value(b, int(t)) for t in tokens]
        ok = np.array([x is not None for x in v], bool)
        return np.array([np.zeros(512) if x is None else x for x in v]).reshape(-1, 512), ok

    def append(self, x, n_new, start, base):
        """x [B, T, 512] float64; the library's whole-sequence rule."""
        B, T, _ = x.shape
        for b in range(B):
            s = int(self.seq_len[b] if start is None else start[b])
            n = int(T if n_new is None else n_new[b])
            if s < 0 or n < 0 or n > T or s + n > self.table.shape[1] * self.P:
                continue
            if any(self.page_of(b, t) < 0 for t in range(s, s + n)):
                continue
            for i in range(n):
                v = x[b, i].copy()
                if base:
                    v[448:] = rotate(v[448:], s + i, base)
                self.store(b, s + i, v)
            self.seq_len[b] = s + n


def visible(p, W, sinks):
    """The tokens that a query at position p sees."""
    if p < 0:
        return np.zeros(0, np.int64)
    t = np.arange(p + 1)
    return t if W is None else t[(t < sinks) | (t > p - W)]


def attention(cache, q, scale, W=None, sinks=0):
    """out [B, Q, H, 512], lse [B, Q, H], and the bounds' parts A (as out), delta and F (as lse)."""
    B, Q, H, _ = q.shape
    out, A = np.zeros((B, Q, H, 512)), np.zeros((B, Q, H, 512))
    lse, delta, F = np.full((B, Q, H), -np.inf), np.zeros((B, Q, H)), np.zeros((B, Q, H))
    for b in range(B):
        n = int(cache.seq_len[b])
        need = sorted(set(int(t) for j in range(Q) for t in visible(n - Q + j, W, sinks)))
        v, ok = cache.values(b, need)
        where = {t: i for i, t in enumerate(need)}
        for j in range(Q):
            see = np.array([t for t in visible(n - Q + j, W, sinks) if ok[where[int(t)]]], np.int64)
            at = np.array([where[int(t)] for t in see], np.int64)
            if not len(at):
                continue
            k = v[at]
            s = scale * (q[b, j] @ k.T)
            m = s.max(1, keepdims=True)
            w = np.exp(s - m)
            l = w.sum(1, keepdims=True)
            out[b, j], A[b, j] = w @ k / l, w @ np.abs(k) / l
            lse[b, j] = (m + np.log(l))[:, 0]
            pv = w / l * np.abs(k[:, :448]).max(1)
            F[b, j] = 32 * np.maximum.reduceat(pv, np.flatnonzero(np.diff(see // 16, prepend=-1)), axis=1).sum(1)
            delta[b, j] = (512 * 2.0 ** -24 * abs(scale) * (np.abs(q[b, j]) @ np.abs(k).T)).max(1)
    return out, lse, A, delta, F


def assert_attention(got, glse, ref, what=""):
    """got (bf16 or fp32 as float64, bf16 flagged by its dtype attribute) within the bounds above."""
    import torch
    out, lse, A, delta, F = ref
    bf = got.dtype == torch.bfloat16
    g, gl = got.double().cpu().numpy(), glse.double().cpu().numpy()
    tol = (2.0 ** -8 + 2 * delta[..., None] + 2.0 ** -21) * A + 2.0 ** -17 * F[..., None] + (2.0 ** -8 * np.abs(out) if bf else 0.0)
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} outputs off, worst {np.abs(g - out)[bad].max():.3g} "
                           f"(allowed {tol[bad][np.abs(g - out)[bad].argmax()]:.3g}) first at {np.argwhere(bad)[0]}")
    none = np.isinf(lse)
    assert np.array_equal(np.isneginf(gl), none), f"{what}: rows with no visible token differ"
    off = np.abs(gl[~none] - lse[~none])
    lim = (delta + 2.0 ** -20 * (1 + np.abs(lse)))[~none]
    assert np.all(off <= lim), f"{what}: lse off by {off.max():.3g}"
