"""The paged-cache operators, as they are measured: the cases, their inputs, their plain form in
elementary torch operations, and the same outputs from the definition in 64 bits.

The operators work on a paged cache of 512-d entries (one shared KV head: an entry is both key and
value; dims 0..447 in 8 or 4 bits, the 64 RoPE dims 448..511 in bf16):

  append        new bf16 tokens -> (RoPE dims rotated at the token's position) -> entries in pages
  read          entries in pages -> bf16 tokens
  window        attention of the newest Q tokens of each sequence over a sliding window plus a few
                first tokens that stay visible
  full          the same over every token of the sequence
  step          append, then full: a decode step with Q draft tokens

Two entry formats.  fp8: 448 E4M3 bytes, then 64 bf16 (576 B per token, tokens of a page in order).
fp4: 368 B per token, kept in chunks of 16 tokens of a page (5888 B):
  bytes    0..3583   [14 groups of 32 dims][16 tokens][16 B] E2M1 codes; a 32-bit word holds 8 dims:
                     dim i's magnitude code in bits 4i..4i+2, its sign in bit 8i+7 (i < 4) or 8(i-4)+3
  bytes 3584..3807   [14 groups][16 tokens] UE8M0 exponents: group scale 2^(byte - 127), the smallest
                     power of two with max|x| <= 6 scale
  bytes 3808..3823   [16 tokens] the largest of the token's 14 exponents; bytes 3824..3839 zero
  bytes 3840..5887   [16 tokens][64] bf16 RoPE dims
"""
import math
import random

import numpy as np
import torch

own = False

D, NOPE, ROPE, GROUPS = 512, 448, 64, 14
BYTES = {"fp8": 576, "fp4": 368}
CHUNK, CHUNK_BYTES = 16, 5888
SCALE = 1.0 / math.sqrt(512.0)
ROPE_BASE = 10000.0
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- the cases ------------------------------------------------------------------------------------
def listed():
    return [
        # one new token for each of 32 sequences: the append of every decode step
        dict(name="append_fp8_decode", op="append", fmt="fp8", B=32, T=1, n=131072, page=64, lens="full"),
        # a prefill chunk, sequences of differing lengths padded to 4096, written and read back in 4 bits
        dict(name="append_fp4_chunk", op="append", fmt="fp4", B=8, T=4096, n=131072, page=64, lens="ragged"),
        # a few tokens of a few sequences read back: a draft's context, an odd count
        dict(name="read_fp8_few", op="read", fmt="fp8", B=4, T=37, n=4096, page=16, lens="full"),
        # a whole 128K-token sequence read back, e.g. to compress it again
        dict(name="read_fp4_128k", op="read", fmt="fp4", B=1, T=131072, n=131072, page=128, lens="full"),
        # one decode token of 8 sequences at 1M tokens, window 128: latency
        dict(name="window_fp8_decode", op="window", fmt="fp8", B=8, Q=1, H=16, W=128, S=4, n=1048576, page=64, lens="full"),
        # a large decode batch with a wider window
        dict(name="window_fp4_batch", op="window", fmt="fp4", B=256, Q=1, H=16, W=1024, S=16, n=32768, page=32, lens="ragged"),
        # 4 draft tokens of 32 sequences, lengths from nothing to 4096, some shorter than the window
        dict(name="window_fp8_drafts", op="window", fmt="fp8", B=32, Q=4, H=16, W=512, S=4, n=4096, page=64, lens="short"),
        # 64 heads on the one entry stream, a long window
        dict(name="window_fp4_heads64", op="window", fmt="fp4", B=16, Q=1, H=64, W=4096, S=128, n=65536, page=64, lens="full"),
        # one sequence of 1M tokens in 4 bits
        dict(name="full_fp4_1m", op="full", fmt="fp4", B=1, Q=1, H=16, n=1048576, page=64, lens="full"),
        # 32 sequences of very unlike lengths, up to 128K tokens
        dict(name="full_fp4_ragged", op="full", fmt="fp4", B=32, Q=1, H=16, n=131072, page=64, lens="ragged"),
        # 8 sequences of 64K tokens in 8 bits
        dict(name="full_fp8_64k", op="full", fmt="fp8", B=8, Q=1, H=16, n=65536, page=64, lens="full"),
        # a decode step with 4 draft tokens: the last accepted length, 4 tokens appended there, attended
        dict(name="step_fp4_drafts", op="step", fmt="fp4", B=8, Q=4, H=16, n=32768, page=128, lens="full"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "window", "window", "full", "full", "step"])
    c = dict(op=op, fmt=rng.choice(["fp8", "fp4"]), page=rng.choice([16, 32, 48, 64, 128, 256]),
             lens=rng.choice(["full", "ragged", "short"]))
    if op in ("append", "read"):
        c["B"] = _log_int(rng, 1, 64)
        c["T"] = _log_int(rng, 1, max(1, 131072 // c["B"] // (4 if op == "append" else 1)))
        c["n"] = max(_log_int(rng, 64, 131072), c["T"] + 1)
        return c
    c["Q"] = rng.choice([1, 1, 1, 2, 3, 4, 8])
    c["H"] = rng.choice([16, 16, 16, 1, 5, 8, 24, 32, 64, 128])
    rows = c["Q"] * -(-c["H"] // 16)
    if op == "window":
        c["B"] = _log_int(rng, 1, max(1, 256 // rows))
        c["W"] = _log_int(rng, 1, max(2, min(4096, 262144 // (c["B"] * rows))))
        c["S"] = rng.choice([0, 1, 4, 4, 16, 100, 128])
        c["n"] = _log_int(rng, 1, 1048576)
    else:
        c["B"] = _log_int(rng, 1, max(1, 64 // rows))
        c["n"] = _log_int(rng, 1, max(64, 1048576 // (c["B"] * rows)))
    return c


def _lengths(c):
    """The sequences' lengths, from the case alone: all n; log-uniform up to n; or from 0 on."""
    r = random.Random("%s %s %s %s" % (c["op"], c["B"], c["n"], c["lens"]))
    n = c["n"]
    if c["lens"] == "full":
        return [n] * c["B"]
    if c["lens"] == "ragged":
        return [_log_int(r, max(1, n // 64), n) for _ in range(c["B"])]
    return [r.choice([0, 1, r.randint(0, n), r.randint(0, n), n]) for _ in range(c["B"])]


def _spans(c):
    """Per sequence: (length, new tokens or tokens read, where those begin)."""
    out = []
    for i, n in enumerate(_lengths(c)):
        if c["op"] == "append":      # up to T tokens that end at n
            k = min(n, c["T"] if c["lens"] == "full" else max(0, c["T"] - (i * c["T"]) // (2 * c["B"])))
            out.append((n, k, n - k))
        elif c["op"] == "read":      # T tokens that end at n; places past the end read as zeros
            out.append((n, min(n, c["T"]), max(0, n - c["T"])))
        elif c["op"] == "step":
            k = min(n, c["Q"])
            out.append((n, k, n - k))
        else:
            out.append((n, 0, n))
    return out


def _visible(c):
    """Per sequence the tokens that any of its queries sees: (first tokens [0, s), the rest [lo, n))."""
    out = []
    for n, _, start in _spans(c):
        if c["op"] in ("append", "read"):
            out.append((0, start, n))
        elif c["op"] == "window":
            lo = max(0, n - c["Q"] + 1 - c["W"])
            out.append((min(c["S"], lo), lo, n))
        else:
            out.append((0, 0, n))
    return out


def work(c):
    e, spans = BYTES[c["fmt"]], _spans(c)
    tokens = sum(k for _, k, _ in spans)
    if c["op"] == "append":
        # bf16 tokens in, entries out; the fp4 case also reads them back
        back = (e + 2 * D) * tokens if c["fmt"] == "fp4" else 0
        return {"bytes": (2 * D + e) * tokens + back + 12 * c["B"], "flops": 6 * ROPE * tokens}
    if c["op"] == "read":
        return {"bytes": e * tokens + 2 * D * c["B"] * c["T"], "flops": 0}
    seen = [s + n - lo for s, lo, n in _visible(c)]
    io = c["B"] * c["Q"] * c["H"] * (2 * D + 2 * D + 4)
    new = (2 * D + e) * tokens if c["op"] == "step" else 0
    pairs = 0
    for n, _, _ in spans:
        for j in range(c["Q"]):
            t = n - c["Q"] + 1 + j
            if t > 0:
                pairs += min(t, c["W"] + min(c["S"], max(0, t - c["W"]))) if c["op"] == "window" else t
    return {"bytes": e * sum(seen) + io + new, "flops": 4 * D * c["H"] * pairs}


# ---- the inputs -----------------------------------------------------------------------------------
def _encode_fp4(x):
    """fp32 [N, 512] -> fp4 codes as [N, 14, 4] 32-bit words, exponents [N, 14], RoPE bf16 [N, 64]."""
    g = x[:, :NOPE].reshape(-1, GROUPS, 32)
    m, e = torch.frexp(g.abs().amax(-1))
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(-126, 125)
    a = torch.ldexp(g.abs(), -e[..., None])
    code = (a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int()
    neg = torch.signbit(g).int()
    i = torch.arange(8, device=x.device, dtype=torch.int32)
    sign_bit = torch.where(i < 4, 8 * i + 7, 8 * (i - 4) + 3)
    w = (code.reshape(-1, GROUPS, 4, 8).long() << (4 * i).long()) | (neg.reshape(-1, GROUPS, 4, 8).long() << sign_bit.long())
    w = w.sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int(), (e + 127).to(torch.uint8), x[:, NOPE:].to(torch.bfloat16)


def _tokens(g, n):
    """Raw tokens as the path meets them: N(0,1) dims, token magnitudes spread by about 1.6 times."""
    x = torch.randn(n, D, generator=g, device="cuda")
    return (x * torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))).to(torch.bfloat16)


def _fill(pages, fmt, first, x):
    """Entries of x in the pages' tokens first, first + 1, ... (counted over all pages; a multiple of 16)."""
    n = x.shape[0]
    if fmt == "fp8":
        p = pages.view(-1, 576)[first:first + n]
        p[:, :NOPE] = x[:, :NOPE].float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        p[:, NOPE:] = x[:, NOPE:].contiguous().view(torch.uint8)
        return
    w, e, r = _encode_fp4(x.float())
    p = pages.view(-1, CHUNK_BYTES)[first // CHUNK:(first + n) // CHUNK]
    k = n // CHUNK
    p[:, :3584] = w.view(k, CHUNK, GROUPS, 4).transpose(1, 2).contiguous().view(torch.uint8).view(k, 3584)
    e = e.view(k, CHUNK, GROUPS)
    p[:, 3584:3808] = e.transpose(1, 2).reshape(k, 224)
    p[:, 3808:3824] = e.amax(-1)
    p[:, 3824:3840] = 0
    p[:, 3840:] = r.contiguous().view(torch.uint8).view(k, 2048)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, P = c["B"], c["page"]
    spans, seen = _spans(c), _visible(c)
    n_max = max(n for n, _, _ in spans)
    max_pages = max(1, -(-n_max // P))
    # only pages that some visible token lies in exist; the others' entries are -1, as after eviction
    need = []
    for b, (s, lo, n) in enumerate(seen):
        need += [(b, i) for i in sorted(set(range(-(-s // P))) | set(range(lo // P, -(-n // P))))]
    n_pages = max(1, len(need))
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    order = np.random.RandomState(seed % (1 << 31)).permutation(n_pages)   # pages lie in any order
    if need:
        at = torch.tensor(need)
        table[at[:, 0], at[:, 1]] = torch.from_numpy(order[:len(need)].astype(np.int32))
    pages = torch.empty(n_pages * P * BYTES[c["fmt"]], dtype=torch.uint8, device="cuda")
    for first in range(0, n_pages * P, 131072):
        k = min(131072, n_pages * P - first)
        _fill(pages, c["fmt"], first, _tokens(g, k))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(c, pages=pages.view(n_pages, P * BYTES[c["fmt"]]), table=table.cuda(), start=i32([t for _, _, t in spans]),
             n_new=i32([k for _, k, _ in spans]), seq_len=i32([n for n, _, _ in spans]))
    if c["op"] in ("append", "step"):
        T = c["T"] if c["op"] == "append" else c["Q"]
        s["kv_new"] = _tokens(g, B * T).view(B, T, D)
        s["seq_len"] = s["start"].clone() if c["op"] == "append" else s["seq_len"]
    if c["op"] not in ("append", "read"):
        s["q"] = torch.randn(B, c["Q"], c["H"], D, generator=g, device="cuda").to(torch.bfloat16)
    return s


# ---- the plain form -------------------------------------------------------------------------------
def _rows(s, tok, ok):
    """fp32 values [B, L, 512] of the tokens tok [B, L], zeros where ok is false."""
    P = s["page"]
    page = torch.gather(s["table"].long(), 1, torch.where(ok, tok // P, 0))
    at = torch.where(ok, page * P + tok % P, 0)
    if s["fmt"] == "fp8":
        e = s["pages"].view(-1, 576)[at]
        v = torch.cat([e[..., :NOPE].view(torch.float8_e4m3fn).float(), e[..., NOPE:].contiguous().view(torch.bfloat16).float()], -1)
    else:
        chunks, ch, t = s["pages"].view(-1, CHUNK_BYTES), at // CHUNK, at % CHUNK
        w = chunks[:, :3584].reshape(-1, GROUPS, CHUNK, 16)[ch, :, t].view(torch.int32)          # [B, L, 14, 4]
        e = chunks[:, 3584:3808].reshape(-1, GROUPS, CHUNK)[ch, :, t]                            # [B, L, 14]
        r = chunks[:, 3840:].reshape(-1, CHUNK, 128)[ch, t].view(torch.bfloat16)
        i = torch.arange(8, device=w.device, dtype=torch.int32)
        grid = torch.tensor(GRID, device=w.device)
        mag = grid[((w[..., None] >> (4 * i)) & 7).long()]
        neg = (w[..., None] >> torch.where(i < 4, 8 * i + 7, 8 * (i - 4) + 3)) & 1
        v = torch.where(neg == 1, -mag, mag).flatten(-2) * torch.ldexp(torch.ones((), device=w.device), e.int() - 127)[..., None]
        v = torch.cat([v.flatten(-2), r.float()], -1)
    return torch.where(ok[..., None], v, 0.0)


def _rotated(x, pos):
    """bf16 tokens [B, T, 512] with their RoPE dims turned at the positions pos [B, T]; fp32, rounded to bf16 there."""
    i = torch.arange(ROPE // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[..., None] * torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device=x.device), -i / 32)
    p = x[..., NOPE:].double().unflatten(-1, (ROPE // 2, 2))
    r = torch.stack([p[..., 0] * a.cos() - p[..., 1] * a.sin(), p[..., 0] * a.sin() + p[..., 1] * a.cos()], -1)
    return torch.cat([x[..., :NOPE].float(), r.flatten(-2).to(torch.bfloat16).float()], -1)


def _stored(fmt, x):
    """The values that fp32 tokens stand for once stored."""
    if fmt == "fp8":
        return torch.cat([x[..., :NOPE].clamp(-448, 448).to(torch.float8_e4m3fn).float(), x[..., NOPE:]], -1)
    g = x[..., :NOPE].unflatten(-1, (GROUPS, 32))
    m, e = torch.frexp(g.abs().amax(-1, keepdim=True))
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(-126, 125)
    a = torch.ldexp(g.abs(), -e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = torch.ldexp(torch.copysign((a / step).round() * step, g).clamp(-6, 6), e)
    return torch.cat([v.flatten(-2), x[..., NOPE:]], -1)


def _attend(s, kv, tok, ok, q):
    """softmax(q kv^T) kv over the tokens tok [B, L] that each query sees; bf16 out and fp32 lse."""
    Q, n = s["Q"], s["seq_len"].long()
    p = (n[:, None] - Q + torch.arange(Q, device=n.device))[:, :, None]                          # [B, Q, 1]
    t = tok[:, None, :]
    see = ok[:, None, :] & (t <= p)
    if s["op"] == "window":
        see = see & ((t < s["S"]) | (t > p - s["W"]))
    x = torch.einsum("bqhd,bld->bqhl", q.float(), kv) * SCALE
    x = x.masked_fill(~see[:, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(x - m)
    l = w.sum(-1, keepdim=True)
    out = torch.einsum("bqhl,bld->bqhd", w, kv) / l.clamp(min=1e-30)
    return out.to(torch.bfloat16), (m + torch.log(l))[..., 0]


def _window_tokens(s):
    """[B, S + W + Q - 1] tokens: the first S, then the W + Q - 1 newest; and which of them count."""
    n = s["seq_len"].long()[:, None]
    first = torch.arange(s["S"], device=n.device)[None, :].expand(s["B"], -1)
    last = n - (s["W"] + s["Q"] - 1) + torch.arange(s["W"] + s["Q"] - 1, device=n.device)
    lo = (n - (s["W"] + s["Q"] - 1)).clamp(min=0)
    return torch.cat([first, last], 1), torch.cat([(first < lo), last >= 0], 1)


def _plain(s):
    op = s["op"]
    if op in ("append", "step"):
        T = s["kv_new"].shape[1]
        i = torch.arange(T, device="cuda")
        pos = s["start"].long()[:, None] + i
        new = i < s["n_new"].long()[:, None]
        x = _stored(s["fmt"], _rotated(s["kv_new"], pos))
    if op == "append":
        s["seq_len"].copy_(s["start"] + s["n_new"])
        if s["fmt"] == "fp4":
            return torch.where(new[..., None], x, 0.0).to(torch.bfloat16), s["seq_len"]
        at = (torch.gather(s["table"].long(), 1, torch.where(new, pos // s["page"], 0)) * s["page"] + pos % s["page"])[new]
        flat = s["pages"].view(-1, 576)
        flat[at, :NOPE] = x[new][:, :NOPE].to(torch.float8_e4m3fn).view(torch.uint8)
        flat[at, NOPE:] = x[new][:, NOPE:].to(torch.bfloat16).view(torch.uint8)
        return flat[:, :NOPE].view(torch.float8_e4m3fn), flat[:, NOPE:].view(torch.bfloat16), s["seq_len"]
    if op == "read":
        tok = s["start"].long()[:, None] + torch.arange(s["T"], device="cuda")
        return _rows(s, tok, tok < s["seq_len"].long()[:, None]).to(torch.bfloat16)
    if op == "window":
        tok, ok = _window_tokens(s)
    else:
        tok = torch.arange(s["table"].shape[1] * s["page"], device="cuda")[None, :].expand(s["B"], -1)
        ok = tok < s["seq_len"].long()[:, None]
    if op == "step":
        old = ok & (tok < s["start"].long()[:, None])
        kv = _rows(s, tok, old)
        b = torch.arange(s["B"], device="cuda")[:, None].expand_as(pos)
        kv[b[new], pos[new]] = x[new]
    else:
        kv = _rows(s, tok, ok)
    return _attend(s, kv, tok, ok, s["q"])


# ---- one pass -------------------------------------------------------------------------------------
def _own(s):
    import compressed_sparse_long_decode_b200 as csld

    cache = s.get("cache")
    if cache is None:   # the handle and the workspace that a user's program keeps
        cache = s["cache"] = csld.PagedCache(s["pages"], s["table"], s["seq_len"], s["page"], s["fmt"])
        s["ws"] = csld.paged_attention_workspace(s["pages"].device)
    op = s["op"]
    if op in ("append", "step"):
        csld.kv_cache_append_paged(cache, s["kv_new"], n_new=s["n_new"], start=s["start"], rope_base=ROPE_BASE)
    if op == "append":
        if s["fmt"] == "fp4":
            return csld.kv_cache_read_paged(cache, s["start"], s["T"]), s["seq_len"]
        flat = s["pages"].view(-1, 576)
        return flat[:, :NOPE].view(torch.float8_e4m3fn), flat[:, NOPE:].view(torch.bfloat16), s["seq_len"]
    if op == "read":
        return csld.kv_cache_read_paged(cache, s["start"], s["T"])
    if op == "window":
        return csld.paged_window_attention(cache, s["q"], s["W"], s["S"], SCALE, ws=s["ws"])
    return csld.paged_decode_attention(cache, s["q"], SCALE, ws=s["ws"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits --------------------------------------------------------------------
def _decode64(fmt, raw, token):
    """float64 [len(token), 512] of tokens counted over the pages' bytes, from the format's definition."""
    if fmt == "fp8":
        e = raw.view(-1, 576)[token]
        b = e[:, :NOPE].long()
        s, x, m = b >> 7, (b >> 3) & 15, (b & 7).double()
        v = torch.where(x == 0, m * 2.0 ** -9, (8 + m) * torch.pow(2.0, (x - 10).double())) * (1 - 2 * s)
        h = e[:, NOPE:].long()
        return torch.cat([v, _bf16_64(h[:, 0::2] | (h[:, 1::2] << 8))], 1)
    c = raw.view(-1, CHUNK_BYTES)[token // CHUNK]
    t, k = token % CHUNK, torch.arange(token.numel(), device=raw.device)
    d = torch.arange(NOPE, device=raw.device)
    group, in_word, word = d // 32, d % 8, (d % 32) // 8
    byte = group * 256 + t[:, None] * 16 + word * 4
    mag = (c[k[:, None], byte + in_word // 2].long() >> (4 * (in_word % 2))) & 7
    neg = torch.where(in_word < 4, c[k[:, None], byte + in_word % 4].long() >> 7, c[k[:, None], byte + in_word % 4].long() >> 3) & 1
    ex = c[k[:, None], 3584 + group * 16 + t[:, None]].double() - 127
    v = torch.tensor(GRID, dtype=torch.float64, device=raw.device)[mag] * torch.pow(2.0, ex) * (1 - 2 * neg)
    at = 3840 + t[:, None] * 128 + 2 * torch.arange(ROPE, device=raw.device)
    return torch.cat([v, _bf16_64(c[k[:, None], at].long() | (c[k[:, None], at + 1].long() << 8))], 1)


def _bf16_64(h):
    s, x, m = h >> 15, (h >> 7) & 255, (h & 127).double()
    return torch.where(x == 0, m * 2.0 ** -133, (128 + m) * torch.pow(2.0, (x - 134).double())) * (1 - 2 * s)


def _stored64(fmt, x, pos):
    """Tokens [T, 512] at positions pos [T] as stored: float64 nope values on the format's grid, the
    turned RoPE dims unrounded."""
    x = x.double()
    a = pos.double()[:, None] * ROPE_BASE ** (-torch.arange(32, device=x.device, dtype=torch.float64) / 32)
    u, v = x[:, NOPE::2], x[:, NOPE + 1::2]
    rope = torch.empty(x.shape[0], ROPE, dtype=torch.float64, device=x.device)
    rope[:, 0::2], rope[:, 1::2] = u * torch.cos(a) - v * torch.sin(a), u * torch.sin(a) + v * torch.cos(a)
    y = x[:, :NOPE]
    if fmt == "fp8":
        lead = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
        unit = torch.pow(2.0, lead - 3)
        return torch.cat([((y / unit).round() * unit).clamp(-448, 448), rope], 1)
    g = y.reshape(-1, GROUPS, 32)
    scale = torch.pow(2.0, torch.ceil(torch.log2(g.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100) / 6)))
    z = g.abs() / scale
    unit = torch.pow(2.0, torch.floor(torch.log2(z.clamp(min=1.0))) - 1)
    return torch.cat([(torch.sign(g) * (z / unit).round() * unit * scale).flatten(1), rope], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, P, fmt = s["op"], s["page"], s["fmt"]
    table = s["table"].long()

    def entries(b, tok):
        return _decode64(fmt, s["pages"].view(-1), table[b, tok // P] * P + tok % P)

    spans, dev = _spans(s), "cuda"
    if op == "read":
        out = torch.zeros(s["B"], s["T"], D, dtype=torch.float64, device=dev)
        for b, (n, k, start) in enumerate(spans):
            for i in range(0, k, 16384):
                m = min(16384, k - i)
                out[b, i:i + m] = entries(b, torch.arange(start + i, start + i + m, device=dev))
        return out
    if op == "append":
        ends = torch.tensor([n for n, _, _ in spans])
        if fmt == "fp4":
            out = torch.zeros(s["B"], s["T"], D, dtype=torch.float64, device=dev)
            for b, (n, k, start) in enumerate(spans):
                out[b, :k] = _stored64(fmt, s["kv_new"][b, :k], torch.arange(start, start + k, device=dev))
            return out, ends
        every = torch.cat([_decode64(fmt, s["pages"].view(-1), torch.arange(i, min(i + 16384, s["pages"].numel() // 576), device=dev))
                           for i in range(0, s["pages"].numel() // 576, 16384)])
        for b, (n, k, start) in enumerate(spans):
            tok = torch.arange(start, start + k, device=dev)
            every[table[b, tok // P] * P + tok % P] = _stored64(fmt, s["kv_new"][b, :k], tok)
        return every[:, :NOPE], every[:, NOPE:], ends
    out = torch.zeros(s["B"], s["Q"], s["H"], D, dtype=torch.float64, device=dev)
    lse = torch.full((s["B"], s["Q"], s["H"]), -math.inf, dtype=torch.float64, device=dev)
    for b, ((n, k, start), (first, lo, _)) in enumerate(zip(spans, _visible(s))):
        tok = torch.cat([torch.arange(first, device=dev), torch.arange(lo, n, device=dev)])
        if not len(tok):
            continue
        q = s["q"][b].double()
        acc = torch.zeros(s["Q"], s["H"], D, dtype=torch.float64, device=dev)
        top = torch.full((s["Q"], s["H"]), -math.inf, dtype=torch.float64, device=dev)
        den = torch.zeros(s["Q"], s["H"], dtype=torch.float64, device=dev)
        p = (n - s["Q"] + torch.arange(s["Q"], device=dev))[:, None]
        for i in range(0, len(tok), 65536):
            t = tok[i:i + 65536]
            v = entries(b, t)
            if op == "step":
                mine = t >= start
                fresh = _stored64(fmt, s["kv_new"][b, :k], torch.arange(start, n, device=dev))
                fresh[:, NOPE:] = fresh[:, NOPE:].to(torch.bfloat16).double()   # an entry holds bf16 there
                v[mine] = fresh[t[mine] - start]
            see = t[None, :] <= p
            if op == "window":
                see = see & ((t[None, :] < s["S"]) | (t[None, :] > p - s["W"]))
            x = torch.where(see[:, None, :], (q @ v.T) * SCALE, -math.inf)
            new = torch.maximum(top, x.amax(-1))
            base = torch.where(torch.isinf(new), 0.0, new)
            w = torch.exp(x - base[..., None])
            keep = torch.exp(top - base)
            acc, den, top = acc * keep[..., None] + w @ v, den * keep + w.sum(-1), new
        some = den > 0
        out[b] = torch.where(some[..., None], acc / den.clamp(min=1e-300)[..., None], 0.0)
        lse[b] = torch.where(some, top + torch.log(den.clamp(min=1e-300)), -math.inf)
    return out, lse
