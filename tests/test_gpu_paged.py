"""GPU parity of the paged entry cache: append (with and without rotation), read-back, sliding-window
attention with first tokens kept, and full attention, over fp8 and fp4 entries, against the 64-bit
reference of tests/paged_reference.py."""
import math

import numpy as np
import pytest
import torch

import synth
from tests import paged_reference as R

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(512.0)
BASE = 10000.0


@pytest.fixture(scope="module")
def csld():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import compressed_sparse_long_decode_b200 as m
    return m


def _tokens(g, *shape):
    """bf16 tokens with magnitudes spread from token to token."""
    x = torch.randn(*shape, 512, generator=g) * torch.exp(torch.randn(*shape, 1, generator=g))
    return x.to(torch.bfloat16)


class Pair:
    """The same cache on the device (csld.PagedCache) and in numpy: lens tokens of each sequence already
    stored (encoded by the reference), pages in random order, everything else in them garbage: 0xFF
    bytes, which are NaNs in every part of both formats."""

    def __init__(self, csld, lens, page, fmt, seed, extra=8, keep=None):
        g = synth.gen(seed)
        rng = np.random.default_rng(seed)
        B = len(lens)
        per = max(1, -(-(max(lens) + extra) // page))
        n_pages = B * per + 3
        table = rng.permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
        pages = np.full((n_pages, page * R.ENTRY[fmt]), 0xFF, np.uint8)
        self.ref = R.Cache(pages, table, np.array(lens, np.int32), page, fmt)
        for b, n in enumerate(lens):
            x = _tokens(g, n).double().numpy() if n else np.zeros((0, 512))
            for t in (range(n) if keep is None else [t for t in range(n) if keep(n, t)]):
                self.ref.store(b, t, x[t])
        if keep is not None:   # pages without a kept token are given back
            for b, n in enumerate(lens):
                for i in range(per):
                    if not any(t < n and keep(n, t) for t in range(i * page, (i + 1) * page)):
                        table[b, i] = -1 if i % 2 else n_pages + 5
        self.dev = csld.PagedCache(torch.from_numpy(pages.copy()).cuda(), torch.from_numpy(table).cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda(), page, fmt)

    def check_bytes(self, rope_ulp=0):
        """Device pages equal the reference's; RoPE values within rope_ulp bf16 steps."""
        torch.cuda.synchronize()
        a, r = self.dev.pages.cpu().numpy(), self.ref.pages
        assert np.array_equal(self.dev.seq_len.cpu().numpy(), self.ref.seq_len)
        if rope_ulp == 0:
            assert np.array_equal(a, r)
            return
        if self.ref.fmt == "fp8":
            a, r = a.reshape(-1, 576), r.reshape(-1, 576)
            cut = 448
        else:
            a, r = a.reshape(-1, 5888), r.reshape(-1, 5888)
            cut = 3840
        assert np.array_equal(a[:, :cut], r[:, :cut])
        ab, rb = (x[:, cut:].copy().view(np.uint16) for x in (a, r))
        av, rv = R.bf16_values(ab), R.bf16_values(rb)
        same = ab == rb
        # one bf16 step (2^-7 of the value), or the fp32 turn's own error where a pair cancels
        with np.errstate(invalid="ignore"):
            near = np.abs(av - rv) <= rope_ulp * 2.0 ** -7 * np.abs(rv) + 2.0 ** -20 * 64
        assert np.all(same | near)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("lens,T,page,base,ragged,given", [
    ([0], 1, 16, 0.0, False, False),
    ([0, 15, 16, 17, 63], 1, 16, BASE, False, False),
    ([5, 0, 40], 7, 48, BASE, True, True),
    ([0, 3], 100, 32, 0.0, True, False),
    ([1000, 3, 77], 33, 64, BASE, True, True),
])
def test_append_and_read_match_reference(csld, fmt, lens, T, page, base, ragged, given):
    c = Pair(csld, lens, page, fmt, seed=len(lens) + T, extra=T + 8)
    g = synth.gen(T)
    B = len(lens)
    x = _tokens(g, B, T)
    x[0, 0, 5] = float("inf")
    x[-1, -1, 40:72] = 0.0
    n_new = torch.tensor([(i * T + T - 1) // max(1, B) if i else T for i in range(B)], dtype=torch.int32).clamp(max=T) if ragged else None
    start = torch.tensor([max(0, n - 2) for n in lens], dtype=torch.int32) if given else None
    wide = torch.randn(B, T, 3, 512, generator=g).to(torch.bfloat16).cuda()   # a strided view, as out of a fused projection
    wide[:, :, 1] = x.cuda()
    csld.kv_cache_append_paged(c.dev, wide[:, :, 1], n_new=None if n_new is None else n_new.cuda(),
                               start=None if start is None else start.cuda(), rope_base=base)
    c.ref.append(x.double().numpy(), None if n_new is None else n_new.numpy(), None if start is None else start.numpy(), base)
    c.check_bytes(rope_ulp=1 if base else 0)
    assert c.dev.err.item() == 0
    back0 = torch.tensor([max(0, n - 3) for n in lens], dtype=torch.int32)
    back = csld.kv_cache_read_paged(c.dev, back0.cuda(), T + 9).double().cpu().numpy()
    dev = R.Cache(c.dev.pages.cpu().numpy(), c.ref.table, c.ref.seq_len, page, fmt)
    for b in range(B):
        for i in range(T + 9):
            t = int(back0[b]) + i
            want = dev.value(b, t) if t < c.ref.seq_len[b] else np.zeros(512)
            assert np.array_equal(back[b, i], want), (b, t)


def test_fp4_values_at_the_formats_edges(csld):
    """Zero, smallest, largest, saturating, NaN groups and every rounding midpoint, bytes and values."""
    c = Pair(csld, [0], 16, "fp4", seed=1)
    x = torch.zeros(1, 6, 512)
    x[0, 0, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4) * torch.tensor([1.0, -1.0] * 16)
    x[0, 1, :448] = torch.logspace(-38, 38, 448)
    x[0, 2, 0], x[0, 2, 33], x[0, 2, 64] = float("nan"), float("-inf"), 3.3e38
    x[0, 3, :448] = 1e-40
    x[0, 4, 100] = -0.0
    x[0, 5, :448] = torch.tensor([1.0, 6.0, 6.03125, 3.0, 3.015625, 4.0, 2.0 ** -30] * 64)
    x = x.to(torch.bfloat16)
    csld.kv_cache_append_paged(c.dev, x.cuda())
    v = x.double().numpy()
    v[0, 2, 0] = 0.0    # the group is stored as NaN whatever its codes; compare those apart
    c.ref.append(v, None, None, 0.0)
    torch.cuda.synchronize()
    a = c.dev.pages.cpu().numpy()[c.ref.table[0, 0]]
    r = c.ref.pages[c.ref.table[0, 0]].copy()
    assert a[3584 + 2] == 255
    a = a.copy()
    a[3584 + 2], a[2 * 16:3 * 16] = r[3584 + 2], r[2 * 16:3 * 16]
    assert np.array_equal(a, r)
    back = csld.kv_cache_read_paged(c.dev, torch.zeros(1, dtype=torch.int32).cuda(), 6).double().cpu().numpy()
    assert np.isnan(back[0, 2, :32]).all() and not np.isnan(back[0, 2, 32:]).any()


ATT = [
    # lens, Q, H, page, W, sinks
    ([1], 1, 16, 16, None, 0),
    ([0, 1, 15, 16, 17], 1, 16, 16, None, 0),
    ([95, 96, 97, 193], 1, 16, 48, None, 0),
    ([700, 3], 2, 16, 64, None, 0),
    ([333], 8, 5, 32, None, 0),
    ([5, 0, 2], 8, 16, 16, None, 0),
    ([260], 1, 128, 128, None, 0),
    ([200, 150], 3, 24, 16, None, 0),
    ([1500, 40, 700], 1, 16, 64, 128, 4),
    ([300, 4, 0], 4, 16, 64, 128, 4),
    ([120, 1], 1, 16, 16, 1, 0),
    ([130], 4, 1, 16, 1, 1),
    ([500], 1, 16, 32, 17, 33),
    ([90], 2, 16, 16, 1000, 5),
    ([100], 1, 16, 16, 5, 1000),
    ([400, 399], 8, 32, 48, 64, 16),
]


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("lens,Q,H,page,W,sinks", ATT)
def test_attention_matches_reference(csld, fmt, lens, Q, H, page, W, sinks):
    keep = None
    if W is not None:
        keep = lambda n, t: t < sinks or t > n - Q - W   # noqa: E731
    c = Pair(csld, lens, page, fmt, seed=sum(lens) + Q + H, keep=keep)
    q = torch.randn(len(lens), Q, H, 512, generator=synth.gen(H)).to(torch.bfloat16)
    ref = R.attention(c.ref, q.double().numpy(), SCALE, W, sinks)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full(q.shape, float("nan"), dtype=dt, device="cuda")
        if W is None:
            o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE, out=out)
        else:
            o, l = csld.paged_window_attention(c.dev, q.cuda(), W, sinks, SCALE, out=out)
        torch.cuda.synchronize()
        assert c.dev.err.item() == 0
        R.assert_attention(o, l, ref, f"{fmt} {lens} Q{Q} H{H} W{W} S{sinks} {dt}")


def _widen(csld, c, tokens):
    """The same cache with a page table for that many tokens, the pages behind the stored ones missing. The
    attention's way of dealing out heads follows from the capacity, so short sequences reach the long ones'."""
    wide = np.full((c.ref.table.shape[0], tokens // c.dev.page_size), -1, np.int32)
    wide[:, :c.ref.table.shape[1]] = c.ref.table
    c.ref.table = wide
    c.dev = csld.PagedCache(c.dev.pages, torch.from_numpy(wide).cuda(), c.dev.seq_len, c.dev.page_size, c.dev.fmt)


LONG = 1 << 19   # tokens of capacity: with one query and any number of heads more than 14 tiles of 64 entries an SM


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("lens,Q,H,page,W,sinks", [
    ([1], 1, 32, 16, None, 0),
    ([0, 17, 300], 1, 17, 64, None, 0),
    ([500, 64], 2, 40, 48, None, 0),
    ([2900, 1700], 1, 128, 64, None, 0),
    ([90, 2, 700], 8, 24, 16, None, 0),
    ([1300, 5], 3, 48, 32, 1 << 18, 16),
    ([40 * i % 1201 for i in range(37)], 1, 128, 64, 1000, 4),
])
def test_many_heads_over_a_large_capacity(csld, fmt, lens, Q, H, page, W, sinks):
    keep = None
    if W is not None:
        keep = lambda n, t: t < sinks or t > n - Q - W   # noqa: E731
    c = Pair(csld, lens, page, fmt, seed=sum(lens) + Q + H, keep=keep)
    _widen(csld, c, LONG // page * page)
    q = torch.randn(len(lens), Q, H, 512, generator=synth.gen(H)).to(torch.bfloat16)
    ref = R.attention(c.ref, q.double().numpy(), SCALE, W, sinks)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full(q.shape, float("nan"), dtype=dt, device="cuda")
        if W is None:
            o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE, out=out)
        else:
            o, l = csld.paged_window_attention(c.dev, q.cuda(), W, sinks, SCALE, out=out)
        torch.cuda.synchronize()
        assert c.dev.err.item() == 0
        R.assert_attention(o, l, ref, f"{fmt} {lens} Q{Q} H{H} W{W} S{sinks} {dt}")


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("lens,H,W", [([900, 33], 32, None), ([300, 70, 5], 16, 128)])
def test_output_in_place_of_the_query(csld, fmt, lens, H, W):
    """out may be q: every row's query is read before its output is written, rows cut over CTAs and whole ones."""
    c = Pair(csld, lens, 64, fmt, seed=21)
    q = torch.randn(len(lens), 2, H, 512, generator=synth.gen(5)).to(torch.bfloat16).cuda()
    call = (lambda x, **k: csld.paged_decode_attention(c.dev, x, SCALE, **k)) if W is None else \
        (lambda x, **k: csld.paged_window_attention(c.dev, x, W, 4, SCALE, **k))
    want, lw = call(q)
    o, l = call(q, out=q)
    assert o is q and torch.equal(o, want) and torch.equal(l, lw)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_many_heads_with_rising_and_falling_logits(csld, fmt):
    """Heads whose running maxima move at other tiles than their neighbours', in both groups of a row."""
    n = 1200
    c = Pair(csld, [n], 64, fmt, seed=3)
    d = torch.sign(torch.randn(512, generator=synth.gen(8)))
    for t in range(n):
        c.ref.store(0, t, (d * (t + 1) / 256.0).to(torch.bfloat16).double().numpy())
    c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
    _widen(csld, c, LONG)
    sign = torch.ones(32)
    sign[5:20] = -1.0
    sign[::7] = 0.125
    q = (d * sign[:, None])[None, None].to(torch.bfloat16).contiguous()
    for scale in (SCALE, 4 * SCALE):
        o, l = csld.paged_decode_attention(c.dev, q.cuda(), scale)
        R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), scale), f"{fmt} rising {scale}")


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("scale", [8 * SCALE, -2 * SCALE, 0.0])
def test_attention_with_peaked_flat_and_negative_scales(csld, fmt, scale):
    c = Pair(csld, [1000, 37], 64, fmt, seed=9)
    q = torch.randn(2, 1, 16, 512, generator=synth.gen(4)).to(torch.bfloat16)
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), scale)
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), scale), f"{fmt} scale {scale}")


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_rising_logits_move_the_running_maximum(csld, fmt):
    """Token t's logit grows with t for half of the heads and falls for the others, by far more than any
    lazily kept maximum allows, so every tile brings a new maximum."""
    n = 1200
    c = Pair(csld, [n], 64, fmt, seed=3)
    d = torch.sign(torch.randn(512, generator=synth.gen(8)))
    for t in range(n):
        c.ref.store(0, t, (d * (t + 1) / 256.0).to(torch.bfloat16).double().numpy())
    c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
    q = (d * torch.tensor([1.0, -1.0] * 8)[:, None])[None, None].to(torch.bfloat16).contiguous()
    for scale in (SCALE, 4 * SCALE):
        o, l = csld.paged_decode_attention(c.dev, q.cuda(), scale)
        R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), scale), f"{fmt} rising {scale}")


def test_fp4_entries_of_very_unlike_magnitudes(csld):
    """Neighbouring tokens 2^40 apart, and groups of one token 2^20 apart."""
    g = synth.gen(5)
    c = Pair(csld, [200], 16, "fp4", seed=2)
    for t in range(200):
        x = torch.randn(512, generator=g) * 2.0 ** (-20 if t % 2 else 0)
        if t % 3 == 0:
            x[32:64] *= 2.0 ** -20
        if t % 5 == 0:
            x *= 2.0 ** -20
        c.ref.store(0, t, x.to(torch.bfloat16).double().numpy())
    c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
    q = torch.randn(1, 1, 16, 512, generator=g).to(torch.bfloat16)
    ref = list(R.attention(c.ref, q.double().numpy(), SCALE))
    # A kernel may round a group whose scale lies far below its entry's largest: to 2^-16 of that scale, which
    # is at most 1 here (max|x| < 6), is allowed: 2^-16 on an output (A enters times 2^-8), and on a logit scale *
    # 32 dims * max|q| (< 6) * 2^-16 < 2^-12.
    ref[2] = ref[2] + 2.0 ** -8
    ref[3] = ref[3] + 2.0 ** -12
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE)
    R.assert_attention(o, l, ref, "unlike magnitudes")


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_nan_and_infinite_values_reach_only_the_queries_that_see_them(csld, fmt):
    c = Pair(csld, [64, 300], 16, fmt, seed=7)
    x = torch.randn(512, generator=synth.gen(1)).double().numpy()
    x[3] = np.nan
    c.ref.store(1, 150, x)
    c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
    q = torch.randn(2, 2, 16, 512, generator=synth.gen(2)).to(torch.bfloat16)
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE)
    assert torch.isnan(o[1]).all() and torch.isnan(l[1]).all() and not torch.isnan(o[0]).any()
    o, l = csld.paged_window_attention(c.dev, q.cuda(), 100, 4, SCALE)
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), SCALE, 100, 4), fmt)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_shared_and_missing_pages(csld, fmt):
    c = Pair(csld, [100, 100, 60], 16, fmt, seed=11)
    c.ref.table[1, :4] = c.ref.table[0, :4]     # a shared prefix
    c.ref.table[2, 1] = -1                      # tokens 16..31 of sequence 2 lost
    c.ref.table[2, 2] = 10 ** 6
    c.dev.page_table.copy_(torch.from_numpy(c.ref.table))
    q = torch.randn(3, 1, 16, 512, generator=synth.gen(6)).to(torch.bfloat16)
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE)
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), SCALE), fmt)
    assert c.dev.err.item() == 16
    c.dev.err.zero_()
    back = csld.kv_cache_read_paged(c.dev, torch.tensor([0, 90, 10], dtype=torch.int32).cuda(), 12)
    assert c.dev.err.item() == 16 and (back[2, 6:] == 0).all() and (back[1, 10:] == 0).all() and (back[2, :6] != 0).any()
    # the append of a sequence that misses a page or room (112 tokens here) is refused as a whole, the
    # others go through
    before = c.dev.pages.clone()
    x = _tokens(synth.gen(3), 3, 20)
    for first, lens in ((100, [100, 100, 60]), (92, [112, 100, 60])):
        c.dev.err.zero_()
        start = torch.tensor([first, 10 ** 7, 30], dtype=torch.int32)
        csld.kv_cache_append_paged(c.dev, x.cuda(), start=start.cuda())
        c.ref.append(x.double().numpy(), None, start.numpy(), 0.0)
        c.check_bytes()
        assert c.dev.err.item() == (16 | 1) and list(c.ref.seq_len) == lens
        assert torch.equal(before, c.dev.pages) == (first == 100)
    c.dev.err.zero_()
    csld.kv_cache_append_paged(c.dev, x.cuda(), n_new=torch.tensor([21, -1, 0], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert c.dev.err.item() == 4 and np.array_equal(c.dev.seq_len.cpu().numpy(), c.ref.seq_len)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_decode_run_append_window_and_full_together(csld, fmt):
    """Prefill chunk, then decode steps with 2 draft tokens of which one is accepted: append, window
    attention and full attention on the same cache, as a layer stack would use them; the last step
    captured in a CUDA graph on a side stream and replayed."""
    g = synth.gen(21)
    B = 3
    c = Pair(csld, [0, 0, 0], 32, fmt, seed=5, extra=200)
    ws = csld.paged_attention_workspace()
    pre, n0 = _tokens(g, B, 90), torch.tensor([90, 61, 7], dtype=torch.int32)
    csld.kv_cache_append_paged(c.dev, pre.cuda(), n_new=n0.cuda(), rope_base=BASE)
    c.ref.append(pre.double().numpy(), n0.numpy(), None, BASE)
    x = torch.zeros(B, 2, 512, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B, 2, 16, 512, dtype=torch.bfloat16, device="cuda")
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    res = {}

    def step():
        csld.kv_cache_append_paged(c.dev, x, start=start, rope_base=BASE)
        res["w"] = csld.paged_window_attention(c.dev, q, 32, 4, SCALE, ws=ws)
        res["f"] = csld.paged_decode_attention(c.dev, q, SCALE, ws=ws)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    for s in range(5):
        hx, hq = _tokens(g, B, 2), torch.randn(B, 2, 16, 512, generator=g).to(torch.bfloat16)
        at = n0 + s
        x.copy_(hx)
        q.copy_(hq)
        start.copy_(at)
        torch.cuda.synchronize()
        if s < 3:
            step()
        else:
            if s == 3:
                with torch.cuda.graph(graph, stream=side):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        c.ref.append(hx.double().numpy(), None, at.numpy(), BASE)
        dev = R.Cache(c.dev.pages.cpu().numpy(), c.ref.table, c.ref.seq_len, 32, fmt)
        c.check_bytes(rope_ulp=1)
        R.assert_attention(*res["w"], R.attention(dev, hq.double().numpy(), SCALE, 32, 4), f"{fmt} window step {s}")
        R.assert_attention(*res["f"], R.attention(dev, hq.double().numpy(), SCALE), f"{fmt} full step {s}")
    assert c.dev.err.item() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_decode_stack_with_window_layers(csld, fmt):
    """A stack of a CSA, an HCA and two window layers over 150 steps: the window layers keep a window of 32
    and 5 first tokens in a ring of pages that is smaller than the context, and match the reference
    over the tokens that they were given; the hybrid layers give what a stack without window layers gives."""
    B, steps, W, S, L = 2, 150, 32, 5, 4
    inp = synth.prefill_inputs(8, seed=0)
    make = lambda kinds: csld.DecodeStack(B, kinds, 64, 8, W, 16, inp["bias4"], inp["bias128"], inp["w_idx"],   # noqa: E731
                                          sinks=S, paged_context=200, paged_fmt=fmt, rope_base=BASE)
    kinds = ["window", "csa", "hca", "window"]
    stack, plain = make(kinds), make(["csa", "hca"])
    assert stack.layers[0].pages.shape[0] < B * stack.layers[0].max_pages
    assert stack.kv_bytes_per_sequence(steps) > plain.kv_bytes_per_sequence(steps)
    g = synth.gen(13)
    refs = []
    for _ in range(2):
        per = 4
        pages = np.zeros((B * per, 64 * R.ENTRY[fmt]), np.uint8)
        refs.append(R.Cache(pages, np.arange(B * per, dtype=np.int32).reshape(B, per), np.zeros(B, np.int32), 64, fmt))
    for s in range(steps):
        x = _tokens(g, L, B)
        gate = torch.randn(L, B, generator=g)
        q = torch.randn(L, B, 16, 512, generator=g).to(torch.bfloat16)
        qi, hw = torch.randn(L, B, 4, 64, generator=g), torch.randn(L, B, 4, generator=g).abs()
        a = [t.cuda() for t in (x, gate, q, qi, hw)]
        out, lse = torch.zeros(L, B, 16, 512, device="cuda"), torch.zeros(L, B, 16, device="cuda")
        o2, l2 = torch.zeros(2, B, 16, 512, device="cuda"), torch.zeros(2, B, 16, device="cuda")
        stack.step(*a, SCALE, out, lse)
        plain.step(*[t[1:3].contiguous() for t in a], SCALE, o2, l2)
        for k, i in enumerate((0, 3)):
            refs[k].append(x[i].double().numpy()[:, None], None, None, BASE)
        if s in (0, 20, 70, 149):
            torch.cuda.synchronize()
            assert torch.equal(out[1:3], o2) and torch.equal(lse[1:3], l2)
            for k, i in enumerate((0, 3)):
                ref = R.attention(refs[k], q[i].double().numpy()[:, None], SCALE, W, S)
                # the stored RoPE dims may differ by one bf16 step (2^-7 of the value): on A and on the logits (delta grows
                # from 512 * 2^-24 to 64 dims' 2^-7, at most)
                o, l, A, d, F = ref
                R.assert_attention(out[i][:, None], lse[i][:, None], (o, l, 3 * A, d * 2.0 ** 8, F), f"{fmt} layer {i} step {s}")
    assert stack.err.item() == 0


def test_two_streams_with_their_own_workspaces_and_inputs_of_another_stream(csld):
    """Two attention calls at once on two streams, each with its workspace, give what they give alone; a
    sequence of calls on a side stream is ordered by that stream alone."""
    c = Pair(csld, [3000, 1500, 77], 64, "fp4", seed=31)
    q = [torch.randn(3, 1, 16, 512, generator=synth.gen(k)).to(torch.bfloat16).cuda() for k in range(2)]
    want = [[t.clone() for t in csld.paged_decode_attention(c.dev, x, SCALE)] for x in q]
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [csld.paged_attention_workspace() for _ in range(2)]
    outs = [(torch.zeros(3, 1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 1, 16, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                csld.paged_decode_attention(c.dev, q[k], SCALE, out=outs[k][0], lse=outs[k][1], ws=ws[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(outs[k][0], want[k][0]) and torch.equal(outs[k][1], want[k][1])


def test_results_do_not_depend_on_the_run(csld):
    """Same call, same bits: no atomics decide an order (long and short rows, cut and whole ones)."""
    for fmt in ("fp8", "fp4"):
        c = Pair(csld, [2500, 10, 900], 32, fmt, seed=8)
        for H in (16, 40):
            q = torch.randn(3, 2, H, 512, generator=synth.gen(H)).to(torch.bfloat16).cuda()
            a = [t.clone() for t in csld.paged_decode_attention(c.dev, q, SCALE)]
            for _ in range(5):
                b = csld.paged_decode_attention(c.dev, q, SCALE)
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_offsets_past_2_to_the_31_bytes(csld, fmt):
    """Pages whose bytes begin past 2^31 (and 2^32) in the pool, and many sequences of which most are empty:
    more than the 640 that one pass of the scan covers."""
    page, B = 64, 1500
    entry = R.ENTRY[fmt]
    n_pages = (2 ** 32 + 2 ** 28) // (page * entry)
    pool = torch.empty((n_pages, page * entry), dtype=torch.uint8, device="cuda")
    lens = [0] * B
    for b, n in ((0, 5), (7, 130), (699, 64), (1203, 200), (1499, 1)):
        lens[b] = n
    table = torch.full((B, 4), -1, dtype=torch.int32)
    at = n_pages
    for b in range(B):
        for i in range(-(-lens[b] // page)):
            at -= 1 if b != 7 else (2 ** 31) // (page * entry) // 2
            table[b, i] = at
    seq = torch.tensor(lens, dtype=torch.int32)
    c = csld.PagedCache(pool, table.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"), page, fmt)
    x = _tokens(synth.gen(3), B, 200)
    csld.kv_cache_append_paged(c, x.cuda(), n_new=seq.cuda())
    q = torch.randn(B, 1, 16, 512, generator=synth.gen(5)).to(torch.bfloat16)
    o, l = csld.paged_decode_attention(c, q.cuda(), SCALE)
    torch.cuda.synchronize()
    assert c.err.item() == 0 and torch.equal(c.seq_len.cpu(), seq)
    keep = [b for b in range(B) if lens[b]]
    small = R.Cache(np.zeros((4 * len(keep), page * entry), np.uint8), np.arange(4 * len(keep), dtype=np.int32).reshape(-1, 4),
                    np.zeros(len(keep), np.int32), page, fmt)
    small.append(x[keep].double().numpy(), seq[keep].numpy(), None, 0.0)
    R.assert_attention(o[keep], l[keep], R.attention(small, q[keep].double().numpy(), SCALE), fmt)
    none = [b for b in range(B) if not lens[b]]
    assert (o[none] == 0).all() and torch.isneginf(l[none]).all()
    del pool, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_lengths_out_of_range_are_reported_and_bounded(csld, fmt):
    c = Pair(csld, [40, 40], 16, fmt, seed=12)
    q = torch.randn(2, 1, 16, 512, generator=synth.gen(2)).to(torch.bfloat16)
    c.dev.seq_len.copy_(torch.tensor([-5, 40], dtype=torch.int32))
    o, l = csld.paged_window_attention(c.dev, q.cuda(), 20, 2, SCALE)
    torch.cuda.synchronize()
    assert c.dev.err.item() == 4 and (o[0] == 0).all() and torch.isneginf(l[0]).all()
    c.ref.seq_len[:] = [0, 40]
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), SCALE, 20, 2), fmt)


def test_binding_refuses_bad_tensors(csld):
    c = csld.PagedCache.allocate(2, 100, 16, "fp4")
    q = torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(2, 1, 512, dtype=torch.bfloat16, device="cuda")
    for call in (
        lambda: csld.paged_decode_attention(c, q.float(), SCALE),
        lambda: csld.paged_decode_attention(c, q[:1], SCALE),
        lambda: csld.paged_decode_attention(c, q.cpu(), SCALE),
        lambda: csld.paged_decode_attention(c, q, float("nan")),
        lambda: csld.paged_decode_attention(c, q.expand(2, 9, 16, 512).contiguous(), SCALE),
        lambda: csld.paged_decode_attention(c, q, SCALE, out=torch.zeros(2, 1, 16, 512, device="cuda", dtype=torch.float16)),
        lambda: csld.paged_decode_attention(c, q, SCALE, ws=torch.zeros(64, dtype=torch.uint8, device="cuda")),
        lambda: csld.paged_window_attention(c, q, 0, 4, SCALE),
        lambda: csld.paged_window_attention(c, q, 1 << 32, 4, SCALE),
        lambda: csld.paged_window_attention(c, q, 8, -1, SCALE),
        lambda: csld.kv_cache_append_paged(c, x[:, :, :256]),
        lambda: csld.kv_cache_append_paged(c, x.float()),
        lambda: csld.kv_cache_append_paged(c, x, start=c.seq_len),
        lambda: csld.kv_cache_append_paged(c, x, n_new=torch.ones(3, dtype=torch.int32, device="cuda")),
        lambda: csld.kv_cache_append_paged(c, x, rope_base=0.5),
        lambda: csld.kv_cache_read_paged(c, c.seq_len, 0),
        lambda: csld.kv_cache_read_paged(c, c.seq_len, 4, out=torch.zeros(2, 4, 512, device="cuda")),
        lambda: csld.PagedCache(c.pages, c.page_table, c.seq_len, 16, "fp8"),
        lambda: csld.PagedCache(c.pages, c.page_table, c.seq_len, 16, "int4"),
        lambda: csld.PagedCache(c.pages, c.page_table[0], c.seq_len, 16, "fp4"),
    ):
        with pytest.raises(csld.CsldError):
            call()
    torch.cuda.synchronize()
    assert c.err.item() == 0 and c.seq_len.sum().item() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("rising", [False, True])
def test_sums_of_rows_whose_last_tile_sets_the_marks(csld, fmt, rising):
    """Rows of one tile, whose only tile sets the marks that its sums are relative to, and rows of a few tiles with
    rising logits, whose last one moves them: the sums of all four warps of the tile's group go by the
    new marks, in every one of many calls."""
    rng = np.random.default_rng(17)
    lens = [int(n) for n in rng.integers(1, 65 if not rising else 290, 100 if not rising else 24)]
    c = Pair(csld, lens, 64, fmt, seed=41)
    d = torch.sign(torch.randn(512, generator=synth.gen(8)))
    if rising:
        for b, n in enumerate(lens):
            for t in range(n):
                c.ref.store(b, t, (d * (t + 1) / 64.0).to(torch.bfloat16).double().numpy())
        c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
        q = (d * torch.tensor([1.0, -1.0, 0.5, 0.25] * 4)[:, None]).expand(len(lens), 1, 16, 512).to(torch.bfloat16).contiguous()
    else:
        q = torch.randn(len(lens), 1, 16, 512, generator=synth.gen(6)).to(torch.bfloat16)
    ref, qd = R.attention(c.ref, q.double().numpy(), SCALE), q.cuda()
    first = [t.clone() for t in csld.paged_decode_attention(c.dev, qd, SCALE)]
    R.assert_attention(*first, ref, f"{fmt} {rising}")
    out, lse, same = torch.empty_like(first[0]), torch.empty_like(first[1]), torch.ones((), dtype=torch.bool, device="cuda")
    ws = csld.paged_attention_workspace()
    for _ in range(300):
        csld.paged_decode_attention(c.dev, qd, SCALE, out=out, lse=lse, ws=ws)
        same &= (out == first[0]).all() & (lse == first[1]).all()
    assert same.item() and c.dev.err.item() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_tiles_without_a_chunk_after_full_ones(csld, fmt):
    """Rows that follow one another in a CTA's share and take turns between full tiles, empty sequences and tiles
    whose pages are all missing: nothing of a ring slot's earlier tile counts for a tile that copies nothing."""
    lens = [0 if b % 3 == 1 else 64 + 64 * (b % 4) + b % 5 for b in range(12)]
    c = Pair(csld, lens, 64, fmt, seed=43)
    for b in range(0, 12, 4):
        c.ref.table[b, 1:] = -1 if b else 10 ** 6      # all but the first tile of these rows lost
    c.dev.page_table.copy_(torch.from_numpy(c.ref.table))
    reps = 40                                          # 480 rows: every CTA walks several
    dev = csld.PagedCache(c.dev.pages, c.dev.page_table.repeat(reps, 1), c.dev.seq_len.repeat(reps), 64, fmt)
    q = torch.randn(12, 1, 16, 512, generator=synth.gen(6)).to(torch.bfloat16)
    o, l = csld.paged_decode_attention(dev, q.repeat(reps, 1, 1, 1).cuda(), SCALE)
    ref = R.attention(c.ref, q.double().numpy(), SCALE)
    R.assert_attention(o, l, [np.tile(a, (reps,) + (1,) * (a.ndim - 1)) for a in ref], fmt)
    assert dev.err.item() == 16


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("T,n", [(4, [1, 0, 1]), (3000, [5, 2, 0, 7])])
def test_append_reads_only_the_tokens_that_there_are(csld, fmt, T, n):
    """Sequences that lie right behind one another in the caller's buffer, closer than T tokens, the last ending with it;
    a refused count (T + 1, -1) reads nothing."""
    gap = max(n)
    c = Pair(csld, [3] * len(n), 32, fmt, seed=44, extra=T)
    x = _tokens(synth.gen(9), len(n), gap)
    n_new = torch.tensor(n, dtype=torch.int32)
    rows = (len(n) - 1) * gap + n[-1]            # up to the last sequence's last token
    buf = x.view(-1, 512)[:rows].contiguous().cuda()

    def call(counts):
        counts = counts.cuda()
        assert csld.lib.kv_cache_append_paged(c.dev._ref, buf.data_ptr(), gap * 512, 512, T, counts.data_ptr(), None, BASE,
                                              c.dev.err.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()

    call(n_new)
    full = np.zeros((len(n), T, 512))
    full[:, :gap] = x.double().numpy()
    c.ref.append(full, n_new.numpy(), None, BASE)
    c.check_bytes(rope_ulp=1)
    assert c.dev.err.item() == 0
    before = c.dev.pages.clone()
    call(torch.tensor([T + 1, -1] + [0] * (len(n) - 2), dtype=torch.int32))
    assert c.dev.err.item() == 4 and torch.equal(before, c.dev.pages)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_tensors_assigned_to_a_cache_are_the_ones_that_calls_use(csld, fmt):
    c = Pair(csld, [70, 20], 32, fmt, seed=45)
    q = torch.randn(2, 1, 16, 512, generator=synth.gen(6)).to(torch.bfloat16)
    old = [c.dev.pages, c.dev.page_table, c.dev.seq_len]
    was = [t.clone() for t in old]
    c.ref.seq_len[:] = [33, 20]
    c.dev.seq_len = torch.tensor([33, 20], dtype=torch.int32).cuda()
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE)
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), SCALE), f"{fmt} lengths")
    # a longer table over a pool of its own
    c.ref.pages = np.concatenate([c.ref.pages, np.full_like(c.ref.pages[:2], 0xFF)])[::-1].copy()
    c.ref.n_pages += 2
    c.ref.table = np.concatenate([c.ref.n_pages - 1 - c.ref.table, np.array([[0], [1]], np.int32)], 1)
    c.dev.pages = torch.from_numpy(c.ref.pages.copy()).cuda()
    c.dev.page_table = torch.from_numpy(c.ref.table).cuda()
    c.dev.err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert (c.dev.max_pages, c.dev.n_pages) == (c.ref.table.shape[1], c.ref.n_pages)
    x = _tokens(synth.gen(3), 2, 50)
    csld.kv_cache_append_paged(c.dev, x.cuda())
    c.ref.append(x.double().numpy(), None, None, 0.0)
    c.check_bytes()
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE)
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), SCALE), f"{fmt} pages")
    assert c.dev.err.item() == 0 and all(torch.equal(a, b) for a, b in zip(old, was))


def test_a_cache_refuses_what_does_not_fit_it(csld):
    c = csld.PagedCache.allocate(2, 100, 16, "fp4")
    have = dict(c.__dict__)
    for name, bad in (("seq_len", torch.zeros(3, dtype=torch.int32, device="cuda")), ("seq_len", c.seq_len.long()),
                      ("seq_len", c.seq_len.cpu()), ("page_table", c.page_table[0]), ("page_table", c.page_table.t()),
                      ("pages", c.pages[:, :-16]), ("pages", c.pages.view(torch.int8)), ("err", torch.zeros(1, device="cuda")),
                      ("err", torch.zeros(1, dtype=torch.int32)), ("batch", 1), ("max_pages", 1), ("n_pages", 1), ("page_size", 32),
                      ("fmt", "fp8"), ("entry_bytes", 576), ("device", torch.device("cpu")), ("_struct", None), ("_ref", None)):
        with pytest.raises(csld.CsldError):
            setattr(c, name, bad)
    assert c.__dict__ == have


def test_workspaces_that_are_no_plain_memory_are_refused(csld):
    """A view whose elements lie apart, or one element many times, has fewer bytes in a row than it counts."""
    c = csld.PagedCache.allocate(2, 100, 16, "fp4")
    q = torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    n = csld.paged_attention_workspace().numel()
    for ws in (torch.zeros(1, dtype=torch.uint8, device="cuda").expand(n), torch.zeros(n // 16, 32, dtype=torch.uint8, device="cuda")[:, :16],
               torch.zeros(n, dtype=torch.uint8)):
        for call in (lambda: csld.paged_decode_attention(c, q, SCALE, ws=ws),
                     lambda: csld.paged_window_attention(c, q, 8, 4, SCALE, ws=ws)):
            with pytest.raises(csld.CsldError):
                call()
    torch.cuda.synchronize()
    assert c.err.item() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("page,window,sinks,new", [(16, 40, 5, 4), (64, 32, 0, 1), (32, 64, 40, 8)])
def test_a_prompt_into_a_window_cache(csld, fmt, page, window, sinks, new):
    """Prompts of several lengths through a ring that is shorter than they are, as the documentation says: the first tokens,
    then the last ring_tokens; then draft steps of which some tokens are taken back.  The reference keeps every token."""
    B, context = 3, 400
    dev = csld.PagedCache.allocate(B, context, page, fmt, window=window, sinks=sinks, new_tokens=new)
    k = dev.ring_tokens
    assert window + 2 * new - 2 <= k < context - sinks
    per = -(-context // page)
    ref = R.Cache(np.zeros((B * per, page * R.ENTRY[fmt]), np.uint8), np.arange(B * per, dtype=np.int32).reshape(B, per),
                  np.zeros(B, np.int32), page, fmt)
    lens = [300, k + 3, 17]
    g = synth.gen(46)
    x = _tokens(g, B, 300)
    if sinks:
        csld.kv_cache_append_paged(dev, x[:, :sinks].cuda())
    start = [max(0, n - k) for n in lens]
    tail = torch.zeros(B, k, 512, dtype=torch.bfloat16)
    for b, n in enumerate(lens):
        tail[b, :n - start[b]] = x[b, start[b]:n]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    csld.kv_cache_append_paged(dev, tail.cuda(), n_new=i32([n - s for n, s in zip(lens, start)]), start=i32(start))
    ref.append(x.double().numpy(), lens, None, 0.0)
    at = list(lens)
    for step in range(6):
        hx, q = _tokens(g, B, new), torch.randn(B, new, 16, 512, generator=g).to(torch.bfloat16)
        csld.kv_cache_append_paged(dev, hx.cuda(), start=i32(at))
        ref.append(hx.double().numpy(), None, at, 0.0)
        o, l = csld.paged_window_attention(dev, q.cuda(), window, sinks, SCALE)
        R.assert_attention(o, l, R.attention(ref, q.double().numpy(), SCALE, window, sinks), f"{fmt} step {step}")
        at = [n + max(0, new - 1 - (step + b) % 3) for b, n in enumerate(at)]
    assert dev.err.item() == 0


def test_window_caches_refuse_what_they_do_not_hold(csld):
    c = csld.PagedCache.allocate(2, 400, 16, "fp4", window=40, sinks=5, new_tokens=2)
    k = c.ring_tokens
    q = torch.zeros(2, 2, 16, 512, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(2, k + 1, 512, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: csld.kv_cache_append_paged(c, x), lambda: csld.kv_cache_append_paged(c, x, n_new=c.seq_len + 1),
                 lambda: csld.paged_decode_attention(c, q, SCALE), lambda: csld.paged_window_attention(c, q, 41, 5, SCALE),
                 lambda: csld.paged_window_attention(c, q, 40, 6, SCALE),
                 lambda: csld.paged_window_attention(c, q.repeat(1, 2, 1, 1), 40, 5, SCALE)):
        with pytest.raises(csld.CsldError):
            call()
    torch.cuda.synchronize()
    assert c.err.item() == 0 and c.seq_len.sum().item() == 0
    csld.kv_cache_append_paged(c, x[:, :k])
    csld.paged_window_attention(c, q, 40, 5, SCALE)
    csld.paged_window_attention(c, q.repeat(1, 2, 1, 1), 38, 0, SCALE)
    # a table of the caller's, and a ring that never turns, have no such limits
    whole = csld.PagedCache.allocate(2, 60, 16, "fp4", window=40, sinks=5, new_tokens=2)
    assert whole.ring_tokens is None
    c.page_table = whole.page_table
    assert c.ring_tokens is None
    csld.paged_decode_attention(whole, q, SCALE)
    torch.cuda.synchronize()
    assert c.err.item() == 0 and whole.err.item() == 0


@pytest.mark.parametrize("heads", [16, 40])
@pytest.mark.parametrize("k", [10, 14, 18, 22, 28, 40, 100])
@pytest.mark.parametrize("at", [0, 300, 511])
def test_fp4_entry_far_larger_than_those_that_carry_weight(csld, heads, k, at):
    """One token 2^k above the others.  Half of the heads point away from it: its weight is 0 (its logit lies 2^k below) and
    the result is that of the other tokens, within the bounds formed over those alone.  The other heads see nothing but it."""
    n, g = 512, synth.gen(k + at)
    c = Pair(csld, [n], 64, "fp4", seed=47)
    d = torch.sign(torch.randn(512, generator=g))
    big = (-d * torch.exp2(torch.randint(0, 3, (512,), generator=g).float()) * 2.0 ** k).to(torch.bfloat16).double().numpy()
    c.ref.store(0, at, big)
    c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
    if heads > 16:
        _widen(csld, c, LONG)
    q = 0.5 * torch.randn(1, 1, heads, 512, generator=g) + d
    q[:, :, 1::2] -= 2 * d
    q = q.to(torch.bfloat16)
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE)
    vals = c.ref.values(0, range(n))[0]
    logit = SCALE * (q[0, 0].double().numpy() @ vals.T)
    rest = np.delete(np.arange(n), at)
    lead = np.where(np.arange(heads) % 2 == 0, 1.0, -1.0) * (logit[:, rest].max(1) - logit[:, at])
    assert lead.min() > 200                       # weights below e^-200
    # the reference over the tokens that have weight: the others' values, as they are stored, or the large one
    only = R.Cache(np.zeros((n // 64, 64 * R.ENTRY["fp4"]), np.uint8), np.arange(n // 64, dtype=np.int32)[None], np.zeros(1, np.int32), 64, "fp4")
    for i, t in enumerate(rest):
        only.store(0, i, vals[t])
    only.seq_len[0] = n - 1
    one = R.Cache(np.zeros((1, 64 * R.ENTRY["fp4"]), np.uint8), np.zeros((1, 1), np.int32), np.ones(1, np.int32), 64, "fp4")
    one.store(0, 0, vals[at])
    qd = q.double().numpy()
    R.assert_attention(o[:, :, 0::2], l[:, :, 0::2], R.attention(only, qd[:, :, 0::2], SCALE), f"2^{k} away")
    R.assert_attention(o[:, :, 1::2], l[:, :, 1::2], R.attention(one, qd[:, :, 1::2], SCALE), f"2^{k} alone")


@pytest.mark.parametrize("heads", [16, 24])
@pytest.mark.parametrize("course", ["any", "falling scales", "rising scales", "weight in the smallest", "weight in the largest"])
def test_fp4_scales_and_weights_of_any_course(csld, heads, course):
    """The query meets the RoPE dims alone, so that weights and the scales of the other dims go their own ways: over up to
    2^60 either, against each other and together, from tile to tile and within one."""
    n, g = 900, synth.gen(len(course))
    rng = np.random.default_rng(len(course))
    t = np.arange(n)
    logit, e = {"any": (rng.uniform(-40, 0, n), rng.integers(-30, 30, n)),
                "falling scales": (0.04 * t, np.rint(-0.04 * t / math.log(2))),       # weight times scale stays
                "rising scales": (-0.04 * t, np.rint(0.04 * t / math.log(2))),
                "weight in the smallest": (np.where(t % 7 == 3, 0.0, -30.0) + rng.uniform(0, 1, n), np.where(t % 7 == 3, -30, 10)),
                "weight in the largest": (0.08 * (t // 64 * 64) + rng.uniform(0, 1, n), np.rint(0.05 * t))}[course]
    c = Pair(csld, [n], 48, "fp4", seed=48)
    x = torch.randn(n, 512, generator=g).double().numpy()
    u = np.sign(x[0, 448:])
    x[:, :448] *= 2.0 ** e[:, None]
    x[:, 448:] = (logit / (64 * SCALE))[:, None] * u + 0.01 * x[:, 448:]     # a head that holds u has this logit
    for i in range(n):
        c.ref.store(0, i, torch.from_numpy(x[i]).to(torch.bfloat16).double().numpy())
    c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
    if heads > 16:
        _widen(csld, c, LONG // 48 * 48)
    q = torch.zeros(1, 1, heads, 512)
    q[..., 448:] = torch.from_numpy(u) * torch.tensor([1.0, 0.5, -1.0, 0.125])[torch.arange(heads) % 4][:, None]
    q = q.to(torch.bfloat16)
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE)
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), SCALE), course)


@pytest.mark.parametrize("k", [4, 12, 16, 20, 24, 32])
def test_fp4_weights_keep_their_bits_beside_a_far_larger_entry(csld, k):
    """fp32 outputs over 1,024 tokens of one magnitude and weights around 2^-10, the first token 2^k larger and of weight 0: the
    448 dims within 2^-11 A (f16 weights) and what the logits' rounding moves, for any k."""
    n, g = 1024, synth.gen(77)
    x = torch.randn(n, 512, generator=g)
    d = torch.sign(x[0])
    x[0] = -d * 2.0 ** k
    c = Pair(csld, [1], 64, "fp4", seed=49, extra=n)
    csld.kv_cache_append_paged(c.dev, x[None].to(torch.bfloat16).cuda(), start=torch.zeros(1, dtype=torch.int32, device="cuda"))
    dev = R.Cache(c.dev.pages.cpu().numpy(), c.ref.table, np.array([n], np.int32), 64, "fp4")
    q = (0.25 * torch.randn(1, 1, 16, 512, generator=g) + d).to(torch.bfloat16)
    out = torch.empty(1, 1, 16, 512, device="cuda")
    csld.paged_decode_attention(c.dev, q.cuda(), SCALE, out=out)
    v, qd = dev.values(0, range(n))[0], q.double().numpy()[0, 0]
    s = SCALE * qd @ v.T
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    assert w[:, 0].max() < 2.0 ** -20 / n
    w[:, 0] = 0.0
    delta = (512 * 2.0 ** -24 * SCALE * np.abs(qd) @ np.abs(v[1:]).T).max(1)[:, None]
    ref, A = (w @ v)[:, :448], (w @ np.abs(v))[:, :448]
    got = out[0, 0].double().cpu().numpy()[:, :448]
    # 2^-23: the absolute half steps of f16, 2^-30 of the largest weighted entry (weight below 2^-6, values below 6) for each of
    # 1,024 tokens
    assert np.all(np.abs(got - ref) <= (2.0 ** -11 + 2 * delta + 2.0 ** -21) * A + 2.0 ** -23)


@pytest.mark.parametrize("heads", [16, 24])
@pytest.mark.parametrize("lens,W", [([70], None), ([1, 40], None), ([200, 64], 50)])
def test_entries_that_were_never_stored_read_and_attend_as_zeros(csld, lens, W, heads):
    """An fp4 page of zero bytes (as allocate makes it) within a sequence: its tokens are zeros for the read-back and
    for attention alike, in full and beside stored ones; as in fp8, whose zero bytes are zeros."""
    for fmt in ("fp8", "fp4"):
        c = Pair(csld, lens, 16, fmt, seed=50)
        for b, n in enumerate(lens):
            for i in range(0, -(-n // 16), 2):                  # every other page
                c.ref.pages[c.ref.table[b, i]] = 0
            for t in range(n):
                if (t // 16) % 2 == 0 and t % 5 == 4:           # and some stored in these
                    c.ref.store(b, t, _tokens(synth.gen(t), 1)[0].double().numpy())
        c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
        if heads > 16 and W is None:
            _widen(csld, c, LONG)
        q = torch.randn(len(lens), 1, heads, 512, generator=synth.gen(6)).to(torch.bfloat16)
        call = (lambda: csld.paged_decode_attention(c.dev, q.cuda(), SCALE)) if W is None else \
            (lambda: csld.paged_window_attention(c.dev, q.cuda(), W, 3, SCALE))
        R.assert_attention(*call(), R.attention(c.ref, q.double().numpy(), SCALE, W, 3 if W else 0), f"{fmt} {lens}")
        back = csld.kv_cache_read_paged(c.dev, torch.zeros(len(lens), dtype=torch.int32, device="cuda"), max(lens))
        for b, n in enumerate(lens):
            assert np.array_equal(back[b, :n].double().cpu().numpy(), c.ref.values(b, range(n))[0])


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("heads", [16, 24])
@pytest.mark.parametrize("e", [-126, -118, -105, -60, 60, 100, 112, 116, 119, 122])
def test_queries_of_any_magnitude(csld, fmt, heads, e):
    """Queries 2^e as large under a scale 2^-e as large: the logits are those of e = 0.  Half of the heads 2^-8 of the others."""
    c = Pair(csld, [300, 20], 64, fmt, seed=51)
    if heads > 16:
        _widen(csld, c, LONG)
    q = torch.randn(2, 1, heads, 512, generator=synth.gen(6)).double()
    q[:, :, 1::2] *= 2.0 ** -8
    q = (q * 2.0 ** e).to(torch.bfloat16)
    scale = float(np.float32(SCALE * 2.0 ** -e))
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), scale)
    assert torch.isfinite(q).all() and c.dev.err.item() == 0
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), scale), f"{fmt} 2^{e}")


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** 100, -2.0 ** 112])
def test_logits_near_the_largest_numbers(csld, fmt, scale, wide):
    """Logits of up to 2^126, all of them negative for some heads: the largest one takes all the weight."""
    n = 100
    c = Pair(csld, [n], 32, fmt, seed=52)
    d = torch.sign(torch.randn(512, generator=synth.gen(8)))
    size = [1.0 + (37 * t % n) / 64.0 for t in range(n)]     # powers of two and their halves survive both formats
    for t in range(n):
        c.ref.store(0, t, (d * 2.0 ** round(size[t])).to(torch.bfloat16).double().numpy())
    c.ref.store(0, 61, (d * 0.25).double().numpy())          # the smallest and the largest one
    c.ref.store(0, 12, (d * 16.0).double().numpy())
    c.dev.pages.copy_(torch.from_numpy(c.ref.pages))
    if wide:      # the row cut over two CTAs
        _widen(csld, c, LONG)
    sign = torch.tensor([1.0, -1.0] * 8)
    q = (d * sign[:, None])[None, None].to(torch.bfloat16).contiguous()
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), scale)
    for h in range(16):
        up = sign[h].item() * scale > 0
        val = 16.0 if up else 0.25
        assert torch.equal(o[0, 0, h].float().cpu(), d * val)
        want = sign[h].item() * scale * 512 * val
        assert abs(l[0, 0, h].item() - want) <= 2.0 ** -14 * abs(want)


def _spread(csld, lens, tokens, fmt, seed):
    """A cache of many sequences, a table for `tokens` of each, pages in random order for the few that hold tokens; and
    the same in numpy, those sequences alone."""
    page = 64
    rng = np.random.default_rng(seed)
    keep = [b for b, n in enumerate(lens) if n]
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + 2).astype(np.int32)
    table = np.full((len(lens), tokens // page), -1, np.int32)
    at = 0
    for b in keep:
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    dev = csld.PagedCache(torch.full((len(order), page * R.ENTRY[fmt]), 0xFF, dtype=torch.uint8, device="cuda"), torch.from_numpy(table).cuda(),
                          torch.zeros(len(lens), dtype=torch.int32, device="cuda"), page, fmt)
    x = _tokens(synth.gen(seed), len(keep), max(lens))
    full = torch.zeros(len(lens), max(lens), 512, dtype=torch.bfloat16, device="cuda")
    full[keep] = x.cuda()
    csld.kv_cache_append_paged(dev, full, n_new=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert dev.err.item() == 0
    return dev, R.Cache(dev.pages.cpu().numpy(), table[keep], np.array([lens[b] for b in keep], np.int32), page, fmt), keep


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("Q,H,W", [(1, 16, None), (2, 24, None), (1, 16, 1 << 14)])
def test_more_sequences_than_one_pass_of_the_scan_covers(csld, fmt, Q, H, W):
    """1,500 sequences with a table for 2,560 tokens each: rows are cut, and which sequence a share begins in comes from three
    passes of 640; most are empty, long ones lie in every pass and at both ends."""
    lens = [0] * 1500
    for b, n in ((0, 1000), (3, 1), (638, 700), (639, 64), (640, 2560), (641, 65), (1279, 130), (1281, 1900), (1498, 17), (1499, 640)):
        lens[b] = n
    dev, ref, keep = _spread(csld, lens, 2560, fmt, 61)
    q = torch.randn(len(lens), Q, H, 512, generator=synth.gen(5)).to(torch.bfloat16)
    if W is None:
        o, l = csld.paged_decode_attention(dev, q.cuda(), SCALE)
    else:
        o, l = csld.paged_window_attention(dev, q.cuda(), W, 4, SCALE)
    assert dev.err.item() == 0
    R.assert_attention(o[keep], l[keep], R.attention(ref, q[keep].double().numpy(), SCALE, W, 4 if W else 0), f"{fmt} {Q} {H} {W}")
    none = [b for b, n in enumerate(lens) if not n]
    assert (o[none] == 0).all() and torch.isneginf(l[none]).all()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("B,Q", [(148, 1), (37, 4)])
def test_one_long_sequence_among_as_many_rows_as_sms(csld, fmt, B, Q):
    """The rows are a multiple of the SMs and one sequence is far longer: right, and not in the time that one CTA takes for it (with
    even shares it takes little longer than in a batch of one row less)."""
    n = 64 * 300
    lens = [1 + 7 * b % 200 for b in range(B)]
    lens[5] = n
    dev, ref, keep = _spread(csld, lens, 1 << 16, fmt, 62)
    q = torch.randn(B, Q, 16, 512, generator=synth.gen(5)).to(torch.bfloat16)
    o, l = csld.paged_decode_attention(dev, q.cuda(), SCALE)
    some = [4, 5, 6, B - 1]
    part = R.Cache(ref.pages, ref.table[some], ref.seq_len[some], 64, fmt)
    R.assert_attention(o[some], l[some], R.attention(part, q[some].double().numpy(), SCALE), f"{fmt} {B}")
    less = csld.PagedCache(dev.pages, dev.page_table[:-1].contiguous(), dev.seq_len[:-1].contiguous(), 64, fmt)
    ws, qd = csld.paged_attention_workspace(), q.cuda()
    ql = qd[:-1].contiguous()

    def best(f):
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                f()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    whole, fewer = best(lambda: csld.paged_decode_attention(dev, qd, SCALE, ws=ws)), best(lambda: csld.paged_decode_attention(less, ql, SCALE, ws=ws))
    # even shares: 300 long tiles and about 300 short rows over 148 SMs; one CTA alone: 300 tiles or more in a row
    assert whole < 2 * fewer, (whole, fewer)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_window_layers_token_by_token(csld, fmt):
    """Window layers of a stack over 150 steps through a ring of pages: what lies at every visible token's place is that
    token (the 448 dims byte for byte, the turned RoPE dims within one bf16 step), and attention matches the
    reference over the bytes that lie there, within the plain bounds."""
    B, W, S = 2, 32, 5
    inp = synth.prefill_inputs(8, seed=0)
    stack = csld.DecodeStack(B, ["window", "window"], 64, 8, W, 16, inp["bias4"], inp["bias128"], inp["w_idx"], sinks=S,
                             paged_context=200, paged_fmt=fmt, rope_base=BASE)
    assert stack.layers[0].ring_tokens is not None
    g = synth.gen(14)
    whole = [R.Cache(np.zeros((B * 4, 64 * R.ENTRY[fmt]), np.uint8), np.arange(B * 4, dtype=np.int32).reshape(B, 4), np.zeros(B, np.int32),
                     64, fmt) for _ in range(2)]
    none = torch.zeros(2, B, device="cuda"), torch.zeros(2, B, 4, 64, device="cuda"), torch.zeros(2, B, 4, device="cuda")
    for s in range(150):
        x, q = _tokens(g, 2, B), torch.randn(2, B, 16, 512, generator=g).to(torch.bfloat16)
        out, lse = torch.zeros(2, B, 16, 512, device="cuda"), torch.zeros(2, B, 16, device="cuda")
        stack.step(x.cuda(), none[0], q.cuda(), none[1], none[2], SCALE, out, lse)
        for i in range(2):
            whole[i].append(x[i].double().numpy()[:, None], None, None, BASE)
        if s % 16 != 5 and s not in (0, 63, 64, 128, 149):
            continue
        torch.cuda.synchronize()
        for i, layer in enumerate(stack.layers):
            dev = R.Cache(layer.pages.cpu().numpy(), layer.page_table.cpu().numpy(), layer.seq_len.cpu().numpy(), 64, fmt)
            for b in range(B):
                seen = R.visible(s, W, S)
                a, want = dev.values(b, seen)[0], whole[i].values(b, seen)[0]
                assert np.array_equal(a[:, :448], want[:, :448])
                assert np.all(np.abs(a - want)[:, 448:] <= 2.0 ** -7 * np.abs(want[:, 448:]) + 2.0 ** -20 * 64)
            R.assert_attention(out[i][:, None], lse[i][:, None], R.attention(dev, q[i].double().numpy()[:, None], SCALE, W, S),
                               f"{fmt} layer {i} step {s}")
    assert stack.err.item() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("page,n", [(16, 1), (16, 16), (32, 20)])
def test_a_pool_of_one_page(csld, fmt, page, n):
    """The smallest pool: fewer rows than the largest copy takes at once."""
    c = csld.PagedCache.allocate(1, page, page, fmt)
    assert c.n_pages == 1
    x, q = _tokens(synth.gen(n), 1, n), torch.randn(1, 1, 16, 512, generator=synth.gen(6)).to(torch.bfloat16)
    csld.kv_cache_append_paged(c, x.cuda())
    o, l = csld.paged_decode_attention(c, q.cuda(), SCALE)
    dev = R.Cache(c.pages.cpu().numpy(), c.page_table.cpu().numpy(), c.seq_len.cpu().numpy(), page, fmt)
    R.assert_attention(o, l, R.attention(dev, q.double().numpy(), SCALE), f"{fmt} {page}")
    back = csld.kv_cache_read_paged(c, torch.zeros(1, dtype=torch.int32, device="cuda"), n)
    assert np.array_equal(back[0].double().cpu().numpy(), dev.values(0, range(n))[0]) and c.err.item() == 0


def test_a_cache_takes_a_programs_own_attributes(csld):
    c = csld.PagedCache.allocate(2, 400, 16, "fp4", window=40, sinks=5)
    for v in ("layer 0", "layer 1"):
        c.name = v
        assert c.name == v
    with pytest.raises(csld.CsldError):
        c.ring_tokens = None


@pytest.mark.parametrize("heads", [24, 32])
@pytest.mark.parametrize("k", [18, 28, 100])
@pytest.mark.parametrize("at", [0, 511])
def test_fp4_entry_far_larger_in_rows_of_two_head_groups(csld, heads, k, at):
    test_fp4_entry_far_larger_than_those_that_carry_weight(csld, heads, k, at)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("heads", [33, 48, 80, 113])
def test_head_groups_of_either_number_over_a_large_capacity(csld, fmt, heads):
    """Three, five and eight groups of 16 heads, the last one full or with a single head."""
    c = Pair(csld, [500, 64], 64, fmt, seed=53)
    _widen(csld, c, LONG)
    q = torch.randn(2, 2, heads, 512, generator=synth.gen(heads)).to(torch.bfloat16)
    o, l = csld.paged_decode_attention(c.dev, q.cuda(), SCALE)
    R.assert_attention(o, l, R.attention(c.ref, q.double().numpy(), SCALE), f"{fmt} {heads}")
