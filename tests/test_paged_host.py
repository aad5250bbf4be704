"""The paged cache's reference codec against torch's casts, and the C entry points' refusals, which
happen on the host before anything is launched (no GPU needed)."""
import ctypes as C

import numpy as np
import pytest
import torch

from tests import paged_reference as R
from tests.test_abi import _build_lib


class Paged(C.Structure):
    _fields_ = [("format", C.c_int32), ("page_size", C.c_int32), ("batch", C.c_int32), ("max_pages", C.c_int32),
                ("n_pages", C.c_int64), ("pages", C.c_void_p), ("page_table", C.c_void_p), ("seq_len", C.c_void_p)]


@pytest.fixture(scope="module")
def lib():
    L = C.CDLL(_build_lib())
    P, I, I64, F, S, D = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t, C.c_double
    G = C.POINTER(Paged)
    L.kv_cache_append_paged.argtypes = [G, P, I64, I64, I, P, P, D, P, P]
    L.kv_cache_read_paged.argtypes = [G, P, I64, P, P, P]
    L.paged_decode_attention.argtypes = [G, P, I, I, F, P, I, P, P, S, P, P]
    L.paged_window_attention.argtypes = [G, P, I, I, I, I, F, P, I, P, P, S, P, P]
    L.csld_paged_attention_workspace_size.restype = S
    return L


def cache(**kw):
    c = Paged(4, 64, 2, 10, 20, 16, 16, 16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(format=5), 1), (dict(page_size=24), 1), (dict(page_size=0), 1), (dict(page_size=2048), 1),
              (dict(batch=0), 1), (dict(batch=70000), 1), (dict(max_pages=0), 1), (dict(max_pages=1 << 26), 1),
              (dict(n_pages=0), 1), (dict(n_pages=1 << 26), 1), (dict(pages=None), 1), (dict(page_table=None), 1),
              (dict(seq_len=None), 1), (dict(pages=8), 3)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(lib, kw, status):
    c, ws = cache(**kw), lib.csld_paged_attention_workspace_size()
    assert lib.kv_cache_append_paged(C.byref(c), 16, 512, 512, 1, None, None, 0.0, None, None) == status
    assert lib.kv_cache_read_paged(C.byref(c), 16, 4, 16, None, None) == status
    assert lib.paged_decode_attention(C.byref(c), 16, 16, 1, 0.1, 16, 1, None, 16, ws, None, None) == status
    assert lib.paged_window_attention(C.byref(c), 16, 16, 1, 8, 4, 0.1, 16, 1, None, 16, ws, None, None) == status
    assert lib.kv_cache_append_paged(None, 16, 512, 512, 1, None, None, 0.0, None, None) == 1


@pytest.mark.parametrize("args,status", [
    ((None, 512, 512, 1, None, None, 0.0), 1), ((16, 512, 512, 0, None, None, 0.0), 1),
    ((16, 512, 512, (1 << 20) + 1, None, None, 0.0), 1), ((8, 512, 512, 1, None, None, 0.0), 3),
    ((16, 513, 512, 1, None, None, 0.0), 3), ((16, 512, 516, 2, None, None, 0.0), 3),
    ((16, 512, 504, 2, None, None, 0.0), 2), ((16, -512, 512, 1, None, None, 0.0), 2),
    ((16, 512, 512, 1, None, 16, 0.0), 1),                      # start is seq_len
    ((16, 512, 512, 1, None, None, 1.0), 1), ((16, 512, 512, 1, None, None, float("nan")), 1),
    ((16, 512, 512, 1, None, None, float("inf")), 1), ((16, 512, 512, 1, None, None, -3.0), 1)])
def test_append_refusals(lib, args, status):
    assert lib.kv_cache_append_paged(C.byref(cache()), *args, None, None) == status


def test_read_refusals(lib):
    for args, status in (((None, 4, 16), 1), ((16, 0, 16), 1), ((16, 4, None), 1), ((16, 4, 8), 3), ((16, 1 << 31, 16), 1)):
        assert lib.kv_cache_read_paged(C.byref(cache()), *args, None, None) == status


def test_attention_refusals(lib):
    ws, c = lib.csld_paged_attention_workspace_size(), cache()
    good = dict(q=16, heads=16, Q=1, scale=0.1, out=16, out_type=1, lse=None, ws=16, n=ws)
    for kw, status in ((dict(q=None), 1), (dict(out=None), 1), (dict(heads=0), 6), (dict(heads=129), 6), (dict(Q=0), 1),
                       (dict(Q=9), 1), (dict(out_type=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
                       (dict(q=8), 3), (dict(out=8), 3), (dict(ws=None), 7), (dict(n=ws - 1), 7), (dict(ws=8), 3)):
        a = {**good, **kw}
        tail = (a["scale"], a["out"], a["out_type"], a["lse"], a["ws"], a["n"], None, None)
        assert lib.paged_decode_attention(C.byref(c), a["q"], a["heads"], a["Q"], *tail) == status, kw
        assert lib.paged_window_attention(C.byref(c), a["q"], a["heads"], a["Q"], 8, 4, *tail) == status, kw
    tail = (0.1, 16, 1, None, 16, ws, None, None)
    assert lib.paged_window_attention(C.byref(c), 16, 16, 1, 0, 4, *tail) == 1
    assert lib.paged_window_attention(C.byref(c), 16, 16, 1, 8, -1, *tail) == 1


def test_reference_codecs_against_torch_casts():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(4000, generator=g) * 2.0 ** torch.randint(-12, 12, (4000,), generator=g),
                   torch.tensor([0.0, -0.0, 448.0, 1000.0, 2.0 ** -10, 3 * 2.0 ** -10, -464.0])]).to(torch.bfloat16)
    want = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_codes(x.double().numpy()), want)
    assert np.array_equal(R.E4M3[want], x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy())
    f = torch.randn(5000, generator=g)
    assert np.array_equal(R.bf16_bits(f.numpy()), f.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16))
    assert np.array_equal(R.bf16_values(R.bf16_bits(f.numpy())), f.to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_reference_store_then_value(fmt):
    """A stored token reads back within its format's rounding, at every place of a page, and touches no
    other token's bytes."""
    rng = np.random.default_rng(3)
    c = R.Cache(np.full((2, 32 * R.ENTRY[fmt]), 0xFF, np.uint8), np.array([[1, 0]], np.int32), np.zeros(1, np.int32), 32, fmt)
    x = R.bf16_values(R.bf16_bits(rng.standard_normal((64, 512))))
    for t in rng.permutation(64):
        c.store(0, int(t), x[t])
    v, ok = c.values(0, range(64))
    assert ok.all() and np.array_equal(v[:, 448:], x[:, 448:])
    if fmt == "fp8":
        assert np.all(np.abs(v - x)[:, :448] <= 2.0 ** -4 * np.abs(x[:, :448]) + 2.0 ** -10)
    else:
        amax = np.abs(x[:, :448]).reshape(64, 14, 32).max(2, keepdims=True)
        assert np.all(np.abs(v - x)[:, :448].reshape(64, 14, 32) <= amax / 3.0)   # half a step of 2 at scale <= amax / 3
    assert c.value(0, 64) is None


def test_reference_attention_against_torch_softmax():
    rng = np.random.default_rng(4)
    c = R.Cache(np.zeros((4, 16 * 576), np.uint8), np.array([[3, 0, 2]], np.int32), np.array([37], np.int32), 16, "fp8")
    for t in range(37):
        c.store(0, t, rng.standard_normal(512))
    q = rng.standard_normal((1, 3, 2, 512))
    out, lse = R.attention(c, q, 0.1, 10, 2)[:2]
    k = torch.from_numpy(c.values(0, range(37))[0])
    for j in range(3):
        p = 37 - 3 + j
        see = torch.tensor([t <= p and (t < 2 or t > p - 10) for t in range(37)])
        s = (torch.from_numpy(q[0, j]) @ k.T * 0.1).masked_fill(~see, -np.inf)
        np.testing.assert_allclose(out[0, j], (torch.softmax(s, 1) @ k).numpy(), rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(lse[0, j], torch.logsumexp(s, 1).numpy(), rtol=1e-12)


@pytest.mark.parametrize("n_new,start", [(16, None), (20, None), (12, None), (None, 20), (None, 12), (16, 64)])
def test_append_refuses_lengths_that_lie_over_seq_len(lib, n_new, start):
    """seq_len (two sequences, at 16) is written while n_new and start are read."""
    assert lib.kv_cache_append_paged(C.byref(cache()), 16, 512, 512, 1, n_new, start, 0.0, None, None) == 1
