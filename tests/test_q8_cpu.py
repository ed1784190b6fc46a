"""The 8-bit cache on the CPU: pins of its oracle by closed forms and worked
values, and the library's refusals, which come before any device call."""
import ctypes
import struct

import numpy as np
import pytest
import torch

from compressed_decode_attention_encode_b200 import build as B
from compressed_decode_attention_encode_b200 import tq
from oracle import q8_oracle as O


@pytest.fixture(scope="module")
def lib():
    B.build()
    return tq.lib()


# ---- oracle -----------------------------------------------------------------

def test_e4m3_rounding_equals_torch_on_every_grid_and_midpoint():
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mid = (grid[1:] + grid[:-1]) / 2
    for y in (grid, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), -mid):
        got = O.round_e4m3(y)
        want = torch.from_numpy(y.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
        same = y.astype(np.float32).astype(np.float64) == y
        np.testing.assert_array_equal(got[same], want[same])
    assert O.round_e4m3(np.array([17.0]))[0] == 16.0 and O.round_e4m3(np.array([19.0]))[0] == 20.0


def test_quantise_worked_values():
    x = np.zeros((64, 2), np.float32)
    x[0, 0], x[1, 1], x[2, 0] = 254.0, -3.0, 1.0           # a = 254: int8 scale 2
    c, s = O.quantise_block(x, "int8")
    assert s == np.float32(2.0) and c[0, 0] == 127 and c[1, 1] == -2 and c[2, 0] == 0   # -1.5 -> -2, 0.5 -> 0
    x[0, 0], x[1, 1], x[2, 0] = 896.0, -34.0, 2.0 ** -9    # a = 896: e4m3 scale 2
    c, s = O.quantise_block(x, "e4m3")
    assert s == np.float32(2.0) and c[0, 0] == 448 and c[1, 1] == -16 and c[2, 0] == 0  # 2^-10 ties to 0


def test_quantise_zero_tiny_and_bad_blocks():
    for fmt in ("int8", "e4m3"):
        c, s = O.quantise_block(np.zeros((64, 4)), fmt)
        assert s == 1 and not c.any()
        c, s = O.quantise_block(np.full((64, 4), 2.0 ** -101), fmt)
        assert s == 1 and not c.any()
        c, s = O.quantise_block(np.full((64, 4), 2.0 ** -100), fmt)
        assert c.max() == O.TOP[fmt]
        for bad in (np.nan, np.inf, -np.inf):
            x = np.ones((64, 4))
            x[5, 1] = bad
            c, s = O.quantise_block(x, fmt)
            assert np.isnan(s) and not c.any()


@pytest.mark.parametrize("fmt,bound", [("int8", 0.5 / 127), ("e4m3", 2.0 ** -4)])
def test_quantise_error_bound(fmt, bound):
    x = np.random.default_rng(0).standard_normal((5, 64, 16)).astype(np.float32)
    c, s = O.quantise_block(x, fmt)
    err = np.abs(c * s[:, None, None].astype(np.float64) - x)
    a = np.abs(x).max(axis=(1, 2))[:, None, None]
    # half a code for int8; half a step of the value, or of the least normal code, for e4m3; float32 roundings
    lim = bound * a if fmt == "int8" else np.maximum(bound * np.abs(x), a / 448 * 2.0 ** -10)
    assert (err <= lim + a * 2.0 ** -22).all()


def test_held_keeps_the_open_block():
    x = np.random.default_rng(1).standard_normal((130, 4))
    c, s = O.held(x, 130, "int8")
    np.testing.assert_array_equal(c[128:], x[128:])
    assert (s[128:] == 1).all() and np.unique(s[:64]).size == 1 and s[0] != s[64]
    c, s = O.held(x, 63, "int8")
    np.testing.assert_array_equal(c, x[:63])


def test_attention_equals_torch_and_masks_by_position():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((3, 2, 8)), g.standard_normal((10, 8)), g.standard_normal((10, 8))
    o, w = O.attention(q, k, v)
    mask = torch.ones(3, 10, dtype=torch.bool).tril(7)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), torch.from_numpy(k).expand(2, 10, 8),
        torch.from_numpy(v).expand(2, 10, 8), attn_mask=mask)
    np.testing.assert_allclose(o, want.transpose(0, 1).numpy(), atol=1e-12)
    np.testing.assert_allclose(w.sum(-1), 1.0, atol=1e-12)
    o, _ = O.attention(q, k[:1], v[:1])                    # only the newest query sees the one token
    assert not o[:2].any()
    np.testing.assert_allclose(o[2], np.broadcast_to(v[0], (2, 8)))
    k[9, 0] = np.inf                                       # seen by the newest query alone
    o, _ = O.attention(q, k, v)
    assert np.isnan(o[2]).all() and np.isfinite(o[:2]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_closed_forms(interleaved):
    g = np.random.default_rng(3)
    x, f = g.standard_normal((2, 3, 8)), np.array([1.0, 0.1, 0.01, 0.0])
    zero = O.norm_rope(x, np.zeros(2), f, interleaved=interleaved)
    np.testing.assert_allclose(zero, x, atol=1e-15)
    there = O.norm_rope(x, np.array([7, 131071]), f, interleaved=interleaved)
    back = O.norm_rope(there, np.array([-7, -131071]), f, interleaved=interleaved)
    np.testing.assert_allclose(back, x, atol=1e-10)
    np.testing.assert_allclose((there ** 2).sum(-1), (x ** 2).sum(-1))
    y = O.norm_rope(x, np.zeros(2), f, weight=np.full(8, 2.0), eps=0.0, interleaved=interleaved)
    np.testing.assert_allclose((y ** 2).mean(-1), 4.0)
    e = np.zeros((1, 1, 8))
    e[..., 0] = 1.0                                        # (1, 0) turned by a quarter is (0, 1)
    t = O.norm_rope(e, np.array([1]), np.full(4, np.pi / 2), interleaved=interleaved)
    assert abs(t[0, 0, 1 if interleaved else 4] - 1) < 1e-15


# The argument structs, fields in the order of include/tq.h; None is NULL.
def _pack(fmt, *fields):
    return struct.pack(fmt, *[0 if x is None else x for x in fields])


def _append(lib, ref, *f):
    return lib.tq_q8_append(ref, _pack("@PP6qi4xPP", *f[:-1]), f[-1])


def _attention(lib, ref, *f):
    return lib.tq_q8_attention(ref, _pack("@P3q2iPPf4xPPN", *f[:-1]), f[-1])


def _norm_rope(lib, *f):
    return lib.tq_qk_norm_rope(_pack("@6iP3qP3q4Pfi2P", *f[:-1]), f[-1])


# ---- refusals ---------------------------------------------------------------

def _struct(**kw):
    base = dict(batch=2, num_kv_heads=2, head_dim=64, format=0, dtype=0, capacity=128, k_codes=256, v_codes=512,
                k_scales=1024, v_scales=2048, k_recent=4096, v_recent=8192, status=16384)
    base.update(kw)
    return tq.tq_q8_cache(*[base[n] for n, _ in tq.tq_q8_cache._fields_])


BAD_CACHES = [
    (dict(batch=0), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=96), 2),
    (dict(head_dim=256), 2), (dict(format=2), 1), (dict(dtype=2), 1), (dict(capacity=0), 1),
    (dict(capacity=100), 1), (dict(capacity=-64), 1), (dict(capacity=2 ** 31), 2), (dict(batch=1025), 2),
    (dict(batch=1024, num_kv_heads=64), 2), (dict(k_codes=None), 1), (dict(v_codes=264), 1),
    (dict(k_scales=1026), 1), (dict(v_recent=None), 1), (dict(status=None), 1),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, kw, code):
    c = _struct(**kw)
    r = ctypes.addressof(c)
    size = ctypes.c_size_t()
    assert _append(lib, r, 256, 256, 8, 8, 8, 8, 8, 8, 1, 256, None, None) == code
    assert lib.tq_q8_read(r, 256, 0, 1, 256, 256, None) == code
    assert _attention(lib, r, 256, 8, 8, 8, 4, 1, 256, None, 0.0, 256, 256, 1 << 40, None) == code
    if not any(k in kw for k in ("k_codes", "v_codes", "k_scales", "v_recent", "status")):
        assert lib.tq_q8_attention_bytes(r, 4, 1, ctypes.byref(size)) == code


def test_null_structs(lib):
    r = ctypes.addressof(c := _struct())
    assert lib.tq_q8_append(r, None, None) == 1 and lib.tq_q8_attention(r, None, None) == 1
    assert lib.tq_qk_norm_rope(None, None) == 1
    del c


def test_null_cache(lib):
    assert _append(lib, None, 256, 256, 8, 8, 8, 8, 8, 8, 1, 256, None, None) == 1
    assert lib.tq_q8_read(None, 256, 0, 1, 256, 256, None) == 1
    assert _attention(lib, None, 256, 8, 8, 8, 4, 1, 256, None, 0.0, 256, 256, 1 << 40, None) == 1
    assert lib.tq_q8_attention_bytes(None, 4, 1, None) == 1
    assert lib.tq_q8_get_status(None, None) == 1


@pytest.mark.parametrize("at,value,code", [
    (1, None, 1), (2, None, 1), (1, 257, 1), (2, 264, 1), (3, 4, 1), (4, -8, 1), (5, 12, 1), (6, 4, 1),
    (7, -8, 1), (8, 7, 1), (9, -1, 1), (9, 129, 3), (10, None, 1), (10, 258, 1), (11, 257, 1)])
def test_append_refusals(lib, at, value, code):
    args = [ctypes.addressof(c := _struct()), 256, 256, 8, 8, 8, 8, 8, 8, 1, 256, None, None]
    args[at] = value
    assert _append(lib, *args) == code
    del c


@pytest.mark.parametrize("at,value,code", [(1, None, 1), (1, 258, 1), (2, -1, 1), (3, -1, 1), (4, None, 1),
                                           (5, 264, 1), (2, 128, 0), (3, 0, 0)])
def test_read_refusals(lib, at, value, code):
    args = [ctypes.addressof(c := _struct()), 256, 0, 1, 256, 256, None]
    args[at] = value
    assert lib.tq_q8_read(*args) == code
    del c


@pytest.mark.parametrize("at,value,code", [
    (1, None, 1), (1, 264, 1), (2, 4, 1), (3, -8, 1), (4, 12, 1), (5, 0, 1), (5, 3, 1), (5, 34, 2), (6, 0, 1),
    (6, 65, 2), (7, None, 1), (7, 258, 1), (8, 257, 1), (9, float("nan"), 1), (9, float("inf"), 1),
    (10, None, 1), (10, 264, 1), (11, None, 1), (11, 264, 1)])
def test_attention_refusals(lib, at, value, code):
    args = [ctypes.addressof(c := _struct()), 256, 8, 8, 8, 4, 1, 256, None, 0.0, 256, 256, 1 << 40, None]
    args[at] = value
    assert _attention(lib, *args) == code
    del c


@pytest.mark.parametrize("at,value,code", [
    (0, -1, 1), (1, -1, 1), (2, -1, 1), (3, -1, 1), (4, 0, 1), (4, 96, 2), (5, 2, 1), (6, None, 1), (6, 264, 1),
    (7, 4, 1), (8, -8, 1), (9, 12, 1), (10, None, 1), (11, 7, 1), (12, -1, 1), (13, 4, 1), (14, None, 1),
    (15, None, 1), (16, 264, 1), (17, 264, 1), (18, -1.0, 1), (18, float("nan"), 1), (18, float("inf"), 1),
    (19, 2, 1), (20, None, 1), (21, 264, 1), (2, 70000, 2), (0, 0, 0), (1, 0, 0)])
def test_norm_rope_refusals(lib, at, value, code):
    args = [1, 1, 4, 2, 64, 0, 256, 8, 8, 8, 256, 8, 8, 8, 256, 256, 256, 256, 1e-6, 0, 256, 256, None]
    args[at] = value
    assert _norm_rope(lib, *args) == code


@pytest.mark.parametrize("kw", [dict(format="int4"), dict(dtype=torch.float32), dict(capacity=100), dict(head_dim=96),
                                dict(batch=0)])
def test_python_cache_refusals(lib, kw):
    base = dict(batch=1, num_kv_heads=1, head_dim=64, capacity=64, device="cpu")
    base.update(kw)
    with pytest.raises((ValueError, tq.TQError)):
        tq.TQ8Cache(**base)


def test_python_calls_refuse_other_tensors(lib):
    """Shapes, types, layouts and devices, before any call of the library."""
    c = tq.TQ8Cache(2, 2, 64, 128, device="cpu")
    h, i = dict(dtype=torch.float16), dict(dtype=torch.int32)
    k, lens, q = torch.zeros(2, 2, 3, 64, **h), torch.zeros(2, **i), torch.zeros(2, 1, 4, 64, **h)
    for a in ((k[:, :1], k, lens), (k, k[:, :, :2], lens), (k.float(), k.float(), lens),
              (k.transpose(2, 3).contiguous().transpose(2, 3), k, lens), (k, k, lens.long()), (k, k, lens[:1]),
              (k, k, torch.zeros(4, **i)[::2]), (k[0], k[0], lens), (k, k, lens, lens.long())):
        with pytest.raises(ValueError):
            c.append(*a)
    for a in ((lens.long(), 0, 3), (lens, 0, None), (lens, 0, 3, (k, k.float())), (lens, 0, 2, (k, k)),
              (lens, 0, 3, (k, k.transpose(0, 1)))):
        with pytest.raises(ValueError):
            c.read(*a)
    for a in ((q.float(), lens), (q[:1], lens), (q[..., :32], lens), (q, lens.long()), (q[0, 0], lens),
              (q, lens, lens[:1])):
        with pytest.raises(ValueError):
            c.attention(*a)
    with pytest.raises(ValueError):
        tq.TQ8Cache(2, 2, 64, 128, device="cpu", buffers={f"{x}_{y}": torch.zeros(1) for x in "kv"
                                                          for y in ("codes", "scales", "recent")})
    with pytest.raises(ValueError):   # CPU tensors
        tq.qk_norm_rope(q, k.transpose(1, 2), torch.zeros(2, 1, **i), torch.zeros(32))


def test_python_calls_need_a_cuda_cache(lib):
    """A cache of CPU tensors is refused at every call, whatever the box has."""
    c = tq.TQ8Cache(1, 1, 64, 64, device="cpu")
    k, lens = torch.zeros(1, 1, 1, 64, dtype=torch.float16), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: c.append(k, k, lens), lambda: c.read(lens, 0, 1), lambda: c.attention(k, lens),
                 lambda: c.scratch_bytes(1, 1), lambda: c.get_status()):
        with pytest.raises(ValueError):
            call()
