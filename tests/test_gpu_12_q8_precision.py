"""How near the 8-bit cache's attention comes to the float64 oracle: a result
is what float32 arithmetic gives, rounded once to the cache's type.

The bounds here are of that arithmetic alone; ``float32_bound`` derives them.
"""
import math

import numpy as np
import pytest
import torch

from oracle import q8_oracle as O
from tests.test_gpu_11_q8 import DT, Stream, values

pytestmark = pytest.mark.gpu


def float32_bound(w, q, ck, sk, cv, sv, sigma, dtype, alike=False):
    """|error| [n, G, d] of a result before it is rounded to its type.  With
    A = sum_p w_p |v_p|:

    * a logit sums as many exact products as q has elements that are not zero,
      each addition off by at most 2^-23 of sum |q k|, with four roundings
      around it; bf16 queries enter as fp16 after a power of two, elements below
      2^-31 of the largest off by 2^-40 of it; an error e of a logit changes a
      weight by 2 e (its exponential and the denominator's).  ``alike``: the
      logits that count are computed from the same numbers, e = 0;
    * a weight in two fp16 parts is off by 2^-11 of 2^-11; exponentials by
      2^-22 each, of the weight, of a reference's move, of the join and of the
      result's factor; a block's scale, as a logarithm, by 2^-22 of it;
    * sums: (L / 16 + 64) additions of 2^-23;
    * a weight's last fp16 part ends at 2^-25, where the row's largest
      w_p scale_p so far stands at 2^7 or above, times the code.  Blocks of
      zeros count for nothing; the open block comes last, with scale 1.
    """
    v = cv * sv[:, None]
    length, whole = len(sv), len(sv) // 64 * 64
    top = np.abs(v).max(-1)
    for j in range(0, length, 64):
        top[j:j + 64] = top[j:j + 64].max()
    scale = np.where(top > 0, sv, 0.0)
    ref = (w * scale)[..., :whole].max(-1, initial=0.0)[..., None]
    last = np.maximum(ref, w[..., whole:].max(-1, initial=0.0)[..., None])
    qk = np.einsum("ngd,ld->ngl", np.abs(q), np.abs(ck)) * sk * abs(sigma)
    e = (np.count_nonzero(q, axis=-1)[..., None] + 4) * 2.0 ** -23 * qk
    if dtype == "bf16":
        e = e + 2.0 ** -40 * np.abs(q).max(-1)[..., None] * (np.abs(ck).sum(-1) * sk * abs(sigma))
    e = 0.0 if alike else e.max(-1)[..., None]
    a = w @ np.abs(v)
    logs = np.abs(np.log2(scale[:whole][top[:whole] > 0])).max(initial=0.0)
    return (a * (2 * e + 2.0 ** -22 * (5 + logs) + (length / 16 + 64) * 2.0 ** -23)
            + 2.0 ** -32 * (ref * np.abs(cv[:whole]).sum(0) + last * np.abs(cv[whole:]).sum(0)))


def half_step(x, dtype):
    """Half the distance of neighbours of the type at |x|."""
    t = torch.finfo(DT[dtype])
    _, e = np.frexp(np.maximum(np.abs(x), t.smallest_normal))
    return np.ldexp(t.eps / 2, e - 1)


def assert_rounded(st, q, out, rows=None, sigma=0.0, alike=False, only=None):
    """Every result of rows (of those in ``only``) is the oracle's, rounded, but for float32_bound."""
    b, h, d = st.shape
    n, hq = q.shape[1:3]
    g = hq // h
    got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
    sig = sigma or 1 / math.sqrt(d)
    for i in range(b) if only is None else only:
        r = n if rows is None else rows[i]
        for u in range(h):
            heads = slice(u * g, (u + 1) * g)
            (ck, sk), (cv, sv) = ((c[u], s[u]) for c, s in (st.stored("k", i), st.stored("v", i)))
            o, w = O.attention(qd[i, :r, heads], ck * sk[:, None], cv * sv[:, None], sig)
            lim = float32_bound(w, qd[i, :r, heads], ck, sk, cv, sv, sig, st.dtype, alike)
            over = np.abs(got[i, :r, heads] - o) - half_step(np.abs(o) + lim, st.dtype) - lim
            assert (over <= 0).all(), (i, u, int((over > 0).sum()), float((over / lim).max()))
    assert st.c.get_status() == 0


def single(b, n, hq, d, dtype, value):
    """Queries of one element each, another one in every head."""
    q = torch.zeros(b, n, hq, d, dtype=DT[dtype])
    return q.scatter_(3, torch.arange(b * n * hq).view(b, n, hq, 1) % d, value).cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [1, 3])
def test_a_result_is_rounded_once(fmt, dtype, d, n):
    """Short rows whose queries have one element each: logits without sums, so
    that what is left is the weights' own precision."""
    lens = [64, 128, 63, 100, 17, 3]
    st = Stream(len(lens), 2, d, 128, fmt, dtype)
    st.append(1, max(lens), lens)
    q = single(len(lens), n, 16, d, dtype, 2 * math.sqrt(d))
    assert_rounded(st, q, st.c.attention(q, st.lens()))


@pytest.mark.parametrize("d,n", [(64, 1), (128, 3)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,size", [("bf16", 1e-6), ("bf16", 1e-8), ("bf16", 1e-28), ("fp16", 1e-6), ("fp16", 1.0)])
def test_blocks_of_zeros_take_nothing_from_small_values(fmt, dtype, size, d, n):
    """Whole blocks of small values between blocks of zeros, whose scale is 1."""
    b = 240                                                 # so many that a unit's tiles lie in one CTA's run
    st = Stream(b, 2, d, 320, fmt, dtype)
    k, v = values(3, (3, 320, 2, d), dtype), (values(4, (3, 320, 2, d), dtype).float() * size).to(DT[dtype])
    v[:, 64:128], v[1, :64], v[2, 256:] = 0, -1e-39, 0      # what is below 2^-100 is stored as zeros, of either sign
    st.append(0, 320, k=k.repeat(b // 3, 1, 1, 1), v=v.repeat(b // 3, 1, 1, 1))
    q = single(b, n, 16, d, dtype, 2 * math.sqrt(d))
    assert_rounded(st, q, st.c.attention(q, st.lens()), only=[0, 1, 2, 118, 239])


def test_only_zeros():
    st = Stream(3, 2, 64, 192, "int8", "bf16")
    k = values(5, (3, 190, 2, 64), "bf16")
    st.append(0, 190, [190, 128, 30], k=k, v=torch.zeros_like(k))
    assert not st.c.attention(single(3, 2, 8, 64, "bf16", 16.0), st.lens()).any()


@pytest.mark.parametrize("d,n", [(64, 1), (128, 3)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,size", [("bf16", 1e-6), ("bf16", 1e-8), ("bf16", 1e-28), ("bf16", 1e-38), ("bf16", 1e30),
                                        ("fp16", 1e-6), ("fp16", 1e-3), ("fp16", 500.0)])
def test_the_open_block_takes_nothing_from_small_values(fmt, dtype, size, d, n):
    """Small and large values in whole blocks and the open one, whose values
    are their own codes; one warp's share of the open block is zeros."""
    b = 240                                                 # so many that a unit's tiles lie in one CTA's run
    st = Stream(b, 2, d, 320, fmt, dtype)
    k, v = values(6, (3, 249, 2, d), dtype), (values(7, (3, 249, 2, d), dtype, False).float() * size).to(DT[dtype])
    v[:, 208:224] = 0
    st.append(0, 249, [249, 192, 40] * (b // 3), k=k.repeat(b // 3, 1, 1, 1), v=v.repeat(b // 3, 1, 1, 1))
    q = single(b, n, 16, d, dtype, 2 * math.sqrt(d))
    assert_rounded(st, q, st.c.attention(q, st.lens()), only=[0, 1, 2, 118, 239])


@pytest.mark.parametrize("d,n", [(64, 1), (128, 3)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("large", [2.0 ** 10, 2.0 ** 20, 2.0 ** 24])
def test_a_large_query_element_takes_nothing_from_the_others(fmt, large, d, n):
    """bf16 queries with an element that meets only zero keys."""
    st = Stream(2, 2, d, 256, fmt, "bf16")
    k = values(8, (2, 250, 2, d), "bf16")
    k[..., 5] = 0
    st.append(0, 250, [250, 130], k=k, v=values(9, (2, 250, 2, d), "bf16"))
    q = values(10, (2, n, 16, d), "bf16", False)
    q[..., 5] = large
    q = q.cuda()
    assert_rounded(st, q, st.c.attention(q, st.lens()))


@pytest.mark.parametrize("d,n", [(64, 1), (128, 3)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("sigma", [0.01, 1.0, 30.0, -30.0])
def test_large_logits_that_do_not_differ(fmt, dtype, d, n, sigma):
    """Tokens with the same key, beside one so far away that it weighs nothing:
    the softmax is flat however large its logits are (sigma 10^6 at most)."""
    st = Stream(4, 2, d, 8192, fmt, dtype)
    k = torch.zeros(4, 8192, 2, d, dtype=DT[dtype])
    k[..., 0], k[..., 1] = 100.0, 300.0
    k[:, 70, :, 0] = -100.0 if sigma > 0 else 300.0
    st.append(0, 8192, [64, 192, 40, 8192], k=k, v=values(11, (4, 8192, 2, d), dtype))
    q = torch.zeros(4, n, 8, d, dtype=DT[dtype])
    q[..., 0] = 333.0
    q = q.cuda()
    rows = [min(n, 1)] * 4
    out = st.c.attention(q, st.lens(), torch.tensor(rows, dtype=torch.int32, device="cuda"), softmax_scale=sigma)
    assert_rounded(st, q, out, rows, sigma, alike=True)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("length", [1, 40, 64, 200, 4000])
def test_an_infinite_query_over_keys_of_one_sign_is_no_number(dtype, length):
    """Logits of -inf alone have no softmax; a query without tokens gives zeros."""
    st = Stream(1, 1, 64, 4032, "int8", dtype)
    k = torch.full((1, length, 1, 64), -1.0, dtype=DT[dtype])
    st.append(0, length, k=k, v=values(12, (1, length, 1, 64), dtype))
    q = torch.zeros(1, 3, 4, 64, dtype=DT[dtype])
    q[:, :, 1, 7] = math.inf
    q[:, :, 2, 9] = -math.inf
    out = st.c.attention(q.cuda(), st.lens()).cpu()
    seen = torch.tensor([length - 2, length - 1, length]) > 0
    assert torch.isnan(out[0, seen][:, 1:3]).all() and torch.isfinite(out[0, :, [0, 3]]).all()
    assert not out[0, ~seen].any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,n", [(64, 1), (128, 3)])
def test_a_flat_softmax_errs_by_its_own_rounding(fmt, d, n):
    """fp16, 2000 tokens of either sign that weigh nearly alike: |o| is some
    sqrt(2000) under sum w |v|, so an error of each weight shows.  Float32's
    errors are random, sqrt(2000 / 16 + 64) of 2^-24 of that sum or 2^-15 of
    |o|, beside the result's rounding, whose steps are 2^-11 to 2^-10 of |o|,
    so 2^-12.8 to 2^-11.8 in the mean square: a quarter of it at most, 1.03 for
    both together.  Weights of 11 bits err as much as the rounding does: 1.4."""
    st = Stream(2, 2, d, 2048, fmt, "fp16")
    st.append(13, 2000, [2000, 1920])
    q = values(14, (2, n, 8, d), "fp16", False).cuda()
    got = st.c.attention(q, st.lens(), softmax_scale=0.01).double().cpu().numpy()
    err, own = 0.0, 0.0
    for i in range(2):
        for u in range(2):
            (ck, sk), (cv, sv) = ((c[u], s[u]) for c, s in (st.stored("k", i), st.stored("v", i)))
            o, _ = O.attention(q[i, :, 4 * u:4 * u + 4].double().cpu().numpy(), ck * sk[:, None], cv * sv[:, None], 0.01)
            err += ((got[i, :, 4 * u:4 * u + 4] - o) ** 2).sum()
            own += ((o.astype(np.float16) - o) ** 2).sum()
    assert err <= 1.1 ** 2 * own


@pytest.mark.parametrize("length", [192, 8000])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_small_values_with_small_weights(fmt, length):
    """Values of 2^-95 behind a block of zeros that takes all but 2^-29 of the
    weight: the results are bf16 numbers, their factor alone no float32."""
    st = Stream(2, 2, 64, 8000, fmt, "bf16")
    k, v = values(15, (2, length, 2, 64), "bf16", False), values(16, (2, length, 2, 64), "bf16")
    k[:, 64:128] = 11.0
    v = (v.float() * 2.0 ** -95).bfloat16()
    v[:, 64:128] = 0
    st.append(0, length, k=k, v=v)
    q = single(2, 1, 16, 64, "bf16", 16.0)
    out = st.c.attention(q, st.lens())
    assert out.any(-1).all()
    assert_rounded(st, q, out)


@pytest.mark.parametrize("d,n", [(64, 1), (128, 3)])
@pytest.mark.parametrize("last", ["zeros", "one element", "small"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_the_open_block_of_small_values_takes_the_weight(fmt, last, d, n):
    """Whole blocks of values of 2^-95 with 2^-33 of the weight; the rest lies on
    the open block, whose values are zeros, zeros but for one element of its
    tokens, or as small."""
    st = Stream(2, 2, d, 256, fmt, "bf16")
    k, v = values(17, (2, 250, 2, d), "bf16", False), (values(18, (2, 250, 2, d), "bf16").float() * 2.0 ** -95).bfloat16()
    k[:, 192:] = 11.5
    if last == "zeros":
        v[:, 192:] = 0
    if last == "one element":
        v[:, 192:, :, 1:] = 0
    st.append(0, 250, k=k, v=v)
    q = single(2, n, 16, d, "bf16", 2 * math.sqrt(d))
    out = st.c.attention(q, st.lens())
    assert out.any(-1).all()
    assert_rounded(st, q, out)
