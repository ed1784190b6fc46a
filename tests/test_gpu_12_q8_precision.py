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


def float32_bound(w, q, ck, sk, cv, sv, sigma):
    """|error| [n, G, d] of a result before it is rounded to its type.  With
    A = sum_p w_p |v_p|:

    * a logit sums as many exact products as q has elements that are not zero,
      each addition off by at most 2^-23 of sum |q k|, with four roundings
      around it; an error e of a logit changes a weight by 2 e (its exponential
      and the denominator's);
    * a weight in two fp16 parts is off by 2^-11 of 2^-11; exponentials by
      2^-22 each, of the weight, of a reference's move, of the join and of the
      result's factor; a block's scale, as a logarithm, by 2^-22 of it;
    * sums: (L / 16 + 64) additions of 2^-23;
    * a weight's last fp16 part ends at 2^-25, where the row's largest
      w_p scale_p stands at 2^7 or above, times |code|.
    """
    v = cv * sv[:, None]
    length = len(sv)
    qk = np.einsum("ngd,ld->ngl", np.abs(q), np.abs(ck)) * sk * abs(sigma)
    e = ((np.count_nonzero(q, axis=-1)[..., None] + 4) * 2.0 ** -23 * qk).max(-1)[..., None]
    a = w @ np.abs(v)
    live = sv[np.abs(cv).max(-1) > 0]
    logs = np.abs(np.log2(live)).max() if len(live) else 0.0
    ref = (w * sv).max(-1)[..., None]
    return (a * (2 * e + 2.0 ** -22 * (5 + logs) + (length / 16 + 64) * 2.0 ** -23)
            + 2.0 ** -32 * ref * np.abs(cv).sum(0))


def half_step(x, dtype):
    """Half the distance of neighbours of the type at |x|."""
    t = torch.finfo(DT[dtype])
    _, e = np.frexp(np.maximum(np.abs(x), t.smallest_normal))
    return np.ldexp(t.eps / 2, e - 1)


def assert_rounded(st, q, out, rows=None, sigma=0.0):
    """Every result of rows is the oracle's, rounded, but for float32_bound."""
    b, h, d = st.shape
    n, hq = q.shape[1:3]
    g = hq // h
    got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
    sig = sigma or 1 / math.sqrt(d)
    for i in range(b):
        r = n if rows is None else rows[i]
        for u in range(h):
            heads = slice(u * g, (u + 1) * g)
            (ck, sk), (cv, sv) = ((c[u], s[u]) for c, s in (st.stored("k", i), st.stored("v", i)))
            o, w = O.attention(qd[i, :r, heads], ck * sk[:, None], cv * sv[:, None], sig)
            lim = float32_bound(w, qd[i, :r, heads], ck, sk, cv, sv, sig)
            over = np.abs(got[i, :r, heads] - o) - half_step(np.abs(o) + lim, st.dtype) - lim
            assert (over <= 0).all(), (i, u, int((over > 0).sum()), float((over / lim).max()))
    assert st.c.get_status() == 0


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
    q = torch.zeros(len(lens), n, 16, d, dtype=DT[dtype])
    at = torch.arange(len(lens) * n * 16).view(len(lens), n, 16, 1) % d
    q.scatter_(3, at, 2 * math.sqrt(d))
    q = q.cuda()
    assert_rounded(st, q, st.c.attention(q, st.lens()))
