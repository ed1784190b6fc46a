"""The 8-bit cache and the norm with rotation on the GPU against the float64
oracle.

Codes, scales and the ring are compared bit for bit (the definition is in
float32 operations that are rounded once); read-back values too.  Attention
and the norm with rotation have the bounds that ``attention_bound`` and
``rope_bound`` derive.
"""
import math

import numpy as np
import pytest
import torch

from compressed_decode_attention_encode_b200 import tq
from oracle import q8_oracle as O

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
INT = dict(dtype=torch.int32, device="cuda")


def values(seed, shape, dtype, outliers=True):
    """16-bit values with channel scales as cached keys have them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if outliers:
        s = torch.exp(0.5 * torch.randn(shape[-1], generator=g))
        s[torch.randint(shape[-1], (1,), generator=g)] *= 10
        x = x * s
    return x.to(DT[dtype])


class Stream:
    """A cache on the GPU beside the tokens that were appended to it."""

    def __init__(self, b, h, d, cap, fmt, dtype):
        self.c = tq.TQ8Cache(b, h, d, cap, fmt, DT[dtype])
        self.fmt, self.dtype, self.shape = fmt, dtype, (b, h, d)
        for t in (self.c.k_recent, self.c.v_recent):       # what was never written is never used
            t.fill_(float("nan"))
        self.c.k_scales.fill_(float("nan")), self.c.v_scales.fill_(float("nan"))
        self.c.k_codes.view(torch.uint8).fill_(0x7f), self.c.v_codes.view(torch.uint8).fill_(0x7f)
        self.len = [0] * b
        self.x = {"k": [torch.empty(h, 0, d, dtype=DT[dtype]) for _ in range(b)],
                  "v": [torch.empty(h, 0, d, dtype=DT[dtype]) for _ in range(b)]}

    def lens(self):
        return torch.tensor(self.len, **INT)

    def append(self, seed, n, rows=None, outliers=True, k=None, v=None):
        b, h, d = self.shape
        k = values(2 * seed, (b, n, h, d), self.dtype, outliers) if k is None else k
        v = values(2 * seed + 1, (b, n, h, d), self.dtype, outliers) if v is None else v
        self.c.append(k.cuda().transpose(1, 2), v.cuda().transpose(1, 2), self.lens(),
                      None if rows is None else torch.tensor(rows, **INT))
        for i in range(b):
            r = n if rows is None else rows[i]
            for w, t in (("k", k), ("v", v)):
                self.x[w][i] = torch.cat((self.x[w][i][:, :self.len[i]], t[i, :r].transpose(0, 1)), 1)
            self.len[i] += r

    def check(self):
        """Codes, scales and ring bit for bit."""
        assert self.c.get_status() == 0
        for w in "kv":
            codes = getattr(self.c, w + "_codes").float().cpu().numpy()
            scales = getattr(self.c, w + "_scales").cpu().numpy()
            ring = getattr(self.c, w + "_recent").cpu()
            for i, n in enumerate(self.len):
                x = self.x[w][i]
                whole = n // 64
                c, s = O.quantise_block(x[:, :64 * whole].float().numpy().reshape(x.shape[0], whole, 64, x.shape[2]), self.fmt)
                np.testing.assert_array_equal(scales[i, :, :whole], s)
                np.testing.assert_array_equal(codes[i, :, :64 * whole].reshape(c.shape), c)
                p = torch.arange(max(0, ((n - 1) // 64 - 1) * 64), n)
                assert torch.equal(ring[i][:, p % 128].view(torch.int16), x[:, p].view(torch.int16))

    def stored(self, w, i):
        """(codes' values, scales) [h, len, d], [h, len] in float64, from the GPU's own records."""
        n = self.len[i]
        whole = n // 64 * 64
        c = getattr(self.c, w + "_codes")[i, :, :whole].double().cpu().numpy()
        s = getattr(self.c, w + "_scales")[i, :, :whole // 64].double().cpu().numpy()
        p = torch.arange(whole, n, device="cuda") % 128
        t = getattr(self.c, w + "_recent")[i][:, p].double().cpu().numpy()
        h = c.shape[0]
        return np.concatenate((c, t), 1), np.concatenate((np.repeat(s, 64, 1), np.ones((h, n - whole))), 1)


def attention_bound(o, w, q, ck, sk, cv, sv, sigma, dtype):
    """|error| that the kernel may have in each output [n, G, d].

    With A = sum_p w_p |v_p| (v = code scale):
    * a logit is a sum of d exact products in float32, each addition off by at
      most 2^-23 of sum |q k| (rounding or truncation), then three float32
      roundings of it; bf16 queries enter as fp16 after a power of two, elements
      below 2^-14 of the largest off by 2^-25 of it.  A logit error e changes a
      weight by 2 e relative (its exponential and the sum's);
    * the exponential, the block's scale in the logit (a float32 logarithm) and
      the sums: 2^-20 relative, and (L / 16 + 64) additions of 2^-23;
    * a weight enters the second product as fp16: half a step, 2^-11 relative;
      below fp16's normal range 2^-25 of a reference that is at most the largest
      w_p scale_p, times |code|;
    * the result is rounded to the output type.
    """
    n, g, d = q.shape
    length = ck.shape[0]
    sigma = abs(sigma)                                     # a bound of magnitudes
    v = cv * sv[:, None]
    u = torch.finfo(DT[dtype]).eps / 2
    qk = np.einsum("ngd,ld->ngl", np.abs(q), np.abs(ck)) * sk * sigma
    low = np.abs(q).max(-1)[..., None] * 2.0 ** -25 * (np.abs(ck).sum(-1) * sk * sigma)
    e = ((d + 4) * 2.0 ** -23 * qk + low).max(-1)[..., None] if length else 0.0
    a = w @ np.abs(v)
    ref = (w * sv).max(-1, initial=0.0)[..., None]
    return (u * np.abs(o) + a * (2.0 ** -11 + 2 * e + 2.0 ** -20 + (length / 16 + 64) * 2.0 ** -23)
            + 2.0 ** -25 * ref * np.abs(cv).sum(0) + 2.0 ** -25)


def check_attention(st, q, out, rows=None, sigma=0.0, before=None, only=None):
    b, h, d = st.shape
    n, hq = q.shape[1], q.shape[2]
    g = hq // h
    got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
    sig = sigma or 1 / math.sqrt(d)
    for i in range(b) if only is None else only:
        r = n if rows is None else rows[i]
        for u in range(h):
            heads = slice(u * g, (u + 1) * g)
            (ck, sk), (cv, sv) = ((c[u], s[u]) for c, s in (st.stored("k", i), st.stored("v", i)))
            o, w = O.attention(qd[i, :r, heads], ck * sk[:, None], cv * sv[:, None], sig)
            lim = attention_bound(o, w, qd[i, :r, heads], ck, sk, cv, sv, sig, st.dtype)
            err = np.abs(got[i, :r, heads] - o)
            assert (err <= lim).all(), (i, u, float((err / lim).max()))
            seen = st.len[i] - r + 1 + np.arange(r) > 0
            assert not got[i, :r, heads][~seen].any()
        if before is not None:                              # behind a row's queries: as it was
            assert np.array_equal(got[i, r:], before.double().cpu().numpy()[i, r:])
    assert st.c.get_status() == 0


# ---- append and read ----------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_one_by_one_and_in_chunks_alike(fmt, dtype, d):
    a = Stream(2, 2, d, 448, fmt, dtype)
    b = Stream(2, 2, d, 448, fmt, dtype)
    for n, seed in ((1, 1), (62, 2), (1, 3), (1, 4), (127, 5), (200, 6), (3, 7)):
        a.append(seed, n)
        a.check()
    for t in range(a.len[0]):
        k, v = (torch.stack([x[:, t:t + 1] for x in a.x[w]]).transpose(1, 2) for w in "kv")
        b.append(0, 1, k=k, v=v)
    b.check()


@pytest.mark.parametrize("lens,n,rows", [
    ([0, 0, 0], 1, None), ([0, 63, 64], 1, None), ([5, 0, 127], 64, [64, 1, 0]), ([0, 60, 100], 130, [130, 129, 1]),
    ([1, 2, 3], 500, [500, 62, 63]), ([64, 128, 192], 320, [320, 64, 128]), ([63, 191, 30], 257, [257, 2, 99])])
def test_append_ragged(lens, n, rows):
    st = Stream(3, 1, 64, 768, "int8", "fp16")
    st.append(1, max(max(lens), 1), lens)
    st.check()
    st.append(2, n, rows)
    st.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_special_blocks(fmt):
    """Zeros, subnormals, the largest values, values below 2^-100, and NaN or
    infinities in one block, which leave the others as they are."""
    st = Stream(1, 7, 64, 192, fmt, "bf16")
    k = values(3, (1, 192, 7, 64), "bf16")
    k[:, :64, 0] = 0
    k[:, :64, 1] = 1e-39
    k[:, :64, 2] = k[:, :64, 2].sign() * 3.3e38
    k[:, 70, 3, 5] = float("nan")
    k[:, 70, 4, 5] = float("inf")
    k[:, 70, 5, 5] = float("-inf")
    k[:, :64, 6] *= 2.0 ** -90
    st.append(0, 192, k=k, v=k.flip(1).contiguous())
    st.check()
    kr, vr = st.c.read(st.lens(), 0, 192)
    for h in (3, 4, 5):
        assert torch.isnan(kr[0, h, 64:128]).all() and torch.isfinite(kr[0, h, :64]).all()
        assert torch.isnan(vr[0, h, 64:128]).all()
    st = Stream(1, 1, 64, 64, fmt, "fp16")
    st.append(0, 64, k=torch.full((1, 64, 1, 64), 65504.0).half(), v=torch.full((1, 64, 1, 64), 2.0 ** -24).half())
    st.check()
    kr, vr = st.c.read(st.lens(), 0, 64)
    assert (kr == 65504).all() and (vr == 2.0 ** -24).all()


@pytest.mark.parametrize("dtype,fmt,d", [("fp16", "int8", 128), ("bf16", "e4m3", 64), ("bf16", "int8", 64)])
def test_read_bit_for_bit(dtype, fmt, d):
    st = Stream(3, 2, d, 384, fmt, dtype)
    st.append(4, 300, [300, 0, 63])
    lens = st.lens()
    for start, n in ((0, 300), (0, 384), (250, 60), (63, 2), (299, 1), (300, 5), (383, 1), (1000, 4)):
        out = [torch.full((3, 2, n, d), 7.0, dtype=DT[dtype], device="cuda") for _ in "kv"]
        st.c.read(lens, start, out=out)
        for w, t in zip("kv", out):
            for i in range(3):
                want = torch.full((2, n, d), 7.0, dtype=DT[dtype])
                c, s = st.stored(w, i)
                x = torch.from_numpy(c.astype(np.float32) * s.astype(np.float32)[..., None]).to(DT[dtype])[:, start:start + n]
                want[:, :x.shape[1]] = x
                assert torch.equal(t[i].cpu(), want), (start, n, w, i)
    assert st.c.get_status() == 0


def test_rejected_drafts_are_set_back():
    """A row's length set back by up to 64 tokens: the codes are as if the
    rejected tokens had never been."""
    for back in (1, 5, 37, 64):
        st = Stream(1, 2, 64, 512, "e4m3", "bf16")
        st.append(1, 150)
        st.append(2, back + 3)
        st.len[0] -= back
        run_attention(st, 4, 2, 4)
        st.append(3, 100)
        st.check()
        run_attention(st, 5, 2, 4)


def test_append_refuses_rows_on_the_device():
    st = Stream(4, 1, 64, 128, "int8", "fp16")
    st.append(1, 100, [100, 10, 20, 128 - 28])
    names = [w + "_" + x for w in "kv" for x in ("codes", "scales", "recent")]
    was = {x: getattr(st.c, x).clone().view(torch.uint8) for x in names}
    k = values(9, (4, 1, 40, 64), "fp16").cuda()
    for lens, rows, code in (([100, -1, 20, 100], [0, 1, 0, 0], 1), ([100, 10, 20, 100], [29, 0, 0, 0], 3),
                             ([100, 10, 20, 100], [0, 41, 0, 0], 1), ([100, 10, 20, 100], [0, 0, -5, 0], 1),
                             ([2 ** 31 - 1, 10, 20, 100], [1, 0, 0, 0], 3)):
        st.c.append(k, k, torch.tensor(lens, **INT), torch.tensor(rows, **INT))
        assert st.c.get_status() == code and st.c.get_status() == 0
        for x in names:
            assert torch.equal(getattr(st.c, x).view(torch.uint8), was[x]), x
    st.c.append(k, k, torch.tensor([100, -1, 20, 100], **INT), torch.tensor([0, 3, 40, 0], **INT))
    assert st.c.get_status() == 1                           # the good row is written
    assert torch.equal(st.c.k_recent[2, 0, 20:60], k[2, 0])
    out = torch.full((4, 1, 3, 64), 5.0, dtype=torch.float16, device="cuda")
    st.c.read(torch.tensor([-1, 129, 3, 0], **INT), 0, out=(out, out.clone()))
    assert st.c.get_status() == 1
    assert (out[:2] == 5).all() and (out[3] == 5).all() and (out[2] != 5).any()


# ---- attention ------------------------------------------------------------------

def run_attention(st, seed, n, hq, rows=None, sigma=0.0):
    b, h, d = st.shape
    q = values(seed, (b, n, hq, d), st.dtype, False).cuda()
    before = torch.full((b, n, hq, d), 3.0, dtype=DT[st.dtype], device="cuda")
    out = st.c.attention(q, st.lens(), None if rows is None else torch.tensor(rows, **INT), out=before.clone(),
                         softmax_scale=sigma)
    check_attention(st, q, out, rows, sigma, before)
    return out


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_lengths(fmt, dtype, d):
    """Lengths at and around the block: empty, one token, the open block alone,
    whole blocks alone, both."""
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 200, 320, 449]
    st = Stream(len(lens), 2, d, 512, fmt, dtype)
    st.append(11, max(lens), lens)
    run_attention(st, 12, 1, 8)


@pytest.mark.parametrize("hq,h", [(1, 1), (6, 2), (5, 1), (8, 1), (32, 4), (9, 1), (16, 1), (32, 2)])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_attention_head_groups(hq, h, n):
    st = Stream(3, h, 64, 384, "int8", "fp16")
    st.append(13, 330, [330, 4, 190])
    run_attention(st, 14, n, hq)


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("hq,n", [(4, 8), (4, 16), (20, 1), (4, 6), (12, 2), (4, 5), (32, 1), (28, 1), (32, 2)])
def test_attention_pass_widths(hq, n, fmt, dtype):
    """One to four eights of query rows in a pass, and more than one pass."""
    st = Stream(3, 2, 128, 448, fmt, dtype)
    st.append(60, 400, [400, 66, 128])
    run_attention(st, 61, n, hq)


@pytest.mark.parametrize("n,rows", [(1, [0, 1, 1, 0]), (4, [4, 0, 2, 3]), (17, [17, 1, 16, 9]), (64, [64, 33, 0, 5]),
                                    (64, None), (33, None)])
@pytest.mark.parametrize("d,fmt,dtype", [(128, "e4m3", "bf16"), (64, "int8", "fp16")])
def test_attention_drafts(n, rows, d, fmt, dtype):
    """Several queries a row, fewer in some rows, more queries than tokens."""
    st = Stream(4, 2, d, 384, fmt, dtype)
    st.append(15, 300, [300, 40, 64, 3])
    run_attention(st, 16, n, 8, rows)


@pytest.mark.parametrize("b,length,hq,h,d", [(1, 9000, 32, 8, 128), (1, 20011, 8, 1, 64), (2, 5000, 4, 2, 128)])
@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "fp16")])
def test_attention_long(b, length, hq, h, d, fmt, dtype):
    """Rows that many CTAs share."""
    st = Stream(b, h, d, -(-length // 64) * 64, fmt, dtype)
    st.append(17, length)
    run_attention(st, 18, 1, hq)
    run_attention(st, 19, 3, hq)


def test_attention_ragged_rows():
    lens = [(977 * i * i) % 1500 for i in range(70)]
    st = Stream(70, 2, 64, 1536, "e4m3", "fp16")
    st.append(20, max(lens), lens)
    run_attention(st, 21, 1, 8)


def test_attention_most_rows():
    """1024 rows, a third of them empty; one query each, and three."""
    lens = [0 if i % 3 == 1 else (37 * i) % 200 for i in range(1024)]
    st = Stream(1024, 1, 64, 256, "int8", "fp16")
    st.append(62, max(lens), lens)
    for n in (1, 3):
        q = values(63 + n, (1024, n, 8, 64), "fp16", False).cuda()
        out = st.c.attention(q, st.lens())
        check_attention(st, q, out, only=list(range(0, 1024, 37)) + [1021, 1022, 1023])
        assert not out[1::3].any()


@pytest.mark.parametrize("sigma", [1e-4, 0.5, 4.0, -0.3])
def test_attention_scales(sigma):
    """Flat and one-hot softmaxes: weights over many orders of magnitude."""
    st = Stream(2, 2, 128, 2048, "int8", "fp16")
    st.append(22, 2000, [2000, 70])
    run_attention(st, 23, 2, 8, sigma=sigma)


def test_attention_values_of_very_different_blocks():
    """Blocks whose value scales differ by 2^24, and zero blocks."""
    st = Stream(1, 2, 64, 1024, "int8", "bf16")
    k, v = values(24, (1, 1000, 2, 64), "bf16"), values(25, (1, 1000, 2, 64), "bf16")
    for j in range(16):
        v[:, 64 * j:64 * j + 64] *= 2.0 ** (4 * (j % 7) - 12) if j % 5 else 0.0
        k[:, 64 * j:64 * j + 64] *= 0.0 if j == 9 else 1.0
    st.append(0, 1000, k=k, v=v)
    run_attention(st, 26, 2, 4)


@pytest.mark.parametrize("magnitude", [1e-30, 1e-6, 3000.0, 1e30])
def test_attention_query_magnitudes(magnitude):
    """bf16 queries beyond fp16's range; the scale brings the logits back."""
    st = Stream(1, 1, 64, 512, "int8", "bf16")
    st.append(27, 400)
    q = (values(28, (1, 1, 4, 64), "bf16", False).float() * magnitude).bfloat16().cuda()
    sigma = float(np.float32(0.125 / magnitude))
    check_attention(st, q, st.c.attention(q, st.lens(), softmax_scale=sigma), sigma=sigma)


def test_attention_bad_tokens_reach_only_who_sees_them():
    for fmt in ("int8", "e4m3"):
        st = Stream(2, 2, 64, 256, fmt, "fp16")
        k, v = values(29, (2, 200, 2, 64), "fp16"), values(30, (2, 200, 2, 64), "fp16")
        v[0, 198, 0, 3] = float("inf")                      # the open block: the newest two queries see it
        k[1, 199, 1, 3] = float("nan")                      # the newest one
        v[1, 70, 0, 0] = float("nan")                       # a whole block: every query
        st.append(0, 200, k=k, v=v)
        q = values(31, (2, 4, 4, 64), "fp16", False).cuda()
        out = st.c.attention(q, st.lens())
        bad = torch.isnan(out).all(-1).cpu()
        want = torch.zeros(2, 4, 4, dtype=torch.bool)
        want[0, 2:, :2] = True
        want[1, 3:, 2:] = True
        want[1, :, :2] = True
        assert torch.equal(bad, want)
        assert torch.equal(torch.isfinite(out).all(-1).cpu(), ~want)
        ck = [st.stored(w, 0) for w in "kv"]
        o, w = O.attention(q[0, :, 2:].double().cpu().numpy(), *[c[1] * s[1][:, None] for c, s in ck])
        lim = attention_bound(o, w, q[0, :, 2:].double().cpu().numpy(), ck[0][0][1], ck[0][1][1], ck[1][0][1],
                              ck[1][1][1], 0.125, "fp16")
        assert (np.abs(out[0, :, 2:].double().cpu().numpy() - o) <= lim).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_bad_queries_stay_their_own(dtype, bad):
    """A head whose query is no number gives NaN, its neighbours what they gave."""
    st = Stream(1, 2, 64, 256, "int8", dtype)
    st.append(70, 200)
    q = values(71, (1, 3, 8, 64), dtype, False).cuda()
    a = st.c.attention(q, st.lens())
    q[0, 1, 2, 7] = bad
    b = st.c.attention(q, st.lens())
    keep = torch.ones(1, 3, 8, dtype=torch.bool)
    keep[0, 1, 2] = False
    assert torch.isnan(b[~keep.cuda()]).all() and torch.equal(a[keep.cuda()], b[keep.cuda()])


def test_attention_in_place():
    """out may be q: units in one CTA's run and units that many share."""
    st = Stream(2, 2, 64, 8192, "e4m3", "bf16")
    st.append(72, 8000, [8000, 30])
    q = values(73, (2, 3, 8, 64), "bf16", False).cuda()
    want = st.c.attention(q, st.lens())
    assert st.c.attention(q, st.lens(), out=q) is q and torch.equal(q, want)


def test_attention_refuses_rows_on_the_device():
    st = Stream(4, 1, 64, 128, "int8", "fp16")
    st.append(32, 100, [100, 10, 20, 30])
    q = values(33, (4, 2, 4, 64), "fp16", False).cuda()
    for lens, rows, bad in (([100, -1, 20, 30], [2, 2, 2, 2], 1), ([100, 10, 129, 30], [2, 2, 2, 2], 2),
                            ([100, 10, 20, 30], [2, 2, 2, 3], 3), ([100, 10, 20, 30], [-1, 2, 2, 2], 0)):
        out = st.c.attention(q, torch.tensor(lens, **INT), torch.tensor(rows, **INT))
        assert st.c.get_status() == 1 and st.c.get_status() == 0
        assert torch.isnan(out[bad]).all()
        # the other rows' tiles are split over the card by the lengths that are valid: another order of
        # the same sums, which the bound holds for
        check_attention(st, q, out, only=[i for i in range(4) if i != bad])


def test_attention_query_strides_streams_and_repeats():
    """Queries as a slice of a packed projection, one token without its
    dimension, another stream, a scratch of the caller's; and the same bits
    every time."""
    st = Stream(2, 2, 128, 4096, "e4m3", "bf16")
    st.append(34, 4001, [4001, 1000])
    qkv = values(35, (2, 3, 12, 128), "bf16", False).cuda()
    q, lens = qkv[:, :, :8], st.lens()
    a = st.c.attention(q, lens)
    check_attention(st, q, a)
    one = st.c.attention(q[:, 2], lens)
    check_attention(st, q[:, 2:], one[:, None])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    scratch = torch.full((st.c.scratch_bytes(8, 3),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        b = st.c.attention(q, lens, stream=side)
        c = st.c.attention(q, lens, scratch=scratch)
        side.synchronize()
        assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(tq.TQError):
        st.c.attention(q, lens, scratch=scratch[:-256])


def test_append_padded_beyond_the_capacity():
    """A padded batch may be wider than the cache; the rows' own counts decide."""
    st = Stream(2, 1, 64, 128, "int8", "fp16")
    st.append(80, 300, [128, 5])
    st.check()
    st.c.append(*[torch.zeros(2, 1, 300, 64, dtype=torch.float16, device="cuda")] * 2, st.lens(), torch.tensor([1, 3], **INT))
    assert st.c.get_status() == 3


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_offsets_beyond_32_bits(fmt):
    """The last of 40 rows of 2^20 tokens, its codes 5 GB behind the first's,
    beside a like cache that holds it in its first row: the same plan, the same
    bits."""
    b, cap, d = 40, 2 ** 20, 128
    last, first = (tq.TQ8Cache(b, 1, d, cap, fmt) for _ in range(2))
    where = ((last, b - 1), (first, 0))
    g = torch.Generator("cuda").manual_seed(0)
    for w in "kv":
        raw = torch.randint(0, 120, (cap, d), generator=g, dtype=torch.uint8, device="cuda")
        for c, r in where:
            getattr(c, w + "_codes")[r, 0].view(torch.uint8).copy_(raw)
            getattr(c, w + "_scales")[r, 0] = torch.linspace(0.5, 2.0, cap // 64, device="cuda") / 50
            getattr(c, w + "_recent").fill_(0.25)
    n = cap - 70
    k, v = values(1, (1, 1, 65, d), "fp16").cuda(), values(2, (1, 1, 65, d), "fp16").cuda()
    q = values(3, (1, 2, 4, d), "fp16", False).cuda()
    got = []
    for c, r in where:
        lens, rows = torch.zeros(b, **INT), torch.zeros(b, **INT)
        lens[r], rows[r] = n, 65
        c.append(k.expand(b, -1, -1, -1), v.expand(b, -1, -1, -1), lens, rows)
        lens[r] += 65
        out = c.attention(q.expand(b, -1, -1, -1), lens)
        x = c.read(lens, n - 100, 165)
        others = [i for i in range(b) if i != r]
        assert out[r].isfinite().all() and not out[others].any() and not any(y[others].any() for y in x)
        assert c.get_status() == 0
        got.append([out[r], x[0][r], x[1][r], *[getattr(c, y)[r].view(torch.uint8) for y in
                    ("k_codes", "v_codes", "k_scales", "v_scales", "k_recent", "v_recent")]])
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_nothing_to_attend_to():
    """All rows empty: zeros; no queries in any row: out as it was."""
    for b in (3, 40):
        st = Stream(b, 2, 64, 128, "int8", "fp16")
        q = values(84, (b, 2, 4, 64), "fp16", False).cuda()
        out = st.c.attention(q, st.lens(), out=torch.full_like(q, 5.0))
        assert not out.any()
        st.append(85, 100)
        out = st.c.attention(q, st.lens(), torch.zeros(b, **INT), out=torch.full_like(q, 5.0))
        assert (out == 5).all() and st.c.get_status() == 0


def test_append_strides_of_their_own_and_another_stream():
    """k token by token, v head by head, on a side stream; a broadcast head."""
    st = Stream(2, 3, 64, 256, "e4m3", "fp16")
    k, v = values(86, (2, 70, 3, 64), "fp16"), values(87, (2, 3, 70, 64), "fp16")
    side = torch.cuda.Stream()
    kd, vd, lens = k.cuda(), v.cuda(), st.lens()
    torch.cuda.synchronize()
    st.c.append(kd.transpose(1, 2), vd, lens, stream=side)
    for w, t in (("k", k.transpose(1, 2)), ("v", v)):
        st.x[w] = list(t)
    st.len = [70, 70]
    side.synchronize()
    st.check()
    out = st.c.read(torch.tensor(st.len, **INT), 60, 10, stream=side)
    side.synchronize()
    assert torch.equal(out[0][:, :, 4:].cpu(), k.transpose(1, 2)[:, :, 64:]) and torch.equal(out[1][:, :, 4:].cpu(), v[:, :, 64:])
    one = kd[:, :, :1].transpose(1, 2).expand(-1, 3, -1, -1)
    st.c.append(one, one, lens)
    assert all(torch.equal(st.c.k_recent[:, h, 64:70], kd[:, 64:, 0]) for h in range(3))


def test_a_cache_takes_over_buffers():
    a = Stream(2, 2, 64, 256, "int8", "bf16")
    a.append(88, 100, [100, 33])
    names = [w + x for w in "kv" for x in ("_codes", "_scales", "_recent")]
    b = Stream.__new__(Stream)
    b.__dict__.update(a.__dict__)
    b.c = tq.TQ8Cache(2, 2, 64, 256, "int8", torch.bfloat16, buffers={x: getattr(a.c, x) for x in names})
    b.append(89, 90, [90, 31])
    b.check()
    run_attention(b, 90, 2, 4)
    assert all(getattr(a.c, x) is getattr(b.c, x) for x in names)


def test_norm_rope_on_another_stream():
    qkv = values(92, (2, 5, 8, 64), "fp16").cuda()
    pos, f = torch.arange(5, **INT).expand(2, 5).contiguous(), torch.linspace(0, 1, 32, device="cuda")
    want = tq.qk_norm_rope(qkv[:, :, :4], qkv[:, :, 4:], pos, f)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = tq.qk_norm_rope(qkv[:, :, :4], qkv[:, :, 4:], pos, f, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


# ---- norm and rotation ------------------------------------------------------------

def rope_bound(y, x, weight, dtype):
    """float32: the sum of squares, root, division and weight are within (d / 16
    + 12) 2^-24 relative of a normed value (sums of 16 by lane, then by halves);
    cosine and sine within 2^-22, and two products and a sum of the pair; then
    one rounding to the type."""
    u = torch.finfo(DT[dtype]).eps / 2
    pair = np.abs(x).max(-1, keepdims=True)
    return u * np.abs(y) * (1 + 2.0 ** -10) + pair * 2 * (40 * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -25


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("b,n,hq,h,norm", [(1, 1, 1, 1, True), (2, 3, 32, 8, True), (3, 1, 6, 2, False), (1, 70, 33, 5, True),
                                           (2, 2, 0, 3, True), (2, 2, 3, 0, False)])
def test_norm_rope(d, dtype, interleaved, b, n, hq, h, norm):
    qkv = values(40, (b, n, hq + 2 * h, d), dtype).cuda()
    g = torch.Generator().manual_seed(41)
    pos = torch.randint(-5, 140000, (b, n), generator=g, dtype=torch.int32)
    pos.view(-1)[0] = 0
    pos.view(-1)[-1] = 2 ** 31 - 1
    f = (500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float()
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(DT[dtype]) if norm else None for _ in "qk")
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + h]
    was = qkv.clone()
    qo, ko = tq.qk_norm_rope(q, k, pos.cuda(), f.cuda(), cu(wq), cu(wk), eps=1e-5, interleaved=interleaved)
    assert torch.equal(was, qkv)
    for x, w, y in ((q, wq, qo), (k, wk, ko.transpose(1, 2))):
        x = x.double().cpu().numpy()
        ww = None if w is None else w.double().numpy()
        want = O.norm_rope(x, pos.numpy(), f.numpy(), ww, 1e-5, interleaved)
        normed = O.norm_rope(x, pos.numpy() * 0, f.numpy(), ww, 1e-5, interleaved)
        err = np.abs(y.double().cpu().numpy() - want)
        assert (err <= rope_bound(want, normed, ww, dtype)).all()


def test_norm_rope_zero_vector_and_extremes():
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 1] = 1e30                                          # its squares leave float32
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    p, f = torch.zeros(1, 2, **INT), torch.ones(32, device="cuda")
    qo, _ = tq.qk_norm_rope(q, q, p, f, w, w, eps=1e-6)
    assert not qo[0, 0].any()
    assert torch.allclose(qo[0, 1].float(), torch.ones(64, device="cuda"))
    qo, _ = tq.qk_norm_rope(q[:, :1] + 1e-30, q[:, :1], p[:, :1].contiguous(), f, w, w, eps=0.0)
    assert torch.allclose(qo.float(), torch.ones(64, device="cuda"))


# ---- together -----------------------------------------------------------------------

def test_a_decoding_run_captured_and_replayed():
    """Prompts of several lengths, then steps of two layers, each from a packed
    projection: norm and rotation, append, attention; the step is captured
    once and replayed as the rows grow past several blocks.  Every token's
    outputs equal the eager run's bit for bit, and the last ones the oracle's."""
    b, hq, h, d, cap = 3, 8, 2, 64, 512
    f = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    prompt = values(50, (2, b, 100, hq + 2 * h, d), "fp16").cuda()
    steps = values(51, (150, 2, b, 1, hq + 2 * h, d), "fp16").cuda()
    rows = torch.tensor([100, 37, 64], **INT)

    def start():
        caches = [tq.TQ8Cache(b, h, d, cap, "e4m3") for _ in range(2)]
        pos = torch.arange(100, **INT).expand(b, 100).contiguous()
        for layer, c in enumerate(caches):
            x = prompt[layer]
            _, k = tq.qk_norm_rope(x[:, :, :hq], x[:, :, hq:hq + h], pos, f, w, w)
            c.append(k, x[:, :, hq + h:].transpose(1, 2), torch.zeros(b, **INT), rows)
        return caches, rows.clone()

    def step(caches, lens, x):
        out = []
        after = lens + 1
        for layer, c in enumerate(caches):
            y = x[layer]
            q, k = tq.qk_norm_rope(y[:, :, :hq], y[:, :, hq:hq + h], lens[:, None].contiguous(), f, w, w)
            c.append(k, y[:, :, hq + h:].transpose(1, 2), lens)
            out.append(c.attention(q, after))
        lens.copy_(after)
        return out

    caches, lens = start()
    eager = [[o.clone() for o in step(caches, lens, x)] for x in steps]
    caches2, lens2 = start()
    x = steps[0].clone()
    keep = lens2.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                              # a first eager step loads every kernel
        step(caches2, lens2, x)
    torch.cuda.current_stream().wait_stream(s)
    lens2.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches2, lens2, x)
    lens2.copy_(keep)
    for t in range(150):
        x.copy_(steps[t])
        graph.replay()
        for a, e in zip(out, eager[t]):
            assert torch.equal(a, e), t
    assert torch.equal(lens, lens2) and lens.tolist() == [250, 187, 214]
    for c1, c2 in zip(caches, caches2):
        assert c1.get_status() == 0 and c2.get_status() == 0
        assert torch.equal(c1.k_codes[0, :, :192].view(torch.uint8), c2.k_codes[0, :, :192].view(torch.uint8))
    st = Stream.__new__(Stream)
    st.c, st.dtype, st.shape, st.len = caches2[1], "fp16", (b, h, d), lens2.tolist()
    y = steps[-1][1]
    q, _ = tq.qk_norm_rope(y[:, :, :hq], y[:, :, hq:hq + h], (lens2 - 1)[:, None].contiguous(), f, w, w)
    check_attention(st, q, out[1])


def test_a_forked_capture():
    """A captured step whose calls lie on two streams, after a copy and beside
    other work: rotation and append on one, a memset between them."""
    b, hq, h, d, n = 2, 8, 2, 64, 30
    st = Stream(b, h, d, 512, "int8", "fp16")
    st.append(95, 200, [200, 90])
    qkv = values(96, (b, n, hq + 2 * h, d), "fp16").cuda()
    f = torch.linspace(0, 1, d // 2, device="cuda")
    x, pos, lens, after = torch.empty_like(qkv), torch.arange(n, **INT).expand(b, n).contiguous(), st.lens(), st.lens() + n
    names = [w + y for w in "kv" for y in ("_codes", "_scales", "_recent")]

    def step(side):
        main = torch.cuda.current_stream()
        x.copy_(qkv)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q, k = tq.qk_norm_rope(x[:, :, :hq], x[:, :, hq:hq + h], pos, f)
            pad = torch.zeros(1 << 16, device="cuda")
            st.c.append(k, x[:, :, hq + h:].transpose(1, 2), lens)
        busy = x.float().sum()
        main.wait_stream(side)
        return st.c.attention(q, after), busy, pad, q, k

    side = torch.cuda.Stream()
    want = step(side)[0].clone()
    torch.cuda.synchronize()
    held = {y: getattr(st.c, y).clone() for y in names}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep = step(side)
    for _ in range(5):
        keep[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(keep[0], want)
        assert all(torch.equal(getattr(st.c, y).view(torch.uint8), t.view(torch.uint8)) for y, t in held.items())


def test_two_graphs_and_an_eager_call_at_once():
    """Calls on one cache from two graphs and the current stream, replayed side
    by side: each has its own scratch."""
    st = Stream(2, 2, 128, 8192, "int8", "fp16")
    st.append(90, 8100, [8100, 2500])
    lens = st.lens()
    qs = [values(91 + i, (2, 1 + 2 * i, 8, 128), "fp16", False).cuda() for i in range(3)]
    want = [st.c.attention(q, lens).clone() for q in qs]
    graphs, outs = [], []
    for q in qs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(st.c.attention(q, lens))
        graphs.append(g)
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(30):
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        got = st.c.attention(qs[2], lens)
        torch.cuda.synchronize()
        assert torch.equal(got, want[2]) and torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_the_compressed_cache_takes_the_rotated_keys():
    """qk_norm_rope's outputs are what tq_evict_window and
    tq_decode_attention take: a ring that holds every token gives softmax
    attention over them."""
    from tests.tq_testutil import ATTN_RTOL, rel_err
    b, hq, h, d, n = 2, 8, 2, 64, 48
    qkv = values(60, (b, n, hq + 2 * h, d), "fp16", False).cuda()
    pos = torch.arange(n, **INT).expand(b, n).contiguous()
    f = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    q, k = tq.qk_norm_rope(qkv[:, :, :hq], qkv[:, :, hq:hq + h], pos, f)
    v = qkv[:, :, hq + h:].transpose(1, 2).contiguous()
    cache = tq.TQCache(tq.make_config(b, hq, h, d, 64, 64, 3, 3, 64))
    cache.evict_window(k, v)
    got = cache.decode_attention(q[:, -1].contiguous()).double().cpu().numpy()
    assert cache.get_status() == 0
    c8 = tq.TQ8Cache(b, h, d, 64)
    c8.append(k, v, torch.zeros(b, **INT))
    got8 = c8.attention(q[:, -1], torch.full((b,), n, **INT)).double().cpu().numpy()
    for i in range(b):
        for u in range(h):
            hs = slice(u * 4, u * 4 + 4)
            o, _ = O.attention(q[i, -1:, hs].double().cpu().numpy(), k[i, u].double().cpu().numpy(),
                               v[i, u].double().cpu().numpy())
            assert (rel_err(got[i, hs], o[0]) <= ATTN_RTOL).all()
            assert (rel_err(got8[i, hs], o[0]) <= ATTN_RTOL).all()
    cache.close()


def test_rotated_queries_go_straight_into_the_compressed_decode():
    """tq_decode_attention's first kernel reads q before it waits for the
    kernel before it, which here is the one that writes q: 100 steps without a
    wait give the bits of the same steps with one after every call."""
    b, hq, h, d = 8, 32, 8, 128
    cache = tq.TQCache(tq.make_config(b, hq, h, d, 64, 64, 3, 3, 128))
    kv = values(97, (2, b, h, 64, d), "fp16", False).cuda()
    cache.evict_window(kv[0].contiguous(), kv[1].contiguous())
    qkv = values(98, (100, b, 1, hq + h, d), "fp16", False).cuda()
    f = torch.linspace(0, 1, d // 2, device="cuda")
    q, k = torch.empty(b, 1, hq, d, dtype=torch.float16, device="cuda"), torch.empty(b, h, 1, d, dtype=torch.float16, device="cuda")
    pos = torch.full((b, 1), 77, **INT)
    outs = []
    for wait in (True, False):
        out = torch.empty(100, b, hq, d, device="cuda")
        for i, x in enumerate(qkv):
            tq.qk_norm_rope(x[:, :, :hq], x[:, :, hq:], pos, f, q_out=q, k_out=k)
            if wait:
                torch.cuda.synchronize()
            cache.decode_attention(q[:, 0], out=out[i])
            if wait:
                torch.cuda.synchronize()
        outs.append(out)
    assert cache.get_status() == 0 and torch.equal(*outs)
    cache.close()
