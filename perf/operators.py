"""Cases of the 8-bit cache's operators and of the norm and rotation before it.

Four operators, each in its plain form (elementary torch operations in 32 bits, ``own`` false) and
as a user of the library calls it (``own`` true):

* ``append``     new tokens are written into a cache that keeps whole blocks of 64 tokens in 8 bits,
                 with one scale for each block and kv head, and the newest two blocks in 16 bits too;
* ``read``       a range of positions is read back to 16 bits;
* ``attention``  attention of a row's newest tokens over that cache: one at a decode step, or some
                 drafted ones together;
* ``norm_rope``  the norm of each query and key head with the rotation by position, from the model's
                 packed projection to the layouts that the caches take.

A row of length L has its first 64 floor(L / 64) tokens in 8 bits; the open block's tokens are read
from the 16-bit ring (position p in slot p mod 128).
"""
import math
import random

import torch

own = False

BLOCK = 64
RING = 128
TINY = 2.0 ** -100   # a block without a magnitude of at least this is stored as zeros
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}
# (query heads, kv heads, head dim): this repository's workloads and tests
HEADS = [(32, 8, 128), (32, 4, 64), (4, 1, 64), (6, 2, 64), (64, 8, 128), (8, 8, 128)]


def _case(op, name, heads, batch, longest, n, fmt, dtype, ragged=False, **more):
    hq, hkv, d = heads
    c = {"op": op, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "longest": longest, "n": n, "format": fmt,
         "dtype": dtype, "ragged": ragged, **more}
    if name:
        c["name"] = name
    return c


def listed():
    small, llama = (32, 4, 64), (32, 8, 128)
    return [
        # one decode step of a small model on a short context: launch latency counts
        _case("attention", "attention one short row", small, 1, 1536, 1, "int8", "fp16"),
        # the decode step that this repository's benchmark runs, 32K tokens in each of 8 rows
        _case("attention", "attention 8 rows of 32K", llama, 8, 32768, 1, "e4m3", "fp16"),
        # one long conversation: the context is split over the whole card and joined
        _case("attention", "attention one row of 131K", llama, 1, 131583, 1, "int8", "bf16"),
        # continuous batching: rows of every length, one of them empty
        _case("attention", "attention ragged 33 rows", llama, 33, 9001, 1, "e4m3", "bf16", True),
        # five drafted tokens in each row are verified at once
        _case("attention", "attention 5 drafts", llama, 16, 4109, 5, "int8", "fp16", True),
        # a decode step writes one token in each row
        _case("append", "append one token", llama, 64, 8191, 1, "e4m3", "bf16", True),
        # a chunk of a prompt, as the encode benchmark has it
        _case("append", "append a 4096 chunk", llama, 8, 4096, 4096, "int8", "fp16"),
        # prompts of several lengths in one padded batch
        _case("append", "append padded prompts", small, 13, 0, 1777, "e4m3", "fp16", True),
        # a prefix is taken out of a cache for another batch
        _case("read", "read a 4096 chunk", llama, 8, 32768, 4096, "int8", "fp16", start=8192),
        # the end of short rows, the open block among it
        _case("read", "read short rows", small, 3, 777, 700, "e4m3", "bf16", True, start=100),
        # a decode step's queries and keys
        _case("norm_rope", "norm and rotation one token", llama, 8, 32768, 1, "-", "fp16", True, norm=True, pairs="half"),
        # a prompt's queries and keys
        _case("norm_rope", "norm and rotation of a prompt", llama, 3, 131072, 4099, "-", "bf16", True, norm=True, pairs="half"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "read", "norm_rope"])
    heads = rng.choice(HEADS)
    hq, hkv, d = heads
    fmt, dtype = rng.choice(["int8", "e4m3"]), rng.choice(["fp16", "bf16"])
    batch, ragged = _spread(rng, 1, 64), rng.random() < 0.5
    most = 8 * 32768 * 8 * 128 // (batch * hkv * d)   # tokens a row, for the largest listed cost
    if op == "attention":
        n = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
        longest = _spread(rng, 1, max(2, min(131583, most // n)))
        return _case(op, None, heads, batch, longest, n, fmt, dtype, ragged)
    if op == "append":
        if rng.random() < 0.5:   # a step, or some drafted tokens, anywhere in a block
            return _case(op, None, heads, batch, _spread(rng, 1, 16384), rng.randint(1, 16), fmt, dtype, ragged)
        # a chunk of a prompt, behind whole blocks
        return _case(op, None, heads, batch, 0, _spread(rng, 17, max(18, min(8192, most // 8))), fmt, dtype, ragged)
    if op == "read":
        longest = _spread(rng, 2, max(3, min(32768, most)))
        start = rng.randrange(longest)
        n = rng.randint(1, max(1, min(longest - start + 5, most // 8)))
        return _case(op, None, heads, batch, longest, n, fmt, dtype, ragged, start=start)
    n = _spread(rng, 1, max(2, 3 * 4099 * 5120 // (batch * (hq + hkv) * d)))
    return _case(op, None, heads, batch, rng.randint(0, 131072), n, "-", dtype, ragged, norm=rng.random() < 0.7,
                 pairs=rng.choice(["half", "half", "interleaved"]))


def _lens(case):
    """Tokens in each row before the call, by the case alone."""
    b, longest = case["batch"], case["longest"]
    if not case["ragged"]:
        return [longest] * b
    out = [int(longest * (1.0 - (0.6180339887 * i) % 1.0) ** 2) for i in range(b)]
    if b >= 4:
        out[2] = 0
    if case["op"] == "attention":   # a row that has drafted tokens holds them
        out = [x if x == 0 or x >= case["n"] else case["n"] for x in out]
    return out


def _rows(case):
    """Tokens that each row appends: a padded batch has rows with fewer."""
    b, n = case["batch"], case["n"]
    if not case["ragged"] or n <= 16:
        return [n] * b
    return [max(1, int(n * (1.0 - (0.7548776662 * i) % 1.0))) for i in range(b)]


def _capacity(case):
    tokens = case["longest"] + (case["n"] if case["op"] == "append" else 0)
    return -(-(tokens + 2 * RING) // BLOCK) * BLOCK


def work(case):
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["n"]
    lens = _lens(case)
    byts, flops = 0, 0
    if case["op"] == "attention":
        for length in lens:
            blocks, rest = divmod(length, BLOCK)
            byts += hkv * (2 * d * BLOCK * blocks + 8 * blocks + 4 * d * rest) + 4 * n * hq * d
            flops += 4 * n * hq * d * length
    elif case["op"] == "append":
        for length, new in zip(lens, _rows(case)):
            first, end = length // BLOCK, (length + new) // BLOCK
            byts += hkv * 4 * d * new                                      # the new tokens
            if end > first:
                byts += hkv * (4 * d * (length % BLOCK) + (end - first) * (2 * d * BLOCK + 8))
            last = (length + new - 1) // BLOCK
            byts += hkv * 4 * d * (length + new - max(length, (last - 1) * BLOCK))   # the ring
            flops += hkv * 2 * d * 3 * (end - first) * BLOCK
    elif case["op"] == "read":
        for length in lens:
            a, e = min(case["start"], length), min(case["start"] + n, length)
            whole = max(0, min(e, length // BLOCK * BLOCK) - a)
            byts += hkv * 2 * d * (whole + 2 * (e - a - whole) + 2 * (e - a))
            flops += hkv * 2 * d * whole
    else:
        byts += case["batch"] * n * (hq + hkv) * d * 4 + 4 * case["batch"] * n + 4 * d
        flops += case["batch"] * n * (hq + hkv) * d * 7
    return {"bytes": float(max(1, byts)), "flops": float(flops)}


def _values(gen, shape, scale):
    """Cached values as this repository's workloads have them: N(0, 1) by channel scales, some channels large."""
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale


def _channels(gen, hkv, d):
    s = torch.exp(0.5 * torch.randn((hkv, 1, d), generator=gen, device="cuda"))
    return torch.where(torch.rand((hkv, 1, d), generator=gen, device="cuda") < 0.01, 10.0 * s, s)


def _by(a, number):
    """a / number as a division (torch multiplies by the reciprocal of a plain number)."""
    return a / torch.full_like(a, number)


def _quantise(blocks, fmt):
    """[..., 64, d] in 32 bits -> codes and one scale [...] for each block."""
    a = blocks.abs().amax(dim=(-1, -2))
    live = a >= TINY
    inv = torch.where(live, torch.full_like(a, TOP[fmt]) / torch.where(live, a, 1.0), 0.0)
    scale = torch.where(live, _by(a, TOP[fmt]), 1.0)
    y = blocks * inv[..., None, None]
    return (torch.round(y).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b, hq, hkv, d, n = (case[x] for x in ("batch", "hq", "hkv", "d", "n"))
    dtype, fmt, op = DTYPES[case["dtype"]], case["format"], case["op"]
    ints = dict(dtype=torch.int32, device="cuda")
    s = {"case": case, "lens": torch.tensor(_lens(case), **ints)}
    if op == "norm_rope":
        # one packed projection [batch, tokens, q heads + 2 kv heads, d], as a model computes it
        qkv = torch.randn((b, n, hq + 2 * hkv, d), generator=gen, device="cuda", dtype=torch.float32)
        qkv = (qkv * torch.exp(0.5 * torch.randn((hq + 2 * hkv, d), generator=gen, device="cuda"))).to(dtype)
        s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv]
        s["positions"] = (s["lens"][:, None] + torch.arange(n, **ints)).contiguous()
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)).float()
        for w in ("q_weight", "k_weight"):
            s[w] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype) if case["norm"] else None
        s["q_out"] = torch.empty((b, n, hq, d), dtype=dtype, device="cuda")
        s["k_out"] = torch.empty((b, hkv, n, d), dtype=dtype, device="cuda")
        if own:
            from compressed_decode_attention_encode_b200 import tq
            s["call"] = tq.qk_norm_rope
        return s
    cap = _capacity(case)
    for w in ("k", "v"):
        chan = _channels(gen, hkv, d)
        codes = torch.empty((b, hkv, cap, d), dtype=CODES[fmt], device="cuda")
        scales = torch.empty((b, hkv, cap // BLOCK), dtype=torch.float32, device="cuda")
        recent = torch.empty((b, hkv, RING, d), dtype=dtype, device="cuda")
        step = max(1, (1 << 25) // (hkv * cap * d))
        for i in range(0, b, step):
            rows = min(step, b - i)
            x = _values(gen, (rows, hkv, cap, d), chan).to(dtype).float()
            c, scales[i:i + rows] = _quantise(x.view(rows, hkv, cap // BLOCK, BLOCK, d), fmt)
            codes[i:i + rows] = c.view(rows, hkv, cap, d)
            # the ring holds the newest two blocks of each row
            length = s["lens"][i:i + rows, None].long()
            first = (length - 1).clamp(min=0) // BLOCK * BLOCK - BLOCK
            p = first + (torch.arange(RING, device="cuda") - first) % RING
            at = p.clamp(min=0)[:, None, :, None].expand(rows, hkv, RING, d)
            recent[i:i + rows] = x.gather(2, at).to(dtype)
        s[w + "_codes"], s[w + "_scales"], s[w + "_recent"] = codes, scales, recent
        if op == "append":   # the model's projections lie token by token: [batch, tokens, kv heads, d]
            s[w] = _values(gen, (b, n, hkv, d), chan.transpose(0, 1)).to(dtype).transpose(1, 2)
        if op == "read":
            s[w + "_out"] = torch.zeros((b, hkv, n, d), dtype=dtype, device="cuda")
    if op == "append":
        s["n_rows"] = torch.tensor(_rows(case), **ints)
    if op == "attention":
        s["q"] = torch.randn((b, n, hq, d), generator=gen, device="cuda", dtype=torch.float32).to(dtype)
        s["out"] = torch.empty((b, n, hq, d), dtype=dtype, device="cuda")
    if own:   # the object that a serving program keeps; it takes the tensors above as they are
        from compressed_decode_attention_encode_b200 import tq
        names = [w + x for w in ("k", "v") for x in ("_codes", "_scales", "_recent")]
        s["cache"] = tq.TQ8Cache(b, hkv, d, cap, fmt, dtype, buffers={x: s[x] for x in names})
    return s


def _dequantised(s, w, p):
    """Positions p [tokens] of every row in 32 bits: the 8-bit blocks, and the open block from the ring."""
    codes, scales, recent = s[w + "_codes"], s[w + "_scales"], s[w + "_recent"]
    x = codes.view(torch.int8)[:, :, p].view(codes.dtype).float() * scales[:, :, p // BLOCK][..., None]
    open_block = p[None, :] >= (s["lens"].long() // BLOCK * BLOCK)[:, None]
    return torch.where(open_block[:, None, :, None], recent[:, :, p % RING].float(), x)


def _plain_attention(s):
    case = s["case"]
    b, hq, hkv, d, n = (case[x] for x in ("batch", "hq", "hkv", "d", "n"))
    p = torch.arange(max(1, case["longest"]), device="cuda")
    sees = s["lens"].long()[:, None] - n + 1 + torch.arange(n, device="cuda")            # [b, n]
    seen = (p < sees[..., None])[:, None, :, None, :]                                    # [b, 1, n, 1, L]
    q = s["q"].float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)              # [b, hkv, n, g, d]
    k = _dequantised(s, "k", p)
    logits = (q.reshape(b, hkv, -1, d) @ k.transpose(-1, -2)).view(b, hkv, n, hq // hkv, -1) / math.sqrt(d)
    del k
    logits = torch.where(seen, logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    o = e.view(b, hkv, -1, len(p)) @ torch.where((p < s["lens"][:, None])[:, None, :, None], _dequantised(s, "v", p), 0.0)
    o = o.view(b, hkv, n, hq // hkv, d) / torch.where(total == 0, 1.0, total)
    return o.permute(0, 2, 1, 3, 4).reshape(b, n, hq, d).to(s["q"].dtype)


def _plain_append(s):
    case = s["case"]
    n, d = case["n"], case["d"]
    lens, rows = s["lens"].long(), s["n_rows"].long()
    end = lens + rows
    nb = (n + BLOCK - 1) // BLOCK + 1
    first = lens // BLOCK
    p = first[:, None] * BLOCK + torch.arange(nb * BLOCK, device="cuda")                 # [b, P]
    is_new = (p >= lens[:, None]) & (p < end[:, None])
    whole = (first[:, None] + torch.arange(nb, device="cuda") + 1) * BLOCK <= end[:, None]
    last = (end - 1) // BLOCK
    ring = (last - 1)[:, None] * BLOCK
    ring = ring + (torch.arange(RING, device="cuda") - ring) % RING                      # position of each slot
    ring_new = (ring >= lens[:, None]) & (ring < end[:, None])
    for w in ("k", "v"):
        new, recent, codes, scales = s[w], s[w + "_recent"], s[w + "_codes"], s[w + "_scales"]
        b, hkv = new.shape[:2]

        def at(index, size):
            return index[:, None, :, None].expand(b, hkv, index.shape[1], size)

        from_new = new.gather(2, at((p - lens[:, None]).clamp(0, n - 1), d))
        x = torch.where(is_new[:, None, :, None], from_new, recent.gather(2, at(p % RING, d)))
        c, sc = _quantise(x.float().view(b, hkv, nb, BLOCK, d), case["format"])
        raw, c = codes.view(torch.int8), c.view(b, hkv, nb * BLOCK, d).view(torch.int8)
        keep = whole.repeat_interleave(BLOCK, 1)[:, None, :, None]
        raw.scatter_(2, at(p, d), torch.where(keep, c, raw.gather(2, at(p, d))))
        blk = (first[:, None] + torch.arange(nb, device="cuda"))[:, None].expand(b, hkv, nb)
        scales.scatter_(2, blk, torch.where(whole[:, None], sc, scales.gather(2, blk)))
        fresh = new.gather(2, at((ring - lens[:, None]).clamp(0, n - 1), d))
        recent.copy_(torch.where(ring_new[:, None, :, None], fresh, recent))
    return [s[w + x] for w in ("k", "v") for x in ("_codes", "_scales", "_recent")]


def _plain_read(s):
    case = s["case"]
    p = case["start"] + torch.arange(case["n"], device="cuda")
    held = (p < s["lens"][:, None])[:, None, :, None]
    p = p.clamp(max=s["k_codes"].shape[2] - 1)
    return [torch.where(held, _dequantised(s, w, p).to(s[w + "_out"].dtype), s[w + "_out"]) for w in ("k", "v")]


def _plain_norm_rope(s):
    angle = s["positions"].double()[..., None] * s["inv_freq"].double()                  # [b, n, d / 2]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    out = []
    for w in ("q", "k"):
        x, weight = s[w].float(), s[w + "_weight"]
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        if s["case"]["pairs"] == "half":
            x0, x1 = x.chunk(2, -1)
            y = torch.cat((x0 * cos - x1 * sin, x1 * cos + x0 * sin), -1)
        else:
            x0, x1 = x[..., 0::2], x[..., 1::2]
            y = torch.stack((x0 * cos - x1 * sin, x1 * cos + x0 * sin), -1).flatten(-2)
        out.append(y.to(s[w].dtype))
    return [out[0], out[1].transpose(1, 2).contiguous()]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"attention": _plain_attention, "append": _plain_append, "read": _plain_read,
                "norm_rope": _plain_norm_rope}[op](s)
    if op == "attention":
        return s["cache"].attention(s["q"], s["lens"], out=s["out"])
    if op == "append":
        s["cache"].append(s["k"], s["v"], s["lens"], n_rows=s["n_rows"])
        return [s[w + x] for w in ("k", "v") for x in ("_codes", "_scales", "_recent")]
    if op == "read":
        return s["cache"].read(s["lens"], s["case"]["start"], out=(s["k_out"], s["v_out"]))
    return s["call"](s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"], eps=1e-6,
                     interleaved=s["case"]["pairs"] == "interleaved", q_out=s["q_out"], k_out=s["k_out"])


def exact(case, seed):
    """The definitions in 64 bits, row by row."""
    s = prepare(case, seed)
    lens = _lens(case)
    b, hq, hkv, d, n = (case[x] for x in ("batch", "hq", "hkv", "d", "n"))

    def tokens(w, row, end):
        """The first `end` tokens of a row as the cache holds them: [hkv, end, d]."""
        whole = lens[row] // BLOCK * BLOCK
        blocks = s[w + "_codes"][row, :, :whole].double().view(hkv, -1, BLOCK, d)
        x = blocks * s[w + "_scales"][row, :, :whole // BLOCK].double()[:, :, None, None]
        tail = torch.arange(whole, lens[row], device="cuda") % RING
        return torch.cat((x.reshape(hkv, whole, d), s[w + "_recent"][row][:, tail].double()), 1)[:, :end]

    if case["op"] == "attention":
        out = torch.zeros((b, n, hq, d), dtype=torch.float64, device="cuda")
        for row in range(b):
            if lens[row] == 0:
                continue
            k, v = tokens("k", row, lens[row]), tokens("v", row, lens[row])
            for i in range(n):
                end = lens[row] - n + 1 + i
                if end <= 0:
                    continue
                q = s["q"][row, i].double().view(hkv, hq // hkv, d)
                a = torch.einsum("hgd,hld->hgl", q, k[:, :end]) * d ** -0.5
                out[row, i] = torch.einsum("hgl,hld->hgd", torch.softmax(a, -1), v[:, :end]).reshape(hq, d)
        return out
    if case["op"] == "read":
        out = []
        for w in ("k", "v"):
            o = s[w + "_out"].double()
            for row in range(b):
                x = tokens(w, row, lens[row])[:, case["start"]:case["start"] + n]
                o[row, :, :x.shape[1]] = x
            out.append(o)
        return out
    if case["op"] == "append":
        out = []
        for w in ("k", "v"):
            scales, recent = s[w + "_scales"].double(), s[w + "_recent"].double()
            for row, new in enumerate(_rows(case)):
                old = torch.arange(lens[row] // BLOCK * BLOCK, lens[row], device="cuda") % RING
                x = torch.cat((s[w + "_recent"][row][:, old], s[w][row, :, :new]), 1).double()
                base = lens[row] - len(old)
                whole = x.shape[1] // BLOCK
                a = x[:, :whole * BLOCK].reshape(hkv, whole, -1).abs().amax(-1) if whole else x.new_zeros((hkv, 0))
                scales[row, :, base // BLOCK:base // BLOCK + whole] = torch.where(a >= TINY, a / TOP[case["format"]], 1.0)
                first = max(lens[row], ((lens[row] + new - 1) // BLOCK - 1) * BLOCK)
                p = torch.arange(first, lens[row] + new, device="cuda")
                recent[row][:, p % RING] = x[:, p - base]
            out += [None, scales, recent]
        return out
    out = []
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[..., None] * s["inv_freq"].double())[:, :, None]
    for w in ("q", "k"):
        x = s[w].double()
        if case["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s[w + "_weight"].double()
        if case["pairs"] == "half":
            z = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn
            y = torch.cat((z.real, z.imag), -1)
        else:
            y = torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        out.append(y)
    return [out[0], out[1].transpose(1, 2)]
