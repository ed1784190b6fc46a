"""Calls that the 8-bit cache's contracts allow, beside the ordinary ones."""
import threading

import numpy as np
import pytest
import torch

from compressed_decode_attention_encode_b200 import tq
from oracle import q8_oracle as O
from tests.test_gpu_11_q8 import INT, Stream, rope_bound, run_attention, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("hq,h", [(3, 0), (0, 3), (1, 0), (0, 1), (5, 0), (0, 5)])
def test_norm_rope_of_one_side_with_its_weight(hq, h, dtype, d):
    """Queries alone or keys alone, whose heads leave lanes of a warp idle."""
    x = values(100, (2, 3, hq + h, d), dtype).cuda()
    w = values(101, (d,), dtype, False).cuda()
    pos, f = torch.arange(6, **INT).view(2, 3), torch.linspace(0, 1, d // 2, device="cuda")
    q_out, k_out = tq.qk_norm_rope(x[:, :, :hq], x[:, :, hq:], pos, f, w if hq else None, w if h else None, eps=1e-5)
    got = (q_out if hq else k_out.transpose(1, 2)).double().cpu().numpy()
    xs, ws = x.double().cpu().numpy(), w.double().cpu().numpy()
    want = O.norm_rope(xs, pos.cpu().numpy(), f.cpu().numpy(), ws, 1e-5)
    flat = O.norm_rope(xs, np.zeros((2, 3)), f.cpu().numpy(), ws, 1e-5)
    assert (np.abs(got - want) <= rope_bound(want, flat, ws, dtype)).all()


def test_threads_share_a_cache_and_a_stream():
    """Calls of several host threads on one cache, one stream and one scratch,
    each with units that many CTAs share: every one gives what it gives alone."""
    st = Stream(1, 2, 128, 8192, "int8", "fp16")
    st.append(110, 8100)
    lens = st.lens()
    qs = [values(111 + i, (1, 1 + i, 8, 128), "fp16", False).cuda() for i in range(4)]
    want = [st.c.attention(q, lens) for q in qs]
    scratch = torch.empty(max(st.c.scratch_bytes(8, 1 + i) for i in range(4)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    wrong = [None] * 4

    def calls(i):
        outs = [st.c.attention(qs[i], lens, scratch=s) for _ in range(200) for s in (None, scratch)]
        torch.cuda.synchronize()
        wrong[i] = sum(not torch.equal(o, want[i]) for o in outs)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0] * 4 and st.c.get_status() == 0


def test_layers_share_a_streams_scratch():
    """Twenty caches on one stream, and their calls in turn with growing
    numbers of queries: one buffer, and every call as with scratch of its own."""
    sts = [Stream(1, 2, 64, 4096, "int8", "fp16") for _ in range(20)]
    for i, st in enumerate(sts):
        st.append(120 + i, 4000 - 150 * i)
    qs = [values(140 + i, (1, 1 + 2 * i, 8, 64), "fp16", False).cuda() for i in range(3)]
    side = torch.cuda.Stream()
    need = max(st.c.scratch_bytes(8, 5) for st in sts)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        outs = [torch.empty_like(q) for q in qs for _ in sts]
        lens = [st.lens() for st in sts]
        held = torch.cuda.memory_allocated()
        for i, q in enumerate(qs):
            for j, st in enumerate(sts):
                st.c.attention(q, lens[j], out=outs[20 * i + j])
        assert torch.cuda.memory_allocated() - held <= need + 512
        for i, q in enumerate(qs):
            for j, st in enumerate(sts):
                own = torch.empty(st.c.scratch_bytes(8, 1 + 2 * i), dtype=torch.uint8, device="cuda")
                assert torch.equal(st.c.attention(q, lens[j], scratch=own), outs[20 * i + j])


def assert_held(st):
    """What is read back is the oracle's, bit for bit, of the tokens appended."""
    b, h, d = st.shape
    got = st.c.read(st.lens(), 0, max(st.len + [1]))
    for w, x in zip("kv", got):
        for i, n in enumerate(st.len):
            for u in range(h):
                codes, scales = O.held(st.x[w][i][u, :n].double().numpy(), n, st.fmt)
                want = torch.from_numpy(codes.astype(np.float32) * scales.astype(np.float32)[:, None]).to(x.dtype)
                assert torch.equal(x[i, u, :n].cpu(), want), (w, i, u)


@pytest.mark.parametrize("seed", range(4))
def test_rows_set_back_again_and_again(seed):
    """Random appends and set-backs of three rows, within 64 tokens of the
    greatest length since the last set-back to a multiple of 64, or to one."""
    g = np.random.default_rng(seed)
    st = Stream(3, 1, 64, 1024, "e4m3" if seed % 2 else "int8", "bf16" if seed % 2 else "fp16")
    base, most = [0] * 3, [0] * 3
    for step in range(25):
        rows = [int(g.choice([0, 1, 5, 63, 64, 100, 150])) for _ in range(3)]
        rows = [min(r, 1024 - n) for r, n in zip(rows, st.len)]
        st.append(1000 * seed + step, max(rows + [1]), rows)
        most = [max(m, n) for m, n in zip(most, st.len)]
        assert_held(st)
        run_attention(st, step, 2, 4)
        for i in range(3):
            if g.random() < 0.15:
                base[i] = most[i] = st.len[i] = 64 * int(g.integers(0, st.len[i] // 64 + 1))
            elif g.random() < 0.7:
                st.len[i] = int(g.integers(min(st.len[i], max(base[i], most[i] - 64)), st.len[i] + 1))
        run_attention(st, step, 2, 4)
