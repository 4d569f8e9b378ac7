"""What the calls around the attention promise at their edges: products whose blocks hand their SMs to the next call, and what the
header says of bytes, angles and rows."""
import math

import numpy as np
import pytest
import torch

from helpers import parity
from layer_ref import BLK, U, matmul, rotate, values, weight

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def operands(g, M, N, K):
    w8, sw = weight(g, N, K, DEV)
    a8, _ = weight(g, M, K, DEV)
    return a8, torch.exp2(torch.randn((-(-K // BLK), M), generator=g) * 2 - 6).to(DEV), w8, sw


def test_products_have_ended_when_the_next_call_takes_their_memory(lib):
    """Products of block pairs (and of the other forms) of few K blocks, each followed at once by calls that fill the same SMs' shared
    memory with something else: what a block still had in flight when it left would show in them."""
    calls = []
    for i, (M, N, K) in enumerate([(1500, 2100, 400), (3, 4096, 256), (1111, 2345, 1232), (64, 1000, 4096), (2048, 4096, 512), (300, 900, 3200),
                                   (4000, 4000, 1040), (700, 8200, 384)]):
        a8, sa, w8, sw = operands(gen(i), M, N, K)
        out, err = torch.empty((M, N), dtype=(BF, F32)[i % 2], device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        x = torch.randn((500, 2048), generator=gen(50 + i)).to(BF).to(DEV)
        q, s, w = torch.empty((500, 2048), dtype=torch.uint8, device=DEV), torch.empty((16, 500), device=DEV), torch.ones(2048, device=DEV)
        calls.append(((a8, sa, w8, sw, out, err), (x, q, s, w)))

    def go():
        for mm, quant in calls:
            lib.kv8_matmul8(*mm[:5], err_word=mm[5])
            lib.kv8_quant_blocks(*quant[:3], norm_w=quant[3])
    for mm, quant in calls:  # each by itself
        lib.kv8_matmul8(*mm[:5], err_word=mm[5])
        torch.cuda.synchronize()
        lib.kv8_quant_blocks(*quant[:3], norm_w=quant[3])
        torch.cuda.synchronize()
    alone = [(mm[4].clone(), quant[1].clone(), quant[2].clone()) for mm, quant in calls]
    for (mm, _), (out, _, _) in zip(calls, alone):
        ref, tol = matmul(*mm[:4], out.dtype)
        assert bool(((out.double() - ref).abs() <= tol).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for turn in range(20):
        for mm, quant in calls:
            for t in (mm[4], quant[1], quant[2]):
                t.zero_()
        if turn % 2:
            graph.replay()
        else:
            go()
        torch.cuda.synchronize()
        for (mm, quant), want in zip(calls, alone):
            assert mm[5].item() == 0
            assert all(torch.equal(a, b) for a, b in zip((mm[4], quant[1], quant[2]), want))


def test_the_products_waits_run_to_their_limits(lib):
    """50 ms by the global timer, 10^8 cycles of the SM's clock (48.3 ms at its highest, 2.07 GHz) and, for the product's two waits,
    2.5 * 10^7 each: 122 ms at the least.  (A wait that did not set its abort flag or its error would leave another status.)"""
    err, st = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
    lib.kv8_wait_selftest(1000, err, st)  # (the first launch loads the kernel)
    torch.cuda.synchronize()
    assert err.item() == lib.KV8_ERR_TIMEOUT and st.item() == 2
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    err.zero_(), st.zero_()
    begin.record()
    lib.kv8_wait_selftest(50_000_000, err, st)
    end.record()
    torch.cuda.synchronize()
    assert err.item() == lib.KV8_ERR_TIMEOUT and st.item() == 2
    assert 121 < begin.elapsed_time(end) < 240


# -------------------------------------------------------------------------------------------------------------
# bytes: a normed row is quantized as the row quantizer quantizes the f32 row
# -------------------------------------------------------------------------------------------------------------
def whole_rows(g, n, width, xt):
    """Rows of whole numbers up to 15 (exact in bf16, and any order of the sum of their squares is exact in f32 and a power of two
    below 2^24), their f32 normed values as the header has them: x times the correctly rounded 1 / sqrt(mean), times w."""
    x = torch.randint(-15, 16, (n, width), generator=g).float()
    x[:, 0] += (x == 0).all(1).float()
    w = 1 + 0.3 * torch.randn(width, generator=g)
    mean = (x.double() ** 2).sum(1) / width
    inv = (1 / torch.sqrt(mean)).float()
    return x.to(xt).to(DEV), w.to(DEV), (x * inv[:, None]).to(DEV)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("width,n", [(512, 30000), (1024, 16000), (2048, 8000), (4096, 4000), (8192, 2000), (16384, 1000)])
def test_normed_blocks_are_the_row_quantizers_bytes(lib, width, n, xt):
    g = gen(width)
    x, w, xn = whole_rows(g, n, width, xt)
    w[128:256] = 1e-40  # a block whose 448 / amax overflows, beside the others
    w[384:512] = 0
    q, s = torch.empty((n, width), dtype=torch.uint8, device=DEV), torch.empty((width // BLK, n), device=DEV)
    lib.kv8_quant_blocks(x, q, s, norm_w=w, eps=0.0)
    y = (xn * w).view(n * width // BLK, BLK)
    q2, s2 = torch.empty((n * width // BLK, BLK), dtype=torch.uint8, device=DEV), torch.empty(n * width // BLK, device=DEV)
    lib.kv8_quant_rows_w(y, q2, s2)
    assert int((q.view(-1, BLK) != q2).sum()) == 0 and torch.equal(s.t().contiguous().view(-1), s2)


@pytest.mark.parametrize("xt", [BF, F32])
def test_fresh_rows_are_the_row_quantizers_bytes(lib, xt):
    """Positions of 0 turn nothing: the row that kv8_quant_rows would take is known."""
    g = gen(1)
    n = 40000
    x, w, xn = whole_rows(g, n, 512, xt)
    rope = torch.randn((n, 64), generator=g).to(xt).to(DEV) * torch.exp2(torch.randint(-3, 4, (n, 1), generator=g).float()).to(DEV).to(xt)
    pos, f, dst = torch.zeros(n, dtype=torch.int32, device=DEV), lib.kv8_rope_freqs(64)[0].to(DEV), torch.arange(n, device=DEV)
    kv8, ks = torch.empty((n, 576), dtype=torch.uint8, device=DEV), torch.empty(n, device=DEV)
    q2, s2 = torch.empty_like(kv8), torch.empty_like(ks)
    for layout in (0, 1):
        lib.kv8_norm_rope_rows(torch.cat([x, rope], 1), w, 0.0, pos, f, dst, kv8, ks, layout=layout)
        lib.kv8_quant_rows(torch.cat([xn * w, rope.float()], 1), q2, s2)
        assert int((kv8 != q2).sum()) == 0 and torch.equal(ks, s2)


@pytest.mark.parametrize("size,weight", [(1e8, 1e32), (1e-12, 1e-30), (1e17, 1e28), (1e-20, 1e-36), (2.5e38, 1.0), (1e-41, 1e3)])
def test_a_norm_before_its_weight(lib, size, weight):
    """The normed value is near 1 whatever the row's size, so a weight of any size leaves the product in range: the result is the one
    of a row of size 1, to the norm's own bound (512 values: the sum rounds 16 + 13 times, half of which enters the root, and 6
    roundings come after it: 20.5 U, for each of the two rows; what the scaled row was rounded to, U in a value and in the root; the
    scale's two quotients): below 48 U, and a code then lies at most one border further."""
    g = gen(3)
    x = torch.randn((6, 512), generator=g).clamp(-1, 1) + 0.25
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(DEV) * weight
    got = []
    for k in (size, 1.0):
        xs = (x.double() * k).float().to(DEV)
        if k < 1e-37:  # (subnormal values: what they stand for is taken back to size 1)
            x = xs.double().cpu() / k
        q, s = torch.empty((6, 512), dtype=torch.uint8, device=DEV), torch.empty((4, 6), device=DEV)
        lib.kv8_quant_blocks(xs, q, s, norm_w=w, eps=0.0)
        rows, ks = torch.empty((6, 576), dtype=torch.uint8, device=DEV), torch.empty(6, device=DEV)
        lib.kv8_norm_rope_rows(torch.cat([xs, torch.zeros((6, 64), device=DEV)], 1), w, 0.0, torch.zeros(6, dtype=torch.int32, device=DEV),
                               torch.ones(32, device=DEV), torch.arange(6, device=DEV), rows, ks)
        got.append((q, s, rows[:, :512], ks))
    for (a, b) in zip(got[0][1::2], got[1][1::2]):  # scales
        assert bool(torch.isfinite(a).all()) and bool(((a.double() - b.double()).abs() <= 48 * U * b.double() + 2.0 ** -149).all())
    for (a, b) in zip(got[0][0::2], got[1][0::2]):  # codes: next to one another (of the same sign)
        assert bool(((a.int() - b.int()).abs() <= 1).all())


def test_a_row_with_an_infinity_is_bytes_of_zero(lib):
    x = torch.randn((3, 2048), generator=gen(4)).to(DEV)
    x[0, 5], x[1, 2047], x[2, 77] = math.inf, -math.inf, math.nan
    q, s = torch.empty((3, 2048), dtype=torch.uint8, device=DEV), torch.empty((16, 3), device=DEV)
    lib.kv8_quant_blocks(x, q, s, norm_w=torch.ones(2048, device=DEV))
    assert bool((q == 0).all()) and bool((s == 0).all())
    rows, ks = torch.empty((3, 576), dtype=torch.uint8, device=DEV), torch.empty(3, device=DEV)
    x[1, 511] = -math.inf
    lib.kv8_norm_rope_rows(torch.cat([x[:, :512], x[:, 600:664]], 1), torch.ones(512, device=DEV), 1e-6, torch.zeros(3, dtype=torch.int32, device=DEV),
                           torch.ones(32, device=DEV), torch.arange(3, device=DEV), rows, ks)
    assert bool((rows[:, :512] == 0).all()) and bool((rows[:, 512:] != 0).any(1).all())


# -------------------------------------------------------------------------------------------------------------
# angles
# -------------------------------------------------------------------------------------------------------------
def exact_angle(p, f):
    """p f reduced to [-pi, pi], rounded once to f64: whole-number arithmetic on 1 / (2 pi) to 320 bits (pi by Machin's formula)."""
    bits = 320
    one = 1 << (bits + 32)

    def arctan_of_inverse(k):
        term = total = one // k
        n, sign = 3, -1
        while term:
            term //= k * k
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total
    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))  # times 2^(bits + 32)
    inverse = (one << bits) // (2 * pi)                          # 2^bits / (2 pi)
    m, e = math.frexp(f)
    whole, e = int(m * (1 << 24)), e - 24                          # f = whole 2^e
    t = p * whole * inverse
    t = t << e if e >= 0 else t >> -e
    t &= (1 << bits) - 1
    if t >> (bits - 1):
        t -= 1 << bits
    return 2 * math.pi * (t / (1 << bits))


def turned(lib, pos, f, layout=0):
    """cos and sin as kv8_rope makes them: pairs (1, 0) turned."""
    n, pairs = len(pos), len(f)
    x = torch.zeros((n, 1, pairs, 2), device=DEV)
    x[..., 0] = 1
    x = x if layout == 0 else x.transpose(2, 3)
    rot = torch.empty((n, 1, 2 * pairs), device=DEV)
    lib.kv8_rope(x.reshape(n, 1, 2 * pairs), torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(f, dtype=torch.float32, device=DEV), 0, rot, layout=layout)
    out = rot.view(n, pairs, 2) if layout == 0 else rot.view(n, 2, pairs).transpose(1, 2)
    return out.double().cpu().numpy()


@pytest.mark.parametrize("layout", [0, 1])
def test_angles_of_every_size(lib, layout):
    """A cosine or sine is held to 6 U of itself and what its angle is off by.  The frequency's fraction of a turn is rounded to 2^-64
    (2^-65 off) and |f| 2^-128 off for the 128 bits of 1 / (2 pi) that make it; the position multiplies both.  The rest of the turn
    after whole quarters then rounds three times (conversion, constant, product; 3 U of itself, which a sine below pi/4 takes over
    at most, a cosine to 0.8 of it), the series rounds its last sum once (U), the terms before it, a tenth of a sine and 0.44 of a cosine at
    most, two or three times (below U); they end at 0.05 U of the value."""
    freqs, _ = lib.kv8_rope_freqs(64, 10000.0, 40.0, 4096)
    f = [float(v) for v in freqs] + [float(np.float32(v)) for v in (0.9999, 3.14159274, 12345.678, 1e6, -0.37, -2.5e-5, 1e-9, 0.0)]
    pos = [0, 1, 2, 3, 5, 8, -1, -7, 100, 1001, 4096, 65537, 999999, (1 << 20) - 1, 123456789, (1 << 31) - 1, -(1 << 31), -(1 << 30) + 1]
    got = turned(lib, pos, f, layout)
    worst = 0.0
    for i, p in enumerate(pos):
        for j, v in enumerate(f):
            a = exact_angle(p, v)
            off = 2 * math.pi * abs(p) * (2.0 ** -65 + abs(v) * 2.0 ** -128)
            for k, want in enumerate((math.cos(a), math.sin(a))):
                worst = max(worst, abs(got[i, j, k] - want) / (6 * U * abs(want) + off + 2.0 ** -149))
    assert worst <= 1, f"{worst:.4g} times the bound"


def test_exact_angle_against_f64():
    for p, f in ((1, 1.0), (7, 0.25), (100, 1e-3), (-5, 0.5), (1000, 0.1)):
        v = float(np.float32(f))
        a = math.remainder(p * v, 2 * math.pi)
        assert abs(exact_angle(p, v) - a) < 1e-12 * max(1, abs(p * v))


# -------------------------------------------------------------------------------------------------------------
# calls one after the other
# -------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 40, 700])
def test_a_call_sees_what_the_call_before_it_has_just_written(lib, n):
    """Every call's input is the output of the call before, written again and again into the same memory while the next kernel may
    already run: quantized rows and their scales, products, slots, positions and rotated heads."""
    g = gen(n)
    hid, H, page = 1024, 8, 16
    xs = [torch.randn((n, hid), generator=g).to(BF).to(DEV) for _ in range(3)]
    w, w8, sw = torch.ones(hid, device=DEV), *weight(g, H * 192, hid, DEV)
    v8, sv = weight(g, 576, hid, DEV)
    q, s = torch.empty((n, hid), dtype=torch.uint8, device=DEV), torch.empty((hid // BLK, n), device=DEV)
    heads, fresh, f, lw = torch.empty((n, H * 192), device=DEV), torch.empty((n, 576), device=DEV), lib.kv8_rope_freqs(64)[0].to(DEV), torch.ones(512, device=DEV)
    rot, rest = torch.empty((n, H, 64), device=DEV), torch.empty((n, H, 128), device=DEV)
    rows = -(-n // page) * page
    kv8, ks = torch.zeros((rows, 576), dtype=torch.uint8, device=DEV), torch.zeros(rows, device=DEV)
    per = 256
    B = -(-n // per)  # sequences of up to 256 rows
    counts = [min(per, n - per * b) for b in range(B)]
    start = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device=DEV)
    lens, parent = torch.zeros(B, dtype=torch.int32, device=DEV), torch.cat([torch.arange(-1, c - 1) for c in counts]).to(torch.int32).to(DEV)
    n_pages, table = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros((B, per // page), dtype=torch.int32, device=DEV)
    free, n_free = torch.arange(rows // page, dtype=torch.int32, device=DEV), torch.tensor([rows // page], dtype=torch.int32, device=DEV)
    slots, mask = torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros((n, per // 32), dtype=torch.int32, device=DEV)
    pos, err = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)

    def go(x, each=lambda: None):
        for call in (lambda: lib.kv8_page_plan(lens, start, page, n_pages, table, free, n_free, slots, err_word=err),
                     lambda: lib.kv8_quant_blocks(x, q, s, norm_w=w),
                     lambda: lib.kv8_matmul8(q, s, w8, sw, heads, err_word=err),
                     lambda: lib.kv8_matmul8(q, s, v8, sv, fresh, err_word=err),
                     lambda: lib.kv8_tree_mask(parent, start, lens, mask, position=pos, err_word=err),
                     lambda: lib.kv8_norm_rope_rows(fresh, lw, 1e-6, pos, f, slots, kv8, ks, err_word=err),
                     lambda: lib.kv8_rope(heads.view(n, H, 192), pos, f, 128, rot, rest),
                     lambda: lib.kv8_rope(rot, pos, f, 0, rot),
                     lambda: lib.kv8_quant_blocks(rest.view(n, H * 128), q, s),
                     lambda: lib.kv8_matmul8(q, s, w8, sw, heads, err_word=err)):
            call()
            each()
    outs = (q, s, heads, fresh, rot, rest, kv8, ks, slots, pos)
    want = []
    for x in xs:
        go(x, torch.cuda.synchronize)
        want.append([o.clone() for o in outs])
    assert err.item() == 0 and not torch.equal(want[0][2], want[1][2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x in xs:
            go(x)
    for turn in range(6):
        for _ in range(4):
            if turn % 2:
                graph.replay()
            else:
                for x in xs:
                    go(x)
        got = [o.clone() for o in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, want[-1]))
        go(xs[turn % 2])
        got = [o.clone() for o in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, want[turn % 2]))
    assert err.item() == 0


# -------------------------------------------------------------------------------------------------------------
# products: a row's place does not matter
# -------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("M,N,K", [(1, 1000, 4096), (16, 1000, 4096), (37, 24576, 256), (64, 1000, 4096), (64, 24576, 256), (200, 1000, 4096), (48, 8200, 1024),
                                   (300, 900, 3200), (1024, 1000, 4096), (129, 12200, 528), (700, 8200, 384), (1500, 2100, 400), (2048, 4096, 512)])
@pytest.mark.parametrize("ot", [BF, F32])
def test_products_do_not_depend_on_a_rows_or_columns_place(lib, M, N, K, ot):
    """Three kinds of rows (codes and scales), each at many places of the left operand, tiles' first and last rows among them: bit-equal rows of
    the output.  Likewise three kinds of columns: weight blocks of equal codes and scales."""
    g = gen(M + N)
    kb, nb = -(-K // BLK), -(-N // BLK)
    a3, _ = weight(g, 3, K, DEV)
    s3 = torch.exp2(torch.randn((kb, 3), generator=g) - 6).to(DEV)
    kind = torch.randint(0, 3, (M,), generator=g)
    kind[[0, M - 1]] = 0
    for at in (15, 16, 31, 32, 63, 64, 127, 128, 255, 256):
        if at < M:
            kind[at] = 0
    kind = kind.to(DEV)
    w3, _ = weight(g, 3 * BLK, K, DEV)
    v3 = torch.exp2(torch.randn((3, kb), generator=g) - 6).to(DEV)
    block = torch.randint(0, 3, (nb,), generator=g).to(DEV)
    block[[0, nb - 1]] = 1
    w8 = w3.view(3, BLK, K)[block].reshape(nb * BLK, K)[:N].contiguous()
    out = torch.empty((M, N), dtype=ot, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_matmul8(a3[kind].contiguous(), s3[:, kind].contiguous(), w8, v3[block].contiguous(), out, err_word=err)
    assert err.item() == 0
    ref, tol = matmul(a3, s3, w3, v3, ot)
    for k in range(3):
        rows = out[kind == k]
        assert bool((rows == rows[:1]).all()), f"rows of kind {k}"
        first = torch.full((3 * BLK,), -1, device=DEV, dtype=torch.long)
        for b in range(nb):  # every block of a kind against the kind's reference, and bit for bit against the first of it
            if len(rows) == 0:
                continue
            c, t = slice(b * BLK, min(N, (b + 1) * BLK)), int(block[b])
            got = rows[0, c]
            want = ref[k, t * BLK:t * BLK + len(got)]
            assert bool(((got.double() - want).abs() <= tol[k, t * BLK:t * BLK + len(got)]).all())
            if first[t] < 0:
                first[t] = b
            else:
                assert torch.equal(got, rows[0, int(first[t]) * BLK:int(first[t]) * BLK + len(got)]), f"columns of kind {t}"


@pytest.mark.parametrize("layout", [0, 1])
def test_scores_of_a_long_context(lib, layout):
    """Frequencies for forty times the context, as the header has them used with heads that are rotated in part: rope_scale 1, and
    the scale's square in sm_scale.  Held to the method's definition, whole queries and whole keys times the scale, in 64 bits (the
    rows as quantized), within the library's bound for attention outputs."""
    g = gen(8)
    T, H, at = 700, 16, 100000
    f, scale = lib.kv8_rope_freqs(64, 10000.0, 40.0, 4096)
    f, sm = f.to(DEV), 192.0 ** -0.5
    pos = (at + torch.arange(T)).to(torch.int32).to(DEV)
    kv8, ks = torch.empty((T, 576), dtype=torch.uint8, device=DEV), torch.empty(T, device=DEV)
    lib.kv8_norm_rope_rows(torch.randn((T, 576), generator=g).to(DEV), torch.ones(512, device=DEV), 1e-6, pos, f, torch.arange(T, device=DEV), kv8, ks, layout=layout)
    q_lat, heads = torch.randn((H, 512), generator=g).to(DEV), torch.randn((1, H, 192), generator=g).to(DEV)
    q_rope, last = torch.empty((1, H, 64), device=DEV), pos[-1:].contiguous()
    lib.kv8_rope(heads, last, f, 128, q_rope, layout=layout)
    ws = torch.empty(lib.mla_decode8_workspace_bytes(H, T, 0) // 4, device=DEV)
    out, err = torch.empty((H, 512), device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.mla_absorb_decode8(q_lat, q_rope[0], kv8, ks, T, sm * scale * scale, ws, out, err_word=err)
    assert err.item() == 0
    c = values(kv8) * ks.double()[:, None]
    turned_q, _ = rotate(heads[..., 128:].double(), last, f, 1.0, layout)
    q = scale * torch.cat([q_lat.double(), turned_q[0]], 1)
    want = torch.softmax(sm * (q @ (scale * c).t()), 1) @ c[:, :512]
    parity(out.cpu().numpy(), want.cpu().numpy(), "scores of a long context")
