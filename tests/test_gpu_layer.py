"""What stands around the attention in a layer: rotary positions, normed and rotated rows into the cache, block quantization and
the block-scaled product, each against a plain 64-bit reference (tests/layer_ref.py derives the bounds), and all together."""
import numpy as np
import pytest
import torch

from layer_ref import BLK, OUT_EPS, U, check_codes, matmul, nearest, norm, rotate, values, weight

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, g, dtype=F32):
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


def positions(n, g):
    """Positions of every size, the ends of the type among them."""
    p = torch.randint(0, 1 << 20, (n,), generator=g)
    special = torch.tensor([0, 1, -1, (1 << 20) - 1, (1 << 31) - 1, -(1 << 31), 12345])
    p[:min(n, 7)] = special[:n]
    return p[torch.randperm(n, generator=g)].to(torch.int32).to(DEV)


# -------------------------------------------------------------------------------------------------------------
# rotary positions
# -------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("n,heads,width,at,dim,xt,ot", [
    (1, 128, 192, 128, 64, BF, BF), (1, 1, 64, 0, 64, F32, F32), (37, 16, 192, 128, 64, BF, F32), (300, 20, 128, 0, 64, F32, BF),
    (5, 7, 96, 0, 96, BF, BF), (64, 3, 128, 64, 32, F32, F32), (9, 2, 100, 10, 30, BF, F32), (3, 5, 7, 1, 2, F32, BF), (2, 1, 256, 0, 256, BF, BF),
    (1000, 1, 64, 0, 64, BF, BF), (2, 128, 1024, 400, 176, BF, BF), (700, 128, 192, 128, 64, BF, BF), (11, 3, 48, 16, 16, BF, BF), (4, 2, 40, 16, 24, BF, BF)])
def test_rope(lib, n, heads, width, at, dim, xt, ot, layout):
    g = gen(n * width + layout)
    x, pos = randn((n, heads, width), g, xt), positions(n, g)
    f, _ = lib.kv8_rope_freqs(dim, 10000.0, 4.0, 4096)
    f, scale = f.to(DEV), 1.25
    rot, rest = torch.full((n, heads, dim), 7.0, dtype=ot, device=DEV), torch.full((n, heads, width - dim), 7.0, dtype=ot, device=DEV)
    lib.kv8_rope(x, pos, f, at, rot, rest if width > dim else None, rope_scale=scale, layout=layout)
    ref, tol = rotate(x[..., at:at + dim].double(), pos, f, scale, layout)
    tol = tol + OUT_EPS[ot] * (ref.abs() + tol)
    d = (rot.double() - ref).abs()
    assert bool((d <= tol).all()), f"{float((d / tol).max()):.3g} times the bound"
    if width > dim:
        keep = torch.cat([x[..., :at], x[..., at + dim:]], -1)
        assert torch.equal(rest, keep.to(ot))


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("xt", [BF, F32])
def test_rope_strides_and_in_place(lib, layout, xt):
    """Heads outside rows, gaps, a repeated head, odd offsets; in place; what lies between stays; negative positions undo."""
    g = gen(5)
    n, heads, width, at, dim = 6, 5, 192, 128, 64
    f = lib.kv8_rope_freqs(dim)[0].to(DEV)
    pos = positions(n, g)
    for off in (0, 8, 3):  # at an offset of 3 elements nothing lies on 16 bytes
        big = randn((heads, n + 1, width + 40), g, xt)
        x = big.permute(1, 0, 2)[:n, :, off:off + width]
        want, tol = rotate(x[..., at:].double(), pos, f, 1.0, layout)
        tol = tol + OUT_EPS[xt] * (want.abs() + tol)
        out = torch.full((n, heads, 200), 7.0, dtype=xt, device=DEV)
        rest = torch.full((heads, n, 160), 7.0, dtype=xt, device=DEV)
        lib.kv8_rope(x, pos, f, at, out[..., off:off + dim], rest.permute(1, 0, 2)[..., off:off + at], layout=layout)
        assert bool(((out[..., off:off + dim].double() - want).abs() <= tol).all())
        assert torch.equal(rest.permute(1, 0, 2)[..., off:off + at], x[..., :at])
        assert bool((out[..., :off] == 7).all()) and bool((out[..., off + dim:] == 7).all()) and bool((rest[..., off + at:] == 7).all())
        before = big.clone()
        lib.kv8_rope(x, pos, f, at, x[..., at:], layout=layout)
        assert torch.equal(x[..., at:], out[..., off:off + dim])
        left = big.permute(1, 0, 2).clone()
        left[:n, :, off + at:off + width] = before.permute(1, 0, 2)[:n, :, off + at:off + width]
        assert torch.equal(left, before.permute(1, 0, 2)), "something outside the rotated part was written"
        if xt is F32:
            keep = pos != -(1 << 31)
            lib.kv8_rope(x, -pos, f, at, x[..., at:], layout=layout)
            d = (x[..., at:] - before.permute(1, 0, 2)[:n, :, off + at:off + width]).abs()[keep]
            size = before.permute(1, 0, 2)[:n, :, off + at:off + width].abs().max()
            # A cosine or sine is off by 5 U at most: its angle, pi/4 at most, by pi 2^-32 2 + 3 U pi/4 (conversion, constant, product),
            # its series by 2^-29 and 2 U of roundings.  An element is then off by 2 * 5 U of the largest one and, for its two products
            # and their sum, 2 * 1.42 U: below 24 U.  There are two turns; the values between them, and the first turn's errors in the
            # second, are up to sqrt(2) < 2 times as large.
            assert float(d.max()) <= 2 * 24 * U * 2 * float(size)
    one = randn((n, 1, width), g, xt)
    a, b = (torch.empty((n, heads, dim), dtype=xt, device=DEV) for _ in range(2))
    lib.kv8_rope(one.expand(n, heads, width), pos, f, at, a, layout=layout)
    lib.kv8_rope(one.expand(n, heads, width).contiguous(), pos, f, at, b, layout=layout)
    assert torch.equal(a, b)


def test_rope_values_that_are_not_finite_stay_in_their_pair(lib):
    g = gen(6)
    for layout in (0, 1):
        x = randn((3, 2, 64), g, BF)
        clean = torch.empty((3, 2, 64), device=DEV)
        pos = torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
        f = lib.kv8_rope_freqs(64)[0].to(DEV)
        lib.kv8_rope(x, pos, f, 0, clean, layout=layout)
        x[1, 1, 20] = float("nan")
        x[2, 0, 3] = float("inf")
        out = torch.empty((3, 2, 64), device=DEV)
        lib.kv8_rope(x, pos, f, 0, out, layout=layout)
        hit = torch.zeros((3, 2, 64), dtype=torch.bool, device=DEV)
        for r, h, e in ((1, 1, 20), (2, 0, 3)):
            hit[r, h, e] = hit[r, h, e ^ 1 if layout == 0 else e ^ 32] = True
        assert torch.equal(out[~hit], clean[~hit]) and not bool(torch.isfinite(out[hit]).any())


def test_rope_at_offsets_past_32_bits(lib):
    """Rows whose elements lie more than 2^31 elements apart, on both sides."""
    n, gap = 3, (1 << 30) + 8
    big = torch.empty(2 * gap + 64, dtype=BF, device=DEV)
    out = torch.empty(2 * gap + 64, dtype=BF, device=DEV)
    x, y = torch.as_strided(big, (n, 1, 64), (gap, 64, 1)), torch.as_strided(out, (n, 1, 64), (gap, 64, 1))
    x.copy_(randn((n, 1, 64), gen(7), BF))
    pos, f = torch.tensor([3, 70000, 9], dtype=torch.int32, device=DEV), lib.kv8_rope_freqs(64)[0].to(DEV)
    lib.kv8_rope(x, pos, f, 0, y, layout=1)
    ref, tol = rotate(x.double(), pos, f, 1.0, 1)
    assert bool(((y.double() - ref).abs() <= tol + OUT_EPS[BF] * (ref.abs() + tol)).all())


# -------------------------------------------------------------------------------------------------------------
# fresh rows into the cache
# -------------------------------------------------------------------------------------------------------------
def rows_case(lib, g, n, xt, layout, pad, scale=1.3, eps=EPS, x=None):
    wide = randn((n, 576 + pad), g, F32) * torch.exp2(torch.randint(-6, 7, (n, 1), generator=g).float()).to(DEV)
    wide = wide.to(xt)
    if x is not None:
        wide[:, pad:] = x
    xs, pos = wide[:, pad:], positions(n, g)
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(DEV)
    f = lib.kv8_rope_freqs(64, 10000.0, 40.0)[0].to(DEV)
    rows = n + 9
    dst = torch.randperm(rows, generator=g)[:n].to(DEV)
    kv8 = torch.randint(0, 255, (rows, 576), generator=g, dtype=torch.uint8).to(DEV)
    ks = torch.rand(rows, generator=g).to(DEV)
    return xs, w, pos, f, dst, kv8, ks, scale, layout, eps


def rows_ref(xs, w, pos, f, scale, layout, eps):
    x = xs.double()
    lat, rel = norm(x[:, :512], w.double(), eps)
    rot, tol = rotate(x[:, None, 512:], pos, f, scale, layout)
    y = torch.cat([lat, rot[:, 0]], 1)
    return y, rel, torch.cat([torch.zeros_like(lat), tol[:, 0]], 1)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("n,xt,pad", [(1, BF, 0), (1, F32, 0), (7, BF, 64), (64, F32, 1472), (1000, BF, 0), (333, F32, 4), (4097, BF, 8)])
def test_norm_rope_rows(lib, n, xt, pad, layout):
    g = gen(n + layout)
    xs, w, pos, f, dst, kv8, ks, scale, layout, eps = rows_case(lib, g, n, xt, layout, pad)
    old8, olds, err = kv8.clone(), ks.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_norm_rope_rows(xs, w, eps, pos, f, dst, kv8, ks, rope_scale=scale, layout=layout, err_word=err)
    y, rel, tol = rows_ref(xs, w, pos, f, scale, layout, eps)
    check_codes(kv8[dst], ks[dst], y, rel, tol)
    other = torch.ones(len(ks), dtype=torch.bool, device=DEV)
    other[dst] = False
    assert torch.equal(kv8[other], old8[other]) and torch.equal(ks[other], olds[other])
    assert err.item() == 0


def test_rows_without_a_place_are_left_out(lib):
    g = gen(11)
    xs, w, pos, f, dst, kv8, ks, scale, layout, eps = rows_case(lib, g, 40, BF, 0, 0)
    full8, fulls = kv8.clone(), ks.clone()
    lib.kv8_norm_rope_rows(xs, w, eps, pos, f, dst, full8, fulls)
    some = dst.clone()
    some[3], some[17], some[39] = -1, len(ks), 1 << 40
    got8, gots, err = kv8.clone(), ks.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_norm_rope_rows(xs, w, eps, pos, f, some, got8, gots, err_word=err)
    want8, wants = full8.clone(), fulls.clone()
    for i in (3, 17, 39):
        want8[dst[i]], wants[dst[i]] = kv8[dst[i]], ks[dst[i]]
    assert torch.equal(got8, want8) and torch.equal(gots, wants) and err.item() == lib.KV8_ERR_INDEX
    lib.kv8_norm_rope_rows(xs, w, eps, pos, f, some, got8, gots)  # without an error word
    lib.kv8_norm_rope_rows(xs[:0], w, eps, pos[:0], f, dst[:0], got8, gots)
    assert torch.equal(got8, want8)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("size,eps", [(0.0, 1e-6), (0.0, 0.0), (1e30, 1e-6), (3e38, 1e-6), (1e-15, 0.0), (1e-30, 0.0), (1e-30, 1e-6), (1e-20, 1e-30), (1e-42, 0.0)])
def test_rows_of_any_magnitude(lib, xt, size, eps):
    g = gen(12)
    n = 5
    x = torch.randn((n, 576), generator=g).clamp(-1, 1) * size
    x[:, 512:] = torch.randn((n, 64), generator=g)
    xs, w, pos, f, dst, kv8, ks, scale, layout, eps = rows_case(lib, g, n, xt, 0, 0, eps=eps, x=x.to(DEV))
    lib.kv8_norm_rope_rows(xs, w, eps, pos, f, dst, kv8, ks, rope_scale=scale)
    y, rel, tol = rows_ref(xs, w, pos, f, scale, layout, eps)
    check_codes(kv8[dst], ks[dst], torch.nan_to_num(y, nan=0.0), rel, tol)


def test_rows_that_are_not_finite(lib):
    """As the row quantizer: NaN gives 0; a norm over an infinity leaves zeros; an infinity among the rotated saturates or gives 0."""
    g = gen(13)
    n = 4
    xs, w, pos, f, dst, kv8, ks, scale, layout, eps = rows_case(lib, g, n, F32, 0, 0)
    pos[:] = 0  # no rotation: an infinity times a sine of 0 is NaN in its partner
    xs[0, 100], xs[1, 200], xs[2, 512], xs[3, 575] = float("nan"), float("inf"), float("nan"), -float("inf")
    lib.kv8_norm_rope_rows(xs, w, eps, pos, f, dst, kv8, ks)
    got, s = values(kv8[dst]), ks[dst].double()
    y, rel, tol = rows_ref(xs, w, pos, f, 1.0, layout, eps)
    for r in (0, 1):
        assert bool((got[r, :512] == 0).all())
        amax = xs[r, 512:].double().abs().max()
        assert abs(float(s[r] - amax / 448)) <= 1e-6 * float(amax) / 448 and float(got[r, 512:].abs().max()) == 448
    for r, e in ((2, 512), (3, 575)):
        fin = torch.isfinite(y[r])
        amax = y[r][fin].abs().max()
        assert abs(float(s[r] - amax / 448)) <= 1e-5 * float(amax) / 448
        assert float(got[r, e]) in ((0.0,) if e == 512 else (0.0, -448.0)) and float(got[r, e ^ 1]) == 0.0
        assert float(got[r, :512].abs().max()) > 0


# -------------------------------------------------------------------------------------------------------------
# blocks of 128
# -------------------------------------------------------------------------------------------------------------
def blocks_check(x, w, eps, q, scale):
    y, rel = (x.double(), 0.0) if w is None else norm(x.double(), w.double(), eps)
    for k in range(scale.shape[0]):
        c = slice(k * BLK, (k + 1) * BLK)
        check_codes(q[:, c].contiguous(), scale[k], torch.nan_to_num(y[:, c], nan=0.0) if w is not None else y[:, c], rel,
                    torch.zeros_like(y[:, c]), f"block {k}")


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("n,width,xt,pad", [(1, 16, BF, 0), (3, 112, F32, 4), (9, 128, BF, 8), (2, 144, F32, 0), (17, 512, BF, 0), (5, 528, F32, 16),
                                            (100, 576, BF, 0), (1, 1024, F32, 0), (4, 1040, BF, 0), (33, 2048, F32, 0), (1, 4096, BF, 0),
                                            (3, 4112, F32, 0), (2, 8208, BF, 8), (7, 16384, F32, 0), (1, 16368, BF, 0)])
def test_quant_blocks(lib, n, width, xt, pad, normed):
    g = gen(n * width)
    x = (randn((n, width + pad), g) * torch.exp2(torch.randint(-8, 9, (1, width + pad), generator=g).float()).to(DEV)).to(xt)[:, :width]
    w = (1 + 0.3 * torch.randn(width, generator=g)).to(DEV) if normed else None
    q = torch.empty((n, width), dtype=torch.uint8, device=DEV)
    room = torch.full((-(-width // BLK), n + 3), -1.0, device=DEV)
    lib.kv8_quant_blocks(x, q, room[:, :n], norm_w=w, eps=EPS)
    blocks_check(x, w, EPS, q, room[:, :n])
    assert bool((room[:, n:] == -1).all())


def test_quant_blocks_wider_than_a_norm_takes_and_refused_with_one(lib):
    g = gen(3)
    x, q, s = randn((2, 65536), g), torch.empty((2, 65536), dtype=torch.uint8, device=DEV), torch.empty((512, 2), device=DEV)
    lib.kv8_quant_blocks(x, q, s)
    blocks_check(x, None, 0, q, s)
    with pytest.raises(lib.Kv8Error):
        lib.kv8_quant_blocks(x, q, s, norm_w=torch.ones(65536, device=DEV))


@pytest.mark.parametrize("normed", [False, True])
def test_quant_blocks_zeros_extremes_and_what_is_not_finite(lib, normed):
    g = gen(4)
    for width in (512, 2048):
        x = randn((9, width), g)
        x[1] = 0
        x[2, 128:256] = 0
        x[3] *= 1e30
        x[4] *= 1e-41
        x[5] *= 1e-30
        x[6, 130] = float("nan")
        x[7, 300] = float("inf")
        x[8, 300] = -float("inf")
        w = torch.ones(width, device=DEV) if normed else None
        q, s = torch.empty((9, width), dtype=torch.uint8, device=DEV), torch.empty((width // BLK, 9), device=DEV)
        lib.kv8_quant_blocks(x, q, s, norm_w=w, eps=0.0)
        got = values(q)
        blocks_check(x[:6], w, 0.0, q[:6], s[:, :6])
        if normed:
            assert bool((got[6:] == 0).all()) and bool((s[:, 6:] == 0).all())
        else:
            blocks_check(x[6:], None, 0.0, q[6:], s[:, 6:])
            assert got[6, 130] == 0 and got[7, 300] == 448 and got[8, 300] == -448


def test_one_block_is_the_row_quantizer(lib):
    """A row of 128 is one block: the same bytes and scale as kv8_quant_rows_w's."""
    x = randn((50, 128), gen(9)) * torch.exp2(torch.arange(-25, 25, device=DEV).float())[:, None]
    q, s = torch.empty((50, 128), dtype=torch.uint8, device=DEV), torch.empty((1, 50), device=DEV)
    q2, s2 = torch.empty_like(q), torch.empty(50, device=DEV)
    lib.kv8_quant_blocks(x, q, s)
    lib.kv8_quant_rows_w(x, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s[0], s2)


# -------------------------------------------------------------------------------------------------------------
# the product
# -------------------------------------------------------------------------------------------------------------
SHAPES = [(1, 1, 16), (1, 64, 128), (1, 4096, 16384), (2, 127, 112), (15, 128, 144), (16, 129, 512), (17, 576, 4112), (31, 24576, 256), (33, 200, 2064),
          (48, 8192, 1024), (64, 1343, 1040), (65, 100, 128), (100, 576, 2048), (127, 300, 272), (128, 128, 16), (129, 130, 640), (256, 256, 4096),
          (300, 1000, 1008), (1000, 576, 4112), (700, 8200, 384), (2048, 4096, 512), (1111, 2345, 1232), (3000, 40, 256), (66, 24576, 2048),
          # every form of the kernel and split of K (on 152 SMs)
          (3, 8200, 1600), (3, 100, 1024), (65, 4096, 1024), (65, 4096, 2064), (300, 100, 1024), (300, 100, 2064), (37, 24576, 2048), (129, 5000, 6400),
          (1000, 100, 1600), (700, 100, 2064), (129, 4096, 3200), (300, 900, 3200), (700, 200, 8192), (129, 12200, 528)]


def product(lib, a8, sa, w8, sw, ot, stride=0, off=0):
    """The call into the middle of a larger buffer, whose other elements stay."""
    M, N = a8.shape[0], w8.shape[0]
    room = torch.full((M + 1, N + off + stride), 7.0, dtype=ot, device=DEV)
    out, err = room[:M, off:off + N], torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_matmul8(a8, sa, w8, sw, out, err_word=err)
    assert err.item() == 0
    assert bool((room[M:] == 7).all()) and bool((room[:, :off] == 7).all()) and bool((room[:, off + N:] == 7).all())
    return out


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ot", [BF, F32])
def test_matmul(lib, M, N, K, ot):
    g = gen(M + N + K)
    w8, sw = weight(g, N, K, DEV)
    a8, _ = weight(g, M, K, DEV)
    sa = torch.exp2(torch.randn((-(-K // BLK), M), generator=g) * 2 - 6).to(DEV)
    ref, tol = matmul(a8, sa, w8, sw, ot)
    for stride, off in ((0, 0), (16, 8), (5, 1)):
        d = (product(lib, a8, sa, w8, sw, ot, stride, off).double() - ref).abs()
        assert bool((d <= tol).all()), f"{float((d / tol).max()):.3g} times the bound"


@pytest.mark.parametrize("M,N,K", SHAPES + [(5000, 512, 128), (4500, 4400, 144)])
def test_matmul_of_whole_numbers_is_exact(lib, M, N, K):
    """Codes of -2 .. 2 and scales of 1/2, 1, 2: every sum is a multiple of 1/4 below 2^22, so any order gives the same f32."""
    g = gen(M * 3 + N + K)
    small = torch.tensor([-2.0, -1.0, 0.0, 1.0, 2.0]).to(torch.float8_e4m3fn).view(torch.uint8)
    a8, w8 = (small[torch.randint(0, 5, (r, K), generator=g)].to(DEV) for r in (M, N))
    kb = -(-K // BLK)
    sa = torch.exp2(torch.randint(-1, 2, (kb, M), generator=g).float()).to(DEV)
    sw = torch.exp2(torch.randint(-1, 2, (-(-N // BLK), kb), generator=g).float()).to(DEV)
    ref, _ = matmul(a8, sa, w8, sw, F32)
    assert torch.equal(product(lib, a8, sa, w8, sw, F32).double(), ref)
    assert torch.equal(product(lib, a8, sa, w8, sw, BF, 8, 8).double(), ref.float().to(BF).double())


@pytest.mark.parametrize("M", [1, 40, 64, 200, 3000])
def test_matmul_of_cache_rows(lib, M):
    """The rows of a latent cache as they lie, one scale a row."""
    g = gen(M)
    cache, _ = weight(g, M, 576, DEV)
    cache[:, 512:] = 0x7F  # what lies behind the latent part is not read
    scale = torch.exp2(torch.randn(M, generator=g) - 6).to(DEV)
    w8, sw = weight(g, 512, 512, DEV)
    for ot in (BF, F32):
        ref, tol = matmul(cache[:, :512], scale, w8, sw, ot)
        assert bool(((product(lib, cache[:, :512], scale, w8, sw, ot).double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("M,N,K", [(3, 300, 528), (64, 200, 2048), (200, 300, 528), (1000, 2000, 144)])
def test_matmul_what_is_not_a_number_stays_in_its_row_or_column(lib, M, N, K):
    g = gen(M)
    w8, sw = weight(g, N, K, DEV)
    a8, _ = weight(g, M, K, DEV)
    kb = -(-K // BLK)
    sa = torch.exp2(torch.randn((kb, M), generator=g)).to(DEV)
    clean = product(lib, a8, sa, w8, sw, F32)
    m, n = M // 2, N // 3
    a8[m, K - 1], w8[n, 3], sa[kb - 1, 0] = 0x7F, 0xFF, float("nan")
    got = product(lib, a8, sa, w8, sw, F32)
    hit = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    hit[m], hit[:, n], hit[0] = True, True, True
    assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("M", [1, 64, 65, 1024])
def test_matmul_is_the_same_every_time_and_row_by_row_alike(lib, M):
    g = gen(M)
    w8, sw = weight(g, 1000, 4096, DEV)
    a8, _ = weight(g, M, 4096, DEV)
    sa = torch.exp2(torch.randn((32, M), generator=g)).to(DEV)
    first = product(lib, a8, sa, w8, sw, F32)
    for _ in range(5):
        assert torch.equal(product(lib, a8, sa, w8, sw, F32), first)


def test_matmul_scales_with_room_between_blocks(lib):
    """Scales of more rows than the call takes: the blocks' rows lie further apart."""
    g = gen(8)
    for M, N, K in ((5, 300, 1040), (200, 300, 1040), (1500, 2100, 400)):
        w8, sw = weight(g, N, K, DEV)
        a8, _ = weight(g, M, K, DEV)
        room = torch.full((-(-K // BLK), M + 11), float("nan"), device=DEV)
        room[:, :M] = torch.exp2(torch.randn((-(-K // BLK), M), generator=g)).to(DEV)
        ref, tol = matmul(a8, room[:, :M], w8, sw, F32)
        assert bool(((product(lib, a8, room[:, :M], w8, sw, F32).double() - ref).abs() <= tol).all())


def test_calls_with_nothing_to_do(lib):
    """No rows: nothing is read, nothing written."""
    z = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    u8, i32 = torch.uint8, torch.int32
    lib.kv8_matmul8(z(0, 256, dtype=u8), z(2, 0), z(128, 256, dtype=u8), z(1, 2), z(0, 128))
    lib.kv8_quant_blocks(z(0, 256), z(0, 256, dtype=u8), z(2, 0))
    lib.kv8_rope(z(0, 4, 64), z(0, dtype=i32), z(32), 0, z(0, 4, 64))
    lib.kv8_norm_rope_rows(z(0, 576), z(512), EPS, z(0, dtype=i32), z(32), z(0, dtype=torch.int64), z(5, 576, dtype=u8), z(5))
    torch.cuda.synchronize()


def codes_on_gpu(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, device=DEV, generator=g)
    return c.masked_fill_((c & 0x7F) == 0x7F, 0x3A)


@pytest.mark.parametrize("M,N,K", [(70000, 40, 32768), (3, 70000, 32768), (300, 70000, 32768)])
def test_matmul_operands_past_32_bits(lib, M, N, K):
    a8, w8 = codes_on_gpu(M, K, 1), codes_on_gpu(N, K, 2)
    g = gen(M)
    kb = K // BLK
    sa, sw = (torch.exp2(torch.randn(s, generator=g) - 6).to(DEV) for s in ((kb, M), (-(-N // BLK), kb)))
    out = torch.empty((M, N), device=DEV)
    lib.kv8_matmul8(a8, sa, w8, sw, out)
    rows = torch.arange(M, device=DEV)[-2:] if M > 1000 else torch.arange(2, device=DEV)
    first = N - N % BLK - BLK  # the last whole block of columns and what follows it
    first = max(first, 0)
    ref, tol = matmul(a8[rows], sa[:, rows].contiguous(), w8[first:].contiguous(), sw[first // BLK:].contiguous(), F32)
    assert bool(((out[rows][:, first:].double() - ref).abs() <= tol).all())
    assert bool(torch.isfinite(out).all())


def test_quant_and_rows_past_32_bits(lib):
    n, width = 140000, 16384  # 2.3e9 values
    x = torch.randn((n, width), device=DEV, generator=torch.Generator(device="cuda").manual_seed(1), dtype=BF)
    q, s = torch.empty((n, width), dtype=torch.uint8, device=DEV), torch.empty((width // BLK, n), device=DEV)
    rows = torch.tensor([0, 131071, 131072, n - 1], device=DEV)
    w = torch.ones(width, device=DEV)
    for norm_w in (None, w):
        lib.kv8_quant_blocks(x, q, s, norm_w=norm_w)
        blocks_check(x[rows], norm_w, 1e-6, q[rows], s[:, rows])
    del x, q, s
    g = gen(2)
    xs, w, pos, f, dst, _, _, scale, layout, eps = rows_case(lib, g, 50, BF, 0, 0)
    kv8, ks = torch.empty((4000000, 576), dtype=torch.uint8, device=DEV), torch.empty(4000000, device=DEV)
    dst = (3999999 - dst).contiguous()
    lib.kv8_norm_rope_rows(xs, w, eps, pos, f, dst, kv8, ks, rope_scale=scale)
    check_codes(kv8[dst], ks[dst], *rows_ref(xs, w, pos, f, scale, layout, eps))


def test_matmul_outputs_past_32_bits(lib):
    M, N, K = 70000, 32768, 16  # 2.3e9 outputs
    g = gen(1)
    w8, sw = weight(g, N, K, DEV)
    a8, _ = weight(g, M, K, DEV)
    sa = torch.ones((1, M), device=DEV)
    out = torch.empty((M, N), dtype=BF, device=DEV)
    lib.kv8_matmul8(a8, sa, w8, sw, out)
    rows = torch.tensor([0, 1, 127, 128, 35000, 65535, 65536, 69999], device=DEV)
    ref, tol = matmul(a8[rows], sa[:, rows], w8, sw, BF)
    assert bool(((out[rows].double() - ref).abs() <= tol).all())
    assert bool(torch.isfinite(out[::997]).all())


# -------------------------------------------------------------------------------------------------------------
# arguments, streams, graphs
# -------------------------------------------------------------------------------------------------------------
def test_tensors_that_do_not_fit_are_refused(lib):
    z = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    i32, u8 = torch.int32, torch.uint8
    rope = dict(x=z(4, 2, 192), position=z(4, dtype=i32), inv_freq=z(32), rope_at=128, rot=z(4, 2, 64), rest=z(4, 2, 128))
    lib.kv8_rope(**rope)
    for bad in [dict(x=z(4, 2, 192).half()), dict(x=z(4, 2, 192).cpu()), dict(position=z(4, dtype=torch.int64)), dict(position=z(3, dtype=i32)),
                dict(inv_freq=z(31)), dict(inv_freq=z(32).double()), dict(rot=z(3, 2, 64)), dict(rest=z(4, 2, 127)), dict(rest=z(4, 2, 128).to(BF)),
                dict(rot=z(4, 64, 2).transpose(1, 2)), dict(x=z(4, 192, 2).transpose(1, 2))]:
        with pytest.raises((TypeError, ValueError)):
            lib.kv8_rope(**{**rope, **bad})
    with pytest.raises(lib.Kv8Error):
        lib.kv8_rope(**{**rope, "rope_at": 129})
    rows = dict(x=z(4, 576), norm_w=z(512), eps=EPS, position=z(4, dtype=i32), inv_freq=z(32), dst_rows=torch.arange(4, device=DEV), kv8=z(9, 576, dtype=u8),
                kv_scale=z(9))
    lib.kv8_norm_rope_rows(**rows)
    for bad in [dict(x=z(4, 575)), dict(x=z(576, 4).t()), dict(norm_w=z(511)), dict(norm_w=z(512).to(BF)), dict(dst_rows=torch.arange(4, device=DEV, dtype=i32)),
                dict(kv8=z(9, 575, dtype=u8)), dict(kv_scale=z(8)), dict(kv8=z(9, 576)), dict(err_word=z(2, dtype=i32)), dict(position=z(4))]:
        with pytest.raises((TypeError, ValueError)):
            lib.kv8_norm_rope_rows(**{**rows, **bad})
    quant = dict(x=z(4, 256), q=z(4, 256, dtype=u8), scale=z(2, 4), norm_w=z(256))
    lib.kv8_quant_blocks(**quant)
    for bad in [dict(x=z(4, 255)), dict(q=z(4, 256)), dict(q=z(256, 4, dtype=u8).t()), dict(scale=z(4, 2)), dict(scale=z(4, 2).t()), dict(norm_w=z(255)),
                dict(scale=z(3, 4)), dict(x=z(4, 256).double())]:
        with pytest.raises((TypeError, ValueError)):
            lib.kv8_quant_blocks(**{**quant, **bad})
    mm = dict(a8=z(4, 256, dtype=u8), a_scale=z(2, 4), w8=z(128, 256, dtype=u8), w_scale=z(1, 2), out=z(4, 128))
    lib.kv8_matmul8(**mm)
    for bad in [dict(a8=z(4, 255, dtype=u8)), dict(a_scale=z(4, 2)), dict(a_scale=z(3)), dict(w8=z(128, 240, dtype=u8)), dict(w_scale=z(2, 2)), dict(out=z(4, 127)),
                dict(out=z(128, 4).t()), dict(out=z(4, 128).half()), dict(w8=z(256, 128, dtype=u8).t()), dict(a8=z(4, 256))]:
        with pytest.raises((TypeError, ValueError)):
            lib.kv8_matmul8(**{**mm, **bad})
    with pytest.raises(lib.Kv8Error):  # rows that do not lie on 16 bytes
        lib.kv8_matmul8(**{**mm, "a8": z(4, 264, dtype=u8)[:, :256]})
    with pytest.raises(lib.Kv8Error):  # the first byte of a8 off 16
        lib.kv8_matmul8(**{**mm, "a8": z(4, 272, dtype=u8)[:, 8:264]})


def layer_calls(lib, g, n):
    """Every call of this file on a batch of its own: (a function that makes them, its outputs)."""
    hid, H = 512, 16
    x = randn((n, hid), g, BF)
    nw = (1 + 0.2 * torch.randn(hid, generator=g)).to(DEV)
    w8, sw = weight(g, H * 192, hid, DEV)
    v8, sv = weight(g, 576, hid, DEV)
    lw = (1 + 0.2 * torch.randn(512, generator=g)).to(DEV)
    pos, f = positions(n, g), lib.kv8_rope_freqs(64)[0].to(DEV)
    q, s = torch.empty((n, hid), dtype=torch.uint8, device=DEV), torch.empty((hid // BLK, n), device=DEV)
    heads, fresh = torch.empty((n, H * 192), dtype=BF, device=DEV), torch.empty((n, 576), device=DEV)
    rot, rest = torch.empty((n, H, 64), dtype=BF, device=DEV), torch.empty((n, H, 128), dtype=BF, device=DEV)
    kv8, ks = torch.zeros((n, 576), dtype=torch.uint8, device=DEV), torch.zeros(n, device=DEV)
    dst = torch.randperm(n, generator=g).to(DEV)

    def go(stream=None):
        lib.kv8_quant_blocks(x, q, s, norm_w=nw, stream=stream)
        lib.kv8_matmul8(q, s, w8, sw, heads, stream=stream)
        lib.kv8_matmul8(q, s, v8, sv, fresh, stream=stream)
        lib.kv8_rope(heads.view(n, H, 192), pos, f, 128, rot, rest, stream=stream)
        lib.kv8_norm_rope_rows(fresh, lw, EPS, pos, f, dst, kv8, ks, stream=stream)
    return go, (q, s, heads, fresh, rot, rest, kv8, ks), x


def test_captured_replayed_and_on_two_streams(lib):
    made = [layer_calls(lib, gen(20 + i), n) for i, n in enumerate((3, 150))]
    want = []
    for go, outs, _ in made:
        go()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(3):
        for (_, outs, _) in made:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        for st, (go, _, _) in zip(streams, made):
            go(st)
        torch.cuda.synchronize()
        for (_, outs, _), w in zip(made, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, w))
    graphs = []
    for st, (go, _, _) in zip(streams, made):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            go()
        graphs.append(graph)
    new = [randn(tuple(x.shape), gen(30 + i), BF) for i, (_, _, x) in enumerate(made)]
    for (_, outs, x), y in zip(made, new):
        x.copy_(y)
    torch.cuda.synchronize()
    for st, graph in zip(streams, graphs):
        with torch.cuda.stream(st):
            graph.replay()
    torch.cuda.synchronize()
    replayed = [[o.clone() for o in outs] for _, outs, _ in made]
    for (go, outs, _), r in zip(made, replayed):
        go()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, r))


@pytest.mark.parametrize("lens,n", [([0], [1]), ([70, 0, 33], [1, 9, 4]), ([500], [130])])
def test_a_layer(lib, lens, n):
    """A layer's attention block as a serving loop runs it, over the paged cache: norm, projections, rotation, fresh rows,
    absorbed tree attention (a chain), value projection, output projection.  Held to the same layer in 64 bits with the
    same quantized rows and activations: what is left are bf16 roundings (2^-8 a value) of the queries and of the attention's
    weights and the f32 steps: 2 % of the output's size is four of the former at their worst."""
    g = gen(len(lens))
    hid, H, page, R = 1024, 8, 16, sum(n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    qw, qs = weight(g, H * 192, hid, DEV)
    kw, ks_ = weight(g, 576, hid, DEV)
    bw, bs = weight(g, H * 256, 512, DEV)
    ow, os_ = weight(g, hid, H * 128, DEV)
    qs, ks_, bs, os_ = qs / 8, ks_ / 8, bs / 4, os_ / 4
    nw, lw = ((1 + 0.2 * torch.randn(m, generator=g)).to(DEV) for m in (hid, 512))
    f, scale = lib.kv8_rope_freqs(64, 10000.0, 4.0, 4096)
    f = f.to(DEV)
    need = [-(-(a + b) // page) for a, b in zip(lens, n)]
    most = max(need) + 1
    table, n_pages = torch.full((len(n), most), -1, dtype=torch.int32, device=DEV), torch.zeros(len(n), dtype=torch.int32, device=DEV)
    total = sum(need) + 2
    free, n_free = torch.randperm(total, generator=g).to(torch.int32).to(DEV), i32([total])
    kv8, kv_scale = torch.full((total * page, 576), 0x7F, dtype=torch.uint8, device=DEV), torch.full((total * page,), float("nan"), device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def fresh_rows(x, at, starts, pos):
        R = x.shape[0]
        a8, a_s = torch.empty((R, hid), dtype=torch.uint8, device=DEV), torch.empty((hid // BLK, R), device=DEV)
        lib.kv8_quant_blocks(x, a8, a_s, norm_w=nw)
        rows, slots = torch.empty((R, 576), device=DEV), torch.empty(R, dtype=torch.int64, device=DEV)
        lib.kv8_matmul8(a8, a_s, kw, ks_, rows, err_word=err)
        lib.kv8_page_plan(i32(at), i32(starts), page, n_pages, table, free, n_free, slots, err_word=err)
        lib.kv8_norm_rope_rows(rows, lw, EPS, pos, f, slots, kv8, kv_scale, rope_scale=scale, err_word=err)
        return a8, a_s

    # the context, in steps of up to 256 rows a sequence
    done = [0] * len(lens)
    while done != lens:
        step = [min(256, t - d) for t, d in zip(lens, done)]
        starts = [0] + np.cumsum(step).tolist()
        pos = torch.cat([torch.arange(d, d + m) for d, m in zip(done, step)]).to(torch.int32).to(DEV)
        fresh_rows(randn((sum(step), hid), g, BF), done, starts, pos)
        done = [d + m for d, m in zip(done, step)]
    # the step
    x = randn((R, hid), g, BF)
    starts = [0] + np.cumsum(n).tolist()
    pos = torch.cat([torch.arange(t, t + m) for t, m in zip(lens, n)]).to(torch.int32).to(DEV)
    a8, a_s = fresh_rows(x, lens, starts, pos)
    heads = torch.empty((R, H * 192), dtype=BF, device=DEV)
    lib.kv8_matmul8(a8, a_s, qw, qs, heads, err_word=err)
    q_rope, q_nope = torch.empty((R, H, 64), dtype=BF, device=DEV), torch.empty((R, H, 128), dtype=BF, device=DEV)
    lib.kv8_rope(heads.view(R, H, 192), pos, f, 128, q_rope, q_nope, rope_scale=scale)
    q_lat = torch.empty((R, H, 512), dtype=BF, device=DEV)
    lib.mla_q_absorb8(q_nope, bw, bs, q_lat, err_word=err)
    ctx = torch.empty((R, H, 512), device=DEV)
    ws = torch.empty(lib.mla_tree8_workspace_bytes(R, H, len(n), BF), dtype=torch.uint8, device=DEV)
    sm = 192.0 ** -0.5
    lib.mla_absorb_tree8(q_lat, q_rope, i32(starts), i32(lens), None, kv8, kv_scale, table, page, sm, ws, ctx, err_word=err)
    value = torch.empty((R, H, 128), device=DEV)
    lib.mla_out_project8(ctx, bw, bs, value, err_word=err)
    o8, o_s = torch.empty((R, H * 128), dtype=torch.uint8, device=DEV), torch.empty((H, R), device=DEV)
    lib.kv8_quant_blocks(value.view(R, H * 128), o8, o_s)
    out = torch.empty((R, hid), dtype=BF, device=DEV)
    lib.kv8_matmul8(o8, o_s, ow, os_, out, err_word=err)
    assert err.item() == 0

    # the same in 64 bits, from the quantized activations and cache rows
    def full(w8, s):
        return values(w8) * s.double().repeat_interleave(BLK, 0)[:w8.shape[0]].repeat_interleave(BLK, 1)[:, :w8.shape[1]]
    act = values(a8) * a_s.double().t().repeat_interleave(BLK, 1)
    y, _ = norm(x.double(), nw.double(), EPS)
    assert float((act - y).norm() / y.norm()) < 2.0 ** -4  # half a step of e4m3 at the worst
    hq = (act @ full(qw, qs).t()).view(R, H, 192)
    rot, _ = rotate(hq[..., 128:], pos, f, scale, 0)
    kvb = full(bw, bs).view(H, 256, 512)
    tab, want = table.long().cpu(), torch.empty((R, H, 128), dtype=torch.float64, device=DEV)
    for b, (t, m) in enumerate(zip(lens, n)):
        p = torch.arange(t + m)
        rows = (tab[b, p // page] * page + p % page).to(DEV)
        c = values(kv8[rows]) * kv_scale[rows].double()[:, None]
        r = slice(starts[b], starts[b + 1])
        k = torch.einsum("tc,hdc->thd", c[:, :512], kvb[:, :128])
        v = torch.einsum("tc,hdc->thd", c[:, :512], kvb[:, 128:])
        s = sm * (torch.einsum("rhd,thd->hrt", hq[r, :, :128], k) + torch.einsum("rhd,td->hrt", rot[r], c[:, 512:]))
        off = torch.arange(t + m, device=DEV)[None] > t + torch.arange(m, device=DEV)[:, None]
        want[r] = torch.einsum("hrt,thd->rhd", torch.softmax(s.masked_fill(off, -torch.inf), -1), v)
    assert float((value.double() - want).norm() / want.norm()) < 0.02
    oo = values(o8) * o_s.double().t().repeat_interleave(BLK, 1)
    assert float((oo - value.double().view(R, -1)).norm() / value.double().norm()) < 2.0 ** -4
    last = oo @ full(ow, os_).t()
    assert float((out.double() - last).norm() / last.norm()) < 2.0 ** -8
