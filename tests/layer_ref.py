"""Plain references, in 64 bits, of the calls that stand around the attention in a layer, and the bounds of their outputs.

A rounding is off by half a step of its type at most, relative: U = 2^-24 (f32), 2^-8 (bf16), 2^-4 (e4m3)."""
from __future__ import annotations

import torch

U = 2.0 ** -24
OUT_EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BLK = 128


def nearest(y):
    """The e4m3 value next to y (f64), ties to even, at most 448; NaN gives 0."""
    y = torch.nan_to_num(y, nan=0.0, posinf=448.0, neginf=-448.0)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def values(codes):
    """e4m3 codes as f64."""
    return codes.view(torch.float8_e4m3fn).double()


def rotate(x, position, inv_freq, scale, layout):
    """x [n][heads][dim] f64 -> (rotated, what an element of it may be off by before its output rounding).

    The bound: an angle's fraction of a turn is held to 2^-32; the rest after whole quarters, pi/4 at most, is off by that and
    three roundings (conversion, constant, product): 2 pi 2^-32 + 3 U pi/4 < 2.4 U.  The series of its cosine and sine end 2^-29
    (0.04 U) early and round twice at the end: below 5 U.  The scale, a product and the sum round once each: under 12 U
    (|u| + |v|) |scale| in all, with room for the products of errors."""
    a = (position.double()[:, None] * inv_freq.double())[:, None]
    d = x.shape[-1]
    i, j = (slice(0, None, 2), slice(1, None, 2)) if layout == 0 else (slice(0, d // 2), slice(d // 2, d))
    u, v = x[..., i], x[..., j]
    out, tol = torch.empty_like(x), torch.empty_like(x)
    out[..., i] = scale * (u * torch.cos(a) - v * torch.sin(a))
    out[..., j] = scale * (u * torch.sin(a) + v * torch.cos(a))
    tol[..., i] = tol[..., j] = 12 * U * (u.abs() + v.abs()) * abs(scale)
    return out, tol


def norm(x, w, eps):
    """x [n][width] f64 -> (normed, relative bound of an element).  The f32 sum of squares rounds once for each term and level of
    its tree, at most width / 32 + 13 times U in a row, half of which enters the root; the mean, the root and three products
    round once each."""
    width = x.shape[-1]
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return y, ((width / 32 + 13) / 2 + 6) * U


def check_codes(codes, scales, y, rel, tol, what=""):
    """Codes [n][width] and scales [n] of rows y (f64) that the kernel holds to rel |y| + tol: the scale is amax / 448, every
    code is the nearest value to what y times 448 / amax may be (two roundings more)."""
    fin = torch.isfinite(y)
    amax = torch.where(fin, y.abs(), torch.zeros_like(y)).amax(-1)
    slack = rel * amax + torch.where(fin, tol, torch.zeros_like(y)).amax(-1)  # the largest element's own error
    s = scales.double()
    assert bool(((s - amax / 448).abs() <= (slack + 2 * U * amax) / 448 + 2.0 ** -149).all()), f"{what}: scales"
    some = amax > 0
    inv = torch.where(some, 448 / torch.where(some, amax, torch.ones_like(amax)), torch.ones_like(amax))[:, None]
    z = y * inv
    off = (rel * y.abs() + tol) * inv + z.abs() * (slack[:, None] * inv / 448 + 4 * U)
    off = torch.nan_to_num(off, nan=0.0, posinf=0.0)
    got = values(codes)
    bad = ~((got >= nearest(z - off)) & (got <= nearest(z + off)))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes, the first at {bad.nonzero()[0].tolist()}"


def matmul(a8, a_scale, w8, w_scale, out_dtype):
    """(out f64, bound).  S = the sum of the terms' sizes.  Products of two e4m3 values are exact; the tensor cores add 128 of
    them in f32 and may cut a term at the last bit of the sum (2 U at most each): 256 U; a scaled block's sum rounds its factor,
    its product and its place in the sum over blocks: kb + 4 times U."""
    M, K = a8.shape
    N = w8.shape[0]
    kb = -(-K // BLK)
    a, w = values(a8.contiguous()), values(w8)
    sa = a_scale.double()[None].expand(kb, M) if a_scale.dim() == 1 else a_scale.double()
    sw = w_scale.double().repeat_interleave(BLK, 0)[:N]
    out = torch.zeros((M, N), dtype=torch.float64, device=a8.device)
    size = torch.zeros_like(out)
    for k in range(kb):
        c = slice(k * BLK, (k + 1) * BLK)
        x, y = a[:, c] * sa[k][:, None], w[:, c] * sw[:, k:k + 1]
        out += x @ y.t()
        size += x.abs() @ y.abs().t()
    tol = size * (256 + kb + 4) * U
    return out, tol + OUT_EPS[out_dtype] * (out.abs() + tol) + 1e-37


def weight(g, N, K, device):
    """A random fmt=8 weight: codes [N][K] without NaN, scales [ceil(N/128)][ceil(K/128)]."""
    codes = torch.randint(0, 256, (N, K), generator=g, dtype=torch.uint8)
    codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)
    scale = torch.exp2(torch.randn((-(-N // BLK), -(-K // BLK)), generator=g) * 2 - 8)
    return codes.to(device), scale.to(device)
