"""Plain references of the paged calls, in 64 bits and one sequence at a time, and the bounds of the
attention's outputs."""
from __future__ import annotations

import numpy as np
import torch

SM = float(np.float32(1.0 / np.sqrt(192.0)))
TABLE = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
BAD_INDEX, BAD_PAGES = 1, 4


def closure(parent):
    """[n][n] bool: which tokens each one attends (itself and its ancestors)."""
    n = len(parent)
    sees = np.zeros((n, n), dtype=bool)
    for i in range(n):
        a = i
        while a >= 0:
            sees[i, a] = True
            a = parent[a]
    return sees


def pack(sees, words):
    """Rows of [R][words] int32 bits of [n][m] bools."""
    out = np.zeros((sees.shape[0], words), dtype=np.uint32)
    for i, j in zip(*np.nonzero(sees)):
        out[i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    return out.view(np.int32)


def attend(q, sees, ctx, rows, valid, kv8, scale, out_eps, f32):
    """Outputs [n][H][512] of one sequence and what each element may be off by.

    q [n][H][576] f64, sees [n][n] bool, rows: cache rows of positions 0 .. ctx+n-1, valid: those that count.
    The bound, term by term (A = sum_t p_t s_t |v_t|, the size of the sum's terms):
      scores   |d score| <= sm s_t (u q_max sum|k| + v sum|q||k|): u the part of a head's largest query element
               that a query element is rounded to (bf16: 2^-17, f32: 2^-39), v the sum's, 576 2^-24: for bf16 2^-24 a
               step of at most 576; for f32 18 products of 16 elements each a quarter, whose 17 terms may each be cut at
               2^-24 of the largest, and 2^-22 of an element that its two pieces leave: 306 + 3 + 4 steps of 2^-24.
               Each weight is then off by exp(+-2 d) relative.
      weights  2 steps of exp2 and a product.  f32: two f16 pieces of w = p_t s_t, which leave 2^-22 of it, or 2^-25 where
               the step's largest is 2^13 or more.  bf16: the weights w = p_t s_t of 32 rows (positions 32 i to 32 i +
               31) are held in units that put the largest of them at 2^7 or more, or, in a tile of 64 context rows with
               scales within 2^8 of one another, the largest p_t times the power of two above the largest s_t; rounded to 11 bits (2^-12 w at most),
               then to an e4m3 value, which leaves at most 2^-4 w (2^-10 where it is subnormal, or all of w below that),
               and that to another (2^-4 of it, or 2^-10 where that is subnormal): at most 2^-8 w + 2^-10, each times the
               row's |e4m3 value|.
      sum      32 bits, one step for each row and one for each part; f32: in 64 rows 8 products of 17 terms, as above
      output   out_eps relative (half a step of its type)
    """
    n, H, _ = q.shape
    k = TABLE[kv8[rows]] * scale[rows].astype(np.float64)[:, None]
    T = len(rows)
    out = np.zeros((n, H, 512))
    tol = np.zeros((n, H, 512))
    for i in range(n):
        on = valid.copy()
        on[ctx:] &= sees[i]
        if not on.any():
            continue
        kk = k[on]
        s = SM * q[i] @ kk.T
        qk = SM * np.abs(q[i]) @ np.abs(kk).T
        d = 576 * 2.0 ** -24 * qk
        d = d + (2.0 ** -39 if f32 else 2.0 ** -17) * SM * np.abs(q[i]).max(1)[:, None] * np.abs(kk).sum(1)[None]
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[i] = p @ kk[:, :512]
        A = p @ np.abs(kk[:, :512])
        # exp(2 d) - 1 for every row, weighted as the terms are, twice: numerator and denominator
        e = np.expm1(2 * d)
        tol[i] = (p * e) @ np.abs(kk[:, :512]) + (p * e).sum(1)[:, None] * A
        tol[i] += A * (2.0 ** -21 + (2 * T + 64) * 2.0 ** -24)
        ps = p * scale[rows[on]].astype(np.float64)
        if f32:
            tol[i] += A * (2.0 ** -22 + 136 * 2.0 ** -24)
            tol[i] += 2.0 ** -38 * ps.max(1, keepdims=True) * np.abs(TABLE[kv8[rows[on]]][:, :512]).sum(0)
        else:
            block = np.nonzero(on)[0] // 32
            st = scale[rows[on]].astype(np.float64)
            unit, pm, sm_, sl = (np.zeros((H, T // 32 + 2)) for _ in range(4))
            np.maximum.at(unit.T, block, ps.T)
            np.maximum.at(pm.T, block, p.T)
            np.maximum.at(sm_.T, block, np.broadcast_to(st[:, None], ps.T.shape))
            sl[:] = np.inf
            np.minimum.at(sl.T, block, np.broadcast_to(st[:, None], ps.T.shape))
            unit = np.where(sm_ <= 256 * sl, np.maximum(unit, 2 * pm * sm_), unit)
            off = (2.0 ** -8 + 2.0 ** -12) * ps + 2.0 ** -10 * unit[:, block] / 128
            tol[i] += off @ np.abs(TABLE[kv8[rows[on]]][:, :512])
        tol[i] += out_eps * (np.abs(out[i]) + tol[i]) + 1e-30
    return out, tol


def plan(lens, n, page, n_pages, table, free, n_free, most):
    """kv8_page_plan on lists; returns (slots per sequence or None, err); the lists are updated."""
    err, B = 0, len(lens)
    want = []
    for b in range(B):
        if lens[b] < 0 or n[b] < 0 or n[b] > 256 or not 0 <= n_pages[b] <= most:
            want.append(None)
            err |= BAD_INDEX
        else:
            want.append(-(-(lens[b] + n[b]) // page))
    give = []
    for b in range(B):
        if want[b] is not None and want[b] <= most:
            give += table[b][want[b]:n_pages[b]]
    if not 0 <= n_free <= len(free) or n_free + len(give) > len(free):
        return [None] * B, n_free, err | BAD_INDEX
    free[n_free:n_free + len(give)] = give[::-1]
    top = n_free + len(give)
    asked = took = 0
    slots = []
    for b in range(B):
        if want[b] is None:
            slots.append(None)
            continue
        ok = want[b] <= most
        need = max(0, want[b] - n_pages[b]) if ok else 0
        if ok and need:
            asked += need
            ok = asked <= top
        if not ok:
            err |= BAD_PAGES
            slots.append([-1] * n[b])
            continue
        for k in range(need):
            table[b][n_pages[b] + k] = free[top - 1 - took]
            took += 1
        n_pages[b] = want[b]
        slots.append([table[b][(lens[b] + i) // page] * page + (lens[b] + i) % page for i in range(n[b])])
    return slots, top - took, err
