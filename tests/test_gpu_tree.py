"""Drafted tokens over a paged cache: plan, mask, tree attention and commit against plain references, each alone
and together as a serving loop runs them.

Attention outputs are held to a bound for every element (tests/tree_ref.py derives it); whole numbers and moved
bytes are equal."""
import numpy as np
import pytest
import torch

import synth
from tree_ref import BAD_INDEX, BAD_PAGES, SM, attend, closure, pack, plan

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
GARBAGE = 0x7F  # an e4m3 NaN code


def i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int64), dtype=torch.int64).to(torch.int32).to(DEV)


def build(oracle, rng, lens, n, page, spare=3, lo=0.5, hi=2.0):
    """A scattered paged cache whose unused rows hold NaN codes and scales: (kv8, scale, table, rows per sequence)."""
    need = [-(-(x + y) // page) for x, y in zip(lens, n)]
    total = sum(need) + spare
    perm = rng.permutation(total)
    kv8 = np.full((total * page, 576), GARBAGE, dtype=np.uint8)
    scale = np.full(total * page, np.nan, dtype=np.float32)
    table = np.full((len(lens), max(max(need), 1) + 1), -7, dtype=np.int64)
    at, rows = 0, []
    for b, (t, m) in enumerate(zip(lens, n)):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        pos = np.arange(t + m)
        r = table[b, pos // page] * page + pos % page
        if t + m:
            kv8[r], scale[r] = oracle.quant_rows(synth.latent_rows(rng, t + m, lo, hi))
        rows.append(r)
    return kv8, scale, table, rows


def run_tree(lib, q, q_dtype, out_dtype, n, lens, mask, kv8, scale, table, page, fill=7.0, rows=None, sm=SM, start=None):
    """The call, on tensors; rows: how many q rows the batch really has (more than the sequences' sum allowed)."""
    R, H = q.shape[0], q.shape[1]
    ql = torch.from_numpy(np.ascontiguousarray(q[..., :512])).to(DEV).to(q_dtype)
    qr = torch.from_numpy(np.ascontiguousarray(q[..., 512:])).to(DEV).to(q_dtype)
    out = torch.full((R, H, 512), fill, dtype=out_dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full((lib.mla_tree8_workspace_bytes(R, H, len(lens), q_dtype),), 0xFF, dtype=torch.uint8, device=DEV)
    start = i32(np.concatenate([[0], np.cumsum(n)]) if start is None else start)
    lib.mla_absorb_tree8(ql, qr, start, i32(lens), None if mask is None else torch.from_numpy(mask).to(DEV),
                         torch.from_numpy(kv8).to(DEV), torch.from_numpy(scale).to(DEV), i32(table), page, sm, ws, out,
                         err_word=err)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), err.item()


def check(got, q, n, lens, sees, kv8, scale, rows, out_dtype, f32, valid=None, what=""):
    at = 0
    for b in range(len(lens)):
        on = np.ones(lens[b] + n[b], dtype=bool) if valid is None else valid[b]
        ref, tol = attend(q[at:at + n[b]].astype(np.float64), sees[b], lens[b], rows[b], on, kv8, scale, EPS[out_dtype], f32)
        d = np.abs(got[at:at + n[b]] - ref)
        assert np.isfinite(got[at:at + n[b]]).all(), f"{what} sequence {b}: not finite"
        assert (d <= tol).all(), f"{what} sequence {b}: off by {(d - tol).max():.3g} over the bound, {(d / tol).max():.3g} times it"
        at += n[b]


def queries(rng, R, H, f32):
    q = rng.standard_normal((R, H, 576)).astype(np.float32)
    return q if f32 else synth.to_bf16_values(q)


def trees(rng, n):
    return [[int(rng.integers(max(-1, i - 6), i)) for i in range(m)] for m in n]


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("H,q_dtype,out_dtype,page,lens,n", [
    (16, F32, F32, 16, [5], [1]),
    (5, F32, F32, 32, [0, 63, 64, 65], [1, 3, 0, 7]),
    (128, F32, BF, 64, [200, 0], [2, 9]),
    (33, F32, F32, 128, [700], [4]),
    (1, BF, F32, 16, [0], [1]),
    (128, BF, BF, 64, [127], [1]),
    (128, BF, F32, 128, [128], [1]),
    (128, BF, BF, 64, [1000], [16]),
    (16, BF, BF, 16, [0, 127, 128, 129, 640, 1], [13, 1, 0, 5, 31, 32]),
    (65, BF, BF, 32, [300, 17], [3, 2]),
    (100, BF, F32, 256, [257, 3, 255], [5, 1, 40]),
    (7, BF, BF, 1024, [1500, 20], [64, 1]),
    (20, BF, BF, 16, [31, 511], [33, 100]),
])
def test_tree_attention(lib, oracle, H, q_dtype, out_dtype, page, lens, n):
    rng = np.random.default_rng(H * 1000 + page + sum(lens))
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    parent = trees(rng, n)
    sees = [closure(p) for p in parent]
    words = max(1, -(-max(n) // 32))
    mask = np.concatenate([pack(s, words) for s in sees]) if sum(n) else np.zeros((0, words), np.int32)
    q = queries(rng, sum(n), H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, out_dtype, n, lens, mask, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, sees, kv8, scale, rows, out_dtype, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_chain_without_a_mask_and_the_longest_draft(lib, oracle, q_dtype):
    rng = np.random.default_rng(3)
    H, lens, n, page = 8, [70, 0], [256, 5], 64
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    q = queries(rng, sum(n), H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, [np.tril(np.ones((m, m), bool)) for m in n], kv8, scale, rows, F32, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_many_sequences_more_than_the_shares(lib, oracle, q_dtype):
    rng = np.random.default_rng(4)
    B, H, page = 300, 16, 16
    lens = [int(x) for x in rng.integers(0, 200, B)]
    n = [int(x) for x in rng.integers(0, 4, B)]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    parent = trees(rng, n)
    sees = [closure(p) for p in parent]
    mask = np.concatenate([pack(s, 1) for s in sees])
    q = queries(rng, sum(n), H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, BF, n, lens, mask, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, sees, kv8, scale, rows, BF, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_any_bits_empty_rows_and_garbage_where_nobody_attends(lib, oracle, q_dtype):
    """Masks that are no tree, tokens that attend nothing, drafted rows of NaN codes and of NaN / infinite / huge
    scales that only some tokens leave out, and rows behind the last sequence."""
    rng = np.random.default_rng(5)
    H, lens, n, page = 16, [0, 150, 0], [6, 40, 3], 32
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    sees = [rng.random((m, m)) < 0.4 for m in n]
    sees[0][2] = False            # attends nothing at all: zeros
    sees[2][:] = False
    for b, j, kind in [(0, 4, "codes"), (1, 7, "nan"), (1, 8, "inf"), (1, 9, "huge"), (1, 20, "codes")]:
        r = rows[b][lens[b] + j]
        if kind == "codes":
            kv8[r, ::3] = 0xFF
        else:
            scale[r] = {"nan": np.nan, "inf": np.inf, "huge": 1e30}[kind]
        sees[b][:, j] = False
    mask = np.concatenate([pack(s, 2) for s in sees])
    extra = 2
    mask = np.concatenate([mask, np.full((extra, 2), -1, np.int32)])
    q = queries(rng, sum(n) + extra, H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, mask, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, sees, kv8, scale, rows, F32, q_dtype == F32)
    assert not got[2].any() and not got[46:49].any()
    assert (got[sum(n):] == 7.0).all()
    # a token that does attend the NaN codes says so; one that does not is unchanged
    sees[1][5, 20] = True
    mask2 = np.concatenate([np.concatenate([pack(s, 2) for s in sees]), np.full((extra, 2), -1, np.int32)])
    got2, _ = run_tree(lib, q, q_dtype, F32, n, lens, mask2, kv8, scale, table, page)
    keep = np.ones(len(got), bool)
    keep[6 + 5] = False
    assert np.isnan(got2[6 + 5][:, 0]).all() and np.array_equal(got2[keep], got[keep])


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_queries_that_are_not_finite(lib, oracle, q_dtype):
    """A NaN or an infinity of either sign in a (token, head)'s query, latent or RoPE, makes that output NaN and leaves
    every other as it was; a token that attends nothing gives zeros all the same."""
    rng = np.random.default_rng(31)
    H, lens, n, page = 24, [130, 0], [5, 3], 64
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    sees = [np.tril(np.ones((m, m), bool)) for m in n]
    sees[1][1] = False
    mask = np.concatenate([pack(s, 1) for s in sees])
    q = queries(rng, sum(n), H, q_dtype == F32)
    q[6, 0, 7] = 0.0
    ref, _ = run_tree(lib, q, q_dtype, F32, n, lens, mask, kv8, scale, table, page)
    bad = [(0, 0, 3, np.nan), (1, 5, 511, np.inf), (2, 23, 512, -np.inf), (4, 9, 575, np.nan), (5, 2, 100, -np.inf)]
    hit = np.zeros((sum(n), H), bool)
    for r, h, k, v in bad:
        q[r, h, k] = v
        hit[r, h] = True
    q[6, 0, 7] = np.inf           # attends nothing
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, mask, kv8, scale, table, page)
    assert err == 0
    assert np.isnan(got[hit]).all()
    assert np.array_equal(got[~hit], ref[~hit]) and not got[6].any()


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_pages_that_sequences_share(lib, oracle, q_dtype):
    """Three sequences whose contexts begin with the same two pages, each with its own pages behind them."""
    rng = np.random.default_rng(37)
    H, page, lens, n = 16, 64, [130, 128, 190], [9, 3, 1]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    for b in (1, 2):
        table[b, :2] = table[0, :2]
        rows[b] = np.concatenate([rows[0][:128], rows[b][128:]])
    sees = [np.tril(np.ones((m, m), bool)) for m in n]
    q = queries(rng, sum(n), H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, sees, kv8, scale, rows, F32, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_the_most_sequences(lib, oracle, q_dtype):
    """4096 sequences of 0 to 2 tokens over contexts of 0 to 70 rows; every 37th is checked."""
    rng = np.random.default_rng(39)
    B, H, page = 4096, 8, 16
    n = [int(x) for x in rng.integers(0, 3, B)]
    lens = [int(x) for x in rng.integers(0, 71, B)]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    q = queries(rng, sum(n), H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    assert err == 0 and np.isfinite(got).all()
    at = np.concatenate([[0], np.cumsum(n)])
    pick = [b for b in range(0, B, 37) if n[b]]
    own = np.concatenate([np.arange(at[b], at[b + 1]) for b in pick])
    check(got[own], q[own], [n[b] for b in pick], [lens[b] for b in pick], [np.tril(np.ones((n[b], n[b]), bool)) for b in pick],
          kv8, scale, [rows[b] for b in pick], F32, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_a_long_context(lib, oracle, q_dtype):
    """50000 rows: many steps of one column's sums, and every share a part of two groups."""
    rng = np.random.default_rng(41)
    H, page, lens, n = 3, 128, [50000], [2]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    q = queries(rng, sum(n), H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, [np.tril(np.ones((2, 2), bool))], kv8, scale, rows, F32, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_softmax_scales_of_either_sign_and_zero(lib, oracle, q_dtype):
    """A negative sm_scale is the positive one with the queries' signs turned (the products' signs alone differ, so to the
    bit); with 0 every row counts the same, to the bounds of a query of zeros."""
    rng = np.random.default_rng(33)
    H, lens, n, page = 20, [200, 0], [7, 4], 64
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    sees = [np.tril(np.ones((m, m), bool)) for m in n]
    q = queries(rng, sum(n), H, q_dtype == F32)
    pos, _ = run_tree(lib, -q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    neg, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page, sm=-SM)
    assert err == 0 and np.array_equal(neg, pos)
    flat, _ = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page, sm=0.0)
    check(flat, 0 * q, n, lens, sees, kv8, scale, rows, F32, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_starts_that_go_back_spare_the_sequences_after_them(lib, oracle, q_dtype):
    """q_start 9, 0, 4, 9: the first sequence is impossible, the others are as they would be alone."""
    rng = np.random.default_rng(35)
    H, lens, n, page = 128, [40, 130, 7], [1, 4, 5], 16
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    q = queries(rng, 9, H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page, start=[9, 0, 4, 9])
    assert err == BAD_INDEX
    check(got, q, n[1:], lens[1:], [np.tril(np.ones((m, m), bool)) for m in n[1:]], kv8, scale, rows[1:], F32, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_zero_and_tiny_rows_count_in_the_softmax(lib, oracle, q_dtype):
    """Rows of zeros (scale 0), of a subnormal maximum, and of magnitudes eleven binary orders apart."""
    rng = np.random.default_rng(6)
    H, lens, n, page = 16, [260], [3], 64
    kv8, scale, table, rows = build(oracle, rng, lens, n, page, lo=1e-2, hi=2.0)
    r = rows[0]
    kv8[r[:40]], scale[r[:40]] = oracle.quant_rows(np.zeros((40, 576), np.float32))
    kv8[r[40:60]], scale[r[40:60]] = oracle.quant_rows((rng.standard_normal((20, 576)) * 1e-39).astype(np.float32))
    q = queries(rng, 3, H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, [np.tril(np.ones((3, 3), bool))], kv8, scale, rows, F32, q_dtype == F32)
    # nothing but zero rows: zeros, not a division by zero
    kv8[r], scale[r] = oracle.quant_rows(np.zeros((263, 576), np.float32))
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    assert err == 0 and not got.any()


@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("at", ["first", "last", "draft"])
def test_whole_tiles_of_zero_rows(lib, oracle, q_dtype, at):
    """Tiles, and whole shares of the work, that hold nothing but zero rows; drafted zero rows that only some tokens
    attend; rows of small magnitude beside them."""
    rng = np.random.default_rng(61)
    H, lens, n, page = 16, [1500, 200], [3, 40], 64
    kv8, scale, table, rows = build(oracle, rng, lens, n, page, lo=1e-3, hi=2e-3)
    for b, r in enumerate(rows):
        z = {"first": r[:lens[b] * 3 // 4], "last": r[lens[b] // 4:], "draft": r[lens[b]:][::2]}[at]
        kv8[z], scale[z] = oracle.quant_rows(np.zeros((len(z), 576), np.float32))
    sees = [rng.random((m, m)) < 0.5 for m in n]
    mask = np.concatenate([pack(s, 2) for s in sees])
    q = queries(rng, sum(n), H, q_dtype == F32) * 64
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, mask, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, sees, kv8, scale, rows, F32, q_dtype == F32)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_bad_pages_and_impossible_sequences(lib, oracle, q_dtype):
    rng = np.random.default_rng(7)
    H, lens, n, page = 16, [100, 90, 60, 10], [3, 2, 4, 2], 32
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    table[0, 1] = 10 ** 6          # pages outside the cache: their rows are left out
    table[2, 0] = -1
    valid = [np.ones(x + m, bool) for x, m in zip(lens, n)]
    valid[0][32:64] = False
    valid[2][:32] = False
    told = list(lens)
    told[1] = 10 ** 9              # more positions than its table holds: skipped
    told[3] = -5
    sees = [np.tril(np.ones((m, m), bool)) for m in n]
    q = queries(rng, sum(n), H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, told, None, kv8, scale, table, page)
    assert err == BAD_INDEX
    for b in (0, 2):
        at = sum(n[:b])
        ref, tol = attend(q[at:at + n[b]].astype(np.float64), sees[b], lens[b], np.where(valid[b], rows[b], 0), valid[b],
                          kv8, scale, EPS[F32], q_dtype == F32)
        assert (np.abs(got[at:at + n[b]] - ref) <= tol).all()
    for b in (1, 3):
        at = sum(n[:b])
        assert (got[at:at + n[b]] == 7.0).all()


def test_one_token_each_agrees_with_the_batched_decode(lib, oracle):
    rng = np.random.default_rng(8)
    B, H, T, page = 3, 128, 1024, 64
    lens = [900, 17, 511]
    rows = synth.latent_rows(rng, B * T, 0.5, 2.0)
    kv8, scale = oracle.quant_rows(rows)
    table = np.arange(B * T // page).reshape(B, -1)
    q = queries(rng, B, H, False)
    got, err = run_tree(lib, q, BF, F32, [1] * B, lens, None, kv8, scale, table, page)
    ql, qr = (torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(BF) for x in (q[..., :512], q[..., 512:]))
    out = torch.empty((B, H, 512), dtype=F32, device=DEV)
    ws = torch.empty(lib.mla_batch_decode8_workspace_bytes(B, H, T), dtype=torch.uint8, device=DEV)
    lib.mla_absorb_batch_decode8(ql, qr, torch.from_numpy(kv8).to(DEV), torch.from_numpy(scale).to(DEV), T, T,
                                 i32([x + 1 for x in lens]), SM, ws, out)
    other = out.double().cpu().numpy()
    assert err == 0
    # each is within 2^-8 or so of the same value: their difference within twice that
    assert np.linalg.norm(got - other) <= 2.0 ** -7 * np.linalg.norm(other)


def test_rows_behind_the_31st_bit_of_the_byte_offset(lib, oracle):
    rng = np.random.default_rng(9)
    page, H, lens, n = 256, 16, [600], [5]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    far = 16_000_000 // page        # rows from 16,000,000 on: 9.2 GB into the cache
    big = torch.empty(((far + 8) * page, 576), dtype=torch.uint8, device=DEV)
    sc = torch.empty((far + 8) * page, dtype=F32, device=DEV)
    big[far * page:far * page + len(kv8)] = torch.from_numpy(kv8).to(DEV)
    sc[far * page:far * page + len(kv8)] = torch.from_numpy(scale).to(DEV)
    q = queries(rng, 5, H, False)
    want, _ = run_tree(lib, q, BF, F32, n, lens, None, kv8, scale, table, page)
    out = torch.empty((5, H, 512), dtype=F32, device=DEV)
    for dt in (BF, F32):
        ws = torch.empty(lib.mla_tree8_workspace_bytes(5, H, 1, dt), dtype=torch.uint8, device=DEV)
        ql, qr = (torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(dt) for x in (q[..., :512], q[..., 512:]))
        lib.mla_absorb_tree8(ql, qr, i32([0, 5]), i32(lens), None, big, sc, i32(np.where(table >= 0, table + far, -1)), page,
                             SM, ws, out)
        if dt == BF:
            assert np.array_equal(out.double().cpu().numpy(), want)
        else:
            check(out.double().cpu().numpy(), q, n, lens, [np.tril(np.ones((5, 5), bool))], kv8, scale, rows, F32, True)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_captured_replayed_and_on_two_streams(lib, oracle, q_dtype):
    """A replayed graph follows lengths, tables and queries that change in place; two calls at once with a workspace
    each give what one gives."""
    rng = np.random.default_rng(10)
    H, page, B = 32, 32, 2
    lens, n = [400, 90], [4, 7]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    R = sum(n)
    t = dict(q_start=i32([0, 4, 11]), lens=i32(lens), mask=None, kv8=torch.from_numpy(kv8).to(DEV),
             kv_scale=torch.from_numpy(scale).to(DEV), block_table=i32(table), page_size=page, sm_scale=SM)
    q = queries(rng, R, H, q_dtype == F32)
    ql, qr = (torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(q_dtype) for x in (q[..., :512], q[..., 512:]))
    ws = [torch.empty(lib.mla_tree8_workspace_bytes(R, H, B, q_dtype), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [torch.empty((R, H, 512), dtype=F32, device=DEV) for _ in range(3)]
    lib.mla_absorb_tree8(ql, qr, workspace=ws[0], out=outs[0], **t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                lib.mla_absorb_tree8(ql, qr, workspace=ws[k], out=outs[1 + k], **t)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.mla_absorb_tree8(ql, qr, workspace=ws[0], out=outs[1], **t)
    new_lens = [250, 12]
    t["lens"].copy_(i32(new_lens))
    t["q_start"].copy_(i32([0, 1, 6]))
    outs[1].fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    got = outs[1].double().cpu().numpy()
    n2 = [1, 5]
    check(got, q, n2, new_lens, [np.tril(np.ones((m, m), bool)) for m in n2], kv8, scale,
          [r[:x + m] for r, x, m in zip(rows, new_lens, n2)], F32, q_dtype == F32)
    assert (got[6:] == 7.0).all()


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_many_small_terms_beside_a_large_one(lib, q_dtype):
    """One row whose term is 2^17 times each other's, and 2^17 others that make up half of the sum."""
    T, H, page = 1 << 17, 16, 1024
    kv8 = np.zeros((T + page, 576), np.uint8)
    one = np.uint8(0x38)                        # 1.0
    kv8[:, 0] = one                             # every row's value in dim 0, so that lost terms show
    kv8[T // 2, 1] = one                        # the row that the query asks for
    scale = np.ones(T + page, np.float32)
    q = np.zeros((1, H, 576), np.float32)
    q[:, :, 1] = round(17 * np.log(2) / SM)     # its score: 17 log 2, to the query's whole number
    p = np.exp(SM * q[0, 0, 1])
    got, err = run_tree(lib, q, q_dtype, F32, [1], [T], None, kv8, scale, np.arange(T // page + 1)[None], page)
    assert err == 0
    # every block of 32 rows has its own power of two, so each weight is within 2^-8 (the 31 beside the large one are lost)
    assert np.abs(got[0, :, 0] - 1).max() <= 2.0 ** -8 + 31 / (p + T) + 1e-3
    assert np.abs(got[0, :, 1] - p / (p + T)).max() <= 2.0 ** -8 + 1e-3


@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("up", [True, False])
def test_scores_hundreds_of_binary_orders_apart(lib, q_dtype, up):
    """Scores that climb (or fall) by about 150 binary orders every 100 rows: what came before is rescaled to nothing,
    and the largest term alone is left."""
    T, H, page = 700, 16, 64
    rng = np.random.default_rng(12)
    kv8 = rng.integers(0x30, 0x40, ((T + page) // page * page, 576)).astype(np.uint8)
    kv8[:, 512:] = 0
    step = (np.arange(len(kv8)) // 100) * (1 if up else -1) + (0 if up else 7)
    kv8[:, 512] = torch.tensor(step, dtype=F32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    scale = np.ones(len(kv8), np.float32)
    q = np.zeros((2, H, 576), np.float32)
    q[:, :, 512] = 1440 + 64 * (np.arange(H) % 4)     # SM * 1440 log2 e: about 150
    q[1] *= -1
    table = np.arange(len(kv8) // page)[None]
    got, err = run_tree(lib, q, q_dtype, F32, [2], [T - 2], None, kv8, scale, table, page)
    assert err == 0
    check(got, q, [2], [T - 2], [np.tril(np.ones((2, 2), bool))], kv8, scale, [np.arange(T)], F32, q_dtype == F32)


# ------------------------------------------------------------------------------------------------------------
def run_plan(lib, lens, n, page, state, R=None):
    R = sum(max(x, 0) for x in n) if R is None else R
    slots = torch.full((R,), -9, dtype=torch.int64, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_page_plan(i32(lens), i32(np.concatenate([[0], np.cumsum(n)])), page, state["n_pages"], state["table"],
                      state["free"], state["n_free"], slots, err_word=err)
    torch.cuda.synchronize()
    return slots.tolist(), err.item()


def plan_state(rng, B, most, total):
    perm = [int(x) for x in rng.permutation(total)]
    host = {"n_pages": [0] * B, "table": [[-7] * most for _ in range(B)], "free": perm, "n_free": total}
    return host, {"n_pages": i32(host["n_pages"]), "table": i32(host["table"]), "free": i32(perm), "n_free": i32([total])}


def same(host, dev):
    assert dev["n_pages"].tolist() == host["n_pages"]
    assert dev["table"].tolist() == host["table"]
    assert dev["free"].tolist() == host["free"]
    assert dev["n_free"].tolist() == [host["n_free"]]


@pytest.mark.parametrize("B,page,most,total,top", [(1, 16, 8, 8, 100), (5, 16, 20, 60, 200), (33, 64, 9, 200, 500),
                                                   (300, 32, 16, 900, 100), (1500, 16, 7, 4000, 70),
                                                   (4096, 16, 6, 20000, 60)])
def test_plan_over_many_steps(lib, B, page, most, total, top):
    """Growth, shrinking, returns of everything, lists that run dry and tables that are too narrow, step after step."""
    rng = np.random.default_rng(B + page)
    host, dev = plan_state(rng, B, most, total)
    for step in range(8):
        lens = [int(x) for x in rng.integers(0, top, B)]
        n = [int(x) for x in rng.integers(0, 5 if B > 64 else 40, B)]
        if step == 5:
            lens, n = [0] * B, [0] * B
        slots, err = run_plan(lib, lens, n, page, dev)
        want, host["n_free"], err_w = plan(lens, n, page, host["n_pages"], host["table"], host["free"], host["n_free"], most)
        assert err == err_w
        assert slots == [x for s in want for x in s]
        same(host, dev)
        held = [p for b in range(B) for p in host["table"][b][:host["n_pages"][b]]] + host["free"][:host["n_free"]]
        assert sorted(held) == sorted(range(total))  # no page lost, none held twice


def test_plan_returns_what_it_took(lib):
    rng = np.random.default_rng(1)
    B, page, most = 40, 16, 12
    host, dev = plan_state(rng, B, most, 300)
    lens = [int(x) for x in rng.integers(0, 90, B)]
    run_plan(lib, lens, [0] * B, page, dev)
    before = {k: v.clone() for k, v in dev.items()}
    first, _ = run_plan(lib, lens, [20] * B, page, dev)
    run_plan(lib, lens, [0] * B, page, dev)
    assert torch.equal(dev["n_free"], before["n_free"]) and torch.equal(dev["free"], before["free"])
    again, _ = run_plan(lib, lens, [20] * B, page, dev)
    assert first == again


def test_plan_impossible_numbers(lib):
    rng = np.random.default_rng(2)
    host, dev = plan_state(rng, 4, 6, 30)
    slots, err = run_plan(lib, [3, -1, 40, 5], [2, 3, 300, 1], 16, dev)
    assert err == BAD_INDEX and slots[:2] == [host["free"][29] * 16 + 3, host["free"][29] * 16 + 4]
    assert slots[2:305] == [-9] * 303 and slots[305] == host["free"][28] * 16 + 5
    assert dev["n_pages"].tolist() == [1, 0, 0, 1]
    # a count that no table can hold, then a list that is shorter than it says: nothing changes
    dev["n_pages"][1] = 99
    _, err = run_plan(lib, [3, 3, 0, 5], [2, 3, 0, 1], 16, dev)
    assert err == BAD_INDEX and dev["n_pages"].tolist() == [1, 99, 0, 1]
    dev["n_pages"][1] = 0
    before = {k: v.clone() for k, v in dev.items()}
    dev["n_free"][0] = 31
    slots, err = run_plan(lib, [30, 30, 30, 30], [1, 1, 1, 1], 16, dev)
    assert err == BAD_INDEX and slots == [-9] * 4
    assert all(torch.equal(dev[k], before[k]) for k in ("n_pages", "table", "free")) and dev["n_free"].item() == 31


@pytest.mark.parametrize("n", [[1], [0, 5, 32, 0, 31], [33, 64, 2], [256, 0, 255, 129], [7] * 700])
def test_mask(lib, n):
    rng = np.random.default_rng(len(n))
    parent = trees(rng, n)
    if n[0] == 256:
        parent[0] = list(range(-1, 255))  # the deepest tree
        parent[2] = [-1] * 255            # the flattest
    R, words = sum(n), max(1, -(-max(n) // 32))
    lens = [int(x) for x in rng.integers(0, 1000, len(n))]
    mask = torch.full((R + 1, words), 99, dtype=torch.int32, device=DEV)
    pos = torch.full((R + 1,), 99, dtype=torch.int32, device=DEV)
    par = i32([p for t in parent for p in t] + [0])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_tree_mask(par, i32(np.concatenate([[0], np.cumsum(n)])), i32(lens), mask, pos, err_word=err)
    torch.cuda.synchronize()
    want = np.concatenate([pack(closure(t), words) for t in parent if len(t)])
    depth = np.concatenate([lens[b] + closure(t).sum(1) - 1 for b, t in enumerate(parent) if len(t)])
    assert err.item() == 0
    assert np.array_equal(mask.cpu().numpy()[:R], want) and np.array_equal(pos.cpu().numpy()[:R], depth)
    assert (mask[R:] == 99).all() and (pos[R:] == 99).all()


def test_mask_bad_parents_and_too_few_words(lib):
    par = i32([-1, 1, 5, -3, 0] + [-1] * 40)
    mask = torch.full((45, 1), 99, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_tree_mask(par, i32([0, 5, 45]), None, mask, None, err_word=err)
    torch.cuda.synchronize()
    assert err.item() == BAD_INDEX
    assert mask[:5, 0].tolist() == [1, 2, 4, 8, 17] and (mask[5:] == 99).all()


# ------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("layers,page,n", [(1, 16, [1, 5, 0, 20]), (3, 64, [64, 33, 7]), (2, 16, [256, 100])])
def test_commit(lib, layers, page, n):
    rng = np.random.default_rng(layers + page)
    B, most = len(n), max(max(n) // 2, 6)
    lens = [int(x) for x in rng.integers(0, 100, B)]
    need = [-(-(x + y) // page) for x, y in zip(lens, n)]
    perm = rng.permutation(sum(need))
    table = np.full((B, max(need)), -1)
    at = 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    rows = sum(need) * page
    kv8 = rng.integers(0, 256, (layers, rows, 576)).astype(np.uint8)
    scale = rng.random((layers, rows)).astype(np.float32)
    count = [int(rng.integers(0, min(most, m) + 1)) for m in n]
    count[0] = min(most, n[0])
    accept = np.full((B, most), -3)
    for b in range(B):
        accept[b, :count[b]] = np.sort(rng.choice(n[b], count[b], replace=False)) if count[b] else []
    want, want_s = kv8.copy(), scale.copy()
    for b in range(B):
        row = lambda t: table[b, t // page] * page + t % page  # noqa: E731
        for k in range(count[b]):
            want[:, row(lens[b] + k)] = kv8[:, row(lens[b] + accept[b, k])]
            want_s[:, row(lens[b] + k)] = scale[:, row(lens[b] + accept[b, k])]
    k, s = torch.from_numpy(kv8).to(DEV), torch.from_numpy(scale).to(DEV)
    if layers == 1:
        k, s = k[0], s[0]
    new, err = torch.full((B,), -9, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_tree_commit(i32(np.concatenate([[0], np.cumsum(n)])), i32(lens), i32(accept), i32(count), k, s, i32(table), page,
                        new, err_word=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and new.tolist() == [x + c for x, c in zip(lens, count)]
    assert np.array_equal(k.cpu().numpy().reshape(want.shape), want) and np.array_equal(s.cpu().numpy().reshape(want_s.shape), want_s)


@pytest.mark.parametrize("B,layers", [(135, 40), (40, 61), (1100, 3)])
def test_commit_of_several_layers_by_a_block(lib, B, layers):
    """More (sequence, layer) pairs than blocks that fit the device at once."""
    g = torch.Generator(device=DEV).manual_seed(B)
    page, n, most = 16, 9, 9
    lens = torch.arange(B, device=DEV) * 5 % 23
    table = torch.randperm(2 * B, generator=g, device=DEV).view(B, 2)
    kv8 = torch.randint(0, 256, (layers, 2 * B * page, 576), generator=g, dtype=torch.uint8, device=DEV)
    scale = torch.rand((layers, 2 * B * page), generator=g, device=DEV)
    count = torch.arange(B, device=DEV) % (n + 1)
    accept = torch.rand((B, n), generator=g, device=DEV).argsort(1)
    k = torch.arange(n, device=DEV)
    accept = torch.where(k < count[:, None], accept, n).sort(1).values
    on = k < count[:, None]
    row = lambda t: table.gather(1, t // page) * page + t % page  # noqa: E731
    src, dst = row(torch.where(on, lens[:, None] + accept, 0))[on], row(torch.where(on, lens[:, None] + k, 0))[on]
    want, want_s = kv8.clone(), scale.clone()
    want[:, dst], want_s[:, dst] = kv8[:, src], scale[:, src]
    new, err = torch.empty(B, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    to = torch.int32
    lib.kv8_tree_commit((torch.arange(B + 1, device=DEV) * n).to(to), lens.to(to), accept.to(to), count.to(to), kv8, scale,
                        table.to(to), page, new, err_word=err)
    assert err.item() == 0 and torch.equal(new.long(), lens + count)
    assert torch.equal(kv8, want) and torch.equal(scale, want_s)


@pytest.mark.parametrize("accept,count,table", [([2, 2, 4], 3, [0, 1]), ([3, 1, 4], 3, [0, 1]), ([0, 1, 6], 3, [0, 1]),
                                                ([-1, 1, 2], 3, [0, 1]), ([0, 1, 2], 4, [0, 1]), ([0, 1, 2], -1, [0, 1]),
                                                ([1, 2, 3], 3, [0, 9]), ([1, 2, 3], 3, [0, -1])])
def test_commit_refuses_what_is_no_branch(lib, accept, count, table):
    page, lens, n = 16, [14, 14], 6
    kv8 = torch.randint(0, 256, (64, 576), dtype=torch.uint8, device=DEV)
    scale = torch.rand(64, device=DEV)
    before, before_s = kv8.clone(), scale.clone()
    new, err = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_tree_commit(i32([0, n, 2 * n]), i32(lens), i32([accept, [1, 3, 5]]), i32([count, 2]), kv8, scale,
                        i32([table, [2, 3]]), page, new, err_word=err)
    torch.cuda.synchronize()
    assert err.item() == BAD_INDEX and new.tolist() == [14, 16]
    before[32 + 14], before[32 + 15] = before[32 + 15].clone(), before[32 + 17].clone()  # the other sequence moves
    before_s[32 + 14], before_s[32 + 15] = before_s[32 + 15].clone(), before_s[32 + 17].clone()
    assert torch.equal(kv8, before) and torch.equal(scale, before_s)


# ------------------------------------------------------------------------------------------------------------
def test_a_serving_loop(lib, oracle):
    """Plan, mask, projection, append, attention, projection, commit and the next step's plan, captured once and
    replayed for every step, against a host model that keeps each sequence's rows as a list."""
    rng = np.random.default_rng(11)
    B, H, N, page, most, layers = 3, 16, 9, 16, 20, 2
    total = 40
    lens0, R = [33, 0, 120], B * N
    host, dev = plan_state(rng, B, most, total)
    kv8 = torch.full((layers, total * page, 576), GARBAGE, dtype=torch.uint8, device=DEV)
    scale = torch.full((layers, total * page), float("nan"), device=DEV)
    hist = [[synth.latent_rows(rng, x, 0.5, 2.0) for _ in range(layers)] for x in lens0]
    # the contexts are planned and appended as drafts of up to 256 rows
    ctx = torch.zeros(sum(lens0), dtype=torch.int64, device=DEV)
    lib.kv8_page_plan(i32([0] * B), i32(np.concatenate([[0], np.cumsum(lens0)])), page, dev["n_pages"], dev["table"],
                      dev["free"], dev["n_free"], ctx)
    for la in range(layers):
        x = torch.from_numpy(np.concatenate([hist[b][la] for b in range(B)])).to(DEV)
        lib.kv8_quant_rows_scatter(x, ctx, kv8[la], scale[la])
    w8, w_scale = synth.kvb_fmt8(H)
    w8, w_scale = torch.from_numpy(w8).to(DEV), torch.from_numpy(w_scale).to(DEV)
    s = {"lens": i32(lens0), "q_start": i32(range(0, R + 1, N)), "parent": i32([0] * R), "new_lens": i32([0] * B),
         "accept": i32([[0] * N] * B), "n_accept": i32([0] * B)}
    slots = torch.empty(R, dtype=torch.int64, device=DEV)
    mask, pos = torch.empty((R, 1), dtype=torch.int32, device=DEV), torch.empty(R, dtype=torch.int32, device=DEV)
    x = torch.zeros((layers, R, 576), device=DEV)
    q_nope, q_rope = torch.zeros((R, H, 128), dtype=BF, device=DEV), torch.zeros((R, H, 64), dtype=BF, device=DEV)
    q_lat = torch.empty((R, H, 512), dtype=BF, device=DEV)
    out, y = torch.empty((layers, R, H, 512), device=DEV), torch.empty((layers, R, H, 128), device=DEV)
    ws = torch.empty(lib.mla_tree8_workspace_bytes(R, H, B, BF), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def draft():
        lib.kv8_page_plan(s["lens"], s["q_start"], page, dev["n_pages"], dev["table"], dev["free"], dev["n_free"], slots,
                          err_word=err)
        lib.kv8_tree_mask(s["parent"], s["q_start"], s["lens"], mask, pos, err_word=err)
        for la in range(layers):
            lib.kv8_quant_rows_scatter(x[la], slots, kv8[la], scale[la], err_word=err)
            lib.mla_q_absorb8(q_nope, w8, w_scale, q_lat, err_word=err)
            lib.mla_absorb_tree8(q_lat, q_rope, s["q_start"], s["lens"], mask, kv8[la], scale[la], dev["table"], page, SM, ws,
                                 out[la], err_word=err)
            lib.mla_out_project8(out[la], w8, w_scale, y[la], err_word=err)

    def commit():
        lib.kv8_tree_commit(s["q_start"], s["lens"], s["accept"], s["n_accept"], kv8, scale, dev["table"], page,
                            s["new_lens"], err_word=err)
        lib.kv8_copy(s["lens"], s["new_lens"])

    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, f in zip(graphs, (draft, commit)):
        with torch.cuda.graph(g):
            f()
    for step in range(4):
        parent = trees(rng, [N] * B)
        fresh = [[synth.latent_rows(rng, N, 0.5, 2.0) for _ in range(layers)] for _ in range(B)]
        s["parent"].copy_(i32([p for t in parent for p in t]))
        for la in range(layers):
            x[la].copy_(torch.from_numpy(np.concatenate([fresh[b][la] for b in range(B)])))
        q_nope.copy_(torch.from_numpy(rng.standard_normal((R, H, 128)).astype(np.float32)))
        q_rope.copy_(torch.from_numpy(rng.standard_normal((R, H, 64)).astype(np.float32)))
        graphs[0].replay()
        torch.cuda.synchronize()
        q = torch.cat([q_lat, q_rope], -1).float().cpu().numpy()
        for b in range(B):
            sees, T = closure(parent[b]), len(hist[b][0])
            assert pos[b * N:(b + 1) * N].tolist() == [T + int(v) - 1 for v in sees.sum(1)]
            for la in range(layers):
                k, sc = oracle.quant_rows(np.concatenate([hist[b][la], fresh[b][la]]))
                ref, tol = attend(q[b * N:(b + 1) * N].astype(np.float64), sees, T, np.arange(T + N),
                                  np.ones(T + N, bool), k, sc, EPS[F32], False)
                assert (np.abs(out[la, b * N:(b + 1) * N].double().cpu().numpy() - ref) <= tol).all(), (step, b, la)
        # accept the branch of some token, or nothing
        leaf = [int(rng.integers(-1, N)) for _ in range(B)]
        acc = [[int(j) for j in np.nonzero(closure(parent[b])[leaf[b]])[0]] if leaf[b] >= 0 else [] for b in range(B)]
        s["accept"].copy_(i32([a + [0] * (N - len(a)) for a in acc]))
        s["n_accept"].copy_(i32([len(a) for a in acc]))
        graphs[1].replay()
        for b in range(B):
            for la in range(layers):
                hist[b][la] = np.concatenate([hist[b][la], fresh[b][la][acc[b]]])
        torch.cuda.synchronize()
        assert s["lens"].tolist() == [len(h[0]) for h in hist] and err.item() == 0
    # the projection of the last step's attention, against the same weights in 64 bits
    ref = oracle.out_project(out[0].cpu().numpy(), w8.cpu().numpy(), w_scale.cpu().numpy())
    assert np.linalg.norm(y[0].cpu().numpy() - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
