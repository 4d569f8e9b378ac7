"""The paged calls at the edges of what their header allows: batch sizes where a launch changes its form, starts that
are not in order, row scales from one end of their range to the other, caches that end inside a page."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_tree import BF, DEV, F32, build, check, i32, queries, run_tree
from tree_ref import BAD_INDEX, SM, TABLE, pack

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def chains(n):
    return [np.tril(np.ones((m, m), bool)) for m in n]


def test_plan_of_any_batch_size_as_a_process_first_call():
    """Batches whose shared memory is about the launch's default limit, before any larger one has raised it."""
    code = ("import sys; sys.path[:0] = sys.argv[1:]\n"
            "import fp8_latent_kv_gb300 as kv, test_gpu_tree as t\n"
            "kv.load()\n"
            "for B in (3039, 3040, 3041, 3055, 3071):\n"
            "    t.test_plan_over_many_steps(kv, B, 16, 6, 4 * B, 60)\n")
    r = subprocess.run([sys.executable, "-c", code, os.path.dirname(HERE), HERE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("start,good", [([0, 4, -1, 9], [0]), ([0, 4, -200, 4, 9], [0, 3]), ([0, 4, -(1 << 31), 9], [0])])
def test_impossible_starts_spare_the_sequences_before_them(lib, oracle, q_dtype, start, good):
    """A start out of range makes the two sequences that it belongs to impossible; the others are as they would be alone."""
    rng = np.random.default_rng(len(start))
    H, page, B = 128, 16, len(start) - 1
    n = [max(0, y - x) if b in good else 0 for b, (x, y) in enumerate(zip(start, start[1:]))]
    lens = [130, 40, 7, 75][:B]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    q = queries(rng, 9, H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page, start=start)
    assert err == BAD_INDEX
    left = np.ones(9, bool)
    for b in good:
        at = slice(start[b], start[b] + n[b])
        check(got[at], q[at], n[b:b + 1], lens[b:b + 1], chains(n[b:b + 1]), kv8, scale, rows[b:b + 1], F32, q_dtype == F32)
        left[at] = False
    assert (got[left] == 7.0).all()


BACK = [([8, 12, 0, 4], 12, "a sequence before an earlier one"), ([0, 8, 4, 12], 12, "rows of two sequences"),
        ([0, 8, 4, 12, 2, 9], 12, "rows of three"), ([0] + [5, 0] * 500 + [5, 9], 9, "the same rows, many times")]


@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("start,R,what", BACK, ids=[x[2] for x in BACK])
def test_rows_that_go_back_are_left(lib, oracle, q_dtype, start, R, what):
    """Possible sequences whose rows are not in order: nothing is written, and the error word says so."""
    rng = np.random.default_rng(R)
    H, page, B = 16, 16, len(start) - 1
    lens = [int(x) for x in rng.integers(0, 60, B)]
    kv8, scale, table, rows = build(oracle, rng, lens, [12] * B, page)
    q = queries(rng, R, H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, None, lens, None, kv8, scale, table, page, start=start)
    assert err == BAD_INDEX and (got == 7.0).all()


@pytest.mark.parametrize("start,R,what", BACK, ids=[x[2] for x in BACK])
def test_plan_of_rows_that_go_back_changes_nothing(lib, start, R, what):
    B = len(start) - 1
    state = dict(n_pages=[1] * B, block_table=np.arange(4 * B).reshape(B, 4), free_list=4 * B + np.arange(3 * B), n_free=[3 * B])
    state = {k: i32(v) for k, v in state.items()}
    before = {k: v.clone() for k, v in state.items()}
    slots, err = torch.full((R,), -9, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_page_plan(i32([20] * B), i32(start), 16, slots=slots, err_word=err, **state)
    assert err.item() == BAD_INDEX and (slots == -9).all()
    assert all(torch.equal(state[k], before[k]) for k in state)


def test_plan_spares_possible_sequences_in_order(lib):
    """An impossible start between sequences whose rows are in order, empty sequences with any start among them."""
    start, lens = [9, 9, 0, 3, 3, -1, 3, 9], [1, 2, 17, 4, 5, 6, 15]
    state = dict(n_pages=[0] * 7, block_table=np.full((7, 4), -7), free_list=np.arange(20), n_free=[20])
    state = {k: i32(v) for k, v in state.items()}
    slots, err = torch.full((9,), -9, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.kv8_page_plan(i32(lens), i32(start), 16, slots=slots, err_word=err, **state)
    assert err.item() == BAD_INDEX
    # sequences 0 (2 positions' page, no rows), 2 (two pages), 3 (one) and 6 (two) from the top of the list
    assert state["n_pages"].tolist() == [1, 0, 2, 1, 0, 0, 2] and state["n_free"].item() == 14
    assert slots.tolist() == [17 * 16 + 1, 17 * 16 + 2, 17 * 16 + 3, 15 * 16 + 15] + [14 * 16 + i for i in range(5)]


def with_scales(oracle, rng, lens, n, page, scales):
    """build()'s cache with other row scales."""
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    for r in rows:
        scale[r] = scales(len(r)).astype(np.float32)
    return kv8, scale, table, rows


@pytest.mark.parametrize("q_dtype,top", [(BF, 60), (F32, 60), (F32, 80)])
@pytest.mark.parametrize("kind", ["small", "large", "both"])
def test_row_scales_at_the_ends_of_their_range(lib, oracle, q_dtype, top, kind):
    """Whole caches with scales next to 2^-60 (f32 queries: 2^-80 too) or 2^60, and both in one sequence, under queries that
    bring the scores back to ordinary sizes."""
    rng = np.random.default_rng(71)
    H, page, lens, n = 24, 64, [700, 0, 63], [3, 9, 1]
    low, high = 2.0 ** -top, 2.0 ** top

    def scales(m):
        s = rng.uniform(1, 4, m) * low
        h = rng.uniform(0.25, 1, m) * high
        return {"small": s, "large": h, "both": np.where(rng.random(m) < 0.5, s, h)}[kind]

    kv8, scale, table, rows = with_scales(oracle, rng, lens, n, page, scales)
    for r in rows:  # the ends themselves
        if len(r) > 2 and kind != "large":
            scale[r[1]] = low
        if len(r) > 2 and kind != "small":
            scale[r[2]] = high
    q = queries(rng, sum(n), H, q_dtype == F32) * np.float32(2.0 ** -8 * (high if kind == "small" else low))
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, chains(n), kv8, scale, rows, F32, q_dtype == F32)


@pytest.mark.parametrize("at", [5, 320, 701])
@pytest.mark.parametrize("big", [float(np.nextafter(np.float32(2.0 ** 60), np.float32(np.inf))), 2.0 ** 90, 2.0 ** 127])
def test_larger_scales_than_bf16_queries_take_say_so(lib, oracle, big, at):
    """One attended row beyond the range: NaN for every token that attends it, the others as they were."""
    rng = np.random.default_rng(73)
    H, page, lens, n = 16, 64, [700], [4]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    q = queries(rng, 4, H, False)
    ref, _ = run_tree(lib, q, BF, F32, n, lens, None, kv8, scale, table, page)
    scale[rows[0][at]] = big
    got, err = run_tree(lib, q, BF, F32, n, lens, None, kv8, scale, table, page)
    first = max(0, at - 700)
    assert err == 0 and np.isnan(got[first:]).all()
    assert np.array_equal(got[:first], ref[:first])


def test_smaller_scales_than_bf16_queries_take_count_as_zero_rows(lib, oracle):
    """Below 2^-60 a row's score counts as 0 and its value as zeros; at 2^-60 and above it is itself.  The queries are such
    that the scores of those rows would show."""
    rng = np.random.default_rng(79)
    H, page, lens, n = 16, 64, [300, 10], [3, 20]
    edge = np.float32(2.0 ** -60)
    below = np.nextafter(edge, np.float32(0))
    kv8, scale, table, rows = with_scales(oracle, rng, lens, n, page, lambda m: np.where(rng.random(m) < 0.5, edge, below))
    q = queries(rng, sum(n), H, False) * np.float32(2.0 ** 52)
    as_zero = np.where(scale < edge, np.float32(0), scale)
    sees = [rng.random((m, m)) < 0.6 for m in n]
    mask = np.concatenate([pack(x, 1) for x in sees])
    got, err = run_tree(lib, q, BF, F32, n, lens, mask, kv8, scale, table, page)
    assert err == 0
    check(got, q, n, lens, sees, kv8, as_zero, rows, F32, False)


def test_f32_sums_of_many_small_terms(lib):
    """2^17 rows that together weigh as much as one: sums of f32 queries are held to f32, not to the bf16 form's weights.

    The bound, in steps of 2^-24 of the sums (all terms are positive): a weight's two f16 pieces leave 2^-22 (4); 64 rows are 8
    products whose 17 terms may each be cut (136); a share is at most 2^17 / 32 / 100 + 1 units of 32 rows (100 shares or
    more), so 21 such steps, each an addition to the context (21) and four to each of sixteen warps' sums (84 + 16); the merge adds
    at most 2 x 152 parts (304, context and sums: at most as many again); the large row's score, 17 ln 2, has a product,
    a factor and a constant (3 x 17 log2 e ln 2 = 51), exp2 and the merge's own (2 + 2).  In all 4 + 136 + 21 + 100 + 608 + 55 =
    924: less than 2^-14."""
    T, H, page = 1 << 17, 16, 1024
    kv8 = np.zeros((T + page, 576), np.uint8)
    kv8[:, 0] = 0x38                            # 1.0 in every row
    kv8[T // 2, 1] = 0x38                       # the row that the query asks for
    scale = np.ones(T + page, np.float32)
    q = np.zeros((1, H, 576), np.float32)
    q[:, :, 1] = round(17 * np.log(2) / SM)
    p = np.exp(SM * float(q[0, 0, 1]))
    got, err = run_tree(lib, q, F32, F32, [1], [T], None, kv8, scale, np.arange(T // page + 1)[None], page)
    assert err == 0
    assert np.abs(got[0, :, 0] - 1).max() <= 2.0 ** -14
    assert np.abs(got[0, :, 1] - p / (p + T)).max() <= 2.0 ** -14


@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_a_cache_that_ends_inside_a_page(lib, oracle, q_dtype, page):
    """cache_rows no multiple of the page: the last page's rows past the end are left out, with the error bit."""
    rng = np.random.default_rng(83)
    H, lens, n = 16, [3 * page + 5, 20], [7, 2]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    end = max(int(r.max()) for r in rows) - 4        # inside the page that holds the highest row
    valid = [r < end for r in rows]
    q = queries(rng, sum(n), H, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8[:end].copy(), scale[:end].copy(), table, page)
    assert err == BAD_INDEX
    check(got, q, n, lens, chains(n), kv8, scale, [np.where(v, r, 0) for v, r in zip(valid, rows)], F32, q_dtype == F32, valid=valid)


@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_a_step_without_drafted_tokens(lib, oracle, q_dtype):
    rng = np.random.default_rng(89)
    kv8, scale, table, rows = build(oracle, rng, [30, 0], [0, 0], 16)
    q = queries(rng, 3, 16, q_dtype == F32)
    got, err = run_tree(lib, q, q_dtype, F32, [0, 0], [30, 0], None, kv8, scale, table, 16)
    assert err == 0 and (got == 7.0).all()


@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("bad", ["scale", "codes"])
@pytest.mark.parametrize("at", [3, 9000, 20001])
def test_a_row_that_is_not_a_number_shows_whatever_the_others_weigh(lib, q_dtype, bad, at):
    """One attended row of NaN among shares whose largest scores lie hundreds of binary orders above and below its share's."""
    page, T, H = 128, 20002, 16
    kv8 = np.full((T + page, 576), 0x38, np.uint8)       # 1.0
    kv8[:, 512:] = 0
    kv8[:, 512] = torch.tensor(np.arange(T + page) // 2000 % 8 * 2.0, dtype=F32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    scale = np.ones(T + page, np.float32)
    q = np.zeros((2, H, 576), np.float32)
    q[:, :, 512] = 2000 * np.where(np.arange(H) % 2, 1, -1)   # about 200 binary orders a level
    table = np.arange(T // page + 1)[None]
    ref, _ = run_tree(lib, q, q_dtype, F32, [2], [T - 2], None, kv8, scale, table, page)
    assert np.isfinite(ref).all()
    if bad == "scale":
        scale[at] = np.nan
    else:
        kv8[at, :512:3] = 0x7F
    got, err = run_tree(lib, q, q_dtype, F32, [2], [T - 2], None, kv8, scale, table, page)
    sees = [at < T - 1, True]
    assert err == 0
    for i in range(2):
        assert np.isnan(got[i, :, 0]).all() if sees[i] else np.array_equal(got[i], ref[i])


@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("base", [0.0156, 0.058, 9.8])
@pytest.mark.parametrize("uneven", [False, True])
@pytest.mark.parametrize("side", [1, -1])
def test_scores_far_from_zero(lib, q_dtype, side, uneven, base):
    """Scores of all sizes, every column's of one sign.  From about 2^12 on the largest row is all that is left, and the output is its
    values, to the weights' rounding (bf16: 2^-8 and 2^-12; f32: 2^-22) and a few steps of 2^-24.  Scores
    from 2^23 log 2 (bf16 queries) or 2^25 log 2 on are beyond what the exponents hold, and the output is NaN, nothing else."""
    rng = np.random.default_rng(97)
    page, T, powers = 64, 300, np.arange(4, 112)
    H = len(powers)
    kv8 = rng.integers(0x30, 0x40, (512, 576)).astype(np.uint8)
    kv8[:, 512:] = 0
    level = rng.permutation(np.arange(T) % 11)           # whole numbers that e4m3 has
    level = level if side > 0 else -2 - level
    top = 108
    level[top] = 13 if side > 0 else -1
    table = rng.permutation(8)[None]
    row = table[0, np.arange(T) // page] * page + np.arange(T) % page
    kv8[row, 520] = torch.tensor(level, dtype=F32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    scale = np.ones(512, np.float32)
    scale[row] = base * rng.uniform(0.9, 1, T)
    if uneven:  # (rows of score 0, or far below all others)
        some = np.nonzero(level == 0 if side > 0 else level < -10)[0]
        scale[row[some]] = base * rng.choice(np.float32([2.0 ** (-7 * side), 2.0 ** 6, 1.5]), len(some))
    q = np.zeros((2, H, 576), np.float32)
    q[:, :, 520] = np.ldexp(1.0 + rng.integers(0, 128, H) / 128, powers)  # exact in bf16
    got, err = run_tree(lib, q, q_dtype, F32, [2], [T - 2], None, kv8, scale, table, page)
    assert err == 0
    score = SM / np.log(2) * q[0, :, 520:521].astype(np.float64) * (level * scale[row].astype(np.float64))  # [H][T]
    want = TABLE[kv8[row[top], :512]] * float(scale[row[top]])
    gap = score[:, top] - np.delete(score, top, 1).max(1)
    far = 2.0 ** (23 if q_dtype == BF else 25)
    fine, beyond = (gap > 40) & (np.abs(score).max(1) < far), np.abs(score[:, top]) > 1.01 * far
    assert fine.sum() >= 5 and beyond.sum() >= 60
    eps = 2.0 ** -8 + 2.0 ** -11 if q_dtype == BF else 2.0 ** -21
    off = np.abs(got / want - 1).max((0, 2))
    assert (off[fine] <= eps).all(), off
    assert np.isnan(got[:, beyond]).all(), off


@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("at", [5, 400, 701])
def test_an_infinite_scale_shows_whatever_its_scores_sign(lib, oracle, q_dtype, at):
    """An attended row of infinite scale: NaN, where its score would be minus infinity too."""
    rng = np.random.default_rng(101)
    H, page, lens, n = 16, 64, [700], [4]
    kv8, scale, table, rows = build(oracle, rng, lens, n, page)
    q = queries(rng, 4, H, q_dtype == F32)
    sign = TABLE[kv8[rows[0][at]]] @ q.reshape(-1, 576).T.astype(np.float64) > 0
    assert 8 < sign.sum() < 56
    ref, _ = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    scale[rows[0][at]] = np.inf
    got, err = run_tree(lib, q, q_dtype, F32, n, lens, None, kv8, scale, table, page)
    first = max(0, at - 700)
    assert err == 0 and np.isnan(got[first:]).all() and np.array_equal(got[:first], ref[:first])
