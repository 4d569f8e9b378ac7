"""The paged calls at the edges of what their header allows: batch sizes where a launch changes its form, starts that
are not in order, row scales from one end of their range to the other, caches that end inside a page."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_tree import BF, DEV, F32, build, check, i32, queries, run_tree
from tree_ref import BAD_INDEX, SM, pack

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
