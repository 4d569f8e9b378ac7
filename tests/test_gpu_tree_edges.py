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
