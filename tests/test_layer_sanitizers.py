"""The host side of the calls around the attention under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: the sources
that answer them are compiled with the sanitizers and run by tests/sanitize/layer_driver.cpp with every GPU hidden."""
from __future__ import annotations

import glob
import os
import subprocess

import pytest

from test_sanitizers import ENV, ROOT, SAN, _gcc_has_sanitizers, _run


def test_layer_calls_host_side_under_asan_ubsan(tmp_path):
    from fp8_latent_kv_gb300 import build as kvbuild
    try:
        nvcc = kvbuild._nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    if not _gcc_has_sanitizers(str(tmp_path)):
        pytest.skip("gcc with the address / undefined sanitizers is not available")
    flags = ["-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "--expt-relaxed-constexpr",
             "-I", os.path.join(ROOT, "include"), "-I", kvbuild.CSRC, "-Xcompiler", ",".join(SAN)]
    mine = ("kv8mla_api", "rope_rows", "quant_blocks", "matmul8")
    others = [s for s in sorted(glob.glob(os.path.join(kvbuild.CSRC, "*.cu"))) if os.path.basename(s)[:-3] not in mine]
    procs, objs = [], []
    for s in [os.path.join(kvbuild.CSRC, f"{m}.cu") for m in mine] + [os.path.join(ROOT, "tests", "sanitize", "layer_driver.cpp")]:
        objs.append(str(tmp_path / (os.path.basename(s) + ".o")))
        procs.append((s, subprocess.Popen([nvcc, *flags, "-c", s, "-o", objs[-1]], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    kvbuild.build()
    objs += [os.path.join(kvbuild.BUILD, os.path.basename(s)[:-3] + ".o") for s in others]
    for s, p in procs:
        _, err = p.communicate(timeout=600)
        assert p.returncode == 0, f"nvcc failed on {s}:\n{err[-4000:]}"
    cudart = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    exe = str(tmp_path / "layer_asan")
    _run(["g++", *SAN, *objs, "-L" + cudart, "-lcudart_static", "-ldl", "-lpthread", "-lrt", "-o", exe])
    r = _run([exe], env=dict(ENV, CUDA_VISIBLE_DEVICES=""))
    assert "layer driver ok" in r.stdout


@pytest.mark.parametrize("rope_dim", [-2, 0, 1, 257, 258, 1 << 20, (1 << 31) - 2])
def test_frequencies_of_a_size_out_of_range_allocate_nothing(rope_dim):
    """The binding makes no table for a size that the call refuses."""
    import tracemalloc

    import torch  # noqa: F401  (its import is not the call's)
    import fp8_latent_kv_gb300 as kv
    from fp8_latent_kv_gb300 import build as kvbuild
    kvbuild.build()
    kv.load()
    tracemalloc.start()
    with pytest.raises(kv.Kv8Error):
        kv.kv8_rope_freqs(rope_dim)
    most = tracemalloc.get_traced_memory()[1]
    tracemalloc.stop()
    assert most < 1 << 20
