"""What the calls around the attention promise at their edges: products whose blocks hand their SMs to the next call, and what the
header says of bytes, angles and rows."""
import pytest
import torch

from layer_ref import BLK, U, matmul, weight

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
