"""The calls around the attention in a layer: what they refuse before any launch, and the frequency table.  CPU only."""
import ctypes
import math

import pytest
import torch

import fp8_latent_kv_gb300 as kv
from fp8_latent_kv_gb300 import build as kvbuild

FAKE = 0x100000  # 16-byte aligned, never dereferenced
BF, F32 = kv.KV8_BF16, kv.KV8_F32
EINVAL, OK = kv.KV8_EINVAL, kv.KV8_OK


@pytest.fixture(scope="module")
def lib():
    kvbuild.build()
    return kv.load()


def test_rope_refusals(lib):
    def call(**k):
        a = dict(x=FAKE, xt=BF, n=4, h=8, w=192, at=128, d=64, xr=8 * 192, xh=192, pos=FAKE, f=FAKE, s=1.0, l=0, rot=FAKE, rr=512, rh=64,
                 rest=FAKE, er=1024, eh=128, ot=BF)
        a.update(k)
        return lib.kv8_rope(a["x"], a["xt"], a["n"], a["h"], a["w"], a["at"], a["d"], a["xr"], a["xh"], a["pos"], a["f"], a["s"], a["l"],
                            a["rot"], a["rr"], a["rh"], a["rest"], a["er"], a["eh"], a["ot"], None)
    assert call(n=0, x=None, rot=None, pos=None) == OK
    for bad in [dict(n=-1), dict(n=(1 << 20) + 1), dict(h=0), dict(h=129), dict(d=0), dict(d=63), dict(d=258, w=512), dict(at=-1), dict(at=129),
                dict(w=65537), dict(w=63, at=0), dict(xt=2), dict(ot=-1), dict(l=2), dict(l=-1), dict(s=math.nan), dict(s=math.inf),
                dict(x=None), dict(x=FAKE + 1), dict(x=FAKE + 2, xt=F32), dict(rot=None), dict(rot=FAKE + 2, ot=F32), dict(rest=FAKE + 1),
                dict(pos=FAKE + 2), dict(pos=None), dict(f=None), dict(f=FAKE + 2), dict(xr=-1), dict(xh=-192),
                # outputs whose heads or rows touch one another
                dict(rh=63), dict(rr=511), dict(eh=127), dict(er=1023), dict(rr=0), dict(rh=0), dict(rr=-512),
                dict(rr=1 << 41), dict(xr=1 << 41), dict(er=1 << 41)]:
        assert call(**bad) == EINVAL, bad


def test_norm_rope_rows_refusals(lib):
    def call(**k):
        a = dict(x=FAKE, xt=BF, n=4, xs=576, w=FAKE, eps=1e-6, pos=FAKE, f=FAKE, s=1.0, l=0, dst=FAKE, kv8=FAKE, ks=FAKE, rows=10)
        a.update(k)
        return lib.kv8_norm_rope_rows(a["x"], a["xt"], a["n"], a["xs"], a["w"], a["eps"], a["pos"], a["f"], a["s"], a["l"], a["dst"],
                                      a["kv8"], a["ks"], a["rows"], None, None)
    assert call(n=0, x=None, w=None, dst=None) == OK
    for bad in [dict(n=-1), dict(rows=-1), dict(xt=2), dict(l=2), dict(s=math.inf), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf),
                dict(xs=575), dict(xs=577), dict(xs=580), dict(xs=578, xt=F32), dict(xs=1 << 41), dict(x=FAKE + 8), dict(x=None), dict(w=None),
                dict(w=FAKE + 4), dict(pos=None), dict(f=None), dict(dst=None), dict(dst=FAKE + 4), dict(kv8=FAKE + 8), dict(ks=None)]:
        assert call(**bad) == EINVAL, bad


def test_quant_blocks_refusals(lib):
    def call(**k):
        a = dict(x=FAKE, xt=BF, n=4, w=256, xs=256, nw=FAKE, eps=1e-6, q=FAKE, s=FAKE, ss=4)
        a.update(k)
        return lib.kv8_quant_blocks(a["x"], a["xt"], a["n"], a["w"], a["xs"], a["nw"], a["eps"], a["q"], a["s"], a["ss"], None)
    assert call(n=0, x=None, q=None, s=None) == OK
    for bad in [dict(n=-1), dict(n=(1 << 20) + 1, ss=1 << 21), dict(w=0), dict(w=8), dict(w=250), dict(w=16400, xs=16400), dict(w=65552, xs=65552, nw=None),
                dict(xt=3), dict(eps=-1.0), dict(eps=math.nan), dict(xs=255), dict(xs=260), dict(xs=258, xt=F32), dict(ss=3), dict(ss=-4),
                dict(x=FAKE + 8), dict(nw=FAKE + 4), dict(q=FAKE + 8), dict(q=None), dict(s=FAKE + 2), dict(s=None)]:
        assert call(**bad) == EINVAL, bad


def test_matmul_refusals(lib):
    def call(**k):
        a = dict(a=FAKE, ast=256, s=FAKE, ss=4, M=4, N=128, K=256, w=FAKE, ws=FAKE, o=FAKE, ot=BF, os=128)
        a.update(k)
        return lib.kv8_matmul8(a["a"], a["ast"], a["s"], a["ss"], a["M"], a["N"], a["K"], a["w"], a["ws"], a["o"], a["ot"], a["os"], None, None)
    assert call(M=0, a=None, w=None, o=None) == OK
    for bad in [dict(M=-1), dict(M=(1 << 20) + 1), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=8), dict(K=250), dict(K=65552, ast=65552),
                dict(ot=2), dict(ast=240), dict(ast=260), dict(ss=3), dict(ss=-1), dict(os=127), dict(os=1 << 37), dict(a=FAKE + 8), dict(a=None),
                dict(s=FAKE + 2), dict(s=None), dict(w=FAKE + 4), dict(ws=None), dict(o=FAKE + 1), dict(o=FAKE + 2, ot=F32), dict(o=None)]:
        assert call(**bad) == EINVAL, bad


def test_frequencies(lib):
    f, s = kv.kv8_rope_freqs(64)
    assert s == 1.0 and f.dtype == torch.float32 and f.shape == (32,)
    ref = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert bool(((f.double() - ref).abs() <= 2.0 ** -24 * ref).all())
    # by parts: pairs with more than 32 turns in the context keep theirs, those with fewer than one are slowed down, between them linear
    g, s = kv.kv8_rope_freqs(64, 10000.0, 40.0, 4096, 32.0, 1.0)
    assert abs(s - (1 + 0.1 * math.log(40))) < 1e-6
    turns = 4096 * ref / (2 * math.pi)
    low, high = int((turns > 32).sum()) - 1, int((turns >= 1).sum())
    share = ((torch.arange(32) - low) / (high - low)).clamp(0, 1).double()
    want = ref * (1 - share) + ref / 40 * share
    assert bool(((g.double() - want).abs() <= 2.0 ** -23 * want).all())
    assert bool((g[:low + 1] == f[:low + 1]).all()) and bool(((g[high:] * 40 - f[high:]).abs() <= 1e-6 * f[high:]).all())
    # the two borders at one pair: a step, no division by zero
    h, _ = kv.kv8_rope_freqs(64, 10000.0, 8.0, 4096, 7.0, 7.0)
    at = 64 * math.log(4096 / (7 * 2 * math.pi)) / (2 * math.log(10000.0))
    assert bool((h[:math.floor(at)] == f[:math.floor(at)]).all()) and bool((h[math.ceil(at):] * 8 == f[math.ceil(at):]).all())
    # a context in which no pair makes a turn: all slowed down; one in which all make many: none
    assert bool((kv.kv8_rope_freqs(64, 10000.0, 8.0, 2)[0] * 8 == f).all())
    assert torch.equal(kv.kv8_rope_freqs(64, 10000.0, 8.0, 1e9)[0], f)


@pytest.mark.parametrize("bad", [dict(rope_dim=0), dict(rope_dim=7), dict(rope_dim=258), dict(theta=1.0), dict(theta=math.nan), dict(factor=0.5),
                                 dict(factor=math.inf), dict(context=0), dict(beta_slow=0.0), dict(beta_slow=40.0), dict(beta_fast=math.nan)])
def test_frequency_refusals(lib, bad):
    with pytest.raises(kv.Kv8Error):
        kv.kv8_rope_freqs(**{"rope_dim": 64, **bad})
    assert lib.kv8_rope_freqs(64, 1e4, 1.0, 4096.0, 32.0, 1.0, None, ctypes.addressof(ctypes.c_float())) == EINVAL
