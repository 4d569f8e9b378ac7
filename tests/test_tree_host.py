"""The paged calls' refusals, on the CPU: scalars, alignment and workspace through the C ABI before any CUDA call,
tensors' types, shapes, strides and devices in the Python binding, and the size of the workspace."""
import ctypes

import pytest
import torch

import fp8_latent_kv_gb300 as kv
from fp8_latent_kv_gb300 import build as kvbuild

FAKE, MIS2, MIS4, MIS8 = 0x100000, 0x100002, 0x100004, 0x100008  # never dereferenced


@pytest.fixture(scope="module")
def so():
    kvbuild.build()
    return kv.load()


def call(fn, good, order, **kw):
    a = dict(good, **kw)
    return fn(*[a[k] for k in order])


def test_plan_refusals(so):
    order = "B lens q_start R page most n_pages table free cap n_free slots err st".split()
    good = dict(B=2, lens=FAKE, q_start=FAKE, R=4, page=64, most=5, n_pages=FAKE, table=FAKE, free=FAKE, cap=9, n_free=FAKE,
                slots=FAKE, err=None, st=None)
    for bad in (dict(B=0), dict(B=kv.KV8_MAX_SEQS + 1), dict(R=-1), dict(R=kv.KV8_MAX_ROWS + 1), dict(page=8), dict(page=48),
                dict(page=0), dict(page=-64), dict(page=1 << 17), dict(most=0), dict(lens=None), dict(lens=MIS2),
                dict(q_start=MIS2), dict(n_pages=None), dict(table=MIS2), dict(free=None), dict(cap=-1), dict(n_free=None),
                dict(slots=MIS4), dict(slots=None)):
        assert call(so.kv8_page_plan, good, order, **bad) == kv.KV8_EINVAL, bad


def test_mask_refusals(so):
    order = "B q_start lens R parent mask words position err st".split()
    good = dict(B=2, q_start=FAKE, lens=FAKE, R=4, parent=FAKE, mask=FAKE, words=1, position=FAKE, err=None, st=None)
    for bad in (dict(B=0), dict(words=0), dict(words=9), dict(R=-1), dict(q_start=None), dict(lens=MIS2), dict(parent=None),
                dict(mask=MIS2), dict(position=MIS2)):
        assert call(so.kv8_tree_mask, good, order, **bad) == kv.KV8_EINVAL, bad
    assert call(so.kv8_tree_mask, good, order, R=0, parent=None, mask=None) == kv.KV8_OK


def test_attention_refusals(so):
    order = "ql qr dt R H B q_start lens mask words kv8 sc rows table most page sm ws wsb err out odt st".split()
    good = dict(ql=FAKE, qr=FAKE, dt=kv.KV8_BF16, R=4, H=16, B=2, q_start=FAKE, lens=FAKE, mask=FAKE, words=1, kv8=FAKE,
                sc=FAKE, rows=1000, table=FAKE, most=5, page=64, sm=0.07, ws=FAKE, wsb=1 << 40, err=None, out=FAKE,
                odt=kv.KV8_BF16, st=None)
    for bad in (dict(ql=MIS8), dict(qr=None), dict(dt=2), dict(R=0), dict(R=kv.KV8_MAX_ROWS + 1), dict(H=0), dict(H=129),
                dict(B=0), dict(B=4097), dict(q_start=MIS2), dict(lens=None), dict(mask=MIS2), dict(words=0), dict(words=9),
                dict(kv8=MIS8), dict(sc=MIS2), dict(rows=0), dict(rows=1 << 31), dict(table=None), dict(most=0),
                dict(page=8), dict(page=100), dict(page=1 << 17), dict(sm=float("nan")), dict(sm=float("inf")), dict(ws=MIS8),
                dict(out=None), dict(out=MIS4), dict(odt=5)):
        assert call(so.mla_absorb_tree8, good, order, **bad) == kv.KV8_EINVAL, bad
    assert call(so.mla_absorb_tree8, good, order, wsb=1024) == kv.KV8_EWORKSPACE
    sz = ctypes.c_size_t(0)
    for a in ((0, 16, 2, 1), (4, 0, 2, 1), (4, 129, 2, 1), (4, 16, 0, 1), (4, 16, 4097, 1), (4, 16, 2, 7)):
        assert so.mla_tree8_workspace_bytes(*a, ctypes.addressof(sz)) == kv.KV8_EINVAL
    assert so.mla_tree8_workspace_bytes(4, 16, 2, 1, None) == kv.KV8_EINVAL


def test_commit_refusals(so):
    order = "B q_start lens accept count most layers kv8 sc rows table pages page new err st".split()
    good = dict(B=2, q_start=FAKE, lens=FAKE, accept=FAKE, count=FAKE, most=5, layers=1, kv8=FAKE, sc=FAKE, rows=100,
                table=FAKE, pages=4, page=16, new=FAKE + 64, err=None, st=None)
    for bad in (dict(B=0), dict(accept=None), dict(count=MIS2), dict(most=0), dict(most=257), dict(layers=0),
                dict(layers=65536), dict(kv8=MIS8), dict(sc=MIS2), dict(rows=0), dict(rows=1 << 31), dict(table=None),
                dict(pages=0), dict(page=24), dict(new=None), dict(new=FAKE)):
        assert call(so.kv8_tree_commit, good, order, **bad) == kv.KV8_EINVAL, bad


def test_binding_refuses_wrong_tensors(monkeypatch):
    """The checks themselves need no GPU: the current device is taken to be the tensors' (-1 for the CPU)."""
    i32 = torch.int32
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    t = torch.zeros((4, 6), dtype=i32)
    kv._args("f", ("t", t, i32, (4, 6)), ("none", None, i32, (1,)))
    with pytest.raises(TypeError, match="f: t must be"):
        kv._args("f", ("t", t.long(), i32, (4, 6)))
    with pytest.raises(ValueError, match="shape"):
        kv._args("f", ("t", t, i32, (6, 4)))
    with pytest.raises(ValueError, match="strides"):
        kv._args("f", ("t", t.t(), i32, (6, 4)))
    with pytest.raises(ValueError, match="contiguous"):
        kv._args("f", ("t", t[:, ::2], i32, (4, 3)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        kv._args("f", ("t", t, i32, (4, 6)))
    with pytest.raises(TypeError, match="bfloat16"):
        kv.mla_tree8_workspace_bytes(1, 1, 1, torch.float16)


def test_commit_refuses_lengths_that_overlap(so):
    """Blocks of other layers still read lens while new_lens is written."""
    order = "B q_start lens accept n_accept most layers kv8 sc rows table pages page new st".split()
    order.insert(order.index("st"), "err")
    good = dict(B=4, q_start=FAKE, lens=FAKE, accept=FAKE, n_accept=FAKE, most=4, layers=1, kv8=FAKE, sc=FAKE, rows=1000,
                table=FAKE, pages=5, page=64, new=FAKE, err=None, st=None)
    for new in (FAKE, FAKE + 4, FAKE + 12, FAKE - 12):
        assert call(so.kv8_tree_commit, good, order, new=new) == kv.KV8_EINVAL, new


def test_the_current_stream_is_found_by_its_public_name_too(monkeypatch):
    """torch's raw lookup is no public name: without it the same stream comes from torch.cuda.current_stream."""
    class Fake:
        cuda_stream = 77

    asked = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: asked.append(dev) or Fake)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    assert kv._stream(None) == 103 and kv._stream(None, 1) == 101 and asked == []
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert kv._stream(None) == 77 and kv._stream(None, 1) == 77 and asked == [3, 1]
    assert kv._stream(5) == 5 and kv._stream(Fake) == 77
