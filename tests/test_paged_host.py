"""Host-side refusals of the paged and prompt calls (no GPU: every error below is found before any launch)."""

import ctypes

import pytest
import torch

from kv_cache_quantization_turboquantprod_b200 import tq

A = 1 << 20  # an aligned address that is never dereferenced


def _cache(**kw):
    x = dict(d=128, h_kv=8, page=64, pages=10, data=A) | kw
    return ctypes.byref(tq._PagedCacheStruct(x["d"], x["h_kv"], x["page"], x["pages"], x["data"]))


def _batch(**kw):
    x = dict(batch=2, max_pages=4, stride=4, len=A, table=A) | kw
    return ctypes.byref(tq._PagedBatchStruct(x["batch"], x["max_pages"], x["stride"], x["len"], x["table"]))


def _rope(**kw):
    x = dict(rot=128, most=64, inter=0, table=A) | kw
    return ctypes.byref(tq._RopeStruct(x["rot"], x["most"], x["inter"], x["table"]))


BAD_POOL = [(dict(data=None), 1), (dict(data=A + 16), 1), (dict(d=96), 2), (dict(page=8), 2), (dict(page=48), 2),
            (dict(page=2048), 2), (dict(h_kv=0), 1), (dict(pages=0), 1)]
BAD_BATCH = [(dict(batch=0), 1), (dict(max_pages=0), 1), (dict(stride=3), 1), (dict(len=None), 1), (dict(table=None), 1),
             (dict(len=A + 2), 1), (dict(max_pages=1 << 28, stride=1 << 28), 3)]


def _append(c=None, b=None, rope=None, **kw):
    x = dict(cu=A, q=A, k=A, v=A, dt=1, hq=32, T=4, qs=4096, ks=1024, vs=1024, qo=2 * A, ko=3 * A, qos=4096, kos=1024) | kw
    return tq.load().tq_paged_append(c or _cache(), b or _batch(), rope, x["cu"], x["q"], x["k"], x["v"], x["dt"], x["hq"], x["T"],
                                     x["qs"], x["ks"], x["vs"], x["qo"], x["ko"], x["qos"], x["kos"], None)


@pytest.mark.parametrize("pool,want", BAD_POOL)
def test_bad_pools(pool, want):
    lib = tq.load()
    assert _append(c=_cache(**pool)) == want
    assert lib.tq_paged_gather(_cache(**pool), _batch(), A, None, 4, A, A, 1, 1024, 1024, None) == want
    assert lib.tq_paged_decode_attention(_cache(**pool), _batch(), A, 1, 32, 4096, 0.1, A, 4096, A, 1 << 30, None) == want
    assert lib.tq_paged_decode_workspace_size(_cache(**pool), 2, 32) == 0
    x = dict(d=128, h_kv=8, page=64, pages=10) | {k: v for k, v in pool.items() if k != "data"}
    assert ("data" in pool) == (lib.tq_paged_bytes(x["d"], x["h_kv"], x["page"], x["pages"]) > 0)


@pytest.mark.parametrize("batch,want", BAD_BATCH)
def test_bad_batches(batch, want):
    lib = tq.load()
    assert _append(b=_batch(**batch)) == want
    assert lib.tq_paged_gather(_cache(), _batch(**batch), A, None, 4, A, A, 1, 1024, 1024, None) == want
    assert lib.tq_paged_decode_attention(_cache(), _batch(**batch), A, 1, 32, 4096, 0.1, A, 4096, A, 1 << 30, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dt=3), 2), (dict(T=-1), 1), (dict(T=0, k=None, v=None), 0), (dict(cu=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(k=A + 8), 1), (dict(ks=1023), 1), (dict(ks=1028), 1), (dict(vs=512), 1), (dict(q=A + 2), 1), (dict(qo=None), 1),
    (dict(hq=12), 1), (dict(hq=4), 1), (dict(qs=4000), 1), (dict(ko=A + 8), 1), (dict(ko=A, kos=2048), 1),
    (dict(qo=A, qos=8192), 1), (dict(T=0x7fffffff), 3), (dict(hq=72, qs=9216, qos=9216), 2)])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


@pytest.mark.parametrize("kw,want", [(dict(rot=8), 2), (dict(rot=144), 2), (dict(rot=24), 2), (dict(table=None), 1),
                                     (dict(table=A + 4), 1), (dict(most=0), 1)])
def test_rope_refusals(kw, want):
    assert _append(rope=_rope(**kw)) == want


@pytest.mark.parametrize("kw,want", [(dict(rows=-1), 1), (dict(rows=0, k=None), 0), (dict(cu=None), 1), (dict(first=A + 1), 1),
                                     (dict(k=None), 1), (dict(v=A + 4), 1), (dict(ks=512), 1), (dict(dt=9), 2)])
def test_gather_refusals(kw, want):
    x = dict(cu=A, first=None, rows=4, k=A, v=A, dt=1, ks=1024, vs=1024) | kw
    assert tq.load().tq_paged_gather(_cache(), _batch(), x["cu"], x["first"], x["rows"], x["k"], x["v"], x["dt"], x["ks"], x["vs"],
                                     None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(dt=0), 2), (dict(dt=3), 2), (dict(hq=12), 1), (dict(hq=4), 1), (dict(hq=72), 2),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(scale=3e38), 1), (dict(qs=128), 1), (dict(os=4100), 1), (dict(ws=None), 4),
    (dict(ws=A + 16), 4)])
def test_decode_refusals(kw, want):
    x = dict(q=A, dt=1, hq=32, qs=4096, scale=0.1, out=A, os=4096, ws=A, wsb=1 << 30) | kw
    qs = x["qs"] if "qs" in kw else max(x["qs"], x["hq"] * 128)
    os_ = x["os"] if "os" in kw else max(x["os"], x["hq"] * 128)
    assert tq.load().tq_paged_decode_attention(_cache(), _batch(), x["q"], x["dt"], x["hq"], qs, x["scale"], x["out"], os_,
                                               x["ws"], x["wsb"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(out=None), 1), (dict(dt=0), 2), (dict(d=80), 2), (dict(hq=12), 1), (dict(hkv=0), 1),
    (dict(hq=72), 2), (dict(Tq=-1), 1), (dict(Tk=-1), 1), (dict(batch=0), 1), (dict(cu=None), 1), (dict(cu=A + 2), 1),
    (dict(scale=float("nan")), 1), (dict(scale=-3e38), 1), (dict(qs=64), 1), (dict(vs=1028), 1), (dict(Tq=0, q=None), 0), (dict(Tq=(1 << 30) + 1), 3),
    (dict(batch=(1 << 20) + 1), 3)])
def test_prompt_refusals(kw, want):
    x = dict(q=A, k=A, v=A, dt=1, Tq=4, Tk=4, hq=32, hkv=8, d=128, qs=1 << 14, ks=1024, vs=1024, cu=A, batch=2, scale=0.1, out=A,
             os=1 << 14) | kw
    assert tq.load().tq_prompt_attention(x["q"], x["k"], x["v"], x["dt"], x["Tq"], x["Tk"], x["hq"], x["hkv"], x["d"], x["qs"],
                                         x["ks"], x["vs"], x["cu"], x["cu"], x["batch"], x["scale"], x["out"], x["os"], None) == want


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        tq.PagedCache(128, 1, 16, 1, buffer=torch.zeros(2560, dtype=torch.uint8))
    with pytest.raises(tq.TQError):
        tq.PagedCache(96, 1, 16, 1, buffer=torch.zeros(2560, dtype=torch.uint8))
    with pytest.raises(ValueError):
        tq.PagedBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(TypeError):
        tq.PagedBatch(torch.zeros(2, dtype=torch.int64), torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        tq.Rope(torch.zeros(4, 32))
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tq.tq_prompt_attention(x, x, x, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), x)
    with pytest.raises(TypeError):
        tq.tq_prompt_attention(x.float(), x, x, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), x)
