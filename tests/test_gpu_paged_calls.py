"""Calls of the paged and prompt operators that their documentation allows and that are easily got wrong: single rows of any stride,
block tables cut from wider ones, first calls under capture, calls from several threads, row boundaries outside the rows, NaN in
cached groups, the widest groups of heads."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import paged_bounds as pb
from kv_cache_quantization_turboquantprod_b200 import tq
from oracle import paged

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kv_cache_quantization_turboquantprod_b200 import build
    build.build()
    tq.load()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _world(d, h_kv, page, total):
    need = [-(-n // page) for n in total]
    table, at = np.zeros((len(total), max(need)), np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        at += n
    cache = tq.PagedCache(d, h_kv, page, at)
    cache.buffer.zero_()
    return cache, tq.PagedBatch(_i32(list(total)), torch.from_numpy(table).to(DEV))


@pytest.mark.parametrize("stride", [129 * 8 + 1, 3])
def test_one_row_of_any_stride(stride):
    """A decode step of one sequence, its rows cut from wider tensors: the same as packed rows."""
    d, h_q, h_kv = 64, 4, 2
    x = torch.randn(4, 8192, device=DEV).to(BF16)
    row = lambda i, h: x[i].as_strided((1, h, d), (stride, d, 1), x[i].storage_offset())  # noqa: E731
    got = []
    for pack in (False, True):
        cache, batch = _world(d, h_kv, 16, [1])
        q, k, v = row(0, h_q), row(1, h_kv), row(2, h_kv)
        out = torch.zeros(1, 4096, device=DEV, dtype=BF16).as_strided((1, h_q, d), (stride, d, 1))
        ko, vo = (torch.zeros(1, 4096, device=DEV, dtype=BF16).as_strided((1, h_kv, d), (stride, d, 1)) for _ in range(2))
        if pack:
            q, k, v, out, ko, vo = (t.reshape(-1).clone().view(t.shape) for t in (q, k, v, out, ko, vo))
        po = torch.zeros(1, h_q, d, dtype=BF16, device=DEV)
        tq.tq_paged_append(cache, batch, _i32([0, 1]), k, v)
        tq.tq_paged_gather(cache, batch, _i32([0, 1]), ko, vo)
        tq.tq_paged_decode_attention(cache, batch, q, out, tq.paged_workspace_for(cache, batch, h_q))
        tq.tq_prompt_attention(q, k, v, _i32([0, 1]), _i32([0, 1]), po)
        got.append([cache.buffer.clone()] + [t.clone() for t in (ko, vo, out, po)])
    for a, b in zip(*got):
        assert torch.equal(a.reshape(-1), b.reshape(-1))
    assert got[0][3].any() and tq.tq_device_errors() == 0


def test_a_table_cut_from_a_wider_one():
    """Rows of the block table further apart than their length, with page numbers behind them that are no pages."""
    d, h_kv, total = 128, 2, [100, 33, 64]
    g = torch.Generator(device=DEV).manual_seed(0)
    k, v = (torch.randn(sum(total), h_kv, d, generator=g, device=DEV) for _ in range(2))
    q = torch.randn(3, 8, d, generator=g, device=DEV).to(BF16)
    cu = _i32([0, 100, 133, 197])
    got = []
    for wide in (False, True):
        cache, batch = _world(d, h_kv, 16, total)
        if wide:
            table = torch.full((3, 11), -77, dtype=torch.int32, device=DEV)
            table[:, 2 : 2 + batch.max_pages] = batch.block_table
            batch = tq.PagedBatch(batch.len_dev, table[:, 2 : 2 + batch.max_pages])
        out, ko, vo = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        tq.tq_paged_append(cache, batch, cu, k, v)
        tq.tq_paged_gather(cache, batch, cu, ko, vo)
        tq.tq_paged_decode_attention(cache, batch, q, out, tq.paged_workspace_for(cache, batch, 8))
        got.append((cache.buffer, out, ko, vo))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and tq.tq_device_errors() == 0


@pytest.mark.parametrize("B", [1, 31, 32, 33, 40, 300])
def test_gather_from_first_positions_of_many_sequences(B):
    """Histories from a position of each sequence on, on either side of the 32 sequences that a warp looks up at once."""
    rng = np.random.default_rng(B)
    total = [int(x) for x in rng.integers(1, 60, B)]
    first = [int(rng.integers(0, n)) for n in total]
    count = [int(rng.integers(0, n - f + 1)) for n, f in zip(total, first)]
    cache, batch = _world(64, 1, 16, total)
    x = torch.randn(sum(total), 1, 64, device=DEV)
    cu = np.concatenate([[0], np.cumsum(total)])
    tq.tq_paged_append(cache, batch, _i32(cu.tolist()), x, -x)
    every = [torch.zeros_like(x) for _ in range(2)]
    tq.tq_paged_gather(cache, batch, _i32(cu.tolist()), *every)
    rows = np.concatenate([np.arange(c + f, c + f + n) for c, f, n in zip(cu, first, count)]).astype(np.int64)
    some = [torch.full((len(rows) + 2, 1, 64), 5.0, device=DEV) for _ in range(2)]
    tq.tq_paged_gather(cache, batch, _i32(np.concatenate([[0], np.cumsum(count)]).tolist()), *some, first=_i32(first))
    for a, b in zip(every, some):
        assert torch.equal(a[torch.from_numpy(rows).to(DEV)], b[: len(rows)]) and (b[len(rows) :] == 5.0).all()
    assert tq.tq_device_errors() == 0


@pytest.mark.parametrize("cu", [[0, 5, 2 ** 31 - 1], [-7, 5, 9], [-2 ** 31, 5, 10 ** 6], [5, 5, 5]])
def test_row_boundaries_outside_the_rows_are_clamped(cu):
    """Boundaries before the first and behind the last row: nothing is read or written outside the rows."""
    T, d = 8, 64
    inside = [min(max(c, 0), T) for c in cu]
    total = [b - a for a, b in zip(inside, inside[1:])]
    cache, batch = _world(d, 1, 16, [max(n, 1) for n in total])
    batch.len_dev.copy_(_i32(total))
    x = torch.randn(T, 1, d, device=DEV).to(BF16)
    guard = [torch.full((T + 64, 1, d), 5.0, dtype=BF16, device=DEV) for _ in range(4)]
    part = [t[32 : 32 + T] for t in guard]
    tq.tq_paged_append(cache, batch, _i32(cu), x, x, k_out=part[0])
    tq.tq_paged_gather(cache, batch, _i32(cu), part[1], part[2])
    tq.tq_prompt_attention(x, x, x, _i32(cu), _i32(cu), part[3])
    lo, hi = inside[0], inside[-1]
    assert torch.equal(part[0][lo:hi], x[lo:hi])
    for t in guard:
        assert (t[: 32 + lo] == 5.0).all() and (t[32 + hi :] == 5.0).all()
    want = torch.full_like(x, 5.0)
    tq.tq_prompt_attention(x, x, x, _i32(inside), _i32(inside), want)
    assert torch.equal(part[3], want) and tq.tq_device_errors() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_in_cached_groups_reaches_its_channels_only(d, dtype):
    """A value group with a NaN or an infinity (at any token) makes its 32 channels NaN and leaves the others right; a key row with
    one makes its KV head's rows NaN."""
    n, h_kv, G = 300, 2, 4
    rng = np.random.default_rng(d)
    x, y = (rng.standard_normal((n, h_kv, d)).astype(np.float32) for _ in range(2))
    bad = y.copy()
    bad[150, 0, 3] = np.nan
    bad[299, 1, 40] = np.inf
    g = torch.Generator().manual_seed(1)
    q = (0.5 * torch.randn(1, G * h_kv, d, generator=g)).to(dtype).to(DEV)

    def decode(keys, values):
        cache, batch = _world(d, h_kv, 16, [n])
        tq.tq_paged_append(cache, batch, _i32([0, n]), torch.from_numpy(keys).to(DEV), torch.from_numpy(values).to(DEV))
        out = torch.zeros_like(q)
        tq.tq_paged_decode_attention(cache, batch, q, out, tq.paged_workspace_for(cache, batch, G * h_kv))
        return out.double().cpu().numpy()[0].reshape(h_kv, G, d)

    got = decode(x, bad)
    assert np.isnan(got[0, :, :32]).all() and np.isnan(got[1, :, 32:64]).all()
    for h in range(h_kv):
        key, val = paged.encode(x[:, h]), paged.encode(y[:, h])
        k, v = (r["codes"] * r["scale16"].repeat(32, 1) + r["zero16"].repeat(32, 1) for r in (key, val))
        other = np.ones(d, bool)
        other[32 * h : 32 * h + 32] = False
        for i in range(G):
            qi = q[0, h * G + i].double().cpu().numpy()
            o, tol = pb.attend(qi, k, v, d ** -0.5)[1], pb.bound(qi, k, key, v, val, d ** -0.5, 8 if dtype == BF16 else 11)
            assert (np.abs(got[h, i] - o) <= tol)[other].all()
    worse = x.copy()
    worse[7, 1, d - 1] = -np.inf
    got = decode(worse, y)
    assert np.isnan(got[1]).all() and np.isfinite(got[0]).all()
    assert tq.tq_device_errors() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,h_kv", [(64, 2), (128, 1), (256, 1)])
def test_eight_heads_a_kv_head(d, h_kv, dtype):
    """The widest groups: a block's largest shared memory."""
    n = (1000, 3)
    rng = np.random.default_rng(d)
    x, y = (rng.standard_normal((sum(n), h_kv, d)).astype(np.float32) for _ in range(2))
    cache, batch = _world(d, h_kv, 64, list(n))
    tq.tq_paged_append(cache, batch, _i32([0, n[0], sum(n)]), torch.from_numpy(x).to(DEV), torch.from_numpy(y).to(DEV))
    g = torch.Generator().manual_seed(1)
    q = (0.5 * torch.randn(2, 8 * h_kv, d, generator=g)).to(dtype).to(DEV)
    out = torch.zeros_like(q)
    tq.tq_paged_decode_attention(cache, batch, q, out, tq.paged_workspace_for(cache, batch, 8 * h_kv))
    got, at = out.double().cpu().numpy(), 0
    for b, m in enumerate(n):
        for h in range(h_kv):
            key, val = paged.encode(x[at : at + m, h]), paged.encode(y[at : at + m, h])
            k, v = (r["codes"] * r["scale16"].repeat(32, 1) + r["zero16"].repeat(32, 1) for r in (key, val))
            for i in range(8 * h, 8 * h + 8):
                qi = q[b, i].double().cpu().numpy()
                o, tol = pb.attend(qi, k, v, d ** -0.5)[1], pb.bound(qi, k, key, v, val, d ** -0.5, 8 if dtype == BF16 else 11)
                assert (np.abs(got[b, i] - o) <= tol).all()
        at += m


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from kv_cache_quantization_turboquantprod_b200 import tq
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
cache = tq.PagedCache(128, 2, 16, 8)
cache.buffer.zero_()
batch, cu = tq.PagedBatch(i32([40]), torch.arange(8, dtype=torch.int32, device="cuda")[None]), i32([0, 40])
q, k = torch.randn(40, 8, 128, device="cuda").half(), torch.randn(40, 2, 128, device="cuda").half()
v, out, ko, vo, one = k.clone(), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(k), torch.zeros_like(q[:1])
ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
calls = dict(append=lambda: tq.tq_paged_append(cache, batch, cu, k, v), gather=lambda: tq.tq_paged_gather(cache, batch, cu, ko, vo),
             decode=lambda: tq.tq_paged_decode_attention(cache, batch, q[:1], one, ws),
             prompt=lambda: tq.tq_prompt_attention(q, k, v, cu, cu, out))
call, state = calls[sys.argv[1]], (cache.buffer, ko, vo, one, out)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in state]
call()
torch.cuda.synchronize()
assert all(torch.equal(a.nan_to_num() if a.is_floating_point() else a, b.nan_to_num() if b.is_floating_point() else b)
           for a, b in zip(got, state))
assert tq.tq_device_errors() == 0
print("same")
"""


@pytest.mark.parametrize("which", ["append", "gather", "decode", "prompt"])
def test_a_first_call_may_be_captured(which):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root), which], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr


def test_calls_from_several_threads():
    """Four host threads, each with its stream, pool, workspace and lengths, at once: what each gets alone."""
    d, h_q, h_kv = 128, 8, 2

    def job(i, results):
        with torch.cuda.stream(torch.cuda.Stream()):
            g = torch.Generator(device=DEV).manual_seed(i)
            total = [200 + 37 * i, 5]
            cu = _i32([0, total[0], sum(total)])
            q, k, v = (torch.randn(sum(total), h, d, generator=g, device=DEV).to(BF16) for h in (h_q, h_kv, h_kv))
            cache, batch = _world(d, h_kv, 16, total)
            ws, got = tq.paged_workspace_for(cache, batch, h_q), []
            for _ in range(20):
                out, one = torch.zeros_like(q), torch.zeros_like(q[:2])
                tq.tq_paged_append(cache, batch, cu, k, v)
                tq.tq_prompt_attention(q, k, v, cu, cu, out)
                tq.tq_paged_decode_attention(cache, batch, q[:2], one, ws)
                got.append((out, one))
            torch.cuda.current_stream().synchronize()
            assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got)
            results[i] = (got[0][0], got[0][1], cache.buffer)

    alone, together = {}, {}
    for i in range(4):
        job(i, alone)
    threads = [threading.Thread(target=job, args=(i, together)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert sorted(together) == [0, 1, 2, 3]
    for i in range(4):
        assert all(torch.equal(a, b) for a, b in zip(alone[i], together[i]))
    assert tq.tq_device_errors() == 0


def test_an_explicit_stream():
    """stream= takes a stream's handle or object: the calls run there and not on the current one."""
    d, total = 64, [70]
    x = torch.randn(70, 1, d, device=DEV).to(BF16)
    cu, side = _i32([0, 70]), torch.cuda.Stream()
    cache, batch = _world(d, 1, 16, total)
    got = torch.zeros_like(x)
    ko, vo = torch.zeros_like(x), torch.zeros_like(x)
    one, ws = torch.zeros_like(x[:1]), tq.paged_workspace_for(cache, batch, 1)
    torch.cuda.synchronize()
    tq.tq_paged_append(cache, batch, cu, x, x, stream=side)
    tq.tq_paged_gather(cache, batch, cu, ko, vo, stream=side)
    tq.tq_prompt_attention(x, ko, vo, cu, cu, got, stream=side)
    tq.tq_paged_decode_attention(cache, batch, x[69:], one, ws, stream=side)
    side.synchronize()
    ref = torch.zeros_like(x)
    tq.tq_prompt_attention(x, ko, vo, cu, cu, ref)
    assert torch.equal(got, ref) and (one - got[69:]).abs().max() < 0.05 and tq.tq_device_errors() == 0
