"""The paged and prompt calls whose bounded waits run out while their own copies and products go on: every call returns, says so,
writes nothing that is finite and wrong, and leaves the kernels beside and behind it alone."""

import numpy as np
import pytest
import torch

from kv_cache_quantization_turboquantprod_b200 import tq

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kv_cache_quantization_turboquantprod_b200 import build
    build.build()
    tq.load()


@pytest.fixture
def hook():
    """Sets the test hook; always off again at the end."""
    tq.tq_device_errors(clear=True)
    try:
        yield tq.tq_test_withhold_handoffs
    finally:
        tq.tq_test_withhold_handoffs(0)
        tq.tq_set_wait_limit_ns(0)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cu(n):
    return _i32(np.concatenate([[0], np.cumsum(n)]).tolist())


def _pool(d, h_kv, page, total, fill):
    need = [-(-n // page) for n in total]
    table, at = np.zeros((len(total), max(need)), np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        at += n
    cache = tq.PagedCache(d, h_kv, page, at)
    cache.buffer.fill_(fill)
    return cache, tq.PagedBatch(_i32(list(total)), torch.from_numpy(table).to(DEV))


@pytest.mark.parametrize("d,h_q,h_kv,dtype", [(128, 8, 2, BF16), (64, 6, 3, F16), (256, 8, 1, F32)])
@pytest.mark.parametrize("rows", [(1, 1), (500, 1203)])
def test_append_that_gives_up_waits_for_its_copies(hook, d, h_q, h_kv, dtype, rows):
    """Appends that count their copies as late write no page and no row; appends beside them on another stream and right behind
    them (whose blocks take over the same shared memory) store what they store alone."""
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(sum(rows), h_q + 2 * h_kv, d, generator=g, device=DEV).to(dtype)
    q, k, v = x[:, :h_q], x[:, h_q : h_q + h_kv], x[:, h_q + h_kv :]
    cu, rope = _cu(rows), tq.Rope(tq.tq_make_rope_table(max(rows), d).to(DEV))

    def append(world, qo):
        tq.tq_paged_append(*world, cu, k, v, q=q, rope=rope, q_out=qo)

    worlds = [_pool(d, h_kv, 64, rows, 0x5A) for _ in range(3)]
    rows_out = [torch.full((sum(rows), h_q, d), 7.0, dtype=dtype, device=DEV) for _ in range(3)]
    append(worlds[0], rows_out[0])
    want, want_rows = worlds[0][0].buffer.clone(), rows_out[0].clone()
    assert tq.tq_device_errors() == 0 and not torch.equal(want, worlds[1][0].buffer)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        hook(2)
        append(worlds[1], rows_out[1])
        hook(0)
        worlds[0][0].buffer.fill_(0x5A)
        append(worlds[0], rows_out[0])
        with torch.cuda.stream(side):
            worlds[2][0].buffer.fill_(0x5A)
            append(worlds[2], rows_out[2])
        torch.cuda.synchronize()
        assert (worlds[1][0].buffer == 0x5A).all() and (rows_out[1] == 7.0).all()
        for i in (0, 2):
            assert torch.equal(worlds[i][0].buffer, want) and torch.equal(rows_out[i], want_rows)
    assert tq.tq_device_errors(clear=True) == tq.ERRF_QUANTIZE_WAIT
