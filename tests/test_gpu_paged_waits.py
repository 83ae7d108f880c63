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


def _prompt_inputs(d, h_q, h_kv, dtype, n, step=64):
    """Keys that are small in the first step and large behind it, so that the running maximum moves at the second."""
    g = torch.Generator(device=DEV).manual_seed(d + n)
    q = (1.5 * torch.randn(n, h_q, d, generator=g, device=DEV)).to(dtype)
    size = torch.where(torch.arange(n, device=DEV) < step, 0.25, 12.0)
    k = (torch.randn(n, h_kv, d, generator=g, device=DEV) * size[:, None, None]).to(dtype)
    return q, k, torch.randn(n, h_kv, d, generator=g, device=DEV).to(dtype)


def _many(tiles_a_head):
    """KV heads that give more than two tiles an SM."""
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count // tiles_a_head + 1


PROMPT = [
    # d, h_q / h_kv, h_kv (None: many tiles), dtype, tokens, keys of a step, tokens of a tile whose rows see one step only
    (64, 1, 2, BF16, 100, 64, 0),       # the failing step is the last one
    (128, 2, 2, F16, 100, 64, 64),
    (256, 1, 1, BF16, 120, 64, 0),
    (128, 1, 2, BF16, 200, 64, 0),      # more steps behind it
    (128, 1, 2, F16, 500, 128, 128),    # 128 keys a step, one tile
    (64, 1, None, BF16, 1400, 128, 0),  # two tiles, three score buffers
]


@pytest.mark.parametrize("d,group,h_kv,dtype,n,step,whole", PROMPT)
def test_prompt_wait_that_runs_out_for_one_half_of_a_row(hook, d, group, h_kv, dtype, n, step, whole):
    """A wait for the tile's products that runs out in one of a row's two threads: both leave, the call returns, and no row is
    finite and wrong (tiles of one step wait for no product)."""
    h_kv = h_kv or _many(n // (128 // group) + 1)
    q, k, v = _prompt_inputs(d, group * h_kv, h_kv, dtype, n, step)
    cu = _cu([n])
    clean = torch.full_like(q, 3.0)
    tq.tq_prompt_attention(q, k, v, cu, cu, clean)
    assert torch.isfinite(clean).all() and tq.tq_device_errors() == 0
    out = torch.full_like(q, 3.0)
    tq.tq_set_wait_limit_ns(2_000_000)
    hook(2)
    tq.tq_prompt_attention(q, k, v, cu, cu, out)
    assert tq.tq_device_errors(clear=True) == tq.ERRF_PROMPT_WAIT
    nan = torch.isnan(out).all(-1)
    assert nan[whole:].all() and not nan[:whole].any()
    assert torch.equal(out[:whole], clean[:whole])
    hook(0)
    tq.tq_set_wait_limit_ns(0)
    tq.tq_prompt_attention(q, k, v, cu, cu, out)
    assert torch.equal(out, clean) and tq.tq_device_errors() == 0


@pytest.mark.parametrize("d,h_q,h_kv,n", [(64, 2, 2, 300), (128, 8, 2, 1000), (256, 2, 1, 200)])
def test_prompt_without_its_copies_is_nan(hook, d, h_q, h_kv, n):
    q, k, v = _prompt_inputs(d, h_q, h_kv, BF16, n)
    cu = _cu([n])
    out = torch.full_like(q, 3.0)
    tq.tq_set_wait_limit_ns(2_000_000)
    hook(1)
    tq.tq_prompt_attention(q, k, v, cu, cu, out)
    assert tq.tq_device_errors(clear=True) == tq.ERRF_PROMPT_WAIT
    assert torch.isnan(out).all()
