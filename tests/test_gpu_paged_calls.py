"""Calls of the paged and prompt operators that their documentation allows: single rows of any stride."""

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
