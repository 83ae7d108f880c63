"""More of the paged calls' host side (no GPU): pools whose size does not fit an address, rows whose stride has no meaning."""

import pytest
import torch

from kv_cache_quantization_turboquantprod_b200 import tq
from test_paged_host import A, _append, _batch, _cache

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("d,h_kv,page,pages,fits", [(256, MOST, 1024, MOST, False), (64, MOST, 16, MOST, False), (256, 1 << 20, 1024, MOST, False),
                                                    (64, 1 << 20, 16, MOST, True), (128, 8, 1024, MOST, True)])
def test_pools_beyond_an_address(d, h_kv, page, pages, fits):
    want = pages * h_kv * (page // 16) * 20 * d
    assert fits == (want < 1 << 64)
    lib = tq.load()
    assert lib.tq_paged_bytes(d, h_kv, page, pages) == (want if fits else 0)
    if fits:
        return
    pool = lambda: _cache(d=d, h_kv=h_kv, page=page, pages=pages)  # noqa: E731
    assert _append(c=pool()) == 3
    assert lib.tq_paged_gather(pool(), _batch(), A, None, 4, A, A, 1, 1024, 1024, None) == 3
    assert lib.tq_paged_decode_attention(pool(), _batch(), A, 1, 32, 4096, 0.1, A, 4096, A, 1 << 30, None) == 3
    assert lib.tq_paged_decode_workspace_size(pool(), 2, 32) == 0
    with pytest.raises(tq.TQError):
        tq.PagedCache(d, h_kv, page, pages, buffer=torch.zeros(16, dtype=torch.uint8))


@pytest.mark.parametrize("stride", [0, 7, 129, 1027])
def test_one_row_has_no_stride(stride):
    """A single token's rows count as packed, whatever lies between it and a next one."""
    x = torch.zeros(4096, dtype=torch.bfloat16)
    one = x.as_strided((1, 2, 64), (stride, 64, 1))
    assert tq._token_rows("k", one, 2, 64, torch.bfloat16, x.device, 1) == 128
    assert tq._token_rows("k", x.as_strided((0, 2, 64), (stride, 64, 1)), 2, 64, torch.bfloat16, x.device, 0) == 128
    two = x.as_strided((2, 2, 64), (stride, 64, 1))
    assert tq._token_rows("k", two, 2, 64, torch.bfloat16, x.device, 2) == stride
