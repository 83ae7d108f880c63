"""The paged decode against its 64-bit definition, channel by channel, within the bounds of paged_bounds (test_paged_bounds shows
that these see a lost token, a shifted tail and a wrong scale): ordinary data, groups of unlike sizes, tokens of unlike sizes, and
the number of sequences at which the splitting changes."""

import numpy as np
import pytest
import torch

import paged_bounds as pb
from kv_cache_quantization_turboquantprod_b200 import tq
from oracle import paged

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16
BITS = {BF16: 8, F16: 11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kv_cache_quantization_turboquantprod_b200 import build
    build.build()
    tq.load()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _part_cells(total, h_kv, d):
    """Cells of a warp's part of the batch: the steps (two cells) are cut into equal ranges, eight a block."""
    blocks = torch.cuda.get_device_properties(0).multi_processor_count * (1 if d == 256 else 2)
    steps = sum(-(-n // 32) for n in total) * h_kv
    return 2 * (-(-steps // (8 * blocks)) + 1)


class World:
    """Encoded keys and values of several sequences, in pages and as the oracle has them."""

    def __init__(self, x, y, d, h_kv, page, total):
        """x, y: float32 keys and values [T, h_kv, d]"""
        need = [-(-n // page) for n in total]
        order = np.random.default_rng(0).permutation(sum(need))
        table, at = np.zeros((len(total), max(1, max(need))), np.int32), 0
        for b, n in enumerate(need):
            table[b, :n] = order[at : at + n]
            at += n
        self.cache = tq.PagedCache(d, h_kv, page, at)
        self.cache.buffer.fill_(0xFF)
        self.batch = tq.PagedBatch(_i32(list(total)), torch.from_numpy(table).to(DEV))
        cu = np.concatenate([[0], np.cumsum(total)])
        tq.tq_paged_append(self.cache, self.batch, _i32(cu.tolist()), torch.from_numpy(x).to(DEV), torch.from_numpy(y).to(DEV))
        self.d, self.h_kv, self.total = d, h_kv, list(total)
        self.of = lambda b, h: [paged.encode(z[cu[b] : cu[b + 1], h]) for z in (x, y)]

    def check(self, q, scale=None, units=None):
        """Every channel of every head (or of the given (sequence, KV head) units) within its bound; the largest share of it."""
        d, G = self.d, q.shape[1] // self.h_kv
        out = torch.full_like(q, 9.0)
        ws = tq.paged_workspace_for(self.cache, self.batch, q.shape[1])
        ws.fill_(0xFF)
        tq.tq_paged_decode_attention(self.cache, self.batch, q, out, ws, softmax_scale=scale)
        scale = d ** -0.5 if scale is None else scale
        cells = _part_cells(self.total, self.h_kv, d)
        qs, got, most = q.double().cpu().numpy(), out.double().cpu().numpy(), 0.0
        for b, n in enumerate(self.total):
            for h in range(self.h_kv):
                if n == 0:
                    assert not got[b].any()
                    continue
                if units is not None and (b, h) not in units:
                    continue
                key, val = self.of(b, h)
                k, v = (r["codes"] * r["scale16"].repeat(32, 1) + r["zero16"].repeat(32, 1) for r in (key, val))
                for hq in range(h * G, h * G + G):
                    o = pb.attend(qs[b, hq], k, v, scale)[1]
                    share = np.abs(got[b, hq] - o) / pb.bound(qs[b, hq], k, key, v, val, scale, BITS[q.dtype], cells)
                    assert (share <= 1).all(), (b, hq, np.flatnonzero(~(share <= 1)), np.nanmax(share), np.abs(got[b, hq] - o).max())
                    most = max(most, float(share.max()))
        assert tq.tq_device_errors() == 0
        return most


def _data(seed, total, h_kv, d, sizes=(1.0,), k_size=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, sum(total), h_kv, d)) * np.exp(0.5 * rng.standard_normal((2, 1, h_kv, d)))
    x[0] *= k_size
    x[1] = np.clip(x[1] * np.resize(sizes, d // 32).repeat(32), -6e4, 6e4)  # (fp16 zeros)
    return x.astype(np.float32)


def _query(seed, B, h_q, d, dtype, size):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(B, h_q, d, generator=g)).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,h_q,h_kv,page,total", [(128, 8, 2, 16, (1, 15, 16, 17, 0, 257)), (64, 8, 1, 32, (333, 2, 48)),
                                                   (256, 6, 3, 64, (70, 150)), (128, 5, 5, 128, (64, 129, 200))])
@pytest.mark.parametrize("size", [0.375, 1.5])
def test_ordinary_values(d, h_q, h_kv, page, total, dtype, size):
    w = World(*_data(d, total, h_kv, d), d, h_kv, page, total)
    print("share of the bound", w.check(_query(1, len(total), h_q, d, dtype, size)))


UNLIKE = [(1000.0, 0.1), (1000.0, 0.01), (4000.0, 0.01), (4000.0, 0.001), (0.001, 20000.0), (1e-4, 1.0, 1e3, 1e-2)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sizes", UNLIKE)
def test_groups_of_unlike_sizes(d, sizes, dtype):
    """Groups of 32 channels up to 2e7 times larger than their neighbours: each as accurate as it is alone."""
    total = (90, 2048 if d == 64 else 600)
    w = World(*_data(d, total, 1, d, sizes), d, 1, 64, total)
    print("share of the bound", w.check(_query(2, len(total), 4, d, dtype, 0.75)))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_tokens_of_unlike_sizes(d, dtype):
    """A group's values grow and shrink along the sequence, each group at another token: the bounds of the groups move apart, in
    the middle of parts and between them."""
    total = (700,)
    x, y = _data(d, total, 2, d)
    rng = np.random.default_rng(5)
    for j in range(d // 32):
        at = np.sort(rng.integers(0, 700, 6))
        for a, s in zip(at, (0.01, 30.0, 500.0, 0.1, 3000.0, 1.0)):
            y[a:, :, 32 * j : 32 * j + 32] = rng.standard_normal((700 - a, 2, 32)) * s
    w = World(x, y, d, 2, 16, total)
    print("share of the bound", w.check(_query(3, 1, 8, d, dtype, 0.75)))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scale_k,scale_v,softmax", [(1e-3, 1e-3, None), (30.0, 300.0, None), (1.0, 1e-5, 0.5), (8.0, 1.0, -0.3),
                                                     (1.0, 1.0, 0.0)])
def test_ranges(scale_k, scale_v, softmax, dtype):
    total = (77, 200)
    w = World(*_data(11, total, 2, 128, (scale_v,), scale_k), 128, 2, 32, total)
    print("share of the bound", w.check(_query(4, 2, 8, 128, dtype, 1.0), softmax))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B", [255, 256, 257, 296, 297])
def test_one_head_of_as_many_sequences_as_threads_and_blocks(B, dtype):
    """One KV head and some 256 sequences (a block's threads) or 296 (two blocks an SM): where the prefix sums take a second round
    and the joining changes its form."""
    rng = np.random.default_rng(B)
    total = [int(n) for n in rng.integers(0, 70, B)]
    total[B // 2] = 3000  # one that many ranges share
    w = World(*_data(B, total, 1, 64), 64, 1, 16, total)
    units = {(b, 0) for b in list(range(0, B, 17)) + [B // 2 - 1, B // 2, B // 2 + 1, 255, 256, B - 2, B - 1]}
    print("share of the bound", w.check(_query(6, B, 2, 64, dtype, 0.375), units=units))
