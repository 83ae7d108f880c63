"""The prompt attention against its 64-bit definition, channel by channel: blocks of two tiles of unlike lengths in both types, keys
of a hundred thousand tokens, batches of many and of very unlike sequences.

Bound of a channel's error, in normalised weights w (SIGMA and the rule of sums as in paged_bounds):
 * output: one rounding, eps / 2; p in the operand type, eps / 2 of w v each, independent: SIGMA sqrt(sum (w v)^2); fp16's smallest
   step, 2^-25 of the largest weight, which is 1 or more.
 * logits: d + 8 roundings of 2^-23 of sum |q k| scale and 2^-20 of the exponential, which move the output by w (v - o).
 * float32 sums that truncate: 2^-23 of the sum so far for each 16 keys, of the largest product for each of the 16, and for some
   twenty moves of the maximum; 2^-24 of the sum of weights for each 32 keys.
"""

import numpy as np
import pytest
import torch

from kv_cache_quantization_turboquantprod_b200 import tq
from paged_bounds import SIGMA

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kv_cache_quantization_turboquantprod_b200 import build
    build.build()
    tq.load()


def _cu(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]).tolist(), dtype=torch.int32, device=DEV)


def _heads_for_two_tiles(new, G):
    """KV heads that give more than two tiles an SM, which blocks of two tiles take (from 2048 keys a sequence on)."""
    tiles = sum(new) // (128 // G) + len(new)
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count // tiles + 1


def _check_rows(q, k, v, past, got):
    """Queries [n, d] behind `past` keys of k, v [m, d]; the largest share of the bound."""
    (n, d), m, dt = q.shape, k.shape[0], q.dtype
    half = torch.finfo(dt).eps / 2
    q, k, v, got = (x.double() for x in (q, k, v, got))
    scale = d ** -0.5
    s = q @ k.T * scale
    hidden = torch.arange(m, device=DEV) > torch.arange(n, device=DEV)[:, None] + past
    w = torch.softmax(s.masked_fill(hidden, -torch.inf), -1)
    seen = ~hidden[:, 0] if m else torch.zeros(n, dtype=torch.bool, device=DEV)
    assert not got[~seen].any()
    if not seen.any():
        return 0.0
    w = w.masked_fill(~seen[:, None], 0.0)
    o = w @ v
    logit = (d + 8) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T) + 2.0 ** -20
    wl = w * logit
    tol = half * o.abs() + SIGMA * half * ((w * w) @ (v * v)).sqrt() + wl @ v.abs() + wl.sum(-1, keepdim=True) * o.abs()
    if dt == F16:
        tol = tol + w.amax(-1, keepdim=True) * 2.0 ** -25 * v.abs().sum(0)
    pad = -m % 64
    w64 = torch.nn.functional.pad(w, (0, pad)).view(n, -1, 64)
    v64 = torch.nn.functional.pad(v, (0, 0, 0, pad)).view(-1, 64, d)
    so_far = torch.einsum("ncj,cjd->ncd", w64, v64).cumsum(1).abs().amax(1)
    top = w64.reshape(n, -1, 16).amax(-1) @ v64.abs().reshape(-1, 16, d).amax(1)
    tol = tol + 2.0 ** -23 * ((m / 16 + 20) * so_far + 16 * top) + (m / 32 + 10) * 2.0 ** -24 * o.abs() + 2.0 ** -25
    share = ((got - o).abs() / tol)[seen]
    assert bool((share <= 1).all()), (float(share.nan_to_num(9e9).max()), int((~(share <= 1)).sum()), share.shape)
    return float(share.max())


def _run(new, nk, h_q, h_kv, d, dtype, heads, grow=None, seed=0, sequences=None):
    g = torch.Generator(device=DEV).manual_seed(seed + d + h_q)
    q = torch.randn(sum(new), h_q, d, generator=g, device=DEV).to(dtype)
    k = torch.randn(sum(nk), h_kv, d, generator=g, device=DEV)
    if grow is not None:
        k *= torch.cat([torch.linspace(*grow, m, device=DEV) for m in nk])[:, None, None]
    k = k.to(dtype)
    v = torch.randn(sum(nk), h_kv, d, generator=g, device=DEV).to(dtype)
    out = torch.full_like(q, 3.0)
    cu_q, cu_k = _cu(new), _cu(nk)
    tq.tq_prompt_attention(q, k, v, cu_q, cu_k, out)
    a = c = 0
    most = 0.0
    for b, (n, m) in enumerate(zip(new, nk)):
        if n and (sequences is None or b in sequences):
            for h in heads:
                most = max(most, _check_rows(q[a : a + n, h], k[c : c + m, h * h_kv // h_q], v[c : c + m, h * h_kv // h_q], m - n,
                                             out[a : a + n, h]))
        a, c = a + n, c + m
    again = torch.zeros_like(out)
    tq.tq_prompt_attention(q, k, v, cu_q, cu_k, again)
    assert torch.equal(out, again) and tq.tq_device_errors() == 0
    print("share of the bound", most)


UNLIKE = [((1,), (2048,)), ((20,), (2100,)), ((300, 100), (170, 4000)), ((100, 700), (2177, 2305)), ((129, 257, 31), (2049, 2300, 2048))]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("new,nk", UNLIKE)
def test_two_tiles_of_unlike_lengths(new, nk, G, d, dtype):
    """Blocks of two tiles whose second has no rows, whose first sees no key, and that see different numbers of steps; keys that
    grow along the sequence, so that the running maximum moves again and again."""
    h_kv = _heads_for_two_tiles(new, G)
    _run(new, nk, G * h_kv, h_kv, d, dtype, sorted({0, h_kv * G // 2, h_kv * G - 1}), grow=(0.25, 8.0))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,G", [(128, 4), (64, 1), (128, 8)])
def test_two_tiles_and_special_values(d, G, dtype):
    """NaN and infinities of value rows in blocks of two tiles: only queries from their token on, in their channel."""
    n = 2300
    h_kv = _heads_for_two_tiles([n], G)
    g = torch.Generator(device=DEV).manual_seed(d + G)
    q = torch.randn(n, G * h_kv, d, generator=g, device=DEV).to(dtype)
    k, v = (torch.randn(n, h_kv, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    cu = _cu([n])
    clean, out = torch.zeros_like(q), torch.zeros_like(q)
    tq.tq_prompt_attention(q, k, v, cu, cu, clean)
    want = torch.ones(n, G * h_kv, d, dtype=torch.bool, device=DEV)
    for (t, h, c), x in {(n - 150, 0, 3): float("nan"), (n - 149, h_kv - 1, d - 1): float("inf"), (n - 64, 0, 17): float("-inf"),
                         (n - 1, h_kv // 2, 0): float("nan"), (200, 0, 5): float("nan")}.items():
        v[t, h, c] = x
        want[t:, h * G : h * G + G, c] = False
    tq.tq_prompt_attention(q, k, v, cu, cu, out)
    assert torch.equal(torch.isfinite(out), want)
    assert torch.equal(out[want], clean[want])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,h_q,h_kv", [(64, 4, 1), (128, 6, 2), (256, 2, 1)])
def test_a_hundred_thousand_keys(d, h_q, h_kv, dtype):
    """Few queries behind long histories: one tile a block."""
    _run((40, 1, 7), (100_003, 65_536, 131_072), h_q, h_kv, d, dtype, (0, h_q - 1))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
def test_a_hundred_thousand_keys_in_two_tiles(d, dtype):
    new = (200,)
    h_kv = _heads_for_two_tiles(new, 8)
    _run(new, (100_001,), 8 * h_kv, h_kv, d, dtype, (0, 8 * h_kv - 1))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B", [31, 32, 33, 1023, 1025])
@pytest.mark.parametrize("d", [64, 256])
def test_many_sequences(B, d, dtype):
    rng = np.random.default_rng(B)
    new = [int(x) for x in rng.integers(0, 40, B)]
    nk = [max(0, n + int(x)) for n, x in zip(new, rng.integers(-10, 90, B))]
    _run(new, nk, 4, 2, d, dtype, (0, 3), sequences={0, 1, 30, 31, 32, 33, B // 2, B - 2, B - 1})


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first", [False, True])
def test_one_long_prompt_among_short_ones(first, d, dtype):
    new = [16] * 15 + [3001]
    new = new[::-1] if first else new
    _run(new, new, 16, 4, d, dtype, (0, 15), sequences={0, 1, 14, 15})
