"""GPU parity of the paged 4-bit cache and of the prompt attention against the float64 oracle.

Stored bytes and gathered values are exact.  Attention tolerances, elementwise, from the roundings that the kernels make:
one rounding of the output to its type (eps / 2 of the value), one of each probability to the operand type (eps / 2 of
sum p |v| / l), and logits in float32 (d + 8 roundings of 2^-23 of sum |q k| scale, each of which moves every probability
by its relative size, twice: numerator and sum), with 2^-20 for the exponential's approximation.
"""

import numpy as np
import pytest
import torch

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


def _cu(n):
    return _i32(np.concatenate([[0], np.cumsum(n)]).tolist())


def _np(t):
    return t.double().cpu().numpy()


def _tables(rng, total, page, extra=2):
    need = [-(-max(n, 0) // page) for n in total]
    most = max(1, max(need))
    order = rng.permutation(sum(need) + extra)
    rows, at = np.zeros((len(need), most), np.int32), 0
    for b, n in enumerate(need):
        rows[b, :n] = order[at : at + n]
        at += n
    return rows, sum(need) + extra


def _tolerance(out, spread, biggest, d, dtype, p_dtype):
    logit = (d + 8) * 2.0 ** -23 * biggest + 2.0 ** -20
    return torch.finfo(dtype).eps / 2 * np.abs(out) + (torch.finfo(p_dtype).eps / 2 + 2 * logit) * spread + 1e-7


def _decode_tolerance(out, spread, largest, biggest, d, dtype):
    """_tolerance, with the roundings of the cached values' two terms in the place of the probabilities' own: p scale code and
    p zero are formed apart, of sizes that add up to at most spread + 2 max |v| (zero is a group's smallest value, scale code
    what lies above it).  bf16 outputs: p, p scale, and the sums of four p zero are fp16 (2^-11 each, at most five in a row).
    fp16 outputs: two fp16 parts each (2^-22), the same number of times, and additions that truncate (2^-23, sixteen a product
    and two products)."""
    r = 5 * 2.0 ** -11 if dtype == BF16 else 5 * 2.0 ** -22 + 32 * 2.0 ** -23
    return _tolerance(out, spread, biggest, d, dtype, F32) + r * (spread + 2 * largest)


class Setup:
    """A pool filled with a byte pattern, its oracle twin, and sequences of given total lengths."""

    def __init__(self, d, h_kv, page, total, seed=0, fill=0xFF):
        self.rng = np.random.default_rng(seed)
        self.table, self.pages = _tables(self.rng, total, page)
        self.spec = paged.PagedSpec(d, h_kv, page, self.pages)
        self.host = np.full(self.spec.nbytes(), fill, np.uint8)
        self.buffer = torch.from_numpy(self.host.copy()).to(DEV)
        self.cache = tq.PagedCache(d, h_kv, page, self.pages, buffer=self.buffer)
        self.batch = tq.PagedBatch(_i32(total), torch.from_numpy(self.table).to(DEV))
        self.total = list(total)

    def fill(self, scale_k=1.0, scale_v=1.0):
        """Random encoded tokens for every position, written by the oracle; returns per (b, h) (keys, values)."""
        d, h_kv = self.spec.d, self.spec.h_kv
        got = {}
        for b, n in enumerate(self.total):
            for h in range(h_kv):
                ch = np.exp(0.5 * self.rng.standard_normal((2, 1, d)))
                x = (self.rng.standard_normal((2, n, d)) * ch).astype(np.float32)
                key, val = paged.encode(x[0] * np.float32(scale_k)), paged.encode(x[1] * np.float32(scale_v))
                self.spec.write_sequence(self.host, self.table[b], h, 0, key, val)
                dq = [r["codes"] * r["scale16"].repeat(32, 1) + r["zero16"].repeat(32, 1) for r in (key, val)]
                got[b, h] = dq
        self.buffer.copy_(torch.from_numpy(self.host))
        return got


APPEND = [
    # d, h_q, h_kv, page, dtype, rotary, interleaved, new, past
    (128, 8, 2, 16, BF16, 128, False, (1, 1, 1), (0, 15, 16)),
    (128, 4, 1, 64, BF16, 128, True, (37, 0, 16, 1), (5, 9, 0, 63)),
    (64, 6, 3, 32, F16, 32, False, (33, 17), (0, 31)),
    (64, 2, 2, 16, F32, 16, True, (16, 48), (16, 8)),
    (256, 8, 1, 128, BF16, 64, False, (130, 3), (1, 126)),
    (256, 2, 2, 16, F32, 0, False, (20,), (12,)),
]


@pytest.mark.parametrize("d,h_q,h_kv,page,dtype,rotary,inter,new,past", APPEND)
@pytest.mark.parametrize("fused", [False, True])
def test_append_bytes_and_rows(d, h_q, h_kv, page, dtype, rotary, inter, new, past, fused):
    """Every byte of the pool (slots of other tokens untouched), and the rotated rows, exactly; rows behind the last
    sequence are left as they are."""
    total = [a + b for a, b in zip(new, past)]
    st = Setup(d, h_kv, page, total, seed=d + page, fill=0xA5)
    T, pad = sum(new), 3
    g = torch.Generator().manual_seed(d)
    x = torch.randn(T + pad, h_q + 2 * h_kv, d, generator=g)
    x[:, :, 1] *= 20
    x[0, -1] = 0.25  # a group of equal values: scale 0
    x = x.to(dtype)
    parts = x[:, :h_q], x[:, h_q : h_q + h_kv], x[:, h_q + h_kv :]
    qkv = x.to(DEV)
    q, k, v = qkv[:, :h_q], qkv[:, h_q : h_q + h_kv], qkv[:, h_q + h_kv :]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    table = tq.tq_make_rope_table(max(total) + 1, rotary, 10000.0) if rotary else None
    rope = tq.Rope(table.to(DEV), interleaved=inter) if rotary else None
    qo, ko = (torch.full((T + pad, h, d), 7.0, dtype=dtype, device=DEV) for h in (h_q, h_kv))
    tq.tq_paged_append(st.cache, st.batch, _cu(new), k, v, q=q, rope=rope, q_out=qo, k_out=ko)
    pos = np.concatenate([np.arange(b, a + b) for a, b in zip(new, past)]).astype(int)
    want = [paged.rotate(_np(p[:T]), table.numpy() if rotary else None, pos, inter) for p in parts[:2]]
    for got, w in zip((qo, ko), want):
        assert torch.equal(got[:T].cpu(), torch.from_numpy(w).float().to(dtype))
        assert (got[T:] == 7.0).all()
    at = 0
    for b, n in enumerate(new):
        for h in range(h_kv):
            st.spec.write_sequence(st.host, st.table[b], h, past[b], paged.encode(want[1][at : at + n, h]),
                                   paged.encode(_np(parts[2])[at : at + n, h])) if n else None
        at += n
    got = st.buffer.cpu().numpy()
    assert np.array_equal(got, st.host), np.nonzero(got != st.host)[0][:8]
    assert tq.tq_device_errors() == 0
    # in place: the rotated rows overwrite q and k
    if not fused:
        tq.tq_paged_append(st.cache, st.batch, _cu(new), k, v, q=q, rope=rope, q_out=q, k_out=k)
        assert torch.equal(q[:T], qo[:T]) and torch.equal(k[:T], ko[:T])
        assert np.array_equal(st.buffer.cpu().numpy(), st.host)


def test_append_ties_round_half_even_and_exactly():
    """Values on and next to the rounding boundaries of their group: codes as the float64 oracle's."""
    d, n = 128, 64
    st = Setup(d, 1, 64, [n], seed=3)
    rng = np.random.default_rng(9)
    scale = np.float16(2.0 ** rng.integers(-6, 3, (n, 4))).astype(np.float64)
    code = rng.integers(0, 30, (n, 4, 32)) * 0.5
    code[..., 0], code[..., 1] = 0, 15
    x = (code * scale[..., None]).reshape(n, d)
    x = x * (1 + rng.integers(-1, 2, x.shape) * 2.0 ** -23)  # on, just below and just above
    x = torch.from_numpy(x.astype(np.float32)).to(DEV).unsqueeze(1)
    tq.tq_paged_append(st.cache, st.batch, _cu([n]), x, x)
    rec = paged.encode(_np(x)[:, 0])
    st.spec.write_sequence(st.host, st.table[0], 0, 0, rec, rec)
    assert np.array_equal(st.buffer.cpu().numpy(), st.host)


@pytest.mark.parametrize("bad", [-1, 99, None])
def test_append_skips_bad_pages_and_positions(bad):
    """A page outside the pool, a length beyond the table's row and a position outside the rotation's table: the token is
    not stored, its rotated rows are NaN where it has no angle, and the device's error word says so."""
    d, page = 64, 16
    st = Setup(d, 1, page, [40, 20], seed=1, fill=0x11)
    if bad is not None:
        st.batch.block_table[0, 1] = bad
    else:
        st.batch.len_dev[0] = 40 + 16  # three pages hold 48
    x = torch.randn(60, 1, d, device=DEV)
    qo = torch.zeros_like(x)
    rope = tq.Rope(tq.tq_make_rope_table(30, 16).to(DEV))
    tq.tq_device_errors(clear=True)
    tq.tq_paged_append(st.cache, st.batch, _cu([40, 20]), x, x, q=x, rope=rope, q_out=qo)
    assert tq.tq_device_errors(clear=True) == tq.ERRF_PAGE | tq.ERRF_POSITION
    first = 0 if bad is not None else 16
    nan = torch.isnan(qo).any(-1).squeeze(1).cpu()
    want = torch.tensor([first + i >= 30 for i in range(40)] + [False] * 20)
    assert torch.equal(nan, want)
    xs = _np(x)[:, 0]
    rot = paged.rotate(_np(x), rope.table.cpu().numpy(), np.minimum(np.concatenate([np.arange(first, first + 40), np.arange(20)]), 29),
                       False)[:, 0]
    for b, (r0, n, f) in enumerate([(0, 40, first), (40, 20, 0)]):
        for i in range(n):
            pos = f + i
            if pos >= 30 or pos >= 48 or (b == 0 and bad is not None and pos // page == 1):
                continue
            st.spec.write_sequence(st.host, st.table[b], 0, pos, paged.encode(rot[r0 + i : r0 + i + 1]),
                                   paged.encode(xs[r0 + i : r0 + i + 1]))
    assert np.array_equal(st.buffer.cpu().numpy(), st.host)


@pytest.mark.parametrize("d,h_kv,page,dtype", [(64, 3, 16, F32), (128, 2, 64, BF16), (256, 1, 32, F16), (128, 1, 1024, F32)])
def test_gather_is_exact(d, h_kv, page, dtype):
    total = [50, 1, 33, 0]
    st = Setup(d, h_kv, page, total, seed=5)
    kv = st.fill()
    first, count = [3, 0, 16, 0], [47, 1, 9, 0]
    T, pad = sum(count), 2
    ko, vo = (torch.full((T + pad, 2 * h_kv, d), 5.0, dtype=dtype, device=DEV)[:, :h_kv] for _ in range(2))  # strided rows
    tq.tq_paged_gather(st.cache, st.batch, _cu(count), ko, vo, first=_i32(first))
    for got, i in ((ko, 0), (vo, 1)):
        want = np.concatenate([np.stack([kv[b, h][i][first[b] : first[b] + count[b]] for h in range(h_kv)], 1) for b in range(4)])
        assert torch.equal(got[:T].cpu(), torch.from_numpy(want).float().to(dtype))
        assert (got[T:] == 5.0).all()
    # rows behind a sequence's length and rows of a bad page
    tq.tq_device_errors(clear=True)
    st.batch.len_dev[0] = 20
    tq.tq_paged_gather(st.cache, st.batch, _cu(count), ko, vo, first=_i32(first))
    assert torch.isnan(ko[17:47]).all() and torch.isnan(vo[17:47]).all() and not torch.isnan(ko[:17]).any()
    st.batch.block_table[2, 16 // page] = -7
    tq.tq_paged_gather(st.cache, st.batch, _cu(count), ko, vo, first=_i32(first))
    assert torch.isnan(ko[48:57]).all() and not torch.isnan(ko[47:48]).any()
    assert tq.tq_device_errors(clear=True) == tq.ERRF_PAGE


def _check_decode(st, kv, q, out, scale, lens=None):
    dt = q.dtype
    d, G = q.shape[2], q.shape[1] // st.spec.h_kv
    qs, got = _np(q), _np(out)
    for b, n in enumerate(st.total if lens is None else lens):
        for hq in range(q.shape[1]):
            k, v = kv[b, hq // G]
            o, spread, big = paged.attend(qs[b, hq], k, v, n, scale)
            tol = _decode_tolerance(o, spread, np.abs(v[:n]).max() if n else 0.0, big, d, dt)
            assert (np.abs(got[b, hq] - o) <= tol).all(), (b, hq, np.abs(got[b, hq] - o).max())


DECODE = [
    # d, h_q, h_kv, page, dtype, lengths
    (128, 8, 2, 16, BF16, (1, 15, 16, 17, 0)),
    (128, 32, 8, 64, BF16, (257,)),
    (128, 12, 2, 64, F16, (100, 300, 31)),
    (128, 5, 5, 128, F16, (64, 129)),
    (64, 8, 1, 16, BF16, (333, 2, 48)),
    (64, 10, 2, 32, F16, (90, 0, 47)),
    (256, 7, 1, 16, BF16, (95, 16)),
    (256, 6, 3, 64, F16, (70, 150)),
]


@pytest.mark.parametrize("d,h_q,h_kv,page,dtype,total", DECODE)
def test_decode_parity(d, h_q, h_kv, page, dtype, total):
    st = Setup(d, h_kv, page, total, seed=d + h_q)  # slots behind a length hold NaN halves (0xFF)
    kv = st.fill()
    g = torch.Generator().manual_seed(1)
    q = (1.5 * torch.randn(len(total), h_q, d, generator=g)).to(dtype).to(DEV)
    out = torch.full_like(q, 9.0)
    ws = tq.paged_workspace_for(st.cache, st.batch, h_q)
    ws.fill_(0xFF)
    tq.tq_paged_decode_attention(st.cache, st.batch, q, out, ws)
    _check_decode(st, kv, q, out, d ** -0.5)
    for b, n in enumerate(total):
        if n == 0:
            assert not out[b].any()
    again = torch.zeros_like(out)
    tq.tq_paged_decode_attention(st.cache, st.batch, q, again, ws)
    assert torch.equal(out, again)  # no order of arrival in the result
    assert tq.tq_device_errors() == 0


@pytest.mark.parametrize("scale_k,scale_v,softmax", [(1e-3, 1e-3, None), (30.0, 300.0, None), (1.0, 1e-6, 0.5), (8.0, 1.0, -0.3),
                                                     (1.0, 1.0, 0.0)])
def test_decode_ranges(scale_k, scale_v, softmax):
    """Small and large keys and values, sharp, flat and negative softmax scales."""
    st = Setup(128, 2, 32, (77, 200), seed=11)
    kv = st.fill(scale_k, scale_v)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(2, 8, 128, generator=g).to(BF16).to(DEV)
    out = torch.zeros_like(q)
    tq.tq_paged_decode_attention(st.cache, st.batch, q, out, tq.paged_workspace_for(st.cache, st.batch, 8), softmax_scale=softmax)
    _check_decode(st, kv, q, out, 128 ** -0.5 if softmax is None else softmax)


@pytest.mark.parametrize("d,h_q,h_kv,dtype", [(64, 4, 4, F16), (128, 8, 4, BF16), (256, 4, 2, BF16)])
@pytest.mark.parametrize("spread", [False, True])
def test_decode_more_units_than_ranges(d, h_q, h_kv, dtype, spread):
    """More (sequence, KV head) units than blocks: few, many or no steps in a unit, one that spans many blocks, empty
    sequences at both ends."""
    rng = np.random.default_rng(3)
    total = [0, 0, 1] + [int(x) for x in rng.integers(0, 40 if spread else 400, 290)] + [4000 if spread else 700, 0, 33, 0]
    table, pages = _tables(rng, total, 32)
    cache = tq.PagedCache(d, h_kv, 32, pages)
    batch = tq.PagedBatch(_i32(total), torch.from_numpy(table).to(DEV))
    g = torch.Generator(device=DEV).manual_seed(0)
    k, v = (torch.randn(sum(total), h_kv, d, generator=g, device=DEV) for _ in range(2))
    tq.tq_paged_append(cache, batch, _cu(total), k, v)
    kc, vc = torch.zeros_like(k), torch.zeros_like(v)
    tq.tq_paged_gather(cache, batch, _cu(total), kc, vc)
    q = torch.randn(len(total), h_q, d, generator=g, device=DEV).to(dtype)
    out = torch.full_like(q, 7.0)
    ws = tq.paged_workspace_for(cache, batch, h_q)
    ws.fill_(0xFF)
    tq.tq_paged_decode_attention(cache, batch, q, out, ws)
    at = 0
    for b, n in enumerate(total):
        if n == 0:
            assert not out[b].any()
            continue
        kb, vb = (x[at : at + n].double().transpose(0, 1) for x in (kc, vc))
        w = torch.softmax(q[b].double().view(h_kv, -1, d) @ kb.transpose(1, 2) * d ** -0.5, -1)
        o, size = w @ vb, w @ vb.abs()
        big = float((q[b].double().abs().view(h_kv, -1, d) @ kb.abs().transpose(1, 2)).max() * d ** -0.5)
        tol = _decode_tolerance(_np(o), _np(size), float(vb.abs().max()), big, d, dtype)
        assert (np.abs(_np(out[b].view(h_kv, -1, d)) - _np(o)) <= tol).all(), b
        at += n
    again = torch.zeros_like(out)
    tq.tq_paged_decode_attention(cache, batch, q, again, ws)
    assert torch.equal(out, again)
    assert tq.tq_device_errors() == 0


def test_decode_long_and_ragged():
    """Many splits: one long sequence among short ones, against float64 on the device."""
    total = (20000, 1, 700, 16, 5003)
    d, h_q, h_kv, page = 128, 16, 4, 64
    rng = np.random.default_rng(0)
    table, pages = _tables(rng, total, page)
    cache = tq.PagedCache(d, h_kv, page, pages)
    batch = tq.PagedBatch(_i32(total), torch.from_numpy(table).to(DEV))
    g = torch.Generator(device=DEV).manual_seed(0)
    T = sum(total)
    k, v = (torch.randn(T, h_kv, d, generator=g, device=DEV) for _ in range(2))
    tq.tq_paged_append(cache, batch, _cu(total), k, v)
    kc, vc = torch.zeros_like(k), torch.zeros_like(v)
    tq.tq_paged_gather(cache, batch, _cu(total), kc, vc)
    q = torch.randn(len(total), h_q, d, generator=g, device=DEV).to(F16)
    out = torch.zeros_like(q)
    tq.tq_paged_decode_attention(cache, batch, q, out, tq.paged_workspace_for(cache, batch, h_q))
    at = 0
    for b, n in enumerate(total):
        kb, vb = (x[at : at + n].double().transpose(0, 1) for x in (kc, vc))
        s = q[b].double().view(h_kv, -1, d) @ kb.transpose(1, 2) * d ** -0.5
        w = torch.softmax(s, -1)
        o, spread = w @ vb, w @ vb.abs()
        big = float((q[b].double().abs().view(h_kv, -1, d) @ kb.abs().transpose(1, 2)).max() * d ** -0.5)
        tol = _decode_tolerance(_np(o), _np(spread), float(vb.abs().max()), big, d, F16)
        assert (np.abs(_np(out[b].view(h_kv, -1, d)) - _np(o)) <= tol).all()
        at += n


def test_decode_bad_page_is_nan_and_flagged():
    st = Setup(64, 2, 16, (40, 33, 20), seed=2)
    kv = st.fill()
    st.batch.block_table[0, 2] = 1 << 20
    st.batch.len_dev[2] = 49  # the table's rows hold 48 positions
    q = torch.randn(3, 4, 64, device=DEV).to(BF16)
    out = torch.zeros_like(q)
    tq.tq_device_errors(clear=True)
    tq.tq_paged_decode_attention(st.cache, st.batch, q, out, tq.paged_workspace_for(st.cache, st.batch, 4))
    assert torch.isnan(out[0]).all() and torch.isnan(out[2]).all() and not torch.isnan(out[1]).any()
    assert tq.tq_device_errors(clear=True) == tq.ERRF_PAGE
    o, _, _ = paged.attend(_np(q)[1, 3], *kv[1, 1], 33, 64 ** -0.5)
    assert np.abs(_np(out)[1, 3] - o).max() < 0.05


def test_pool_beyond_four_gigabytes():
    """Pages whose byte offsets do not fit 32 bits."""
    d, h_kv, page = 128, 8, 128
    per = tq.tq_paged_bytes(d, h_kv, page, 1)
    pages = (5 << 30) // per
    cache = tq.PagedCache(d, h_kv, page, pages)
    n = 200
    batch = tq.PagedBatch(_i32([n]), _i32([[pages - 1, pages - 2]]))
    g = torch.Generator(device=DEV).manual_seed(0)
    k, v = (torch.randn(n, h_kv, d, generator=g, device=DEV) for _ in range(2))
    tq.tq_paged_append(cache, batch, _cu([n]), k, v)
    kc, vc = torch.zeros_like(k), torch.zeros_like(v)
    tq.tq_paged_gather(cache, batch, _cu([n]), kc, vc)
    for x, y in ((k, kc), (v, vc)):
        rec = paged.encode(_np(x).reshape(-1, d))
        want = rec["codes"] * rec["scale16"].repeat(32, 1) + rec["zero16"].repeat(32, 1)
        assert np.array_equal(_np(y).reshape(-1, d), want.astype(np.float32))
    q = torch.randn(1, 16, d, generator=g, device=DEV).to(BF16)
    out = torch.zeros_like(q)
    tq.tq_paged_decode_attention(cache, batch, q, out, tq.paged_workspace_for(cache, batch, 16))
    for hq in range(16):
        o, spread, big = paged.attend(_np(q)[0, hq], _np(kc)[:, hq // 2], _np(vc)[:, hq // 2], n, d ** -0.5)
        tol = _decode_tolerance(o, spread, np.abs(_np(vc)[:, hq // 2]).max(), big, d, BF16)
        assert (np.abs(_np(out)[0, hq] - o) <= tol).all()


PROMPT = [
    # d, h_q, h_kv, dtype, queries, history
    (128, 8, 2, BF16, (1, 130, 257, 64), (0, 0, 0, 0)),
    (128, 6, 1, F16, (300, 3), (0, 200)),
    (128, 5, 1, BF16, (129, 0, 31), (128, 7, 1)),
    (128, 2, 2, F16, (511,), (0,)),
    (64, 8, 1, BF16, (140, 129), (17, 0)),
    (64, 7, 1, F16, (90, 1, 1, 260), (0, 0, 300, 0)),
    (256, 4, 2, BF16, (70, 200), (0, 33)),
    (256, 3, 3, F16, (129, 64), (0, 0)),
]


def _prompt_inputs(d, h_q, h_kv, dtype, nq, nk, seed=0, pad=5):
    g = torch.Generator().manual_seed(seed)
    q = (1.5 * torch.randn(sum(nq) + pad, h_q, d, generator=g)).to(dtype)
    k = torch.randn(sum(nk) + pad, h_kv, d, generator=g).to(dtype)
    v = torch.randn(sum(nk) + pad, h_kv, d, generator=g).to(dtype)
    k[sum(nk):], v[sum(nk):] = float("nan"), float("inf")  # behind the last sequence
    return q, k, v


def _check_prompt(q, k, v, nq, nk, out, scale, rows=None):
    d, G, dt = q.shape[2], q.shape[1] // k.shape[1], q.dtype
    qs, ks, vs, got = _np(q), _np(k), _np(v), _np(out)
    a = c = 0
    for n, m in zip(nq, nk):
        for i in range(n):
            if rows is not None and i not in rows(n):
                continue
            for hq in range(q.shape[1]):
                o, spread, big = paged.attend(qs[a + i, hq], ks[c : c + m, hq // G], vs[c : c + m, hq // G], min(m, i + 1 + m - n), scale)
                tol = _tolerance(o, spread, big, d, dt, dt)
                assert (np.abs(got[a + i, hq] - o) <= tol).all(), (n, m, i, hq, np.abs(got[a + i, hq] - o).max())
        a, c = a + n, c + m


@pytest.mark.parametrize("d,h_q,h_kv,dtype,new,past", PROMPT)
@pytest.mark.parametrize("fused", [False, True])
def test_prompt_parity(d, h_q, h_kv, dtype, new, past, fused):
    nk = [a + b for a, b in zip(new, past)]
    q, k, v = _prompt_inputs(d, h_q, h_kv, dtype, new, nk)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    if fused:  # keys and values as parts of wider rows
        kv = torch.cat([kd, vd], 1)
        kd, vd = kv[:, :h_kv], kv[:, h_kv:]
    out = torch.full((q.shape[0], 2 * h_q, d), 3.0, dtype=dtype, device=DEV)[:, :h_q] if fused else torch.full_like(qd, 3.0)
    tq.tq_prompt_attention(qd, kd, vd, _cu(new), _cu(nk), out)
    T = sum(new)
    assert (out[T:] == 3.0).all()
    few = (lambda n: set(range(0, n, 13)) | {n - 1, n - 2, 1, 31, 32, 127, 128}) if T > 40 else None
    _check_prompt(q, k, v, new, nk, out, d ** -0.5, few)
    again = torch.zeros_like(qd)
    tq.tq_prompt_attention(qd, kd, vd, _cu(new), _cu(nk), again)
    assert torch.equal(again[:T], out[:T])
    assert tq.tq_device_errors() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_keyless_queries_and_empty_sequences(d):
    """Fewer keys than queries: the first queries see nothing and get zeros; no keys at all: zeros throughout."""
    new, nk = (200, 0, 5, 150), (50, 3, 0, 149)
    q, k, v = _prompt_inputs(d, 4, 2, BF16, new, nk, seed=4)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    out = torch.full_like(qd, 3.0)
    tq.tq_prompt_attention(qd, kd, vd, _cu(new), _cu(nk), out)
    assert not out[:150].any() and out[150:200].any(-1).all() and not out[200:205].any() and not out[205].any()
    assert (out[355:] == 3.0).all()
    _check_prompt(q, k, v, new, nk, out, d ** -0.5, lambda n: {0, n - 1, n - 50, n - 49, 1, 2})
    none = torch.zeros(0, 2, d, dtype=BF16, device=DEV)
    out.fill_(3.0)
    tq.tq_prompt_attention(qd, none, none, _cu(new), _i32([0] * 5), out)
    assert not out[:355].any() and (out[355:] == 3.0).all()


@pytest.mark.parametrize("d,h_q,h_kv", [(128, 8, 2), (64, 4, 4), (256, 2, 1)])
@pytest.mark.parametrize("softmax", [0.0, 2.0, -0.2])
def test_prompt_scales_and_infinite_neighbours(d, h_q, h_kv, softmax):
    """Flat, sharp and negative softmax scales; a neighbouring sequence of infinities and NaN reaches no result, and a
    masked key's infinities in the key row reach none either."""
    new = (60, 100, 40)
    q, k, v = _prompt_inputs(d, h_q, h_kv, F16, new, new, seed=6)
    k[60:160], v[60:160] = float("inf"), float("nan")
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    out = torch.zeros_like(qd)
    tq.tq_prompt_attention(qd, kd, vd, _cu(new), _cu(new), out, softmax_scale=softmax)
    for a, n in ((0, 60), (160, 40)):
        _check_prompt(q[a : a + n], k[a : a + n], v[a : a + n], [n], [n], out[a : a + n], softmax)
    k, v = torch.randn_like(k), torch.randn_like(v)
    k[59] = float("nan")
    tq.tq_prompt_attention(qd, k.to(DEV), v.to(DEV), _cu(new), _cu(new), out, softmax_scale=softmax)
    k[59] = 0
    _check_prompt(q[:59], k[:59], v[:59], [59], [59], out[:59], softmax)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,h_q,h_kv", [(128, 8, 2), (64, 3, 3), (256, 6, 1), (128, 4, 4)])
@pytest.mark.parametrize("long", [False, True])
def test_prompt_special_values_reach_only_who_sees_them(d, h_q, h_kv, dtype, long):
    """A NaN or an infinity in one channel of a value row: NaN or that infinity for the queries from its token on, in that
    channel alone; a NaN key row: NaN for those queries; nothing for earlier ones."""
    n = 2300 if long else 210  # one tile a block, and two
    q, k, v = _prompt_inputs(d, h_q, h_kv, dtype, [n], [n], seed=8, pad=0)
    cu = _cu([n])
    clean = torch.zeros_like(q, device=DEV)
    tq.tq_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), cu, cu, clean)
    hit = {n - 150: 3, n - 149: d - 1, n - 64: 17, n - 1: 0}
    bad = v.clone()
    for (t, c), x in zip(hit.items(), (float("nan"), float("inf"), float("-inf"), float("nan"))):
        bad[t, 0, c] = x
    out = torch.zeros_like(clean)
    tq.tq_prompt_attention(q.to(DEV), k.to(DEV), bad.to(DEV), cu, cu, out)
    want = torch.ones(n, h_q, d, dtype=torch.bool, device=DEV)
    for t, c in hit.items():
        want[t:, : h_q // h_kv, c] = False
    assert torch.equal(torch.isfinite(out), want)
    assert torch.equal(out[want], clean[want])
    bad = k.clone()
    bad[n - 70, 0, 5] = float("nan")
    tq.tq_prompt_attention(q.to(DEV), bad.to(DEV), v.to(DEV), cu, cu, out)
    want[:] = True
    want[n - 70 :, : h_q // h_kv] = False
    assert torch.equal(torch.isfinite(out), want)
    assert torch.equal(out[want], clean[want])


def _check_on_device(q, k, v, new, nk, out):
    h_q, h_kv, d, dt = q.shape[1], k.shape[1], q.shape[2], q.dtype
    a = c = 0
    for n, m in zip(new, nk):
        i, j = torch.arange(n, device=DEV)[:, None], torch.arange(m, device=DEV)
        seen = (i[:, 0] + m - n >= 0).cpu().numpy()
        for hq in range(h_q):
            kk, vv = (x[c : c + m, hq * h_kv // h_q].double() for x in (k, v))
            s = q[a : a + n, hq].double() @ kk.T * d ** -0.5
            w = torch.softmax(s.masked_fill(j > i + m - n, -torch.inf), -1)
            big = float((q[a : a + n, hq].double().abs() @ kk.abs().T).max() * d ** -0.5)
            o, got = _np(w @ vv), _np(out[a : a + n, hq])
            tol = _tolerance(o, _np(w @ vv.abs()), big, d, dt, dt)
            assert (np.abs(got - o) <= tol)[seen].all(), (n, m, hq)
            assert not got[~seen].any()
        a, c = a + n, c + m


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", [(2, 2), (8, 1)])
@pytest.mark.parametrize("new,nk", [((1,), (2048,)), ((20,), (2100,)), ((300, 100), (170, 4000)), ((100, 700), (2177, 2305)),
                                    ((129, 257, 31), (2049, 2300, 2048))])
def test_prompt_two_tiles_of_unlike_lengths(d, h_q, h_kv, new, nk):
    """Blocks of two tiles whose second has no rows, whose first sees no key, and that see different numbers of steps; keys
    that grow along the sequence, so that the running maximum moves again and again."""
    g = torch.Generator(device=DEV).manual_seed(d + h_q)
    for dt in (BF16, F16):
        q = torch.randn(sum(new), h_q, d, generator=g, device=DEV).to(dt)
        grow = torch.cat([torch.linspace(0.25, 8.0, m, device=DEV) for m in nk])[:, None, None]
        k = (torch.randn(sum(nk), h_kv, d, generator=g, device=DEV) * grow).to(dt)
        v = torch.randn(sum(nk), h_kv, d, generator=g, device=DEV).to(dt)
        out = torch.full_like(q, 3.0)
        tq.tq_prompt_attention(q, k, v, _cu(new), _cu(nk), out)
        _check_on_device(q, k, v, new, nk, out)
        again = torch.zeros_like(q)
        tq.tq_prompt_attention(q, k, v, _cu(new), _cu(nk), again)
        assert torch.equal(out, again)
    assert tq.tq_device_errors() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("new,nk", [((1,), (2048,)), ((20,), (2100,)), ((300, 100), (170, 4000)), ((100, 700), (2177, 2305)),
                                    ((129, 257, 31), (2049, 2300, 2048))])
def test_prompt_two_tiles_with_many_heads(d, G, new, nk):
    """The same with more tiles than two an SM, which blocks of two tiles take; a few of the heads are looked at."""
    tiles = sum(new) // (128 // G) + len(new)
    h_kv = 300 // tiles + 2
    g = torch.Generator(device=DEV).manual_seed(d + G)
    dt = BF16 if G == 1 else F16
    q = torch.randn(sum(new), h_kv * G, d, generator=g, device=DEV).to(dt)
    grow = torch.cat([torch.linspace(0.25, 8.0, m, device=DEV) for m in nk])[:, None, None]
    k = (torch.randn(sum(nk), h_kv, d, generator=g, device=DEV) * grow).to(dt)
    v = torch.randn(sum(nk), h_kv, d, generator=g, device=DEV).to(dt)
    out = torch.full_like(q, 3.0)
    tq.tq_prompt_attention(q, k, v, _cu(new), _cu(nk), out)
    for h in (0, h_kv // 2, h_kv - 1):
        _check_on_device(q[:, h * G : h * G + G], k[:, h : h + 1], v[:, h : h + 1], new, nk, out[:, h * G : h * G + G])
    again = torch.zeros_like(q)
    tq.tq_prompt_attention(q, k, v, _cu(new), _cu(nk), again)
    assert torch.equal(out, again)
    assert tq.tq_device_errors() == 0


@pytest.mark.parametrize("d,h_q,h_kv", [(128, 20, 5), (64, 18, 18)])
def test_prompt_special_values_with_many_heads(d, h_q, h_kv):
    test_prompt_special_values_reach_only_who_sees_them(d, h_q, h_kv, BF16, True)


def test_prompt_long_against_float64_on_device():
    d, h_q, h_kv, new, past = 128, 8, 2, (2000, 3, 1111), (0, 3000, 517)
    nk = [a + b for a, b in zip(new, past)]
    g = torch.Generator(device=DEV).manual_seed(0)
    for dt in (BF16, F16):
        q = (1.5 * torch.randn(sum(new), h_q, d, generator=g, device=DEV)).to(dt)
        k, v = (torch.randn(sum(nk), h_kv, d, generator=g, device=DEV).to(dt) for _ in range(2))
        out = torch.zeros_like(q)
        tq.tq_prompt_attention(q, k, v, _cu(new), _cu(nk), out)
        a = c = 0
        for n, m in zip(new, nk):
            i, j = torch.arange(n, device=DEV)[:, None], torch.arange(m, device=DEV)
            for hq in range(h_q):
                kk, vv = (x[c : c + m, hq * h_kv // h_q].double() for x in (k, v))
                s = q[a : a + n, hq].double() @ kk.T * d ** -0.5
                w = torch.softmax(s.masked_fill(j > i + m - n, -torch.inf), -1)
                big = float((q[a : a + n, hq].double().abs() @ kk.abs().T).max() * d ** -0.5)
                o = _np(w @ vv)
                tol = _tolerance(o, _np(w @ vv.abs()), big, d, dt, dt)
                assert (np.abs(_np(out[a : a + n, hq]) - o) <= tol).all()
            a, c = a + n, c + m


def _chain(d, h_q, h_kv, dtype, page, prompts, steps, stream=None):
    """Prompts appended and attended, the second half as a chunk behind gathered history, then decode steps; returns the
    outputs and what the oracle needs to check them."""
    B = len(prompts)
    rng = np.random.default_rng(0)
    table, pages = _tables(rng, [n + steps for n in prompts], page)
    cache = tq.PagedCache(d, h_kv, page, pages)
    cache.buffer.fill_(0xFF)
    len_dev = _i32([0] * B)
    batch = tq.PagedBatch(len_dev, torch.from_numpy(table).to(DEV))
    rope = tq.Rope(tq.tq_make_rope_table(max(prompts) + steps, d, 10000.0).to(DEV))
    g = torch.Generator().manual_seed(3)
    parts = [[n // 2 for n in prompts], [n - n // 2 for n in prompts]]
    log, done = [], [0] * B
    for n in parts:
        T = sum(n)
        qkv = torch.randn(T, h_q + 2 * h_kv, d, generator=g).to(dtype).to(DEV)
        q, k, v = qkv[:, :h_q], qkv[:, h_q : h_q + h_kv], qkv[:, h_q + h_kv :]
        total = [a + b for a, b in zip(done, n)]
        len_dev.copy_(_i32(total))
        qo = torch.empty(T, h_q, d, dtype=dtype, device=DEV)
        tq.tq_paged_append(cache, batch, _cu(n), k, v, q=q, rope=rope, q_out=qo)
        kc, vc = (torch.empty(sum(total), h_kv, d, dtype=dtype, device=DEV) for _ in range(2))
        tq.tq_paged_gather(cache, batch, _cu(total), kc, vc)
        out = torch.empty_like(qo)
        tq.tq_prompt_attention(qo, kc, vc, _cu(n), _cu(total), out)
        log.append(("prompt", n, total, qo, kc, vc, out))
        done = total
    ws = tq.paged_workspace_for(cache, batch, h_q)
    for _ in range(steps):
        qkv = torch.randn(B, h_q + 2 * h_kv, d, generator=g).to(dtype).to(DEV)
        len_dev.add_(1)
        done = [x + 1 for x in done]
        qo = torch.empty(B, h_q, d, dtype=dtype, device=DEV)
        tq.tq_paged_append(cache, batch, _i32(list(range(B + 1))), qkv[:, h_q : h_q + h_kv], qkv[:, h_q + h_kv :], q=qkv[:, :h_q],
                           rope=rope, q_out=qo)
        out = torch.empty_like(qo)
        tq.tq_paged_decode_attention(cache, batch, qo, out, ws)
        kc, vc = (torch.empty(sum(done), h_kv, d, device=DEV) for _ in range(2))
        tq.tq_paged_gather(cache, batch, _cu(done), kc, vc)
        log.append(("decode", [1] * B, list(done), qo, kc, vc, out))
    return log


@pytest.mark.parametrize("d,h_q,h_kv,dtype,page", [(128, 8, 2, BF16, 16), (64, 6, 1, F16, 64), (256, 2, 2, BF16, 32)])
def test_a_serving_run(d, h_q, h_kv, dtype, page):
    """Append, gather, prompt attention in two chunks, then decode steps: each against the oracle on the cached values."""
    for kind, n, total, q, k, v, out in _chain(d, h_q, h_kv, dtype, page, [45, 2, 130], 3):
        if kind == "prompt":
            _check_prompt(q, k, v, n, total, out, d ** -0.5, lambda m: {0, m // 2, m - 1})
        else:
            at = 0
            for b, m in enumerate(total):
                for hq in range(h_q):
                    kk, vv = _np(k)[at : at + m, hq * h_kv // h_q], _np(v)[at : at + m, hq * h_kv // h_q]
                    o, spread, big = paged.attend(_np(q)[b, hq], kk, vv, m, d ** -0.5)
                    tol = _decode_tolerance(o, spread, np.abs(vv).max(), big, d, dtype)
                    assert (np.abs(_np(out)[b, hq] - o) <= tol).all()
                at += m


def test_captured_steps_follow_the_batch():
    """Two decode steps captured into graphs with workspaces of their own and replayed as the lengths grow, on a side stream:
    the same outputs as eager calls."""
    d, h_q, h_kv, page, B, steps = 128, 8, 2, 16, 3, 20
    g = torch.Generator(device=DEV).manual_seed(0)
    rng = np.random.default_rng(0)
    table, pages = _tables(rng, [40 + steps] * B, page)
    x = torch.randn(steps, B, h_q + 2 * h_kv, d, generator=g, device=DEV).to(BF16)
    rope = tq.Rope(tq.tq_make_rope_table(64, d).to(DEV))
    cu = _i32(list(range(B + 1)))

    def world():
        cache = tq.PagedCache(d, h_kv, page, pages)
        cache.buffer.zero_()
        batch = tq.PagedBatch(_i32([1, 14, 39]), torch.from_numpy(table).to(DEV))
        return cache, batch, tq.paged_workspace_for(cache, batch, h_q)

    def step(w, qkv, qo, out):
        w[1].len_dev.add_(1)
        tq.tq_paged_append(w[0], w[1], cu, qkv[:, h_q : h_q + h_kv], qkv[:, h_q + h_kv :], q=qkv[:, :h_q], rope=rope, q_out=qo)
        tq.tq_paged_decode_attention(w[0], w[1], qo, out, w[2])

    w, want = world(), []
    qo, out = (torch.empty(B, h_q, d, dtype=BF16, device=DEV) for _ in range(2))
    for i in range(steps):
        step(w, x[i], qo, out)
        want.append(out.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    worlds = [world(), world()]
    io = [[torch.empty(B, h_q + 2 * h_kv, d, dtype=BF16, device=DEV)] + [torch.empty(B, h_q, d, dtype=BF16, device=DEV) for _ in range(2)]
          for _ in worlds]
    lens = [u[1].len_dev.clone() for u in worlds]
    graphs = [torch.cuda.CUDAGraph() for _ in worlds]
    torch.cuda.synchronize()
    for u, t, gr in zip(worlds, io, graphs):
        with torch.cuda.graph(gr, stream=side):
            step(u, *t)
    for u, n in zip(worlds, lens):
        u[1].len_dev.copy_(n)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for i in range(steps):  # the two graphs run side by side
        for t, gr, s in zip(io, graphs, (side, other)):
            with torch.cuda.stream(s):
                t[0].copy_(x[i])
                gr.replay()
        torch.cuda.synchronize()
        for t in io:
            assert torch.equal(t[2], want[i])


def test_bounded_waits_give_up():
    """With the copies withheld and the wait limit at 2 ms every call returns: NaN rows and the device's error word (append:
    the pages stay as they were), and the next calls are right."""
    st = Setup(128, 2, 64, (100, 300), seed=3)
    kv = st.fill()
    q = torch.randn(2, 8, 128, device=DEV).to(BF16)
    out = torch.zeros_like(q)
    ws = tq.paged_workspace_for(st.cache, st.batch, 8)
    x = torch.randn(200, 2, 128, device=DEV).to(BF16)
    po = torch.zeros_like(x)
    cu = _cu([50, 150])
    tq.tq_device_errors(clear=True)
    try:
        tq.tq_set_wait_limit_ns(2_000_000)
        tq.tq_test_withhold_handoffs(True)
        tq.tq_paged_decode_attention(st.cache, st.batch, q, out, ws)
        assert tq.tq_device_errors(clear=True) == tq.ERRF_DECODE_WAIT
        tq.tq_prompt_attention(x, x, x, cu, cu, po)
        assert tq.tq_device_errors(clear=True) == tq.ERRF_PROMPT_WAIT
        tq.tq_paged_append(st.cache, st.batch, cu, x, x)
        assert tq.tq_device_errors(clear=True) == tq.ERRF_QUANTIZE_WAIT
    finally:
        tq.tq_test_withhold_handoffs(False)
        tq.tq_set_wait_limit_ns(0)
    assert torch.isnan(out).all() and torch.isnan(po).all()
    assert np.array_equal(st.buffer.cpu().numpy(), st.host)
    tq.tq_paged_decode_attention(st.cache, st.batch, q, out, ws)
    _check_decode(st, kv, q, out, 128 ** -0.5)
    tq.tq_prompt_attention(x, x, x, cu, cu, po)
    _check_prompt(x, x, x, [50, 150], [50, 150], po, 128 ** -0.5, lambda n: {0, n - 1})
    assert tq.tq_device_errors() == 0


def test_another_stream_and_lengths_out_of_range():
    """Calls on a side stream (inputs made on it), and lengths and first positions at the ends of 32 bits: nothing is
    dereferenced, rows are NaN, zero or left as the lengths say."""
    st = Setup(64, 1, 16, (20, 33), seed=4, fill=0x33)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.randn(53, 1, 64, device=DEV)
        tq.tq_paged_append(st.cache, st.batch, _cu([20, 33]), x, x)
        k, v = torch.zeros_like(x), torch.zeros_like(x)
        tq.tq_paged_gather(st.cache, st.batch, _cu([20, 33]), k, v)
    side.synchronize()
    rec = paged.encode(_np(x)[:, 0])
    want = (rec["codes"] * rec["scale16"].repeat(32, 1) + rec["zero16"].repeat(32, 1)).astype(np.float32)
    assert np.array_equal(k[:, 0].cpu().numpy(), want) and torch.equal(k, v)
    before = st.buffer.clone()
    q = torch.randn(2, 4, 64, device=DEV).to(BF16)
    out = torch.zeros_like(q)
    ws = tq.paged_workspace_for(st.cache, st.batch, 4)
    tq.tq_device_errors(clear=True)
    for lens in ([2 ** 31 - 1, -2 ** 31], [-5, 2 ** 30 + 7]):
        st.batch.len_dev.copy_(_i32(lens))
        tq.tq_paged_append(st.cache, st.batch, _cu([20, 33]), x, x)
        assert torch.equal(st.buffer, before)
        assert tq.tq_device_errors(clear=True) == tq.ERRF_PAGE
        tq.tq_paged_decode_attention(st.cache, st.batch, q, out, ws)
        for b, n in enumerate(lens):
            assert torch.isnan(out[b]).all() if n > 0 else not out[b].any()
        tq.tq_device_errors(clear=True)
    st.batch.len_dev.copy_(_i32([20, 33]))
    for first in ([2 ** 31 - 1, -2 ** 31], [17, 40]):
        k.fill_(1.0)
        tq.tq_paged_gather(st.cache, st.batch, _cu([20, 33]), k, v, first=_i32(first))
        if first[0] == 17:
            assert torch.equal(k[:3, 0].cpu(), torch.from_numpy(want[17:20])) and torch.isnan(k[3:]).all()
        else:
            assert torch.isnan(k).all()
    assert tq.tq_device_errors(clear=True) == tq.ERRF_PAGE


@pytest.mark.parametrize("start", [0, 40])
def test_rows_before_the_first_sequence_and_repeated_boundaries(start):
    """Row arrays whose first entry is not 0: the rows before it belong to nobody and are left as they are."""
    st = Setup(64, 1, 16, (9, 0, 0, 30), seed=5, fill=0)
    T = start + 39 + 4
    cu = _i32([start, start + 9, start + 9, start + 9, start + 39])
    x = torch.randn(T, 1, 64, device=DEV).to(BF16)
    ko = torch.full_like(x, 2.0)
    tq.tq_paged_append(st.cache, st.batch, cu, x, x, k_out=ko)
    k, v, o = (torch.full_like(x, 2.0) for _ in range(3))
    tq.tq_paged_gather(st.cache, st.batch, cu, k, v)
    tq.tq_prompt_attention(x, x, x, cu, cu, o)
    assert torch.equal(ko[start : start + 39], x[start : start + 39])
    for y in (ko, k, v, o):
        assert (y[:start] == 2.0).all() and (y[start + 39 :] == 2.0).all()
    rec = paged.encode(_np(x)[start : start + 39, 0])
    want = torch.from_numpy(rec["codes"] * rec["scale16"].repeat(32, 1) + rec["zero16"].repeat(32, 1)).float().to(BF16)
    assert torch.equal(k[start : start + 39, 0].cpu(), want)
    y = x[start:]
    _check_prompt(y, y, y, [9, 0, 0, 30], [9, 0, 0, 30], o[start:], 64 ** -0.5)
