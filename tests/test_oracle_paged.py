"""Pins of the paged oracle: the layout against hand-computed bytes, the codec's bounds, the rotation and the attention
against independent forms."""

import numpy as np
import pytest

from kv_cache_quantization_turboquantprod_b200 import tq
from oracle import paged


@pytest.mark.parametrize("d", [64, 128, 256])
def test_every_byte_of_a_cell_has_one_owner(d):
    spec = paged.PagedSpec(d, 2, 32, 3)
    seen = np.zeros(2 * spec.cell_bytes, np.int64)  # nibbles
    for at in (spec.key_byte, spec.val_byte):
        np.add.at(seen, (2 * at + spec.shift // 4).ravel(), 1)
    for at in (spec.key_scale, spec.key_zero, spec.val_scale, spec.val_zero):
        for k in range(4):
            np.add.at(seen, (2 * at + k).ravel(), 1)
    assert (seen == 1).all()
    assert tq.tq_paged_bytes(d, 2, 32, 3) == spec.nbytes() == 3 * 2 * 2 * 20 * d


def test_hand_placed_bytes():
    spec = paged.PagedSpec(128, 3, 64, 4)
    buf = np.zeros(spec.nbytes(), np.uint8)
    blank = lambda: {"codes": np.zeros((1, 128), np.int64), "scale16": np.zeros((1, 4)), "zero16": np.zeros((1, 4))}  # noqa: E731
    key, val = blank(), blank()
    key["codes"][0, 77] = 9    # group 2, channel 13 of it: word u = 1, nibble 5
    val["codes"][0, 77] = 6    # quad g = 3, nibble 1
    key["scale16"][0, 3] = 1.0  # 0x3C00
    key["zero16"][0, 1] = -2.0  # 0xC000
    val["scale16"][0, 0] = 0.5  # 0x3800
    val["zero16"][0, 2] = 2.0   # 0x4000
    pos = 64 + 27               # page index 1; cell 1 of the page, token 11 = 8 + 2 + 1
    spec.write(buf, 3, 2, pos, key, val, 0)
    base = 3 * 3 * 4 * 2560 + (2 * 4 + 1) * 2560
    want = {base + 11 * 64 + 16 + 8 + 2: 0x90,                                # key code, high half
            base + 1024 + 512 + (3 * 4 + 1) * 16 + 2 * 4 + 2 + 0: 0x60,       # value code, high half, odd token
            base + 2048 + 1 * 32 + 3 * 8 + 4 + 2 + 1: 0x3C,                   # key scale
            base + 2176 + (11 * 4 + 1) * 2 + 1: 0xC0,                         # key zero
            base + 2304 + 1 * 32 + 0 + 4 + 2 + 1: 0x38,                       # value scale
            base + 2432 + 1 * 32 + 2 * 8 + 4 + 2 + 1: 0x40}                   # value zero
    assert {int(i): int(buf[i]) for i in np.nonzero(buf)[0]} == want


@pytest.mark.parametrize("d", [64, 128, 256])
def test_write_then_read(d):
    rng = np.random.default_rng(d)
    spec = paged.PagedSpec(d, 2, 16, 5)
    buf = rng.integers(0, 256, spec.nbytes()).astype(np.uint8)
    row = [4, 1, 3]
    x, y = rng.standard_normal((40, d)).astype(np.float32), rng.standard_normal((40, d)).astype(np.float32)
    key, val = paged.encode(x), paged.encode(y)
    spec.write_sequence(buf, row, 1, 3, key, val)
    k, v = spec.read(buf, row, 1, 3, 40)
    for got, src, rec in ((k, x, key), (v, y, val)):
        step = rec["scale16"].repeat(32, 1)
        # half a step, and the fp16 roundings of zero and of fifteen scales at the ends of the range
        room = step * 0.5 + 16 * 2.0 ** -11 * np.abs(src).max()
        assert (np.abs(got - src) <= room).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_turns_pairs(interleaved):
    rng = np.random.default_rng(0)
    rot, d = 32, 64
    table = tq.tq_make_rope_table(50, rot, 10000.0).numpy()
    x = rng.standard_normal((7, 3, d))
    pos = np.array([0, 1, 2, 7, 31, 40, 49])
    y = paged.rotate(x, table, pos, interleaved)
    assert np.array_equal(y[..., rot:], x[..., rot:].astype(np.float32))
    assert np.allclose(y[0], x[0], rtol=0, atol=1e-7)  # position 0 does not turn
    for i in range(7):
        for j in range(rot // 2):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
            w = pos[i] * 10000.0 ** (-2 * j / rot)
            m = np.array([[np.cos(w), -np.sin(w)], [np.sin(w), np.cos(w)]])
            assert np.allclose(y[i][:, [a, b]], x[i][:, [a, b]] @ m.T, rtol=0, atol=1e-6)


def test_rope_table_matches_numpy_and_refuses():
    t = tq.tq_make_rope_table(1000, 64, 500000.0).numpy()
    a = np.arange(1000)[:, None] * 500000.0 ** (-2 * np.arange(32) / 64)
    # one rounding to float32, and float64 angles a few units in the last place apart
    assert np.allclose(t, np.concatenate([np.cos(a), np.sin(a)], 1), rtol=0, atol=2.0 ** -24 + 1e-10)
    lib = tq.load()
    assert lib.tq_make_rope_table(8, 16, 1e4, None) == 1
    for bad in ((0, 16, 1e4), (8, 16, 0.0), (8, 16, float("inf")), (8, 16, float("nan"))):
        assert lib.tq_make_rope_table(*bad, t.ctypes.data) == 1
    for rot in (0, 8, 24, 272):
        assert lib.tq_make_rope_table(1, rot, 1e4, t.ctypes.data) == 2


def test_attend_against_a_loop():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal(8), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    w = [np.exp(sum(q[c] * k[t, c] for c in range(8)) * 0.3) for t in range(4)]
    out = sum(w[t] * v[t] for t in range(4)) / sum(w)
    got, a, m = paged.attend(q, k, v, 4, 0.3)
    assert np.allclose(got, out, rtol=1e-13, atol=0)
    assert (a >= np.abs(got) - 1e-15).all() and m >= max(abs(k[t] @ q) * 0.3 for t in range(4))
    assert not paged.attend(q, k, v, 0, 0.3)[0].any()
