"""The bounds that the paged decode is held to are tight enough to see a lost token, a shifted tail, a wrong scale and weights that
belong to other values, and wide enough for the roundings that they are made of."""

import numpy as np
import pytest

import paged_bounds as pb
from oracle import paged


def _case(rng, n, d, sizes, k_size, q_size=0.375):
    """Encoded keys and values whose groups of 32 channels have the given sizes, and a query that gives every token a weight
    (logits within one or two of each other)."""
    x = rng.standard_normal((2, n, d)) * np.exp(0.5 * rng.standard_normal((2, 1, d)))
    x[0] *= k_size
    x[1] *= np.resize(sizes, d // 32).repeat(32)
    key, val = (paged.encode(y.astype(np.float32)) for y in x)
    k, v = (r["codes"] * r["scale16"].repeat(32, 1) + r["zero16"].repeat(32, 1) for r in (key, val))
    return q_size * rng.standard_normal(d), k, key, v, val


CASES = [
    # tokens, d, sizes of the groups, of the keys, softmax scale
    (257, 128, [1.0], 1.0, None),
    (200, 128, [1.0], 1e-3, None),
    (200, 128, [300.0], 1.0, 0.0),
    (333, 64, [1.0], 1.0, None),
    (150, 256, [1.0, 1e-3], 1.0, None),
    (120, 128, [1000.0, 0.01, 1.0, 0.1], 1.0, None),
]


@pytest.mark.parametrize("n,d,sizes,k_size,scale", CASES)
@pytest.mark.parametrize("out_bits", [8, 11])
def test_the_bound_sees_small_mistakes(n, d, sizes, k_size, scale, out_bits):
    rng = np.random.default_rng(n + d)
    scale = d ** -0.5 if scale is None else scale
    for _ in range(8):
        q, k, key, v, val = _case(rng, n, d, sizes, k_size)
        tol = pb.bound(q, k, key, v, val, scale, out_bits)
        w, o = pb.attend(q, k, v, scale)
        tail = v.copy()
        tail[n - 16 :] = np.roll(v[n - 16 :], 1, 0)
        wrong = v.copy()
        wrong[n - 1, -32:] += val["scale16"][n - 1, -1] * 8
        assert (np.abs(pb.attend(q, k[:-1], v[:-1], scale)[1] - o) > tol).any()  # the last token left out
        assert (np.abs(w @ wrong - o) > tol).any()                               # half its codes' range off in one group
        if scale != 0.0 and k_size == 1.0:                                       # (equal weights: the same sum)
            assert (np.abs(w @ tail - o) > tol).any()                            # the tail's values one token on


def _rounded(q, k, val, scale):
    """The bf16 path's roundings in turn: p, p 2^-E, p s 2^-E and the sums of four p z 2^-E in fp16."""
    x = k @ q * scale * np.log2(np.e)
    p = np.float16(2.0 ** (x - x.max() + 9)).astype(np.float64)[:, None]
    s, z = val["scale16"], val["zero16"]
    E = np.maximum(np.floor(np.log2(np.maximum(np.maximum(s, np.abs(z)).max(0), 2.0 ** -24))) + 1, -2)
    pk = np.float16(p * 2.0 ** -E)
    ps = np.float16(pk.astype(np.float64) * s).astype(np.float64)
    n = len(p)
    pad = -n % 4
    pk4, z4 = (np.pad(y.astype(np.float64), ((0, pad), (0, 0))).reshape(-1, 4, y.shape[1]) for y in (pk, z))
    zs = np.zeros(pk4[:, 0].shape)
    for i in range(4):
        zs = np.float16(zs + pk4[:, i] * z4[:, i]).astype(np.float64)
    out = (ps.repeat(32, 1) * val["codes"]).sum(0) + zs.sum(0).repeat(32)
    return out * 2.0 ** E.repeat(32) / p.sum()


@pytest.mark.parametrize("n,d,sizes,k_size,scale", CASES)
@pytest.mark.parametrize("q_size", [0.375, 1.5])
def test_the_bound_holds_the_roundings_that_it_names(n, d, sizes, k_size, scale, q_size):
    rng = np.random.default_rng(n)
    scale = d ** -0.5 if scale is None else scale
    for _ in range(4):
        q, k, key, v, val = _case(rng, n, d, sizes, k_size, q_size)
        o = pb.attend(q, k, v, scale)[1]
        assert (np.abs(_rounded(q, k, val, scale) - o) <= pb.bound(q, k, key, v, val, scale, 8)).all()
