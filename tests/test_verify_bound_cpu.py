"""The bounds of tests/verify_bound.py against a model of the kernels' roundings of the weights: what the kernels do
is inside, what a mistake would cost is outside."""
import numpy as np
import pytest
import torch

from tests import verify_bound as VB


def rows(ctx, size, seed, sink=0.0, d=64):
    """One query over INT8 rows: q, k, v (values), scales, codes."""
    rng = np.random.default_rng(seed)
    q, k = rng.standard_normal((1, 1, d)), rng.standard_normal((ctx, 1, d))
    if sink:
        q[..., 0], k[:, :, 0] = 8.0, 0.0
        k[0, 0, 0] = sink * d ** 0.5 / 8
    v = rng.standard_normal((ctx, 1, d)) * size
    if sink:
        v[0] *= 2.0 ** -8
    s = (np.abs(v).max(-1) / 127).astype(np.float32)
    c = np.rint(v / s[..., None].astype(np.float64))
    return q, k, s, c


def model(q, k, s, c, factor, counted=True, residual=True, drop=()):
    """Weights 2^(z - M) s 2^factor as an fp16 pair, everything else in 64 bits; counted: M counts the scale."""
    d, s = q.shape[-1], s.astype(np.float64)
    z = (q[:, 0] @ k[:, 0].T)[0] / np.sqrt(d) / np.log(2)
    with np.errstate(divide="ignore"):
        m = (z + np.log2(s[:, 0]) if counted else z).max()
    p = np.exp2(z - m + factor)
    w = p * s[:, 0]
    hi = w.astype(np.float16)
    lo = (w - hi).astype(np.float16) if residual else np.float16(0)
    x = hi.astype(np.float64) + lo
    x[list(drop)] = 0.0
    return torch.tensor((x @ c[:, 0] / p.sum()).astype(np.float16).astype(np.float64))


def reference(q, k, s, c):
    t = lambda a: torch.tensor(np.asarray(a, np.float64))  # noqa: E731
    n = k.shape[0]
    o, bound = VB.attention(t(q), t(k), t(c * s[..., None]), t(s), t(np.abs(c)), [1], q.shape[-1] ** -0.5, n - 1, False)
    return o[0, 0], bound[0, 0]


@pytest.mark.parametrize("ctx", [4, 300, 8000])
@pytest.mark.parametrize("size,sink", [(1.0, 0), (2.0 ** -7, 0), (2.0 ** -10, 0), (2.0 ** -14, 0), (1.0, 12.0)])
def test_the_kernels_weights_are_inside(ctx, size, sink):
    r = rows(ctx, size, 1, sink)
    o, bound = reference(*r)
    got = model(*r, 6.0)
    assert ((got - o).abs() <= bound).all() and VB.rms(got - o) <= VB.rms_bound(o, ctx)


@pytest.mark.parametrize("size,sink", [(2.0 ** -7, 0), (2.0 ** -10, 0), (2.0 ** -14, 0), (1.0, 12.0)])
def test_weights_that_shrink_with_v_are_outside(size, sink):
    """(2^-7 is found by the root mean square alone: a single element's bound has to allow every rounding at its worst.)"""
    r = rows(8000, size, 1, sink)
    o, bound = reference(*r)
    got = model(*r, -2.0, counted=False)
    assert VB.rms(got - o) > VB.rms_bound(o, 8000) and (size == 2.0 ** -7 or ((got - o).abs() > bound).any())


@pytest.mark.parametrize("ctx,tile", [(300, 0), (8000, 32), (20000, 19968)])
def test_a_lost_tile_is_outside(ctx, tile):
    r = rows(ctx, 1.0, 2)
    o, bound = reference(*r)
    got = model(*r, 6.0, drop=range(tile, tile + 32))
    assert ((got - o).abs() > bound).any() and VB.rms(got - o) > VB.rms_bound(o, ctx)


def test_a_lost_residual_is_outside():
    worst = 0.0
    for seed in range(20):
        r = rows(4, 1.0, seed)
        o, bound = reference(*r)
        worst = max(worst, ((model(*r, 6.0, residual=False) - o).abs() / bound).max().item())
    assert worst > 1.0
