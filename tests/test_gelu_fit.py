"""The fit behind the bf16 GeLU, against erfc: its coefficients in 64 bits, its fp32
evaluation with the approximate instructions at the ends of their error bounds, and the
activation's gradient on a GPU for every bf16 argument."""
import os
import re

import numpy as np
import pytest
import torch

from _lib import ROOT, build_and_import

f32 = np.float32


@pytest.fixture(scope="module")
def coefficients():
    with open(os.path.join(ROOT, "fine_grained_moe_router_b200", "csrc", "linear_epilogue.cuh")) as f:
        src = f.read()
    horner = src[src.index("Pair h ="):src.index("q = mul2")]
    c = [float(v) for v in re.findall(r"pair_of\((-?0\.\d+)f\)", horner)]
    assert len(c) == 9
    return c


def test_fit(coefficients):
    from scipy.special import erfcx
    x = np.linspace(0, 10, 400001)
    t = 1 / (1 + x / 2)
    h = np.zeros_like(t)
    for k in coefficients:
        h = h * t + float(f32(k))
    assert np.abs(h * t / erfcx(x) - 1).max() < 8.2e-8


@pytest.mark.parametrize("ex2", [-1, 0, 1])
@pytest.mark.parametrize("rcp", [-1, 0, 1])
def test_tail_in_fp32(coefficients, ex2, rcp):
    """ex2.approx is good to 2^-22 relative, rcp.approx to 2^-23."""
    from scipy.special import erfc
    z = np.linspace(0, 12, 400001).astype(f32)

    def fma(a, b, c):
        return (a.astype(np.float64) * b.astype(np.float64) + np.float64(c)).astype(f32)
    m = (z * z) * f32(-0.72134752044448170368)
    u = fma(z, np.full_like(z, 0.35355339059327376), 1)
    e = (np.exp2(m.astype(np.float64)) * (1 + ex2 * 2.0 ** -22)).astype(f32)
    t = (1 / u.astype(np.float64) * (1 + rcp * 2.0 ** -23)).astype(f32)
    h = np.full_like(z, coefficients[0])
    for k in coefficients[1:]:
        h = fma(h, t, f32(k))
    q = ((h * t) * (e * f32(0.5))).astype(np.float64)
    ref = 0.5 * erfc(z.astype(np.float64) / np.sqrt(2))
    assert np.abs(q - ref).max() < 4.1e-7
    assert np.abs(q / ref - 1)[z <= 4].max() < 1.4e-6
    assert np.abs(q / ref - 1).max() < 8e-6


@pytest.mark.gpu
def test_gradient_for_every_bf16_argument():
    """The bias gradient of one token with dy = 1 is act'(z) = Phi(z) + z phi(z) in fp32. The
    tail errs by 4.1e-7; z phi (at most 0.25) by 2^-22 of itself for ex2.approx and by
    |z|^3 phi / 2 <= 0.24 times 2^-23 for the rounding of z^2; five roundings of values below
    1.13 add 2^-24 of it each."""
    from scipy.special import erfc
    M = build_and_import()
    every = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = every[every.float().abs() <= 13]
    z = z[:len(z) // 8 * 8].view(1, -1).cuda()
    n = z.shape[1]
    d = M.make_linear(1, 8, n, M.MOE_BF16, "gelu")
    db = torch.empty(n, device="cuda")
    M.moe_linear_backward(d, torch.ones_like(z), None, None, z, None, None, db, M.alloc_workspace(d))
    v = z[0].cpu().double().numpy()
    ref = 0.5 * erfc(-v / np.sqrt(2)) + v * np.exp(-v * v / 2) / np.sqrt(2 * np.pi)
    err = np.abs(db.cpu().double().numpy() - ref)
    assert err.max() <= 4.1e-7 + 0.25 * 2.0 ** -22 + 0.24 * 2.0 ** -23 + 5 * 1.13 * 2.0 ** -24
