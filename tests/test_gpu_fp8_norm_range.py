"""The RMS norm over the range of its inputs: squares that leave fp32's range on either side,
eps from 0 to the largest.

x = s / sqrt(mean(s^2) + eps) * weight in fp32, rounded once to bf16: off by at most half a step,
2^-8 of the value, and by a few fp32 roundings (the sum of squares is one of positive numbers:
2^-24 sqrt(d) on average, under 2^-17 for every d); below the normal range by half a subnormal
step of bf16 (2^-134) and fp32's own (2^-149)."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, to_np
from tenant_serving_amd import bitdelta as B

pytestmark = pytest.mark.gpu


def check(h, w, eps, residual=None):
    s, x, (codes, scales) = B.rmsnorm_fp8(h.to(DEV), w.to(DEV), eps, residual=None if residual is None else residual.to(DEV))
    v = h.double() if residual is None else (h.float() + residual.float()).to(h.dtype).double()
    if residual is not None:
        assert torch.equal(s.cpu().double(), v)
    e32 = float(np.float32(eps))
    ref = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + e32) * w.double()
    got = x.cpu().double()
    tol = ref.abs() * (2.0 ** -8 + 2.0 ** -17) + 2.0 ** -134 + 2.0 ** -149
    ok = (got - ref).abs() <= tol
    assert bool(ok.all()), (got[~ok][:4], ref[~ok][:4], eps)
    oc, os_ = O.fp8_quantize_tokens(to_np(x), dtype=O.BF16)
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), oc) and np.array_equal(to_np(scales), os_)


EXPONENTS = [-140, -126, -110, -100, -75, -63, -51, -40, 0, 40, 57, 60, 63, 64, 80, 100, 124]


@pytest.mark.parametrize("d", [64, 4096, 10240, 20480])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_every_magnitude(d, dtype):
    g = torch.Generator().manual_seed(d)
    exps = torch.tensor([e for e in EXPONENTS if dtype is torch.float32 or e >= -126])[:, None]
    h = torch.ldexp(torch.randn(len(exps), d, generator=g).clamp(-4, 4) + 0.25, exps).to(dtype)
    w = 1 + 0.1 * torch.randn(d, generator=g)
    for eps in (0.0, 1e-6, 1e-12, 2.0 ** -120, 1e-38, 1e10, 3e38):
        check(h, w, eps)
    check(h, w, 1e-6, residual=torch.ldexp(torch.randn(h.shape, generator=g), exps))


def test_one_large_value_among_small_ones():
    h = torch.full((4, 512), 1e-3)
    h[0, 5], h[1, 500], h[2, 0] = 1e30, -3e38, 2.0 ** 64
    h[3] = 0.0
    h[3, 77] = 1e-40
    check(h, torch.ones(512), 1e-6)
    check(h, torch.ones(512), 0.0)


def test_rows_that_are_not_finite_or_zero():
    h = torch.randn(5, 576, generator=torch.Generator().manual_seed(3))
    h[0, 3], h[1, 4], h[2] = float("inf"), float("nan"), 0.0
    h[3] *= 1e30
    h[3, 9] = float("-inf")
    _, x, (_, scales) = B.rmsnorm_fp8(h.to(DEV), torch.ones(576, device=DEV), 0.0)
    x = x.cpu().float()
    for r, c in ((0, 3), (3, 9)):  # Inf / Inf, and the finite values over Inf
        assert torch.isnan(x[r, c]) and bool((x[r, torch.arange(576) != c] == 0).all())
    assert torch.isnan(x[1]).all() and torch.isnan(x[2]).all()  # (a row of zeros with eps = 0 is 0 / 0)
    assert torch.isfinite(x[4]).all()
    _, x, _ = B.rmsnorm_fp8(h.to(DEV), torch.ones(576, device=DEV), 1e-6)
    assert bool((x[2] == 0).all())
