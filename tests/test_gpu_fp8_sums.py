"""FP8 base products are fp32 sums: against binary64, on activations with loud channels, and on
large products that cancel.

Two e4m3 values multiply exactly (4 + 4 significant bits), so the error is that of fp32
additions: at most K / 4 inside the matrix instructions (pairs of lanes' four columns at a time,
at the finest) and one per 128 columns behind them, each off by at most 2^-23 of its partial sum
(a truncation; half that if it rounds).  The partial sums of random signs have at most s, s^2 =
sum (x w)^2, as their root mean square, and independent errors add as the root of their number:
over many outputs the error's norm stays within 2^-23 sqrt(K / 4 + K / 128 + 1) of that of s.
A matrix instruction that cuts products 13 places below the largest of its group is 1.3e-5 to
2.5e-5 off on such tokens, three times the bar at 17408 columns and more at fewer."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV
from tenant_serving_amd import bitdelta as B

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def loud_tokens(T, cols, seed):
    """Normal activations, one channel in 128 eight times as large: FP8 form and values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, cols, generator=g)
    x *= torch.where(torch.rand(cols, generator=g) < 1 / 128, 8.0, 1.0)
    x = x.to(torch.bfloat16)
    c, s = O.fp8_quantize_tokens(x.float().numpy())
    return x.to(DEV), (torch.from_numpy(c).to(DEV).view(E4M3), torch.from_numpy(s).to(DEV)), O.fp8_token_values(c, s)


def checkpoint(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    c, s = O.fp8_quantize((torch.randn(rows, cols, generator=g) * 0.02).numpy())
    s = (s * (0.5 + torch.rand(s.shape, generator=g)).numpy()).astype(np.float32)
    return (torch.from_numpy(c).to(DEV).view(E4M3), torch.from_numpy(s).to(DEV)), O.fp8_dequantize(c, s)


def assert_fp32_sums(y, xv, wv):
    K = xv.shape[1]
    ref, s2 = xv @ wv.T, (xv * xv) @ (wv * wv).T
    bar = 2.0 ** -23 * np.sqrt(K / 4 + K / 128 + 1) * np.sqrt(s2.sum())
    off = np.linalg.norm(y.double().cpu().numpy() - ref)
    assert off <= bar, (off / np.linalg.norm(ref), bar / np.linalg.norm(ref))


CASES = [(1, 4096, 6144), (7, 576, 333), (16, 14336, 256), (17, 4096, 700), (33, 1088, 1000), (64, 4096, 2560),
         (70, 5120, 1024), (129, 4096, 4096), (300, 17408, 640), (333, 8256, 700), (700, 2048, 2050),
         (1144, 17408, 640), (2300, 1024, 2500)]


@pytest.mark.parametrize("T,cols,rows", CASES)
def test_products_are_fp32_sums(T, cols, rows):
    base, wv = checkpoint(rows, cols, seed=rows)
    _, xq, xv = loud_tokens(T, cols, seed=T)
    (y,) = B.base_gemm_fp8(xq, [base])
    assert_fp32_sums(y, xv, wv)
    (h,) = B.base_gemm_fp8(xq, [base], y_dtype=torch.bfloat16)
    assert torch.equal(h, y.to(torch.bfloat16))


@pytest.mark.parametrize("T,cols,mode", [(1, 512, "matrix"), (16, 4096, "row"), (16, 1088, "matrix"), (12, 576, "col"),
                                         (9, 4160, "matrix"), (40, 1024, "col"), (300, 2048, "matrix")])
@pytest.mark.parametrize("given", [True, False])
def test_applies_base_part_is_fp32_sums(T, cols, mode, given):
    """Tokens of the base model (user -1): the apply is its base product."""
    rows, U = 320, 2
    base, wv = checkpoint(rows, cols, seed=rows + 1)
    x, xq, xv = loud_tokens(T, cols, seed=T)
    signs = torch.zeros(U, rows, cols // 64, dtype=torch.int64, device=DEV)
    n = {"matrix": 1, "row": rows, "col": cols}[mode]
    y = B.apply_fp8(x, *base, signs, torch.ones(U, n, device=DEV), B.params(mode), torch.full((T,), -1, dtype=torch.int32, device=DEV),
                    xq=xq if given else None, check=True)
    assert_fp32_sums(y, xv, wv)


@pytest.mark.parametrize("T", [1, 16, 17, 40, 64, 65, 150, 300, 700, 1200])
@pytest.mark.parametrize("small", [4.0, 0.5, 2.0 ** -6])
def test_small_products_beside_large_ones_that_cancel(T, small):
    """448 x 448, -448 x 448 and a small product, next to each other or far apart: every partial
    sum in any order is a multiple of the small one under 2^24 of it, so fp32 sums are exact."""
    cols, rows = 1088, 200
    sets = [(0, 1, 2), (16, 24, 18), (3, 70, 4), (5, 1087, 6), (511, 512, 513), (64, 96, 80)]
    x, w = torch.zeros(T, cols), torch.zeros(rows, cols)
    for a, b, c in sets:
        x[:, a], x[:, b], x[:, c] = 448.0, 448.0, 0.5
    for r in range(rows):  # (a row reads its own three columns)
        a, b, c = sets[r % 6]
        w[r, a], w[r, b], w[r, c] = 448.0, -448.0, small / 0.5
    xv = x.to(E4M3).double()
    wv = w.to(E4M3).double()
    assert torch.equal(xv, x.double()) and torch.equal(wv, w.double())
    want = xv @ wv.t()
    assert torch.equal(want, torch.full_like(want, small))
    nb = (cols + 127) // 128
    xs = torch.zeros(T, B.bd_fp8_scale_stride(cols), dtype=torch.uint8)
    xs[:, :nb] = 127
    ws = torch.ones((rows + 127) // 128, nb)
    (y,) = B.base_gemm_fp8((x.to(E4M3).to(DEV), xs.to(DEV)), [(w.to(E4M3).to(DEV), ws.to(DEV))])
    assert torch.equal(y.double().cpu(), want), (y.cpu()[0, :6], want[0, :6])
