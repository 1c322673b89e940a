"""FP8 products with scales near the ends of their range: a token's 2^E and a weight's scale
meet as their product, which is all that has to be a normal fp32 number."""
import pytest
import torch

from gpu_util import DEV
from tenant_serving_amd import bitdelta as B

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def codes_of(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * 100).clamp(-448, 448).to(E4M3).to(DEV)


@pytest.mark.parametrize("T", [1, 16, 20, 40, 65, 300, 1100])
def test_opposite_scales_leave_the_sums(T):
    """Every block's scales multiply to 1, from 2^-127 x 2^127 to 2^120 x 2^-120: the same bits as
    with scales of 1."""
    rows, cols = 200, 2112
    nb, ld = (cols + 127) // 128, B.bd_fp8_scale_stride(cols)
    x, w = codes_of(T, cols, T), codes_of(rows, cols, 1)
    ones = torch.zeros(T, ld, dtype=torch.uint8, device=DEV)
    ones[:, :nb] = 127
    e = torch.linspace(-127, 120, nb).round().int()
    xs = torch.zeros(T, ld, dtype=torch.uint8, device=DEV)
    xs[:, :nb] = (e + 127).to(torch.uint8).to(DEV)
    ws = torch.ldexp(torch.ones(nb), -e).expand((rows + 127) // 128, nb).contiguous().to(DEV)
    assert bool((ws > 0).all()) and bool(torch.isfinite(ws).all())
    (want,) = B.base_gemm_fp8((x, ones), [(w, torch.ones_like(ws))])
    (got,) = B.base_gemm_fp8((x, xs), [(w, ws)])
    assert torch.isfinite(want).all() and torch.equal(got, want)
    p = B.params("matrix")
    signs = torch.zeros(1, rows, cols // 64, dtype=torch.int64, device=DEV)
    one, ids = torch.ones(1, 1, device=DEV), torch.full((T,), -1, dtype=torch.int32, device=DEV)
    xb = torch.zeros(T, cols, dtype=torch.bfloat16, device=DEV)  # (the base part reads the codes alone)
    a = B.apply_fp8(xb, w, torch.ones_like(ws), signs, one, p, ids, xq=(x, ones), check=True)
    b = B.apply_fp8(xb, w, ws, signs, one, p, ids, xq=(x, xs), check=True)
    assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_blocks_that_are_not_finite(T):
    """Byte 255 under any codes, and weight scales of Inf or NaN: the outputs that multiply the
    block, and no others."""
    rows, cols = 200, 576
    nb, ld = 5, B.bd_fp8_scale_stride(cols)
    x, w = codes_of(T, cols, T), codes_of(rows, cols, 1)
    xs = torch.zeros(T, ld, dtype=torch.uint8, device=DEV)
    xs[:, :nb] = 127
    ws = torch.ones(2, nb, device=DEV)
    (want,) = B.base_gemm_fp8((x, xs), [(w, ws)])
    bad = xs.clone()
    bad[T // 2, 4] = 255
    (y,) = B.base_gemm_fp8((x, bad), [(w, ws)])
    keep = torch.arange(T, device=DEV) != T // 2
    assert torch.isnan(y[T // 2]).all() and torch.equal(y[keep], want[keep])
    nan = ws.clone()
    nan[1, 0] = float("nan")
    (y,) = B.base_gemm_fp8((x, xs), [(w, nan)])
    assert torch.isnan(y[:, 128:]).all() and torch.equal(y[:, :128], want[:, :128])
    inf = ws.clone()
    inf[0, 3] = float("inf")
    (y,) = B.base_gemm_fp8((x, xs), [(w, inf)])
    assert not torch.isfinite(y[:, :128]).any() and torch.equal(y[:, 128:], want[:, 128:])


CODES = torch.arange(256, dtype=torch.uint8)


@pytest.mark.parametrize("T", [1, 16, 40, 256, 700])
def test_every_code(T):
    """Each of the 256 codes, as a weight under tokens of 1 and as a token over weights of 1, in the
    column that its index picks: finite ones exactly (subnormals and both zeros too), the two NaN codes
    in their own outputs alone."""
    cols, rows = 320, 256
    nb, ld = (cols + 127) // 128, B.bd_fp8_scale_stride(cols)
    one = torch.ones((), dtype=torch.float32).to(E4M3).view(torch.uint8)
    xs = torch.zeros(T, ld, dtype=torch.uint8, device=DEV)
    xs[:, :nb] = 127
    w = torch.zeros(rows, cols, dtype=torch.uint8)
    w[CODES.long(), (7 * CODES.long()) % cols] = CODES
    x = one.expand(T, cols).contiguous()
    ws = torch.ones((rows + 127) // 128, nb, device=DEV)
    val = CODES.view(E4M3).float().to(DEV)
    (y,) = B.base_gemm_fp8((x.view(E4M3).to(DEV), xs), [(w.view(E4M3).to(DEV), ws)])
    assert torch.equal(torch.nan_to_num(y, nan=1e9), torch.nan_to_num(val, nan=1e9).expand(T, rows))
    t = torch.arange(T)
    x = torch.zeros(T, cols, dtype=torch.uint8)
    x[t, (11 * t) % cols] = CODES[t % 256]
    (y,) = B.base_gemm_fp8((x.view(E4M3).to(DEV), xs), [(one.expand(rows, cols).contiguous().view(E4M3).to(DEV), ws)])
    assert torch.equal(torch.nan_to_num(y, nan=1e9), torch.nan_to_num(val[t % 256], nan=1e9)[:, None].expand(T, rows))
    # the apply's base part (user -1), in one launch up to 16 tokens
    p, ids = B.params("matrix"), torch.full((T,), -1, dtype=torch.int32, device=DEV)
    signs = torch.zeros(1, rows, cols // 64, dtype=torch.int64, device=DEV)
    a = B.apply_fp8(torch.zeros(T, cols, dtype=torch.bfloat16, device=DEV), one.expand(rows, cols).contiguous().view(E4M3).to(DEV), ws,
                    signs, torch.ones(1, 1, device=DEV), p, ids, xq=(x.view(E4M3).to(DEV), xs), check=True)
    assert torch.equal(torch.nan_to_num(a, nan=1e9), torch.nan_to_num(y, nan=1e9))
