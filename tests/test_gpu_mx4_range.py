"""The MX4 operators at the ends of their range: K parts and long rows on the large tiles,
every scale byte and code, blocks at the smallest and the largest scale in the products,
groups under 128 columns and the widest rows in the multi-tenant apply.

Bars: products as in test_gpu_mx4 (only the fp32 sums round; the values at the ends of the
scale range are exact in bf16, subnormal ones included); the delta term of groups under 128
columns is fp32 sums of exact bf16 products (1e-5 rms), of the others the encoding's bound."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import (DEV, TOL_BF16, assert_delta_within_bound, bf16_to_f64, custom, gpu_bank,
                      max_err_vs_rms, o_sdtype, oracle_bank, to_np, tol_delta)
from tenant_serving_amd import bitdelta as B
from tenant_serving_amd import synth as S

pytestmark = pytest.mark.gpu


def assert_product(got, xv, wv, what=""):
    """got [T][N] (fp32) against xv [T][K] . wv [N][K]^T in binary64."""
    K = xv.shape[1]
    ref = xv @ wv.T
    s = np.sqrt((xv * xv) @ (wv * wv).T)
    excess = np.abs(got.astype(np.float64) - ref) - 36 * np.sqrt(K / 4) * 2.0 ** -23 * s
    assert np.all(excess <= 0), (what, float(np.nanmax(excess)), np.unravel_index(excess.argmax(), excess.shape))


def product(x4, x, base):
    """(y, the tokens' values in binary64) of one base matrix."""
    if not x4:
        return B.base_gemm_mx4(x, [base])[0], x.double().cpu().numpy()
    xq = B.quantize_mx4(x)
    return B.base_gemm_mx4x4(xq, [base])[0], O.mx4_dequantize(to_np(xq[0]), to_np(xq[1]))


# (MX4 tokens, d_out, d_in, T, K parts): parts with a ragged last one on each of the tiles of
# 128 rows or more, and rows of many 512-column periods without parts
LARGE = [
    (True, 73, 8320, 4214, 6), (True, 4483, 10304, 204, 7), (True, 11178, 15936, 133, 4),
    (True, 16000, 4160, 300, 1), (True, 7000, 4160, 1500, 1), (True, 4000, 8256, 1000, 1),
    (False, 5120, 17408, 1144, 2), (False, 8923, 8384, 105, 6), (False, 3000, 8256, 140, 2),
    (False, 5120, 8256, 1144, 1), (False, 7700, 4160, 1144, 1), (False, 12000, 8256, 100, 1),
]


@pytest.mark.parametrize("x4,d_out,d_in,T,parts", LARGE)
def test_products_of_k_parts_and_long_rows(x4, d_out, d_in, T, parts):
    query = B.bd_base_gemm_mx4x4_n_workspace_bytes if x4 else B.bd_base_gemm_mx4_n_workspace_bytes
    assert query(T, d_in, [d_out]) // (4 * T * d_out) == (parts if parts > 1 else 0)  # the plan's split
    g = torch.Generator(DEV).manual_seed(d_in + T)
    w = torch.randn(d_out, d_in, generator=g, device=DEV)
    w *= torch.exp2(torch.randint(-6, 7, (d_out, d_in // 32), generator=g, device=DEV).float()).repeat_interleave(32, 1)
    x = torch.randn(T, d_in, generator=g, device=DEV).bfloat16()
    base = B.quantize_mx4(w)
    y, xv = product(x4, x, base)
    rows = sorted({0, d_out - 1} | set(np.random.default_rng(T).choice(d_out, min(d_out, 48), replace=False).tolist()))
    wv = O.mx4_dequantize(to_np(base[0])[rows], to_np(base[1])[rows])
    assert_product(y.cpu().numpy()[:, rows], xv, wv, (x4, d_out, d_in, T))
    assert torch.equal(y, product(x4, x, base)[0])


# ------------------------------------------------------- scale bytes and codes

def test_every_scale_byte_and_code_dequantised():
    """All 16 codes under all 256 scale bytes, in fp32 and bf16: exact, Inf beyond the range
    (codes of 2 and more at byte 254, of 4 and more at 253), NaN at 255."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)  # every pair of codes: 512 columns
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 16)
    want = O.mx4_dequantize(codes.numpy(), scales.numpy())
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)  # exact, or Inf
    assert np.isinf(want[254]).any() and np.isinf(want[253]).any() and np.isfinite(want[252]).all()
    for dt in (torch.float32, torch.bfloat16):
        got = B.dequantize_mx4(codes.to(DEV), scales.to(DEV), dt).float().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)
        assert np.array_equal(np.signbit(got[:255]), np.signbit(want[:255]))  # -0 too


def test_values_of_every_scale_byte_that_finite_blocks_reach():
    """values_out and the dequantised codes under the bytes 0..252: what the codes stand for."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], np.float64)
    blk = np.zeros(32)
    blk[:27] = np.concatenate([mids, mids * (1 - 2.0 ** -7), -mids * (1 + 2.0 ** -7)])
    blk[27:] = [-0.25, -5.0, -1.75, 4.0, 7.5]
    rows = np.stack([np.ldexp(blk, e) for e in range(-127, 126)]).astype(np.float32)
    for dtype in (torch.float32, torch.bfloat16):
        w = torch.from_numpy(np.concatenate([rows, rows[::-1]], axis=1)).to(dtype)
        codes, scales, values = B.quantize_mx4(w.to(DEV), values=True)
        oc, os_ = O.mx4_quantize(to_np(w), dtype=O.BF16 if dtype == torch.bfloat16 else O.F32)
        assert np.array_equal(to_np(codes), oc) and np.array_equal(to_np(scales), os_)
        ov = O.mx4_dequantize(oc, os_)
        assert np.array_equal(values.double().cpu().numpy(), ov)
        assert np.array_equal(B.dequantize_mx4(codes, scales, dtype).double().cpu().numpy(), ov)


def extreme_base(rows, cols, byte, seed, top=16):
    """Random codes (magnitudes below index top) under one scale byte, and their values."""
    r = np.random.default_rng(seed)
    mag = r.integers(0, top, (rows, cols)) | r.integers(0, 2, (rows, cols)) << 3
    codes = (mag[:, 0::2] | mag[:, 1::2] << 4).astype(np.uint8)
    scales = np.zeros((rows, 16 * ((cols + 511) // 512)), np.uint8)
    scales[:, :cols // 32] = byte
    return (torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)), O.mx4_dequantize(codes, scales)


# (scale byte, codes in use, exponent of the tokens that makes the sums ordinary numbers):
# byte 0: weights down to 2^-128, subnormal in bf16 and fp32; 252: the largest of a block of
# finite values; 253 and 254: from a foreign checkpoint, codes that stay within the range
EXTREME = [(0, 8, 118), (1, 8, 117), (252, 8, -120), (253, 6, -120), (254, 4, -121)]


@pytest.mark.parametrize("x4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("T", [1, 9, 80, 300])
@pytest.mark.parametrize("byte,top,e", EXTREME, ids=lambda v: str(v))
def test_products_at_the_ends_of_the_scales(byte, top, e, T, x4):
    d_in = 576
    base, wv = extreme_base(130, d_in, byte, byte + T, top)
    g = torch.Generator().manual_seed(T)
    x = (torch.randn(T, d_in, generator=g).clamp(-3, 3) * 2.0 ** e).bfloat16().to(DEV)
    y, xv = product(x4, x, base)
    assert_product(y.cpu().numpy(), xv, wv, (byte, T))


@pytest.mark.parametrize("byte,top,e", EXTREME, ids=lambda v: str(v))
def test_apply_base_at_the_ends_of_the_scales(byte, top, e):
    """The one-launch decode apply's base product (tokens of the base model)."""
    d_in, T = 576, 9
    base, wv = extreme_base(50, d_in, byte, byte, top)
    g = torch.Generator().manual_seed(byte)
    x = (torch.randn(T, d_in, generator=g).clamp(-3, 3) * 2.0 ** e).bfloat16().to(DEV)
    signs = torch.zeros((1, 50, d_in // 64), dtype=torch.int64, device=DEV)
    ids = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    y = B.apply_mx4(x, *base, signs, torch.zeros(1, 1, device=DEV), B.params("matrix"), ids, check=True)
    assert_product(y.cpu().numpy(), x.double().cpu().numpy(), wv, byte)


# ------------------------------------------------------------------ the apply

APPLY = [
    # (mode, group, scale dtype, d_out, d_in, T, n_users, y dtype)
    ("group", 32, B.BD_F32, 136, 1152, 40, 4, torch.float32),
    ("group", 64, B.BD_F16, 136, 1152, 9, 4, torch.bfloat16),
    ("group", 16, B.BD_F32, 50, 576, 100, 3, torch.float32),
    ("group", 256, B.BD_F32, 136, 2048, 70, 5, torch.float32),
    ("group", 512, B.BD_F16, 80, 4096, 12, 3, torch.bfloat16),
    ("group", 128, B.BD_F32, 96, 17408, 33, 3, torch.float32),
    ("row", 128, B.BD_F16, 100, 14336, 16, 5, torch.float32),
    ("matrix", 128, B.BD_F32, 64, 17408, 1, 1, torch.bfloat16),
    ("col", 128, B.BD_F16, 64, 17408, 70, 4, torch.float32),
    ("matrix", 128, B.BD_F32, 128, 14336, 200, 40, torch.bfloat16),
]


@pytest.mark.parametrize("tokens", ["bf16", "mx4"])
@pytest.mark.parametrize("case", APPLY, ids=lambda c: f"{c[0]}{c[1]}-{c[3]}x{c[4]}-T{c[5]}")
def test_apply_groups_and_wide_rows(case, tokens):
    mode, grp, sd, d_out, d_in, T, U, ydt = case
    ids = np.random.default_rng(T + d_in).integers(-1, U, T).astype(np.int32)
    w = custom(d_out, d_in, S.BF16, n_users=U, T=T, b=5e-3, cid=2800 + grp + T)
    p = B.params(mode, grp, 0.0, sd)
    x_dev = S.dev_x(w, 0)
    codes, scales, values = B.quantize_mx4(S.dev_wbase(w, 0), values=True)
    vb = to_np(values)
    signs, dsc = gpu_bank(w, 0, values, p, range(U))
    words, osc = oracle_bank(w, 0, vb, p, range(U))
    assert np.array_equal(to_np(signs), words)
    ids_dev = torch.from_numpy(ids).to(DEV)
    y = B.apply_mx4(x_dev, codes, scales, signs, dsc, p, ids_dev, y_dtype=ydt, tokens=tokens, check=True)
    y0 = B.apply_mx4(x_dev, torch.zeros_like(codes), scales, signs, dsc, p, ids_dev, tokens=tokens, check=True)
    xb = S.host_x(w, 0)
    _, yb, yd = O.apply(xb, vb, words, osc, p.mode, ids, g=grp, sdtype=o_sdtype(p), xdtype=O.BF16, wdtype=O.BF16)
    if tokens == "mx4":
        yb = O.mx4_dequantize(*O.mx4_quantize(xb, dtype=O.BF16)) @ bf16_to_f64(vb).T
    err, rms = max_err_vs_rms(y.float().cpu().numpy(), yb + yd)
    assert err <= TOL_BF16 * rms, (err, rms)
    g0 = y0.cpu().numpy()
    if (ids >= 0).any():
        err0, rms0 = max_err_vs_rms(g0, yd)
        if mode == "group" and grp < 128:
            assert err0 <= 1e-5 * rms0, (err0, rms0)
        else:
            assert err0 <= tol_delta(mode) * rms0, (err0, rms0)
            assert_delta_within_bound(g0, yd, xb, osc, p, ids)
    assert np.all(g0[ids < 0] == 0)
    y2 = B.apply_mx4(x_dev, codes, scales, signs, dsc, p, ids_dev, y_dtype=ydt, tokens=tokens)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("T", [5, 80])
def test_products_of_values_beyond_the_range(T):
    """Codes of 2 and more under byte 254 (2^128 and above; no block quantised from finite
    values has them): the bf16-token product widens the weights to bf16, where they are Inf;
    the MX4-token product never forms the value, and its sums are ordinary."""
    base, wv = extreme_base(20, 576, 254, T)
    g = torch.Generator().manual_seed(T)
    x = (torch.randn(T, 576, generator=g).clamp(-3, 3) * 2.0 ** -120).bfloat16().to(DEV)
    y, _ = product(False, x, base)
    assert not torch.isfinite(y).any()
    y4, xv = product(True, x, base)
    assert_product(y4.cpu().numpy(), xv, wv, T)
