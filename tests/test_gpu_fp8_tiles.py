"""FP8 base products in every kernel, tile and split of the plan (fp8_tile_cases.py, which the
plan itself is held to on the CPU), ragged in rows and tokens: against binary64 on sampled rows,
between guards, the same bits on every call and in both output types.

Bound: fp32 additions, at most K / 4 inside the matrix instructions and one per 128 columns
behind them, each off by at most 2^-23 of a partial sum that stays within 6 s, s^2 = sum (x w)^2,
independent, 6 standard deviations: 36 sqrt(K / 4 + K / 128 + 1) 2^-23 s.  One dropped or misplaced
product is about s / sqrt(K), a block's wrong scale more."""
import numpy as np
import pytest
import torch

from fp8_tile_cases import CASES
from gpu_util import DEV
from tenant_serving_amd import bitdelta as B

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
GUARD = 64


def random_fp8(rows, cols, seed, tokens):
    """Codes and scales of many magnitudes on the GPU, and the values in binary64."""
    g = torch.Generator(DEV).manual_seed(seed)
    c = (torch.randn(rows, cols, device=DEV, generator=g) * 100).clamp(-448, 448).to(E4M3)
    nb = (cols + 127) // 128
    if tokens:
        s = torch.zeros(rows, B.bd_fp8_scale_stride(cols), dtype=torch.uint8, device=DEV)
        s[:, :nb] = torch.randint(121, 134, (rows, nb), device=DEV, generator=g).to(torch.uint8)
        f = torch.exp2(s[:, :nb].double() - 127)
    else:
        s = (0.5 + torch.rand((rows + 127) // 128, nb, device=DEV, generator=g)) * torch.exp2(
            torch.randint(-6, 7, ((rows + 127) // 128, nb), device=DEV, generator=g).float())
        f = s.double().repeat_interleave(128, 0)[:rows]
    return (c, s), lambda r: c[r].double() * f[r].repeat_interleave(128, 1)[:, :cols]


def guarded(T, n, dtype):
    flat = torch.full((T * n + 2 * GUARD,), 7.5, device=DEV, dtype=dtype)
    return flat, flat[GUARD:GUARD + T * n].view(T, n)


@pytest.mark.parametrize("tile,S,T,d_outs,d_in", [c for c in CASES if c[2] * sum(c[3]) * c[4] < 1 << 36],
                         ids=lambda v: str(v).replace(" ", ""))
def test_tile(tile, S, T, d_outs, d_in):
    xq, xval = random_fp8(T, d_in, T, True)
    bases, wvals = zip(*[random_fp8(n, d_in, 7 * n + i, False) for i, n in enumerate(d_outs)])
    need = B.bd_base_gemm_fp8_n_workspace_bytes(T, d_in, d_outs)
    assert (need > 0) == (S > 1)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    outs = {}
    for name, dtype, work in (("f32", torch.float32, ws), ("again", torch.float32, ws), ("bf16", torch.bfloat16, ws),
                              ("whole", torch.float32, None)):
        flat, ys = zip(*[guarded(T, n, dtype) for n in d_outs])
        assert B.bd_base_gemm_fp8_n(*xq, list(bases), list(ys), None if work is None else work[:need] if need else None) == B.BD_OK
        torch.cuda.synchronize()
        for f in flat:
            assert bool((f[:GUARD] == 7.5).all()) and bool((f[-GUARD:] == 7.5).all()), name
        outs[name] = ys
    assert bool((ws[need:] == 0x5A).all())
    xv = xval(torch.arange(T, device=DEV)).cpu().numpy()
    rng = np.random.default_rng(T)
    for i, n in enumerate(d_outs):
        y, again, h, whole = (outs[k][i] for k in ("f32", "again", "bf16", "whole"))
        assert torch.equal(y, again) and torch.equal(h, y.to(torch.bfloat16))
        rows = sorted({0, n - 1, n // 2} | set(rng.choice(n, min(n, 48), replace=False).tolist()))
        wv = wvals[i](torch.tensor(rows, device=DEV)).cpu().numpy()
        ref, s = xv @ wv.T, np.sqrt((xv * xv) @ (wv * wv).T)
        tol = 36 * np.sqrt(d_in / 4 + d_in / 128 + 1) * 2.0 ** -23 * s
        for k, v in (("parts", y), ("whole", whole)):
            off = np.abs(v[:, rows].double().cpu().numpy() - ref) - tol
            assert np.all(off <= 0), (k, n, float(off.max()), np.unravel_index(off.argmax(), off.shape))
        # every row: a tile that took another's place or was left out shows in the sums over rows
        full = wvals[i](torch.arange(n, device=DEV))
        xs = xval(torch.tensor([0, T - 1], device=DEV))
        d = (y[[0, T - 1]].double() - xs @ full.t()).abs()
        ss = torch.sqrt((xs * xs) @ (full * full).t())
        assert bool((d <= 36 * (d_in / 4 + d_in / 128 + 1) ** 0.5 * 2.0 ** -23 * ss).all())
