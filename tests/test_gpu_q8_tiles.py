"""The INT8 base product (no valid user: every id -1) on each tile of the plan, unsplit,
with tokens that were written long before the call: the caches are swept by a large fill,
so the first stage's copies are the slowest of the call.

Token (8 significant bits) times code (7) is exact in fp32, so only the sums and the row's
scale round.  A sum of K terms takes at most K / 4 accumulations of at most 2^-23 |partial
sum| each (truncation allowed); with s = sqrt(sum (x q)^2) the partial sums stay within
6 s, and independent errors add as sqrt(K / 4) with 6 standard deviations:
|err| <= scale 36 sqrt(K / 4) 2^-23 s, and 2^-24 |y| for the product with the scale."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, bf16_to_f64, to_np
from tenant_serving_amd import bitdelta as B

pytestmark = pytest.mark.gpu

CASES = {
    "64x64": (4096, 14336, 256), "64x64 ragged": (1000, 1088, 77), "64x128": (3200, 1024, 385),
    "128x128": (4100, 576, 1000), "128x256": (25600, 448, 250), "256x256": (14336, 576, 1024),
}


@pytest.mark.parametrize("tile", CASES)
def test_int8_product_on_cold_tokens(tile):
    d_out, d_in, T = CASES[tile]
    g = torch.Generator(DEV).manual_seed(d_in)
    w = torch.randn(d_out, d_in, generator=g, device=DEV).bfloat16()
    x = torch.randn(T, d_in, generator=g, device=DEV).bfloat16()
    q, s = B.quantize_base(w)
    signs = torch.zeros((1, d_out, d_in // 64), dtype=torch.int64, device=DEV)
    sc = torch.zeros((1, 1), dtype=torch.float32, device=DEV)
    ids = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    p = B.params("matrix")
    junk = torch.empty(1 << 28, device=DEV)  # 1 GB, four times the last-level cache
    ys = []
    for rep in range(3):
        junk.fill_(1e30 + rep)
        ys.append(B.apply_q8(x, q, s, signs, sc, p, ids, check=True))
    rows = sorted({0, 1, d_out - 1} | set(np.random.default_rng(T).choice(d_out, 61, replace=False).tolist()))
    oq, os_ = O.quantize_rows(to_np(w)[rows], dtype=O.BF16)
    assert np.array_equal(to_np(q)[rows], oq) and np.array_equal(to_np(s)[rows], os_)
    xv, qv, sv = bf16_to_f64(to_np(x)), oq.astype(np.float64), os_.astype(np.float64)
    ref = (xv @ qv.T) * sv
    bar = sv * 36 * np.sqrt(d_in / 4) * 2.0 ** -23 * np.sqrt((xv * xv) @ (qv * qv).T) + 2.0 ** -24 * np.abs(ref)
    err = np.abs(ys[0].cpu().numpy()[:, rows].astype(np.float64) - ref) - bar
    assert np.all(err <= 0), (float(err.max()), np.unravel_index(err.argmax(), err.shape))
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
