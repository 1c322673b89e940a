"""MX4 base weights and tokens against the oracle: codes, scales and values bit for bit;
the products and the multi-tenant apply within bars derived from their arithmetic.

Products: code, scale and token multiply exactly in fp32 (2 + 8 significant bits), so only
the fp32 sums round.  A sum of K terms takes at most K / 4 accumulations of at most 2^-23
|partial sum| each (truncation allowed); with s = sqrt(sum (x w)^2) the partial sums stay
within 6 s, and independent errors add as sqrt(K / 4) with 6 standard deviations:
|err| <= 36 sqrt(K / 4) 2^-23 s per element.  One dropped product is about s / sqrt(K),
far outside for every K here."""
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
    assert np.all(excess <= 0), (what, float(excess.max()), np.unravel_index(excess.argmax(), excess.shape))


def rand_w(rows, cols, dtype=torch.float32, seed=0, spread=True):
    """Weights whose blocks differ by many powers of two (every scale byte matters)."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(rows, cols, generator=g)
    if spread:
        w *= torch.exp2(torch.randint(-6, 7, (rows, cols // 32), generator=g).float()).repeat_interleave(32, 1)
    return w.to(dtype)


def base_of(rows, cols, seed=0):
    """(codes, scales) on the GPU and the dense values in binary64, from the oracle."""
    c, s = O.mx4_quantize(rand_w(rows, cols, seed=seed).numpy())
    return (torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV)), O.mx4_dequantize(c, s)


def tokens_of(T, cols, seed=1):
    x = rand_w(T, cols, torch.bfloat16, seed, spread=False)
    return x, x.double().numpy()


# ------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 64), (3, 192), (5, 512), (130, 576), (33, 1088), (257, 4096), (2, 17408)])
def test_quantize_matches_oracle(rows, cols, dtype):
    w = rand_w(rows, cols, dtype, seed=rows + cols)
    w[0, :32] = 0.0
    w[-1, -32:] = -0.0
    codes, scales, values = B.quantize_mx4(w.to(DEV), values=True)
    oc, os_ = O.mx4_quantize(to_np(w), dtype=O.BF16 if dtype == torch.bfloat16 else O.F32)
    assert np.array_equal(to_np(scales), os_)
    assert np.array_equal(to_np(codes), oc)
    ov = O.mx4_dequantize(oc, os_)
    assert np.array_equal(values.double().cpu().numpy(), ov)
    for dt in (torch.float32, torch.bfloat16):
        assert np.array_equal(B.dequantize_mx4(codes, scales, dt).double().cpu().numpy(), ov)
    c2, s2 = B.quantize_mx4(w.to(DEV))  # without values: the same codes
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


def test_every_grid_tie_and_scale_byte():
    """All midpoints of the grid (and their neighbours) under every scale byte that finite
    fp32 blocks reach, subnormal ones included."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], np.float64)
    lo, hi = mids * (1 - 2.0 ** -20), mids * (1 + 2.0 ** -20)
    blk = np.zeros(32)
    blk[:27] = np.concatenate([mids, lo, hi])
    blk[27:] = [-0.25, -5.0, -1.75, 4.0, 7.5]
    rows = np.stack([np.ldexp(blk, e) for e in range(-127, 126)]).astype(np.float32)
    w = np.concatenate([rows, rows[::-1]], axis=1)
    codes, scales = B.quantize_mx4(torch.from_numpy(w).to(DEV))
    oc, os_ = O.mx4_quantize(w)
    assert np.array_equal(to_np(scales), os_) and os_.max() == 252 and os_[:, :2].min() == 0
    assert np.array_equal(to_np(codes), oc)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_non_finite_blocks(dtype):
    w = rand_w(6, 576, dtype, seed=9)
    w[1, 3], w[2, 575], w[4, 64], w[4, 65] = float("nan"), float("inf"), -float("inf"), float("nan")
    codes, scales, values = B.quantize_mx4(w.to(DEV), values=True)
    oc, os_ = O.mx4_quantize(to_np(w), dtype=O.BF16 if dtype == torch.bfloat16 else O.F32)
    assert np.array_equal(to_np(codes), oc) and np.array_equal(to_np(scales), os_)
    ov = O.mx4_dequantize(oc, os_)
    assert np.isnan(ov).sum() == 96
    assert np.array_equal(values.double().cpu().numpy(), ov, equal_nan=True)
    assert np.array_equal(B.dequantize_mx4(codes, scales, dtype).double().cpu().numpy(), ov, equal_nan=True)
    # products: the rows (and tokens) that hold such a block are NaN, the others are not
    ok = np.array([0, 3, 5])
    for T in (5, 80):
        x, xv = tokens_of(T, 576)
        (y,) = B.base_gemm_mx4(x.to(DEV), [(codes, scales)])
        got = y.cpu().numpy()
        assert np.isnan(got[:, [1, 2, 4]]).all()
        assert_product(got[:, ok], xv, ov[ok])
        (y4,) = B.base_gemm_mx4x4(B.quantize_mx4(x.to(DEV)), [(codes, scales)])
        assert np.isnan(y4.cpu().numpy()[:, [1, 2, 4]]).all() and np.isfinite(y4.cpu().numpy()[:, ok]).all()
        x[3, 575] = float("inf")  # a token's infinity stays that token's
        for y in B.base_gemm_mx4(x.to(DEV), [(codes, scales)]) + \
                B.base_gemm_mx4x4(B.quantize_mx4(x.to(DEV)), [(codes, scales)]):
            fin = np.isfinite(y.cpu().numpy()[:, ok])
            assert not fin[3].any() and np.delete(fin, 3, 0).all()
    clean = base_of(16, 576)[0]
    (y4t,) = B.base_gemm_mx4x4((codes, scales), [clean])  # the same rows as tokens
    bad = np.isnan(y4t.cpu().numpy())
    assert bad[[1, 2, 4]].all() and not bad[ok].any()


def test_quantize_in_place_and_padding():
    """values_out may be w itself; the scales' padding is written (zeros)."""
    w = rand_w(9, 192, torch.bfloat16, seed=4).to(DEV)
    ref = B.quantize_mx4(w, values=True)
    codes = torch.empty_like(ref[0])
    scales = torch.full_like(ref[1], 77)
    assert B.bd_quantize_mx4(w, codes, scales, w) == B.BD_OK
    assert torch.equal(codes, ref[0]) and torch.equal(scales, ref[1]) and torch.equal(w, ref[2])
    assert not scales[:, 6:].any()
    empty = B.quantize_mx4(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV))
    assert empty[0].shape == (0, 64) and empty[1].shape == (0, 16)


# ----------------------------------------------------------------- products

TS = [1, 2, 15, 16, 17, 33, 64, 65, 129, 300]
SHAPES = [((1,), 64), ((17, 16), 192), ((130,), 512), ((33, 1, 64), 576), ((257,), 1088),
          ((48, 16, 16, 300), 4096), ((100,), 4160), ((40, 24), 14336)]


def run_product(x4, x, bases, guard=3, workspace=True):
    """(outputs, the tokens' values in binary64); every output stands in a larger buffer
    whose rest must stay as it was."""
    T, d_in = x.shape
    outs = [c.shape[0] for c, _ in bases]
    bufs = [torch.full((T * n + guard,), 7.5, device=DEV) for n in outs]
    ys = [b[:T * n].view(T, n) for b, n in zip(bufs, outs)]
    query = B.bd_base_gemm_mx4x4_n_workspace_bytes if x4 else B.bd_base_gemm_mx4_n_workspace_bytes
    need = query(T, d_in, outs) if workspace else 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV) if need else None
    if x4:
        xc, xs = B.quantize_mx4(x.to(DEV))
        xv = O.mx4_dequantize(to_np(xc), to_np(xs))
        st = B.bd_base_gemm_mx4x4_n(xc, xs, bases, ys, None if ws is None else ws[:need])
    else:
        xv = x.double().numpy()
        st = B.bd_base_gemm_mx4_n(x.to(DEV), bases, ys, None if ws is None else ws[:need])
    assert st == B.BD_OK
    torch.cuda.synchronize()
    for b, n in zip(bufs, outs):
        assert bool((b[T * n:] == 7.5).all()), "written past the output"
    if ws is not None:
        assert bool((ws[need:] == 0xFF).all()), "written past the workspace"
    return ys, xv


@pytest.mark.parametrize("x4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("d_outs,d_in", SHAPES, ids=lambda v: str(v).replace(" ", ""))
@pytest.mark.parametrize("T", TS)
def test_products_match_oracle(T, d_outs, d_in, x4):
    bases, vals = zip(*[base_of(n, d_in, seed=7 * i + n) for i, n in enumerate(d_outs)])
    x, _ = tokens_of(T, d_in, seed=T)
    for workspace in (True, False):
        ys, xv = run_product(x4, x, list(bases), workspace=workspace)
        for y, wv in zip(ys, vals):
            assert_product(y.cpu().numpy(), xv, wv, (T, d_outs, d_in, workspace))


TILE_CASES = [((14336,), 512, 512), ((4100, 300), 1088, 1000), ((700,), 1536, 333), ((4096,), 4096, 129),
              ((1024, 1024, 4096), 2048, 257), ((5120,), 8192, 70), ((160,), 64, 2100),
              ((2050,), 1088, 1000), ((2050,), 1088, 3000), ((5123,), 448, 2060), ((2050,), 2112, 4100),
              ((700,), 8256, 333), ((1000,), 8256, 257), ((2050,), 8256, 520), ((2050,), 8256, 1000)]


@pytest.mark.parametrize("x4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("d_outs,d_in,T", TILE_CASES, ids=lambda v: str(v).replace(" ", ""))
def test_products_over_tile_shapes(d_outs, d_in, T, x4):
    """Larger batches and matrices: every tile and split of the plan, ragged edges; all
    tokens of sampled rows, and the same bits from one call to the next."""
    rng = np.random.default_rng(T)
    bases = [B.quantize_mx4(torch.randn(n, d_in, device=DEV, generator=torch.Generator(DEV).manual_seed(n)))
             for n in d_outs]
    x, _ = tokens_of(T, d_in, seed=T)
    ys, xv = run_product(x4, x, bases)
    ys2, _ = run_product(x4, x, bases)
    for y, y2, (c, s) in zip(ys, ys2, bases):
        assert torch.equal(y, y2)
        n = c.shape[0]
        rows = sorted({0, n - 1} | set(rng.choice(n, min(n, 64), replace=False).tolist()))
        assert_product(y.cpu().numpy()[:, rows], xv, O.mx4_dequantize(to_np(c)[rows], to_np(s)[rows]))


@pytest.mark.parametrize("x4", [False, True], ids=["bf16", "mx4"])
def test_products_captured_and_on_another_stream(x4):
    """Two captured graphs with a workspace each, replayed in turn with other inputs, and
    eager work between the replays, against the eager call."""
    d_in, outs = 4096, (96, 33)
    bases = [base_of(n, d_in, seed=n)[0] for n in outs]
    made = []
    for T in (5, 80):
        x = tokens_of(T, d_in, seed=T)[0].to(DEV)
        ys = [torch.empty(T, n, device=DEV) for n in outs]
        query = B.bd_base_gemm_mx4x4_n_workspace_bytes if x4 else B.bd_base_gemm_mx4_n_workspace_bytes
        ws = B.workspace(query(T, d_in, outs), DEV)
        xc, xs = B.quantize_mx4(x)

        def call(x=x, xc=xc, xs=xs, ys=ys, ws=ws):
            if x4:
                assert B.bd_quantize_mx4(x, xc, xs) == B.BD_OK
                assert B.bd_base_gemm_mx4x4_n(xc, xs, bases, ys, ws) == B.BD_OK
            else:
                assert B.bd_base_gemm_mx4_n(x, bases, ys, ws) == B.BD_OK

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()  # on a stream of its own first
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        made.append((g, x, ys, call))  # (the graph's workspace and token buffers live in call)
    for rep in range(3):
        for g, x, ys, _ in made:
            x.copy_(tokens_of(x.shape[0], d_in, seed=100 + rep)[0])
            g.replay()
            got = [y.clone() for y in ys]
            want = B.base_gemm_mx4x4(B.quantize_mx4(x), bases) if x4 else B.base_gemm_mx4(x, bases)
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("as_int", [False, True], ids=["stream", "handle"])
def test_helpers_on_a_given_stream(as_int):
    """What a helper allocates for a call on another stream is that stream's: blocks that
    the current stream has freed with work on them still to run are not handed to it."""
    T, n, d_in = 80, 96, 4096
    base, _ = base_of(n, d_in)
    x = tokens_of(T, d_in, seed=3)[0].to(DEV)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side
    calls = [lambda s: B.base_gemm_mx4(x, [base], stream=s)[0],
             lambda s: B.base_gemm_mx4x4(B.quantize_mx4(x, stream=s), [base], stream=s)[0],
             lambda s: B.dequantize_mx4(*base, torch.float32, stream=s)]
    p = B.params("matrix")
    signs = torch.randint(-2 ** 62, 2 ** 62, (2, n, d_in // 64), device=DEV)
    sc = torch.rand(2, 1, device=DEV)
    ids = (torch.arange(T, device=DEV) % 2).int()
    calls += [lambda s: B.apply_mx4(x, *base, signs, sc, p, ids, stream=s, check=True),
              lambda s: B.apply_mx4(x, *base, signs, sc, p, ids, tokens="mx4", stream=s)]
    want = [f(None) for f in calls]

    def same(i, got, what):
        d = (got != want[i]).nonzero()
        assert d.shape[0] == 0, (what, i, d.shape[0], float((got - want[i]).abs().max()), d[:8].tolist())

    with pytest.raises(ValueError):
        B.base_gemm_mx4(x.cpu(), [base], stream=stream)  # the call's own refusal, not the stream's
    for i, f in enumerate(calls):  # the default stream's handle is 0: in order with what follows
        for _ in range(10):
            same(i, f(torch.cuda.default_stream().cuda_stream), "default stream")
    big = torch.ones(8192, 8192, device=DEV)
    for i, f in enumerate(calls):
        torch.cuda.synchronize()
        for _ in range(4):
            big @ big  # the current stream is busy ...
        junk = [torch.empty(m, dtype=torch.uint8, device=DEV) for m in [T * n * 4, n * d_in * 4] * 4 + [1 << 23] * 2]
        for j in junk:
            j.fill_(0xFF)
        del junk, j  # ... and these blocks, free for its next tensors, are still to be filled
        got = f(stream)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        same(i, got, "side stream")
        del got


def test_empty_batch():
    base = base_of(40, 128)[0]
    x = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    assert B.base_gemm_mx4(x, [base])[0].shape == (0, 40)
    assert B.base_gemm_mx4x4(B.quantize_mx4(x), [base])[0].shape == (0, 40)


# ------------------------------------------------------- multi-tenant apply

def seeded_ids(seed, T, U):
    return np.random.default_rng(seed).integers(-1, U, T).astype(np.int32)


APPLY = [
    # (mode, scale dtype, d_out, d_in, ids, n_users, y dtype)
    ("matrix", B.BD_F32, 200, 1024, np.random.default_rng(1).permutation(16).astype(np.int32), 16, torch.float32),
    ("matrix", B.BD_F32, 17, 64, np.array([0], np.int32), 1, torch.float32),
    ("row", B.BD_F16, 130, 1088, np.array([2, 0, -1, 2, 1, 2, 0], np.int32), 3, torch.bfloat16),
    ("matrix", B.BD_F32, 64, 4096, np.array([1, 1, 0], np.int32), 2, torch.float32),
    ("row", B.BD_F32, 33, 448, np.full(16, -1, np.int32), 2, torch.float32),
    ("matrix", B.BD_F32, 200, 1024, seeded_ids(2, 40, 4), 4, torch.float32),
    ("row", B.BD_F16, 130, 4608, np.array([0, 2, 1, 1, -1, 0, 2, 2, 0], np.int32), 3, torch.bfloat16),
    ("col", B.BD_F16, 96, 1088, seeded_ids(3, 12, 3), 3, torch.float32),
    ("group", B.BD_F32, 136, 2048, seeded_ids(4, 70, 5), 5, torch.float32),
    ("group", B.BD_F32, 136, 1024, seeded_ids(5, 9, 5), 5, torch.bfloat16),
    ("matrix", B.BD_F32, 300, 576, seeded_ids(6, 260, 7), 7, torch.bfloat16),
    ("col", B.BD_F32, 12288, 192, seeded_ids(7, 6, 3), 3, torch.bfloat16),
    ("col", B.BD_F32, 12291, 192, seeded_ids(7, 6, 3), 3, torch.float32),
    ("matrix", B.BD_F32, 80, 128, np.full(64, 1, np.int32), 2, torch.float32),
    ("row", B.BD_F32, 80, 128, np.full(65, 1, np.int32), 2, torch.bfloat16),
    ("matrix", B.BD_F32, 80, 128, seeded_ids(8, 1025, 40), 40, torch.float32),
    ("row", B.BD_F32, 48, 64, seeded_ids(9, 8192, 300), 300, torch.float32),
    ("matrix", B.BD_F32, 48, 64, np.full(8192, -1, np.int32), 1, torch.float32),
]


@pytest.mark.parametrize("tokens", ["bf16", "mx4"])
@pytest.mark.parametrize("case", APPLY, ids=lambda c: f"{c[0]}-{c[2]}x{c[3]}-T{len(c[4])}")
def test_quantize_compress_and_apply_together(case, tokens):
    """The run a user makes: the base quantised with its values, each user's delta
    compressed against those values, the batch applied on codes and banks."""
    mode, sd, d_out, d_in, ids, U, ydt = case
    T = len(ids)
    w = custom(d_out, d_in, S.BF16, n_users=U, T=T, b=5e-3, cid=2600 + d_out)
    p = B.params(mode, 128, 0.0, sd)
    x_dev = S.dev_x(w, 0)
    codes, scales, values = B.quantize_mx4(S.dev_wbase(w, 0), values=True)
    oc, os_ = O.mx4_quantize(S.host_wbase(w, 0), dtype=O.BF16)
    assert np.array_equal(to_np(codes), oc) and np.array_equal(to_np(scales), os_)
    ov = O.mx4_dequantize(oc, os_)
    vb = to_np(values)
    assert np.array_equal(bf16_to_f64(vb), ov)
    signs, dsc = gpu_bank(w, 0, values, p, range(U))
    words, osc = oracle_bank(w, 0, vb, p, range(U))
    assert np.array_equal(to_np(signs), words)
    ids_dev = torch.from_numpy(ids).to(DEV)
    y = B.apply_mx4(x_dev, codes, scales, signs, dsc, p, ids_dev, y_dtype=ydt, tokens=tokens, check=True)
    y0 = B.apply_mx4(x_dev, torch.zeros_like(codes), scales, signs, dsc, p, ids_dev, tokens=tokens,
                     check=True)
    torch.cuda.synchronize()
    xb = S.host_x(w, 0)
    _, yb, yd = O.apply(xb, vb, words, osc, p.mode, ids, g=128, sdtype=o_sdtype(p), xdtype=O.BF16,
                        wdtype=O.BF16)
    if tokens == "mx4":
        yb = O.mx4_dequantize(*O.mx4_quantize(xb, dtype=O.BF16)) @ ov.T
    yr = yb + yd
    err, rms = max_err_vs_rms(y.float().cpu().numpy(), yr)
    assert err <= TOL_BF16 * rms, (err, rms)
    g0 = y0.cpu().numpy()
    if (ids >= 0).any():
        err0, rms0 = max_err_vs_rms(g0, yd)
        assert err0 <= tol_delta(mode) * rms0, (err0, rms0)
        assert_delta_within_bound(g0, yd, xb, osc, p, ids)
    assert np.all(g0[ids < 0] == 0)
    # tokens of the base model: the base product alone, within its own bar
    if (ids < 0).any() and ydt == torch.float32:
        xv = O.mx4_dequantize(*O.mx4_quantize(xb, dtype=O.BF16)) if tokens == "mx4" else bf16_to_f64(xb)
        assert_product(y.cpu().numpy()[ids < 0], xv[ids < 0], ov)


@pytest.mark.parametrize("tokens", ["bf16", "mx4"])
@pytest.mark.parametrize("T", [1, 16, 70])
def test_apply_reports_bad_user_ids(T, tokens):
    w = custom(48, 512, S.BF16, n_users=2, T=T, b=5e-3, cid=2700)
    p = B.params("row")
    codes, scales, values = B.quantize_mx4(S.dev_wbase(w, 0), values=True)
    signs, dsc = gpu_bank(w, 0, values, p, range(2))
    ids = torch.full((T,), 2, dtype=torch.int32, device=DEV)  # outside [0, 2)
    y = torch.empty(T, 48, device=DEV)
    ws = B.workspace(B.bd_apply_mx4_workspace_bytes(p, T, 2, 48, 512, B.BD_BF16, B.BD_F32, tokens), DEV)
    x = S.dev_x(w, 0)
    assert B.bd_apply_mx4(x, codes, scales, signs, dsc, p, 2, ids, y, ws, tokens) == B.BD_OK
    assert B.bd_device_status(ws) == B.BD_ERR_USER_ID
    xv = O.mx4_dequantize(*O.mx4_quantize(S.host_x(w, 0), dtype=O.BF16)) if tokens == "mx4" \
        else bf16_to_f64(S.host_x(w, 0))
    assert_product(y.cpu().numpy(), xv, O.mx4_dequantize(to_np(codes), to_np(scales)))


@pytest.mark.parametrize("tokens", ["bf16", "mx4"])
@pytest.mark.parametrize("T,mode", [(9, "matrix"), (9, "col"), (130, "row")])
def test_apply_repeats_and_replays(T, mode, tokens):
    w = custom(72, 1088, S.BF16, n_users=3, T=T, b=5e-3, cid=2750)
    p = B.params(mode)
    codes, scales, values = B.quantize_mx4(S.dev_wbase(w, 0), values=True)
    signs, dsc = gpu_bank(w, 0, values, p, range(3))
    ids = torch.from_numpy(seeded_ids(T, T, 3)).to(DEV)
    x = S.dev_x(w, 0)
    y = torch.empty(T, 72, dtype=torch.bfloat16, device=DEV)
    ws = B.workspace(B.bd_apply_mx4_workspace_bytes(p, T, 3, 72, 1088, B.BD_BF16, B.BD_BF16, tokens), DEV)
    assert B.bd_apply_mx4(x, codes, scales, signs, dsc, p, 3, ids, y, ws, tokens) == B.BD_OK
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert B.bd_apply_mx4(x, codes, scales, signs, dsc, p, 3, ids, y, ws, tokens) == B.BD_OK
    for rep in range(3):
        x.copy_(x.roll(1, 0))
        y.fill_(float("nan"))
        g.replay()
        want = B.apply_mx4(x, codes, scales, signs, dsc, p, ids, y_dtype=torch.bfloat16, tokens=tokens)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    empty = B.apply_mx4(x[:0], codes, scales, signs, dsc, p, ids[:0], tokens=tokens, check=True)
    assert empty.shape == (0, 72)
