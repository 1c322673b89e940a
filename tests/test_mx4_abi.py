"""The MX4 entry points' checks on the host: every call below fails validation (fake,
never dereferenced device addresses), so no kernel is launched; the binding's checks of
tensors run on host tensors."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tenant_serving_amd import bitdelta as B  # noqa: E402

A = 1 << 12  # an aligned fake address


def test_scale_stride():
    assert B.bd_mx4_scale_stride(64) == 16
    assert B.bd_mx4_scale_stride(512) == 16
    assert B.bd_mx4_scale_stride(576) == 32
    assert B.bd_mx4_scale_stride(17408) == 17408 // 32
    for bad in (0, -64, 32, 100):
        assert B.bd_mx4_scale_stride(bad) == 0


def test_quantize_and_dequantize_refusals():
    L = B.lib()

    def q(w=A, dt=B.BD_BF16, rows=4, cols=128, c=A, s=A, v=None):
        return int(L.bd_quantize_mx4(w, dt, rows, cols, c, s, v, None))

    def d(c=A, s=A, rows=4, cols=128, o=A, dt=B.BD_F32):
        return int(L.bd_dequantize_mx4(c, s, rows, cols, o, dt, None))

    assert q(dt=B.BD_F16) == B.BD_ERR_DTYPE and d(dt=B.BD_F16) == B.BD_ERR_DTYPE
    assert q(dt=7) == B.BD_ERR_DTYPE
    for f in (q, d):
        assert f(rows=-1) == B.BD_ERR_INVALID_ARG
        assert f(cols=96) == B.BD_ERR_SHAPE
        assert f(cols=0) == B.BD_ERR_SHAPE
        assert f(cols=-64) == B.BD_ERR_SHAPE
        assert f(rows=1 << 31) == B.BD_ERR_SHAPE
        assert f(c=None) == B.BD_ERR_INVALID_ARG
        assert f(s=A + 8) == B.BD_ERR_INVALID_ARG
        assert f(c=A + 4) == B.BD_ERR_INVALID_ARG
        assert f(rows=0, c=None) == B.BD_OK  # nothing to do
    assert q(w=None) == B.BD_ERR_INVALID_ARG
    assert q(w=A + 2) == B.BD_ERR_INVALID_ARG
    assert q(v=A + 2) == B.BD_ERR_INVALID_ARG
    assert d(o=None) == B.BD_ERR_INVALID_ARG
    assert d(o=A + 4) == B.BD_ERR_INVALID_ARG


def test_product_refusals():
    L = B.lib()
    P, N = ctypes.c_void_p * 4, ctypes.c_int64 * 4

    def args(n, w, s, d, y, ws, wsb):
        return (n, P(*[w] * 4), P(*[s] * 4), N(*[d] * 4), P(*[y] * 4), ws, wsb, None)

    def g(x=A, xd=B.BD_BF16, T=8, d_in=128, n=2, w=A, s=A, d=64, y=A, ws=None, wsb=0):
        return int(L.bd_base_gemm_mx4_n(x, xd, T, d_in, *args(n, w, s, d, y, ws, wsb)))

    def g4(x=A, xs=A, T=8, d_in=128, n=2, w=A, s=A, d=64, y=A, ws=None, wsb=0):
        return int(L.bd_base_gemm_mx4x4_n(x, xs, T, d_in, *args(n, w, s, d, y, ws, wsb)))

    assert g(xd=B.BD_F32) == B.BD_ERR_DTYPE
    assert g4(xs=None) == B.BD_ERR_INVALID_ARG
    assert g4(xs=A + 8) == B.BD_ERR_INVALID_ARG
    for f in (g, g4):
        assert f(T=-1) == B.BD_ERR_INVALID_ARG
        assert f(n=0) == B.BD_ERR_INVALID_ARG
        assert f(n=5) == B.BD_ERR_INVALID_ARG
        assert f(d_in=96) == B.BD_ERR_SHAPE
        assert f(d=0) == B.BD_ERR_SHAPE
        assert f(d_in=1 << 20, d=1 << 13) == B.BD_ERR_UNSUPPORTED  # 32-bit offsets
        assert f(T=1 << 19, d_in=1 << 14) == B.BD_ERR_UNSUPPORTED
        assert f(d_in=1 << 62, d=4) == B.BD_ERR_UNSUPPORTED  # sizes whose product wraps to 0
        assert f(T=1 << 58) == B.BD_ERR_UNSUPPORTED
        assert f(d=1 << 58) == B.BD_ERR_UNSUPPORTED
        assert f(x=None) == B.BD_ERR_INVALID_ARG
        assert f(x=A + 8) == B.BD_ERR_INVALID_ARG
        assert f(w=None) == B.BD_ERR_INVALID_ARG
        assert f(w=A + 8) == B.BD_ERR_INVALID_ARG
        assert f(s=A + 8) == B.BD_ERR_INVALID_ARG
        assert f(y=A + 4) == B.BD_ERR_INVALID_ARG
        assert f(T=0, x=None) == B.BD_OK
    for query in (B.bd_base_gemm_mx4_n_workspace_bytes, B.bd_base_gemm_mx4x4_n_workspace_bytes):
        assert query(0, 128, [64]) == 0
        assert query(8, 96, [64]) == 0
        assert query(8, 128, [0]) == 0
        assert query(8, 128, [64] * 5) == 0
    # a workspace smaller than the query, or misaligned, is refused where K is split
    for query, f in ((B.bd_base_gemm_mx4_n_workspace_bytes, g),
                     (B.bd_base_gemm_mx4x4_n_workspace_bytes, g4)):
        need = query(64, 17408, [256, 256])
        if need:
            assert f(T=64, d_in=17408, d=256, ws=A, wsb=need - 1) == B.BD_ERR_WORKSPACE
            assert f(T=64, d_in=17408, d=256, ws=A + 16, wsb=need) == B.BD_ERR_WORKSPACE


def test_apply_refusals():
    L = B.lib()

    def ap(p=B.params("matrix"), xd=B.BD_BF16, T=4, d_in=512, wc=A, wsc=A, U=2, yd=B.BD_F32,
           tok=B.BD_MX4_TOKENS_BF16, ids=A, bank=A, y=A, ws=1 << 16, wsb=1 << 30):
        return int(L.bd_apply_mx4(A, xd, T, d_in, wc, wsc, 64, bank, A,
                                  None if p is None else ctypes.byref(p), U, ids, y, yd, tok, ws, wsb,
                                  None))

    assert ap(p=None) == B.BD_ERR_INVALID_ARG
    assert ap(tok=2) == B.BD_ERR_INVALID_ARG
    assert ap(tok=-1) == B.BD_ERR_INVALID_ARG
    assert ap(p=B.params("group", 256), d_in=384) == B.BD_ERR_SHAPE
    assert ap(p=B.params("group", 100)) == B.BD_ERR_UNSUPPORTED
    assert ap(T=9000) == B.BD_ERR_UNSUPPORTED
    assert ap(T=-1) == B.BD_ERR_INVALID_ARG
    assert ap(xd=B.BD_F32) == B.BD_ERR_UNSUPPORTED
    assert ap(yd=B.BD_F16) == B.BD_ERR_DTYPE
    assert ap(d_in=100) == B.BD_ERR_SHAPE
    assert ap(ws=0) == B.BD_ERR_WORKSPACE
    assert ap(ws=(1 << 16) + 16) == B.BD_ERR_WORKSPACE
    assert ap(wc=None) == B.BD_ERR_INVALID_ARG
    assert ap(wc=A + 8) == B.BD_ERR_INVALID_ARG
    assert ap(wsc=A + 8) == B.BD_ERR_INVALID_ARG
    assert ap(ids=None) == B.BD_ERR_INVALID_ARG
    assert ap(ids=A + 2) == B.BD_ERR_INVALID_ARG
    assert ap(bank=None) == B.BD_ERR_INVALID_ARG
    assert ap(y=A + 2) == B.BD_ERR_INVALID_ARG
    for tok in ("bf16", "mx4"):
        for T, d_in, mode in ((4, 512, "row"), (40, 4608, "col"), (8192, 576, "matrix")):
            p = B.params(mode)
            need = B.bd_apply_mx4_workspace_bytes(p, T, 2, 64, d_in, B.BD_BF16, B.BD_BF16, tok)
            assert need > 0
            assert ap(p=p, T=T, d_in=d_in, yd=B.BD_BF16, tok=B.MX4_TOKENS[tok],
                      wsb=need - 1) == B.BD_ERR_WORKSPACE
    assert B.bd_apply_mx4_workspace_bytes(B.params(), 4, 2, 64, 96, B.BD_BF16, B.BD_F32) == 0


def test_binding_checks_tensors():
    bf, u8 = torch.bfloat16, torch.uint8
    w = torch.zeros(8, 128, dtype=bf)
    c, s = torch.zeros(8, 64, dtype=u8), torch.zeros(8, 16, dtype=u8)
    for call in (lambda: B.quantize_mx4(w), lambda: B.dequantize_mx4(c, s),
                 lambda: B.base_gemm_mx4(w, [(c, s)], ws=torch.zeros(256, dtype=u8)),
                 lambda: B.base_gemm_mx4x4((c, s), [(c, s)], ws=torch.zeros(256, dtype=u8))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        B.quantize_mx4(w.half())
    with pytest.raises(TypeError):
        B._mx4(c.to(torch.int8), s, "base")
    with pytest.raises(ValueError, match="expected \\(rows"):
        B._mx4(c, s, "base", cols=192)
    with pytest.raises(ValueError, match="contiguous"):
        B._dev(c.t(), "base codes", (u8,))
    with pytest.raises(ValueError, match="1..4 matrices"):
        B._mx4_bases([], 0, 128)
    with pytest.raises(ValueError, match="tokens is"):
        B._tokens("fp8")
