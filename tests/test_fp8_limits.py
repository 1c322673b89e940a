"""The ends of the sizes that the FP8 calls take, as the header states them: refused on the host
(fake addresses, never dereferenced: a size that is taken meets the refusal of a NULL operand)."""
import ctypes

import pytest

pytest.importorskip("torch")

from tenant_serving_amd import bitdelta as B  # noqa: E402

A = 1 << 12


def product(T, d_in, d=64):
    P, N = ctypes.c_void_p * 1, ctypes.c_int64 * 1
    return int(B.lib().bd_base_gemm_fp8_n(None, A, T, d_in, 1, P(A), P(A), N(d), P(A), B.BD_F32, None, 0, None))


@pytest.mark.parametrize("T,d_in,d,taken", [
    ((1 << 20) - 1, 64, 64, True), (1 << 20, 64, 64, False),          # tokens
    ((1 << 15) - 1, 1 << 16, 64, True), (1 << 15, 1 << 16, 64, False),  # an operand's bytes: the tokens'
    (1, 1 << 11, (1 << 20) - 1, True), (1, 1 << 11, 1 << 20, False),    # ... and a matrix's
    (1, 64, (1 << 22) - 1, True), (1, 64, 1 << 22, False),            # rows
    (1, 1 << 22, 64, True), (1, (1 << 22) + 64, 64, False),           # columns
])
def test_products(T, d_in, d, taken):
    assert product(T, d_in, d) == (B.BD_ERR_INVALID_ARG if taken else B.BD_ERR_UNSUPPORTED)
    if not taken:
        assert B.bd_base_gemm_fp8_n_workspace_bytes(T, d_in, [d]) == 0


def test_quantised_weights():
    """Under 2^24 blocks of 128 x 128."""
    def q(rows, cols):
        return int(B.lib().bd_quantize_fp8(None, B.BD_BF16, rows, cols, A, A, None, None))

    assert q(128, 1 << 30) == B.BD_ERR_INVALID_ARG  # 2^23 of them
    assert q(129, 1 << 30) == B.BD_ERR_UNSUPPORTED
    assert q(((1 << 24) - 1) * 128, 64) == B.BD_ERR_INVALID_ARG
    assert q(((1 << 24) - 1) * 128 + 1, 64) == B.BD_ERR_UNSUPPORTED


def test_norm():
    def n(T, d):
        return int(B.lib().bd_rmsnorm_fp8(None, B.BD_BF16, None, 0, A, B.BD_BF16, T, d, 1e-6, None, A, A, A, None))

    assert n((1 << 22) - 1, 64) == B.BD_ERR_INVALID_ARG and n(1 << 22, 64) == B.BD_ERR_UNSUPPORTED
    assert n(1, 32768) == B.BD_ERR_INVALID_ARG and n(1, 32768 + 64) == B.BD_ERR_UNSUPPORTED
