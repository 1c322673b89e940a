"""bd_batch_prepare at the C entry: x is not read for bf16 batches and may be NULL."""
import numpy as np
import pytest
import torch

from gpu_util import DEV
from tenant_serving_amd import bitdelta as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,U", [(1, 1), (64, 5), (65, 5), (700, 40)])
def test_bf16_batch_without_tokens(T, U):
    """The same batch, byte for byte, with and without the token pointer."""
    ids = torch.from_numpy(np.random.default_rng(T).integers(-1, U, T).astype(np.int32)).to(DEV)
    x = torch.zeros(T, 128, dtype=torch.bfloat16, device=DEV)
    need = B.bd_batch_workspace_bytes(T, U, 128, B.BD_BF16)
    got = []
    for ptr in (x.data_ptr(), None):
        ws = torch.full((need,), 0x5A, dtype=torch.uint8, device=DEV)
        st = B.lib().bd_batch_prepare(ptr, B.BD_BF16, T, 128, ids.data_ptr(), U, ws.data_ptr(), need,
                                      torch.cuda.current_stream().cuda_stream)
        assert int(st) == B.BD_OK
        assert B.bd_device_status(ws) == B.BD_OK
        got.append(ws)
    assert torch.equal(*got)
    assert int(B.lib().bd_batch_prepare(None, B.BD_F32, T, 128, ids.data_ptr(), U, got[0].data_ptr(), 1 << 40,
                                        None)) == B.BD_ERR_INVALID_ARG
