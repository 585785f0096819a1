"""layer_norm_bwd at the edges of what its checks accept."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,code", [(BF, txl.TXL_BF16), (F32, txl.TXL_F32)])
@pytest.mark.parametrize("d", [1, 64, 130, 512, 1001, 16384])
def test_no_rows_need_no_gamma(dtype, code, d):
    """Without rows gamma is not read, so it may be null or start off the alignment:
    zeros in dgamma and dbeta, and nothing around them written."""
    out = torch.full((2, 16640), 7.0, device="cuda")
    rc = txl.load().txl_layer_norm_bwd(None, None, None, None, None, None, None, 0, d, None, out[0].data_ptr(),
                                       out[1].data_ptr(), code, None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and not out[:, :d].any() and bool((out[:, d:] == 7).all())
    x = torch.empty(0, d, dtype=dtype, device="cuda")
    gamma = torch.ones(d + 1, dtype=dtype, device="cuda")[1:]
    got = txl.layer_norm_bwd(x, x, gamma, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"))
    torch.cuda.synchronize()
    assert got["dx"].shape == (0, d) and not got["dgamma"].any() and not got["dbeta"].any()
    assert txl.sync_status() == 0
