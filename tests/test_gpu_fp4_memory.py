"""An output or a workspace that the device has no room for is torch's own error, as
on the other routes, and leaves the library usable."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8

pytestmark = pytest.mark.gpu


def test_no_room_for_an_output():
    rows = i8.FP4Rows.empty(1 << 22, 32, "mxfp4")        # 4M channels: an output of 2^22 x 2^22 is 35 TB
    x = torch.zeros(1 << 22, 32, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(1, 1, 64, device="cuda", dtype=torch.bfloat16)
    for call in (lambda: i8.linear_fp4(x, rows), lambda: i8.gemm_fp4_bias_bf16(rows, rows),
                 lambda: i8.gated_linear_fp4(x, rows, rows), lambda: i8.gemm_fp4_gated_bf16(rows, rows, rows)):
        with pytest.raises(torch.OutOfMemoryError):
            call()
    w = torch.zeros(8, 64, device="cuda").bfloat16()
    y = i8.linear_fp4(q[0], i8.quant_rows_fp4(w, "mxfp4"))
    assert not y.any()
    i8.sync_check()

