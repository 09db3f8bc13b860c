"""Rows longer than the C calls' 32-bit lengths are refused by the binding, not cut to them."""
import pytest
import torch

import hadamard_rotation_int4_amd as hr


def _meta(n, dtype=torch.bfloat16):
    return torch.empty((1, n), dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda n: hr.rotate(_meta(n)),
    lambda n: hr.rotate_quant_int4(_meta(n), 64),
    lambda n: hr.rotate_quant_int8(_meta(n), 64),
    lambda n: hr.quant_int4(_meta(n), 64),
    lambda n: hr.quant_int8(_meta(n), 64),
    lambda n: hr.harp_apply(_meta(n, torch.float32), (2, 2), _meta(8, torch.float32)),
    lambda n: hr.dequant_int4(_meta(n, torch.uint8), _meta(n // 32, torch.float16), 64),
    lambda n: hr.rotate_quant_fp6(_meta(n), 64),
    lambda n: hr.w4a4_to_fp6(_meta(n, torch.uint8)),
])
@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 2048])
def test_rows_past_the_c_type_are_refused(call, n):
    with pytest.raises(ValueError, match=f"rows of {n} elements"):
        call(n)
