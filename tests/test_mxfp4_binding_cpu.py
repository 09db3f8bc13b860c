"""CPU-only checks of the MXFP4 and norm bindings: what they hand to the C calls."""
import pytest
import torch

import hadamard_rotation_int4_amd as hr

LONG = 2 ** 32 + 64


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_the_c_type_of_a_row_length_is_too_short_for_it():
    """What a call without the check below would do: the call sees 64 elements."""
    p = 0x10000
    assert hr.lib.hr_quant_mxfp4(p, hr.HR_BF16, LONG, 0, 2 ** 20, 0, p, p, None) == hr.HR_EUNSUPPORTED
    assert hr.lib.hr_quant_mxfp4(p, hr.HR_BF16, LONG, 0, LONG, 0, p, p, None) == hr.HR_OK


@pytest.mark.parametrize("call", [
    lambda n: hr.quant_mxfp4(_meta(1, n)),
    lambda n: hr.rotate_quant_mxfp4(_meta(1, n), 64),
    lambda n: hr.dequant_mxfp4(_meta(1, n // 2, dtype=torch.uint8), _meta(1, n // 32, dtype=torch.uint8)),
    lambda n: hr.norm_residual(_meta(1, n)),
    lambda n: hr.norm_residual(_meta(2, n), _meta(2, n)),
    lambda n: hr.norm_residual_quant_mxfp4(_meta(1, n)),
])
@pytest.mark.parametrize("n", [2 ** 31, LONG])
def test_rows_past_the_c_type_are_refused(call, n):
    """Not cut to it: 2^32 + 64 elements would run as 64."""
    with pytest.raises(ValueError, match=f"rows of {n} elements"):
        call(n)


def test_outputs_where_the_quick_way_takes_other_arguments(monkeypatch):
    """A private function of torch that has changed is left alone from then on; running
    out of memory is not that."""
    calls, made = [], []

    def other(size, stride, dtype, device):
        calls.append(size)

    def full(*a):
        raise torch.OutOfMemoryError("out of memory")

    monkeypatch.setattr(hr, "_get_device", lambda: 0)
    monkeypatch.setattr(hr, "_empty_cuda", full)
    with pytest.raises(torch.OutOfMemoryError):
        hr._new(0, 3, 5, torch.uint8)
    assert hr._empty_cuda is full
    monkeypatch.setattr(hr, "_empty_cuda", other)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append((a, k)))
    for _ in range(2):
        hr._new(0, 3, 5, torch.uint8)
    want = (((3, 5),), {"dtype": torch.uint8, "device": torch.device("cuda", 0)})
    assert made == [want, want] and hr._empty_cuda is None and not calls
