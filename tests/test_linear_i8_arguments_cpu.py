"""Arguments of the channel products that contradict each other are refused by the binding, without a GPU."""
import pytest
import torch

import sparse_gather_contraction_amd as sgc

Q, S = torch.zeros((6, 32), dtype=torch.int8), torch.ones(6)
W, WS = torch.zeros((4, 32), dtype=torch.int8), torch.ones(4)
GY = torch.zeros((6, 4), dtype=torch.bfloat16)
FIELD, FS = torch.zeros((2, 3, 5, 32), dtype=torch.int8), torch.ones(2, 3, 5)


# each output is one that its call takes, but not of as many channels as are asked for
@pytest.mark.parametrize("call", [
    lambda: sgc.disco_dequantize_i8(Q, S, channels=20, out=torch.zeros((6, 21), dtype=torch.bfloat16)),
    lambda: sgc.disco_dequantize_i8(FIELD, FS, channels=20, out=torch.zeros((2, 30, 3, 5), dtype=torch.bfloat16)),
    lambda: sgc.disco_dequantize_i8(FIELD, FS, channels=20, axis=-1, out=torch.zeros((2, 3, 5, 30), dtype=torch.bfloat16)),
    lambda: sgc.disco_linear_i8_bwd_input(GY, W, WS, channels=20, gx=torch.zeros((6, 32), dtype=torch.bfloat16)),
    lambda: sgc.disco_linear_i8_bwd_weight(GY, Q, S, channels=20, dw=torch.zeros((4, 32), dtype=torch.bfloat16)),
], ids=["dequantize rows", "dequantize field", "dequantize last", "bwd_input", "bwd_weight"])
def test_channels_that_a_given_output_does_not_have(call):
    with pytest.raises(sgc.DiscoError) as e:
        call()
    assert e.value.status_name == "DISCO_ERR_SHAPE" and "channels" in str(e.value)


@pytest.mark.parametrize("call", [
    lambda: sgc.disco_dequantize_i8(Q, S, channels=20, out=torch.zeros((6, 20), dtype=torch.bfloat16)),
    lambda: sgc.disco_dequantize_i8(FIELD, FS, channels=20, axis=-1, out=torch.zeros((2, 3, 5, 20), dtype=torch.bfloat16)),
    lambda: sgc.disco_dequantize_i8(Q, S, out=torch.zeros((6, 20), dtype=torch.bfloat16)),
    lambda: sgc.disco_linear_i8_bwd_input(GY, W, WS, channels=20, gx=torch.zeros((6, 20), dtype=torch.bfloat16)),
    lambda: sgc.disco_linear_i8_bwd_weight(GY, Q, S, channels=20, dw=torch.zeros((4, 20), dtype=torch.bfloat16)),
], ids=["dequantize", "dequantize last", "not asked for", "bwd_input", "bwd_weight"])
def test_channels_that_agree_pass_on_to_the_device_check(call):
    with pytest.raises(sgc.DiscoError) as e:   # host memory: refused where the shapes are in order
        call()
    assert e.value.status_name != "DISCO_ERR_SHAPE"


def test_what_is_no_tensor_is_a_type_error_as_before():
    for call in (lambda: sgc.disco_dequantize_i8(Q, S, channels=20, out=[1.0]), lambda: sgc.disco_dequantize_i8(Q, S, channels=20, axis="1"),
                 lambda: sgc.disco_linear_i8_bwd_weight(GY, Q, S, channels=20, dw=1.0)):
        with pytest.raises(TypeError):
            call()
