"""What the layer for a few tokens says to weights of other types and to a backward that
it does not have.  No GPU needed."""
import pytest
import torch

OTHER = [torch.float16, torch.float64, torch.int32, torch.float8_e4m3fn]


@pytest.mark.parametrize("dt", OTHER)
def test_workspace_size_refuses_other_types(dt):
    import padding_free_expert_amd as xm
    with pytest.raises(TypeError, match="dtype"):
        xm.xmoe_layer_few_workspace_size(4, 64, 8, 2, 32, 0, dt)
    for good in (torch.bfloat16, torch.float32):
        assert xm.xmoe_layer_few_workspace_size(4, 64, 8, 2, 32, 0, good) > 0


@pytest.mark.parametrize("dt", OTHER)
def test_layer_refuses_weights_of_other_types(dt):
    from padding_free_expert_amd.layer import PaddingFreeMoE
    e = lambda *s: torch.empty(s, dtype=dt)
    w = dict(wg=e(64, 8), w1=e(8, 64, 32), w3=e(8, 64, 32), w2=e(8, 32, 64))
    with pytest.raises(TypeError, match="dtype"):
        PaddingFreeMoE(w, 4, 2, backward=False, few=True)


def test_a_layer_for_few_tokens_has_no_backward():
    from padding_free_expert_amd.layer import PaddingFreeMoE
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16)
    w = dict(wg=e(64, 8), w1=e(8, 64, 32), w3=e(8, 64, 32), w2=e(8, 32, 64))
    layer = PaddingFreeMoE(w, 4, 2, backward=False, few=True)
    with pytest.raises(RuntimeError, match="no backward"):
        layer.backward(e(4, 64))
