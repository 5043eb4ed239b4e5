"""rotary gives gradients to q and k alone: a table that asks for one is refused, not left without it."""
import pytest
import torch


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


@pytest.mark.parametrize("which", ["cos", "sin", "both", "computed"])
@pytest.mark.parametrize("call", ["rotary", "attn_rotary"])
def test_a_table_that_asks_for_a_gradient_is_refused(ea, which, call):
    q = torch.zeros(4, 2, 64).bfloat16()
    cos, sin = torch.ones(8, 32), torch.zeros(8, 32)
    if which in ("cos", "both"):
        cos.requires_grad_()
    if which in ("sin", "both"):
        sin.requires_grad_()
    if which == "computed":
        cos = torch.zeros(8, 32, requires_grad=True).cos()
    for k in (q, None):
        with pytest.raises(ValueError, match="gradient"):
            getattr(ea, call)(q, k, cos, sin)


def test_not_where_no_gradient_is_recorded(ea):
    """The call then gets as far as the tensors' own checks."""
    q = torch.zeros(4, 2, 64).bfloat16()
    cos, sin = torch.ones(8, 32, requires_grad=True), torch.zeros(8, 32)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        ea.rotary(q, q, cos, sin)
