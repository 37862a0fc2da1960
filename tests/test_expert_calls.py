"""CPU tests of the expert products' binding: tensors of a type that the library does not know are
refused, whatever else the call leaves out (nothing is launched)."""
import pytest

from expert_slot_cache_amd import binding
from test_expert_refusals import on_cpu, tensors  # noqa: F401

torch = pytest.importorskip("torch")

OTHER = [torch.float16, torch.float64, torch.int32]


@pytest.mark.parametrize("kind", OTHER)
@pytest.mark.parametrize("act", ["none", "relu", "swiglu"])
@pytest.mark.parametrize("wanted", ["both", "d_bias", "d_pre"])
def test_activation_backward_knows_the_type_of_pre(on_cpu, kind, act, wanted):  # noqa: F811
    """With the bias' gradient alone nothing else names the type of pre: half as many bytes as fp32
    would be read past their end."""
    args = dict(tensors("activation_backward"), act=act)
    if act == "swiglu":
        args["d_out"] = torch.zeros(8, 12)
    args["pre"] = args["pre"].to(kind)
    if wanted == "d_bias":
        args["d_pre"] = None
    elif wanted == "d_pre":
        args["d_bias"] = None
    with pytest.raises(binding.MoeError):
        binding.activation_backward(**args)


@pytest.mark.parametrize("call,name", [("expert_product", "x"), ("expert_product", "out"), ("activation_backward", "d_out"),
                                       ("activation_backward", "d_pre"), ("expert_product_backward", "d_pre"),
                                       ("expert_product_backward", "d_w"), ("route_groups", "logits"),
                                       ("route_groups_backward", "d_logits")])
@pytest.mark.parametrize("kind", OTHER)
def test_other_types_are_refused(on_cpu, call, name, kind):  # noqa: F811
    good = tensors(call)
    with pytest.raises(binding.MoeError):
        getattr(binding, call)(**dict(good, **{name: good[name].to(kind)}))


def test_a_workspace_for_sizes_that_are_refused_is_none():
    f = binding.activation_backward_workspace_bytes
    assert f(100, 4, 64) > 0 and f(100, 4, 4) > 0      # 4 columns are a piece of fp32
    assert f(100, 4, 5) == 0 and f(100, 4, 62) == 0    # no format has such rows
    assert f(1 << 24, 1, 1 << 12) > 0 and f(1 << 24, 1, 1 << 13) == 0    # 2^36 values are the most
    assert f(100, 4, (1 << 18) + 4) == 0 and f((1 << 24) + 1, 4, 64) == 0 and f(100, 4097, 64) == 0
