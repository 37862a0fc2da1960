"""CPU tests: every tensor that an operator's binding needs, left out, is refused as a missing
argument.  The place is set to the CPU's (device -1), and the library is never reached."""
import pytest

from expert_slot_cache_amd import binding

torch = pytest.importorskip("torch")


def tensors(call):
    f32 = lambda *s: torch.zeros(s)                                  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)               # noqa: E731
    f8 = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)        # noqa: E731
    return {
        "route": dict(logits=f32(4, 8), topk_ids=i32(4, 2), topk_w=f32(4, 2)),
        "route_backward": dict(logits=f32(4, 8), topk_ids=i32(4, 2), topk_w=f32(4, 2), d_topk_w=f32(4, 2), d_logits=f32(4, 8)),
        "sort_tokens": dict(x=f32(4, 16), topk_ids=i32(4, 2), sorted_x=f32(8, 16), offsets=i32(9), rows=i32(4, 2)),
        "combine_rows": dict(ys=f32(8, 16), rows=i32(4, 2), out=f32(4, 16)),
        "combine_rows_backward": dict(d_out=f32(4, 16), ys=f32(8, 16), rows=i32(4, 2), topk_w=f32(4, 2), d_ys=f32(8, 16),
                                      d_topk_w=f32(4, 2)),
        "scaled_product": dict(x=f8(4, 32), x_scales=f32(4, 1), w=f8(1, 256, 32), w_scales=f32(1, 2, 1), out=f32(4, 256)),
    }[call]


class Reached(Exception):
    pass


class NoLibrary:
    def moe_sort_workspace_bytes(self, *_):
        return 0

    def __getattr__(self, name):
        raise Reached(name)


MISSING = [(call, name) for call in ("route", "route_backward", "sort_tokens", "combine_rows", "combine_rows_backward",
                                     "scaled_product") for name in tensors(call)
           if (call, name) not in (("route_backward", "logits"), ("sort_tokens", "x"))]     # these two may be left out


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(binding, "_place", lambda torch, stream: (-1, None))
    monkeypatch.setattr(binding, "lib", lambda: NoLibrary())


@pytest.mark.parametrize("call,name", MISSING)
def test_a_missing_tensor_is_refused(on_cpu, call, name):
    args = tensors(call)
    with pytest.raises(Reached):
        getattr(binding, call)(**args)                # as they are, they pass
    args[name] = None
    with pytest.raises(binding.MoeError, match=f"{name} is missing") as e:
        getattr(binding, call)(**args)
    assert e.value.status == binding.EINVAL


def test_a_missing_swiglu_output_is_refused(on_cpu):
    args = dict(tensors("scaled_product"), out=None, swiglu_scales=torch.zeros(4, 1))
    with pytest.raises(binding.MoeError, match="out is missing"):
        binding.scaled_product(**args)
