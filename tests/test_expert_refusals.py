"""CPU tests of the argument checks of the grouped router and the expert products: every refused
call returns before any GPU call (the addresses below are never touched)."""
import pytest

from expert_slot_cache_amd import binding

P = 1 << 20        # an aligned address that is not null
F32, BF16 = binding.A_F32, binding.A_BF16
INF, NAN = float("inf"), float("nan")


def _refused(name, args):
    lib = binding.lib()
    assert getattr(lib, name)(*args) == binding.EINVAL, args
    assert lib.moe_last_error()


def _with(base, **change):
    out = dict(base)
    assert set(change) <= set(out)
    out.update(change)
    return list(out.values())


ROUTE = dict(atype=BF16, logits=P, stride=64, bias=P, T=4, E=64, K=8, score=1, norm=1, groups=8, kept=4, top=2, scale=1.0,
             ids=P, w=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(atype=2), dict(logits=None), dict(logits=P + 1), dict(stride=63), dict(bias=P + 2), dict(T=-1), dict(T=1 << 22),
    dict(E=0), dict(E=4160, stride=4160), dict(K=0), dict(K=65, E=128, stride=128), dict(K=33), dict(score=2), dict(score=-1),
    dict(norm=2), dict(groups=0), dict(groups=7), dict(groups=128, E=128, stride=128), dict(kept=0), dict(kept=9), dict(top=0),
    dict(top=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=INF), dict(scale=NAN), dict(ids=None), dict(ids=P + 2),
    dict(w=None), dict(w=P + 1)])
def test_route_groups_refuses(change):
    _refused("moe_route_groups", _with(ROUTE, **change))


BACK = dict(atype=F32, logits=P, stride=64, ids=P, w=P, dw=P, T=4, E=64, K=8, score=1, norm=1, scale=1.0, dl=P, dstride=64,
            stream=None)


@pytest.mark.parametrize("change", [
    dict(atype=-1), dict(logits=None), dict(logits=None, score=0, norm=0), dict(logits=P + 2), dict(stride=63), dict(ids=None),
    dict(w=None), dict(dw=None), dict(T=-1), dict(E=4097), dict(K=65), dict(K=65, E=128, dstride=128, stride=128),
    dict(score=3), dict(norm=-1), dict(scale=0.0), dict(scale=NAN), dict(dl=None), dict(dl=P + 2), dict(dstride=63)])
def test_route_groups_backward_refuses(change):
    _refused("moe_route_groups_backward", _with(BACK, **change))


PRODUCT = dict(atype=BF16, x=P, w=P, bias=P, offsets=P, resid=P, M=8, G=4, N=64, K=128, act=4, ot=BF16, out=P, pre=P, stream=None)
SIZES = [dict(atype=2), dict(M=-1), dict(M=(1 << 24) + 1), dict(G=0), dict(G=4097), dict(offsets=None), dict(offsets=P + 2),
         dict(N=0), dict(N=4), dict(N=60), dict(N=(1 << 18) + 16), dict(M=1 << 24, N=1 << 13)]
DEPTHS = [dict(K=0), dict(K=4), dict(K=12), dict(K=(1 << 17) + 8), dict(M=1 << 24, K=1 << 13),
          dict(G=4096, N=1 << 13, K=1 << 12), dict(K=132)]


@pytest.mark.parametrize("change", SIZES + DEPTHS + [
    dict(N=72), dict(atype=F32, ot=F32, N=68), dict(act=5), dict(act=-1), dict(ot=2), dict(atype=F32, ot=BF16), dict(x=None),
    dict(x=P + 8), dict(w=None), dict(w=P + 8), dict(bias=P + 2), dict(resid=P + 8), dict(out=None), dict(out=P + 4),
    dict(pre=P + 8)])
def test_expert_product_refuses(change):
    _refused("moe_expert_product", _with(PRODUCT, **change))


ACTIVATION = dict(atype=BF16, dout=P, ot=F32, pre=P, offsets=P, M=8, G=4, N=64, act=4, dpre=P, dbias=P, ws=P, wsb=1 << 20,
                  stream=None)


@pytest.mark.parametrize("change", SIZES + [
    dict(N=72), dict(act=5), dict(ot=2), dict(atype=F32, ot=BF16), dict(dout=None), dict(dout=P + 8), dict(pre=None),
    dict(pre=P + 8), dict(dpre=P + 8), dict(dpre=None, dbias=None), dict(dbias=P + 2), dict(ws=None), dict(ws=P + 8),
    dict(wsb=64)])
def test_activation_backward_refuses(change):
    _refused("moe_activation_backward", _with(ACTIVATION, **change))


GRADS = dict(atype=BF16, dpre=P, x=P, w=P, offsets=P, M=8, G=4, N=64, K=128, dx=P, dwt=F32, dw=P, ws=P, wsb=1 << 40, stream=None)


@pytest.mark.parametrize("change", SIZES + DEPTHS + [
    dict(dpre=None), dict(dpre=P + 8), dict(x=None), dict(x=P + 8), dict(w=None), dict(w=P + 8), dict(dx=P + 8),
    dict(dw=P + 8), dict(dx=None, dw=None), dict(dwt=2), dict(atype=F32, dwt=BF16)])
def test_expert_product_backward_refuses(change):
    _refused("moe_expert_product_backward", _with(GRADS, **change))


@pytest.mark.parametrize("name,args", [
    ("moe_route_groups", _with(ROUTE, T=0, logits=None, ids=None, w=None)),
    ("moe_route_groups_backward", _with(BACK, T=0, logits=None, ids=None, w=None, dw=None, dl=None)),
    ("moe_expert_product", _with(PRODUCT, M=0, x=None, w=None, out=None, resid=None)),
    ("moe_activation_backward", _with(ACTIVATION, M=0, dout=None, pre=None, dbias=None, ws=None)),
    ("moe_expert_product_backward", _with(GRADS, M=0, dpre=None, x=None, w=None, dw=None, ws=None))])
def test_no_rows_is_accepted_and_does_nothing(name, args):
    assert getattr(binding.lib(), name)(*args) == binding.OK


def test_workspaces():
    f, g = binding.activation_backward_workspace_bytes, binding.expert_product_backward_workspace_bytes
    assert f(100, 4, 64) > 0 and f(100, 4, 64) % 4 == 0
    assert f(-1, 4, 64) == 0 and f(100, 0, 64) == 0 and f(100, 1 << 33, 64) == 0
    assert g("bf16", 100, 4, 60, 64) == 0 and g("f32", -1, 4, 64, 64) == 0 and g("f32", 100, 4, 64, 1 << 33) == 0


torch = pytest.importorskip("torch")


class Reached(Exception):
    pass


class NoLibrary:
    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *_: 0
        raise Reached(name)


def tensors(call):
    f32 = lambda *s: torch.zeros(s)                                  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)               # noqa: E731
    return {
        "route_groups": dict(logits=f32(4, 8), topk_ids=i32(4, 2), topk_w=f32(4, 2), bias=f32(8)),
        "route_groups_backward": dict(logits=f32(4, 8), topk_ids=i32(4, 2), topk_w=f32(4, 2), d_topk_w=f32(4, 2),
                                      d_logits=f32(4, 8), score="sigmoid"),
        "expert_product": dict(x=f32(8, 16), w=f32(2, 24, 16), out=f32(8, 24), bias=f32(2, 24), resid=f32(8, 24),
                               pre=f32(8, 24), act="silu", offsets=i32(3)),
        "activation_backward": dict(d_out=f32(8, 24), pre=f32(8, 24), d_pre=f32(8, 24), d_bias=f32(2, 24), act="silu",
                                    offsets=i32(3)),
        "expert_product_backward": dict(d_pre=f32(8, 24), x=f32(8, 16), w=f32(2, 24, 16), d_x=f32(8, 16), d_w=f32(2, 24, 16),
                                        offsets=i32(3)),
    }[call]


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(binding, "_place", lambda torch, stream: (-1, 0))
    monkeypatch.setattr(binding, "lib", lambda: NoLibrary())


@pytest.mark.parametrize("call", ["route_groups", "route_groups_backward", "expert_product", "activation_backward",
                                  "expert_product_backward"])
def test_a_whole_call_reaches_the_library(on_cpu, call):
    with pytest.raises(Reached):
        getattr(binding, call)(**tensors(call))


CALLS = ["route_groups", "route_groups_backward", "expert_product", "activation_backward", "expert_product_backward"]
NEEDED = {"route_groups": ["logits", "topk_ids", "topk_w"], "route_groups_backward": ["topk_ids", "topk_w", "d_topk_w", "d_logits"],
          "expert_product": ["x", "w", "out"], "activation_backward": ["d_out", "pre"],
          "expert_product_backward": ["d_pre", "x", "w"]}


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in NEEDED[c]])
def test_a_missing_tensor_is_refused_as_one(on_cpu, call, name):
    with pytest.raises(binding.MoeError, match="missing"):
        getattr(binding, call)(**dict(tensors(call), **{name: None}))


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n, v in tensors(c).items() if isinstance(v, torch.Tensor)
                                       if (c, n) != ("route_groups_backward", "topk_ids")])
def test_a_tensor_of_another_shape_type_or_layout_is_refused(on_cpu, call, name):
    good = tensors(call)
    t = good[name]
    # one row more, another type, and the same shape with its last two dimensions turned round
    others = [torch.zeros((t.shape[0] + 1, *t.shape[1:]), dtype=t.dtype), t.to(torch.float64)]
    if t.dim() > 1 and name not in ("logits", "d_logits"):
        others.append(torch.zeros(*t.shape[:-2], t.shape[-1], t.shape[-2], dtype=t.dtype).transpose(-1, -2))
    elif t.dim() > 1:
        others.append(torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype)[:, ::2])
    for other in others:
        with pytest.raises(binding.MoeError):
            getattr(binding, call)(**dict(good, **{name: other}))


@pytest.mark.parametrize("call,change", [
    ("route_groups", dict(score="max")), ("route_groups_backward", dict(score="")), ("expert_product", dict(act="tanh")),
    ("activation_backward", dict(act=None)),
    ("expert_product", dict(out=torch.zeros(8, 24, dtype=torch.bfloat16), resid=None)),      # fp32 rows, bf16 output
    ("expert_product", dict(act="swiglu")),                                                  # out has N columns, not N/2
    ("activation_backward", dict(d_out=torch.zeros(8, 24, dtype=torch.bfloat16))),
    ("expert_product_backward", dict(d_w=torch.zeros(2, 24, 16, dtype=torch.bfloat16))),
    ("expert_product_backward", dict(d_x=None, d_w=None))])
def test_other_choices_are_refused(on_cpu, call, change):
    with pytest.raises(binding.MoeError):
        getattr(binding, call)(**dict(tensors(call), **change))
