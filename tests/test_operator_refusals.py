"""CPU tests of the argument checks of the operators around the experts: every refused call
returns before any GPU call (the addresses below are never touched)."""
import pytest

from expert_slot_cache_amd import binding

P = 1 << 20        # an aligned address that is not null
F32, BF16 = binding.A_F32, binding.A_BF16


def _refused(name, args):
    lib = binding.lib()
    assert getattr(lib, name)(*args) == binding.EINVAL, args
    assert lib.moe_last_error()


def _with(base, **change):
    out = dict(base)
    out.update(change)
    return list(out.values())


ROUTE = dict(atype=BF16, logits=P, stride=64, T=4, E=64, K=8, norm=1, ids=P, w=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(atype=2), dict(logits=None), dict(logits=P + 1), dict(stride=63), dict(stride=-64), dict(T=-1), dict(E=0),
    dict(E=4097, stride=4097), dict(K=0), dict(K=65, E=128, stride=128), dict(K=9, E=8), dict(norm=2), dict(ids=None),
    dict(ids=P + 2), dict(w=None), dict(w=P + 2), dict(T=1 << 22)])
def test_route_refuses(change):
    _refused("moe_route", _with(ROUTE, **change))


BACK = dict(atype=F32, logits=P, stride=64, ids=P, w=P, dw=P, T=4, E=64, K=8, norm=0, dl=P, dstride=64, stream=None)


@pytest.mark.parametrize("change", [
    dict(atype=-1), dict(logits=None), dict(logits=P + 2), dict(stride=63), dict(ids=None), dict(w=None), dict(dw=None),
    dict(T=-1), dict(E=4097), dict(K=65), dict(norm=-1), dict(dl=None), dict(dl=P + 2), dict(dstride=63)])
def test_route_backward_refuses(change):
    _refused("moe_route_backward", _with(BACK, **change))


SORT = dict(atype=BF16, x=P, stride=256, ids=P, T=8, K=4, E=16, H=256, f8=1, out=P, scales=P, offsets=P, rows=P, ws=None,
            wsb=0, stream=None)


@pytest.mark.parametrize("change", [
    dict(atype=7), dict(x=P + 1), dict(stride=255), dict(ids=None), dict(T=-1), dict(K=0), dict(K=65), dict(E=0),
    dict(E=4097), dict(H=0), dict(H=250, stride=250), dict(f8=2), dict(out=None), dict(out=P + 8), dict(scales=None),
    dict(offsets=None), dict(rows=None), dict(T=4096), dict(T=4096, ws=P, wsb=64), dict(T=4096, ws=P + 2, wsb=1 << 20),
    dict(H=1 << 18, stride=1 << 18), dict(T=1 << 23)])
def test_sort_refuses(change):
    _refused("moe_sort_tokens", _with(SORT, **change))


def test_sort_workspace_bytes():
    f = binding.sort_workspace_bytes
    assert f(1, 8, 64) == 0 and f(256, 8, 64) == 0
    assert f(257, 8, 64) == 3 * 64 * 4            # three workgroups' counts
    assert f(1 << 20, 16, 64) == 256 * 64 * 4     # never more than 256 of them
    assert f(-1, 8, 64) == 0 and f(8, 0, 64) == 0 and f(8, 8, 5000) == 0


COMBINE = dict(atype=BF16, ys=P, rows=P, w=P, resid=P, T=8, K=4, H=256, out=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(atype=3), dict(ys=None), dict(ys=P + 1), dict(rows=None), dict(w=P + 2), dict(resid=P + 1), dict(T=-2), dict(K=0),
    dict(K=65), dict(H=0), dict(H=(1 << 17) + 1), dict(T=1 << 24, K=1), dict(out=None), dict(out=P + 1)])
def test_combine_refuses(change):
    _refused("moe_combine_rows", _with(COMBINE, **change))


COMBINE_BACK = dict(atype=BF16, dout=P, ys=P, rows=P, w=P, T=8, K=4, H=256, dys=P, dw=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(atype=3), dict(dout=None), dict(ys=None), dict(rows=None), dict(w=None), dict(T=-2), dict(K=0), dict(H=0),
    dict(dys=None), dict(dys=P + 1), dict(dw=None), dict(dw=P + 2)])
def test_combine_backward_refuses(change):
    _refused("moe_combine_rows_backward", _with(COMBINE_BACK, **change))


PRODUCT = dict(x=P, xs=P, w=P, ws=P, offsets=P, M=8, G=4, N=256, K=128, ep=2, out=P, os=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(x=P + 8), dict(xs=None), dict(xs=P + 2), dict(w=None), dict(w=P + 8), dict(ws=None),
    dict(offsets=None), dict(offsets=P + 2), dict(M=-1), dict(M=(1 << 24) + 1),
    dict(M=1 << 23, N=(1 << 13) + 256), dict(G=0), dict(G=4097), dict(N=0),
    dict(N=128), dict(N=384), dict(K=0), dict(K=8), dict(K=120), dict(K=1 << 18), dict(ep=3), dict(ep=-1),
    dict(out=None), dict(out=P + 4), dict(os=None), dict(ep=0, out=P + 2), dict(ep=1, out=P + 1)])
def test_scaled_product_refuses(change):
    _refused("moe_scaled_product", _with(PRODUCT, **change))


@pytest.mark.parametrize("name,args", [
    ("moe_route", _with(ROUTE, T=0, logits=None, ids=None, w=None)),
    ("moe_route_backward", _with(BACK, T=0, logits=None, ids=None, w=None, dw=None, dl=None)),
    ("moe_combine_rows", _with(COMBINE, T=0, ys=None, rows=None, out=None)),
    ("moe_combine_rows_backward", _with(COMBINE_BACK, T=0, dout=None, ys=None, rows=None, w=None, dys=None, dw=None)),
    ("moe_scaled_product", _with(PRODUCT, M=0, x=None, xs=None, w=None, ws=None, out=None, os=None))])
def test_no_tokens_is_accepted_and_does_nothing(name, args):
    assert getattr(binding.lib(), name)(*args) == binding.OK


def test_sizes_past_int32_are_refused_not_wrapped():
    """A size is passed on as int32: 2^32 + 4 rows must not become four."""
    torch = pytest.importorskip("torch")
    big = torch.empty(1, dtype=torch.int32).expand((1 << 32) + 4, 1)
    with pytest.raises(binding.MoeError, match="sizes above"):
        binding._array("topk_ids", big, torch.int32, -1)
    with pytest.raises(binding.MoeError, match="sizes above"):
        binding._rows("x", big, -1)
    assert tuple(binding._array("topk_ids", big[:4].contiguous(), torch.int32, -1)) == (4, 1)
    assert binding.sort_workspace_bytes((1 << 32) + 4000, 8, 64) == 0


def test_missing_tensors_are_refused():
    for call in (lambda: binding._array("topk_ids", None, None, 0), lambda: binding._rows("x", None, 0),
                 lambda: binding._check_tensor("rows", None, None, (1, 1), 0)):
        with pytest.raises(binding.MoeError, match="is missing"):
            call()
