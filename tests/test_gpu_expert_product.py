"""GPU tests of the expert products and their gradients against oracle/experts.py in float64.

Tolerances: u = 2^-24 is half a step of fp32.  The matrix instruction adds exact (bf16) or rounded
(fp32) products in fp32, each addition within a whole step (it need not round to nearest): a sum
of n is off by at most 2 (n + 4) u of the sum of the magnitudes, in any order.  An activation
passes its argument's error on by its slope (|act'| < 1.13) and adds its own: silu's exponential
and reciprocal (|h| + 4) 2 u of the value, erfc's argument and its own rounding (2 h^2 + 40) u.
A bf16 output adds half a step, 2^-8 of the value.  Where |h| > 87 an exponential has no normal
number: |h| 2^-125."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from oracle import experts as oe
from test_gpu_operators import HALF, TYPES, U, dev, host, within

pytestmark = pytest.mark.gpu

NAN = float("nan")
MARGIN = 4096      # bytes before and behind


class Guarded:
    """A tensor between two margins that no call may touch."""

    def __init__(self, shape, kind, fill=3.0):
        t = TYPES[kind]
        n = int(np.prod(shape)) * torch.empty(0, dtype=t).element_size()
        self.whole = torch.full((n + 2 * MARGIN,), 0x5A, dtype=torch.uint8, device=DEV)
        self.t = self.whole[MARGIN:MARGIN + n].view(t).view(shape)
        self.t.fill_(fill)

    def check(self, what=""):
        n = self.whole.numel()
        assert bool((self.whole[:MARGIN] == 0x5A).all()) and bool((self.whole[n - MARGIN:] == 0x5A).all()), what


def offsets_for(M, G, seed, holes=True):
    """Uneven groups, some without rows; with holes rows before the first and behind the last."""
    if G == 1 and not holes:
        return None
    rng = np.random.default_rng(seed)
    lo, hi = (min(1, M), M - min(2, M // 3)) if holes else (0, M)
    cuts = np.sort(rng.integers(lo, hi + 1, G - 1)) if G > 1 else np.empty(0, int)
    if G > 3:
        cuts[G // 2] = cuts[G // 2 - 1]
    return np.concatenate([[lo], cuts, [hi]]).astype(np.int32)


def rows_for(shape, seed, kind, std=1.0):
    v = np.random.default_rng(seed).normal(size=shape).astype(np.float32) * np.float32(std)
    return dev(v, kind)


def sum_err(n):
    return 2 * (n + 4) * U


def act_err(h, e, act):
    """Of act(h) where h is off by e."""
    a = np.abs(oe.activate(h, act))
    if act == "silu":
        return 1.13 * e + a * (np.abs(h) + 4) * 2 * U + np.abs(h) * 2.0 ** -125
    if act == "gelu":
        return 1.13 * e + a * (2 * h * h + 40) * U + np.abs(h) * 2.0 ** -125
    return e


def slope_err(h, act):
    """Of act'(h), absolute."""
    if act == "silu":
        return oe.sigmoid(h) * (1 + np.abs(h)) * (np.abs(h) + 6) * 2 * U + (1 + np.abs(h)) * 2.0 ** -125
    if act == "gelu":
        return (oe.normal_cdf(h) + np.abs(h) * np.exp(-h * h / 2)) * (2 * h * h + 40) * U + (1 + np.abs(h)) * 2.0 ** -125
    return 0 * h


def product_case(M, G, N, K, kind, out, act, bias, resid, pre, holes=True, seed=0, offsets="make"):
    x, w = rows_for((M, K), seed + 1, kind), rows_for((G, N, K), seed + 2, kind, 1.5 / K ** 0.5)
    if isinstance(offsets, str):
        offsets = offsets_for(M, G, seed + 3, holes)
    b = rows_for((G, N), seed + 4, "f32", 0.5) if bias else None
    cols = N // 2 if act == "swiglu" else N
    r = rows_for((M, cols), seed + 5, out) if resid else None
    o, p = Guarded((M, cols), out), Guarded((M, N), kind) if pre else None
    binding.expert_product(x, w, o.t, bias=b, resid=r, pre=p.t if pre else None, act=act,
                           offsets=None if offsets is None else dev(offsets))
    x, w = host(x), host(w)
    b, r = host(b) if bias else None, host(r) if resid else None
    ref, h = oe.product(x, w, offsets, b, r, act)
    ref_abs, _ = oe.product(np.abs(x), np.abs(w), offsets, None if b is None else np.abs(b))
    e = ref_abs * sum_err(K)
    if act == "swiglu":
        g, u, eg, eu = h[:, :cols], h[:, cols:], e[:, :cols], e[:, cols:]
        a, ea = oe.activate(g, "silu"), act_err(g, eg, "silu")
        plain, bound = a * u, ea * np.abs(u) + np.abs(a) * eu + ea * eu + np.abs(a * u) * 2 * U
    else:
        plain, bound = oe.activate(h, act), act_err(h, e, act)
    if resid:
        bound = bound + (np.abs(plain) + np.abs(r)) * 2 * U
    out_of = np.isnan(ref).all(axis=1)
    got = host(o.t)
    assert (got[out_of] == 3.0).all()
    within(got[~out_of], ref[~out_of], (bound + np.abs(ref) * HALF[out] + bound * HALF[out])[~out_of], "out")
    o.check("out")
    if pre:
        got = host(p.t)
        assert (got[out_of] == 3.0).all()
        within(got[~out_of], h[~out_of], (e + (np.abs(h) + e) * HALF[kind])[~out_of], "pre")
        p.check("pre")


TYPINGS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]
# (rows, groups, columns, depth): one row, one group, more groups than rows, odd row counts, a last
# tile of every kind in columns and depth
SHAPES = [(1, 1, 8, 8), (1, 1, 256, 512), (3, 1, 64, 2048), (8, 64, 64, 128), (5, 3, 16, 24), (17, 2, 40, 72), (64, 1, 128, 64),
          (129, 5, 136, 200), (300, 200, 48, 96), (333, 1, 1000, 1040), (700, 4, 264, 328), (1500, 3, 512, 264)]


@pytest.mark.parametrize("kind,out", TYPINGS)
@pytest.mark.parametrize("M,G,N,K", SHAPES)
def test_product(M, G, N, K, kind, out):
    product_case(M, G, N, K, kind, out, "none", False, False, False, holes=M % 2 == 1)


@pytest.mark.parametrize("kind,out", TYPINGS)
@pytest.mark.parametrize("act", oe.ACTS)
@pytest.mark.parametrize("M,G,N,K", [(1, 1, 16, 16), (7, 4, 48, 40), (200, 3, 272, 136), (700, 2, 640, 200)])
def test_epilogue(M, G, N, K, act, kind, out):
    for i, (bias, resid, pre) in enumerate([(True, True, True), (True, False, False), (False, True, False), (False, False, True)]):
        product_case(M, G, N, K, kind, out, act, bias, resid, pre, seed=i)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("act", oe.ACTS)
def test_activations_far_out(act, kind):
    """Arguments to +-120 through a unit matrix, where exponentials run over and out."""
    N = 64
    x = torch.linspace(-120, 120, 200, device=DEV)[:, None].repeat(1, N).to(TYPES[kind])
    w = torch.eye(N, device=DEV)[None].to(TYPES[kind]).contiguous()
    cols = N // 2 if act == "swiglu" else N
    out = torch.empty(200, cols, device=DEV)
    binding.expert_product(x, w, out, act=act)
    h = host(x)
    ref = oe.activate(h, act)
    bound = act_err(h[:, :cols], 0, "silu") * np.abs(h[:, cols:]) if act == "swiglu" else act_err(h, 0, act)
    within(host(out), ref, bound + np.abs(ref) * 3 * U, act)


def test_residual_may_be_the_output():
    x, w = rows_for((50, 64), 1, "bf16"), rows_for((2, 48, 64), 2, "bf16", 0.2)
    resid, off = rows_for((50, 48), 3, "bf16"), dev(np.int32([2, 20, 45]))
    a, b = resid.clone(), resid.clone()
    binding.expert_product(x, w, a, resid=resid, act="relu", offsets=off)
    binding.expert_product(x, w, b, resid=b, act="relu", offsets=off)
    assert torch.equal(a, b)


# ---- back through the epilogue ---------------------------------------------------------------


@pytest.mark.parametrize("kind,out", TYPINGS)
@pytest.mark.parametrize("act", oe.ACTS)
@pytest.mark.parametrize("M,G,N", [(1, 1, 16), (5, 3, 48), (64, 1, 256), (333, 70, 1040), (2000, 3, 528), (1, 1, 4112)])
def test_activation_backward(M, G, N, act, kind, out):
    cols = N // 2 if act == "swiglu" else N
    d_out, pre = rows_for((M, cols), 1, out), rows_for((M, N), 2, kind, 2.0)
    offsets = offsets_for(M, G, 3, holes=M > 1)
    off = None if offsets is None else dev(offsets)
    dp, db = Guarded((M, N), kind), Guarded((G, N), "f32")
    binding.activation_backward(d_out, None if act == "none" else pre, dp.t, d_bias=db.t, act=act, offsets=off)
    d, h = host(d_out), host(pre)
    ref, ref_b = oe.activation_grad(d, h, offsets, N, act)
    if act == "swiglu":
        g, u = h[:, :cols], h[:, cols:]
        e = np.concatenate([np.abs(d * u) * (slope_err(g, "silu") + np.abs(oe.slope(g, "silu")) * 3 * U),
                            np.abs(d) * (act_err(g, 0, "silu") + np.abs(oe.activate(g, "silu")) * 3 * U)], axis=1)
    else:
        e = np.abs(d) * (slope_err(h, act) + np.abs(oe.slope(h, act)) * 2 * U * (act != "none"))
    out_of = np.isnan(ref).all(axis=1)
    got = host(dp.t)
    assert (got[out_of] == 3.0).all()
    within(got[~out_of], ref[~out_of], (e + (np.abs(ref) + e) * HALF[kind])[~out_of], "d_pre")
    e[out_of] = 0
    mag = np.where(np.isnan(ref), 0, np.abs(ref)) + e
    bound = np.stack([(e[a:b] + mag[a:b] * (b - a + 4) * U).sum(0) for _, a, b in oe.runs(offsets, M)])
    within(host(db.t), ref_b, bound, "d_bias")
    dp.check("d_pre")
    db.check("d_bias")
    # each alone, and the gradient in place of what it is taken from
    alone, alone_b = torch.full_like(dp.t, 3.0), torch.empty_like(db.t)
    binding.activation_backward(d_out, pre, alone, act=act, offsets=off)
    binding.activation_backward(d_out, pre, None, d_bias=alone_b, act=act, offsets=off)
    assert torch.equal(alone, dp.t) and torch.equal(alone_b, db.t)
    if act == "none" and kind == out:
        same = d_out.clone()
        binding.activation_backward(same, None, same, offsets=off)
        assert torch.equal(same, d_out)
    if act != "none":
        binding.activation_backward(d_out, pre, pre, act=act, offsets=off)
        rows = torch.from_numpy(~out_of).to(DEV)
        assert torch.equal(pre[rows], dp.t[rows])


def test_a_bias_of_many_groups_and_none_of_them_has_rows():
    for M, off in ((0, [0] * 71), (9, [9] * 71), (9, [4] * 71)):
        db = torch.full((70, 24), 7.0, device=DEV)
        binding.activation_backward(torch.ones(M, 24, device=DEV), None, None, d_bias=db, offsets=dev(np.int32(off)))
        assert (db == 0).all()


# ---- back through the product ----------------------------------------------------------------


def grad_case(M, G, N, K, kind, dw_kind, which="both", holes=True, seed=0, offsets="make"):
    dp, x = rows_for((M, N), seed + 1, kind), rows_for((M, K), seed + 2, kind)
    w = rows_for((G, N, K), seed + 3, kind)
    if isinstance(offsets, str):
        offsets = offsets_for(M, G, seed + 4, holes)
    off = None if offsets is None else dev(offsets)
    dx = Guarded((M, K), kind) if which != "w" else None
    dw = Guarded((G, N, K), dw_kind) if which != "x" else None
    binding.expert_product_backward(dp, x if dw else None, w if dx else None, d_x=dx.t if dx else None, d_w=dw.t if dw else None,
                                    offsets=off)
    dp, x, w = host(dp), host(x), host(w)
    ref_x, ref_w = oe.product_grad(dp, x, w, offsets)
    abs_x, abs_w = oe.product_grad(np.abs(dp), np.abs(x), np.abs(w), offsets)
    if dx:
        out_of = np.isnan(ref_x).all(axis=1)
        got = host(dx.t)
        assert (got[out_of] == 3.0).all()
        e = abs_x * sum_err(N)
        within(got[~out_of], ref_x[~out_of], (e + (np.abs(ref_x) + e) * HALF[kind])[~out_of], "d_x")
        dx.check("d_x")
    if dw:
        n = np.array([b - a for _, a, b in oe.runs(offsets, M)])[:, None, None]
        e = abs_w * sum_err(n)
        within(host(dw.t), ref_w, e + (np.abs(ref_w) + e) * HALF[dw_kind], "d_w")
        dw.check("d_w")


@pytest.mark.parametrize("kind,dw_kind", TYPINGS)
@pytest.mark.parametrize("M,G,N,K", SHAPES)
def test_product_backward(M, G, N, K, kind, dw_kind):
    grad_case(M, G, N, K, kind, dw_kind, holes=M % 2 == 1)


@pytest.mark.parametrize("which", ["x", "w"])
def test_one_gradient_alone(which):
    grad_case(90, 4, 72, 136, "bf16", "f32", which)
    grad_case(90, 4, 72, 136, "f32", "f32", which)


@pytest.mark.parametrize("kind,dw_kind", TYPINGS)
def test_matrices_of_groups_without_rows_have_no_gradient(kind, dw_kind):
    for M, off in ((0, [0] * 6), (9, [9] * 6), (9, [4, 4, 5, 5, 5, 5])):
        grad_case(M, 5, 24, 40, kind, dw_kind, "both" if M else "w", offsets=np.int32(off))


def test_gradients_are_the_differences_of_the_forward():
    """The call's own forward in fp32: a loss' differences along a random direction."""
    M, G, N, K = 37, 3, 48, 40
    for act in oe.ACTS:
        x, w, b = rows_for((M, K), 1, "f32"), rows_for((G, N, K), 2, "f32", 0.2), rows_for((G, N), 3, "f32")
        cols = N // 2 if act == "swiglu" else N
        d_out, off = rows_for((M, cols), 4, "f32"), dev(np.int32([0, 20, 20, 37]))
        out, pre = torch.empty(M, cols, device=DEV), torch.empty(M, N, device=DEV)
        binding.expert_product(x, w, out, bias=b, pre=pre, act=act, offsets=off)
        dp, db = torch.empty_like(pre), torch.empty(G, N, device=DEV)
        binding.activation_backward(d_out, pre, dp, d_bias=db, act=act, offsets=off)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        binding.expert_product_backward(dp, x, w, d_x=dx, d_w=dw, offsets=off)

        def loss(x, w, b):
            return (oe.product(host(x), host(w), [0, 20, 20, 37], host(b), None, act)[0] * host(d_out)).sum()

        for i, (v, g) in enumerate([(x, dx), (w, dw), (b, db)]):
            step = rows_for(tuple(v.shape), 9, "f32", 2.0 ** -12)
            args, size = [x, w, b], [x, w, b]
            args[i], size[i] = v + step, v - step
            slope = (host(args[i]) - host(size[i]))
            diff = loss(*args) - loss(*size)
            want = (host(g) * slope).sum()
            # the third differences along the step, and the gradient's own rounding; a kink of relu that the step
            # crosses moves the loss by at most its share
            scale = np.abs(host(g) * slope).sum()
            assert abs(diff - want) <= (2e-2 if act == "relu" else 1e-4) * scale, (act, i, diff, want)


# ---- as a user runs them ---------------------------------------------------------------------

def test_same_bits_on_another_stream_and_captured():
    M, G, N, K = 200, 6, 96, 136
    x, w, b = rows_for((M, K), 1, "bf16"), rows_for((G, N, K), 2, "bf16", 0.1), rows_for((G, N), 3, "f32")
    off = dev(offsets_for(M, G, 4))
    d_out = rows_for((M, N // 2), 5, "bf16")
    L = binding
    ws1 = torch.empty(L.activation_backward_workspace_bytes(M, G, N), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(max(16, L.expert_product_backward_workspace_bytes("bf16", M, G, N, K)), dtype=torch.uint8, device=DEV)

    def buffers():
        return [torch.full((M, N // 2), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV),
                torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV), torch.empty(G, N, device=DEV),
                torch.full((M, K), 3.0, dtype=torch.bfloat16, device=DEV), torch.empty(G, N, K, device=DEV)]

    def step(o, a, c):
        out, pre, dp, db, dx, dw = o
        L.expert_product(x, w, out, bias=b, pre=pre, act="swiglu", offsets=off)
        L.activation_backward(d_out, pre, dp, d_bias=db, act="swiglu", offsets=off, workspace=a)
        L.expert_product_backward(dp, x, w, d_x=dx, d_w=dw, offsets=off, workspace=c)

    ref, got = buffers(), buffers()
    step(ref, ws1, ws2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got, None, None)
    side = torch.cuda.Stream()
    ws3, ws4 = torch.empty_like(ws1), torch.empty_like(ws2)
    for i in range(4):
        x.copy_(rows_for((M, K), 10 + i, "bf16"))
        for t in got[3:4] + got[5:]:
            t.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        other = buffers()
        with torch.cuda.stream(side):
            step(other, ws3, ws4)
        step(ref, ws1, ws2)
        torch.cuda.synchronize()
        for a, c, d in zip(ref, got, other):
            assert torch.equal(a, c) and torch.equal(a, d), i


def test_a_stream_that_is_not_torchs_needs_its_workspace():
    other = torch.cuda.Stream()
    d, db = torch.ones(4, 16, device=DEV), torch.empty(1, 16, device=DEV)
    with pytest.raises(binding.MoeError, match="workspace"):
        binding.activation_backward(d, None, None, d_bias=db, stream=other.cuda_stream)
    ws = torch.empty(binding.activation_backward_workspace_bytes(4, 1, 16), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    binding.activation_backward(d, None, None, d_bias=db, workspace=ws, stream=other.cuda_stream)
    other.synchronize()
    assert (db == 4).all()
