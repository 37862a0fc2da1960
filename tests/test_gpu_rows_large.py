"""GPU tests of the rows' movers where a call is large: on both sides of the sizes from which rows
are stored past the caches."""
import pytest
import torch

import test_gpu_operators as ops
from _gpu_helpers import DEV
from expert_slot_cache_amd import binding

pytestmark = pytest.mark.gpu

MIB = 1 << 20


def places(T, K, E, seed):
    """ids and the sort's offsets and rows of T tokens, a few of them without an expert."""
    ids = ops.dev(ops.ids_for(T, K, E, seed, holes=0.05))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    rows = torch.full((T, K), -5, dtype=torch.int32, device=DEV)
    return ids, offsets, rows


def tokens(T, H, seed, kind):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randn(T, H, generator=gen, device=DEV).to(ops.TYPES[kind])


# (tokens, k, hidden, type): rows of 120 and 256 MiB lie between these
LARGE = [(1000, 8, 2048, "bf16"), (1030, 8, 2050, "bf16"), (3700, 8, 2048, "bf16"), (3901, 8, 2056, "bf16"), (3100, 5, 2049, "f32"),
         (4000, 8, 4096, "bf16"), (4200, 8, 4100, "bf16"), (260, 33, 8192, "f32")]


@pytest.mark.parametrize("T,K,H,kind", LARGE)
def test_rows_there_and_back(T, K, H, kind):
    """Every row bit for bit; the sums against 64 bits, token by token, on a part of them."""
    E = 40
    ids, offsets, rows = places(T, K, E, T)
    x = tokens(T, H, 1, kind)
    out = torch.full((T * K, H), 3.0, dtype=ops.TYPES[kind], device=DEV)
    binding.sort_tokens(x, ids, out, offsets, rows)
    at = rows.long()
    live = at >= 0
    assert torch.equal(out[at[live]], x[:, None].expand(T, K, H)[live])
    n = int(offsets[-1])
    assert n == int(live.sum()) and bool((out[n:] == 3.0).all())
    assert torch.equal(torch.sort(at[live]).values, torch.arange(n, device=DEV))

    part = torch.arange(0, T, 7, device=DEV)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    w = torch.rand(T, K, generator=gen, device=DEV)
    got = torch.full((T, H), 9.0, dtype=ops.TYPES[kind], device=DEV)
    binding.combine_rows(out, rows, got, topk_w=w, resid=x)
    wl = torch.where(live, w.double(), 0.0)[part]
    xd = x[part].double()
    ref = xd + (wl.sum(1)[:, None] * xd)               # each row is its token
    size = xd.abs() * (1 + wl.sum(1)[:, None])
    # as in test_combine_rows; the reference's own sum of weights adds nothing at 2^-53
    assert bool(((got[part].double() - ref).abs() <= size * (K + 3) * ops.U + ref.abs() * ops.HALF[kind]).all())

    d = tokens(T, H, 3, kind)
    d_ys = torch.full((T * K, H), 9.0, dtype=ops.TYPES[kind], device=DEV)
    d_w = torch.full((T, K), 9.0, device=DEV)
    binding.combine_rows_backward(d, out, rows, w, d_ys, d_w)
    want = (w[:, :, None] * d.float()[:, None]).to(ops.TYPES[kind]) if T * K * H < 64 * MIB else None
    if want is not None:                               # one product in fp32, rounded once: the same bits
        assert torch.equal(d_ys[at[live]], want[live])
    else:
        for k in range(K):
            m = live[:, k]
            assert torch.equal(d_ys[at[m, k]], (w[m, k, None] * d[m].float()).to(ops.TYPES[kind]))
    assert bool((d_ys[n:] == 9.0).all())
    dot = (d[part].double() * xd).sum(1)
    size = (d[part].double() * xd).abs().sum(1)
    ref_w = torch.where(live[part], dot[:, None], 0.0)
    assert bool(((d_w[part].double() - ref_w).abs() <= size[:, None] * (H + 2) * ops.U).all())
