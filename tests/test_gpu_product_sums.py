"""GPU tests of how scaled_product sums: every output format holds a block's 128 products and the
blocks in 32 bits, also where products of very different size meet in one sum."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from oracle import rows as orows
from test_gpu_operators import F8, HALF, TYPES, U, Product, dev, host, offsets_for, within

pytestmark = pytest.mark.gpu


def codes(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(F8)


def one_large(rows, depth, value, sign):
    """448 at one place of each eight, `value` at its others.  `sign`: the 448 of every other eight
    is negative, so that products of two such rows cancel across the eights."""
    v = np.full((rows, depth // 8, 8), value)
    v[:, :, 3] = 448.0
    if sign:
        v[:, 1::2, 3] = -448.0
    return v.reshape(rows, depth)


def channels(rows, depth, seed, times):
    """Normal values; one channel in eight is `times` the others."""
    v = np.random.default_rng(seed).normal(size=(rows, depth))
    v[:, 5::8] *= times
    return np.clip(v * (100.0 / times if times > 16 else 1.0), -448, 448)


def large_and_small(M, G, N, K, seed):
    """(x, w) by name: products 2^13 and more below the largest of their eight, the large ones
    cancelling or not; channels 16 and 256 times the others; codes of all sizes, all positive."""
    rng = np.random.default_rng(seed)
    any_code = lambda *s: orows.e4m3_widen(rng.integers(0, 0x7F, s))     # noqa: E731
    out = {"cancel": (one_large(M, K, 3.0, False), one_large(G * N, K, 5.0, True)),
           "add": (one_large(M, K, 3.0, False), one_large(G * N, K, 5.0, False)),
           "all sizes": (any_code(M, K), any_code(G * N, K))}
    for times in (16, 256):
        out[f"channels x {times}"] = channels(M, K, seed + times, times), channels(G * N, K, seed + 2 * times, times)
    return {name: (x, w.reshape(G, N, K)) for name, (x, w) in out.items()}


@pytest.mark.parametrize("M,G,N,K", [(1, 1, 40, 128), (9, 3, 130, 272), (60, 1, 257, 400), (700, 3, 520, 256), (2000, 5, 1300, 144),
                                     (2100, 2, 4100, 144)])
def test_sums_are_held_in_32_bits(M, G, N, K):
    nb, kb = -(-N // 128), -(-K // 128)
    offsets = offsets_for(M, G, M) if G > 1 else np.array([0, M], np.int32)
    for name, (x, w) in large_and_small(M, G, N, K, M + N).items():
        x, w = codes(x), codes(w)
        # powers of two, so that the scales round nothing
        xs = np.exp2(np.random.default_rng(M).integers(-6, -2, (M, kb))).astype(np.float32)
        ws = np.exp2(np.random.default_rng(N).integers(-6, -2, (G, nb, kb))).astype(np.float32)
        xv, wv = orows.widen_rows(host(x), xs), [orows.widen_matrix(host(w[g]), ws[g]) for g in range(G)]
        ref = orows.scaled_product(xv, wv, offsets)
        # a block's 128 products are exact and added in fp32, at most two half steps an addition
        # (it may truncate), then kb blocks: (256 + 2 kb) u of the magnitudes' sum
        bound = orows.scaled_product(np.abs(xv), [np.abs(v) for v in wv], offsets) * (256 + 2 * kb) * U
        got = {}
        for kind in ("f32", "bf16"):
            out = torch.full((M, N), 7.0, dtype=TYPES[kind], device=DEV)
            binding.scaled_product(x.to(DEV), dev(xs), w.to(DEV), dev(ws), out, offsets=dev(offsets))
            within(host(out), ref, bound * (1 + HALF[kind]) + np.abs(ref) * HALF[kind], f"{name}, {kind}")
            got[kind] = out
        assert torch.equal(got["f32"].to(torch.bfloat16), got["bf16"]), name    # rounded once, from the same sums


@pytest.mark.parametrize("M,G,N,K", [(7, 1, 300, 640), (200, 30, 1030, 528), (333, 1, 1000, 1040), (700, 30, 700, 528),
                                     (3500, 20, 1100, 272), (4100, 4, 1300, 656)])
def test_bf16_is_the_fp32_output_rounded(M, G, N, K):
    p = Product(M, G, N, K, M + N, offsets_for(M, G, M) if G > 1 else None)
    wide, out = torch.zeros((M, N), device=DEV), torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    p.call(wide)
    p.call(out)
    assert torch.equal(wide.to(torch.bfloat16), out)
