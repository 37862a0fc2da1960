"""GPU tests of every tile of the expert products and their gradients, with rows that use each stage of
the ring again, at whole and shorter last stages, and of a matrix' gradient in parts.  (A CPU test holds
the tile of each case; the oracle and tolerances are those of test_gpu_expert_product.)"""
import numpy as np
import pytest

from test_gpu_expert_product import grad_case, product_case

pytestmark = pytest.mark.gpu

# (columns, rows of a tile): (rows, groups, output columns, depth) of products
BF16 = {
    (256, 256): [(3000, 2, 4096, 256), (3001, 2, 4112, 328)],
    (256, 128): [(1600, 8, 2560, 384), (1601, 8, 2576, 360)],
    (128, 64): [(1000, 16, 896, 384), (1001, 16, 912, 328)],
    (64, 64): [(700, 16, 512, 384), (701, 16, 528, 392)],
    (64, 32): [(60, 30, 320, 448), (61, 30, 336, 520), (333, 1, 1000, 1040)],
    (32, 32): [(20, 3, 64, 512), (21, 3, 80, 600), (1, 1, 2048, 1024)],
}
F32 = {
    (64, 64): [(700, 16, 512, 192), (701, 16, 528, 196), (3000, 8, 512, 196)],
    (64, 32): [(120, 60, 320, 224), (121, 60, 336, 228)],
    (32, 32): [(20, 3, 64, 256), (21, 3, 80, 292), (333, 1, 1000, 260)],
}
F32_SWIGLU = {                                        # and this one, which SwiGLU alone takes in fp32
    (128, 64): [(1700, 2, 896, 192), (1701, 2, 912, 212)],
}
# (columns, rows of a tile, parts): (rows, groups, columns, depth) of a product whose matrix' gradient it is
MATRICES = {
    (256, 256, 1): [(1700, 4, 1792, 1792), (1601, 4, 1800, 1784)],
    (256, 128, 1): [(700, 24, 512, 512), (5000, 24, 520, 504)],
    (128, 128, 1): [(700, 24, 512, 256), (6001, 24, 456, 248)],
    (128, 64, 1): [(333, 1, 1000, 1040), (700, 4, 264, 328), (4000, 1, 64, 256)],
    (128, 64, 2): [(13000, 3, 72, 264)],
    (128, 64, 4): [(8300, 1, 64, 256)],
}


@pytest.mark.parametrize("M,G,N,K", [c for cases in BF16.values() for c in cases])
def test_products_in_bf16(M, G, N, K):
    product_case(M, G, N, K, "bf16", "bf16", "none", False, True, False, holes=M % 2 == 1)
    if N % 16 == 0:
        product_case(M, G, N, K, "bf16", "f32", "swiglu", True, False, True, holes=M % 2 == 0, seed=5)


@pytest.mark.parametrize("M,G,N,K", [c for table in (F32, F32_SWIGLU) for cases in table.values() for c in cases])
def test_products_in_fp32(M, G, N, K):
    product_case(M, G, N, K, "f32", "f32", "none", False, True, False, holes=M % 2 == 1)
    if N % 8 == 0:
        product_case(M, G, N, K, "f32", "f32", "swiglu", True, False, True, holes=M % 2 == 0, seed=5)


@pytest.mark.parametrize("kind,M,G,N,K", [(kind, *c) for kind, table in (("bf16", BF16), ("f32", F32))
                                          for cases in table.values() for c in cases])
def test_back_to_the_rows(kind, M, G, N, K):
    grad_case(M, G, K, N, kind, "f32", "x", holes=M % 2 == 1)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,G,N,K", [c for cases in MATRICES.values() for c in cases])
def test_back_to_the_matrices(M, G, N, K, kind):
    grad_case(M, G, N, K, kind, kind, "w", holes=M % 2 == 1)


def test_parts_of_uneven_groups():
    """Groups that differ in rows by far more than a part holds, and one without any."""
    for off in ([0, 100, 100, 13000], [7, 12990, 12991, 13000], [0, 4300, 8600, 13000]):
        grad_case(13000, 3, 40, 72, "bf16", "bf16", "w", offsets=np.int32(off))
        grad_case(13000, 3, 40, 72, "f32", "f32", "w", offsets=np.int32(off))
