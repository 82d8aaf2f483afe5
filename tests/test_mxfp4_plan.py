"""The MXFP4 product's choice of tiles, on the host (nothing is launched): up to 16 tokens it does not
depend on their number, so that decoding and verifying form a token's sums in the same order."""
import ctypes

import pytest

import q8_block_quantized_act_gb300 as q8
from q8_block_quantized_act_gb300 import build as q8build

SMS = 152

# Sizes that between them reach every variant of the product: (m, n, k) -> (tokens a tile, CTAs a tile's k
# or 0 for pairs, CTAs to an SM, activation quantized by the CTAs).  tests/test_gpu_mxfp4_plans.py runs them.
REACHED = {
    (1, 4096, 4096): (16, 4, 1, 1), (7, 185, 2048): (16, 8, 1, 1), (16, 128, 4096): (16, 8, 1, 1),
    (2, 5719, 7680): (16, 2, 1, 1), (3, 4999, 3840): (16, 2, 1, 1), (5, 1001, 2560): (16, 8, 1, 1),
    (2, 9900, 4096): (16, 1, 1, 1), (1, 9900, 4352): (16, 1, 1, 0),          # 16 steps of k are kept at most
    (10, 300, 6144): (16, 8, 1, 1), (11, 300, 6144): (16, 8, 1, 0),          # 32 token-steps a CTA at most
    (12, 19467, 256): (16, 1, 2, 1), (13, 19467, 256): (16, 1, 2, 0),        # 12 with two CTAs to an SM
    (6, 19999, 512): (16, 1, 2, 1), (7, 19999, 512): (16, 1, 2, 0),
    (5, 4900, 3584): (16, 2, 1, 0), (11, 1928, 2560): (16, 4, 1, 0), (1, 2500, 20480): (16, 4, 1, 0),
    (29, 1941, 2560): (32, 1, 1, 0), (23, 4866, 3584): (32, 2, 1, 0), (17, 3844, 8704): (32, 4, 1, 0),
    (25, 50, 2048): (32, 8, 1, 0), (17, 19531, 256): (32, 1, 2, 0),
    (49, 333, 2560): (64, 1, 1, 0), (33, 4912, 4608): (64, 2, 1, 0), (971, 200, 4608): (64, 4, 1, 0),
    (34, 70, 4096): (64, 8, 1, 0), (33, 19891, 256): (64, 1, 2, 0),
    (65, 9746, 256): (128, 1, 1, 0), (67, 5905, 14592): (128, 2, 1, 0), (68, 2888, 11520): (128, 4, 1, 0),
    (112, 954, 15872): (128, 8, 1, 0), (131, 12935, 256): (192, 1, 1, 0),
    (129, 9731, 2304): (192, 0, 1, 0), (65, 20164, 3328): (192, 0, 1, 0),    # pairs: whole, cut in three
    (193, 9829, 1280): (256, 0, 1, 0), (402, 13098, 2304): (256, 0, 1, 0),   # whole, cut in two,
    (195, 20644, 2304): (256, 0, 1, 0),                                      # in four
}


@pytest.fixture(scope="module", autouse=True)
def built():
    q8build.build()


def plan(m, n, k, sms=SMS):
    """(tokens a tile, CTAs a tile's k or 0 for pairs, CTAs to an SM, activation quantized by the CTAs)"""
    p = (ctypes.c_int32 * 4)()
    q8.check(q8.q8act_debug_gemm_mxfp4_plan(sms, m, n, k, p))
    return tuple(p)


def test_few_tokens_have_one_plan():
    splits = set()
    for n in [*range(1, 129, 9), *range(128, 20480, 331), 4096, 5120, 5152, 20480, 64448, 10 ** 6]:
        for k in [256, 512, 768, 1024, 1280, 1792, 2048, 2304, 2560, 4096, 5120, 7168, 8192, 10240, 20480, 65536]:
            plans = {plan(m, n, k)[:3] for m in range(1, 17)}
            assert len(plans) == 1, (n, k, plans)
            splits |= plans
    assert splits == {(16, 1, 1), (16, 2, 1), (16, 4, 1), (16, 8, 1), (16, 1, 2)}


def test_variants_are_reached():
    assert {size: plan(*size) for size in REACHED} == REACHED


def test_plan_refusals():
    p = (ctypes.c_int32 * 4)()
    assert q8.q8act_debug_gemm_mxfp4_plan(SMS, 1, 8, 256, None) == q8.Q8ACT_ERR_NULL
    for args in ((0, 1, 8, 256), (SMS, 0, 8, 256), (SMS, 1, 0, 256), (SMS, 1, 8, 100)):
        assert q8.q8act_debug_gemm_mxfp4_plan(*args, p) == q8.Q8ACT_ERR_DIMS
