"""The MXFP4 product's choice of tiles, on the host (nothing is launched): up to 16 tokens it does not
depend on their number, so that decoding and verifying form a token's sums in the same order."""
import ctypes

import pytest

import q8_block_quantized_act_gb300 as q8
from q8_block_quantized_act_gb300 import build as q8build

SMS = 152


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


def test_plan_refusals():
    p = (ctypes.c_int32 * 4)()
    assert q8.q8act_debug_gemm_mxfp4_plan(SMS, 1, 8, 256, None) == q8.Q8ACT_ERR_NULL
    for args in ((0, 1, 8, 256), (SMS, 0, 8, 256), (SMS, 1, 0, 256), (SMS, 1, 8, 100)):
        assert q8.q8act_debug_gemm_mxfp4_plan(*args, p) == q8.Q8ACT_ERR_DIMS
