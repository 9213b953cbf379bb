"""Limits of the routed-expert operators' sizes: refused before any CUDA call."""
import pytest

import moe_shared_expert_gb300 as mse
from moe_shared_expert_gb300 import _build

FAKE = 1 << 20
MANY = 1 << 62


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mse.lib()


@pytest.mark.parametrize("kw", [dict(rows=(1 << 30) + 1), dict(K=(1 << 22) + 1, ldx=1 << 23, ldq=1 << 23),
                                dict(ldx=(1 << 32) + 1), dict(rows=1 << 30, K=1 << 22, ldx=1 << 22, ldq=1 << 22, br=128)])
def test_quantise_refuses_sizes_beyond_its_limits(L, kw):
    a = dict(rows=5, K=130, ldx=130, br=1, ldq=144)
    a.update(kw)
    assert L.fp8_block_quantise(FAKE, a["rows"], a["K"], a["ldx"], a["br"], FAKE, a["ldq"], MANY, FAKE, MANY, None) == \
        mse.STATUS_CODE["MSE_ERR_INVALID_ARG"]


@pytest.mark.parametrize("kw", [dict(T=(1 << 30) + 1), dict(N=(1 << 22) + 1), dict(K=(1 << 22) + 1, ld=1 << 23),
                                dict(ld=(1 << 32) + 16)])
def test_products_refuse_sizes_beyond_their_limits(L, kw):
    a = dict(T=3, N=7, K=512, ld=512)
    a.update(kw)
    assert L.fp8_block_matmul(FAKE, a["ld"], FAKE, FAKE, a["ld"], FAKE, a["T"], a["N"], a["K"], FAKE, mse.F32, MANY, None) == \
        mse.STATUS_CODE["MSE_ERR_INVALID_ARG"]


def test_launch_plans_refuse_what_the_calls_refuse(L):
    import ctypes
    out = (ctypes.c_int32 * 8)()
    bad = mse.STATUS_CODE["MSE_ERR_INVALID_ARG"]
    assert L.mse_fp8_launch_plan(3, 7, 500, None) == bad and L.mse_moe_launch_plan(3, 2, 4, 256, 128, None) == bad
    for sizes in ((0, 7, 500), (3, 0, 500), (3, 7, -1), ((1 << 30) + 1, 7, 500), (3, (1 << 22) + 1, 500)):
        assert L.mse_fp8_launch_plan(*sizes, out) == bad, sizes
    for sizes in ((0, 2, 4, 256, 128), (3, 33, 4, 256, 128), (3, 2, 1025, 256, 128), (3, 2, 4, 0, 128), (1 << 29, 3, 4, 256, 128)):
        assert L.mse_moe_launch_plan(*sizes, out) == bad, sizes
