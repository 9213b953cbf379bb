"""Refusals and sizes of the routed-expert operators: argument checks come before any CUDA call."""
import pytest

import moe_shared_expert_gb300 as mse
from moe_shared_expert_gb300 import _build

FAKE = 1 << 20
INF = 1 << 40


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mse.lib()


def code(name):
    return mse.STATUS_CODE[name]


def route(L, **kw):
    a = dict(logits=FAKE, dtype=mse.F32, T=4, E=64, ld=64, bias=None, scoring=1, n_group=8, topk_group=4, group_top=2,
             top_k=8, renormalise=1, scale=1.0, ids=FAKE, weights=FAKE, capacity=32, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.moe_route(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), "MSE_ERR_INVALID_ARG"), (dict(ids=None), "MSE_ERR_INVALID_ARG"),
    (dict(weights=None), "MSE_ERR_INVALID_ARG"), (dict(T=0), "MSE_ERR_INVALID_ARG"),
    (dict(E=0), "MSE_ERR_INVALID_ARG"), (dict(E=1032, ld=1032), "MSE_ERR_INVALID_ARG"),
    (dict(ld=63), "MSE_ERR_INVALID_ARG"), (dict(dtype=2), "MSE_ERR_INVALID_ARG"),
    (dict(scoring=2), "MSE_ERR_INVALID_ARG"), (dict(n_group=0), "MSE_ERR_INVALID_ARG"),
    (dict(n_group=64, topk_group=1, top_k=1), "MSE_ERR_INVALID_ARG"), (dict(topk_group=9), "MSE_ERR_INVALID_ARG"),
    (dict(topk_group=0), "MSE_ERR_INVALID_ARG"), (dict(group_top=3), "MSE_ERR_INVALID_ARG"),
    (dict(top_k=0), "MSE_ERR_INVALID_ARG"), (dict(top_k=33, capacity=INF), "MSE_ERR_INVALID_ARG"),
    (dict(top_k=9, topk_group=1, capacity=INF), "MSE_ERR_INVALID_ARG"),
    (dict(n_group=7), "MSE_ERR_NOT_DIVISIBLE"), (dict(capacity=31), "MSE_ERR_GEOMETRY"),
])
def test_route_refuses(L, kw, want):
    assert route(L, **kw) == code(want)


def test_quantise_refuses(L):
    def call(x=FAKE, rows=5, K=130, ldx=130, br=1, q=FAKE, ldq=144, qc=4 * 144 + 130, s=FAKE, sc=10):
        return L.fp8_block_quantise(x, rows, K, ldx, br, q, ldq, qc, s, sc, None)
    bad = code("MSE_ERR_INVALID_ARG")
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(rows=0), dict(K=0), dict(ldx=129), dict(ldq=129),
               dict(br=2), dict(br=0)):
        assert call(**kw) == bad, kw
    assert call(qc=4 * 144 + 129) == code("MSE_ERR_GEOMETRY")
    assert call(sc=9) == code("MSE_ERR_GEOMETRY")
    assert call(br=128, sc=1) == code("MSE_ERR_GEOMETRY")


def test_products_refuse(L):
    def matmul(xq=FAKE, ldx=512, xs=FAKE, wq=FAKE, ldw=512, ws=FAKE, T=3, N=7, K=500, out=FAKE, dt=mse.BF16, cap=21):
        return L.fp8_block_matmul(xq, ldx, xs, wq, ldw, ws, T, N, K, out, dt, cap, None)

    def linear(x=FAKE, ldx=500, wq=FAKE, ldw=512, ws=FAKE, T=3, N=7, K=500, y=FAKE, dt=mse.BF16, cap=21, buf=FAKE,
               n=1 << 20):
        return L.fp8_block_linear(x, ldx, wq, ldw, ws, T, N, K, y, dt, cap, buf, n, None)
    bad = code("MSE_ERR_INVALID_ARG")
    for kw in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(out=None), dict(T=0), dict(N=-1),
               dict(K=0), dict(ldx=499), dict(ldw=499), dict(dt=5)):
        assert matmul(**kw) == bad, kw
    assert matmul(cap=20) == code("MSE_ERR_GEOMETRY")
    for kw in (dict(x=None), dict(wq=None), dict(ws=None), dict(y=None), dict(T=0), dict(ldx=499), dict(dt=-1)):
        assert linear(**kw) == bad, kw
    assert linear(cap=20) == code("MSE_ERR_GEOMETRY")
    need = mse.fp8_linear_workspace_bytes(3, 7, 500)
    for kw in (dict(buf=None), dict(n=need - 1), dict(buf=FAKE + 128)):
        assert linear(**kw) == code("MSE_ERR_WORKSPACE"), kw


def test_experts_refuse(L):
    T, k, E, H, I = 3, 2, 4, 256, 128
    need = mse.moe_workspace_bytes(T, k, E, H, I)

    def call(x=FAKE, T=T, H=H, ids=FAKE, w=FAKE, k=k, gu=FAKE, ldg=256, sg=FAKE, d=FAKE, ldd=128, sd=FAKE, E=E, I=I,
             first=0, shared=None, y=FAKE, cap=3 * 256, buf=FAKE, n=need):
        return L.moe_experts_forward(x, T, H, ids, w, k, gu, ldg, sg, d, ldd, sd, E, I, first, shared, y, cap, buf, n,
                                     None)
    bad = code("MSE_ERR_INVALID_ARG")
    for kw in (dict(x=None), dict(ids=None), dict(w=None), dict(gu=None), dict(sg=None), dict(d=None), dict(sd=None),
               dict(y=None), dict(T=0), dict(H=0), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(I=0),
               dict(ldg=255), dict(ldd=127), dict(first=-1)):
        assert call(**kw) == bad, kw
    assert call(cap=3 * 256 - 1) == code("MSE_ERR_GEOMETRY")
    for kw in (dict(buf=None), dict(n=need - 1), dict(buf=FAKE + 64)):
        assert call(**kw) == code("MSE_ERR_WORKSPACE"), kw


def test_workspace_sizes(L):
    assert mse.fp8_linear_workspace_bytes(0, 1, 1) == 0 and mse.moe_workspace_bytes(1, 33, 4, 8, 8) == 0
    lin = [mse.fp8_linear_workspace_bytes(T, 2112, 7168) for T in range(1, 300)]
    assert all(a <= b for a, b in zip(lin, lin[1:])) and lin[63] >= 64 * (7168 + 4 * 56)
    for k, E in ((1, 1), (2, 300), (8, 32), (32, 1024)):
        moe = [mse.moe_workspace_bytes(T, k, E, 512, 300) for T in [*range(1, 200), 1000, 5000]]
        assert all(a <= b for a, b in zip(moe, moe[1:]))
    # smaller in any other size: not more
    full = mse.moe_workspace_bytes(100, 8, 64, 1024, 512)
    for smaller in ((99, 8, 64, 1024, 512), (100, 7, 64, 1024, 512), (100, 8, 63, 1024, 512),
                    (100, 8, 64, 1023, 512), (100, 8, 64, 1024, 511)):
        assert mse.moe_workspace_bytes(*smaller) <= full


def test_bindings_refuse():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        mse.moe_route(x, 2)                                        # not on a GPU
    with pytest.raises(ValueError):
        mse.fp8_block_quantise(torch.zeros(4, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mse.fp8_block_linear(x, x, x)
    with pytest.raises(ValueError):
        mse.moe_experts_forward(None, None, None, None, None, None, None)


def test_calls_in_c_take_the_arguments_of_the_library(L):
    import ctypes
    import os
    import sysconfig
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("no Python headers: calls go through ctypes")
    from moe_shared_expert_gb300 import _calls
    names = ("moe_route", "fp8_block_linear", "fp8_block_matmul", "moe_experts_forward")
    _calls.bind(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names))
    calls = {
        "moe_route": [FAKE, mse.F32, 4, 64, 64, None, 1, 7, 4, 2, 8, 1, 1.0, FAKE, FAKE, 32, None],
        "fp8_block_linear": [FAKE, 500, FAKE, 512, FAKE, 3, 7, 500, FAKE, 0, 20, FAKE, 1 << 21, None],
        "fp8_block_matmul": [FAKE, 512, FAKE, FAKE, 512, FAKE, 3, 7, 500, FAKE, 0, 20, None],
        "moe_experts_forward": [FAKE, 3, 256, FAKE, FAKE, 2, FAKE, 256, FAKE, FAKE, 128, FAKE, 4, 128, 0, None, FAKE,
                                3 * 256 - 1, FAKE, 1 << 30, None],
    }
    want = {"moe_route": "MSE_ERR_NOT_DIVISIBLE"}
    for name, a in calls.items():
        f = getattr(_calls, name)
        assert f(*a) == getattr(L, name)(*a) == code(want.get(name, "MSE_ERR_GEOMETRY")), name
        # every pointer argument in turn: null is refused alike
        for i, v in enumerate(a):
            b = [*a[:i], None if v == FAKE else 0, *a[i + 1:]]
            if v is not None and not isinstance(v, float):
                assert f(*b) == getattr(L, name)(*b), (name, i)
        with pytest.raises(TypeError):
            f(*a[:-1])
        with pytest.raises(TypeError):
            f("x", *a[1:])
