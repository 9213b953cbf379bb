"""What the sorted rows' calls and the 8-bit integer products refuse: the library before any CUDA call, the bindings before the library."""
import pytest

torch = pytest.importorskip("torch")

import moe_shared_expert_gb300 as mse
from moe_shared_expert_gb300 import _build, routed, rows
from tests.test_routed_bindings_cpu import On

FAKE, FAR = 1 << 20, 1 << 50   # never read: the calls fail before; FAR lies behind everything at FAKE
MANY = 1 << 62
BAD, SMALL, SPACE = (mse.STATUS_CODE["MSE_ERR_" + n] for n in ("INVALID_ARG", "GEOMETRY", "WORKSPACE"))
GOOD = mse.STATUS_CODE["MSE_ERR_UNSUPPORTED_DEVICE"]   # all arguments were taken; there is no GPU here

CALLS = {
    "moe_sort": dict(x=FAKE, value_bytes=2, T=5, H=8, ldx=8, ids=FAKE, top_k=2, E=4, first_expert=0, scales=FAKE, rows=FAR, ldr=8,
                     rows_capacity=80, row_scales=FAR + 4096, place=FAR + 8192, offsets=FAKE, workspace=FAKE, workspace_bytes=1 << 20, stream=None),
    "moe_unsort": dict(rows=FAKE, rows_dtype=0, n_rows=10, ldr=8, place=FAKE, weights=FAKE, T=5, H=8, top_k=2, base=None, y=FAR,
                       y_dtype=0, y_capacity=40, stream=None),
    "moe_unsort_backward": dict(dy=FAKE, dy_dtype=0, place=FAKE, weights=FAKE, rows=FAKE, rows_dtype=0, ldr=8, n_rows=10, T=5, H=8,
                                top_k=2, drows=FAR, ldd=8, drows_capacity=80, dweights=FAKE, stream=None),
    "int8_quantise": dict(x=FAKE, x_dtype=0, rows=5, K=8, ldx=16, swiglu=1, last=None, q=FAR, ldq=16, q_capacity=80, scales=FAKE,
                          stream=None),
    "int8_matmul": dict(xq=FAKE, ldx=16, xs=FAKE, wq=FAKE, ldw=16, ws=FAKE, T=5, N=7, K=9, out=FAR, out_dtype=0, out_capacity=35,
                        workspace=FAKE, workspace_bytes=1 << 20, stream=None),
    "int8_grouped_matmul": dict(xq=FAKE, ldx=16, xs=FAKE, offsets=FAKE, groups=3, wq=FAKE, ldw=16, ws=FAKE, T=5, N=7, K=9, out=FAR,
                                out_dtype=0, out_capacity=35, workspace=FAKE, workspace_bytes=1 << 20, stream=None),
    "int8_linear": dict(x=FAKE, x_dtype=1, ldx=16, wq=FAKE, ldw=16, ws=FAKE, T=5, N=7, K=9, y=FAR, y_dtype=0, y_capacity=35,
                        workspace=FAKE, workspace_bytes=1 << 20, stream=None),
}
POINTERS = {"x", "ids", "rows", "place", "offsets", "y", "dy", "drows", "q", "scales", "xq", "xs", "wq", "ws", "out"}
OPTIONAL = {("moe_sort", "scales"), ("int8_quantise", "rows")}   # (the latter a number)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mse.lib()


def status(L, name, **other):
    return getattr(L, name)(*{**CALLS[name], **other}.values())


@pytest.mark.parametrize("name", CALLS)
def test_good_arguments_reach_the_device(L, name):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    assert status(L, name) == GOOD


@pytest.mark.parametrize("name,arg", [(n, a) for n, c in CALLS.items() for a in c if a in POINTERS and (n, a) not in OPTIONAL])
def test_null_pointers(L, name, arg):
    assert status(L, name, **{arg: None}) == BAD


@pytest.mark.parametrize("name,arg", [(n, a) for n, c in CALLS.items() for a in c if a in ("T", "H", "N", "K", "rows", "E", "top_k", "n_rows", "groups")
                                      and not (n in ("moe_sort", "moe_unsort", "moe_unsort_backward") and a == "rows")])
def test_sizes(L, name, arg):
    for wrong in (0, -1, (1 << 30) + 1):
        assert status(L, name, **{arg: wrong}) == BAD, wrong


@pytest.mark.parametrize("name,other", [
    ("moe_sort", dict(top_k=33)), ("moe_sort", dict(E=1025)), ("moe_sort", dict(T=1 << 29, top_k=4)), ("moe_sort", dict(value_bytes=8)),
    ("moe_sort", dict(value_bytes=0)), ("moe_sort", dict(ldx=7)), ("moe_sort", dict(ldr=7)), ("moe_sort", dict(first_expert=-1)),
    ("moe_sort", dict(scales=None)), ("moe_sort", dict(row_scales=None)), ("moe_sort", dict(rows=FAKE + 64)), ("moe_sort", dict(ldx=(1 << 32) + 1)),
    ("moe_sort", dict(place=FAKE)), ("moe_sort", dict(place=FAKE + 36)), ("moe_sort", dict(row_scales=FAKE)),
    ("moe_sort", dict(row_scales=FAKE + 16)),
    ("moe_sort", dict(H=(1 << 22) + 1, ldx=1 << 23, ldr=1 << 23, rows_capacity=MANY)),
    ("moe_unsort", dict(rows_dtype=2)), ("moe_unsort", dict(y_dtype=-1)), ("moe_unsort", dict(ldr=7)), ("moe_unsort", dict(top_k=33)),
    ("moe_unsort", dict(y=FAKE + 158)), ("moe_unsort", dict(base=FAR + 2)),
    ("moe_unsort_backward", dict(dweights=None)), ("moe_unsort_backward", dict(weights=None)), ("moe_unsort_backward", dict(rows=None)),
    ("moe_unsort_backward", dict(ldd=7)), ("moe_unsort_backward", dict(ldr=7)), ("moe_unsort_backward", dict(dy_dtype=3)),
    ("moe_unsort_backward", dict(drows=FAKE + 2)), ("moe_unsort_backward", dict(drows=FAR, rows=FAR, ldr=9)),
    ("int8_quantise", dict(x_dtype=5)), ("int8_quantise", dict(ldx=15)), ("int8_quantise", dict(ldq=7)), ("int8_quantise", dict(q=FAKE + 3)),
    ("int8_matmul", dict(K=1 << 17, ldx=1 << 18, ldw=1 << 18, workspace_bytes=MANY)), ("int8_matmul", dict(ldx=8)), ("int8_matmul", dict(ldw=8)),
    ("int8_matmul", dict(out_dtype=2)), ("int8_matmul", dict(out=FAKE)), ("int8_matmul", dict(N=(1 << 22) + 1, out_capacity=MANY)),
    ("int8_grouped_matmul", dict(groups=1025)), ("int8_grouped_matmul", dict(groups=1024, N=1 << 21, out_capacity=MANY)),
    ("int8_grouped_matmul", dict(out=FAKE + 40)), ("int8_linear", dict(x_dtype=2)), ("int8_linear", dict(ldx=8)),
], ids=lambda v: v if isinstance(v, str) else "-".join(v))
def test_bad_arguments(L, name, other):
    assert status(L, name, **other) == BAD


@pytest.mark.parametrize("name,arg", [("moe_sort", "rows_capacity"), ("moe_unsort", "y_capacity"), ("moe_unsort_backward", "drows_capacity"),
                                      ("int8_quantise", "q_capacity"), ("int8_matmul", "out_capacity"),
                                      ("int8_grouped_matmul", "out_capacity"), ("int8_linear", "y_capacity")])
def test_small_outputs(L, name, arg):
    least = {"int8_quantise": 4 * 16 + 8}.get(name, CALLS[name][arg])
    assert status(L, name, **{arg: least - 1}) == SMALL


@pytest.mark.parametrize("name", ["moe_sort", "int8_matmul", "int8_grouped_matmul", "int8_linear"])
def test_workspaces(L, name):
    for wrong in (dict(workspace=None), dict(workspace=FAKE + 16), dict(workspace_bytes=0)):
        assert status(L, name, **wrong) == SPACE


def test_workspaces_of_fewer_tokens_are_no_larger(L):
    sizes = [L.moe_sort_workspace_bytes(T, 8, 64) for T in range(1, 20000, 37)]
    assert sizes == sorted(sizes)
    sizes = [L.int8_workspace_bytes(T, 700, 1000, 1) for T in range(1, 9000, 31)]
    assert sizes == sorted(sizes)
    assert L.moe_sort_workspace_bytes(0, 8, 64) == 0 == L.int8_workspace_bytes(5, 7, 1 << 17, 1)


# ------------------------------------------------------------------------------------ bindings

@pytest.fixture
def reached(monkeypatch):
    _build.build()
    rows._ready()
    names = []

    class C:
        pass

    for n in CALLS:
        setattr(C, n, staticmethod(lambda *a, n=n: names.append(n) or 0))
    monkeypatch.setattr(rows, "_C", C)
    monkeypatch.setattr(routed, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(routed, "_current", lambda: 0)
    return names


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def i8(*shape):
    return torch.zeros(*shape, dtype=torch.int8)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


SPACE_T = torch.zeros(1 << 16, dtype=torch.uint8)
BINDINGS = {
    "moe_sort": (mse.moe_sort, dict(x=bf16(5, 8), ids=i32(5, 2), num_experts=4, scales=torch.zeros(5), rows=bf16(10, 8),
                                    row_scales=torch.zeros(10), place=i32(5, 2), offsets=i32(5), workspace=SPACE_T)),
    "moe_unsort": (mse.moe_unsort, dict(rows=bf16(10, 8), place=i32(5, 2), weights=torch.zeros(5, 2), base=bf16(5, 8), y=bf16(5, 8))),
    "moe_unsort_backward": (mse.moe_unsort_backward, dict(dy=bf16(5, 8), place=i32(5, 2), rows=bf16(10, 8), weights=torch.zeros(5, 2),
                                                          drows=bf16(10, 8), dweights=torch.zeros(5, 2))),
    "int8_quantise": (mse.int8_quantise, dict(x=bf16(5, 8), offsets=i32(3), q=i8(5, 8), scales=torch.zeros(5))),
    "int8_matmul": (mse.int8_matmul, dict(xq=i8(5, 8), xs=torch.zeros(5), wq=i8(7, 8), ws=torch.zeros(7), out=bf16(5, 7), workspace=SPACE_T)),
    "int8_grouped_matmul": (mse.int8_grouped_matmul, dict(xq=i8(5, 8), xs=torch.zeros(5), offsets=i32(4), wq=i8(3, 7, 8), ws=torch.zeros(3, 7),
                                                          out=bf16(5, 7), workspace=SPACE_T)),
    "int8_linear": (mse.int8_linear, dict(x=bf16(5, 8), wq=i8(7, 8), ws=torch.zeros(7), y=bf16(5, 7), workspace=SPACE_T)),
}


def arguments(op, index=0, **other):
    f, a = BINDINGS[op]
    return f, {n: On(v, index) if isinstance(v, torch.Tensor) else v for n, v in {**a, **other}.items()}


@pytest.mark.parametrize("op", BINDINGS)
def test_bindings_reach_the_library(reached, op):
    f, a = arguments(op)
    f(**a)
    assert reached == [op]


@pytest.mark.parametrize("op,arg", [(op, n) for op, (_, a) in BINDINGS.items() for n, v in a.items() if isinstance(v, torch.Tensor)])
def test_bindings_refuse_another_device_or_the_cpu(reached, op, arg):
    f, a = arguments(op)
    for wrong in (On(a[arg].t, 1), a[arg].t):
        with pytest.raises(ValueError):
            f(**{**a, arg: wrong})
    f, a = arguments(op, index=1)
    with pytest.raises(ValueError):
        f(**a)
    assert reached == []


@pytest.mark.parametrize("op,other", [
    ("moe_sort", dict(x=torch.zeros(5, 8, dtype=torch.float64))), ("moe_sort", dict(ids=torch.zeros(5, 2, dtype=torch.int64))),
    ("moe_sort", dict(ids=i32(4, 2))), ("moe_sort", dict(rows=bf16(9, 8))), ("moe_sort", dict(rows=torch.zeros(10, 8))),
    ("moe_sort", dict(offsets=i32(4))), ("moe_sort", dict(place=i32(2, 5))), ("moe_sort", dict(x=bf16(8, 5).t())),
    ("moe_unsort", dict(weights=torch.zeros(5, 3))), ("moe_unsort", dict(base=torch.zeros(5, 8))), ("moe_unsort", dict(y=bf16(5, 9))),
    ("moe_unsort", dict(rows=torch.zeros(10, 8, dtype=torch.float16))),
    ("moe_unsort_backward", dict(rows=bf16(10, 9))), ("moe_unsort_backward", dict(drows=bf16(11, 8))),
    ("moe_unsort_backward", dict(drows=torch.zeros(10, 8))), ("moe_unsort_backward", dict(place=i32(4, 2))),
    ("int8_quantise", dict(q=i8(5, 9))), ("int8_quantise", dict(scales=torch.zeros(4))), ("int8_quantise", dict(x=torch.zeros(5, 8, dtype=torch.float16))),
    ("int8_matmul", dict(wq=i8(7, 9))), ("int8_matmul", dict(xs=torch.zeros(6))), ("int8_matmul", dict(ws=torch.zeros(8))),
    ("int8_matmul", dict(xq=torch.zeros(5, 8, dtype=torch.uint8))), ("int8_grouped_matmul", dict(offsets=i32(3))),
    ("int8_grouped_matmul", dict(wq=i8(7, 8))), ("int8_grouped_matmul", dict(ws=torch.zeros(21))), ("int8_linear", dict(x=i8(5, 8))),
    ("int8_linear", dict(wq=i8(8, 7).t())),
], ids=lambda v: v if isinstance(v, str) else "-".join(v))
def test_bindings_refuse_other_types_and_shapes(reached, op, other):
    f, a = arguments(op, **other)
    with pytest.raises(ValueError):
        f(**a)
    assert reached == []


def test_bindings_refuse_what_does_not_go_together(reached):
    f, a = arguments("moe_sort")
    with pytest.raises(ValueError, match="row_scales"):
        f(**{**a, "scales": None})
    f, a = arguments("moe_unsort_backward")
    with pytest.raises(ValueError, match="rows"):
        f(**{**a, "rows": None})
    with pytest.raises(ValueError, match="dweights"):
        f(**{**a, "weights": None})
    f, a = arguments("int8_quantise", x=bf16(5, 9), q=None)
    with pytest.raises(ValueError, match="even"):
        f(**{**a, "swiglu": True})
    assert reached == []


# ------------------------------------------------------------------------------------ the entry in C

ARGUMENTS = {n: len(c) for n, c in CALLS.items()}
FLAGS = {"moe_sort": (1, 6), "moe_unsort": (1, 8, 11), "moe_unsort_backward": (1, 5, 10), "int8_quantise": (1, 5), "int8_matmul": (10,),
         "int8_grouped_matmul": (12,), "int8_linear": (1, 10)}


@pytest.fixture
def entry():
    import ctypes
    import os
    import sysconfig
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("no Python headers: calls go through ctypes")
    _build.build()
    from moe_shared_expert_gb300 import _calls
    seen = []
    kinds = {n: list(getattr(mse.lib(), n).argtypes) for n in CALLS}
    made = [ctypes.CFUNCTYPE(ctypes.c_int, *kinds[n])(lambda *a, n=n: seen.append((n, a)) or 5) for n in rows._NAMES]
    _calls.bind_rows(*(ctypes.cast(f, ctypes.c_void_p).value for f in made))
    yield _calls, seen
    _calls.bind_rows(*(ctypes.cast(getattr(mse.lib(), n), ctypes.c_void_p).value for n in rows._NAMES))


@pytest.mark.parametrize("name", CALLS)
def test_the_entry_in_c_hands_on_every_argument(entry, name):
    calls, seen = entry
    a = list(range(1, ARGUMENTS[name] + 1))
    assert getattr(calls, name)(*a) == 5 and seen == [(name, tuple(a))]
    with pytest.raises(TypeError):
        getattr(calls, name)(*a[:-1])


@pytest.mark.parametrize("name,at", [(n, i) for n, flags in FLAGS.items() for i in flags])
def test_the_entry_in_c_refuses_numbers_beyond_an_int(entry, name, at):
    calls, seen = entry
    for number in (2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1):
        a = [0] * ARGUMENTS[name]
        a[at] = number
        with pytest.raises(OverflowError):
            getattr(calls, name)(*a)
    assert seen == []
