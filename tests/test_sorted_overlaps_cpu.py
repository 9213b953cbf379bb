"""Outputs that lie over an input or over another output are refused before any CUDA call: CTAs read while others write."""
import itertools

import pytest

torch = pytest.importorskip("torch")

import moe_shared_expert_gb300 as mse
from moe_shared_expert_gb300 import _build
from tests.test_sorted_refusals_cpu import BAD, CALLS, GOOD

# name: (other arguments, bytes of each pointer's memory, written ones, read ones, pairs that may be the same memory)
CASES = {
    "moe_sort": (dict(ldx=9, ldr=10, rows_capacity=98),
                 dict(x=(4 * 9 + 8) * 2, ids=40, scales=20, rows=(9 * 10 + 8) * 2, row_scales=40, place=40, offsets=20, workspace=256),
                 ("rows", "place", "row_scales"), ("x", "ids", "scales", "offsets", "workspace"), ()),
    "moe_unsort": (dict(ldr=9), dict(rows=(9 * 9 + 8) * 2, place=40, weights=40, base=80, y=80), ("y",),
                   ("rows", "place", "weights", "base"), (("y", "base"),)),
    "moe_unsort_backward": (dict(ldr=9, ldd=10, drows_capacity=98),
                            dict(dy=80, place=40, weights=40, rows=(9 * 9 + 8) * 2, drows=(9 * 10 + 8) * 2, dweights=40),
                            ("drows",), ("dy", "place", "weights", "rows", "dweights"), ()),
    "int8_quantise": (dict(ldx=17), dict(x=(4 * 17 + 16) * 2, last=4, q=4 * 16 + 8, scales=20), ("q",), ("x", "last", "scales"), ()),
    "int8_matmul": (dict(ldx=17), dict(xq=4 * 17 + 9, xs=20, wq=6 * 16 + 9, ws=28, out=70, workspace=1024), ("out",),
                    ("xq", "xs", "wq", "ws", "workspace"), ()),
    "int8_grouped_matmul": (dict(ldx=17, out_dtype=1), dict(xq=4 * 17 + 9, xs=20, offsets=16, wq=20 * 16 + 9, ws=84, out=140, workspace=1024),
                            ("out",), ("xq", "xs", "offsets", "wq", "ws", "workspace"), ()),
    "int8_linear": (dict(ldx=17), dict(wq=6 * 16 + 9, ws=28, y=70, workspace=1024, x=(4 * 17 + 9) * 4), ("y",), ("wq", "ws", "workspace"), ()),
}


@pytest.fixture(scope="module")
def L():
    _build.build()
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    return mse.lib()


def arguments(name):
    """The call's arguments, every pointer to memory of its own."""
    other, sizes, *_ = CASES[name]
    return {**CALLS[name], **other, **{p: (i + 1) << 40 for i, p in enumerate(sizes)}}


@pytest.mark.parametrize("name", CASES)
def test_memory_apart_is_taken(L, name):
    assert getattr(L, name)(*arguments(name).values()) == GOOD


def pairs():
    for name, (_, sizes, written, read, same) in CASES.items():
        for w, o in itertools.chain(itertools.product(written, read), itertools.combinations(written, 2)):
            yield name, w, o, sizes[w], sizes[o], (w, o) in same


@pytest.mark.parametrize("name,w,o,w_bytes,o_bytes,same", list(pairs()), ids=lambda v: str(v))
def test_memory_that_meets_is_refused(L, name, w, o, w_bytes, o_bytes, same):
    a = arguments(name)

    def at(shift):
        return getattr(L, name)(*{**a, w: a[o] + shift}.values())

    # (a workspace's address is a multiple of 256: what lies over it moves, not the workspace)
    for shift in (1 - w_bytes, o_bytes - 1):
        assert at(shift) == BAD, shift
    assert same or at(0) == BAD
    for shift in (-w_bytes, o_bytes):   # side by side
        assert at(shift) == GOOD, shift


def test_what_may_lie_over_what(L):
    a = arguments("moe_unsort_backward")
    a.update(ldd=9, drows_capacity=89, drows=a["rows"], dweights=a["weights"])
    assert L.moe_unsort_backward(*a.values()) == GOOD
    a = arguments("moe_unsort")
    assert L.moe_unsort(*{**a, "y": a["base"]}.values()) == GOOD
    a = arguments("int8_linear")
    for shift in (-69, 0, 300):
        assert L.int8_linear(*{**a, "y": a["x"] + shift}.values()) == GOOD
    # without weights, rows is not read
    a = arguments("moe_unsort_backward")
    a.update(weights=None, dweights=None, rows=a["drows"] + 2)
    assert L.moe_unsort_backward(*a.values()) == GOOD
