"""The entry of the routed-expert calls in C (csrc/calls.c), with stand-ins for the library's functions."""
import ctypes
import os
import sysconfig
import threading
import time

import pytest

import moe_shared_expert_gb300 as mse
from moe_shared_expert_gb300 import _build

NAMES = ("moe_route", "fp8_block_linear", "fp8_block_matmul", "moe_experts_forward")
ARGUMENTS = {"moe_route": 17, "fp8_block_linear": 14, "fp8_block_matmul": 13, "moe_experts_forward": 21}


@pytest.fixture
def calls():
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("no Python headers: calls go through ctypes")
    _build.build()
    from moe_shared_expert_gb300 import _calls
    yield _calls
    _calls.bind(*(ctypes.cast(getattr(mse.lib(), n), ctypes.c_void_p).value for n in NAMES))


def numbers(name, first=0):
    a = [0] * ARGUMENTS[name]
    a[0] = first
    if name == "moe_route":
        a[12] = 1.0
    return a


@pytest.mark.parametrize("name", NAMES)
def test_other_threads_run_during_a_call(calls, name):
    # usleep in the place of a launch that waits for room in its queue: 0.4 s, given as the first argument
    sleeper = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    calls.bind(sleeper, sleeper, sleeper, sleeper)
    ticks, done = [], threading.Event()

    def tick():
        while not done.wait(0.005):
            ticks.append(time.monotonic())

    other = threading.Thread(target=tick)
    other.start()
    begin = time.monotonic()
    status = getattr(calls, name)(*numbers(name, 400000))
    end = time.monotonic()
    done.set()
    other.join()
    assert status == 0 and end - begin >= 0.4
    assert sum(begin < t < end for t in ticks) >= 10


def test_the_entry_in_c_belongs_to_this_interpreter(calls):
    # another Python, or another machine, finds no file of its own and takes ctypes
    assert os.path.basename(_build.CALLS) == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.samefile(calls.__file__, _build.CALLS)


@pytest.mark.parametrize("name,at", [("moe_route", i) for i in (1, 6, 7, 8, 9, 10, 11)]
                         + [("fp8_block_linear", 9), ("fp8_block_matmul", 10), ("moe_experts_forward", 5)])
def test_numbers_beyond_an_int_are_refused(calls, name, at):
    # 2^32 + 1 groups are not one group
    def never(*_):
        raise AssertionError("called")

    made = ctypes.CFUNCTYPE(ctypes.c_int)(never)
    calls.bind(*[ctypes.cast(made, ctypes.c_void_p).value] * 4)
    for number in (2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1):
        a = numbers(name)
        a[at] = number
        with pytest.raises(OverflowError):
            getattr(calls, name)(*a)
