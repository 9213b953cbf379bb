"""Rounding to 8-bit integers: gates at the ends of the range, every kernel that the columns choose, more rows than the grid has turns."""
import math

import pytest

from tests import sorted_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

mse = pytest.importorskip("moe_shared_expert_gb300")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from moe_shared_expert_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mse.lib()
    yield
    torch.cuda.synchronize()
    assert mse.poll_device_error() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(x, q, s, rel):
    """q s is silu(gate) up of rows x, each value of which is within `rel` of itself before it is rounded."""
    h = ref.swiglu(x)
    a = h.abs().amax(1)
    # the scale is the largest over 127, in 32 bits; a quotient has two such values, and is rounded to an integer once
    assert bool(((s.double() - a / 127).abs() <= (a / 127) * (rel + 2.0 ** -23)).all())
    assert bool(((q.double() - 127 * h / a[:, None]).abs() <= 0.5 + 127 * 2 * (rel + 2.0 ** -22)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("K", [1, 64, 300, 1500, 3000, 5000, 9000])
def test_gates_whose_exponential_is_nearly_infinite(K, dtype):
    # 1 + e^-g is above 2^126 from g = -87.34 on, and its reciprocal below the normal numbers; e^-g is finite up to 88.72
    g = torch.tensor([-87.0, -87.5, -88.0, -88.5])[torch.randint(0, 4, (5, K), generator=gen(K))]
    x = torch.cat([g, torch.randn(5, K, generator=gen(1)) * 2.0 ** 100], 1).to(dtype)
    q, s = mse.int8_quantise(x.cuda(), swiglu=True)
    # e^-g is off by 1.3 |g| 2^-24 of itself (116 of them) and 2^-22 more, its reciprocal by 2^-23 and, below the normal numbers,
    # by half of 2^-149 of at least 2^-128; three products follow
    close(x, q.cpu(), s.cpu(), (116 + 4 + 2 + 4 + 3) * 2.0 ** -24)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_gates_and_factors_that_are_not_finite(dtype):
    K, odd = 40, [(math.inf, 1.0), (-math.inf, 1.0), (math.nan, 1.0), (0.0, math.inf), (-200.0, -math.inf), (1.0, math.nan), (-math.inf, 0.0)]
    g, u = torch.randn(len(odd) + 1, K, generator=gen(1)), torch.randn(len(odd) + 1, K, generator=gen(2))
    for r, (a, b) in enumerate(odd):
        g[r, 7], u[r, 7] = a, b
    g[-1, 7], u[-1, 7] = -1e30, 1.0    # silu(g) is 0
    x = torch.cat([g, u], 1).to(dtype)
    q, s = mse.int8_quantise(x.cuda(), swiglu=True)
    n = len(odd)
    assert bool(s[:n].isnan().all()) and bool((q[:n] == 0).all()) and bool(s[n].isfinite()) and int(q[n, 7]) == 0


def rows_of_many_sizes(rows, K, dtype, seed):
    """Neighbouring rows differ in size by 2^10 to 2^40: a maximum taken from another row shows."""
    size = 2.0 ** (20 * ((torch.arange(rows) * 7 % 5).double() - 2))[:, None]
    return (torch.randn(rows, K, generator=gen(seed)) * size).to(dtype)


# the columns that each kernel takes, and more rows than its grid has at a time (39,000 of up to 1024, 4,900, 1,200 of more than 8192)
ROWS = [(3, 1025), (64, 1500), (33, 2048), (40_000, 64), (39_500, 260), (10_300, 1100), (5_000, 2300), (5_100, 5000), (2_600, 8200)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,K", ROWS)
def test_rows(rows, K, dtype):
    # (the scale is compared bit for bit with the CPU's quotient: torch divides by a number on the GPU by its reciprocal)
    x = rows_of_many_sizes(rows, K, dtype, K)
    q, s = mse.int8_quantise(x.cuda())
    if dtype is torch.bfloat16:
        want, scale = ref.quantised(x)
    else:   # the quotient in 32 bits
        a = x.abs().amax(1, keepdim=True).clamp_min(ref.FLOOR)
        want, scale = torch.round(x * (127.0 / 512) / a * 512), a[:, 0] / 127
    assert torch.equal(q.cpu().to(want.dtype), want) and torch.equal(s.cpu(), scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,K", ROWS + [(64, 3000), (9, 9000)])
def test_rows_of_swiglu(rows, K, dtype):
    gate = (2 * torch.randn(rows, K, generator=gen(K))).to(dtype)
    x = torch.cat([gate, rows_of_many_sizes(rows, K, dtype, 1)], 1).cuda()
    q, s = mse.int8_quantise(x, swiglu=True)
    # e^-g is off by 1.3 |g| 2^-24 of itself and a few 2^-23 more, |g| < 16 here
    close(x, q, s, 2.0 ** -19)


@pytest.mark.parametrize("T,K", [(700, 300), (300, 700), (5_000, 1100), (1_300, 8200)])
def test_rows_in_fp16_within_a_product(T, K):
    """int8_linear rounds its rows straight to fp16: the product of the same integers as int8_quantise makes."""
    x = rows_of_many_sizes(T, K, torch.bfloat16, K)
    w = (torch.arange(96 * K) % 255 - 127).view(96, K).to(torch.int8)
    wq = torch.zeros(96, -(-K // 16) * 16, dtype=torch.int8, device="cuda")[:, :K].copy_(w)
    ws = torch.rand(96, generator=gen(2)).cuda()
    assert mse.int8_launch_plan(T, 96, K)["tile_rows"] > 4
    q, s = ref.quantised(x)
    y = mse.int8_linear(x.cuda(), wq, ws, y_dtype=torch.float32)
    assert torch.equal(y, ref.product(q.cuda(), s.cuda(), wq, ws))
