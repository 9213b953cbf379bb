"""Routed-expert operators at the edges of their arguments: infinite and undefined logits and biases, sizes beyond a
grid's second dimension."""
import math

import pytest

from tests.helpers import kernel_path
from tests.test_gpu_routed import gen, make_experts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

mse = pytest.importorskip("moe_shared_expert_gb300")

LOWEST = torch.finfo(torch.float32).min
# n_group, topk_group, group_top
GROUPS = [(1, 1, 1), (4, 2, 2), (4, 2, 1), (8, 3, 2)]


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


# ------------------------------------------------------------------------------------ an infinite logit

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("groups", GROUPS, ids=str)
@pytest.mark.parametrize("E", [40, 320, 1000])
def test_softmax_of_an_infinite_logit_is_nan(E, groups, renormalise, with_bias, dtype):
    # e^(l - max) / sum is NaN for every open expert: the choices are equal, the weights NaN
    G, keep, top = groups
    logits = torch.randn(5, E, generator=gen(E)).to(dtype)
    logits[1, E // 2] = math.inf
    logits[2, 0] = logits[2, E - 1] = math.inf
    logits[3, ::2] = -math.inf
    logits[3, 1] = math.inf
    logits[4] = -math.inf
    logits[4, E - 2] = math.inf
    bias = torch.linspace(-1, 1, E) if with_bias else None
    call = dict(scoring="softmax", bias=None if bias is None else bias.cuda(), n_group=G, topk_group=keep,
                group_top=top, renormalise=renormalise)
    ids, w = mse.moe_route(logits.cuda(), 6, **call)
    ids, w = ids.cpu(), w.cpu()
    size = E // G
    for t in range(1, 5):
        open_ = [e for e in range(E) if float(logits[t, e]) > -math.inf]
        kept = sorted({e // size for e in open_})[:keep if G > 1 else None]
        want = [e for e in open_ if e // size in kept][:6]
        assert ids[t].tolist() == want + [-1] * (6 - len(want))
        assert torch.isnan(w[t, :len(want)]).all() and not w[t, len(want):].any()
    # the other tokens are as without it
    alone, w0 = mse.moe_route(logits[:1].cuda(), 6, **call)
    assert torch.equal(ids[:1], alone.cpu()) and torch.equal(w[:1], w0.cpu())


def test_an_infinite_logit_reaches_the_layers_output():
    E, H, I, T = 6, 256, 128, 4
    weights = make_experts(E, H, I, 3)
    x = torch.randn(T, H, generator=gen(4)).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=gen(5))
    logits[2, 3] = math.inf
    y = mse.moe_experts_forward(x, *mse.moe_route(logits.cuda(), 2, scoring="softmax"), *weights, shared=x)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3]]).all()


def test_sigmoid_of_an_infinite_logit_is_one():
    logits = torch.zeros(2, 50)
    logits[0, 9] = logits[0, 33] = math.inf
    ids, w = mse.moe_route(logits.cuda(), 3, scoring="sigmoid", renormalise=False)
    assert ids.cpu().tolist() == [[9, 33, 0], [0, 1, 2]] and w.cpu().tolist() == [[1.0, 1.0, 0.5], [0.5] * 3]


# ------------------------------------------------------------------------------------ a bias that is NaN, infinite or lowest

@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_a_nan_bias_counts_for_nothing_in_its_group(scoring):
    E, G = 64, 2
    for nan_at in (19, 3, 35):
        logits = torch.full((1, E), -8.0)
        logits[0, 5], logits[0, 5 + 32], logits[0, 6 + 32] = 3.0, 2.5, 2.4     # one good expert against two
        # lane r of a group's sixteen has experts r and r + 16: the best one, then the undefined one, and the other way
        best = (nan_at + 16) % 32 + nan_at // 32 * 32
        if nan_at < 32:
            logits[0, 5], logits[0, best] = -8.0, 3.0
        logits[0, nan_at] = 6.0
        bias = torch.zeros(E)
        bias[nan_at] = math.nan
        ids, w = mse.moe_route(logits.cuda(), 2, scoring=scoring, bias=bias.cuda(), n_group=G, topk_group=1)
        assert ids.cpu().tolist() == [[37, 38]], nan_at
        assert torch.isfinite(w).all()
        # without groups: the expert is never chosen
        ids, _ = mse.moe_route(logits.cuda(), E, scoring=scoring, bias=bias.cuda()) if E <= 32 else \
            mse.moe_route(logits.cuda(), 32, scoring=scoring, bias=bias.cuda())
        assert nan_at not in ids.cpu()[0].tolist()


@pytest.mark.parametrize("n_group", [1, 2])
def test_an_infinite_bias(n_group):
    # -inf: no choice is lower, the expert is never chosen; +inf: always, equal ones by index
    E = 40
    bias = torch.zeros(E)
    bias[3:] = -math.inf
    bias[[30, 10]] = math.inf
    ids, w = mse.moe_route(torch.zeros(1, E).cuda(), 6, bias=bias.cuda(), n_group=n_group, topk_group=1 if n_group == 1 else 2)
    assert ids.cpu().tolist() == [[10, 30, 0, 1, 2, -1]]
    assert torch.allclose(w.cpu(), torch.tensor([[0.2] * 5 + [0.0]]))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("low", [LOWEST, -3.3895313892515355e38, -1e38, -1e4])
@pytest.mark.parametrize("E,k", [(8, 8), (40, 12), (500, 9)])
def test_a_low_bias_puts_an_expert_last(E, k, low, scoring):
    # the bias moves the choice; it is the logit that closes an expert
    logits = torch.randn(3, E, generator=gen(E)) * 1e-3
    bias = torch.zeros(E)
    bias[2:E - 2] = low
    ids, w = mse.moe_route(logits.cuda(), k, scoring=scoring, bias=bias.cuda(), renormalise=False)
    score = torch.sigmoid(logits.double()) if scoring == "sigmoid" else torch.softmax(logits.double(), 1)
    for t in range(3):
        first = sorted((0, 1, E - 2, E - 1), key=lambda e: -float(logits[t, e]))
        rest = list(range(2, E - 2))
        if low == -1e4:   # its rounding leaves an order among the low ones
            got = ids.cpu()[t].tolist()
            assert got[:4] == first and set(got[4:]) <= set(rest) and len(set(got)) == k
        else:
            assert ids.cpu()[t].tolist() == (first + rest)[:k]
        assert torch.allclose(w.cpu()[t].double(), score[t][ids.cpu()[t].long()], rtol=1e-6)


@pytest.mark.parametrize("group_top", [1, 2])
def test_a_low_bias_in_every_group(group_top):
    E, G = 48, 4
    logits = torch.zeros(2, E)
    logits[1, :12] = -math.inf                     # the first group is closed to the second token
    bias = torch.full((E,), LOWEST)
    ids, w = mse.moe_route(logits.cuda(), 3, bias=bias.cuda(), n_group=G, topk_group=2, group_top=group_top)
    assert ids.cpu().tolist() == [[0, 1, 2], [12, 13, 14]]
    assert torch.allclose(w.cpu(), torch.full((2, 3), 1 / 3), rtol=1e-6)


def test_empty_slots_have_weight_zero_whatever_the_scale():
    logits = torch.full((2, 9), -math.inf)
    logits[1, 4] = 0.0
    for scale in (math.inf, -1.0, math.nan):
        ids, w = mse.moe_route(logits.cuda(), 2, scale=scale)
        assert ids.cpu().tolist() == [[-1, -1], [4, -1]]
        w = w.cpu()
        assert [math.copysign(1.0, v) * (v == 0) for v in (*w[0].tolist(), float(w[1, 1]))] == [1.0] * 3, scale


# ------------------------------------------------------------------------------------ sizes beyond 65535 tiles

@pytest.mark.parametrize("N", [1048560, 1048561, 1048700, 2100001])
def test_generic_product_of_many_weight_rows(N):
    T, K, pitch = 3, 20, 21                        # rows of an odd pitch: the generic kernel; whole numbers: no rounding
    g = gen(N)
    w = torch.randint(-8, 9, (N, K), generator=g).float()
    x = torch.randint(-8, 9, (T, K), generator=g).float()
    wq = torch.zeros(N, pitch, dtype=torch.uint8, device="cuda")[:, :K]
    wq.copy_(w.to(torch.float8_e4m3fn).view(torch.uint8))
    ws = torch.randint(1, 5, (-(-N // 128), 1), generator=g).float()
    out = mse.fp8_block_matmul(x.to(torch.float8_e4m3fn).cuda(), torch.ones(T, 1, device="cuda"), wq, ws.cuda(),
                               out_dtype=torch.float32)
    want = (x @ w.t()) * ws.repeat_interleave(128, 0)[:N, 0]
    assert torch.equal(out.cpu(), want)


def test_generic_experts_of_a_long_row():
    E, H, I, T = 1, 1048560 + 130, 16, 2
    qgu, sgu, qd, sd = make_experts(E, H, I, 6)
    x = torch.randn(T, H, generator=gen(7)).to(torch.bfloat16).cuda()
    ids, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    y = mse.moe_experts_forward(x, ids, w, qgu, sgu, qd, sd)
    with kernel_path(mse.PATH_GENERIC):
        z = mse.moe_experts_forward(x, ids, w, qgu, sgu, qd, sd)
    # the same 8-bit operands and one h of 16 values a token: a value of h that falls on the other side of two e4m3
    # numbers moves by 1/8 at most, and the results round to bf16
    assert float((y.double() - z.double()).norm() / y.double().norm()) < 0.05
    assert torch.isfinite(z).all()


def test_quantise_of_many_row_blocks():
    rows, K = 65535 * 128 + 131, 3                 # 65,537 blocks of rows
    x = torch.randn(rows, K, generator=gen(8)).to(torch.bfloat16).cuda()
    q, s = mse.fp8_block_quantise(x, block_rows=128)
    assert s.shape == (65537, 1)
    for r0 in (0, 128 * 40000, 65535 * 128, 65536 * 128):
        part, ps = mse.fp8_block_quantise(x[r0:r0 + 128].clone(), block_rows=128)
        assert torch.equal(q[r0:r0 + 128].float(), part.float()) and torch.equal(s[r0 // 128:r0 // 128 + 1], ps)
