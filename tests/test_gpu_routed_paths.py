"""Every kernel and split that a rule of the routed-expert operators chooses: shapes with the launch plan they are here
for.  Where a rule is tuned anew, other shapes take these places."""
import math

import pytest

from tests.test_gpu_routed import EPS32, assert_experts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

mse = pytest.importorskip("moe_shared_expert_gb300")

BLOCK = 128


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


def normal(seed, *shape, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def rows_of(q, s):
    """q [.., K] e4m3 times its scales [.., K / 128], in 64 bits."""
    return q.double() * s.double().repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def weight_of(q, s):
    N, K = q.shape
    return q.double() * s.double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


# ------------------------------------------------------------------------------------ products

PRODUCTS = [
    # T, N, K: tile rows, parts
    # the CTA-pair kernel, a tile to a pair or several
    (2048, 4097, 512, 256, 1),      # rows that start anywhere
    (2048, 4096, 512, 256, 1),      # whole rows by TMA
    (3000, 5000, 640, 256, 1),      # the last rows of T by the lanes
    (4000, 2561, 300, 256, 1),
    (8192, 1024, 130, 256, 1),
    # two pairs to a tile (more tiles than clusters of eight fit any GPU: how many do differs a little)
    (300, 4000, 5000, 256, 2), (1024, 1400, 7168, 256, 2), (1024, 1401, 7168, 256, 2), (1000, 1408, 7168, 256, 2),
    # four
    (512, 1536, 8192, 256, 4), (512, 1500, 8192, 256, 4), (700, 1000, 9000, 256, 4), (700, 1001, 9000, 256, 4),
    # the swap-AB kernel: tiles of 64, 32 and 16 tokens, split or not
    (640, 1001, 3200, 64, 3), (64, 512, 8192, 64, 8), (64, 7168, 768, 64, 1), (70, 700, 9000, 64, 5),
    (33, 12288, 5120, 64, 3), (200, 12288, 300, 64, 1), (17, 300, 1000, 32, 4), (32, 1024, 4200, 32, 8), (20, 24000, 4300, 32, 1),
    (16, 1024, 4096, 16, 8), (13, 24000, 4300, 16, 1), (8, 1000, 4300, 16, 8), (8, 30000, 500, 16, 1),
]


@pytest.mark.parametrize("T,N,K,tile_rows,parts", PRODUCTS)
def test_product(T, N, K, tile_rows, parts):
    plan = mse.fp8_launch_plan(T, N, K)
    assert (plan["tile_rows"], plan["parts"]) == (tile_rows, parts), plan
    x, w = normal(T + K, T, K), normal(N + K, N, K, sigma=1 / math.sqrt(K))
    wq, ws = mse.fp8_block_quantise(w, block_rows=128)
    xq, xs = mse.fp8_block_quantise(x)
    xv, wv = rows_of(xq, xs), weight_of(wq, ws)
    exact, total = xv @ wv.t(), xv.abs() @ wv.abs().t()
    # K products in 32 bits in any order, each sum perhaps cut off (2^-23 of it), three roundings of the factors, and
    # the result's own rounding
    sums = (K + 3) * 2.0 ** -23 * total + 1e-30
    f32 = mse.fp8_block_matmul(xq, xs, wq, ws, out_dtype=torch.float32)
    assert torch.all((f32.double() - exact).abs() <= 2.0 ** -22 * exact.abs() + sums)
    bf16 = mse.fp8_block_matmul(xq, xs, wq, ws)
    assert torch.all((bf16.double() - exact).abs() <= 2.0 ** -8 * exact.abs() + sums)
    assert torch.equal(f32.to(torch.bfloat16), bf16)               # the same sums, rounded once
    assert torch.equal(mse.fp8_block_linear(x, wq, ws), bf16)
    # around the output nothing is written
    around = torch.full((T * N + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    mse.fp8_block_matmul(xq, xs, wq, ws, out=around[32:32 + T * N].view(T, N))
    assert torch.equal(around[32:32 + T * N].view(T, N), bf16)
    assert torch.all(around[:32] == -7.0) and torch.all(around[32 + T * N:] == -7.0)


def test_product_of_several_tiles_to_a_pair():
    for T, N, K in ((2048, 4097, 512), (3000, 5000, 640), (4000, 2561, 300)):
        assert -(-T // 256) * -(-N // 256) > mse.fp8_launch_plan(T, N, K)["ctas"] // 2


@pytest.mark.parametrize("T,N,K,one", [(1, 2112, 7168, 1), (8, 1000, 4300, 1), (9, 1000, 4300, 0), (8, 7168, 6144, 0)])
def test_linear_in_one_launch_or_two(T, N, K, one):
    assert mse.fp8_launch_plan(T, N, K)["one_launch"] == one
    x = normal(T, T, K)
    wq, ws = mse.fp8_block_quantise(normal(N, N, K), block_rows=128)
    assert torch.equal(mse.fp8_block_linear(x, wq, ws), mse.fp8_block_matmul(*mse.fp8_block_quantise(x), wq, ws))


# ------------------------------------------------------------------------------------ the experts' layer

EXPERTS = [
    # T, k, E, H, I: tile rows, parts of gate_up and of down, tiles from the ids
    (1, 4, 4, 4096, 1024, 16, 5, 1, 1),       # one token, gate_up split
    (2, 4, 8, 1280, 640, 16, 2, 1, 1),
    (5, 2, 6, 5000, 300, 16, 5, 1, 1),
    (12, 3, 8, 4224, 256, 16, 5, 1, 0),
    (100, 2, 8, 4096, 256, 32, 5, 1, 0),      # tiles of 32 tokens, split
    (100, 2, 4, 4096, 1100, 32, 3, 1, 0),
    (64, 2, 4, 512, 2300, 32, 1, 5, 0),       # down split
    (160, 2, 40, 4224, 512, 16, 1, 1, 0),     # more k-blocks than scales are kept at a time, unsplit
    (160, 2, 40, 512, 4224, 16, 1, 1, 0),
    (400, 4, 40, 4224, 512, 32, 1, 1, 0),
    (400, 4, 40, 512, 4224, 32, 1, 1, 0),
    (400, 2, 6, 333, 200, 256, 1, 1, 0),      # CTA pairs; rows of y that end inside a word
    (900, 3, 5, 640, 256, 256, 1, 1, 0),
    (700, 4, 12, 1100, 1500, 256, 1, 1, 0),   # several tiles to a pair
]


def experts_in_64_bits(x, ids, w, qgu, sgu, qd, sd, shared):
    E, H, I = qd.shape
    nb, ib = -(-I // BLOCK), -(-I // BLOCK) * BLOCK
    xq, xs = mse.fp8_block_quantise(x)
    xr = rows_of(xq, xs)
    y = shared.double().clone()
    for e in range(E):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if not token.numel():
            continue
        g = xr[token] @ weight_of(qgu[e, :I], sgu[e, :nb]).t()
        u = xr[token] @ weight_of(qgu[e, I:], sgu[e, nb:]).t()
        h = torch.nn.functional.pad(g / (1 + torch.exp(-g)) * u, (0, ib - I)).unflatten(-1, (-1, BLOCK))
        a = h.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
        h = ((448 * h / a).float().to(torch.float8_e4m3fn).double() * (a / 448)).flatten(-2)[:, :I]
        y.index_add_(0, token, w[token, slot].double()[:, None] * (h @ weight_of(qd[e], sd[e]).t()))
    return y


@pytest.mark.parametrize("T,k,E,H,I,tile_rows,gate_up,down,from_ids", EXPERTS)
def test_experts(T, k, E, H, I, tile_rows, gate_up, down, from_ids):
    plan = mse.moe_launch_plan(T, k, E, H, I)
    assert (plan["tile_rows"], plan["gate_up_parts"], plan["down_parts"], plan["tiles_from_ids"]) == \
        (tile_rows, gate_up, down, from_ids), plan
    qgu, sgu = mse.fp8_block_quantise(normal(E + H, 2 * E, I, H, sigma=1 / math.sqrt(H)), block_rows=128)
    qgu = qgu.as_strided((E, 2 * I, H), (2 * I * qgu.stride(1), qgu.stride(1), 1))
    sgu = sgu.reshape(E, -1, sgu.shape[-1])
    qd, sd = mse.fp8_block_quantise(normal(E + I, E, H, I, sigma=1 / math.sqrt(I)), block_rows=128)
    x, shared = normal(T, T, H), normal(T + 1, T, H)
    g = torch.Generator(device="cuda").manual_seed(k)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    y = mse.moe_experts_forward(x, ids, w, qgu, sgu, qd, sd, shared=shared)
    assert_experts(y, experts_in_64_bits(x, ids, w, qgu, sgu, qd, sd, shared).cpu())
    buf = mse.new_moe_workspace(T, k, E, H, I)
    buf.fill_(0xFF)
    around = torch.full((T * H + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    mse.moe_experts_forward(x, ids, w, qgu, sgu, qd, sd, shared=shared, y=around[32:32 + T * H].view(T, H), workspace=buf)
    assert torch.equal(around[32:32 + T * H].view(T, H), y)
    assert torch.all(around[:32] == -7.0) and torch.all(around[32 + T * H:] == -7.0)


# ------------------------------------------------------------------------------------ many tokens' routes

@pytest.mark.parametrize("T,E,k,scoring,with_bias,G,keep,top", [
    (65536, 160, 6, "softmax", True, 8, 3, 2), (20001, 448, 8, "sigmoid", True, 8, 4, 2), (30000, 72, 4, "sigmoid", False, 18, 7, 1),
    (16384, 384, 8, "sigmoid", True, 1, 1, 2), (40001, 33, 5, "softmax", False, 1, 1, 2), (9000, 1000, 10, "softmax", True, 1, 1, 2),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_of_many_tokens(T, E, k, scoring, with_bias, G, keep, top, dtype):
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = (torch.randn(T, E, generator=g, device="cuda") * 1.5).to(dtype)
    bias = torch.randn(E, generator=g, device="cuda") * 0.05 if with_bias else None
    ids, w = mse.moe_route(logits, k, scoring=scoring, bias=bias, n_group=G, topk_group=keep, group_top=top)
    l = logits.double()
    score = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 1)
    choice = score if bias is None else score + bias.double()
    gap = torch.full((T,), math.inf, dtype=torch.float64, device="cuda")
    if G > 1:
        value = choice.view(T, G, -1).topk(top, 2).values.sum(2)
        order = value.sort(dim=1, descending=True, stable=True)
        gap = torch.minimum(gap, order.values[:, keep - 1] - order.values[:, keep])
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order.indices[:, :keep], True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    order = choice.sort(dim=1, descending=True, stable=True)
    gap = torch.minimum(gap, (order.values[:, :k] - order.values[:, 1:k + 1]).amin(1))
    # choices are held in 32 bits: rows decided by less than ten roundings of at most about 4 may go either way
    sure = gap > 40 * EPS32
    assert float(sure.double().mean()) > (0.9 if dtype == torch.float32 or with_bias else 0.2)
    assert torch.equal(ids[sure].long(), order.indices[sure][:, :k])
    want = score.gather(1, order.indices[:, :k])
    want = want / want.sum(1, keepdim=True)
    assert torch.all((w.double() - want)[sure].abs() <= 32 * EPS32 * want[sure] + 1e-37)
