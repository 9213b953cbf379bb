"""Routing, 8-bit block products and the experts' layer against plain 64-bit forms."""
import math

import pytest

from tests import routed_ref as ref
from tests.helpers import kernel_path

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

mse = pytest.importorskip("moe_shared_expert_gb300")

EPS32 = 2.0 ** -24


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


@pytest.fixture(params=["generic", "auto"])
def path(request):
    with kernel_path(mse.PATH_GENERIC if request.param == "generic" else mse.PATH_AUTO):
        yield request.param


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------------ routing

ROUTES = [
    # T, E, k, scoring, bias, n_group, topk_group, group_top, renormalise
    (1, 256, 8, "sigmoid", True, 8, 4, 2, True),
    (5, 8, 2, "softmax", False, 1, 1, 1, True),
    (33, 160, 6, "softmax", True, 8, 3, 2, False),
    (33, 160, 6, "softmax", False, 8, 3, 1, False),
    (9, 384, 8, "sigmoid", True, 1, 1, 2, True),
    (4, 1, 1, "sigmoid", False, 1, 1, 1, True),
    (3, 31, 31, "softmax", False, 1, 1, 1, True),
    (3, 1024, 32, "sigmoid", True, 32, 16, 2, True),
    (6, 72, 5, "sigmoid", True, 18, 7, 2, False),
    (6, 33, 7, "softmax", True, 3, 2, 2, True),
    (1025, 64, 4, "sigmoid", False, 1, 1, 1, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c)))
def test_route(case, dtype):
    T, E, k, scoring, with_bias, G, keep, top, renorm = case
    g = gen(T * 1000 + E)
    logits = (torch.randn(T, E, generator=g) * 1.5).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    bias = torch.randn(E, generator=g) * 0.05 if with_bias else None
    ids, w = mse.moe_route(logits.cuda(), k, scoring=scoring, bias=None if bias is None else bias.cuda(), n_group=G,
                           topk_group=keep, group_top=top, renormalise=renorm, scale=2.5)
    rid, rw, gap = ref.route(logits, k, scoring, bias, G, keep, top, renorm, 2.5)
    # choices are held in 32 bits: rows that are decided by less than their rounding (a score and a sum,
    # of at most about 4, in ten roundings) may go either way, unless the scores are equal bit by bit
    sure = gap > 40 * EPS32
    tied = gap == 0
    assert int(sure.sum() + tied.sum()) >= 0.8 * T
    if with_bias:
        tied &= False
    rows = sure | tied
    assert torch.equal(ids.cpu()[rows], rid[rows])
    # score: exp (2 ulp), sum, quotient; then the sum of k and a quotient: 16 roundings
    assert torch.all((w.cpu().double() - rw)[rows].abs() <= 16 * 2 * EPS32 * rw[rows] + 1e-37)


def test_route_ties_go_to_the_lower_index():
    ids, w = mse.moe_route(torch.zeros(3, 96, device="cuda"), 5, scoring="softmax")
    assert ids.cpu().tolist() == [[0, 1, 2, 3, 4]] * 3
    assert torch.allclose(w.cpu(), torch.full((3, 5), 0.2), rtol=1e-6)
    ids, _ = mse.moe_route(torch.zeros(2, 96, device="cuda"), 5, n_group=4, topk_group=2)
    assert ids.cpu().tolist() == [[0, 1, 2, 3, 4]] * 2
    logits = torch.zeros(1, 64)
    logits[0, 40] = logits[0, 7] = 1.0
    assert mse.moe_route(logits.cuda(), 3)[0].cpu().tolist() == [[7, 40, 0]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_closed_experts(scoring, dtype):
    E = 40
    low = torch.finfo(dtype).min
    logits = torch.randn(6, E, generator=gen(3)).to(dtype)
    logits[0] = -math.inf                                  # nothing open
    logits[1] = low                                        # nothing open
    logits[2, 1:] = -math.inf                              # one open
    logits[3, 10:] = float("nan")                          # NaN closes
    logits[4, ::2] = low
    bias = torch.full((E,), 3.0)                           # a bias opens nothing
    ids, w = mse.moe_route(logits.cuda(), 4, scoring=scoring, bias=bias.cuda())
    rid, rw, _ = ref.route(logits, 4, scoring, bias)
    ids, w = ids.cpu(), w.cpu()
    assert ids[0].tolist() == [-1] * 4 and ids[1].tolist() == [-1] * 4 and ids[2].tolist() == [0, -1, -1, -1]
    assert torch.all(ids[3] < 10) and torch.all(ids[4] % 2 == 1)
    assert torch.all(w[:2] == 0) and w[2].tolist() == [1.0, 0, 0, 0]
    assert torch.allclose(w.double(), rw, rtol=1e-4, atol=1e-30)
    # groups: one open expert in group 1, none in the others
    logits = torch.full((1, E), -math.inf, dtype=dtype)
    logits[0, 13] = -5.0
    ids, w = mse.moe_route(logits.cuda(), 3, scoring=scoring, n_group=4, topk_group=1)
    assert ids.cpu().tolist() == [[13, -1, -1]] and w.cpu()[0, 1:].tolist() == [0, 0]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_of_crowded_scores(scoring):
    # more experts near the top_k-th best than are ranked at once: saturated, tiny and equal scores
    E = 300
    g = gen(41)
    rows = [torch.full((E,), 30.0), torch.full((E,), -90.0), torch.zeros(E), torch.randn(E, generator=g) * 1e-4,
            torch.cat([torch.full((150,), 20.0), torch.full((150,), -20.0)]), torch.randn(E, generator=g) * 30 - 200,
            torch.cat([torch.tensor([50.0]), torch.zeros(E - 1)])]
    logits = torch.stack(rows)
    logits[3, 100:] = logits[3, 0]
    for bias in (None, torch.linspace(0, 1e-3, E)):
        ids, w = mse.moe_route(logits.cuda(), 8, scoring=scoring, bias=None if bias is None else bias.cuda())
        l = logits                                         # in 32 bits, as the choices are defined
        s = 1.0 / (1.0 + torch.exp(-l)) if scoring == "sigmoid" else torch.softmax(l.double(), 1).float()
        c = s if bias is None else s + bias
        ids, w = ids.cpu().long(), w.cpu()
        for t in range(len(rows)):
            best = c[t].sort(descending=True, stable=True)
            # nothing left out is better than what was taken by more than 32-bit rounding
            taken = c[t][ids[t]]
            assert len(set(ids[t].tolist())) == 8 and torch.all(ids[t] >= 0)
            assert torch.all((taken - best.values[:8]).abs() <= 8 * EPS32 * (best.values[:8].abs() + 1e-30) + 1e-42)
            want = s[t][ids[t]].double()
            if want.sum() > 0:
                assert torch.allclose(w[t].double(), want / want.sum(), rtol=1e-5, atol=1e-6)
    same, _ = mse.moe_route(logits[:3].cuda(), 8, scoring=scoring)
    assert same.cpu().tolist() == [list(range(8))] * 3


def test_route_of_a_pitched_view_and_extreme_logits():
    big = torch.randn(7, 100, generator=gen(4))
    big[1] = 80.0
    big[2] = -80.0
    big[3, 20] = 3e38
    ids, w = mse.moe_route(big.cuda()[:, 10:74], 6, scoring="softmax")
    rid, rw, _ = ref.route(big[:, 10:74], 6, "softmax")
    assert torch.equal(ids.cpu(), rid) and torch.allclose(w.cpu().double(), rw, rtol=2e-6, atol=1e-37)


# ------------------------------------------------------------------------------------ rounding to 8 bits

@pytest.mark.parametrize("rows,K", [(1, 1), (3, 128), (2, 129), (17, 1000), (130, 300), (5, 7168)])
def test_quantise_rows_has_one_value(rows, K):
    x = (torch.randn(rows, K, generator=gen(K)) * torch.logspace(-3, 3, rows)[:, None]).to(torch.bfloat16)
    x[0, :min(K, 128)] = 0.0
    q, s = mse.fp8_block_quantise(x.cuda())
    rq, rs = ref.rounded(x.double())
    assert q.shape == (rows, K) and q.stride(0) % 16 == 0 and s.shape == (rows, ref.blocks(K))
    assert torch.equal(q.cpu().double(), rq)          # exact: no quotient of bf16 numbers is near a tie
    assert torch.all((s.cpu().double() - rs).abs() <= EPS32 * rs)


@pytest.mark.parametrize("rows,K", [(1, 1), (128, 128), (129, 257), (300, 500)])
def test_quantise_tiles(rows, K):
    x = torch.randn(rows, K, generator=gen(K)).to(torch.bfloat16)
    q, s = mse.fp8_block_quantise(x.cuda(), block_rows=128)
    assert s.shape == (ref.blocks(rows), ref.blocks(K))
    for r in range(s.shape[0]):
        for k in range(s.shape[1]):
            v = x[r * 128:(r + 1) * 128, k * 128:(k + 1) * 128].double()
            a = v.abs().max().clamp_min(ref.FLOOR)
            got = q[r * 128:(r + 1) * 128, k * 128:(k + 1) * 128].cpu().double()
            assert torch.equal(got, ref.e4m3(448.0 * v / a))
            assert abs(float(s[r, k]) - float(a / 448)) <= EPS32 * float(a / 448)
    stacked = torch.stack([x, -x]).cuda()
    q3, s3 = mse.fp8_block_quantise(stacked, block_rows=128)
    assert torch.equal(q3[0].cpu().float(), q.cpu().float()) and torch.equal(s3[1], s)


def test_quantise_of_extreme_blocks():
    x = torch.zeros(5, 256, dtype=torch.bfloat16)
    x[0, 3], x[1, 4], x[2, 200] = math.inf, math.nan, 3.3895313892515355e38
    x[3, 0] = 1e-38
    q, s = mse.fp8_block_quantise(x.cuda())
    v = (q.cpu().float() * s.cpu().repeat_interleave(128, 1))
    assert torch.isnan(v[0, :128]).all() and torch.isnan(v[1, :128]).all()
    assert not v[0, 128:].any() and not v[4].any() and not v[3].any()
    assert float(q[2, 200]) == 448.0 and torch.isfinite(v[2]).all()


@pytest.mark.parametrize("rows,K,pitch,offset", [(70, 200, 208, 8), (70, 200, 204, 4), (70, 136, 138, 2), (70, 300, 301, 0),
                                                 (33, 128, 136, 3), (6000, 900, 900, 0)])
def test_quantise_of_views(rows, K, pitch, offset):
    # rows at multiples of 16, 8, 4 and 2 bytes, and more rows than are on their way at once
    flat = torch.randn(rows * pitch + offset, generator=gen(K)).to(torch.bfloat16).cuda()
    x = torch.as_strided(flat, (rows, K), (pitch, 1), offset)
    rq, rs = ref.rounded(x.cpu().double())
    q, s = mse.fp8_block_quantise(x)
    assert torch.equal(q.cpu().double(), rq) and torch.all((s.cpu().double() - rs).abs() <= EPS32 * rs)
    q, s = mse.fp8_block_quantise(x, block_rows=128)
    q2, s2 = mse.fp8_block_quantise(x.clone(), block_rows=128)
    assert torch.equal(q.cpu().float(), q2.cpu().float()) and torch.equal(s, s2)


# ------------------------------------------------------------------------------------ products

def assert_product(got, x_values, w_values, roundings=2.0 ** -8):
    """got against x w^T: K products summed in 32 bits in any order, each sum perhaps cut off rather than
    rounded (2^-23 of the largest partial sum), the scales (3 roundings), and the rounding of the result."""
    exact = x_values @ w_values.t()
    total = x_values.abs() @ w_values.abs().t()
    bound = roundings * exact.abs() + (x_values.shape[1] + 3) * 2.0 ** -23 * total + 1e-30
    off = (got.cpu().double() - exact).abs() / bound
    assert torch.all(off <= 1), float(off.max())


MATMULS = [
    (1, 1, 1), (1, 2112, 7168), (2, 128, 128), (3, 130, 257), (16, 256, 384), (17, 300, 1000), (64, 1000, 640),
    (65, 384, 2048), (100, 131, 4100), (129, 128, 520), (200, 700, 130), (257, 513, 1024), (333, 2111, 610),
    (600, 256, 128), (1030, 260, 784), (2, 11000, 4500), (33, 9000, 300), (520, 5001, 300), (300, 4000, 5000),
]


@pytest.mark.parametrize("T,N,K", MATMULS)
def test_matmul_and_linear(T, N, K, path):
    g = gen(T + N + K)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16)
    w = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(torch.bfloat16)
    wq, ws = mse.fp8_block_quantise(w.cuda(), block_rows=128)
    wv = ref.weight(wq.cpu(), ws.cpu())
    xq, xs = mse.fp8_block_quantise(x.cuda())
    xv = ref.spread_rows(xq.cpu().double(), xs.cpu().double())
    f32 = mse.fp8_block_matmul(xq, xs, wq, ws, out_dtype=torch.float32)
    assert_product(f32, xv, wv, 2.0 ** -22)
    bf16 = mse.fp8_block_matmul(xq, xs, wq, ws)
    assert bf16.dtype == torch.bfloat16
    assert_product(bf16, xv, wv)
    y = mse.fp8_block_linear(x.cuda(), wq, ws)
    assert torch.equal(y, bf16)
    # the same call twice, and into a kept workspace: the same bits
    ws_buf = mse.new_fp8_linear_workspace(T + 5, N, K)
    ws_buf.fill_(0xFF)
    assert torch.equal(mse.fp8_block_linear(x.cuda(), wq, ws, workspace=ws_buf), y)


def test_forced_tensor_cores_refuse_what_they_cannot_serve():
    T, N, K = 5, 130, 200
    x = torch.randn(T, K, generator=gen(31)).to(torch.bfloat16).cuda()
    wq, ws = mse.fp8_block_quantise(torch.randn(N, K, generator=gen(32)).to(torch.bfloat16).cuda(), block_rows=128)
    odd = torch.zeros(N, K + 1, dtype=torch.uint8, device="cuda")[:, :K]
    odd.copy_(wq.view(torch.uint8))
    with kernel_path(mse.PATH_TENSORCORE):
        y = mse.fp8_block_linear(x, wq, ws)
        with pytest.raises(mse.MSEError, match="MSE_ERR_UNSUPPORTED_SHAPE"):
            mse.fp8_block_linear(x, odd, ws)
    assert_product(y, ref.spread_rows(*ref.rounded(x.cpu().double())), ref.weight(wq.cpu(), ws.cpu()))


def test_bindings_refuse_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    wq, ws = mse.fp8_block_quantise(torch.ones(8, 64, dtype=torch.bfloat16, device="cuda"), block_rows=128)
    for bad in (dict(x=x.t()), dict(x=x.float()), dict(x=x[:, :60]), dict(wq=wq.t()), dict(ws=ws.double()),
                dict(y=torch.empty(4, 9, device="cuda", dtype=torch.bfloat16)), dict(x=x[:0])):
        a = dict(x=x, wq=wq, ws=ws, y=None)
        a.update(bad)
        with pytest.raises((ValueError, mse.MSEError)):
            mse.fp8_block_linear(a["x"], a["wq"], a["ws"], y=a["y"])
    with pytest.raises(ValueError):
        mse.moe_route(x, 2, scoring="relu")
    with pytest.raises(mse.MSEError):
        mse.moe_route(x, 65)
    with pytest.raises(ValueError):
        mse.moe_route(x, 2, bias=torch.zeros(63, device="cuda"))


def test_matmul_takes_any_pitch_and_alignment():
    T, N, K = 20, 150, 300
    g = gen(11)
    x = torch.randn(T, K + 3, generator=g).to(torch.bfloat16).cuda()[:, 3:]
    w = torch.randn(N, K, generator=g).to(torch.bfloat16)
    wq, ws = mse.fp8_block_quantise(w.cuda(), block_rows=128)
    y = mse.fp8_block_linear(x, wq, ws)
    odd = torch.zeros(N, K + 7, dtype=torch.uint8, device="cuda")[:, 5:5 + K]
    odd.copy_(wq.view(torch.uint8))
    y2 = mse.fp8_block_linear(x, odd, ws)
    wide = torch.full((N, K + 20), 0x7F, dtype=torch.uint8, device="cuda")[:, :K]   # NaN between the rows
    wide.copy_(wq.view(torch.uint8))
    y3 = mse.fp8_block_linear(x, wide, ws)
    xv = ref.spread_rows(*ref.rounded(x.cpu().double()))
    for got in (y, y2, y3):
        assert_product(got, xv, ref.weight(wq.cpu(), ws.cpu()))


def test_matmul_keeps_rows_and_columns_apart(path):
    # a NaN row of x or of W spoils its own row or column and nothing else
    T, N, K = 70, 260, 384
    g = gen(12)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16)
    w = torch.randn(N, K, generator=g).to(torch.bfloat16)
    wq, ws = mse.fp8_block_quantise(w.cuda(), block_rows=128)
    clean = mse.fp8_block_linear(x.cuda(), wq, ws)
    x[33, 200] = math.nan
    wq = wq.clone()
    wq.view(torch.uint8)[131, 7] = 0x7F
    y = mse.fp8_block_linear(x.cuda(), wq, ws)
    assert torch.isnan(y[33]).all() and torch.isnan(y[:, 131]).all()
    keep = torch.ones(T, N, dtype=torch.bool, device="cuda")
    keep[33] = False
    keep[:, 131] = False
    assert torch.equal(y[keep], clean[keep])


# ------------------------------------------------------------------------------------ the experts' layer

def make_experts(E, H, I, seed):
    g = gen(seed)
    wgu = (torch.randn(E, 2 * I, H, generator=g) / math.sqrt(H)).to(torch.bfloat16).cuda()
    wd = (torch.randn(E, H, I, generator=g) / math.sqrt(I)).to(torch.bfloat16).cuda()
    qgu, sgu = mse.fp8_block_quantise(wgu.view(2 * E, I, H), block_rows=128)
    qgu = torch.as_strided(qgu, (E, 2 * I, H), (2 * I * qgu.stride(1), qgu.stride(1), 1))
    qd, sd = mse.fp8_block_quantise(wd, block_rows=128)
    return qgu, sgu.reshape(E, 2 * ref.blocks(I), ref.blocks(H)), qd, sd


def assert_experts(y, want):
    # the rounding of the result (2^-8), and of h: about one value in a thousand lies so near the middle of two e4m3
    # numbers that 32-bit sums move it, by 1/16 at most: 0.2% of a row's size in the mean, six times that at worst
    want = want.to(torch.float64)
    rms = want.square().mean().sqrt()
    off = (y.cpu().double() - want).abs()
    assert torch.all(off <= 2.0 ** -8 * want.abs() + 0.012 * rms), float((off / (2.0 ** -8 * want.abs() + 0.012 * rms)).max())
    assert float(off.norm() / want.norm()) <= 2.0 ** -8


EXPERTS = [
    # T, E, total, k, H, I, shared
    (1, 4, 4, 2, 256, 128, True),
    (1, 8, 8, 8, 384, 256, False),
    (3, 3, 9, 2, 200, 100, True),
    (16, 4, 8, 3, 512, 384, True),
    (40, 6, 6, 2, 1000, 700, False),
    (70, 2, 2, 1, 256, 200, True),
    (150, 5, 10, 4, 384, 128, True),
    (530, 3, 4, 2, 256, 300, False),
    (4, 5, 5, 5, 256, 128, True),          # up to 32 pairs: tiles from the ids
    (1, 40, 64, 32, 128, 128, False),
    (30, 300, 400, 9, 128, 60, True),      # more experts than pairs of any
    (1100, 4, 5, 4, 128, 130, True),       # above 4096 pairs: counted apart
    (700, 9, 9, 7, 200, 128, False),
]


@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: "-".join(map(str, c)))
def test_experts(case, path):
    T, E, total, k, H, I, with_shared = case
    g = gen(T * 7 + I)
    first = (total - E) // 2
    weights = make_experts(E, H, I, 100 + T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    ids = torch.randn(T, total, generator=g).topk(k, 1).indices.to(torch.int32)
    ids[T // 2, 0] = -1
    w = torch.rand(T, k, generator=g)
    shared = torch.randn(T, H, generator=g).to(torch.bfloat16) if with_shared else None
    want = ref.experts(x, ids, w, *[t.cpu().float() if i % 2 == 0 else t.cpu() for i, t in enumerate(weights)],
                       first=first, shared=shared)
    args = (x.cuda(), ids.cuda(), w.cuda(), *weights)
    y = mse.moe_experts_forward(*args, first_expert=first, shared=None if shared is None else shared.cuda())
    assert_experts(y, want)
    # a kept workspace that a larger call has left full of its own rows; y over x and over shared: the same bits
    buf = mse.new_moe_workspace(T + 9, k, E, H, I)
    buf.fill_(0xFF)
    out = x.cuda().clone() if shared is None else shared.cuda().clone()
    if shared is None:
        mse.moe_experts_forward(out, *args[1:], first_expert=first, y=out, workspace=buf)
    else:
        mse.moe_experts_forward(*args, first_expert=first, shared=out, y=out, workspace=buf)
    assert torch.equal(out, y)


def test_experts_of_many_chunks_and_unaligned_rows(path):
    # 277 chunks of tokens, 40 experts; x, shared and y that begin in the middle of a word
    T, E, k, H, I = 17700, 40, 4, 36, 16
    weights = make_experts(E, H, I, 31)
    g = gen(32)
    flat = torch.randn(2, T * H + 1, generator=g).to(torch.bfloat16).cuda()
    x, shared = flat[0, 1:].view(T, H), flat[1, 1:].view(T, H)
    ids = torch.randn(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    w = torch.rand(T, k, generator=g)
    y = torch.empty(T * H + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H)
    mse.moe_experts_forward(x, ids.cuda(), w.cuda(), *weights, shared=shared, y=y)
    some = torch.cat([torch.arange(200), torch.arange(9000, 9200), torch.arange(T - 200, T)])
    want = ref.experts(x.cpu()[some], ids[some], w[some],
                       *[t.cpu().float() if i % 2 == 0 else t.cpu() for i, t in enumerate(weights)], shared=shared.cpu()[some])
    assert_experts(y[some.cuda()], want)
    aligned = mse.moe_experts_forward(x.clone(), ids.cuda(), w.cuda(), *weights, shared=shared.clone())
    assert torch.equal(aligned, y)


def test_experts_of_a_few_tokens_with_repeated_ids(path):
    # up to 32 pairs: repeated experts of one token, experts with more pairs than a tile has rows, holes
    E, H, I = 7, 256, 128
    weights = make_experts(E, H, I, 23)
    cpu = [t.cpu().float() if i % 2 == 0 else t.cpu() for i, t in enumerate(weights)]
    for T, k, fill in ((1, 32, "one"), (2, 16, "two"), (4, 8, "any"), (1, 1, "any"), (3, 7, "holes")):
        g = gen(T + k)
        x = torch.randn(T, H, generator=g).to(torch.bfloat16)
        ids = {"one": torch.full((T, k), 5), "two": torch.arange(T * k).view(T, k) % 2 * 3 + 1,
               "any": torch.randint(0, E, (T, k), generator=g),
               "holes": torch.randint(-3, E + 3, (T, k), generator=g)}[fill].to(torch.int32)
        w = torch.rand(T, k, generator=g)
        y = mse.moe_experts_forward(x.cuda(), ids.cuda(), w.cuda(), *weights)
        assert_experts(y, ref.experts(x, ids, w, *cpu))


def test_experts_without_a_pair(path):
    E, H, I, T = 3, 256, 128, 5
    weights = make_experts(E, H, I, 5)
    x = torch.randn(T, H, generator=gen(6)).to(torch.bfloat16).cuda()
    shared = torch.randn(T, H, generator=gen(7)).to(torch.bfloat16).cuda()
    w = torch.ones(T, 2, device="cuda")
    for ids in (torch.full((T, 2), -1), torch.full((T, 2), 7), torch.full((T, 2), -2 ** 31), torch.full((T, 2), 2 ** 31 - 1)):
        ids = ids.to(torch.int32).cuda()
        assert torch.equal(mse.moe_experts_forward(x, ids, w, *weights, shared=shared), shared)
        assert not mse.moe_experts_forward(x, ids, w, *weights).any()


def test_experts_all_tokens_to_one_expert_and_twice(path):
    E, H, I, T = 5, 256, 256, 90
    weights = make_experts(E, H, I, 8)
    x = torch.randn(T, H, generator=gen(9)).to(torch.bfloat16)
    ids = torch.full((T, 2), 3, dtype=torch.int32)
    w = torch.rand(T, 2, generator=gen(10))
    y = mse.moe_experts_forward(x.cuda(), ids.cuda(), w.cuda(), *weights)
    assert_experts(y, ref.experts(x, ids, w, *[t.cpu().float() if i % 2 == 0 else t.cpu() for i, t in enumerate(weights)]))


def test_experts_keep_tokens_apart(path):
    # a token's result does not depend on the others in its batch, nor on a NaN among them
    E, H, I, T = 4, 384, 256, 37
    weights = make_experts(E, H, I, 13)
    x = torch.randn(T, H, generator=gen(14)).to(torch.bfloat16).cuda()
    ids = torch.randint(0, E, (T, 2), generator=gen(15)).to(torch.int32).cuda()
    w = torch.rand(T, 2, generator=gen(16)).cuda()
    y = mse.moe_experts_forward(x, ids, w, *weights)
    x2 = x.clone()
    x2[20, 5] = math.nan
    y2 = mse.moe_experts_forward(x2, ids, w, *weights)
    assert torch.isnan(y2[20]).all()
    rest = [t for t in range(T) if t != 20]
    assert torch.equal(y2[rest], y[rest])


def test_calls_on_another_stream_and_in_a_graph():
    E, H, I, T = 4, 256, 256, 24
    weights = make_experts(E, H, I, 17)
    x = torch.randn(T, H, generator=gen(18)).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=gen(19)).cuda()

    def layer(stream=None):
        ids, w = mse.moe_route(logits, 2, stream=stream)
        return mse.moe_experts_forward(x, ids, w, *weights, stream=stream)

    y = layer()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    z = layer(other)
    other.synchronize()
    assert torch.equal(z, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)


def test_experts_beside_the_shared_expert():
    # the layer as a model runs it: router, shared expert, routed experts on top of it
    E, H, I, T = 6, 512, 256, 48
    weights = make_experts(E, H, I, 21)
    g = gen(22)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    wgu = (torch.randn(2 * I, H, generator=g) / math.sqrt(H)).to(torch.bfloat16).cuda()
    wd = (torch.randn(H, I, generator=g) / math.sqrt(I)).to(torch.bfloat16).cuda()
    router = torch.randn(E, H, generator=g).to(torch.bfloat16).cuda()
    old = mse.set_tuning(mse.TUNE_X_EARLY, 1)
    try:
        ids, w = mse.moe_route(x @ router.t(), 2)
        y = mse.mlp_swiglu_forward(x, wgu, wd)
        y = mse.moe_experts_forward(x, ids, w, *weights, shared=y)
        z = mse.mlp_swiglu_forward(y, wgu, wd)
    finally:
        mse.set_tuning(mse.TUNE_X_EARLY, old)
    shared = mse.mlp_swiglu_forward(x, wgu, wd)
    cpu = [t.cpu().float() if i % 2 == 0 else t.cpu() for i, t in enumerate(weights)]
    assert_experts(y, ref.experts(x.cpu(), ids.cpu(), w.cpu(), *cpu, shared=shared.cpu()))
    assert torch.equal(z, mse.mlp_swiglu_forward(y, wgu, wd))


def test_example_layer():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "moe_layer.py"), "--tokens", "24", "--experts", "6",
                        "--top-k", "2", "--hidden", "512", "--intermediate", "256", "--steps", "3", "--check"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "us a layer" in r.stdout
