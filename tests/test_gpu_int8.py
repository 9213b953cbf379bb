"""Products in 8-bit integers, plain and by expert, against plain 64-bit forms."""
import math

import pytest

from tests import sorted_ref as ref
from tests.helpers import kernel_path

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


@pytest.fixture(params=["generic", "auto"])
def path(request):
    with kernel_path(mse.PATH_GENERIC if request.param == "generic" else mse.PATH_AUTO):
        yield request.param


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows_with_pitch(t, pitch, fill=0, shift=0):
    """t's values on the GPU in rows of a pitch, begun `shift` values late, in a buffer of `fill` bytes."""
    *lead, rows, cols = t.shape
    n = math.prod(lead) * rows
    raw = torch.full(((n * pitch + shift) * t.element_size(),), fill, dtype=torch.uint8, device="cuda")
    out = raw.view(t.dtype)[shift:].as_strided((n, cols), (pitch, 1))
    out.copy_(t.reshape(n, cols))
    return out.as_strided(t.shape, (*([rows * pitch] if lead else []), pitch, 1))


# ------------------------------------------------------------------------------------ rounding

ROUNDS = [(1, 7168, 0), (3, 1, 0), (5, 2, 1), (17, 129, 0), (64, 1000, 8), (33, 1001, 2), (2, 8200, 0), (300, 256, 0),
          (1, 40000, 0), (1300, 64, 0), (2, 16388, 4)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,K,extra", ROUNDS)
def test_quantise(rows, K, extra, dtype):
    x = (torch.randn(rows, K, generator=gen(K)) * torch.exp(3 * torch.randn(rows, 1, generator=gen(1)))).to(dtype)
    x[rows // 2] = 0
    q, s = mse.int8_quantise(rows_with_pitch(x, K + extra, 0xEE))
    assert q.dtype is torch.int8 and q.stride(0) == -(-K // 16) * 16 and s.shape == (rows,)
    if dtype is torch.bfloat16:
        want, scale = ref.quantised(x)
    else:   # the quotient in 32 bits
        a = x.abs().amax(1, keepdim=True).clamp_min(ref.FLOOR)
        want, scale = torch.round(x * (127.0 / 512) / a * 512), a[:, 0] / 127
    assert torch.equal(q.cpu().double(), want.double()) and torch.equal(s.cpu(), scale)


@pytest.mark.parametrize("top", [127.0, 254.0, 508.0, 1.0, 2.0 ** 100, 2.0 ** -90])
def test_ties_go_to_even(top):
    # 127 v / top: halves of integers where top is 254 or 508 times a power of two, in every other place integers and more
    n = torch.arange(-254, 255).double()
    x = torch.cat([n * top / 254, torch.tensor([top], dtype=torch.float64)]).to(torch.bfloat16)[None]
    q, s = mse.int8_quantise(x.cuda())
    want, scale = ref.quantised(x)
    assert torch.equal(q.cpu().double(), want) and torch.equal(s.cpu(), scale)


def test_every_pair_of_fractions():
    # the rounding of bf16 v / a depends on their fractions and on the distance of their exponents alone
    a = (128 + torch.arange(128)).double()
    v = torch.cat([(128 + torch.arange(128)).double() * 2.0 ** -e for e in range(10)])
    v = torch.where(v[None] <= a[:, None], v[None], 0.0)
    x = torch.cat([a[:, None], v, -v], 1).to(torch.bfloat16)
    q, s = mse.int8_quantise(x.cuda())
    want, scale = ref.quantised(x)
    assert torch.equal(q.cpu().double(), want) and torch.equal(s.cpu(), scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_rows_at_the_ends_of_the_range(dtype):
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    x = torch.tensor([[big, -big, big / 3], [small, -small, 0], [2.0 ** -100, 2.0 ** -101, -2.0 ** -107], [0, 0, 0],
                      [1, math.inf, 0], [math.nan, 1, 2], [-math.inf, math.inf, 1], [3, 1, -2]]).to(dtype)
    q, s = mse.int8_quantise(x.cuda())
    want, scale = ref.quantised(x)
    assert torch.equal(q.cpu().double(), want)
    assert torch.equal(s.cpu().nan_to_num(nan=-1), scale.nan_to_num(nan=-1)) and bool((s[4:7].isnan()).all())
    w = torch.ones(5, 3, dtype=torch.int8, device="cuda")
    y = mse.int8_linear(x.cuda(), w, torch.ones(5, device="cuda"), y_dtype=torch.float32)
    assert bool(y[4:7].isnan().all()) and bool(y[7].isfinite().all()) and bool((y[3] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,K,extra", [(1, 2048, 0), (5, 1, 0), (33, 700, 4), (3, 1001, 1), (64, 512, 0), (2, 5000, 0)])
def test_quantise_of_swiglu(rows, K, extra, dtype):
    x = (2 * torch.randn(rows, 2 * K, generator=gen(K))).to(dtype)
    q, s = mse.int8_quantise(rows_with_pitch(x, 2 * K + extra, 0xEE), swiglu=True)
    h = ref.swiglu(x)
    a = h.abs().amax(1)
    # e^-g is off by 1.3 |g| 2^-24 of itself and a few 2^-23 more, |g| < 12 here: h within 2^-19, the scale and each quotient too
    rel = 2.0 ** -19
    assert bool(((s.cpu().double() - a / 127).abs() <= (a / 127) * (rel + 2.0 ** -23)).all())
    ratio = 127 * h / a[:, None]
    assert bool(((q.cpu().double() - ratio).abs() <= 0.5 + 127 * 2 * (rel + 2.0 ** -22)).all())


def test_rows_behind_the_last_are_left_alone():
    x = torch.randn(9, 40, generator=gen(1)).to(torch.bfloat16).cuda()
    for n in (0, 4, 9, 12, -3):
        offsets = torch.tensor([0, 1, n], dtype=torch.int32, device="cuda")
        q = torch.full((9, 48), 99, dtype=torch.int8, device="cuda")
        s = torch.full((9,), 5.0, device="cuda")
        mse.int8_quantise(x, offsets=offsets, q=q[:, :40], scales=s)
        want, scale = ref.quantised(x.cpu())
        n = min(max(n, 0), 9)
        assert torch.equal(q[:n, :40].cpu().double(), want[:n]) and torch.equal(s[:n].cpu(), scale[:n])
        assert bool((q[n:] == 99).all()) and bool((q[:, 40:] == 99).all()) and bool((s[n:] == 5).all())


def test_weights_of_experts_in_one_call():
    w = torch.randn(3, 20, 50, generator=gen(1)).to(torch.bfloat16)
    q, s = mse.int8_quantise(w.cuda())
    want, scale = ref.quantised(w)
    assert q.shape == w.shape and q.stride() == (20 * 64, 64, 1) and s.shape == (3, 20)
    assert torch.equal(q.cpu().double(), want) and torch.equal(s.cpu(), scale)


# ------------------------------------------------------------------------------------ products

def integers(*shape, seed, top=127):
    return torch.randint(-top - (top == 128), min(top, 127) + 1, shape, generator=gen(seed)).clamp_min(-128).to(torch.int8)


def scales(*shape, seed):
    return torch.exp(torch.randn(*shape, generator=gen(seed))) * 1e-3


def expected(xq, xs, wq, ws, dtype):
    return ref.product(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda()).to(dtype)


PRODUCTS = [(1, 2112, 7168), (1, 1, 1), (2, 3, 17), (3, 904, 966), (4, 128, 128), (5, 129, 130), (8, 1024, 1024), (9, 700, 1000),
            (16, 256, 512), (17, 33, 4097), (31, 127, 1025), (33, 2111, 1031), (64, 1536, 2048), (65, 300, 96), (100, 640, 640),
            (128, 513, 1024), (129, 257, 1152), (200, 2112, 1536), (257, 384, 384), (333, 2111, 610), (520, 1000, 700),
            (1025, 260, 2050), (2049, 512, 144)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_matmul(T, N, K, dtype, path):
    xq, wq, xs, ws = integers(T, K, seed=1), integers(N, K, seed=2), scales(T, seed=3), scales(N, seed=4)
    pitch = -(-K // 16) * 16
    got = mse.int8_matmul(rows_with_pitch(xq, pitch, 0x7F), xs.cuda(), rows_with_pitch(wq, pitch, 0x7F), ws.cuda(), out_dtype=dtype)
    assert torch.equal(got, expected(xq, xs, wq, ws, dtype))


@pytest.mark.parametrize("T,N,K", [(1, 64, 5000), (7, 130, 3000), (16, 128, 9000), (40, 200, 4100), (70, 64, 131071), (130, 128, 2100), (300, 256, 3200),
                                   (2, 5, 131071)])
@pytest.mark.parametrize("sign", [1, -1])
def test_largest_sums_are_exact(T, N, K, sign, path):
    # -128 x -128 throughout, but for a few: sums up to 2^14 K, beyond what 24 bits hold
    xq = torch.full((T, K), -128, dtype=torch.int8)
    wq = torch.full((N, K), -128 if sign > 0 else 127, dtype=torch.int8)
    xq[torch.rand(T, K, generator=gen(1)) < 0.01] = 3
    wq[torch.rand(N, K, generator=gen(2)) < 0.01] = -1
    xs, ws = torch.full((T,), 1.0), torch.full((N,), 1.0)
    pitch = -(-K // 16) * 16
    got = mse.int8_matmul(rows_with_pitch(xq, pitch), xs.cuda(), rows_with_pitch(wq, pitch), ws.cuda(), out_dtype=torch.float32)
    assert torch.equal(got, expected(xq, xs, wq, ws, torch.float32))


@pytest.mark.parametrize("T", [1, 5, 20, 70, 300])
@pytest.mark.parametrize("px,pw,sx,sw", [(0, 0, 0, 0), (1, 0, 0, 0), (0, 1, 0, 0), (7, 8, 3, 0), (0, 12, 0, 4), (0, 0, 0, 1), (48, 32, 16, 16)])
def test_pitches_and_alignments(T, px, pw, sx, sw, path):
    N, K = 200, 304
    xq, wq, xs, ws = integers(T, K, seed=1), integers(N, K, seed=2), scales(T, seed=3), scales(N, seed=4)
    got = mse.int8_matmul(rows_with_pitch(xq, K + px, 0x7F, sx), xs.cuda(), rows_with_pitch(wq, K + pw, 0x7F, sw), ws.cuda())
    assert torch.equal(got, expected(xq, xs, wq, ws, torch.bfloat16))


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("T,N,K", [(1, 2112, 7168), (1, 5, 3), (2, 300, 1001), (3, 904, 966), (8, 1024, 1024), (9, 129, 700), (16, 700, 520), (33, 200, 1000),
                                   (64, 1536, 2048), (130, 257, 999), (300, 640, 1536), (1030, 300, 777)])
def test_linear(T, N, K, x_dtype, path):
    x = torch.randn(T, K, generator=gen(1)).to(x_dtype)
    wq, ws = mse.int8_quantise(torch.randn(N, K, generator=gen(2)).to(torch.bfloat16).cuda())
    q, s = mse.int8_quantise(x.cuda())
    got = mse.int8_linear(rows_with_pitch(x, K + 3, 0xEE), wq, ws)
    assert torch.equal(got, expected(q, s, wq, ws, torch.bfloat16))
    assert torch.equal(mse.int8_linear(x.cuda(), wq, ws), got)


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_y_over_x(T, path):
    x = torch.randn(T, 512, generator=gen(1)).to(torch.bfloat16).cuda()
    wq, ws = mse.int8_quantise(torch.randn(512, 512, generator=gen(2)).to(torch.bfloat16).cuda())
    want = mse.int8_linear(x, wq, ws)
    assert mse.int8_linear(x, wq, ws, y=x) is x and torch.equal(x, want)


GROUPS = [
    # rows of each group, rows behind them, N, K
    ([1] * 8, 0, 4096, 7168),
    ([0, 0, 3, 0], 2, 40, 33),
    ([5], 0, 129, 1000),
    ([0], 4, 16, 16),
    ([90, 0, 1, 17, 300, 16, 0, 129, 0], 7, 700, 1000),
    ([2, 7, 1, 0, 12, 9, 3, 8], 300, 520, 2048),
    ([0] * 63 + [9], 0, 64, 512),
    ([3] * 100, 11, 72, 160),
    ([256, 256, 1, 255], 0, 384, 1056),
    ([1000, 30, 513], 20, 256, 640),
    ([40] * 40, 0, 300, 528),
    ([64, 70, 60, 66], 0, 1024, 512),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("case", GROUPS, ids=lambda c: f"{len(c[0])}groups-{sum(c[0])}+{c[1]}-{c[2]}-{c[3]}")
def test_grouped(case, dtype, path):
    counts, behind, N, K = case
    G, P = len(counts), sum(counts) + behind
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    xq, wq, xs, ws = integers(P, K, seed=1), integers(G, N, K, seed=2), scales(P, seed=3), scales(G, N, seed=4)
    pitch = -(-K // 16) * 16
    out = torch.full((P, N), 77.0, dtype=dtype, device="cuda")
    mse.int8_grouped_matmul(rows_with_pitch(xq, pitch, 0x7F), xs.cuda(), offsets.cuda(), rows_with_pitch(wq, pitch, 0x7F),
                            ws.cuda(), out=out)
    for g in range(G):
        a, b = int(offsets[g]), int(offsets[g + 1])
        if a < b:
            assert torch.equal(out[a:b], expected(xq[a:b], xs[a:b], wq[g], ws[g], dtype)), g
    assert bool((out[sum(counts):] == 77).all())


def test_grouped_rows_that_begin_late_or_end_beyond(path):
    N, K, P = 40, 64, 30
    xq, wq, xs, ws = integers(P, K, seed=1), integers(3, N, K, seed=2), scales(P, seed=3), scales(3, N, seed=4)
    offsets = torch.tensor([4, 10, 10, 1000], dtype=torch.int32)
    out = torch.full((P, N), 77.0, device="cuda")
    mse.int8_grouped_matmul(xq.cuda(), xs.cuda(), offsets.cuda(), wq.cuda(), ws.cuda(), out=out)
    assert torch.equal(out[4:10], expected(xq[4:10], xs[4:10], wq[0], ws[0], torch.float32)) and bool((out[:4] == 77).all())
    assert torch.equal(out[10:], expected(xq[10:], xs[10:], wq[2], ws[2], torch.float32))


@pytest.mark.parametrize("P,groups", [(14, 8), (400, 12), (2048, 32), (20000, 60)])
def test_offsets_that_do_not_ascend_lead_nowhere_else(P, groups, path):
    """More tiles than a rising row of offsets makes, and numbers far outside."""
    N, K = 520, 200
    xq, wq, xs, ws = integers(P, K, seed=1), integers(groups, N, K, seed=2), scales(P, seed=3), scales(groups, N, seed=4)
    offsets = torch.tensor([0, P] * groups, dtype=torch.int32)[:groups]
    offsets = torch.cat([offsets, torch.tensor([P], dtype=torch.int32)])
    offsets[groups // 2], offsets[groups // 2 + 1] = -2 ** 31, 2 ** 31 - 1
    around = torch.full((P + 600, N), 77.0, device="cuda")
    mse.int8_grouped_matmul(xq.cuda(), xs.cuda(), offsets.cuda(), wq.cuda(), ws.cuda(), out=around[300:-300])
    torch.cuda.synchronize()
    assert bool((around[:300] == 77).all()) and bool((around[-300:] == 77).all())
    # a rising row of offsets is answered as before
    offsets = (torch.arange(groups + 1) * P // groups).int()
    out = mse.int8_grouped_matmul(xq.cuda(), xs.cuda(), offsets.cuda(), wq.cuda(), ws.cuda(), out_dtype=torch.float32)
    g = groups - 1
    a, b = int(offsets[g]), int(offsets[g + 1])
    assert torch.equal(out[a:b], expected(xq[a:b], xs[a:b], wq[g], ws[g], torch.float32))


# Every kernel and split that the rules choose, each with its launch plan.
PLANS = [
    # T, N, K, counts of the groups or None, tile rows, parts
    (1, 300, 700, None, 1, 1), (2, 300, 700, None, 2, 1), (2, 5000, 260, None, 2, 1), (3, 300, 700, None, 4, 1), (4, 5000, 260, None, 4, 1),
    (2, 130, 60000, None, 16, 8), (5, 300, 700, None, 16, 1), (16, 1300, 1100, None, 16, 2), (9, 140, 3300, None, 16, 6),
    (13, 2112, 7168, None, 16, 5), (16, 12288, 1600, None, 16, 3), (16, 2500, 2100, None, 16, 4), (32, 300, 5000, None, 32, 8),
    (24, 7168, 2600, None, 32, 5), (33, 900, 900, None, 64, 2), (64, 2500, 3300, None, 64, 5), (64, 12288, 700, None, 64, 1), (100, 130, 9000, None, 64, 8),
    (257, 12288, 1100, None, 256, 1), (2300, 1024, 4000, None, 256, 2), (2250, 1000, 3990, None, 256, 2), (2177, 1025, 1200, None, 256, 1), (5000, 1500, 1000, None, 256, 1),
    (9, 500, 900, [1, 0, 3, 0, 0, 4], 2, 1), (60, 500, 900, [9, 11, 2, 0, 17, 9, 3, 8], 16, 2), (60, 500, 4100, [9, 31, 20], 32, 5),
    (300, 500, 900, [90, 31, 0, 150, 3], 64, 2), (40, 40, 60, [40], 64, 1), (2000, 3000, 1100, [700, 129, 128, 1, 1000], 256, 1), (1600, 700, 8100, [1400, 150], 256, 2),
    (16, 700, 900, [5, 5, 6], 2, 1),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("T,N,K,counts,tile,parts", PLANS)
def test_every_kernel_and_split(T, N, K, counts, tile, parts, dtype):
    G = len(counts) if counts else 0
    plan = mse.int8_launch_plan(T, N, K, G)
    assert (plan["tile_rows"], plan["parts"]) == (tile, parts) and plan["one_launch"] == (tile == 1 and not counts)
    # magnitudes that need all of 32 bits in the longest sums
    pitch = -(-K // 16) * 16
    xq, wq = integers(T, K, seed=1, top=128).abs().clamp_max(127).to(torch.int8), integers(max(G, 1), N, K, seed=2, top=128)
    xs, ws = scales(T, seed=3), scales(max(G, 1), N, seed=4)
    out = torch.full((T, N), 77.0, dtype=dtype, device="cuda")
    w = rows_with_pitch(wq, pitch, 0x7F)
    if counts:
        offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
        mse.int8_grouped_matmul(rows_with_pitch(xq, pitch, 0x7F), xs.cuda(), offsets.cuda(), w, ws.cuda(), out=out)
        end = offsets.tolist()
    else:
        mse.int8_matmul(rows_with_pitch(xq, pitch, 0x7F), xs.cuda(), w[0], ws[0].cuda(), out=out)
        end = [0, T]
    for g, (a, b) in enumerate(zip(end, end[1:])):
        if a < b:
            assert torch.equal(out[a:b], expected(xq[a:b], xs[a:b], wq[g], ws[g], dtype)), g
    assert bool((out[end[-1]:] == 77).all())


# ------------------------------------------------------------------------------------ together

def layer(x, ids, weights, E, first, wgu, wd, shared, stages=None):
    q, s = mse.int8_quantise(x)
    rows, place, offsets, rs = mse.moe_sort(q, ids, E, first_expert=first, scales=s)
    gu = mse.int8_grouped_matmul(rows, rs, offsets, *wgu, out_dtype=torch.float32)
    h, hs = mse.int8_quantise(gu, swiglu=True, offsets=offsets)
    o = mse.int8_grouped_matmul(h, hs, offsets, *wd, out_dtype=torch.float32)
    if stages is not None:
        stages.update(rows=rows, place=place, offsets=offsets, rs=rs, gu=gu, h=h, hs=hs, o=o)
    return mse.moe_unsort(o, place, weights, base=shared, y_dtype=torch.bfloat16)


def layer_inputs(T, H, I, E, total, k, seed=0):
    x = torch.randn(T, H, generator=gen(seed)).to(torch.bfloat16).cuda()
    ids, w = mse.moe_route(torch.randn(T, total, generator=gen(seed + 1)).cuda(), k)
    wgu = mse.int8_quantise((torch.randn(E, 2 * I, H, generator=gen(seed + 2)) / math.sqrt(H)).to(torch.bfloat16).cuda())
    wd = mse.int8_quantise((torch.randn(E, H, I, generator=gen(seed + 3)) / math.sqrt(I)).to(torch.bfloat16).cuda())
    shared = torch.randn(T, H, generator=gen(seed + 4)).to(torch.bfloat16).cuda()
    return x, ids, w, E, (total - E) // 2, wgu, wd, shared


@pytest.mark.parametrize("T,H,I,E,total,k", [(1, 1024, 512, 8, 8, 4), (40, 1000, 700, 6, 12, 3), (300, 512, 256, 16, 16, 8)])
def test_experts_in_8_bit_integers(T, H, I, E, total, k, path):
    x, ids, w, E, first, wgu, wd, shared = args = layer_inputs(T, H, I, E, total, k)
    st = {}
    y = layer(*args, stages=st)
    place, order, offsets = ref.sort(ids.cpu(), E, first)
    n = len(order)
    of = torch.tensor(order, dtype=torch.long) // k
    xq, xs = ref.quantised(x.cpu())
    assert torch.equal(st["rows"][:n].cpu().double(), xq[of]) and torch.equal(st["rs"][:n].cpu(), xs[of])
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        assert torch.equal(st["gu"][a:b], expected(st["rows"][a:b], st["rs"][a:b], wgu[0][e], wgu[1][e], torch.float32))
        assert torch.equal(st["o"][a:b], expected(st["h"][a:b], st["hs"][a:b], wd[0][e], wd[1][e], torch.float32))
    h = ref.swiglu(st["gu"][:n].cpu())
    held = st["h"][:n].cpu().double() * st["hs"][:n].cpu().double()[:, None]
    # half a step of 1 / 127 of the row's largest, and h's own error
    assert bool(((held - h).abs() <= h.abs().amax(1, keepdim=True) * (0.5 / 127 + 2.0 ** -17)).all())
    want, size = ref.unsort(st["o"].cpu(), place, w.cpu(), shared.cpu())
    bound = (2 * k + 1) * 2.0 ** -24 * size * 2 + 2.0 ** -8 * want.abs()
    assert bool(((y.double().cpu() - want).abs() <= bound).all())


def test_kernels_agree_bit_for_bit():
    args = layer_inputs(70, 512, 384, 8, 8, 4)
    with kernel_path(mse.PATH_GENERIC):
        a = layer(*args)
    assert torch.equal(a, layer(*args))


def test_a_captured_layer_follows_its_inputs():
    x, ids, w, *rest = layer_inputs(24, 512, 256, 8, 16, 4)
    rest = tuple(rest)
    layer(x, ids, w, *rest)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, ids, w, *rest)
    for seed in (11, 12, 13):
        x2, ids2, w2, *_ = layer_inputs(24, 512, 256, 8, 16, 4, seed)
        x.copy_(x2)
        ids.copy_(ids2)
        w.copy_(w2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer(x2, ids2, w2, *rest))


@pytest.mark.parametrize("T", [3, 40])
def test_on_another_stream(T):
    args = layer_inputs(T, 512, 256, 8, 8, 4)
    want = layer(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = layer(*args)
    side.synchronize()
    assert torch.equal(got, want)
    torch.cuda._sleep(20_000_000)
    wq, ws = args[5][0][0], args[5][1][0]
    a = mse.int8_linear(args[0], wq, ws, stream=side)
    side.synchronize()
    assert torch.equal(a, mse.int8_linear(args[0], wq, ws))


def test_calls_in_turn_share_a_workspace():
    wq, ws = mse.int8_quantise(torch.randn(700, 1000, generator=gen(2)).to(torch.bfloat16).cuda())
    xs = [torch.randn(T, 1000, generator=gen(T)).to(torch.bfloat16).cuda() for T in (300, 1, 64, 9, 130, 8)]
    want = [mse.int8_linear(x, wq, ws) for x in xs]
    space = mse.new_int8_workspace(300, 700, 1000)
    ys = [torch.empty_like(w) for w in want]
    for _ in range(20):
        for x, y in zip(xs, ys):
            mse.int8_linear(x, wq, ws, y=y, workspace=space)
    for y, w in zip(ys, want):
        assert torch.equal(y, w)


def test_a_decode_loop_on_kept_buffers():
    # every call writes what the next one reads, and the next round writes it again
    steps = [layer_inputs(T, 512, 256, 8, 16, 4, seed) for seed, T in enumerate((24, 3, 24, 1, 40, 24))]
    weights = steps[0][5:7]
    steps = [(x, ids, w, E, first, *weights, shared) for x, ids, w, E, first, _, _, shared in steps]
    want = [layer(*s) for s in steps]
    T, k, E, H, I = 40, 4, 8, 512, 256
    P = T * k
    keep = dict(q=torch.empty(T, H, dtype=torch.int8, device="cuda"), s=torch.empty(T, device="cuda"), rows=torch.empty(P, H, dtype=torch.int8, device="cuda"),
                rs=torch.empty(P, device="cuda"), place=torch.empty(T, k, dtype=torch.int32, device="cuda"), off=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                gu=torch.empty(P, 2 * I, device="cuda"), h=torch.empty(P, I, dtype=torch.int8, device="cuda"), hs=torch.empty(P, device="cuda"),
                o=torch.empty(P, H, device="cuda"), space=mse.new_int8_workspace(P, 2 * I, H, E), sort=mse.new_moe_sort_workspace(T, k, E))

    def run(x, ids, w, E, first, wgu, wd, shared):
        t, p, b = x.shape[0], x.shape[0] * k, keep
        q, s = mse.int8_quantise(x, q=b["q"][:t], scales=b["s"][:t])
        rows, place, off, rs = mse.moe_sort(q, ids, E, first_expert=first, scales=s, rows=b["rows"][:p], row_scales=b["rs"][:p], place=b["place"][:t],
                                            offsets=b["off"], workspace=b["sort"])
        gu = mse.int8_grouped_matmul(rows, rs, off, *wgu, out=b["gu"][:p], workspace=b["space"])
        h, hs = mse.int8_quantise(gu, swiglu=True, offsets=off, q=b["h"][:p], scales=b["hs"][:p])
        o = mse.int8_grouped_matmul(h, hs, off, *wd, out=b["o"][:p], workspace=b["space"])
        return mse.moe_unsort(o, place, w, base=shared, y_dtype=torch.bfloat16)

    got = [run(*s) for _ in range(30) for s in steps]
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % len(steps)]), i


def test_two_streams_with_workspaces_of_their_own():
    args = [layer_inputs(T, 512, 256, 8, 8, 4, T) for T in (33, 40)]
    want = [layer(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(*args[i]))
    torch.cuda.synchronize()
    for ys, w in zip(got, want):
        assert all(torch.equal(y, w) for y in ys)


def test_outputs_beyond_32_bits():
    T, N, K = 300_007, 7168, 48
    xq, wq = integers(T, K, seed=1).cuda(), integers(N, K, seed=2).cuda()
    xs, ws = scales(T, seed=3).cuda(), scales(N, seed=4).cuda()
    y = mse.int8_matmul(xq, xs, wq, ws)
    for rows in (slice(0, 9), slice(299_520, 299_700), slice(T - 300, T)):
        assert torch.equal(y[rows], expected(xq[rows], xs[rows], wq, ws, torch.bfloat16))


@pytest.mark.parametrize("tokens", ["24", "300"])
def test_the_example_runs(tokens):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "moe_layer.py"), "--int8", "--tokens", tokens, "--experts", "6", "--top-k", "3",
                        "--hidden", "512", "--intermediate", "256", "--steps", "2", "--check"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "relative error" in r.stdout
