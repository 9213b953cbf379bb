"""Tokens sorted by expert and back, and the gradients of both ways, against plain 64-bit forms."""
import pytest

from tests import sorted_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

mse = pytest.importorskip("moe_shared_expert_gb300")

EPS32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


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


def some_ids(T, k, total, seed, closed=0.2):
    ids = torch.randint(0, total, (T, k), generator=gen(seed), dtype=torch.int32)   # an expert twice now and then
    ids[torch.rand(T, k, generator=gen(seed + 1)) < closed] = -1
    if T > 2:
        ids[T // 2] = -1                                                              # a token without any
    return ids


def pitched(rows, cols, dtype, pitch, fill, shift=0):
    """(tensor [rows, cols] on the GPU in a buffer of `fill` bytes, the buffer): rows of a pitch, begun `shift` values late."""
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full(((rows * pitch + shift) * size,), fill, dtype=torch.uint8, device="cuda")
    return raw.view(dtype)[shift:].as_strided((rows, cols), (pitch, 1)), raw


SORTS = [
    # T, k, E, total, first, H, dtype, pitch of x and of rows beyond H, first value
    (1, 8, 32, 32, 0, 7168, torch.bfloat16, 0, 0, 0),
    (1, 1, 1, 1, 0, 1, torch.float32, 0, 0, 0),
    (2, 32, 5, 9, 3, 33, torch.int8, 0, 15, 0),
    (3, 2, 1024, 1024, 0, 129, torch.bfloat16, 7, 0, 1),
    (64, 8, 32, 128, 48, 7168, torch.bfloat16, 0, 0, 0),
    (33, 3, 10, 10, 0, 1001, torch.float32, 0, 3, 0),
    (300, 5, 7, 7, 0, 100, torch.int8, 12, 28, 4),
    (513, 8, 16, 64, 16, 512, torch.bfloat16, 0, 0, 0),      # more pairs than every CTA counts: 4104
    (512, 8, 16, 64, 16, 512, torch.bfloat16, 0, 0, 0),
    (5000, 6, 256, 256, 0, 72, torch.float32, 0, 0, 0),      # 30,000: counted by a cluster
    (4096, 8, 1024, 1024, 0, 16, torch.bfloat16, 0, 0, 0),   # 32,768
    (4097, 8, 30, 40, 5, 16, torch.bfloat16, 0, 0, 0),       # and beyond
    (20, 8, 5, 5, 0, 2048, torch.bfloat16, 0, 0, 0),
    (9000, 1, 3, 3, 0, 40, torch.float16, 0, 0, 0),
    (2100, 32, 40, 50, 2, 16, torch.float8_e4m3fn, 0, 0, 0),
]


@pytest.mark.parametrize("case", SORTS, ids=lambda c: "-".join(map(str, c)))
def test_sort(case):
    T, k, E, total, first, H, dtype, px, pr, shift = case
    size = torch.empty(0, dtype=dtype).element_size()
    x, _ = pitched(T, H, dtype, H + px, 0, shift)
    bits = torch.randint(0, 256, (T, H * size), generator=gen(T), dtype=torch.uint8)
    x.copy_(bits.view(dtype))
    ids = some_ids(T, k, total, T + 7)
    scales = torch.randn(T, generator=gen(5)).cuda()
    rows, raw = pitched(T * k, H, dtype, H + pr, 0xA5, shift)
    row_scales = torch.full((T * k,), 7.0, device="cuda")
    got, place, offsets, rs = mse.moe_sort(x, ids.cuda(), E, first_expert=first, scales=scales, rows=rows, row_scales=row_scales)
    want_place, order, want_offsets = ref.sort(ids, E, first)
    assert torch.equal(place.cpu(), want_place) and torch.equal(offsets.cpu(), want_offsets)
    n = len(order)
    of = torch.tensor(order, dtype=torch.long) // k
    want = torch.full(((T * k * (H + pr) + shift) * size,), 0xA5, dtype=torch.uint8)
    view = want[shift * size:].view(T * k, (H + pr) * size)
    view[:n, :H * size] = bits[of]
    assert torch.equal(raw.cpu(), want)                       # the rows, and everything else as it was
    assert torch.equal(rs.cpu()[:n], scales.cpu()[of]) and bool((rs[n:] == 7.0).all())


def test_sort_makes_its_own_outputs():
    x = torch.randn(9, 100, generator=gen(1)).cuda()
    ids = some_ids(9, 3, 4, 2)
    rows, place, offsets, scales = mse.moe_sort(x, ids.cuda(), 4)
    want_place, order, want_offsets = ref.sort(ids, 4)
    assert scales is None and rows.shape == (27, 100) and torch.equal(place.cpu(), want_place)
    assert torch.equal(rows[:len(order)].cpu(), x.cpu()[torch.tensor(order) // 3]) and torch.equal(offsets.cpu(), want_offsets)
    q = mse.moe_sort(x.to(torch.int8), ids.cuda(), 4)[0]
    assert q.stride() == (112, 1)                             # as the products want them


def test_ids_far_outside_belong_to_nobody():
    ids = torch.tensor([[0, 2 ** 31 - 1], [-2 ** 31, 5], [7, 4]], dtype=torch.int32)
    x = torch.randn(3, 8, generator=gen(1)).cuda()
    _, place, offsets, _ = mse.moe_sort(x, ids.cuda(), 3, first_expert=4)
    assert place.cpu().tolist() == [[-1, -1], [-1, 1], [-1, 0]] and offsets.cpu().tolist() == [0, 1, 2, 2]


def test_no_pair_at_all():
    rows = torch.full((6, 8), 3.0, device="cuda")
    ids = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    _, place, offsets, _ = mse.moe_sort(torch.randn(3, 8).cuda(), ids, 4, rows=rows)
    assert bool((rows == 3.0).all()) and place.cpu().eq(-1).all() and offsets.cpu().tolist() == [0] * 5
    w = torch.ones(3, 2, device="cuda")
    assert bool((mse.moe_unsort(rows, place, w) == 0).all())
    drows, dw = mse.moe_unsort_backward(torch.randn(3, 8).cuda(), place, rows, w, drows=rows.clone())
    assert bool((drows == 3.0).all()) and bool((dw == 0).all())


UNSORTS = [
    # T, k, E, total, H, pitch beyond H, weights, base
    (1, 8, 32, 32, 7168, 0, True, True),
    (1, 1, 1, 1, 1, 0, False, False),
    (2, 32, 5, 9, 33, 0, True, False),
    (64, 8, 32, 128, 7168, 0, True, True),
    (33, 3, 10, 10, 1001, 3, True, True),
    (7, 5, 10, 10, 1002, 0, False, True),
    (9, 4, 10, 10, 1004, 4, True, "y"),
    (300, 5, 7, 7, 100, 0, False, False),
    (1300, 2, 3, 4, 256, 0, True, False),
]
DTYPES = [(a, b) for a in (torch.bfloat16, torch.float32) for b in (torch.bfloat16, torch.float32)]


def unsort_inputs(case, rows_dtype, y_dtype):
    T, k, E, total, H, pr, weighted, based = case
    place, order, _ = ref.sort(some_ids(T, k, total, T + H), E)
    rows, _ = pitched(T * k, H, rows_dtype, H + pr, 0)
    rows.copy_(torch.randn(T * k, H, generator=gen(1)))
    rows[len(order):] = torch.nan                             # rows that no pair has reach nothing
    w = torch.randn(T, k, generator=gen(2)).masked_fill(place < 0, torch.inf) if weighted else None
    base = torch.randn(T, H, generator=gen(3)).to(y_dtype) if based else None
    return place, rows, w, base


def close(got, want, size, terms, dtype):
    # `terms` roundings to fp32 of at most `size`, then one to dtype
    bound = terms * EPS32 * size + HALF_STEP[dtype] * (want.abs() + terms * EPS32 * size)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp_min(1e-300)).max())


@pytest.mark.parametrize("dtypes", DTYPES, ids=str)
@pytest.mark.parametrize("case", UNSORTS, ids=lambda c: "-".join(map(str, c)))
def test_unsort(case, dtypes):
    place, rows, w, base = unsort_inputs(case, *dtypes)
    y = base.cuda() if case[-1] == "y" else None
    got = mse.moe_unsort(rows, place.cuda(), None if w is None else w.cuda(),
                         base=y if y is not None else None if base is None else base.cuda(), y=y, y_dtype=dtypes[1])
    want, size = ref.unsort(rows.cpu(), place, w, base)
    assert got.dtype is dtypes[1]
    close(got, want, size, 2 * case[1] + 1, dtypes[1])


def test_unsort_leaves_out_places_beyond_the_rows():
    rows = torch.randn(4, 16, generator=gen(1)).cuda()
    place = torch.tensor([[3, 4], [-1, 2 ** 31 - 1], [-2 ** 31, 0]], dtype=torch.int32, device="cuda")
    y = mse.moe_unsort(rows, place)
    assert torch.equal(y[0], rows[3]) and bool((y[1] == 0).all()) and torch.equal(y[2], rows[0])
    dy = torch.randn(3, 16, generator=gen(2)).cuda()
    drows, dw = mse.moe_unsort_backward(dy, place, rows, torch.ones(3, 2, device="cuda"), drows=torch.zeros_like(rows))
    assert torch.equal(drows[3], dy[0]) and torch.equal(drows[0], dy[2]) and bool((drows[1:3] == 0).all())
    assert dw[0, 1] == dw[1, 0] == dw[1, 1] == dw[2, 0] == 0


@pytest.mark.parametrize("dtypes", DTYPES, ids=str)
@pytest.mark.parametrize("case", [c for c in UNSORTS if c[-1] != "y"], ids=lambda c: "-".join(map(str, c)))
def test_unsort_backward(case, dtypes):
    T, k, _, _, H = case[:5]
    place, rows, w, _ = unsort_inputs(case, *dtypes)
    dy = torch.randn(T, H, generator=gen(4)).to(dtypes[1])
    n = int((place >= 0).sum())
    drows, raw = pitched(T * k, H, dtypes[0], H + 5, 0x11)
    before = drows.clone()
    if w is None:
        got, dw = mse.moe_unsort_backward(dy.cuda(), place.cuda(), drows=drows)
        assert dw is None
    else:
        got, dw = mse.moe_unsort_backward(dy.cuda(), place.cuda(), rows, w.cuda(), drows=drows)
    want, want_dw, size = ref.unsort_backward(dy, place, None if w is None else rows.cpu(), w, T * k)
    assert got is drows and torch.equal(got[n:], before[n:])
    assert raw.view(dtypes[0]).view(T * k, H + 5)[:, H:].view(torch.uint8).eq(0x11).all()
    close(got[:n], want[:n], want[:n].abs(), 1, dtypes[0])
    if w is not None:
        # a thread adds at most H / 128 + 8 products; five and four sums of the threads' follow
        bound = (H / 128 + 8 + 9) * EPS32 * size
        assert bool(((dw.double().cpu() - want_dw).abs() <= bound).all())
        assert bool((dw.cpu()[place < 0] == 0).all())


def test_gradients_in_place_of_the_rows():
    place, rows, w, _ = unsort_inputs((33, 4, 5, 6, 264, 0, True, False), torch.bfloat16, torch.bfloat16)
    dy = torch.randn(33, 264, generator=gen(4)).to(torch.bfloat16).cuda()
    want = mse.moe_unsort_backward(dy, place.cuda(), rows, w.cuda(), drows=rows.clone())
    got = mse.moe_unsort_backward(dy, place.cuda(), rows, w.cuda(), drows=rows)
    n = int((place >= 0).sum())
    assert got[0] is rows and torch.equal(got[0][:n], want[0][:n]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,k,H", [(33, 5, 264), (700, 12, 1001)])
def test_weights_gradient_in_place_of_the_weights(T, k, H):
    place, rows, w, _ = unsort_inputs((T, 4, k, 14, H, 0, True, False), torch.bfloat16, torch.float32)
    dy, w = torch.randn(T, H, generator=gen(4)).cuda(), w.cuda()
    want = mse.moe_unsort_backward(dy, place.cuda(), rows, w)
    got = mse.moe_unsort_backward(dy, place.cuda(), rows, w, dweights=w)
    n = int((place >= 0).sum())
    assert got[1] is w and torch.equal(w, want[1]) and torch.equal(got[0][:n], want[0][:n])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_sort_backward(dtype):
    T, k, E, H = 40, 6, 9, 264
    place, order, _ = ref.sort(some_ids(T, k, E, 3), E)
    d = torch.randn(T * k, H, generator=gen(1)).to(dtype).cuda()
    got = mse.moe_sort_backward(d, place.cuda())
    want, size = ref.unsort(d.cpu(), place)
    close(got, want, size, k, dtype)


def test_gradients_are_the_differences():
    """s = <dy, y> is linear in rows, in weights and in x: a step along an input changes it by the gradient times the step."""
    T, k, E, H = 21, 3, 5, 136
    place, order, _ = ref.sort(some_ids(T, k, E, 3), E)
    n = len(order)
    rows = torch.randn(T * k, H, generator=gen(1)).cuda()
    w = torch.randn(T, k, generator=gen(2)).cuda()
    dy = torch.randn(T, H, generator=gen(4)).cuda()
    drows, dw = mse.moe_unsort_backward(dy, place.cuda(), rows, w, drows=torch.zeros_like(rows))

    def s(rows, w):
        return float((mse.moe_unsort(rows, place.cuda(), w).double() * dy.double()).sum())

    at = s(rows, w)
    # the two sums differ by roundings of y: k + 1 of 2^-24 each, of terms whose sizes add up to at most `size`
    size = float((ref.unsort(rows.cpu().abs(), place, w.cpu().abs())[0] * dy.cpu().double().abs()).sum())
    tol = 2 * 2 * (2 * k + 1) * EPS32 * size
    for row in range(0, n, 7):
        for col in (0, 77, H - 1):
            step = torch.zeros_like(rows)
            step[row, col] = 1.0
            assert abs(s(rows + step, w) - at - float(drows[row, col])) <= tol
    for t in range(0, T, 5):
        step = torch.zeros_like(w)
        step[t, 1] = 1.0
        assert abs(s(rows, w + step) - at - float(dw[t, 1])) <= tol
    x = torch.randn(T, H, generator=gen(6)).cuda()
    ids = torch.full((T, k), -1, dtype=torch.int32)
    offsets = ref.sort(some_ids(T, k, E, 3), E)[2]
    for t in range(T):
        for j in range(k):
            if place[t, j] >= 0:
                ids[t, j] = int(torch.searchsorted(offsets, place[t, j], right=True)) - 1
    g = torch.randn(T * k, H, generator=gen(7)).cuda()
    dx = mse.moe_sort_backward(g, place.cuda())

    def r(x):
        out, p, _, _ = mse.moe_sort(x, ids.cuda(), E)
        assert torch.equal(p.cpu(), place)
        return float((out[:n].double() * g[:n].double()).sum())

    at = r(x)
    for t in range(0, T, 4):
        step = torch.zeros_like(x)
        step[t, 3] = 4.0
        # a sum of copies: x + 4 is rounded once, dx by k sums
        assert abs((r(x + step) - at) - 4.0 * float(dx[t, 3])) <= 4 * (k + 2) * EPS32 * 8 * k * float(g.abs().max())


def test_rows_beyond_32_bits():
    # 37,500 tokens of 7168 to eight experts each: more values than 31 bits count
    T, k, E, H = 37_500, 8, 16, 7168
    ids = torch.rand(T, E, generator=gen(1)).topk(k, 1).indices.to(torch.int32).cuda()
    x = torch.arange(T, device="cuda").to(torch.float32)[:, None].expand(T, H).contiguous().to(torch.bfloat16)
    x[:, 0] = (torch.arange(T, device="cuda") % 128).to(torch.bfloat16)
    x[:, 1] = torch.div(torch.arange(T, device="cuda"), 128, rounding_mode="floor").to(torch.bfloat16)
    rows, place, offsets, _ = mse.moe_sort(x, ids, E)
    assert int(offsets[-1]) == T * k and torch.equal(place.flatten().sort().values.long(), torch.arange(T * k, device="cuda"))
    for t in (0, 1, T // 2, T - 1):
        for j in (0, k - 1):
            assert torch.equal(rows[int(place[t, j])], x[t])
    last = int(offsets[-1]) - 1
    t = int((place == last).nonzero()[0, 0])
    assert torch.equal(rows[last], x[t])
    y = mse.moe_unsort(rows, place, torch.full((T, k), 0.125, device="cuda"))
    assert torch.equal(y, x)                                  # eight eighths of the same value
    drows, dw = mse.moe_unsort_backward(x, place, rows, torch.full((T, k), 2.0, device="cuda"))
    assert torch.equal(drows[last], 2 * x[t])
    want = (x[t].double() ** 2).sum()
    assert abs(float(dw[t].double().max() - want)) <= (H / 128 + 17) * EPS32 * float(want)


def test_a_captured_round_trip_follows_its_inputs():
    T, k, E, H = 60, 4, 9, 264
    w = torch.rand(T, k, generator=gen(2)).cuda()
    x, ids = torch.empty(T, H, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")

    def step():
        rows, place, _, _ = mse.moe_sort(x, ids, E, rows=torch.zeros(T * k, H, device="cuda"))
        y = mse.moe_unsort(rows, place, w, base=x)
        drows, dw = mse.moe_unsort_backward(y, place, rows, w, drows=torch.zeros_like(rows))
        return y, drows, dw, mse.moe_sort_backward(drows, place)

    def fill(seed):
        x.copy_(torch.randn(T, H, generator=gen(seed)))
        ids.copy_(some_ids(T, k, E, seed))

    fill(1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (5, 6, 7):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, step()):
            assert torch.equal(a, b)


def test_a_program_s_backward_pass():
    """The calls within an autograd function, experts of one matrix each in torch: gradients as autograd finds them for the plain layer."""
    T, k, E, H = 30, 3, 5, 72

    class Sort(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, ids):
            rows, place, offsets, _ = mse.moe_sort(x, ids, E, rows=torch.zeros(T * k, H, device="cuda"))
            ctx.save_for_backward(place)
            ctx.mark_non_differentiable(place, offsets)
            return rows, place, offsets

        @staticmethod
        def backward(ctx, drows, *_):
            return mse.moe_sort_backward(drows.contiguous(), *ctx.saved_tensors), None

    class Unsort(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, place, w, base):
            ctx.save_for_backward(rows, place, w)
            return mse.moe_unsort(rows, place, w, base=base)

        @staticmethod
        def backward(ctx, dy):
            rows, place, w = ctx.saved_tensors
            drows, dw = mse.moe_unsort_backward(dy.contiguous(), place, rows, w, drows=torch.zeros_like(rows))
            return drows, None, dw, dy

    ids = some_ids(T, k, E, 3)
    leaves = [torch.randn(T, H, generator=gen(1)), torch.rand(T, k, generator=gen(2)), torch.randn(E, H, H, generator=gen(3)) / H ** 0.5]
    dy = torch.randn(T, H, generator=gen(4))
    x, w, m = [v.cuda().requires_grad_() for v in leaves]
    rows, place, offsets = Sort.apply(x, ids.cuda())
    at = offsets.tolist()
    out = torch.cat([rows[at[e]:at[e + 1]] @ m[e] for e in range(E)] + [rows[at[E]:]])
    Unsort.apply(out, place, w, x).backward(dy.cuda())
    X, W, M = [v.double().requires_grad_() for v in leaves]
    y = X
    for j in range(k):
        here = (ids[:, j] >= 0).double()[:, None]
        y = y + here * W[:, j, None] * torch.einsum("th,thg->tg", X, M[ids[:, j].clamp_min(0).long()])
    y.backward(dy.double())
    # fp32 products and sums of up to H k terms of a few units each
    for got, want in ((x, X), (w, W), (m, M)):
        assert float((got.grad.double().cpu() - want.grad).abs().max()) <= 2.0 ** -24 * H * (k + 2) * float(want.grad.abs().max() + 1)
