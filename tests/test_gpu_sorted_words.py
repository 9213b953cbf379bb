"""The gradients of the way back in every word and block size, against the plain 64-bit form."""
import pytest

from tests import sorted_ref as ref
from tests.test_gpu_sorted import DTYPES, EPS32, close, gen, pitched, some_ids

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


# T, k, experts here, in all, H, values between rows, between gradients of rows, values of a word (eight of 32 bits are two loads)
WORDS = [
    (40, 8, 12, 16, 7168, 0, 0, 8), (9, 3, 5, 5, 1000, 8, 16, 8), (33, 4, 5, 6, 256, 0, 8, 8),
    (17, 5, 6, 6, 1004, 0, 4, 4), (5, 2, 3, 3, 2052, 4, 0, 4), (21, 6, 8, 9, 264, 12, 4, 4),
    (7, 5, 10, 10, 1002, 0, 0, 2), (30, 4, 5, 5, 1030, 2, 6, 2), (12, 3, 4, 4, 3080, 0, 2, 2),
    (33, 3, 10, 10, 1001, 0, 0, 1), (8, 9, 12, 12, 1000, 8, 3, 1),
    # blocks of 128 threads from four tokens an SM on
    (700, 3, 7, 8, 1032, 0, 0, 8), (650, 5, 6, 6, 516, 0, 4, 4), (640, 2, 4, 4, 1030, 0, 2, 2), (800, 3, 5, 5, 333, 0, 0, 1), (610, 1, 2, 2, 40, 0, 0, 8),
]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtypes", DTYPES, ids=str)
@pytest.mark.parametrize("case", WORDS, ids=lambda c: "-".join(map(str, c)))
def test_unsort_backward(case, dtypes, weighted):
    T, k, E, total, H, pr, pd, word = case
    assert word == max(w for w in (1, 2, 4, 8) if all(n % w == 0 for n in (H, H + pr, H + pd)))
    place, order, _ = ref.sort(some_ids(T, k, total, T + H), E)
    n = len(order)
    rows, _ = pitched(T * k, H, dtypes[0], H + pr, 0)
    rows.copy_(torch.randn(T * k, H, generator=gen(1)))
    rows[n:] = torch.nan                                      # rows that no pair has reach nothing
    w = torch.randn(T, k, generator=gen(2)).masked_fill(place < 0, torch.inf) if weighted else None
    dy = torch.randn(T, H, generator=gen(4)).to(dtypes[1])
    drows, raw = pitched(T * k, H, dtypes[0], H + pd, 0x11)
    before = raw.clone()
    got, dw = mse.moe_unsort_backward(dy.cuda(), place.cuda(), rows if weighted else None, w.cuda() if weighted else None, drows=drows)
    want, want_dw, size = ref.unsort_backward(dy, place, rows.cpu() if weighted else None, w, T * k)
    assert got is drows
    close(got[:n], want[:n], want[:n].abs(), 1, dtypes[0])
    # nothing between the rows or behind the last one that a pair has
    drows[:n] = before.view(dtypes[0]).as_strided((n, H), (H + pd, 1))
    assert torch.equal(raw, before)
    if weighted:
        # a thread adds at most H / 128 + 8 products; five and four sums of the threads' follow
        bound = (H / 128 + 8 + 9) * EPS32 * size
        assert bool(((dw.double().cpu() - want_dw).abs() <= bound).all())
        assert bool((dw.cpu()[place < 0] == 0).all())
    else:
        assert dw is None


@pytest.mark.parametrize("dtypes", DTYPES, ids=str)
@pytest.mark.parametrize("H,word", [(1000, 8), (1004, 4), (1002, 2), (1001, 1)])
def test_dy_and_rows_that_begin_late(H, word, dtypes):
    """The address of every tensor counts, not its pitch alone."""
    T, k, E = 20, 4, 6
    place, order, _ = ref.sort(some_ids(T, k, E, H), E)
    n = len(order)
    for late in range(3):   # dy, rows, drows
        (rows, _), (drows, _) = (pitched(T * k, H, dtypes[0], H + 8, 0, 1 if late == i else 0) for i in (1, 2))
        dy, _ = pitched(T, H, dtypes[1], H, 0, 1 if late == 0 else 0)
        rows.copy_(torch.randn(T * k, H, generator=gen(1)))
        dy.copy_(torch.randn(T, H, generator=gen(4)))
        w = torch.randn(T, k, generator=gen(2))
        _, dw = mse.moe_unsort_backward(dy, place.cuda(), rows, w.cuda(), drows=drows)
        want, want_dw, size = ref.unsort_backward(dy.cpu(), place, rows.cpu(), w)
        close(drows[:n], want[:n], want[:n].abs(), 1, dtypes[0])
        assert bool(((dw.double().cpu() - want_dw).abs() <= (H / 128 + 17) * EPS32 * size).all())
