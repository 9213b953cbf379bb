"""Workspaces, and small outputs, that lie over an input are refused on the host: CTAs read while others write."""
import pytest

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


def over(t, dtype, n):
    """The first n values of `dtype` in t's memory."""
    return t.flatten().view(torch.uint8).view(dtype)[:n]


def refused(f, inputs, **arguments):
    before = [t.clone() for t in inputs]
    with pytest.raises(mse.MSEError, match="INVALID_ARG"):
        f(**arguments)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(inputs, before))


@pytest.mark.parametrize("T", [40, 600])   # every CTA counts all ids, and kernels before the sort count them
@pytest.mark.parametrize("taken", ["x", "ids", "scales"])
@pytest.mark.parametrize("by", ["offsets", "workspace"])
def test_sort(T, taken, by):
    k, E, H = 8, 32, 64
    a = dict(x=torch.randn(T, H, device="cuda"), ids=torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda"),
             scales=torch.randn(max(T, 4096), device="cuda")[:T], num_experts=E)
    if by == "offsets":
        a["offsets"] = over(a[taken], torch.int32, E + 1)
    else:
        # (begun a step before the input's end, in memory of the test's own)
        room = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        t = a[taken]
        a[taken] = room[4096:4096 + t.nbytes].view(t.dtype).view(t.shape).copy_(t)
        a["workspace"] = room[(4096 + t.nbytes - 1) // 256 * 256:]
    refused(mse.moe_sort, [a["x"], a["ids"], a["scales"]], **a)
    del a[by]
    rows, place, offsets, scales = mse.moe_sort(**a)
    assert int(offsets[-1]) == T * k and torch.equal(rows[place[3, 2]], a["x"][3]) and float(scales[place[3, 2]]) == float(a["scales"][3])


@pytest.mark.parametrize("taken", ["dy", "place", "rows", "weights"])
def test_unsort_backward(taken):
    T, k, H = 40, 8, 64
    room = torch.randn(4 * T * k, device="cuda")
    a = dict(dy=torch.randn(T, H, device="cuda"), place=torch.arange(T * k, device="cuda").int().view(T, k),
             rows=torch.randn(T * k, H, device="cuda"), weights=room[:T * k].view(T, k), drows=torch.zeros(T * k, H, device="cuda"))
    # (the weights' own memory is allowed, but not all of it but one)
    dweights = room[1:T * k + 1] if taken == "weights" else over(a[taken], torch.float32, T * k)
    refused(mse.moe_unsort_backward, [a["dy"], a["place"], a["rows"], a["weights"], a["drows"]], dweights=dweights.view(T, k), **a)
    drows, dw = mse.moe_unsort_backward(**a, dweights=room[T * k:2 * T * k].view(T, k))
    assert torch.equal(drows[5 * k + 2], a["weights"][5, 2] * a["dy"][5])


@pytest.mark.parametrize("taken", ["x", "offsets"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_quantise(taken, swiglu):
    x, room = torch.randn(40, 64, device="cuda"), torch.full((80,), 40, dtype=torch.int32, device="cuda")
    offsets = room[:41]
    scales = over(x, torch.float32, 40) if taken == "x" else room.view(torch.float32)[40:]   # (the last offset is read)
    refused(mse.int8_quantise, [x, room], x=x, swiglu=swiglu, offsets=offsets, scales=scales)
    q, s = mse.int8_quantise(x, swiglu=swiglu, offsets=offsets, scales=torch.zeros(40, device="cuda"))
    assert bool((q.abs().amax(1) == 127).all()) and bool((s > 0).all())


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("name,taken", [("int8_matmul", t) for t in ("xq", "xs", "wq", "ws")] + [("int8_linear", t) for t in ("x", "wq", "ws")] +
                         [("int8_grouped_matmul", t) for t in ("xq", "xs", "offsets", "wq", "ws")])
def test_products(name, taken, T):
    N, K, G = 256, 512, 3
    room = torch.zeros(1 << 21, dtype=torch.uint8, device="cuda")
    lead = (G,) if name == "int8_grouped_matmul" else ()
    a = dict(wq=torch.randint(-127, 128, (*lead, N, K), device="cuda").to(torch.int8), ws=torch.rand(*lead, N, device="cuda"))
    if name == "int8_linear":
        a["x"] = torch.randn(T, K, device="cuda")
    else:
        a["xq"], a["xs"] = torch.randint(-127, 128, (T, K), device="cuda").to(torch.int8), torch.rand(T, device="cuda")
    if lead:
        a["offsets"] = torch.tensor([0, T, T, T], dtype=torch.int32, device="cuda")
    t = a[taken]
    a[taken] = room[4096:4096 + t.nbytes].view(t.dtype).view(t.shape).copy_(t)   # the workspace begins where it ends, or just before
    refused(getattr(mse, name), list(a.values()), workspace=room[(4096 + t.nbytes - 1) // 256 * 256:], **a)
    y = getattr(mse, name)(workspace=room[(4096 + t.nbytes + 255) // 256 * 256:], **a)
    assert torch.equal(y, getattr(mse, name)(**a))
