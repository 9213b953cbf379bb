"""Calls in turn on one workspace, without a pause between them: each reads what its own kernels wrote."""
import pytest

from tests.test_gpu_routed import gen, make_experts

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


@pytest.mark.parametrize("T,N,K", [(3, 500, 900), (64, 3000, 2000), (300, 4000, 5000), (1500, 2560, 512)])
def test_linear_calls_in_turn(T, N, K):
    wq, ws = mse.fp8_block_quantise(torch.randn(N, K, generator=gen(N)).to(torch.bfloat16).cuda(), block_rows=128)
    # tokens whose scales differ by powers of two from call to call: a stale scale or value is far off
    xs = [(torch.randn(T, K, generator=gen(i)) * 4.0 ** (i - 3)).to(torch.bfloat16).cuda() for i in range(6)]
    want = [mse.fp8_block_linear(x, wq, ws) for x in xs]
    torch.cuda.synchronize()
    buf = mse.new_fp8_linear_workspace(T, N, K)
    for _ in range(5):
        got = [torch.empty_like(y) for y in want]
        torch.cuda.synchronize()
        for x, y in zip(xs, got):
            mse.fp8_block_linear(x, wq, ws, y=y, workspace=buf)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 9, 90, 900])
def test_experts_calls_in_turn_with_and_without_pairs(T):
    # calls of which the rank holds no pair between others on the same workspace
    E, H, I, k = 5, 640, 256, 3
    weights = make_experts(E, H, I, 9)
    x = [(torch.randn(T, H, generator=gen(i)) * 4.0 ** (i % 3 - 1)).to(torch.bfloat16).cuda() for i in range(6)]
    ids = [(torch.randint(0, E, (T, k), generator=gen(10 + i)) if i % 2 else torch.full((T, k), 77)).to(torch.int32).cuda()
           for i in range(6)]
    w = torch.rand(T, k, generator=gen(20)).cuda()
    want = [mse.moe_experts_forward(a, i, w, *weights) for a, i in zip(x, ids)]
    assert all(want[i].any() == (i % 2 == 1) for i in range(6))
    buf = mse.new_moe_workspace(T, k, E, H, I)
    for _ in range(5):
        got = [torch.empty_like(y) for y in want]
        torch.cuda.synchronize()
        for a, i, y in zip(x, ids, got):
            mse.moe_experts_forward(a, i, w, *weights, y=y, workspace=buf)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 3, 40])
def test_a_decode_loop_on_kept_buffers(T):
    # every step routes into the same ids and weights, and its experts read them at once
    E, H, I, k = 12, 512, 256, 4
    weights = make_experts(E, H, I, 30)
    steps = 8
    logits = torch.randn(steps, T, E, generator=gen(31)).cuda()
    x = torch.randn(steps, T, H, generator=gen(32)).to(torch.bfloat16).cuda()
    want = torch.empty_like(x)
    for i in range(steps):
        torch.cuda.synchronize()
        want[i] = mse.moe_experts_forward(x[i], *mse.moe_route(logits[i], k), *weights)
    torch.cuda.synchronize()
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    buf = mse.new_moe_workspace(T, k, E, H, I)

    def loop(y):
        for i in range(steps):
            mse.moe_route(logits[i], k, ids=ids, weights=w)
            mse.moe_experts_forward(x[i], ids, w, *weights, y=y[i], workspace=buf)

    for _ in range(5):
        y = torch.empty_like(x)
        torch.cuda.synchronize()
        loop(y)
        assert torch.equal(y, want)
    y = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop(y)
    for _ in range(3):
        y.zero_()
        graph.replay()
        assert torch.equal(y, want)


@pytest.mark.parametrize("T", [1, 8, 9, 70, 600])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_onto_its_own_tokens(T, dtype):
    N, K = 512, 1024
    wq, ws = mse.fp8_block_quantise(torch.randn(N, K, generator=gen(40)).to(torch.bfloat16).cuda(), block_rows=128)
    x = torch.randn(T, K, generator=gen(41)).to(torch.bfloat16).cuda()
    want = mse.fp8_block_linear(x, wq, ws, y_dtype=dtype)
    for _ in range(5):
        over = x.clone()
        flat = over.view(-1).view(dtype)
        y = flat[:T * N].view(T, N)                    # bf16: the first half of x; fp32: all of it
        mse.fp8_block_linear(over, wq, ws, y=y)
        assert torch.equal(y, want)
        if dtype is torch.bfloat16:                    # and its second half
            over = x.clone()
            y = over.view(-1)[T * N:].view(T, N)
            mse.fp8_block_linear(over, wq, ws, y=y)
            assert torch.equal(y, want)
