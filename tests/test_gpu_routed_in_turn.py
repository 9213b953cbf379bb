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
