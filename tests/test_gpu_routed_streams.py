"""The routed experts' operators on another stream than the current one, while the current one is busy."""
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


@pytest.mark.parametrize("as_handle", [False, True])
def test_outputs_on_a_side_stream_are_not_the_current_streams_old_blocks(as_handle):
    E, H, I, T, N = 4, 512, 256, 300, 700
    weights = make_experts(E, H, I, 1)
    x = torch.randn(T, H, generator=gen(2)).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=gen(3)).cuda()
    wq, ws = mse.fp8_block_quantise(torch.randn(N, H, generator=gen(4)).to(torch.bfloat16).cuda(), block_rows=128)

    def layer(stream=None):
        ids, w = mse.moe_route(logits, 2, stream=stream)
        y = mse.moe_experts_forward(x, ids, w, *weights, stream=stream)
        z = mse.fp8_block_linear(y, wq, ws, stream=stream)
        return ids, w, y, z, *mse.fp8_block_quantise(z, stream=stream)

    want = [t.clone() for t in layer()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        # blocks of every size that the calls ask for, written late by the current stream and dropped at once
        torch.cuda._sleep(20_000_000)
        for n in (256, T * 2 * 4, T * H * 2, T * N * 2, T * N, 1 << 20, 4 << 20, 16 << 20):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7F)
        got = layer(side.cuda_stream if as_handle else side)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                               b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)
        del got
    torch.cuda.synchronize()


def test_a_handle_of_zero_is_the_default_stream():
    logits = torch.randn(9, 40, generator=gen(5)).cuda()
    ids, w = mse.moe_route(logits, 3)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        ids0, w0 = mse.moe_route(logits, 3, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids0) and torch.equal(w, w0)
