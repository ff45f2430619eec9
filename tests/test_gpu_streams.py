"""The serving calls on the default stream's handle: ordered behind what the default stream was given before."""
import pytest
import torch

from post_weight_quantization_hessian_b200 import slim
import grouped_util as U

pytestmark = pytest.mark.gpu


def slow(t, value):
    """t becomes `value` on the current stream, behind some 10 ms of other work."""
    a = torch.ones((8192, 8192), device="cuda")
    for _ in range(12):
        a = (a @ a).clamp_(0, 1)
    t.copy_(value + 0 * a[0, 0])


@pytest.mark.parametrize("R", [3, 100])
def test_grouped_product_on_handle_zero(R):
    layer = U.random_layers(1, 200, 1024, 128, 2, 1)
    want_x = torch.randn((R, 1024), device="cuda")
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    want = slim.slim_dequant_grouped_gemm(*layer, 128, 2, want_x, off)
    torch.cuda.synchronize()
    assert torch.cuda.current_stream().cuda_stream == 0
    for stream in (0, torch.cuda.default_stream(), None):
        x = torch.zeros_like(want_x)
        slow(x, want_x)
        y = slim.slim_dequant_grouped_gemm(*layer, 128, 2, x, off, stream=stream)
        slim.slim_async_status(stream=stream)
        assert torch.equal(y, want)


def test_log_probabilities_on_handle_zero():
    want_l = torch.randn((50, 3001), device="cuda")
    want = slim.slim_token_logprobs(want_l, top_k=3)
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.default_stream(), None):
        l = torch.zeros_like(want_l)
        slow(l, want_l)
        got = slim.slim_token_logprobs(l, top_k=3, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
