"""slim_dequant_grouped_gemm with an index into no rows of x (T = 0): every index is outside, every product zero."""
import pytest
import torch

import grouped_util as U
from post_weight_quantization_hessian_b200 import build, slim

EINVAL, ENODEV, EINJECTED = 1, 6, 7


def test_x_may_be_null_without_rows(monkeypatch):
    """Accepted by the checks of arguments (the injected failure comes behind them, before any launch)."""
    build.build()
    monkeypatch.setenv("SLIM_FAULT", "dequant_grouped_gemm")

    def call(x, T):
        return slim._lib().slim_dequant_grouped_gemm(0x1000, 0x2000, 0x3000, 0x4000, 4, 256, 640, 128, 2, x, 1, T, 0x8000,
                                                     0x6000, 100, 0x7000, 1, None, 0, None)

    assert call(None, 0) in (ENODEV, EINJECTED)
    assert call(None, 1) == EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R", [1, 20, 90])
def test_no_rows_of_x(R, dtype):
    m, n = 150, 512
    layer = U.random_layers(2, m, n, 64, 2, 1)
    index = torch.randint(-3, 5, (R + 1,), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, R // 2, R], dtype=torch.int32, device="cuda")
    y = torch.full((R + 1, m), 7.0, device="cuda")
    slim.slim_dequant_grouped_gemm(*layer, 64, 2, torch.empty((0, n), dtype=dtype, device="cuda"), off, row_index=index, y=y)
    slim.slim_async_status()
    assert torch.count_nonzero(y[:R]) == 0 and torch.all(y[R:] == 7.0)
