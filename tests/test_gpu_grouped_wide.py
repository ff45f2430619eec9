"""slim_dequant_grouped_gemm on the widest layers that it accepts (n <= 65535, n / group <= 1024), by the few-rows and
the many-rows kernel. Tolerance: the derivation of test_gpu_grouped_mean.py, delta = 3 * 2^-23 (k + g / 16)."""
import pytest
import torch

import grouped_util as U
from post_weight_quantization_hessian_b200 import slim

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n, group, avg", [(53248, 128, 2), (65408, 128, 3), (65472, 64, 2), (40000, 64, 3),
                                           (32768, 64, 2), (32832, 64, 2), (32768, 32, 2)])
@pytest.mark.parametrize("counts, xdt, ydt", [([1], "bf16", "bf16"), ([5, 0, 12], "bf16", "f32"), ([3, 20], "f32", "f32"),
                                              ([2, 70], "bf16", "bf16"), ([40], "f32", "f32")])
def test_wide_layers(n, group, avg, counts, xdt, ydt):
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    E, R, m = len(counts), sum(counts), 200
    layer = U.random_layers(E, m, n, group, avg, n + R)
    x = torch.randn((R, n), generator=torch.Generator("cuda").manual_seed(R), device="cuda").to(dt[xdt])
    offsets = [sum(counts[:e]) for e in range(E + 1)]
    y = slim.slim_dequant_grouped_gemm(*layer, group, avg, x, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                                       y_dtype=dt[ydt])
    slim.slim_async_status()
    steps = group / 16 * (3 if xdt == "f32" else 1)
    U.check64(y, U.product64(layer, group, x, offsets), 3 * 2.0 ** -23 * (n // group + steps), f"{n} {counts}")
