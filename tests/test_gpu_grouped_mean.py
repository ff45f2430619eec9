"""slim_dequant_grouped_gemm on inputs of one sign or with a mean (activations behind a ReLU, for example).

Tolerance. With x of magnitude a, u = s 2^b the groups' span and v = (q - c) 2^-b, c any number within 0.1 of the range of
the zero z, a result is sum_c u (sum_j x_j v_j + (c - z) 2^-b sum_j x_j). Codes are uniform and zeros within 0.1 of the
range of its middle, so
  y's rms       Y = a u sqrt(n / 12 + k (0.058 g)^2),
  the groups' sums of x v are at most that of a group's share of y, Y when k of them are joined at random,
  the running sum of the zeros' terms is at most a u 0.058 g sqrt(k), Y at most.
The tensor core may truncate every step at 2^-23 of the running sum; a group takes g / 16 steps (three times as many
for fp32 x), the zeros' terms, eight columns a group, k / 2, and the groups join in k fp32 additions of 2^-24. With
sums up to 3 times their rms an output is off by at most
  delta = 3 * 2^-23 (k + g / 16) of Y  (fp32 x: 3 g / 16),
1.4e-5 for k = 32 and g = 128, and the norm, where sums have their rms, by a third of it. Half a step of the output
type comes on top. A factor of the zeros' terms in 16 bits would leave 1e-4 and more.
"""
import pytest
import torch

import grouped_util as U
from post_weight_quantization_hessian_b200 import slim

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["relu", "mean 1", "mean 4"])
@pytest.mark.parametrize("group, avg", [(32, 2), (64, 3), (128, 2), (128, 7), (64, 5)])
@pytest.mark.parametrize("R, xdt, ydt", [(8, "bf16", "bf16"), (32, "bf16", "bf16"), (33, "bf16", "bf16"),
                                         (300, "bf16", "bf16"), (300, "f32", "bf16"), (20, "f32", "f32"),
                                         (200, "bf16", "f32"), (200, "f32", "f32")])
def test_inputs_with_a_mean(kind, group, avg, R, xdt, ydt):
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    k, m = 32, 520
    n = k * group
    layer = U.random_layers(1, m, n, group, avg, R + group)
    x = torch.randn((R, n), generator=torch.Generator("cuda").manual_seed(R), device="cuda")
    x = (x.relu() if kind == "relu" else x + float(kind[-1])).to(dt[xdt])
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    y = slim.slim_dequant_grouped_gemm(*layer, group, avg, x, off, y_dtype=dt[ydt])
    slim.slim_async_status()
    steps = group / 16 * (3 if xdt == "f32" else 1)
    U.check64(y, U.product64(layer, group, x, [0, R]), 3 * 2.0 ** -23 * (k + steps), f"{kind} {R} {xdt} {ydt}")
