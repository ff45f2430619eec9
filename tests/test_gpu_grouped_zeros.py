"""slim_dequant_grouped_gemm where zeros lie outside or at the ends of the codes' range: groups of equal weights (the
quantizer gives them scale 1, codes 0 and the weight as minus the zero: padded outputs, pruned rows), weights of one sign.

Tolerance. With v = (q - c) 2^-b, c the zero rounded to 2^(b - 7) and met at the ends of the codes' range, a group adds
s 2^b sum x v + s (c - z) sum x. |s 2^b v| is at most the weight and r = s 2^(b - 8), and |s (c - z)| at most r or, for a zero
outside the range, the weight, so all partial sums stay below B = sum_j |x_j| (|w_j| + 2 r). (A group of equal weights has
zeros of less than 2^-8 of the range or is met at its end: r = 0 there.) The tensor core may truncate each of g / 16
steps (three times as many for fp32 x) and of the k / 2 steps of the zeros' terms by 2^-23, sums of x take 8 more, the
groups' additions k, and products and parts a few: |dy| <= 2^-23 (planes g / 16 + 2 k + 16) B, and half a step of y's type.
An output of zero weights is exactly zero."""
import pytest
import torch

import grouped_util as U
from post_weight_quantization_hessian_b200 import slim

pytestmark = pytest.mark.gpu


def repack(q, bits, group):
    """Codes [m, k, group] -> packed words [m, row words]."""
    m, k, _ = q.shape
    b = [int(v) for v in bits]
    words = torch.zeros((m, sum(b) * group // 32 + 1), dtype=torch.int64, device=q.device)
    pos = 0
    for c in range(k):
        for j in range(group):
            w, s = divmod(pos, 32)
            v = q[:, c, j].long() << s
            words[:, w] |= v & 0xFFFFFFFF
            words[:, w + 1] |= v >> 32
            pos += b[c]
    words = words[:, :-1]
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).contiguous()


def layer_with_equal_groups(m, k, group, avg, seed):
    """Outputs 0..15 zero weights, 16..31 weights 0.02, 32..47 -0.003, 48..63 another in each group, 64..95 every other
    group so, 96..127 weights of one sign, the rest as usual."""
    codes, bits, scale, zero = U.random_layers(1, m, k * group, group, avg, seed)
    q = U.codes64(codes[0], bits[0], group).view(m, k, group)
    w = torch.zeros((96, k), device="cuda")
    w[16:32], w[32:48] = 0.02, -0.003
    w[48:96] = torch.randn((48, k), generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * 0.02
    w = w.clamp(-0.1, 0.1)
    equal = torch.ones((96, k), dtype=torch.bool, device="cuda")
    equal[64:, 1::2] = False
    # a zero inside the range has to stay below 2^-8 of it for the derivation's r = 0
    w = torch.where(w < 0, w.clamp(min=-2.0 ** -8), w)
    q[:96][equal] = 0
    scale[0, :96][equal] = 1.0
    zero[0, :96][equal] = -w[equal]
    levels = 2.0 ** bits[0].float() - 1
    zero[0, 96:112], zero[0, 112:128] = -0.3 * levels, 1.4 * levels
    return [repack(q, bits[0], group)[None], bits, scale, zero], equal


@pytest.mark.parametrize("mean", [0.0, 1.0])
@pytest.mark.parametrize("group, k, avg", [(32, 20, 2), (64, 12, 3), (128, 8, 2), (128, 9, 7), (64, 16, 5)])
@pytest.mark.parametrize("R, xdt, ydt", [(1, "bf16", "f32"), (20, "f32", "f32"), (32, "bf16", "bf16"), (33, "bf16", "bf16"),
                                         (300, "bf16", "f32"), (300, "f32", "f32")])
def test_equal_weights_and_one_sign(mean, group, k, avg, R, xdt, ydt):
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    m = 200
    layer, equal = layer_with_equal_groups(m, k, group, avg, R + k)
    x = (torch.randn((R, k * group), generator=torch.Generator("cuda").manual_seed(R), device="cuda") + mean).to(dt[xdt])
    y = slim.slim_dequant_grouped_gemm(*layer, group, avg, x, torch.tensor([0, R], dtype=torch.int32, device="cuda"),
                                       y_dtype=dt[ydt])
    slim.slim_async_status()
    w = U.weights64(layer[0][0], layer[1][0], layer[2][0], layer[3][0], group)
    ref = x.double() @ w.t()
    r = layer[2][0].double() * 2.0 ** (layer[1][0].double() - 8)
    r[:96][equal] = 0
    B = x.double().abs() @ (w.abs() + 2 * r.repeat_interleave(group, 1)).t()
    tol = 2.0 ** -23 * ((3 if xdt == "f32" else 1) * group / 16 + 2 * k + 16) * B + U.half_step(ref, dt[ydt])
    err = (y.double() - ref).abs()
    print(f"of the bound {(err / tol.clamp(min=1e-300))[:, 16:].max():.3f}, rms of the errors of equal weights "
          f"{err[:, 16:64].square().mean().sqrt():.1e}, of others {err[:, 128:].square().mean().sqrt():.1e}")
    assert torch.count_nonzero(y[:, :16]) == 0
    assert torch.all(err <= tol)


@pytest.mark.parametrize("R", [3, 80])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_zero_that_is_not_finite_spoils_its_output_alone(R, bad):
    layer = U.random_layers(1, 140, 512, 64, 2, 5)
    x = torch.randn((R, 512), device="cuda")
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    want = slim.slim_dequant_grouped_gemm(*layer, 64, 2, x, off)
    layer[3][0, 70, 3] = bad
    y = slim.slim_dequant_grouped_gemm(*layer, 64, 2, x, off)
    keep = [i for i in range(140) if i != 70]
    assert torch.equal(y[:, keep], want[:, keep]) and not torch.isfinite(y[:, 70]).any()
