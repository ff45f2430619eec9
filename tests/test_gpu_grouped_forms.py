"""The many-rows kernels of slim_dequant_grouped_gemm in each of their forms: row tiles of 64, 128 and 256, CTAs that take
several tiles, several passes over the outputs, more than 32 experts. Each test states the form that its sizes take, by the
kernels' rules, so that a changed rule shows. Tolerance: the derivation of test_gpu_grouped_mean.py."""
import pytest
import torch

import grouped_util as U
from post_weight_quantization_hessian_b200 import slim

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FEW, TILE_BYTES = 32, 1 << 30


def row_tiles(counts, m):
    """(rows a tile, tiles): 256 rows, halved while the tiles fill half of the SMs at most."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = 512
    while True:
        most //= 2
        tiles = sum(-(-c // most) for c in counts if c > FEW) * (-(-m // 128))
        if most == 64 or tiles * 2 > sms:
            return most, tiles, sms


def output_tiles_of_a_pass(counts, n, group):
    boxes = -(-n // 64) + -(-(n // group) // 8)
    return TILE_BYTES // (min(len(counts), sum(counts) // (FEW + 1)) * boxes * 16384)


def run(counts, m, n, group, avg, xdt, ydt, T=0, cols=None):
    E, R = len(counts), sum(counts)
    layer = U.random_layers(E, m, n, group, avg, n + R)
    gen = torch.Generator("cuda").manual_seed(R)
    x = (torch.randn((T or R, n), generator=gen, device="cuda") + 0.5).to(DT[xdt])
    index = torch.randint(-1, T + 1, (R,), generator=gen, device="cuda", dtype=torch.int32) if T else None
    offsets = [sum(counts[:e]) for e in range(E + 1)]
    y = slim.slim_dequant_grouped_gemm(*layer, group, avg, x, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                                       row_index=index, y_dtype=DT[ydt])
    slim.slim_async_status()
    steps = group / 16 * (3 if xdt == "f32" else 1)
    ref = U.product64(layer, group, x, offsets, index, cols)
    got = y if cols is None else y[:, cols]
    U.check64(got, ref, 3 * 2.0 ** -23 * (n // group + steps), f"{counts[:4]} {m}x{n} g{group} {xdt} {ydt}")


SHAPES = [(32, 13, 2), (32, 16, 3), (64, 11, 2), (64, 12, 4), (128, 9, 2), (128, 8, 3)]


@pytest.mark.parametrize("group, k, avg", SHAPES)
@pytest.mark.parametrize("xdt, ydt, T", [("bf16", "bf16", 0), ("bf16", "f32", 500), ("f32", "bf16", 700), ("f32", "f32", 0)])
def test_tiles_of_256_rows_several_a_cta(group, k, avg, xdt, ydt, T):
    counts, m = [1000, 1111, 0, 37, 300, 5], 2500
    most, tiles, sms = row_tiles(counts, m)
    assert most == 256 and tiles > sms
    run(counts, m, k * group, group, avg, xdt, ydt, T)


@pytest.mark.parametrize("group, k, avg", SHAPES)
@pytest.mark.parametrize("xdt, ydt, T", [("bf16", "bf16", 90), ("bf16", "f32", 0), ("f32", "bf16", 0), ("f32", "f32", 100)])
def test_tiles_of_128_rows(group, k, avg, xdt, ydt, T):
    counts, m = [300, 129, 1, 90], 2000
    assert row_tiles(counts, m)[0] == 128
    run(counts, m, k * group, group, avg, xdt, ydt, T)


@pytest.mark.parametrize("group, k, avg", SHAPES)
@pytest.mark.parametrize("xdt, ydt, T", [("bf16", "bf16", 0), ("f32", "f32", 90)])
def test_tiles_of_64_rows(group, k, avg, xdt, ydt, T):
    counts, m = [70, 0, 33, 128, 3], 999
    assert row_tiles(counts, m)[0] == 64
    run(counts, m, k * group, group, avg, xdt, ydt, T)


@pytest.mark.parametrize("xdt, ydt", [("bf16", "bf16"), ("f32", "f32")])
def test_more_experts_than_a_warp_has_lanes(xdt, ydt):
    """The list of experts with many rows, and the tiles before each, go past 32."""
    counts = [33 + e % 9 if e % 5 else e % 3 for e in range(100)]
    assert sum(c > FEW for c in counts) == 80
    run(counts, 300, 512, 64, 2, xdt, ydt)


@pytest.mark.parametrize("xdt, ydt, counts", [("bf16", "bf16", [40, 50]), ("f32", "f32", [300, 2])])
def test_several_passes_over_the_outputs(xdt, ydt, counts):
    m, n, group = 20000, 16384, 128
    a_pass = output_tiles_of_a_pass(counts, n, group)
    assert a_pass < -(-m // 128) < 2 * a_pass                       # two passes, the second a shorter one
    edge = a_pass * 128
    cols = torch.cat([torch.arange(a, b) for a, b in ((0, 130), (edge - 130, edge + 130), (m - 130, m))]).cuda()
    run(counts, m, n, group, 2, xdt, ydt, cols=cols)


def test_passes_over_the_experts():
    """One output tile of each of 60 experts of 1023 + 128 boxes is past the tile budget: the experts go in two passes."""
    n, group = 65472, 64
    counts = [33 + e % 3 for e in range(60)]
    assert output_tiles_of_a_pass(counts, n, group) == 0
    assert TILE_BYTES // ((1023 + 128) * 16384) == 56
    cols = torch.cat([torch.arange(0, 20), torch.arange(120, 140)]).cuda()
    run(counts, 140, n, group, 2, "bf16", "bf16", cols=cols)
