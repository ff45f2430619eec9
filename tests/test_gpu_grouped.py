"""slim_dequant_grouped_gemm against the float64 oracle.

Tolerance. Per group of width b the kernels form D = sum_j x_j f_j with f_j in
[0, 2) (a code scaled by 2^-b, shifted by at most 1) and xs = sum_j x_j, then
add s 2^b D - s (2^b + z) xs (or its shifted equivalent) over the groups. With
B = sum over groups of s 2^b (3 + z 2^-b) sum_j |x_j|, a bound of all partial
sums in magnitude:
  - the tensor core's accumulation takes at most 3 g / 16 + 16 steps a group
    (fp32 x: three parts), each off by at most 2^-23 of the sum's magnitude,
  - xs in fp32 is off by at most g 2^-24 of sum |x_j|,
  - the k groups' terms are added in fp32, at most (k + 16) 2^-24 of B,
  - the three-part split of fp32 x leaves at most 2^-24 |x_j|,
so |dy| <= (3 g / 16 + 16 + g / 2 + k / 2 + 10) 2^-23 B, and half a step of the
output type, eps / 2 |y|, on top. That is the worst case of every output. Over
all outputs the errors are far smaller: a step's error is at most 2^-23 of the
running sum, which is of the order of sqrt(g) |x| s 2^b, about 7 times the
group's share of y (weights span 7 of their deviations); 24 steps that all
truncate lose half a step each on average, 12 * 7 * 2^-23 = 1e-5. So the norm of
the error is held to 2e-5 of the norm of y, plus eps / 2 for a bf16 y.
"""
import numpy as np
import pytest
import torch

from oracle import slim_oracle as O
from post_weight_quantization_hessian_b200 import slim
from post_weight_quantization_hessian_b200 import synthetic as syn

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make_layers(E, m, n, group, avg, seed, widths="sba"):
    """Random packed layers whose dequantized weights look like N(0, 0.02^2) quantized min-max; widths "sba": avg and
    its two neighbours, "wide": any of 1..8 that average to avg."""
    rng = np.random.default_rng(seed)
    k = n // group
    bits = np.empty((E, k), np.uint8)
    for e in range(E):
        b = O.allocation(rng.permutation(k), avg, k // 3)
        if widths == "wide":
            for _ in range(8 * k):
                i, j = rng.integers(k, size=2)
                if i != j and b[i] < 8 and b[j] > 1:
                    b[i] += 1
                    b[j] -= 1
        bits[e] = b
    words = rng.integers(0, 2 ** 32, (E, m, n * avg // 32), dtype=np.uint64).astype(np.uint32)
    levels = 2.0 ** bits[:, None, :].astype(np.float64) - 1
    span = rng.uniform(0.1, 0.14, (E, m, k))
    scale = (span / levels).astype(np.float32)
    zero = (rng.uniform(0.4, 0.6, (E, m, k)) * levels).astype(np.float32)
    return words, bits, scale, zero


def make_x(T, n, xdt, seed):
    x = np.random.default_rng(seed).standard_normal((T, n)).astype(np.float32)
    x[:, :: max(1, n // 3)] *= 25.0
    if xdt == "bf16":
        xb = syn.f32_to_bf16_bits(x)
        return syn.bf16_bits_to_f32(xb), torch.from_numpy(xb.view(np.int16)).cuda().view(torch.bfloat16)
    return x, torch.from_numpy(x).cuda()


def on_device(words, bits, scale, zero):
    return [torch.from_numpy(a).cuda() for a in (words.view(np.int32), bits, scale, zero)]


def bound(bits, scale, zero, group, x, offsets, row_index, ydt, ref):
    k = bits.shape[1]
    c = (3 * group / 16 + 16 + group / 2 + k / 2 + 10) * 2.0 ** -23
    R = ref.shape[0]
    B = np.zeros_like(ref)
    for e in range(len(offsets) - 1):
        r0, r1 = offsets[e], offsets[e + 1]
        at = np.arange(r0, r1) if row_index is None else np.asarray(row_index)[r0:r1]
        inside = (at >= 0) & (at < len(x))
        rows = np.where(inside[:, None], x[np.where(inside, at, 0)], 0)
        ax = np.abs(rows.astype(np.float64)).reshape(len(at), k, group).sum(2)
        p2 = 2.0 ** bits[e].astype(np.float64)
        B[r0:r1] = ax @ (scale[e] * (3 * p2 + np.abs(zero[e]))).T
    return c * B + torch.finfo(DT[ydt]).eps / 2 * np.abs(ref) + 1e-30


def check(y, ref, tol, ydt, what):
    y, got = y.float().cpu().numpy().astype(np.float64), ~np.isnan(ref)
    err = np.abs(y - ref)[got]
    norm = np.linalg.norm(err) / max(np.linalg.norm(ref[got]), 1e-30)
    print(f"{what}: max err / bound {np.max(err / tol[got]) if err.size else 0:.3f}, norm {norm:.2e}")
    assert np.all(err <= tol[got])
    assert norm <= 2e-5 + (torch.finfo(torch.bfloat16).eps / 2 if ydt == "bf16" else 0)


CASES = [
    # counts, m, n, group, avg, x, y, gathered from T rows (0: no index), widths
    ([1], 64, 32, 32, 2, "bf16", "bf16", 0, "sba"),              # the smallest: one group
    ([1], 4096, 4096, 128, 2, "bf16", "bf16", 0, "sba"),
    ([1], 33, 416, 32, 3, "f32", "f32", 0, "sba"),               # rows of 39 words: not 16-byte aligned
    ([8], 257, 1024, 64, 2, "bf16", "f32", 0, "sba"),
    ([9], 130, 1024, 128, 4, "f32", "bf16", 0, "sba"),
    ([16, 0, 1], 1003, 640, 128, 3, "bf16", "f32", 0, "sba"),    # 3-bit codes straddle words; odd width
    ([17, 3], 300, 576, 64, 3, "bf16", "bf16", 11, "sba"),
    ([0, 0, 5, 0], 128, 512, 64, 2, "f32", "f32", 0, "sba"),     # empty experts around
    ([2, 0, 1, 1, 0, 3, 1, 0], 1376, 1024, 128, 2, "bf16", "bf16", 4, "sba"),
    ([31, 33, 64, 65], 200, 768, 32, 2, "bf16", "f32", 0, "sba"),
    ([127, 129, 1], 256, 800, 32, 4, "f32", "f32", 50, "sba"),
    ([255, 257], 384, 512, 128, 3, "bf16", "bf16", 0, "sba"),
    ([300], 129, 1376, 32, 5, "bf16", "f32", 0, "sba"),
    ([5, 40, 300], 140, 1024, 64, 4, "bf16", "f32", 0, "wide"),   # any width from 1 to 8
    ([3, 70], 140, 1024, 32, 4, "f32", "f32", 0, "wide"),
    ([12, 90], 140, 1152, 128, 5, "bf16", "f32", 0, "wide"),
    ([4, 200], 72, 1152, 128, 7, "bf16", "f32", 0, "sba"),        # 6, 7 and 8 bits
    ([2, 0, 700], 513, 352, 32, 3, "f32", "bf16", 99, "sba"),
    ([1] * 40, 96, 256, 64, 2, "bf16", "bf16", 0, "sba"),         # many experts
    ([1100], 1003, 1024, 64, 2, "bf16", "bf16", 0, "sba"),        # several tiles of rows and outputs
]


@pytest.mark.parametrize("counts, m, n, group, avg, xdt, ydt, T, widths", CASES)
def test_grouped(counts, m, n, group, avg, xdt, ydt, T, widths):
    E, R = len(counts), sum(counts)
    rng = np.random.default_rng(R + m)
    layer = make_layers(E, m, n, group, avg, R + n, widths)
    x, xd = make_x(T or R, n, xdt, 5)
    index = rng.integers(0, T, R).astype(np.int32) if T else None
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = slim.slim_dequant_grouped_gemm(*on_device(*layer), group, avg, xd, torch.from_numpy(offsets).cuda(),
                                       row_index=None if index is None else torch.from_numpy(index).cuda(),
                                       y_dtype=DT[ydt])
    slim.slim_async_status()
    assert y.dtype == DT[ydt]
    ref = O.dequant_grouped_matmul(*layer, group, x, offsets, index)
    check(y, ref, bound(*layer[1:], group, x, offsets, index, ydt, ref), ydt, f"{counts} {m}x{n} g{group}")


@pytest.mark.parametrize("counts, first, pad", [([3, 0, 2], 2, 3), ([30, 0, 50], 7, 40), ([300, 20], 1, 1)])
@pytest.mark.parametrize("gather", [False, True])
def test_rows_of_no_expert_are_left_alone_and_bad_indices_read_zeros(counts, first, pad, gather):
    """Rows before offsets[0] and behind offsets[E] keep their contents; an index outside x reads zeros."""
    m, n, group, avg = 150, 512, 64, 2
    E, R = len(counts), first + sum(counts) + pad
    layer = make_layers(E, m, n, group, avg, 3)
    x, xd = make_x(R, n, "bf16", 6)
    offsets = (first + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    index = None
    if gather:
        index = np.random.default_rng(1).integers(0, R, R).astype(np.int32)
        index[first], index[first + 1] = -1, 2 ** 31 - 1
        index[first + 2] = R
    y = torch.full((R, m), 7.0, device="cuda")
    slim.slim_dequant_grouped_gemm(*on_device(*layer), group, avg, xd, torch.from_numpy(offsets).cuda(),
                                   row_index=None if index is None else torch.from_numpy(index).cuda(), y=y)
    ref = O.dequant_grouped_matmul(*layer, group, x, offsets, index)
    check(y, ref, bound(*layer[1:], group, x, offsets, index, "f32", ref), "f32", f"{counts} from {first}")
    assert torch.equal(y[:first], torch.full_like(y[:first], 7.0))
    assert torch.equal(y[R - pad:], torch.full_like(y[R - pad:], 7.0))
    if gather:
        assert torch.count_nonzero(y[first:first + 3]) == 0


@pytest.mark.parametrize("R", [6, 60, 600])
def test_offsets_outside_the_rows_are_clamped(R):
    """Offsets past R stop at R: nothing outside x and y is read or written."""
    m, n = 130, 256
    layer = make_layers(2, m, n, 64, 2, 4)
    x, xd = make_x(R, n, "bf16", 7)
    buf = torch.full((R + 8, m), 7.0, device="cuda")
    slim.slim_dequant_grouped_gemm(*on_device(*layer), 64, 2, xd,
                                   torch.tensor([-5, 4, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), y=buf[:R])
    offsets = [0, 4, R]
    ref = O.dequant_grouped_matmul(*layer, 64, x, offsets)
    check(buf[:R], ref, bound(*layer[1:], 64, x, offsets, None, "f32", ref), "f32", "clamped")
    assert torch.equal(buf[R:], torch.full_like(buf[R:], 7.0))


@pytest.mark.parametrize("R", [3, 20, 300])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_a_row_with_infinity_or_nan_spoils_no_other(R, xdt):
    m, n = 70, 512
    layer = make_layers(1, m, n, 128, 2, 8)
    x, xd = make_x(R, n, xdt, 9)
    dev = on_device(*layer)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    clean = slim.slim_dequant_grouped_gemm(*dev, 128, 2, xd, off)
    bad = xd.clone()
    bad[1, 5] = float("nan")
    bad[1, 300] = float("inf")
    y = slim.slim_dequant_grouped_gemm(*dev, 128, 2, bad, off)
    keep = [r for r in range(R) if r != 1]
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[1]).any()


@pytest.mark.parametrize("R", [5, 333])
def test_invalid_widths_read_nothing_outside(R):
    """Widths outside 1..8 or that do not fill a row leave that expert's y unspecified and the others right."""
    m, n = 130, 512
    layer = list(make_layers(2, m, n, 128, 2, 10))
    x, xd = make_x(2 * R, n, "bf16", 11)
    good = layer[1].copy()
    layer[1][0] = [0, 255, 8, 8]
    y = slim.slim_dequant_grouped_gemm(*on_device(*layer), 128, 2, xd,
                                       torch.tensor([0, R, 2 * R], dtype=torch.int32, device="cuda"),
                                       y_dtype=torch.float32)
    layer[1] = good
    offsets = [0, R, 2 * R]
    ref = O.dequant_grouped_matmul(*layer, 128, x, offsets)
    tol = bound(*layer[1:], 128, x, offsets, None, "f32", ref)
    check(y[R:], ref[R:], tol[R:], "f32", "the other expert")


@pytest.mark.parametrize("counts", [[1], [3, 0, 9], [40, 0, 100], [600, 1]])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_captured_replayed_and_repeated(counts, xdt):
    """Calls repeat bit for bit; a captured call replays on new inputs and new counts, with an eager call in between and
    a second graph of the same operator beside it."""
    m, n, group, avg = 260, 768, 64, 2
    E, R = len(counts), sum(counts)
    dev = on_device(*make_layers(E, m, n, group, avg, 12))
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    off2 = off.clone()
    off2[1:E] = off[E]                      # every row to the first expert
    xs = [make_x(R, n, xdt, s)[1] for s in (1, 2)]
    want = [slim.slim_dequant_grouped_gemm(*dev, group, avg, a, o) for a, o in ((xs[0], off), (xs[1], off2))]
    again = slim.slim_dequant_grouped_gemm(*dev, group, avg, xs[0], off)
    assert torch.equal(again, want[0])
    x, o = xs[0].clone(), off.clone()
    x2 = xs[1].clone()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a, b in ((x, o), (x2, off2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(slim.slim_dequant_grouped_gemm(*dev, group, avg, a, b))
        graphs.append(g)
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
        eager = slim.slim_dequant_grouped_gemm(*dev, group, avg, xs[0], off)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[0])
    x.copy_(xs[1])
    o.copy_(off2)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1])


@pytest.mark.parametrize("R", [4, 500])
def test_another_stream_and_a_caller_workspace(R):
    m, n = 300, 512
    dev = on_device(*make_layers(1, m, n, 128, 2, 13))
    _, x = make_x(R, n, "f32", 14)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    want = slim.slim_dequant_grouped_gemm(*dev, 128, 2, x, off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    need = slim._lib().slim_dequant_grouped_gemm_workspace_bytes(1, m, n, 128, 2, 0, 0, R)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    y1 = slim.slim_dequant_grouped_gemm(*dev, 128, 2, x, off, stream=s)
    y2 = slim.slim_dequant_grouped_gemm(*dev, 128, 2, x, off, ws=ws, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y1, want) and torch.equal(y2, want)
    # the C entry's own workspace
    y3 = torch.empty_like(want)
    rc = slim._lib().slim_dequant_grouped_gemm(*[t.data_ptr() for t in dev], 1, m, n, 128, 2, x.data_ptr(), 0, R, None,
                                               off.data_ptr(), R, y3.data_ptr(), 0, None, 0,
                                               torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(y3, want)
    if need:
        with pytest.raises(slim.SlimError):
            slim.slim_dequant_grouped_gemm(*dev, 128, 2, x, off, ws=ws[: need - 256])
        with pytest.raises(slim.SlimError):
            slim.slim_dequant_grouped_gemm(*dev, 128, 2, x, off, ws=torch.empty(need + 512, dtype=torch.uint8,
                                                                                device="cuda")[16:])


def test_two_calls_at_once():
    """Two streams, each with its own buffers."""
    m, n = 512, 1024
    dev = on_device(*make_layers(2, m, n, 64, 2, 15))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for R in (6, 400):
        xs = [make_x(R, n, "bf16", s)[1] for s in (1, 2)]
        off = torch.tensor([0, R // 3, R], dtype=torch.int32, device="cuda")
        want = [slim.slim_dequant_grouped_gemm(*dev, 64, 2, x, off) for x in xs]
        torch.cuda.synchronize()
        got = [[slim.slim_dequant_grouped_gemm(*dev, 64, 2, x, off, stream=s) for _ in range(10)]
               for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for ys, w in zip(got, want) for y in ys)


@pytest.mark.parametrize("R, m", [(40000, 65536), (3, 1 << 20)])
def test_offsets_past_32_bits(R, m):
    """y of more than 2^31 values, and codes and scales of a very wide layer; sampled rows and outputs checked."""
    n, group, avg = 32, 32, 2
    words, bits, scale, zero = make_layers(1, m, n, group, avg, 16)
    x, xd = make_x(R, n, "bf16", 17)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    y = slim.slim_dequant_grouped_gemm(*on_device(words, bits, scale, zero), group, avg, xd, off)
    slim.slim_async_status()
    rows = np.unique(np.concatenate([[0, R - 1], np.random.default_rng(0).integers(0, R, 20)]))
    cols = np.unique(np.concatenate([[0, m - 1], np.random.default_rng(1).integers(0, m, 200)]))
    got = y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()]
    sub = (words[:, cols], bits, scale[:, cols], zero[:, cols])
    ref = O.dequant_grouped_matmul(*sub, group, x[rows], [0, len(rows)])
    check(got, ref, bound(*sub[1:], group, x[rows], [0, len(rows)], None, "bf16", ref), "bf16", "sampled")


def test_agrees_with_the_gemv():
    """One expert and up to 8 rows is slim_dequant_gemv's product: both within their bounds of the oracle, so of each other."""
    words, bits, scale, zero = make_layers(1, 300, 1024, 128, 2, 18)
    x, xd = make_x(5, 1024, "f32", 19)
    dev = on_device(words, bits, scale, zero)
    a = slim.slim_dequant_gemv(*[t[0] for t in dev], 128, 2, xd)
    b = slim.slim_dequant_grouped_gemm(*dev, 128, 2, xd, torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
    tol = bound(bits, scale, zero, 128, x, [0, 5], None, "f32", a.cpu().numpy().astype(np.float64))
    assert np.all((a - b).abs().cpu().numpy() <= 2 * tol)


def test_injected_failure(monkeypatch):
    dev = on_device(*make_layers(1, 64, 256, 64, 2, 20))
    _, x = make_x(2, 256, "f32", 21)
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    monkeypatch.setenv("SLIM_FAULT", "dequant_grouped_gemm")
    with pytest.raises(slim.SlimError) as e:
        slim.slim_dequant_grouped_gemm(*dev, 64, 2, x, off)
    assert e.value.status == 7


def test_no_rows():
    dev = on_device(*make_layers(2, 64, 256, 64, 2, 20))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = slim.slim_dequant_grouped_gemm(*dev, 64, 2, torch.zeros((0, 256), device="cuda"), off)
    assert y.shape == (0, 64)
    y = torch.full((70, 64), 7.0, device="cuda")                 # rows, but none of an expert
    slim.slim_dequant_grouped_gemm(*dev, 64, 2, torch.zeros((70, 256), device="cuda"), off, y=y)
    assert torch.equal(y, torch.full_like(y, 7.0))


def test_offsets_that_descend_stay_inside():
    """Offsets out of order give unspecified rows, but nothing outside y is written and the device stays usable."""
    E, m, n, R = 9, 130, 256, 150
    layer = make_layers(E, m, n, 64, 2, 22)
    x, xd = make_x(R, n, "bf16", 23)
    buf = torch.full((R + 8, m), 7.0, device="cuda")
    off = torch.tensor([0, R, 0, R, 0, R, 0, R, 0, R], dtype=torch.int32, device="cuda")
    slim.slim_dequant_grouped_gemm(*on_device(*layer), 64, 2, xd, off, y=buf[:R])
    slim.slim_async_status()
    assert torch.equal(buf[R:], torch.full_like(buf[R:], 7.0))
