"""slim_token_logprobs against the float64 oracle.

Tolerance. d = l - max is exact or rounded once (2^-24 |d|), its exponential
takes d log2(e) rounded (2^-24 |d| 1.45, times the exponential's own slope of 1)
and ex2's error of 2^-22; S = sum exp(d) is a fixed tree of fp32 sums, at most
V / 256 + 32 terms long in any chain, so log S is off by at most
c = (V / 256 + 40) 2^-24 + 2^-22 relative of S, plus the terms' own errors
weighted by p, 2.5 sum p |d| 2^-24. logp = d - log S adds 2^-23 (|d| + |log S|).
The entropy log S - sum p d adds the same relative errors of sum p |d|. With
H <= log V and sum p |d| <= H + log S <= 2 log V, |dlogp| and |dH| are below
  2 c (1 + 2 log V) + 8 log V 2^-24 + 2^-23 |logp|.
top_id has to be equal: it is decided on the logits as they are.
"""
import numpy as np
import pytest
import torch

from oracle import slim_oracle as O
from post_weight_quantization_hessian_b200 import slim

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def tolerance(V, ref):
    c = (V / 256 + 40) * 2.0 ** -24 + 2.0 ** -22
    return 2 * c * (1 + 2 * np.log(V)) + 8 * np.log(V) * 2.0 ** -24 + 1e-7 + 2.0 ** -23 * np.abs(ref)


def make(N, V, dt, seed, spread=2.5, ld=None, offset=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((N, V), generator=g) * spread
    l.scatter_add_(1, torch.randint(V, (N, min(4, V)), generator=g), torch.rand((N, min(4, V)), generator=g) * 12)
    buf = torch.zeros(N * (ld or V) + offset, dtype=DT[dt])
    view = buf[offset:].view(N, ld or V)[:, :V]
    view.copy_(l)
    dev = buf.cuda()[offset:].view(N, ld or V)[:, :V]
    return view.double().numpy(), dev, torch.randint(V, (N,), generator=g)


def close(got, ref, V, what):
    got = got.double().cpu().numpy()
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(got)) and np.array_equal(np.isnan(ref), np.isnan(got)), what
    assert np.array_equal(ref[np.isinf(ref)], got[np.isinf(ref)]), what
    err, tol = np.abs(got[fine] - ref[fine]), tolerance(V, ref[fine])
    if err.size:
        print(f"{what}: max err / bound {np.max(err / tol):.3f}")
        assert np.all(err <= tol), what


def check(l, dev, tokens, top_k, what=""):
    V = l.shape[1]
    logp, ent, tl, ti = slim.slim_token_logprobs(dev, None if tokens is None else tokens.cuda(), top_k=top_k)
    rl, re, rtl, rti = O.token_logprobs(l, None if tokens is None else tokens.numpy(), top_k)
    close(ent, re, V, what + "entropy")
    assert (logp is None) == (tokens is None) and (tl is None) == (ti is None) == (top_k == 0)
    if tokens is not None:
        close(logp, rl, V, what + "logp")
    if top_k:
        assert np.array_equal(ti.cpu().numpy(), rti), what
        close(tl, rtl, V, what + "top")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N, V, top_k", [
    (1, 1, 1), (3, 2, 2), (2, 31, 31), (5, 33, 32), (1, 255, 20), (7, 1000, 5), (1, 4097, 32), (1, 32000, 20),
    (2, 50257, 1), (1, 151937, 32), (300, 777, 8), (40, 32000, 0), (1000, 4096, 3), (2000, 130, 4), (17, 100003, 7),
])
def test_logprobs(N, V, top_k, dt):
    l, dev, tokens = make(N, V, dt, N + V)
    check(l, dev, tokens, top_k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V, ld, offset", [(1001, 1008, 0), (1000, 1003, 1), (33000, 33005, 3), (130000, 130001, 7), (8, 9, 1)])
def test_strided_and_unaligned_rows(V, ld, offset, dt):
    l, dev, tokens = make(6, V, dt, 3, ld=ld, offset=offset)
    check(l, dev, tokens, min(6, V))


@pytest.mark.parametrize("N", [2, 400])
def test_tokens_that_are_none(N):
    l, dev, tokens = make(N, 500, "f32", 4)
    tokens[0], tokens[1] = -100, 500
    check(l, dev, tokens, 2)
    tokens[0], tokens[1] = 2 ** 40, -2 ** 62
    check(l, dev, tokens, 0)
    check(l, dev, None, 3)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [5, 700])
@pytest.mark.parametrize("V", [100, 5000, 40000])
def test_masks(N, V, dt):
    """-infinity on part of a row, all but one, all; the type's lowest value in their place."""
    l, dev, tokens = make(N, V, dt, 5)
    for fill in (-np.inf, float(torch.finfo(DT[dt]).min)):
        d, want = dev.clone(), l.copy()
        d[0, : V // 2], want[0, : V // 2] = fill, fill
        d[1], want[1] = fill, fill
        d[2], want[2] = fill, fill
        d[2, V - 1], want[2, V - 1] = 3.0, 3.0
        d[3, 1:], want[3, 1:] = fill, fill
        if np.isfinite(fill):                                     # the type's lowest and highest in one row
            d[4, ::2], want[4, ::2], d[4, 1], want[4, 1] = -fill, -fill, fill, fill
        check(want, d, tokens, 8, f"fill {fill}: ")


@pytest.mark.parametrize("N", [3, 600])
@pytest.mark.parametrize("V", [64, 3000, 70000])
def test_nan_and_infinity(N, V):
    l, dev, tokens = make(N, V, "f32", 6)
    for row, at, v in ((0, V // 2, np.inf), (1, V - 1, np.nan), (2, 0, np.nan), (2, 7, np.inf), (2, 9, -np.inf)):
        l[row, at] = v
        dev[row, at] = float(v)
    check(l, dev, tokens, 5)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 2000, 33333, 128000])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "steps", "zeros", "one lane", "block"])
def test_ties_and_orders(V, kind, dt):
    """Ties rank by index; orders that put the largest values of a row into few threads' hands."""
    v = torch.arange(V, dtype=torch.float64)
    rows = {"equal": torch.full((V,), 2.5), "ascending": v * (20.0 / V), "descending": -v * (20.0 / V),
            "steps": torch.floor(v * 7 / V), "zeros": torch.where(v % 2 == 0, 0.0, -0.0),
            "one lane": torch.where((v // 8) % 32 == 3, 5.0 + (v % 5) * 0.25, 0.0),
            "block": torch.where((v >= V // 2) & (v < V // 2 + 1500), 9.0, 1.0)}
    for N in (1, 500):
        l = rows[kind].to(DT[dt]).expand(N, V).contiguous()
        check(l.double().numpy()[:1].repeat(min(N, 2), 0), l.cuda()[:min(N, 2)], torch.zeros(min(N, 2), dtype=torch.long), 32)
        if N > 2:
            one = slim.slim_token_logprobs(l[:1].cuda(), top_k=32)
            many = slim.slim_token_logprobs(l.cuda(), top_k=32)
            assert torch.equal(many[3], one[3].expand(N, 32))


def test_large_magnitudes():
    """Differences of large logits stay exact: a common offset changes nothing but its rounding."""
    l, dev, tokens = make(4, 3000, "f32", 7)
    far = (dev + 4096.0)
    check(far.double().cpu().numpy(), far, tokens, 4)
    big = (dev * 1e4)
    check(big.double().cpu().numpy(), big, tokens, 4)


def test_outputs_alone():
    """Each output by itself through the C entry."""
    l, dev, tokens = make(9, 3001, "bf16", 8)
    lib, t = slim._lib(), tokens.cuda()
    full = slim.slim_token_logprobs(dev, t, top_k=3)
    s = torch.cuda.current_stream().cuda_stream
    a, b = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    c, d = torch.empty((9, 3), device="cuda"), torch.empty((9, 3), dtype=torch.int32, device="cuda")
    assert lib.slim_token_logprobs(dev.data_ptr(), 1, 9, 3001, 3001, t.data_ptr(), 0, a.data_ptr(), None, None, None, s) == 0
    assert lib.slim_token_logprobs(dev.data_ptr(), 1, 9, 3001, 3001, None, 0, None, b.data_ptr(), None, None, s) == 0
    assert lib.slim_token_logprobs(dev.data_ptr(), 1, 9, 3001, 3001, None, 3, None, None, c.data_ptr(), d.data_ptr(), s) == 0
    torch.cuda.synchronize()
    assert torch.equal(a, full[0]) and torch.equal(b, full[1]) and torch.equal(c, full[2]) and torch.equal(d, full[3])


@pytest.mark.parametrize("N, V", [(1, 32000), (600, 3001)])
def test_captured_repeated_and_on_another_stream(N, V):
    l, dev, tokens = make(N, V, "bf16", 9)
    t = tokens.cuda()
    want = slim.slim_token_logprobs(dev, t, top_k=4)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = slim.slim_token_logprobs(dev, t, top_k=4)
    for _ in range(3):
        for o in got:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    other = slim.slim_token_logprobs(dev, t, top_k=4, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last rows are read where they are."""
    N, V = 17000, 130000
    dev = torch.zeros((N, V), dtype=torch.bfloat16, device="cuda")
    l, rows, tokens = make(3, V, "bf16", 10)
    dev[N - 3:] = rows
    got = slim.slim_token_logprobs(dev, torch.cat([torch.zeros(N - 3, dtype=torch.long), tokens]).cuda(), top_k=5)
    ref = O.token_logprobs(l, tokens.numpy(), 5)
    for a, b, what in zip(got, ref, ("logp", "entropy", "top", "ids")):
        if what == "ids":
            assert np.array_equal(a[N - 3:].cpu().numpy(), b)
        else:
            close(a[N - 3:], b, V, what)
    assert abs(got[1][0].item() - np.log(V)) < 1e-4 and got[3][5].tolist() == [0, 1, 2, 3, 4]


def test_empty_batch():
    out = slim.slim_token_logprobs(torch.zeros((0, 50), device="cuda"), torch.zeros(0, dtype=torch.long, device="cuda"), top_k=3)
    assert [tuple(t.shape) for t in out] == [(0,), (0,), (0, 3), (0, 3)]


@pytest.mark.parametrize("V", [300, 60000])
@pytest.mark.parametrize("left", [0, 1, 3, 31])
def test_fewer_unmasked_logits_than_alternatives(V, left):
    """Constrained decoding: few logits are left; the masked ones follow by index."""
    for N in (1, 400):
        g = torch.Generator().manual_seed(left + V)
        l = torch.full((N, V), -float("inf"))
        for r in range(N):
            l[r, torch.randperm(V, generator=g)[:left]] = torch.randn(left, generator=g)
        check(l.double().numpy()[:3], l.cuda()[:3], torch.zeros(min(N, 3), dtype=torch.long), 32)
        one = slim.slim_token_logprobs(l[-1:].cuda(), top_k=32)
        many = slim.slim_token_logprobs(l.cuda(), top_k=32)
        assert torch.equal(many[3][-1:], one[3])
