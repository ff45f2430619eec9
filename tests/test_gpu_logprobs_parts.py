"""slim_token_logprobs counts every element of a row once: at the borders of the parts that a cluster's blocks take, of
the unaligned head and tail, and of a block's batches of loads.

Tolerance of the mean error over random rows. A result is rounded twice (its value, below 16, and the logarithm taken from
it: 2^-21 each), the exponential is off by 2^-22 of its value at most, which S and T share (T / S is off by 2^-22 of at
most 10), and the sums' 50 or so fp32 steps in a chain add sqrt(50) 2^-25 = 2e-7: 3e-6 in all. One 16-byte vector left out
or counted twice at each border of a row of 130000 changes it by 2e-4, a lost part of a batch by more.
Where only a few hundred elements are not masked, each of them is 1/300 of the sum or more, and the bound is 1e-5 and the
two roundings of the result, 2^-24 of its magnitude each (an alternative of logit -300 is about -305, where a step is
3e-5: l - max is off by half of it, and minus log S by another half)."""
import numpy as np
import pytest
import torch

from oracle import slim_oracle as O
from post_weight_quantization_hessian_b200 import slim

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def parts_of(N, V, size):
    """Blocks a row and their threads, by the launch rule."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    split = 1
    while split < 8 and N * split < 2 * sms and V * size // (2 * split) >= 32768:
        split *= 2
    return split, 128 if V * size // split <= 16384 else 256


def borders(address, V, size, split, threads):
    """Elements on both sides of every border of a row that starts at `address`."""
    vec = 16 // size
    mis = address % 16 // size
    head = min((vec - mis) % vec, V)
    nvec = (V - head) // vec
    at = {0, head - 1, head, head + nvec * vec - 1, head + nvec * vec, V - 1}
    for rank in range(split + 1):
        v = nvec * rank // split
        at |= {head + v * vec + o for o in (-vec - 1, -vec, -1, 0, vec - 1, vec)}
        if rank < split:                                     # the last, partial batch of the part, and its last round
            end = nvec * (rank + 1) // split
            batch = v + (end - v) // (4 * threads) * 4 * threads
            for w in (batch, batch + threads, batch + 2 * threads, batch + 3 * threads, v + threads, v + 32):
                at |= {head + w * vec + o for o in (-1, 0, vec - 1, vec)}
    return sorted(i for i in at if 0 <= i < V)


def rows(N, V, ld, offset, dt):
    buf = torch.zeros(N * ld + offset, dtype=DT[dt], device="cuda")
    return buf[offset:].view(N, ld)[:, :V]


SHAPES = [(3, 130000, 130000, 0), (4, 130001, 130003, 1), (2, 100003, 100003, 3), (5, 33000, 33005, 5), (300, 32001, 32001, 1),
          (2, 4097, 4099, 1), (400, 777, 779, 2), (1, 70000, 70000, 7), (2, 262144, 262144, 0), (7, 8191, 8192, 0)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rest", [-float("inf"), -300.0])
@pytest.mark.parametrize("N, V, ld, offset", SHAPES)
def test_single_elements_at_every_border(N, V, ld, offset, rest, dt):
    size = 4 if dt == "f32" else 2
    split, threads = parts_of(N, V, size)
    dev = rows(N, V, ld, offset, dt)
    dev.fill_(rest)
    g = torch.Generator().manual_seed(V)
    tokens = torch.empty(N, dtype=torch.long)
    for r in range(N):
        at = torch.tensor(borders(dev.data_ptr() + r * ld * size, V, size, split, threads))
        dev[r, at.cuda()] = torch.rand(len(at), generator=g).to(DT[dt]).cuda()
        tokens[r] = at[r % len(at)]
    k = min(32, V)
    got = slim.slim_token_logprobs(dev, tokens.cuda(), top_k=k)
    ref = O.token_logprobs(dev[:16].double().cpu().numpy(), tokens[:16].numpy(), k)
    for name, a, b in zip(("logp", "entropy", "top"), got, ref):
        a, fine = a[:16].double().cpu().numpy(), np.isfinite(b)
        assert np.array_equal(a[~fine], b[~fine])             # alternatives past the unmasked elements
        err, tol = np.abs(a[fine] - b[fine]), 1e-5 + 2.0 ** -23 * np.abs(b[fine])
        print(f"{name} split {split}: {err.max():.2e}, of its bound {(err / tol).max():.3f}")
        assert np.all(err <= tol)
    assert np.array_equal(got[3][:16].cpu().numpy(), ref[3])
    p = torch.softmax(dev.double(), 1)                       # all rows, by torch in 64 bits
    entropy = -(p * torch.log(p.clamp(min=1e-300))).sum(1)
    assert (got[1].double() - entropy).abs().max() <= 1e-5


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N, V, ld, offset", [(64, 130000, 130000, 0), (64, 130001, 130003, 1), (40, 32000, 32000, 0),
                                              (500, 50257, 50257, 0), (2000, 4097, 4099, 1), (100, 100003, 100096, 0)])
def test_mean_error_of_random_rows(N, V, ld, offset, dt):
    dev = rows(N, V, ld, offset, dt)
    gen = torch.Generator("cuda").manual_seed(N)
    dev.copy_(torch.randn((N, V), generator=gen, device="cuda") * 2.5)
    tokens = torch.randint(V, (N,), generator=gen, device="cuda")
    logp, ent, tl, ti = slim.slim_token_logprobs(dev, tokens, top_k=5)
    lp = torch.log_softmax(dev.double(), 1)
    H = -(lp.exp() * lp).sum(1)
    for name, a, b in (("logp", logp, lp.gather(1, tokens[:, None])[:, 0]), ("entropy", ent, H),
                       ("top", tl, lp.topk(5, 1)[0])):
        err = (a.double() - b).abs()
        print(f"{name}: mean {err.mean():.2e}, max {err.max():.2e}")
        assert err.mean() <= 3e-6
