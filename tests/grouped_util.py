"""Packed layers and their products in 64 bits, vectorized on any device, for layers too large for the
oracle's bit by bit unpacking (pinned against it in test_grouped_util.py)."""
import torch

MEAN = 0.1   # of the codes' range: how far zeros lie from its middle at most


def codes64(words, bits, group):
    """Packed words [m, row words] (int32) of widths bits [k] -> codes [m, k * group] as int64."""
    dev = words.device
    b = torch.as_tensor(bits, dtype=torch.int64, device=dev)
    start = (torch.cumsum(b, 0) - b) * group
    j = torch.arange(group, device=dev)
    at = (start[:, None] + j * b[:, None]).flatten()
    width = b.repeat_interleave(group)
    wide = torch.nn.functional.pad(words.long() & 0xFFFFFFFF, (0, 1))
    pair = wide[:, at >> 5] | wide[:, (at >> 5) + 1] << 32
    return (pair >> (at & 31)) & ((1 << width) - 1)


def weights64(words, bits, scale, zero, group):
    q = codes64(words, bits, group).double()
    return scale.double().repeat_interleave(group, 1) * (q - zero.double().repeat_interleave(group, 1))


def product64(layer, group, x, offsets, index=None, cols=None):
    """float64 [R, outputs]; layer = codes, bits, scale, zero of E experts; cols: outputs, all by default. Rows of no
    expert are NaN, an index outside x reads zeros."""
    codes, bits, scale, zero = layer
    R = x.shape[0] if index is None else index.numel()
    m = scale.shape[1]
    cols = torch.arange(m, device=x.device) if cols is None else cols
    y = torch.full((R, cols.numel()), float("nan"), dtype=torch.float64, device=x.device)
    for e in range(len(offsets) - 1):
        r0, r1 = (min(max(int(v), 0), R) for v in offsets[e:e + 2])
        if r1 <= r0:
            continue
        if index is None:
            rows = x[r0:r1].double()
        else:
            at = index[r0:r1].long()
            inside = (at >= 0) & (at < x.shape[0])
            rows = torch.where(inside[:, None], x[torch.where(inside, at, 0)].double(), 0.0)
        for c0 in range(0, cols.numel(), 256):
            c = cols[c0:c0 + 256]
            w = weights64(codes[e][c], bits[e], scale[e][c], zero[e][c], group)
            y[r0:r1, c0:c0 + 256] = rows @ w.t()
    return y


def random_bits(k, avg, gen):
    """SBA's widths: avg, and its two neighbours equally often."""
    b = torch.full((k,), avg, dtype=torch.uint8)
    order = torch.randperm(k, generator=gen)
    p = k // 3
    b[order[:p]] += 1
    b[order[k - p:]] -= 1
    return b


def random_layers(E, m, n, group, avg, seed, device="cuda"):
    """E packed layers: uniform codes over a span of 0.1 to 0.14, zeros within 0.1 of the range around its middle."""
    host, gen = torch.Generator().manual_seed(seed), torch.Generator(device).manual_seed(seed)
    k = n // group
    bits = torch.stack([random_bits(k, avg, host) for _ in range(E)]).to(device)
    codes = torch.randint(-2 ** 31, 2 ** 31, (E, m, n * avg // 32), dtype=torch.int32, generator=gen, device=device)
    levels = (2.0 ** bits.float() - 1)[:, None, :]
    scale = (0.1 + 0.04 * torch.rand((E, m, k), generator=gen, device=device)) / levels
    zero = (0.5 + MEAN * (2 * torch.rand((E, m, k), generator=gen, device=device) - 1)) * levels
    return [codes, bits, scale, zero]


def half_step(ref, dtype):
    """Half the distance between the values of dtype around ref, for normal numbers."""
    t = torch.finfo(dtype)
    exp = torch.floor(torch.log2(ref.abs().clamp(min=float(t.tiny))))
    return torch.exp2(exp) * t.eps / 2


def check64(y, ref, delta, what=""):
    """Each |y - ref| within half a step of y's type and delta of its row's rms; fp32 also in the norm, a third of it."""
    rows = ~torch.isnan(ref[:, 0])
    y, ref, dtype = y[rows].double(), ref[rows], y.dtype
    rms = ref.square().mean(1, keepdim=True).sqrt()
    err = (y - ref).abs()
    over = ((err - half_step(ref, dtype)) / rms.clamp(min=1e-30)).max().item()
    norm = (err.norm() / ref.norm()).item()
    print(f"{what}: beyond half a step {over:.2e} of rms (allowed {delta:.2e}), norm {norm:.2e}")
    assert over <= delta
    if dtype == torch.float32:
        assert norm <= delta / 3
