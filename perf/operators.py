"""Performance cases of the operators that serve and judge a quantized model.

slim_dequant_grouped_gemm: products of ragged groups of rows with packed
mixed-width layers, one layer per expert (one expert: a plain layer).
slim_token_logprobs: log probabilities of given tokens, the entropy of the
distribution and its top alternatives, from logits.

`own` selects the framework's calls; otherwise run() computes the same in
elementary torch operations in 32 bits.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one token through one 2-bit attention projection: decode latency
        gemm_case("gemm_one_token", "1", 4096, 4096, 128, 2, BF16, BF16),
        # four tokens, two experts each, through the up projections of a mixture: the x rows are gathered
        gemm_case("gemm_few_tokens_experts", "2,0,1,1,0,3,1,0", 11008, 4096, 128, 2, BF16, BF16, tokens=4),
        # a few fp32 rows on small groups (three widths, scales a large part of the bytes)
        gemm_case("gemm_few_rows_f32_g32", "1,2,0,2", 13824, 5120, 32, 2, F32, F32),
        # a decode batch over experts, uneven, one expert idle, rows for padding behind the last expert
        gemm_case("gemm_batch_ragged", "5,31,0,17,64,9,1,33", 4096, 11008, 128, 3, BF16, BF16, pad=16),
        # odd output width, 4-bit average, fp32 in and out: a scoring run of a layer in fp32
        gemm_case("gemm_odd_f32", "257,0,519", 1003, 5120, 32, 4, F32, F32),
        # the prompt of one sequence chunk through one projection
        gemm_case("gemm_prompt_dense", "4096", 4096, 4096, 128, 2, BF16, BF16),
        # the prompt's chunk through eight experts, two for each token, uneven: the largest
        gemm_case("gemm_prompt_experts", "1311,702,1,2040,955,1187,480,1516", 11008, 4096, 64, 2, BF16, BF16,
                  tokens=4096),
        # one position of one sequence: sampling's report of 20 alternatives
        logp_case("logp_one_row", 1, 32000, 32000, BF16, 20),
        # a decode batch on a large vocabulary in fp32, part of it masked, one row fully
        logp_case("logp_batch_masked_f32", 64, 128000, 128000, F32, 5, masked=True),
        # scoring a chunk of text: log probability, entropy and the best token
        logp_case("logp_chunk", 4096, 32000, 32000, BF16, 1),
        # padded rows of an odd vocabulary in fp32 with alternatives
        logp_case("logp_padded_f32", 1024, 100003, 100096, F32, 8),
        # odd vocabulary, unaligned bf16 rows, no alternatives: perplexity of a long text
        logp_case("logp_unaligned", 8191, 50257, 50257, BF16, 0),
    ]


def gemm_case(name, rows, m, n, group, avg_bits, xtype, ytype, tokens=0, pad=0):
    """rows: the experts' row counts; tokens > 0: x has that many rows and the grouped rows are gathered from
    them; pad: rows of y behind the last expert's, left as they are."""
    c = {"op": "gemm", "rows": rows, "m": m, "n": n, "group": group, "avg_bits": avg_bits, "x": xtype, "y": ytype,
         "tokens": tokens, "pad": pad}
    return c if name is None else {"name": name, **c}


def logp_case(name, rows, vocab, ld, xtype, top_k, masked=False):
    c = {"op": "logp", "rows": rows, "vocab": vocab, "ld": ld, "x": xtype, "top_k": top_k, "masked": masked}
    return c if name is None else {"name": name, **c}


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.55:
        while True:
            experts = rng.choice([1, 1, 2, 3, 4, 8, 16])
            group = rng.choice([32, 64, 128])
            m, n = log_int(rng, 100, 14000), group * max(1, log_int(rng, 256, 11264) // group)
            total = log_int(rng, 1, 8192)
            weights = [rng.random() ** 2 for _ in range(experts)]
            counts = [int(total * w / sum(weights)) for w in weights]
            counts[rng.randrange(experts)] += total - sum(counts)
            xtype = rng.choice([BF16, BF16, F32])
            cost = 2.0 * total * m * n * (1 if xtype == BF16 else 3)
            if cost <= 7e11 and experts * m * n <= 3.6e8:
                break
        tokens = max(1, total // 2) if rng.random() < 0.4 else 0
        return gemm_case(None, ",".join(map(str, counts)), m, n, group, rng.choice([2, 2, 3, 4]), xtype,
                         rng.choice([BF16, F32]), tokens, rng.choice([0, 0, 5]))
    while True:
        rows, vocab = log_int(rng, 1, 8192), log_int(rng, 500, 152000)
        if rows * vocab <= 2e8:
            break
    ld = rng.choice([vocab, vocab, (vocab + 63) // 64 * 64])
    return logp_case(None, rows, vocab, ld, rng.choice([BF16, F32]), rng.choice([0, 1, 5, 20, 32]),
                     rng.random() < 0.3)


def counts_of(case):
    return [int(v) for v in case["rows"].split(",")]


# ------------------------------------------------------------------ inputs
def pack_width(codes, b):
    """Codes [m, groups, group] of b bits each -> little-endian int32 words [m, groups, group * b / 32]."""
    m, ng, g = codes.shape
    u = codes.to(torch.int64).view(m, ng, g // 32, 32)
    words = torch.zeros((m, ng, g // 32, b + 1), dtype=torch.int64, device=codes.device)
    for t in range(32):
        lo, sh = t * b // 32, t * b % 32
        v = u[..., t] << sh
        words[..., lo] |= v & 0xFFFFFFFF
        words[..., lo + 1] |= v >> 32
    words = words[..., :b]
    words = torch.where(words >= 1 << 31, words - (1 << 32), words)
    return words.to(torch.int32).reshape(m, ng, g * b // 32)


def quantize(case, gen, dev):
    """One layer of random weights with a few salient columns, min-max quantized at the given widths and packed."""
    m, n, g, avg = case["m"], case["n"], case["group"], case["avg_bits"]
    k = n // g
    p = k // 4
    order = torch.randperm(k, generator=gen)
    bits = torch.full((k,), avg, dtype=torch.int64)
    bits[order[:p]] += 1
    bits[order[k - p:]] -= 1
    w = torch.randn((m, n), generator=torch.Generator(dev).manual_seed(int(torch.randint(1 << 40, (1,), generator=gen))),
                    device=dev) * 0.02
    w[:, torch.randperm(n, generator=gen)[: max(1, n // 512)].to(dev)] *= 6.0
    w = w.view(m, k, g)
    lo, hi = w.amin(2), w.amax(2)
    levels = ((1 << bits) - 1).to(dev)
    scale = (hi - lo) / levels
    zero = -lo / scale
    first = (torch.cumsum(bits, 0) - bits) * (g // 32)
    words = torch.empty((m, n * avg // 32), dtype=torch.int32, device=dev)
    for b in sorted(set(bits.tolist())):
        at = torch.nonzero(bits == b).flatten()
        d = at.to(dev)
        q = torch.round(w[:, d] / scale[:, d, None] + zero[:, d, None]).clamp_(0, (1 << b) - 1).to(torch.int32)
        cols = (first[at][:, None] + torch.arange(g * b // 32)).flatten().to(dev)
        words[:, cols] = pack_width(q, b).flatten(1)
    return words, bits.to(torch.uint8).to(dev), scale, zero


def activations(rows, n, dtype, gen, dev):
    x = torch.randn((rows, n), generator=gen, device=dev)
    x[:, torch.randperm(n, generator=gen, device=dev)[: max(1, n // 512)]] *= 25.0
    return x.to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    host, gen = torch.Generator().manual_seed(seed), torch.Generator(dev).manual_seed(seed)
    if case["op"] == "gemm":
        counts = counts_of(case)
        rows = sum(counts)
        layers = [quantize(case, host, dev) for _ in counts]
        codes, bits, scale, zero = (torch.stack(v) for v in zip(*layers))
        x = activations(case["tokens"] or rows, case["n"], DTYPE[case["x"]], gen, dev)
        index = None
        if case["tokens"]:
            index = torch.randint(case["tokens"], (rows,), generator=gen, device=dev, dtype=torch.int32)
        ends = torch.cumsum(torch.tensor([0] + counts), 0)
        y = torch.zeros((rows + case["pad"], case["m"]), dtype=DTYPE[case["y"]], device=dev)
        if index is not None and case["pad"]:
            index = torch.cat([index, index.new_zeros(case["pad"])])
        if index is None and case["pad"]:
            x = torch.cat([x, x.new_zeros((case["pad"], case["n"]))])
        return {"case": case, "codes": codes, "bits": bits, "scale": scale, "zero": zero, "x": x, "row_index": index,
                "offsets": ends.to(torch.int32).to(dev), "ends": ends.tolist(), "widths": bits.tolist(), "y": y}
    rows, vocab = case["rows"], case["vocab"]
    logits = torch.randn((rows, case["ld"]), generator=gen, device=dev) * 2.5
    spikes = torch.randint(vocab, (rows, 4), generator=gen, device=dev)
    logits.scatter_add_(1, spikes, torch.rand((rows, 4), generator=gen, device=dev) * 12.0)
    tokens = torch.randint(vocab, (rows,), generator=gen, device=dev)
    tokens = torch.where(torch.rand(rows, generator=gen, device=dev) < 0.5, spikes[:, 0], tokens)
    if case["masked"]:
        gone = torch.rand(vocab, generator=gen, device=dev) < 0.06
        logits[:, :vocab].masked_fill_(gone, -math.inf)
        if rows > 1:
            logits[rows - 1] = -math.inf
    if rows > 8:
        tokens[rows // 3] = -100  # a position without a given token
    return {"case": case, "logits": logits.to(DTYPE[case["x"]])[:, :vocab], "tokens": tokens}


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if case["op"] == "gemm":
        if own:
            from post_weight_quantization_hessian_b200 import slim
            return slim.slim_dequant_grouped_gemm(state["codes"], state["bits"], state["scale"], state["zero"],
                                                  case["group"], case["avg_bits"], state["x"], state["offsets"],
                                                  row_index=state["row_index"], y=state["y"])
        return plain_gemm(state)
    if own:
        from post_weight_quantization_hessian_b200 import slim
        logp, entropy, top_logp, top_id = slim.slim_token_logprobs(state["logits"], state["tokens"],
                                                                   top_k=case["top_k"])
    else:
        logp, entropy, top_logp, top_id = plain_logprobs(state["logits"], state["tokens"], case["top_k"])
    out = {"logp": logp, "entropy": entropy}
    if case["top_k"]:
        out.update(top_logp=top_logp, top_id=top_id)
    return out


def plain_codes(words, widths, group):
    """Packed words [m, row words] -> codes [m, n] as int32, all groups of one width at a time."""
    m, k, dev = words.shape[0], len(widths), words.device
    first = [0]
    for b in widths:
        first.append(first[-1] + group * b // 32)
    codes = torch.empty((m, k, group // 32, 32), dtype=torch.int32, device=dev)
    for b in sorted(set(widths)):
        at = [c for c in range(k) if widths[c] == b]
        cols = torch.tensor([[first[c] + i for i in range(group * b // 32)] for c in at], device=dev)
        w = words[:, cols.flatten()].view(m, len(at), group // 32, b)
        bit = torch.arange(32, device=dev) * b
        lo, sh = bit // 32, bit % 32
        hi = torch.clamp(lo + 1, max=b - 1)
        # the low part without its sign's copies, the straddling part from the next word
        part = torch.bitwise_right_shift(w[..., lo], sh) & ((1 << (32 - sh).clamp(max=b)) - 1)
        rest = torch.where(sh + b > 32, w[..., hi] << (32 - sh).clamp(max=31), 0)
        codes[:, at] = ((part | rest) & ((1 << b) - 1)).to(torch.int32)
    return codes.view(m, k, group)


def plain_gemm(state):
    case, ends, y = state["case"], state["ends"], state["y"]
    x = state["x"] if state["row_index"] is None else state["x"][state["row_index"].long()]
    for e, (r0, r1) in enumerate(zip(ends, ends[1:])):
        if r1 > r0:
            q = plain_codes(state["codes"][e], state["widths"][e], case["group"])
            w = (q.float() - state["zero"][e][:, :, None]) * state["scale"][e][:, :, None]
            y[r0:r1] = (x[r0:r1].float() @ w.flatten(1).t()).to(y.dtype)
    return y


def plain_logprobs(logits, tokens, top_k):
    x = logits.float()
    top = x.amax(1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    d = x - base
    e = torch.exp(d)
    total = e.sum(1)
    empty = total == 0  # every logit is -inf: no probability anywhere, no entropy
    total = torch.where(empty, torch.ones_like(total), total)
    log_total = torch.log(total)
    entropy = log_total - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1) / total
    given = (tokens >= 0) & (tokens < x.shape[1])
    at = torch.where(given, tokens, torch.zeros_like(tokens))
    logp = d.gather(1, at[:, None])[:, 0] - log_total
    logp = torch.where(given, logp, torch.zeros_like(logp))
    if not top_k:
        return logp, entropy, None, None
    value, index = torch.sort(d, dim=1, descending=True, stable=True)
    return logp, entropy, value[:, :top_k] - log_total[:, None], index[:, :top_k].to(torch.int32)


# ------------------------------------------------------------------ what it cannot do without
def work(case):
    if case["op"] == "gemm":
        counts = counts_of(case)
        rows, m, n, k = sum(counts), case["m"], case["n"], case["n"] // case["group"]
        used = sum(1 for c in counts if c)
        size = {BF16: 2, F32: 4}
        weights = used * (m * n * case["avg_bits"] // 8 + 8 * m * k + k)
        xrows = min(rows, case["tokens"]) if case["tokens"] else rows
        return {"bytes": weights + xrows * n * size[case["x"]] + rows * m * size[case["y"]] + 4 * (len(counts) + 1),
                "flops": 2.0 * rows * m * n}
    rows, vocab = case["rows"], case["vocab"]
    return {"bytes": rows * vocab * (2 if case["x"] == BF16 else 4) + rows * (16 + 8 * case["top_k"]),
            "flops": 5.0 * rows * vocab}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        m, n, g, dev = case["m"], case["n"], case["group"], s["codes"].device
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=dev)
        column = torch.arange(n, device=dev)
        for e, count in enumerate(counts_of(case)):
            r0 = s["ends"][e]
            if not count:
                continue
            width = s["bits"][e].long()
            start = (torch.cumsum(width, 0) - width) * g
            bit = start[column // g] + (column % g) * width[column // g]
            mask = (1 << width[column // g]) - 1
            rows = torch.arange(r0, r0 + count, device=dev)
            if s["row_index"] is not None:
                rows = s["row_index"][rows].long()
            x = s["x"][rows].double()
            for i in range(0, m, 1024):
                bytes_ = s["codes"][e][i:i + 1024].contiguous().view(torch.uint8).long()
                bytes_ = torch.nn.functional.pad(bytes_, (0, 2))
                pair = bytes_[:, bit // 8] | bytes_[:, bit // 8 + 1] << 8
                q = (pair >> (bit % 8)) & mask
                sc = s["scale"][e][i:i + 1024].double().repeat_interleave(g, 1)
                ze = s["zero"][e][i:i + 1024].double().repeat_interleave(g, 1)
                y[r0:r0 + count, i:i + 1024] = x @ (sc * (q.double() - ze)).t()
        return y
    out = {"logp": [], "entropy": [], "top_logp": [], "top_id": None}
    for i in range(0, case["rows"], 512):
        x, t = s["logits"][i:i + 512].double(), s["tokens"][i:i + 512]
        lse = torch.logsumexp(x, 1, keepdim=True)
        lp = torch.where(lse == -math.inf, x, x - lse)
        p = lp.exp()
        out["entropy"].append(-(p * lp.clamp(min=-1e300)).sum(1))
        known = (t >= 0) & (t < case["vocab"])
        out["logp"].append(lp.gather(1, t.clamp(0, case["vocab"] - 1)[:, None])[:, 0].masked_fill(~known, 0.0))
        if case["top_k"]:
            out["top_logp"].append(lp.topk(case["top_k"], 1)[0])
    got = {k: torch.cat(v) for k, v in out.items() if v}
    if case["top_k"]:
        got["top_id"] = None
    return got
