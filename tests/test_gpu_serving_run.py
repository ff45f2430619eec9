"""The serving operators together, as a user runs them: layers quantized by the
library, a mixture's experts multiplied group by group, an output head on the
result, and the log probabilities of the next tokens."""
import numpy as np
import pytest
import torch

from oracle import slim_oracle as O
from post_weight_quantization_hessian_b200 import slim
from post_weight_quantization_hessian_b200 import synthetic as syn

pytestmark = pytest.mark.gpu


def quantized(m, n, group, seed):
    spec = syn.LayerSpec(name="s", m=m, n=n, N=1024, x_dtype="bf16", group=group, avg_bits=2, seed=seed,
                         n_w_salient=4, w_scale=6.0, n_x_outliers=2, x_scale=25.0)
    W = torch.from_numpy(syn.make_weight(spec)).cuda()
    X = torch.from_numpy(syn.make_activations(spec).view(np.int16)).cuda().view(torch.bfloat16)
    codes, scale, zero, bits = slim.slim_quantize_layer(W, X, group, 2)
    return codes, bits, scale, zero


@pytest.mark.parametrize("tokens", [3, 40, 300])
def test_experts_head_and_log_probabilities(tokens):
    n, m, V, group, E = 512, 256, 1003, 128, 4
    experts = [quantized(m, n, group, 30 + e) for e in range(E)]
    head = quantized(V, m, group, 40)
    stacked = [torch.stack(t) for t in zip(*experts)]
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn((tokens, n), generator=g).bfloat16()
    choice = torch.randint(E, (tokens,), generator=g)
    choice[choice == 1] = 2                                   # one expert without tokens
    rows = torch.argsort(choice, stable=True)
    counts = torch.bincount(choice, minlength=E)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int()
    target = torch.randint(V, (tokens,), generator=g)
    target[0] = -100

    def run(x, rows, offsets, target):
        h = slim.slim_dequant_grouped_gemm(*stacked, group, 2, x, offsets, row_index=rows)
        back = torch.empty_like(h).index_copy_(0, rows.long(), h)     # the tokens' own order
        logits = slim.slim_dequant_grouped_gemm(*[t[None] for t in head], group, 2, back, whole,
                                                y_dtype=torch.float32)
        return h, back, logits, slim.slim_token_logprobs(logits, target, top_k=5)

    whole = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    args = (x.cuda(), rows.int().cuda(), offsets.cuda(), target.cuda())
    h, back, logits, out = run(*args)
    slim.slim_async_status()
    host = [t.cpu().numpy() for t in stacked]
    ref_h = O.dequant_grouped_matmul(host[0].view(np.uint32), host[1], host[2], host[3], group, x.float().numpy(),
                                     offsets.tolist(), rows.numpy())
    # bf16 h: half a step of each value, and 1e-5 of the rows' scale for the sums (see test_gpu_grouped.py)
    assert np.all(np.abs(h.float().cpu().numpy() - ref_h)
                  <= 2.0 ** -8 * np.abs(ref_h) + 1e-4 * np.abs(ref_h).max(1, keepdims=True))
    hw = [t.cpu().numpy() for t in head]
    ref_l = O.dequant_matmul(hw[0].view(np.uint32), hw[1], hw[2], hw[3], group, back.float().cpu().numpy())
    got_l = logits.double().cpu().numpy()
    assert np.linalg.norm(got_l - ref_l) <= 2e-5 * np.linalg.norm(ref_l)
    logp, ent, tl, ti = O.token_logprobs(got_l, target.numpy(), 5)
    # fp32 sums over 1003 logits: 2 (V / 256 + 40) 2^-24 (1 + 2 log V) and the values' own rounding
    tol = 2e-4
    assert np.abs(out[0].cpu().numpy() - logp).max() <= tol and np.abs(out[1].cpu().numpy() - ent).max() <= tol
    assert np.array_equal(out[3].cpu().numpy(), ti) and np.abs(out[2].cpu().numpy() - tl).max() <= tol
    assert out[0][0].item() == 0

    # the same run captured and replayed
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = run(*args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured[2], logits) and all(torch.equal(a, b) for a, b in zip(captured[3], out))
