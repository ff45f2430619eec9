"""The vectorized unpacking and products of grouped_util.py against the oracle."""
import numpy as np
import pytest
import torch

import grouped_util as U
from oracle import slim_oracle as O


@pytest.mark.parametrize("group, avg, k", [(32, 2, 3), (32, 3, 13), (64, 7, 6), (128, 4, 5)])
def test_products_of_packed_layers(group, avg, k):
    n, m, E = k * group, 5, 3
    layer = U.random_layers(E, m, n, group, avg, 1, device="cpu")
    host = [t.numpy() for t in layer]
    for e in range(E):
        assert int(host[1][e].sum()) == k * avg
        q = O.unpack_codes(host[0][e].view(np.uint32), host[1][e], group, n)
        assert np.array_equal(U.codes64(layer[0][e], layer[1][e], group).numpy(), q)
    x = torch.randn((6, n), generator=torch.Generator().manual_seed(2))
    offsets, index = [1, 3, 3, 7], [0, 5, -1, 2, 6, 2, 3, 4]
    ref = O.dequant_grouped_matmul(host[0].view(np.uint32), *host[1:], group, x.numpy(), offsets, index)
    got = U.product64(layer, group, x, offsets, torch.tensor(index))
    assert np.array_equal(np.isnan(ref), np.isnan(got.numpy()))
    np.testing.assert_allclose(got.numpy()[1:7], ref[1:7], rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_half_step_is_what_rounding_moves_at_most(dtype):
    v = torch.randn(4000, dtype=torch.float64, generator=torch.Generator().manual_seed(3)) * 10
    moved = (v.to(dtype).double() - v).abs() / U.half_step(v, dtype)
    assert 0.99 < moved.max() <= 1.0
