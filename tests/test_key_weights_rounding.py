"""What the rounding of the probabilities leaves in the output of the prefill that accumulates key weights."""
import numpy as np
import pytest
import torch

from test_key_weights import BF16, _i32, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,starts,n", [(4, 1, [512], 30), (32, 8, [512, 304, 128], 200), (8, 1, [1040], 130)],
                         ids=["spans", "tiles", "long"])
def test_weights_of_an_output_add_up_to_one(Hq, Hkv, starts, n):
    """Every softmax over these keys gives one mean: sixteen keys of one direction each, of whose values nine are u and seven
    the bf16 number behind u.  The mean lies 7/16 of the way between them, 1/16 of it below the middle, 2^-12 of u at least:
    however the weights are rounded, a division by their own sum ends at u."""
    rng = np.random.default_rng(len(starts) + Hq)
    D, B, S = 128, 16, len(starts)
    lens = [s + n for s in starts]
    count = [-(-x // B) for x in lens]
    P = sum(count)
    order, at = rng.permutation(P), 0
    table = np.full((S, max(count)), -1)
    k, v = torch.zeros(P, B, Hkv, D), torch.zeros(P, B, Hkv, D)
    u = torch.tensor(1 + rng.random((Hkv, D)), dtype=torch.float32).to(BF16)
    above = (u.view(torch.int16) + 1).view(BF16).float()
    for s in range(S):
        table[s, :count[s]] = order[at:at + count[s]]
        at += count[s]
        for b in range(count[s]):
            pool = int(table[s, b])
            k[pool] = torch.tensor(rng.standard_normal((1, Hkv, D)), dtype=torch.float32)
            k[pool, :, :, 9] = 0 if b * B < starts[s] else 1e4  # the chunk's own keys: a score below -880
            v[pool] = u.float()
            v[pool, torch.as_tensor(rng.permutation(B)[:7])] = above
    q = torch.tensor(rng.standard_normal((S * n, Hq, D)) * 3, dtype=torch.float32)
    q[..., 9] = -1 - q[..., 9].abs()
    width = max(lens)
    weights = torch.zeros(S, Hkv, width, device="cuda")
    ws = pa.new_prefill_weights_workspace(S, S * n, n, Hq, Hkv, D, B, width)
    out = pa.pa_prefill_chunk_weights(q.to(BF16).cuda(), _i32(np.arange(S + 1) * n), _i32(starts), _i32(range(S)), n,
                                      k.to(BF16).cuda(), v.to(BF16).cuda(), _i32(table), _i32(lens), width, D ** -0.5, weights, ws)
    want = u[:, None].expand(Hkv, Hq // Hkv, D).reshape(Hq, D).cuda()
    assert torch.equal(out, want[None].expand(out.shape))
    # and the weights, from the 32-bit sums, add up to the heads of all queries
    total = weights.double().sum(dim=2).cpu().numpy()
    assert np.all(np.abs(total / (n * Hq // Hkv) - 1) <= 2.0 ** -16)
