"""Infinities and NaN in the attention that accumulates the weight each key draws."""
import numpy as np
import pytest
import torch

from test_key_weights import BF16, F32, _decode_case, _i32, _prefill_args, _prefill_case, _prefill_ws, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa

# dtype, D, Hq, Hkv, B, lengths, blocks without a valid entry: tensor cores (one partition, several, head_dim 64, a group
# without an instance of its own), CUDA cores (16 heads, blocks of 24, fp32)
PATHS = [
    (BF16, 128, 8, 2, 16, [50, 50], ((0, 1), (1, 0))),
    (BF16, 128, 8, 1, 16, [3000, 90], ((0, 3), (0, 100), (1, 5))),
    (BF16, 64, 4, 2, 32, [200, 70], ((0, 0),)),
    (BF16, 128, 6, 2, 16, [100, 40], ((0, 2),)),
    (BF16, 128, 16, 1, 16, [300, 5], ((0, 7),)),
    (BF16, 128, 4, 2, 24, [301, 50], ((0, 3),)),
    (F32, 128, 4, 1, 16, [2500, 40], ((0, 2), (0, 60))),
]
_IDS = [f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[4]}"[6:] for c in PATHS]


def _decode(case, q, k, v, table, before, scale):
    dtype, D, Hq, Hkv, B, lens, holes = case
    weights = torch.tensor(before).cuda()
    ws = pa.new_decode_weights_workspace(len(lens), Hq, Hkv, D, B, max(lens))
    out = pa.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(lens), max(lens), scale, weights, ws)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), weights.cpu().numpy()


def _in_holes(case, s):
    n, B = case[5][s], case[4]
    return np.array([(s, j // B) in case[6] for j in range(n)])


@pytest.mark.gpu
@pytest.mark.parametrize("case", PATHS, ids=_IDS)
def test_nan_query_leaves_weights_in_invalid_blocks(case):
    rng, k, v, table, q, before, scale = _decode_case(case)
    q[0, 0, 7] = float("nan")  # head 0: kv head 0 of sequence 0
    _, w = _decode(case, q, k, v, table, before, scale)
    n, hole = case[5][0], _in_holes(case, 0)
    assert hole.any()
    assert np.array_equal(w[0, 0, :n][hole], before[0, 0, :n][hole]) and np.isnan(w[0, 0, :n][~hole]).all()
    assert np.array_equal(w[0, 0, n:], before[0, 0, n:])
    assert np.isfinite(w[0, 1:]).all() and np.isfinite(w[1:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("case", PATHS, ids=_IDS)
def test_nan_query_gives_nan_on_every_path(case):
    """A query head with a NaN: its outputs are NaN, those of every other head and sequence are not."""
    rng, k, v, table, q, before, scale = _decode_case(case)
    q[0, 1, 3] = float("nan")
    out, _ = _decode(case, q, k, v, table, before, scale)
    assert np.isnan(out[0, 1]).all() and np.isnan(out).sum() == case[1]


@pytest.mark.gpu
@pytest.mark.parametrize("case", PATHS, ids=_IDS)
@pytest.mark.parametrize("keys", ["one", "half"])
def test_nan_keys_reach_their_sequence(case, keys):
    """A NaN in a key of kv head 0: that head's sums over the sequence are NaN, whichever partition the key is in and whether or
    not that partition has another key."""
    rng, k, v, table, q, before, scale = _decode_case(case)
    n, B, G = case[5][0], case[4], case[2] // case[3]
    hole = _in_holes(case, 0)
    tokens = np.arange(n)[~hole]
    for j in tokens[:1] if keys == "one" else tokens[:len(tokens) // 2]:
        k[table[0, j // B], j % B, 0, 5] = float("nan")
    out, w = _decode(case, q, k, v, table, before, scale)
    assert np.isnan(out[0, :G]).all() and np.isnan(out).sum() == G * case[1]
    assert np.isnan(w[0, 0, :n][~hole]).all() and np.isnan(w).sum() == (~hole).sum()


# dtype, D, Hq, Hkv, B, chunks: tensor cores with groups that leave rows of a query tile unused, and that do not; CUDA cores
PREFILLS = [
    (BF16, 128, 3, 1, 16, [(0, 300, 100)], ()),
    (BF16, 128, 10, 2, 32, [(0, 400, 60), (1, 260, 26)], ()),
    (BF16, 128, 12, 2, 16, [(0, 0, 300)], ()),
    (BF16, 128, 8, 2, 16, [(0, 300, 100)], ()),
    (BF16, 64, 3, 1, 16, [(0, 100, 50)], ()),
    (F32, 128, 3, 1, 16, [(0, 100, 50)], ()),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", PREFILLS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{len(c[5])}"[6:])
def test_infinite_keys_that_no_query_looks_at(case):
    """Keys with an infinity that every query scores -inf draw nothing: as keys whose weights are too small for a number."""
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    B = case[4]
    q[..., 9] = -1 - q[..., 9].abs()
    results = []
    for far in (1e4, float("inf")):  # (1e4: a score below -880, 2^-1270)
        for j in (0, 3, 77, 130, 131):
            k[table[0, j // B], j % B, :, 9] = far
        weights = torch.tensor(before).cuda()
        out = pa.pa_prefill_chunk_weights(*_prefill_args(case, lens, q, k, v, table, cu, scale), weights,
                                          _prefill_ws(case, lens, q))
        results.append((out[:int(cu[1])], weights))
    torch.cuda.synchronize()
    (a, wa), (b, wb) = results
    assert torch.isfinite(wb).all()
    # (a chunk that begins at 0 has queries that see no key but such ones: their scores are -inf, their weights those of no
    # key, where the finite ones have a largest)
    first = 4 if case[5][0][1] == 0 else 0
    assert torch.equal(a[first:], b[first:])
    far = torch.zeros(wa.shape, dtype=torch.bool)
    far[0, :, :first] = True
    assert torch.equal(wa.cpu()[~far], wb.cpu()[~far])


@pytest.mark.gpu
@pytest.mark.parametrize("case", PREFILLS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{len(c[5])}"[6:])
@pytest.mark.parametrize("j", [5, 290])
def test_nan_key_reaches_the_queries_that_see_it(case, j):
    """A NaN in a key of kv head 0: NaN for the queries from its own on, and for the weights of all keys that those see."""
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    dtype, D, Hq, Hkv, B, chunks, holes = case
    s, start, n = chunks[0]
    j = min(j, start + n - 2)
    k[table[s, j // B], j % B, 0, 3] = float("nan")
    weights = torch.tensor(before).cuda()
    out = pa.pa_prefill_chunk_weights(*_prefill_args(case, lens, q, k, v, table, cu, scale), weights, _prefill_ws(case, lens, q))
    o, w = out.float().cpu().numpy(), weights.cpu().numpy()
    nan = np.zeros(o.shape, bool)
    nan[max(0, j - start):n, :Hq // Hkv] = True
    assert np.array_equal(np.isnan(o), nan)
    nan = np.zeros(w.shape, bool)
    nan[s, 0, :start + n] = True
    assert np.array_equal(np.isnan(w), nan)
