"""Attention with key weights where every CTA has several items: query tiles and pairs of key tiles of a prefill, whose rings and
buffers go round, and items of a decode."""
import math

import numpy as np
import pytest
import torch

from test_key_weights import BF16, _cache, _i32, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa

# Hq, Hkv, B, chunks of (sequence, start, queries), holes.  Query tiles and (256 keys, tile) units, for 152 CTAs:
CASES = [
    (64, 8, 16, [(0, 1500, 260), (1, 2100, 260), (2, 700, 260), (3, 0, 260)], ()),   # 544 tiles, 2856 units
    (40, 8, 32, [(1, 900, 300), (0, 1300, 310), (1, 1200, 290), (0, 0, 300)], ()),   # groups of 5; 392 tiles, 1768 units
    (16, 8, 64, [(0, 3000, 700)], ()),                                                # 88 tiles in spans, 1200 units
    (64, 8, 16, [(0, 1500, 260), (1, 2100, 260), (2, 700, 260)], ((0, 3), (0, 60), (1, 0), (1, 130), (2, 50))),
]
_IDS = ["tiles", "odd-group", "spans", "holes"]


def _make(case, seed=0):
    Hq, Hkv, B, chunks, holes = case
    rng = np.random.default_rng(seed + Hq)
    lens = [max(st + n for s, st, n in chunks if s == i) for i in range(max(c[0] for c in chunks) + 1)]
    k, v, table = _cache(rng, BF16, lens, B, Hkv, 128, holes)
    cu = np.cumsum([0] + [n for _, _, n in chunks])
    q = torch.tensor(rng.standard_normal((cu[-1], Hq, 128)) * 1.5, dtype=torch.float32).to(BF16)
    before = torch.tensor(rng.random((len(lens), Hkv, max(lens) + 5)), dtype=torch.float32)
    return lens, k, v, table, q, before, cu, 128 ** -0.5


def _run(case, lens, k, v, table, q, before, cu, scale):
    Hq, Hkv, B, chunks, holes = case
    most = max(c[2] for c in chunks)
    ws = pa.new_prefill_weights_workspace(len(chunks), q.shape[0], most, Hq, Hkv, 128, B, max(lens))
    ws.fill_(255)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q.cuda(), _i32(cu), _i32([c[1] for c in chunks]), _i32([c[0] for c in chunks]), most, k.cuda(), v.cuda(),
            _i32(table), _i32(lens), max(lens), scale)
    results = []
    for _ in range(2):
        weights = before.cuda()
        results.append((pa.pa_prefill_chunk_weights(*args, weights, ws, error_count=err), weights))
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return results[0] + (int(err),)


def _reference(case, lens, k, v, table, q, cu, scale):
    """In float64 on the GPU: outputs, softmax |v|, the weights drawn, and a bound of a weight's relative error (as
    eviction_reference.attend's)."""
    Hq, Hkv, B, chunks, holes = case
    G, P = Hq // Hkv, k.shape[0]
    kd, vd, qd = (torch.nan_to_num(t.double().cuda(), nan=0.0) for t in (k, v, q))
    out, mag = torch.zeros_like(qd), torch.zeros_like(qd)
    add, rel = torch.zeros(len(lens), Hkv, max(lens), dtype=torch.float64, device="cuda"), 0.0
    for c, (s, st, n) in enumerate(chunks):
        keys = torch.arange(st + n, device="cuda")
        block = torch.as_tensor(table[s], device="cuda")[keys // B]
        ok = (block >= 0) & (block < P)
        at = torch.where(ok, block, 0)
        see = ok[None] & (keys[None] <= st + torch.arange(n, device="cuda")[:, None])
        for h in range(Hkv):
            kk, vv = kd[at, keys % B, h], vd[at, keys % B, h]
            for g in range(h * G, (h + 1) * G):
                x = qd[cu[c]:cu[c + 1], g]
                score = scale * x @ kk.T
                w = torch.nan_to_num(torch.softmax(score.masked_fill(~see, -math.inf), dim=1), nan=0.0)
                out[cu[c]:cu[c + 1], g], mag[cu[c]:cu[c + 1], g] = w @ vv, w @ vv.abs()
                add[s, h, :st + n] += w.sum(0)
                terms = float((scale * x.abs() @ kk.abs().T).max())
                rel = max(rel, 2 * 136 * 2.0 ** -23 * terms
                          + 8 * 2.0 ** -23 * (float(score.abs().max()) + math.log(st + n) + 1))
    return out, mag, add, rel + 2.0 ** -20


def _check(got, want, mag, rel, rows=None):
    tol = mag * (2.0 ** -8 + 2 * rel) * (1 + 2.0 ** -7) + 2.0 ** -8 * want.abs()
    assert torch.all((got.double() - want).abs() <= tol)


def _check_weights(case, got, before, add, rel, total_q):
    n = add.shape[2]
    want = before.double().cuda()
    want[..., :n] += add
    tol = (rel + (total_q * case[0] // case[1] + 2) * 2.0 ** -24) * (want - before.double().cuda()) + 2.0 ** -24 * want.abs()
    assert torch.all((got.double() - want).abs() <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=_IDS)
def test_many_tiles_of_a_cta(case):
    lens, k, v, table, q, before, cu, scale = _make(case)
    out, weights, errors = _run(case, lens, k, v, table, q, before, cu, scale)
    want, mag, add, rel = _reference(case, lens, k, v, table, q, cu, scale)
    assert (errors > 0) == bool(case[4])
    _check(out, want, mag, rel)
    _check_weights(case, weights, before, add, rel, int(cu[-1]))


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES[:3], ids=_IDS[:3])
def test_values_that_are_no_numbers_stay_with_their_queries(case):
    """Infinities and NaN among the values of a chunk's own keys, in other columns for each kv head and chunk: the queries that
    see the key have NaN or the infinity there, whichever item of a CTA they are in, and nothing else changes."""
    Hq, Hkv, B, chunks, holes = case
    lens, k, v, table, q, before, cu, scale = _make(case, 1)
    rng = np.random.default_rng(7)
    G = Hq // Hkv
    clean = v.clone()
    bad = torch.zeros(q.shape, dtype=torch.bool)
    if len({s for s, _, _ in chunks}) < len(chunks):
        chunks_ = [c for c in range(len(chunks)) if chunks[c][1] + chunks[c][2] == lens[chunks[c][0]]]
    else:
        chunks_ = range(len(chunks))  # (each a sequence's last: no other chunk sees its own keys)
    for c in chunks_:
        s, st, n = chunks[c]
        for h in range(Hkv):
            if (c + h) % 3 == 2:
                continue  # items without any, between
            for _ in range(3):
                i, col = int(rng.integers(n)), int(rng.integers(128))
                j = st + i
                v[table[s, j // B], j % B, h, col] = [float("nan"), float("inf"), -float("inf")][int(rng.integers(3))]
                bad[cu[c] + i:cu[c + 1], h * G:(h + 1) * G, col] = True
    out, weights, errors = _run(case, lens, k, v, table, q, before, cu, scale)
    assert errors == 0
    want, mag, add, rel = _reference(case, lens, k, clean, table, q, cu, scale)
    bad = bad.cuda()
    assert torch.all(~torch.isfinite(out[bad])) and torch.all(torch.isfinite(out[~bad]))
    _check(torch.where(bad, 0.0, out.float()), torch.where(bad, 0.0, want), mag, rel)
    _check_weights(case, weights, before, add, rel, int(cu[-1]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hq,Hkv,B", [(BF16, 32, 8, 16), (BF16, 24, 8, 32), (torch.float32, 8, 4, 16)],
                         ids=["bf16", "groups-of-3", "fp32"])
def test_many_decode_items_of_a_cta(dtype, Hq, Hkv, B):
    """Sixty sequences of up to 2500 tokens, whole partitions and short ones."""
    rng = np.random.default_rng(Hq)
    D, G = 128, Hq // Hkv
    lens = [int(x) for x in rng.integers(1, 2500, 60)]
    k, v, table = _cache(rng, dtype, lens, B, Hkv, D)
    q = torch.tensor(rng.standard_normal((60, Hq, D)) * 1.5, dtype=torch.float32).to(dtype)
    before = torch.tensor(rng.random((60, Hkv, max(lens) + 3)), dtype=torch.float32)
    scale = D ** -0.5
    ws = pa.new_decode_weights_workspace(60, Hq, Hkv, D, B, max(lens))
    weights = before.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pa.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(lens), max(lens), scale, weights, ws,
                               error_count=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    kd, vd, qd = k.double().cuda(), v.double().cuda(), q.double().cuda()
    p = 2.0 ** -8 if dtype == BF16 else 0.0
    for s, n in enumerate(lens):
        keys = torch.arange(n, device="cuda")
        at = torch.as_tensor(table[s], device="cuda")[keys // B]
        kk, vv = kd[at, keys % B], vd[at, keys % B]                      # [n, Hkv, D]
        x = qd[s].view(Hkv, G, D)
        score = scale * torch.einsum("hgd,nhd->hgn", x, kk)
        w = torch.softmax(score, dim=2)
        terms = float((scale * torch.einsum("hgd,nhd->hgn", x.abs(), kk.abs())).max())
        rel = 2.0 ** -20 + 2 * 136 * 2.0 ** -23 * terms + 8 * 2.0 ** -23 * (float(score.abs().max()) + math.log(n) + 1)
        want = torch.einsum("hgn,nhd->hgd", w, vv).view(Hq, D)
        mag = torch.einsum("hgn,nhd->hgd", w, vv.abs()).view(Hq, D)
        tol = mag * (p + 2 * rel) * (1 + 2.0 ** -7) + torch.finfo(dtype).eps / 2 * want.abs()
        assert torch.all((out[s].double() - want).abs() <= tol)
        old, add = before[s].double().cuda(), w.sum(1)
        tol = (rel + (G + 2) * 2.0 ** -24) * add + 2.0 ** -24 * (old[:, :n] + add)
        assert torch.all((weights[s, :, :n].double() - old[:, :n] - add).abs() <= tol)
        assert torch.equal(weights[s, :, n:].cpu(), before[s, :, n:])
