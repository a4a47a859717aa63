"""e4m3 pools with a scale per (block, kv head): attention whose work items have several stages or key tiles, whose CTAs
take several items, and whose contexts are cut into several partitions, against a float64 reference (the expected
output is `_attend`'s, over codes and scales that the tests draw).

Tolerance, as derived in tests/test_fp8_block.py: 2^-8 |out| for the output's rounding, (2^-8 + 2^-10) sum_j w_j |v_j| for
the weights' two e4m3 terms (or f16) and the float32 sums, and 2^-22 max_j(w_j vs_j) sum_j |code_j| for the floor of the
two terms, which is relative to the largest w vs that the row sees."""
import numpy as np
import pytest
import torch

import fp8_block_reference as R
from paged_kv_cache_313_gb300 import build as pa_build
from paged_kv_cache_313_gb300 import pa

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    pa_build.build()
    return pa.lib()


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).cuda()


def _dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def _bf16(rng, shape, gain=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * gain).astype(np.float32)).to(BF)


def _codes(rng, shape):
    """Codes of values from 2^-3 to 1.875 * 2, either sign."""
    return (rng.integers(0, 8, shape, dtype=np.uint8) | (rng.integers(4, 9, shape, dtype=np.uint8) << 3)
            | (rng.integers(0, 2, shape, dtype=np.uint8) << 7))


def _pools(rng, P, B, H):
    """K codes, V codes, K scales, V scales; the scales differ by block and head."""
    codes = [_codes(rng, (P, B, H, 128)) for _ in range(2)]
    return codes + [(2.0 ** rng.integers(-4, 2, (P, H))).astype(np.float32) for _ in range(2)]


def _attend(q, pools, table_row, limits, scale):
    """q [m, Hq, D] float64, row i attends the tokens before limits[i] that lie in valid blocks: (out, sum w |v|,
    max(w vs) sum |code|), each [m, Hq, D]."""
    kc, vc, ks, vs = pools
    P, B, H, D = kc.shape
    m, Hq, _ = q.shape
    G, n = Hq // H, int(max(limits, default=0))
    out, mag, floor = (np.zeros(q.shape) for _ in range(3))
    j = np.arange(n)
    page = table_row[j // B] if n else np.zeros(0, int)
    j = j[(page >= 0) & (page < P)]
    if j.size == 0:
        return out, mag, floor
    b, o = table_row[j // B], j % B
    see = j[None] < np.asarray(limits)[:, None]  # [m, keys]
    some = see.any(axis=1)
    last = np.maximum(see.sum(axis=1) - 1, 0)
    for h in range(H):
        k = R.E4M3[kc[b, o, h]] * ks[b, h].astype(np.float64)[:, None]
        code, s = R.E4M3[vc[b, o, h]], vs[b, h].astype(np.float64)
        v, total = code * s[:, None], np.cumsum(np.abs(code), axis=0)
        for g in range(h * G, h * G + G):
            x = np.where(see, scale * q[:, g] @ k.T, -np.inf)
            w = np.exp(x - np.where(some, x.max(axis=1, initial=-np.inf), 0.0)[:, None])
            w /= np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
            out[:, g], mag[:, g] = w @ v, w @ np.abs(v)
            floor[:, g] = (w * s).max(axis=1)[:, None] * total[last] * some[:, None]
    return out, mag, floor


def _close(got, want, mag, floor, where=None):
    got = got.float().cpu().double().numpy()
    over = np.abs(got - want) / (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -22 * floor + 1e-30)
    if where is not None:
        over = over[where]
    assert np.all(np.isfinite(over)) and over.max(initial=0.0) <= 1.0, f"{np.nanmax(over):.3g} times the tolerance"


def _tables(rng, lens, B, spare=3):
    n = [-(-L // B) for L in lens]
    P = sum(n) + spare
    perm, t, at = rng.permutation(P), np.full((len(lens), max(n)), -1, np.int32), 0
    for s, k in enumerate(n):
        t[s, :k] = perm[at:at + k]
        at += k
    return t, P


def _partials(ws):
    """Rows of partial results that a decode call left in its workspace (zeroed before the call): head_dim outputs, a
    maximum and a sum each, hardly ever zero."""
    return int(torch.count_nonzero(ws.view(torch.float32)[64:])) / 130


# ---------------------------------------------------------------- items of several stages, CTAs of several items
@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,B", [(32, 8, 8), (64, 8, 16), (32, 8, 64), (16, 8, 128)])
def test_decode_partitions_of_several_stages(Hq, Hkv, B):
    """64 contexts of up to 2500 tokens: items of up to eight 128-token stages and of several 32-entry pieces of the table,
    running maxima that grow late, bad pages and far larger or smaller V scales in later stages; NaN in every slot
    without a token."""
    rng = np.random.default_rng(Hq + B)
    lens = [2500, 2049, 2048, 1025, 1024, 1023, 513, 0, 1, 128, 129] + [int(x) for x in rng.integers(1, 2500, 53)]
    order = rng.permutation(64)
    lens = [lens[i] for i in order]
    table, P = _tables(rng, lens, B)
    kc, vc, ks, vs = pools = _pools(rng, P, B, Hkv)
    bad = 0
    for s, L in enumerate(lens):
        blocks = -(-L // B)
        if L > 600 and s % 3 == 0:  # far-apart V scales, and larger scores, from somewhere in the middle on
            far = table[s, blocks // 2:blocks]
            vs[far] *= np.float32(2.0 ** rng.integers(-40, 40))
            ks[far[::2]] *= 2
    held = np.zeros((P, B), bool)
    for s, L in enumerate(lens):
        j = np.arange(L)
        held[table[s, j // B], j % B] = True
    kc[~held], vc[~held] = 0x7f, 0xff
    ks[~held.any(axis=1)], vs[~held.any(axis=1)] = np.nan, np.inf
    for s, L in enumerate(lens):
        if L > 300 and s % 4 == 1:
            at = rng.integers(1, -(-L // B), 2)
            table[s, at] = [-1, P]
            bad += 1
    q = _bf16(rng, (64, Hq, 128))
    q[::5] *= 4
    ws = pa.new_decode_fp8_block_workspace(64, Hq, Hkv, 128, B, 2500)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q.cuda(), *_dev(*pools), _i32(table), _i32(lens), 2500, 128 ** -0.5, ws)
    got = pa.pa_decode_fp8_block(*args, error_count=err)
    assert bad and int(err.item()) > 0
    # the plan has several stages an item, and cuts contexts too
    rows = _partials(ws)
    cut = sum(L for L in lens if L > 1024)
    assert 2 * Hq * sum(L > 1024 for L in lens) < rows and cut * Hq / rows > 2.5 * 128, (rows, cut)
    assert torch.equal(got, pa.pa_decode_fp8_block(*args)), "the same call twice"
    parts = [_attend(q[s:s + 1].double().numpy(), pools, table[s], [L], 128 ** -0.5) for s, L in enumerate(lens)]
    _close(got, *(np.concatenate(x) for x in zip(*parts)))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [4, 8])
def test_decode_of_several_launches_with_partitions(Hq):
    """More sequences than a launch takes, each cut into partitions of several stages: the second launch's rows, partials
    and shorter last partitions are its own."""
    rng = np.random.default_rng(40 + Hq)
    N, B, P = 600, 16, 400
    lens = [int(x) for x in rng.integers(0, 2100, N)]
    lens[511:514] = [2100, 2100, 2049]
    table = rng.integers(0, P, (N, 132)).astype(np.int32)  # (blocks shared among sequences)
    pools = _pools(rng, P, B, 1)
    q = _bf16(rng, (N, Hq, 128), 2.0)
    ws = pa.new_decode_fp8_block_workspace(N, Hq, 1, 128, B, 2100)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q.cuda(), *_dev(*pools), _i32(table), _i32(lens), 2100, 0.1, ws)
    got = pa.pa_decode_fp8_block(*args, error_count=err)
    rows = _partials(ws)
    assert sum(L for L in lens if L > 1024) * Hq / rows > 2.5 * 128
    assert torch.equal(got, pa.pa_decode_fp8_block(*args)) and int(err.item()) == 0
    parts = [_attend(q[s:s + 1].double().numpy(), pools, table[s], [L], 0.1) for s, L in enumerate(lens)]
    _close(got, *(np.concatenate(x) for x in zip(*parts)))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,B", [(32, 8, 16), (64, 8, 64), (24, 8, 8), (8, 8, 32)])
def test_prefill_of_many_items(Hq, Hkv, B):
    """Chunks whose (query tile, kv head) items are more than two for each SM, some of one key tile, some without any,
    some long, in one call: every ring and slot is used again.  Bad pages, NaN codes in V of some chunks' own tokens (NaN
    for the queries that see them, in their head and column), NaN in every slot without a token."""
    rng = np.random.default_rng(60 + Hq + B)
    G, ppt = Hq // Hkv, 128 // (Hq // Hkv)
    chunks = [(0, 1), (5, 300), (700, 129), (0, 0), (1500, 200), (64, 64), (127, 2), (2000, 90), (300, 33), (0, 500)]
    chunks += [(int(o), int(n)) for o, n in zip(rng.integers(0, 600, 12), rng.integers(1, 40, 12))]
    while Hkv * sum(-(-n // ppt) for _, n in chunks) <= 2 * 160:  # (1 query head a kv head: 128 positions a tile)
        chunks += [(int(o), int(n)) for o, n in zip(rng.integers(0, 600, 12), rng.integers(1, 40, 12))]
    lens = [o + n for o, n in chunks]
    table, P = _tables(rng, [max(L, 1) for L in lens], B)
    kc, vc, ks, vs = pools = _pools(rng, P, B, Hkv)
    held = np.zeros((P, B), bool)
    for s, L in enumerate(lens):
        j = np.arange(L)
        held[table[s, j // B], j % B] = True
    kc[~held], vc[~held] = 0xff, 0x7f
    vs[table[4, :40]] *= np.float32(2.0 ** 30)
    vs[table[7, -20:]] *= np.float32(2.0 ** 25)
    table[2, [3, 5]] = [-1, P + 5]
    table[1, 0] = -7
    cu = np.concatenate([[0], np.cumsum([n for _, n in chunks])])
    q = _bf16(rng, (int(cu[-1]), Hq, 128))
    q[int(cu[4]) + 50:int(cu[4]) + 90] *= 5
    order = rng.permutation(len(chunks))
    table, ctx = table[np.argsort(order)], np.array(lens)[np.argsort(order)]  # chunk c is of sequence order[c]
    parts = [_attend(q[int(cu[c]):int(cu[c + 1])].double().numpy(), pools, table[order[c]],
                     [o + i + 1 for i in range(n)], 128 ** -0.5) for c, (o, n) in enumerate(chunks)]
    want, mag, floor = (np.concatenate(x) for x in zip(*parts))
    nan = np.zeros(q.shape, bool)
    for c, pos, h, dims in ((1, 200, 0, [3, 77]), (1, 304, 7, [127]), (4, 1600, 2, [0, 1]), (7, 2089, 5, [64]),
                            (9, 0, 1, [9]), (9, 257, 1, [10]), (8, 310, 3, list(range(128)))):
        vc[table[order[c], pos // B], pos % B, h, dims] = 0x7f
        first = int(cu[c]) + max(pos - chunks[c][0], 0)
        nan[first:int(cu[c + 1]), h * G:h * G + G, dims] = True
    mq = max(n for _, n in chunks)
    ws = pa.new_prefill_fp8_block_workspace(len(chunks), int(cu[-1]), mq, Hq, Hkv, 128, B, max(lens))
    out = torch.full(q.shape, 5.0, dtype=BF, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q.cuda(), _i32(cu), _i32([o for o, _ in chunks]), _i32(order), mq, *_dev(*pools), _i32(table), _i32(ctx),
            max(lens), 128 ** -0.5, ws)
    items = Hkv * sum(-(-n // ppt) for _, n in chunks)
    assert items > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pa.pa_prefill_chunk_fp8_block(*args, out=out, error_count=err)
    assert int(err.item()) > 0
    first = out.cpu()
    pa.pa_prefill_chunk_fp8_block(*args, out=out)
    assert torch.equal(torch.nan_to_num(first, nan=7.0), torch.nan_to_num(out.cpu(), nan=7.0)), "the same call twice"
    assert np.array_equal(torch.isnan(first).numpy(), nan)
    _close(first, want, mag, floor, ~nan)
