"""Attention that accumulates the weight each key draws, for single tokens and for prompts."""
import numpy as np
import pytest
import torch

import eviction_reference as ref
from paged_kv_cache_313_gb300 import build as pa_build
from paged_kv_cache_313_gb300 import pa

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    pa_build.build()
    return pa.lib()


def _i32(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def _cache(rng, dtype, lens, B, Hkv, D, holes=()):
    """Pools with NaN wherever no token lies, a shuffled table, and table entries `holes` (sequence, block) out of range."""
    count = [-(-n // B) for n in lens]
    P = sum(count) + 2
    order = rng.permutation(P)
    width = max(count + [1]) + 1
    table = np.full((len(lens), width), -1)
    k = torch.full((P, B, Hkv, D), float("nan"))
    v = k.clone()
    at = 0
    for s, n in enumerate(lens):
        table[s, :count[s]] = order[at:at + count[s]]
        at += count[s]
        for b in range(count[s]):
            m = min(B, n - b * B)
            if (s, b) in holes:
                table[s, b] = P if b % 2 else -7
                continue
            k[table[s, b], :m] = torch.tensor(rng.standard_normal((m, Hkv, D)), dtype=torch.float32)
            v[table[s, b], :m] = torch.tensor(rng.standard_normal((m, Hkv, D)), dtype=torch.float32)
    return k.to(dtype), v.to(dtype), table


def _np(t):
    return t.double().cpu().numpy()


def _check_out(got, want, mag, rel, dtype):
    """Each weight is off by `rel`; where P is rounded to bf16 for the tensor cores, by half a step more; then one rounding."""
    p = 2.0 ** -8 if dtype == BF16 else 0.0
    tol = mag * (p + 2 * rel) * (1 + 2.0 ** -7) + torch.finfo(dtype).eps / 2 * np.abs(want)
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), np.max(err - tol)


def _check_weights(got, before, add, rel, terms):
    """`terms` numbers are added in some order in 32 bits, then to what was there."""
    want = before + add
    tol = add * (rel + (terms + 2) * 2.0 ** -24) + 2.0 ** -24 * np.abs(want)
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), np.max(err - tol)


# dtype, D, Hq, Hkv, B, lengths, holes
DECODES = [
    (BF16, 128, 32, 8, 16, [1, 0, 40, 17, 64, 65], ()),
    (BF16, 128, 4, 1, 16, [2500], ()),
    (BF16, 128, 8, 1, 64, [3000, 1, 0, 1025, 1024], ()),
    (BF16, 64, 3, 1, 32, [700, 100], ()),
    (BF16, 128, 6, 2, 8, [129, 63], ((0, 1), (0, 2), (1, 0))),
    (BF16, 128, 16, 1, 16, [300, 5], ()),          # 16 heads of a kv head: CUDA cores
    (BF16, 128, 4, 2, 24, [301, 50], ((0, 3),)),   # blocks of 24: CUDA cores
    (F32, 128, 32, 8, 16, [1, 40, 7, 23], ()),
    (F32, 64, 5, 1, 1, [600, 3], ((1, 1),)),
    (F32, 128, 2, 2, 1000, [1500], ()),
    (BF16, 128, 2, 2, 16, [5] * 70, ()),
    (BF16, 128, 4, 4, 16, [48, 16], ((0, 0), (0, 1), (0, 2))),  # a sequence without any valid block
]


def _decode_case(case, seed=0):
    dtype, D, Hq, Hkv, B, lens, holes = case
    rng = np.random.default_rng(seed + D + Hq + len(lens))
    k, v, table = _cache(rng, dtype, lens, B, Hkv, D, holes)
    q = torch.tensor(rng.standard_normal((len(lens), Hq, D)) * 1.5, dtype=torch.float32).to(dtype)
    width = max(lens) + 3
    before = rng.random((len(lens), Hkv, width)).astype(np.float32)
    return rng, k, v, table, q, before, D ** -0.5


def _decode_want(case, q, k, v, table, scale, width):
    dtype, D, Hq, Hkv, B, lens, holes = case
    out, mag, add, rel = [], [], np.zeros((len(lens), Hkv, width)), 0.0
    kd, vd = _np(k), _np(v)
    for s, n in enumerate(lens):
        o, m, w, r = ref.attend(_np(q[s:s + 1]), kd, vd, table[s], [n], scale)
        out.append(o)
        mag.append(m)
        add[s, :, :n] = w
        rel = max(rel, r)
    return np.concatenate(out), np.concatenate(mag), add, rel


@pytest.mark.gpu
@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[4]}-{len(c[5])}"[6:])
def test_decode_weights(case):
    dtype, D, Hq, Hkv, B, lens, holes = case
    rng, k, v, table, q, before, scale = _decode_case(case)
    max_len = max(lens)
    want, mag, add, rel = _decode_want(case, q, k, v, table, scale, before.shape[2])
    ws = pa.new_decode_weights_workspace(len(lens), Hq, Hkv, D, B, max_len)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(lens), max_len, scale)
    results = []
    for _ in range(2):
        weights = torch.tensor(before).cuda()
        out = pa.pa_decode_weights(*args, weights, ws, error_count=err)
        results.append((out, weights))
    torch.cuda.synchronize()
    _check_out(out, want, mag, rel, dtype)
    _check_weights(weights, before, add, rel, Hq // Hkv)
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    assert (int(err) > 0) == bool(holes)
    for s, n in enumerate(lens):
        assert np.array_equal(weights[s, :, n:].cpu().numpy(), before[s, :, n:])
        if n == 0:
            assert torch.all(out[s] == 0)


@pytest.mark.gpu
def test_decode_weights_as_pa_decode():
    """The output is pa_decode's within a rounding of each (bf16: half a step of the value for either)."""
    case = (BF16, 128, 32, 8, 16, [900, 33, 2000], ())
    rng, k, v, table, q, before, scale = _decode_case(case)
    args = (q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(case[5]), 2000, scale)
    a = pa.pa_decode_weights(*args, torch.tensor(before).cuda(), pa.new_decode_weights_workspace(3, 32, 8, 128, 16, 2000))
    b = pa.pa_decode(*args, pa.new_decode_workspace(3, 32, 8, 128, 16, 2000))
    assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 1e-6)


@pytest.mark.gpu
def test_decode_workspace_of_the_largest_call_serves_smaller_ones():
    lens = [1500, 40, 700, 1, 333, 90]
    ws = pa.new_decode_weights_workspace(6, 8, 2, 128, 16, 1500)
    for n in (6, 1, 3, 2):
        case = (BF16, 128, 8, 2, 16, lens[6 - n:] if n < 6 else lens, ())
        rng, k, v, table, q, before, scale = _decode_case(case, n)
        want, mag, add, rel = _decode_want(case, q, k, v, table, scale, before.shape[2])
        weights = torch.tensor(before).cuda()
        out = pa.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(case[5]), max(case[5]), scale, weights, ws)
        _check_out(out, want, mag, rel, BF16)
        _check_weights(weights, before, add, rel, 4)


@pytest.mark.gpu
def test_decode_weights_in_two_graphs_on_one_workspace():
    case = (BF16, 128, 8, 2, 16, [300, 1200], ())
    rng, k, v, table, q, before, scale = _decode_case(case)
    ws = pa.new_decode_weights_workspace(2, 8, 2, 128, 16, 1200)
    weights, out = torch.tensor(before).cuda(), torch.empty(2, 8, 128, dtype=BF16, device="cuda")
    args = (q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(case[5]), 1200, scale, weights, ws)
    pa.pa_decode_weights(*args, out=out)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            pa.pa_decode_weights(*args, out=out)
    want, mag, add, rel = _decode_want(case, q, k, v, table, scale, before.shape[2])
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    _check_out(out, want, mag, rel, BF16)
    _check_weights(weights, before, 5 * add, rel, 4 + 5)


@pytest.mark.gpu
def test_decode_weights_context_beyond_the_limit_is_clamped_and_counted():
    case = (BF16, 128, 4, 1, 16, [100, 60], ())
    rng, k, v, table, q, before, scale = _decode_case(case)
    ws = pa.new_decode_weights_workspace(2, 4, 1, 128, 16, 60)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    weights = torch.tensor(before).cuda()
    out = pa.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32([100, 60]), 60, scale, weights, ws,
                               error_count=err)
    want, mag, add, rel = _decode_want(case[:5] + ([60, 60], ()), q, k, v, table, scale, before.shape[2])
    assert int(err) == 1
    _check_out(out, want, mag, rel, BF16)
    _check_weights(weights, before, add, rel, 4)


@pytest.mark.gpu
def test_decode_weights_nan_query():
    case = (BF16, 128, 8, 2, 16, [50, 50], ())
    rng, k, v, table, q, before, scale = _decode_case(case)
    q[0, 5, 7] = float("nan")
    weights = torch.tensor(before).cuda()
    pa.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32([50, 50]), 50, scale, weights,
                         pa.new_decode_weights_workspace(2, 8, 2, 128, 16, 50))
    w = weights.cpu().numpy()
    assert np.isnan(w[0, 1, :50]).all() and np.isfinite(w[0, 0]).all() and np.isfinite(w[1]).all()
    assert np.array_equal(w[0, 1, 50:], before[0, 1, 50:])


# dtype, D, Hq, Hkv, B, chunks of (sequence, start, queries), holes
PREFILLS = [
    (BF16, 128, 4, 1, 16, [(0, 0, 1)], ()),
    (BF16, 128, 32, 8, 16, [(0, 263, 37)], ()),
    (BF16, 128, 8, 2, 32, [(2, 0, 100), (0, 77, 129), (1, 5, 1), (3, 130, 64)], ()),
    (BF16, 128, 8, 1, 64, [(0, 0, 300), (1, 400, 33)], ()),
    (BF16, 128, 2, 1, 8, [(0, 100, 90), (0, 190, 70), (1, 3, 20), (0, 0, 30)], ()),  # several of one sequence
    (BF16, 128, 2, 2, 128, [(0, 10, 140)], ()),
    (BF16, 128, 3, 1, 16, [(0, 20, 50)], ()),
    (BF16, 64, 4, 2, 16, [(0, 20, 75), (1, 0, 4)], ()),
    (BF16, 128, 4, 1, 24, [(0, 31, 40)], ((0, 1),)),
    (BF16, 128, 4, 1, 16, [(0, 250, 40), (1, 0, 33)], ((0, 0), (0, 9), (1, 0), (1, 1), (1, 2))),
    (F32, 128, 8, 2, 16, [(0, 0, 20), (1, 90, 41)], ()),
    (F32, 64, 16, 1, 1, [(1, 3, 9), (0, 60, 5)], ((0, 2),)),
]


def _prefill_case(case, seed=0):
    dtype, D, Hq, Hkv, B, chunks, holes = case
    rng = np.random.default_rng(seed + D + Hq + len(chunks))
    lens = [max([st + n for s, st, n in chunks if s == i] + [0]) for i in range(max(c[0] for c in chunks) + 1)]
    k, v, table = _cache(rng, dtype, lens, B, Hkv, D, holes)
    total = sum(n for _, _, n in chunks)
    q = torch.tensor(rng.standard_normal((total, Hq, D)) * 1.5, dtype=torch.float32).to(dtype)
    before = rng.random((len(lens), Hkv, max(lens) + 5)).astype(np.float32)
    cu = np.cumsum([0] + [n for _, _, n in chunks])
    return lens, k, v, table, q, before, cu, D ** -0.5


def _prefill_want(case, lens, q, k, v, table, cu, scale, width):
    dtype, D, Hq, Hkv, B, chunks, holes = case
    out, mag, add, rel = np.zeros(q.shape), np.zeros(q.shape), np.zeros((len(lens), Hkv, width)), 0.0
    kd, vd = _np(k), _np(v)
    for c, (s, st, n) in enumerate(chunks):
        o, m, w, r = ref.attend(_np(q[cu[c]:cu[c + 1]]), kd, vd, table[s], [st + i + 1 for i in range(n)], scale)
        out[cu[c]:cu[c + 1]], mag[cu[c]:cu[c + 1]] = o, m
        add[s, :, :st + n] += w
        rel = max(rel, r)
    return out, mag, add, rel


def _prefill_args(case, lens, q, k, v, table, cu, scale):
    chunks = case[5]
    return (q.cuda(), _i32(cu), _i32([c[1] for c in chunks]), _i32([c[0] for c in chunks]), max(c[2] for c in chunks),
            k.cuda(), v.cuda(), _i32(table), _i32(lens), max(lens), scale)


def _prefill_ws(case, lens, q):
    dtype, D, Hq, Hkv, B, chunks, holes = case
    ws = pa.new_prefill_weights_workspace(len(chunks), q.shape[0], max(c[2] for c in chunks), Hq, Hkv, D, B, max(lens))
    ws.fill_(255)  # (needs no zeroing: NaN)
    return ws


@pytest.mark.gpu
@pytest.mark.parametrize("case", PREFILLS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[4]}-{len(c[5])}"[6:])
def test_prefill_weights(case):
    dtype, D, Hq, Hkv, B, chunks, holes = case
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    want, mag, add, rel = _prefill_want(case, lens, q, k, v, table, cu, scale, before.shape[2])
    args, ws = _prefill_args(case, lens, q, k, v, table, cu, scale), _prefill_ws(case, lens, q)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    results = []
    for _ in range(2):
        weights = torch.tensor(before).cuda()
        results.append((pa.pa_prefill_chunk_weights(*args, weights, ws, error_count=err), weights))
    torch.cuda.synchronize()
    out, weights = results[0]
    _check_out(out, want, mag, rel, dtype)
    _check_weights(weights, before, add, rel, q.shape[0] * Hq // Hkv)
    assert torch.equal(out, results[1][0]) and torch.equal(weights, results[1][1])
    assert (int(err) > 0) == bool(holes)
    for s, n in enumerate(lens):
        assert np.array_equal(weights[s, :, n:].cpu().numpy(), before[s, :, n:])


def _rows_behind(case, extra):
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    q = torch.cat([q, torch.full((extra,) + q.shape[1:], float("nan"), dtype=q.dtype)])
    return lens, k, v, table, q, before, cu, scale


@pytest.mark.gpu
@pytest.mark.parametrize("case", [PREFILLS[1], PREFILLS[2], PREFILLS[10]], ids=["tail", "chunks", "f32"])
def test_prefill_weights_rows_behind_the_chunks(case):
    """NaN queries behind the last chunk reach nothing, and their outputs are left as they were."""
    lens, k, v, table, q, before, cu, scale = _rows_behind(case, 9)
    n = int(cu[-1])
    want, mag, add, rel = _prefill_want(case, lens, q[:n], k, v, table, cu, scale, before.shape[2])
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    weights = torch.tensor(before).cuda()
    pa.pa_prefill_chunk_weights(*_prefill_args(case, lens, q, k, v, table, cu, scale), weights, _prefill_ws(case, lens, q),
                                out=out)
    _check_out(out[:n], want, mag, rel, case[0])
    _check_weights(weights, before, add, rel, n * case[2] // case[3])
    assert torch.all(out[n:] == 3.0)


@pytest.mark.gpu
def test_prefill_weights_nan_query_stays_with_its_chunk():
    case = (BF16, 128, 4, 1, 16, [(0, 40, 50), (1, 0, 70)], ())
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    q[60, 1, 3] = float("nan")  # query 10 of sequence 1
    weights = torch.tensor(before).cuda()
    out = pa.pa_prefill_chunk_weights(*_prefill_args(case, lens, q, k, v, table, cu, scale), weights,
                                      _prefill_ws(case, lens, q))
    w, o = weights.cpu().numpy(), out.float().cpu().numpy()
    assert np.isnan(w[1, 0, :11]).all() and np.isfinite(w[1, 0, 11:]).all() and np.isfinite(w[0]).all()
    assert np.isnan(o[60, 1]).all() and np.isnan(o).sum() == 128


@pytest.mark.gpu
def test_prefill_weights_bad_chunks_are_counted_and_left():
    case = (BF16, 128, 4, 1, 16, [(0, 10, 20), (1, 0, 30), (0, 30, 10)], ())
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    args = list(_prefill_args(case, lens, q, k, v, table, cu, scale))
    args[3] = _i32([0, 5, 0])  # no sequence 5
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    weights = torch.tensor(before).cuda()
    out = torch.full(q.shape, 3.0, dtype=BF16, device="cuda")
    pa.pa_prefill_chunk_weights(*args, weights, _prefill_ws(case, lens, q), out=out, error_count=err)
    good = case[:5] + ([case[5][0], case[5][2]], ())
    rows = np.r_[0:20, 50:60]
    want, mag, add, rel = _prefill_want(good, lens, q[rows], k, v, table, np.array([0, 20, 30]), scale, before.shape[2])
    assert int(err) == 1 and torch.all(out[20:50] == 3.0)
    _check_out(out[torch.tensor(rows)], want, mag, rel, BF16)
    _check_weights(weights, before, add, rel, 30 * 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_prefill_weights_positions_beyond_the_largest_int(dtype):
    """A chunk whose last position is no int is counted and left; one that ends at the largest is clamped to its context."""
    case = (dtype, 128, 4, 1, 16, [(0, 10, 20), (1, 0, 30), (0, 30, 10)], ())
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    args = list(_prefill_args(case, lens, q, k, v, table, cu, scale))
    args[2] = _i32([10, 2 ** 31 - 10, 30])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    weights = torch.tensor(before).cuda()
    out = torch.full(q.shape, 3.0, dtype=dtype, device="cuda")
    pa.pa_prefill_chunk_weights(*args, weights, _prefill_ws(case, lens, q), out=out, error_count=err)
    good = case[:5] + ([case[5][0], case[5][2]], ())
    rows = np.r_[0:20, 50:60]
    want, mag, add, rel = _prefill_want(good, lens, q[rows], k, v, table, np.array([0, 20, 30]), scale, before.shape[2])
    assert int(err) == 1 and torch.all(out[20:50] == 3.0)
    _check_out(out[torch.tensor(rows)], want, mag, rel, dtype)
    _check_weights(weights, before, add, rel, 30 * 4)

    args[2] = _i32([10, 2 ** 31 - 1 - 30, 30])
    weights = torch.tensor(before).cuda()
    out = pa.pa_prefill_chunk_weights(*args, weights, _prefill_ws(case, lens, q), error_count=err)
    o, m, w, r = ref.attend(_np(q[20:50]), _np(k), _np(v), table[1], [lens[1]] * 30, scale)
    add[1, :, :lens[1]] += w
    assert int(err) > 1
    _check_out(out[20:50], o, m, r, dtype)
    _check_weights(weights, before, add, max(rel, r), 60 * 4)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [PREFILLS[1], PREFILLS[3], PREFILLS[10]], ids=["tail", "chunks", "f32"])
def test_prefill_weights_loose_bound_of_the_chunks(case):
    """max_q_len far above every chunk, up to the largest int: the same work."""
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    args = list(_prefill_args(case, lens, q, k, v, table, cu, scale))
    got = []
    for longest in (q.shape[0], 2 ** 31 - 1):
        args[4] = longest
        weights = torch.tensor(before).cuda()
        got.append((pa.pa_prefill_chunk_weights(*args, weights, _prefill_ws(case, lens, q)), weights))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    want, mag, add, rel = _prefill_want(case, lens, q, k, v, table, cu, scale, before.shape[2])
    _check_out(got[1][0], want, mag, rel, case[0])
    _check_weights(got[1][1], before, add, rel, q.shape[0] * case[2] // case[3])


@pytest.mark.gpu
def test_prefill_weights_many_chunks_of_few_sequences():
    """More chunks than a launch looks at together, in mixed order: the sums are those of one chunk after the other."""
    rng = np.random.default_rng(11)
    chunks = [(int(s), int(st), 1) for s, st in zip(rng.integers(0, 3, 600), rng.integers(0, 40, 600))]
    case = (F32, 64, 2, 1, 16, chunks, ())
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    want, mag, add, rel = _prefill_want(case, lens, q, k, v, table, cu, scale, before.shape[2])
    weights = torch.tensor(before).cuda()
    out = pa.pa_prefill_chunk_weights(*_prefill_args(case, lens, q, k, v, table, cu, scale), weights,
                                      _prefill_ws(case, lens, q))
    _check_out(out, want, mag, rel, F32)
    _check_weights(weights, before, add, rel, 1200)


def test_decode_weights_refusals():
    L = pa.lib()

    def decode(N=1, Hq=8, Hkv=2, D=128, dtype=pa.PA_BF16, B=16, ctx=16, width=16, ptr=None):
        return L.pa_decode_weights(ptr, ptr, N, Hq, Hkv, D, dtype, ptr, ptr, 4, B, ptr, 1, ptr, ctx, 1.0, ptr, width, None, 0,
                                   None, None)

    assert decode(N=0) == pa.PA_OK
    for bad in (dict(), dict(N=-1), dict(width=15), dict(Hq=7), dict(ctx=-1)):
        assert decode(**bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(D=96), dict(Hq=64), dict(dtype=9), dict(B=2000)):
        assert decode(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    q, pool = torch.zeros(1, 8, 128), torch.zeros(4, 16, 2, 128)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_decode_weights(q, pool, pool, i, i[0], 16, 1.0, torch.zeros(1, 2, 16), None)
    with pytest.raises(ValueError, match="key_weights must be"):
        pa.pa_decode_weights(q, pool, pool, i, i[0], 16, 1.0, torch.zeros(1, 1, 16), None)
    with pytest.raises(TypeError, match="torch.float32"):
        pa.pa_decode_weights(q, pool.bfloat16(), pool.bfloat16(), i, i[0], 16, 1.0, torch.zeros(1, 2, 16), None)


def test_prefill_weights_refusals():
    L = pa.lib()

    def prefill(C=1, T=4, Hq=8, Hkv=2, D=128, dtype=pa.PA_BF16, B=16, ctx=16, width=16, ptr=None):
        return L.pa_prefill_chunk_weights(ptr, ptr, ptr, ptr, ptr, C, T, 4, 1, Hq, Hkv, D, dtype, ptr, ptr, 4, B, ptr, 1, ptr,
                                          ctx, 1.0, ptr, width, None, 0, None, None)

    assert prefill(C=0) == pa.PA_OK and prefill(T=0) == pa.PA_OK
    for bad in (dict(), dict(C=-1), dict(width=15), dict(Hq=7), dict(ctx=-1)):
        assert prefill(**bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(D=96), dict(Hq=64), dict(dtype=9), dict(B=2000)):
        assert prefill(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    assert L.pa_prefill_weights_workspace_size(1, 4, 4, 7, 2, 128, 16, 16) == 0
    q, pool = torch.zeros(4, 8, 128), torch.zeros(4, 16, 2, 128)
    i = torch.zeros(1, 1, dtype=torch.int32)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_prefill_chunk_weights(q, cu, i[0], i[0], 4, pool, pool, i, i[0], 16, 1.0, torch.zeros(1, 2, 16), None)
    with pytest.raises(ValueError, match="disagree"):
        pa.pa_prefill_chunk_weights(q, cu[:1], i[0], i[0], 4, pool, pool, i, i[0], 16, 1.0, torch.zeros(1, 2, 16), None)


@pytest.mark.gpu
def test_workspaces_are_checked():
    case = DECODES[0]
    rng, k, v, table, q, before, scale = _decode_case(case)
    ws = pa.new_decode_weights_workspace(6, 32, 8, 128, 16, 65)
    args = (q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(case[5]), 65, scale, torch.tensor(before).cuda())
    for bad in (None, ws[:256], ws[1:]):
        with pytest.raises(pa.PaError) as e:
            pa.pa_decode_weights(*args, bad)
        assert e.value.status == pa.PA_ERR_WORKSPACE
    case = PREFILLS[1]
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    args, ws = _prefill_args(case, lens, q, k, v, table, cu, scale), _prefill_ws(case, lens, q)
    for bad in (None, ws[:-256], ws[1:]):
        with pytest.raises(pa.PaError) as e:
            pa.pa_prefill_chunk_weights(*args, torch.tensor(before).cuda(), bad)
        assert e.value.status == pa.PA_ERR_WORKSPACE
