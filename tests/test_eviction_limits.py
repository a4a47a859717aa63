"""Sizes, lengths, streams and layouts at the edges of what the calls of caches that evict tokens take."""
import numpy as np
import pytest
import torch

import eviction_reference as ref
from paged_kv_cache_313_gb300 import build as pa_build
from paged_kv_cache_313_gb300 import pa
from test_key_weights import (BF16, F32, _check_out, _check_weights, _decode_case, _decode_want, _i32, _prefill_args,
                              _prefill_case, _prefill_want, _prefill_ws)


@pytest.fixture(scope="module", autouse=True)
def lib():
    pa_build.build()
    return pa.lib()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_no_sequence_has_a_token(dtype):
    k = torch.zeros(2, 16, 1, 128, dtype=dtype, device="cuda")
    q = torch.ones(3, 4, 128, dtype=dtype, device="cuda")
    weights = torch.full((3, 1, 5), 2.0, device="cuda")
    table, lens = _i32(np.full((3, 1), -1)), _i32([0, 0, 0])
    ws = pa.new_decode_weights_workspace(3, 4, 1, 128, 16, 0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pa.pa_decode_weights(q, k, k, table, lens, 0, 1.0, weights, ws, error_count=err)
    assert torch.all(out == 0) and torch.all(weights == 2) and int(err) == 0
    new = pa.pa_evict_tokens(k, k.clone(), table, lens, 0, weights, weights.int(), lens, 4, 0, 0,
                             pa.new_evict_workspace(3, 1, 0, 4), error_count=err)
    assert new.cpu().tolist() == [0, 0, 0] and int(err) == 0


@pytest.mark.gpu
def test_decode_of_more_sequences_than_a_tensor_core_launch_takes():
    lens = [int(n) for n in np.random.default_rng(0).integers(0, 40, 1100)]
    case = (BF16, 128, 2, 1, 16, lens, ())
    rng, k, v, table, q, before, scale = _decode_case(case)
    want, mag, add, rel = _decode_want(case, q, k, v, table, scale, before.shape[2])
    weights = torch.tensor(before).cuda()
    out = pa.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(lens), max(lens), scale, weights,
                               pa.new_decode_weights_workspace(1100, 2, 1, 128, 16, max(lens)))
    _check_out(out, want, mag, rel, BF16)
    _check_weights(weights, before, add, rel, 2)


@pytest.mark.gpu
def test_decode_blocks_of_128_and_an_unaligned_output():
    case = (BF16, 128, 8, 2, 128, [300, 77], ())
    rng, k, v, table, q, before, scale = _decode_case(case)
    want, mag, add, rel = _decode_want(case, q, k, v, table, scale, before.shape[2])
    for B in (128, 16):
        kk, tt = k, table
        vv = v
        if B == 16:  # the same pools as blocks of 16
            kk, vv = k.view(-1, 16, 2, 128), v.view(-1, 16, 2, 128)
            tt = np.where(table[..., None] >= 0, table[..., None] * 8 + np.arange(8), -1).reshape(table.shape[0], -1)
        flat = torch.zeros(q.numel() + 1, dtype=BF16, device="cuda")
        out = flat[1:].view(q.shape)
        weights = torch.tensor(before).cuda()
        pa.pa_decode_weights(q.cuda(), kk.cuda(), vv.cuda(), _i32(tt), _i32(case[5]), 300, scale, weights,
                             pa.new_decode_weights_workspace(2, 8, 2, 128, B, 300), out=out)
        _check_out(out, want, mag, rel, BF16)
        _check_weights(weights, before, add, rel, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_prefill_beyond_the_longest_context_is_clamped_and_counted(dtype):
    """max_context_len, and a context shorter than its chunk: keys behind them are not read."""
    case = (dtype, 128, 4, 1, 16, [(0, 100, 60), (1, 0, 40)], ())
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    args = list(_prefill_args(case, lens, q, k, v, table, cu, scale))
    args[8], args[9] = _i32([160, 25]), 130
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    weights = torch.tensor(before).cuda()
    out = pa.pa_prefill_chunk_weights(*args, weights, _prefill_ws(case, lens, q), error_count=err)
    want, mag, add, rel = np.zeros(q.shape), np.zeros(q.shape), np.zeros(before.shape), 0.0
    kd, vd = k.double().numpy(), v.double().numpy()
    for c, (s, st, n) in enumerate(case[5]):
        limits = [min(st + i + 1, (130, 25)[c]) for i in range(n)]
        want[cu[c]:cu[c + 1]], mag[cu[c]:cu[c + 1]], w, r = ref.attend(q[cu[c]:cu[c + 1]].double().numpy(), kd, vd, table[s],
                                                                       limits, scale)
        add[s, :, :w.shape[1]] += w
        rel = max(rel, r)
    assert int(err) > 0
    _check_out(out, want, mag, rel, dtype)
    _check_weights(weights, before, add, rel, 400)


@pytest.mark.gpu
def test_prefill_workspace_of_the_largest_call_serves_smaller_ones():
    big = pa.new_prefill_weights_workspace(5, 700, 300, 8, 2, 128, 8, 900)
    for chunks in ([(0, 0, 300), (1, 50, 20)], [(0, 700, 3)], [(1, 9, 1), (0, 0, 1), (1, 3, 2), (0, 7, 100), (2, 600, 300)]):
        case = (BF16, 128, 8, 2, 16, chunks, ())
        lens, k, v, table, q, before, cu, scale = _prefill_case(case)
        want, mag, add, rel = _prefill_want(case, lens, q, k, v, table, cu, scale, before.shape[2])
        weights = torch.tensor(before).cuda()
        out = pa.pa_prefill_chunk_weights(*_prefill_args(case, lens, q, k, v, table, cu, scale), weights, big)
        _check_out(out, want, mag, rel, BF16)
        _check_weights(weights, before, add, rel, q.shape[0] * 4)


@pytest.mark.gpu
def test_prefill_few_queries_over_many_keys():
    """The keys of one tile in spans: lengths around the spans' borders, masked blocks within one."""
    for start, holes in ((3000, ()), (127, ()), (383, ()), (384, ()), (1535, ((0, 3), (0, 40)))):
        case = (BF16, 128, 4, 1, 16, [(0, start, 5)], holes)
        lens, k, v, table, q, before, cu, scale = _prefill_case(case)
        want, mag, add, rel = _prefill_want(case, lens, q, k, v, table, cu, scale, before.shape[2])
        weights = torch.tensor(before).cuda()
        out = pa.pa_prefill_chunk_weights(*_prefill_args(case, lens, q, k, v, table, cu, scale), weights,
                                          _prefill_ws(case, lens, q))
        _check_out(out, want, mag, rel, BF16)
        _check_weights(weights, before, add, rel, 20)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(F32, 128, 4, 1, 16), (F32, 64, 6, 2, 8), (BF16, 64, 8, 1, 32), (BF16, 128, 4, 2, 24)], ids=str)
def test_prefill_few_queries_over_many_keys_on_the_cuda_cores(shape):
    """As above: contexts around the spans' borders, chunks of different lengths, spans of masked blocks alone, NaN queries."""
    for chunks, holes in (([(0, 3000, 5)], ()), ([(0, 191, 1)], ()), ([(0, 383, 2), (1, 384, 70), (0, 0, 3)], ()),
                          ([(0, 1535, 17), (1, 2, 4)], tuple((0, i) for i in range(3, 60)))):
        case = shape + (chunks, holes)
        lens, k, v, table, q, before, cu, scale = _prefill_case(case)
        want, mag, add, rel = _prefill_want(case, lens, q, k, v, table, cu, scale, before.shape[2])
        args, ws, got = _prefill_args(case, lens, q, k, v, table, cu, scale), _prefill_ws(case, lens, q), []
        for _ in range(2):
            weights = torch.tensor(before).cuda()
            out = torch.full(q.shape, 3.0, dtype=shape[0], device="cuda")
            got.append((pa.pa_prefill_chunk_weights(*args, weights, ws, out=out), weights))
            ws.fill_(255)
        _check_out(got[0][0], want, mag, rel, shape[0])
        _check_weights(got[0][1], before, add, rel, q.shape[0] * shape[2] // shape[3])
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    q[0] = float("nan")
    out = pa.pa_prefill_chunk_weights(q.cuda(), *args[1:], torch.tensor(before).cuda(), ws)
    assert torch.all(torch.isnan(out[0])) and torch.equal(out[1:], got[0][0][1:])


@pytest.mark.gpu
def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own, on their streams' order alone."""
    dcase, pcase = (BF16, 128, 8, 2, 16, [700, 1300, 5], ()), (BF16, 128, 8, 2, 16, [(0, 100, 150), (1, 0, 33)], ())
    _, k, v, table, q, before, scale = _decode_case(dcase)
    dwant, dmag, dadd, drel = _decode_want(dcase, q, k, v, table, scale, before.shape[2])
    lens, pk, pv, ptable, pq, pbefore, cu, _ = _prefill_case(pcase)
    pwant, pmag, padd, prel = _prefill_want(pcase, lens, pq, pk, pv, ptable, cu, scale, pbefore.shape[2])
    dargs = (q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32(dcase[5]), 1300, scale)
    pargs = _prefill_args(pcase, lens, pq, pk, pv, ptable, cu, scale)
    dws, pws = pa.new_decode_weights_workspace(3, 8, 2, 128, 16, 1300), _prefill_ws(pcase, lens, pq)
    dw, pw = torch.tensor(before).cuda(), torch.tensor(pbefore).cuda()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        dout = pa.pa_decode_weights(*dargs, dw, dws, stream=a)
        pout = pa.pa_prefill_chunk_weights(*pargs, pw, pws, stream=b)
    torch.cuda.synchronize()
    _check_out(dout, dwant, dmag, drel, BF16)
    _check_out(pout, pwant, pmag, prel, BF16)
    _check_weights(dw, before, 8 * dadd, drel, 4 + 8)
    _check_weights(pw, pbefore, 8 * padd, prel, 183 * 4 + 8)


@pytest.mark.gpu
def test_pools_beyond_2_to_the_32_elements():
    """Blocks at the far end of pools of 4.9e9 elements each: written, attended, evicted there."""
    P, B, Hkv, D, Hq = 300000, 16, 8, 128, 16
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    rng = np.random.default_rng(2)
    k, v = (torch.empty(P, B, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    n, blocks = 150, 10
    table = np.stack([P - 1 - rng.permutation(40)[:blocks], rng.permutation(40)[:blocks]])
    qkv = torch.tensor(rng.standard_normal((2 * n, Hq + 2 * Hkv, D)), dtype=torch.float32).to(BF16).cuda()
    seq, pos = np.repeat([0, 1], n), np.tile(np.arange(n), 2)
    weights, places = torch.ones(2, Hkv, 160, device="cuda"), torch.zeros(2, Hkv, 160, dtype=torch.int32, device="cuda")
    freq, axis = (1e4 ** (-np.arange(64) / 64)).astype(np.float32), np.zeros(64, int)
    q = pa.pa_rope_write_kv_paged(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], _i32(pos), torch.tensor(freq).cuda(), None,
                                  k, v, _i32(table), _i32(seq), _i32(pos), key_weights=weights, key_pos=places)
    lens = _i32([n, n])
    out = pa.pa_prefill_chunk_weights(q, _i32([0, n, 2 * n]), _i32([0, 0]), _i32([0, 1]), n, k, v, _i32(table), lens, n, D ** -0.5,
                                      weights, pa.new_prefill_weights_workspace(2, 2 * n, n, Hq, Hkv, D, B, n))
    dec = pa.pa_decode_weights(q[[n - 1, 2 * n - 1]], k, v, _i32(table), lens, n, D ** -0.5, weights,
                               pa.new_decode_weights_workspace(2, Hq, Hkv, D, B, n))
    # the same in small pools: the same bits
    small = np.arange(2 * blocks).reshape(2, blocks)
    k2, v2 = (torch.zeros(2 * blocks, B, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    w2, p2 = torch.ones_like(weights), torch.zeros_like(places)
    q2 = pa.pa_rope_write_kv_paged(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], _i32(pos), torch.tensor(freq).cuda(), None,
                                   k2, v2, _i32(small), _i32(seq), _i32(pos), key_weights=w2, key_pos=p2)
    out2 = pa.pa_prefill_chunk_weights(q2, _i32([0, n, 2 * n]), _i32([0, 0]), _i32([0, 1]), n, k2, v2, _i32(small), lens, n,
                                       D ** -0.5, w2, pa.new_prefill_weights_workspace(2, 2 * n, n, Hq, Hkv, D, B, n))
    dec2 = pa.pa_decode_weights(q2[[n - 1, 2 * n - 1]], k2, v2, _i32(small), lens, n, D ** -0.5, w2,
                                pa.new_decode_weights_workspace(2, Hq, Hkv, D, B, n))
    assert torch.equal(q, q2) and torch.equal(out, out2) and torch.equal(dec, dec2) and torch.equal(weights, w2)
    want, mag = ref.turn(qkv[:, :Hq].double().cpu().numpy(), pos[None], freq, axis, False)
    assert np.all(np.abs(q.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag)
    for kk, vv, tt, ww, pp in ((k, v, table, weights, places), (k2, v2, small, w2, p2)):
        pa.pa_evict_tokens(kk, vv, _i32(tt), lens, n, ww, pp, lens, 64, 2, 8, pa.new_evict_workspace(2, Hkv, n, 64))
    assert torch.equal(weights, w2) and torch.equal(places, p2)
    for s in range(2):
        for pool, other in ((k, k2), (v, v2)):
            a = pool[torch.tensor(table[s][:4]).cuda()]
            assert torch.equal(a, other[torch.tensor(small[s][:4]).cuda()])


@pytest.mark.gpu
def test_rope_strided_and_broadcast_rows():
    """Tokens far apart, and one token's rows broadcast to all."""
    x = torch.randn(7, 3, 6, 64, device="cuda").to(BF16)
    pos, freq = _i32(np.arange(7) * 100), torch.tensor((1e4 ** (-np.arange(32) / 32)).astype(np.float32)).cuda()
    q, k = x[:, 1, :4], x[:, 2, 4:]
    qo, ko = pa.pa_rope(q, k, pos, freq)
    qc, kc = pa.pa_rope(q.contiguous(), k.contiguous(), pos, freq)
    assert torch.equal(qo, qc) and torch.equal(ko, kc)
    one = x[:1, 0].expand(7, 6, 64)
    a, _ = pa.pa_rope(one, k, pos, freq)
    b, _ = pa.pa_rope(one.contiguous(), k, pos, freq)
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_rope_no_heads_of_one_kind():
    x = torch.randn(5, 3, 128, device="cuda")
    pos, freq = _i32(np.arange(5)), torch.ones(64, device="cuda")
    none = torch.empty(5, 0, 128, device="cuda")
    q, k = pa.pa_rope(x, none, pos, freq)
    q2, k2 = pa.pa_rope(none, x, pos, freq)
    assert torch.equal(q, k2) and k.shape == none.shape and q2.shape == none.shape
    empty = torch.empty(0, 3, 128, device="cuda")
    q, k = pa.pa_rope(empty, empty, _i32(np.zeros(0)), freq)
    assert q.shape == empty.shape


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(BF16, 128, 4, 1, 16, [(0, 0, 90)], ()), (BF16, 128, 8, 2, 32, [(0, 60, 140), (1, 3, 200)], ()),
                                  (BF16, 128, 3, 1, 8, [(0, 500, 9)], ()), (F32, 64, 2, 1, 16, [(0, 10, 70)], ())],
                         ids=["one", "two", "spans", "f32"])
def test_prefill_values_that_are_no_numbers_stay_with_the_queries_that_see_them(case):
    """NaN and infinities among V, next to the diagonal: queries before their keys are as if they were not there."""
    dtype, D, Hq, Hkv, B, chunks, _ = case
    lens, k, v, table, q, before, cu, scale = _prefill_case(case)
    bad = {}  # (sequence, key) -> column
    for s, st, n in chunks:
        for key, col, x in ((st + n // 2, 5, np.nan), (st + n // 2 + 1, D - 3, np.inf), (st + n - 1, 40, -np.inf)):
            v[table[s, key // B], key % B, Hkv - 1, col] = float(x)
            bad.setdefault((s, Hkv - 1), []).append((key, col))
    weights = torch.tensor(before).cuda()
    out = pa.pa_prefill_chunk_weights(*_prefill_args(case, lens, q, k, v, table, cu, scale), weights,
                                      _prefill_ws(case, lens, q)).double().cpu().numpy()
    clean = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    want, mag, add, rel = _prefill_want(case, lens, q, k, clean, table, cu, scale, before.shape[2])
    g = Hq // Hkv
    sees = np.zeros(out.shape, bool)
    for c, (s, st, n) in enumerate(chunks):
        for (s2, h), items in bad.items():
            if s2 == s:
                for key, col in items:
                    sees[cu[c] + max(0, key - st):cu[c + 1], h * g:(h + 1) * g, col] = True
    assert np.isfinite(out[~sees]).all() and not np.isfinite(out[sees]).any() and sees.any()
    _check_out(torch.tensor(np.where(sees, 0, out)), np.where(sees, 0, want), mag, rel, dtype)
    _check_weights(weights, before, add, rel, q.shape[0] * g)


def test_contexts_longer_than_launches_reach_are_refused():
    """On the host, before anything is read: the largest ints are no launch's."""
    L, ptr, most = pa.lib(), 256, 2 ** 31 - 1
    for ctx in (65534 * 1024 + 1, 2 ** 30 + 1, most):
        assert L.pa_decode_weights(ptr, ptr, 1, 2, 1, 64, pa.PA_BF16, ptr, ptr, 4, 16, ptr, 2, ptr, ctx, 1.0, ptr, most, ptr, 0,
                                   None, None) == pa.PA_ERR_UNSUPPORTED
        assert L.pa_decode_weights_workspace_size(1, 2, 1, 64, 16, ctx) == 0
    for ctx in (2 ** 30 + 1, most):
        assert L.pa_prefill_chunk_weights(ptr, ptr, ptr, ptr, ptr, 1, 1, 1, 1, 2, 1, 64, pa.PA_BF16, ptr, ptr, 4, 16, ptr, 2, ptr,
                                          ctx, 1.0, ptr, most, ptr, 0, None, None) == pa.PA_ERR_UNSUPPORTED
        assert L.pa_prefill_weights_workspace_size(1, 1, 1, 2, 1, 64, 16, ctx) == 0

    def evict(ctx, budget):
        return L.pa_evict_tokens(ptr, ptr, 4, 16, 1, 64, pa.PA_BF16, ptr, 1, 2, ptr, ctx, ptr, ptr, most, ptr, budget, 0, 0, ptr,
                                 None, 0, None, None)

    for ctx, budget in ((2 ** 30 + 1, 4), (most, 2 ** 30), (2 ** 30, 65535 * 64 + 1), (65535 * 128 + 2, 65535 * 64 + 1)):
        assert evict(ctx, budget) == pa.PA_ERR_UNSUPPORTED, (ctx, budget)
        assert L.pa_evict_workspace_size(1, 1, ctx, budget) == 0
    assert L.pa_evict_workspace_size(1, 1, 65535 * 128, 65535 * 64) > 0
    assert L.pa_evict_workspace_size(1, 1, 2 ** 30, 2 ** 30 - 5) > 0
