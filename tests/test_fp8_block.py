"""e4m3 pools with a scale per (block, kv head): the quantising write, the read back, decode and chunked prefill,
against a float64 reference (tests/fp8_block_reference.py).

Write and read back are bit-exact.  Attention: an output is off by at most its own rounding to bf16, 2^-8 |out|; by
the rounding of the probabilities to bf16-like precision (two e4m3 terms: 2^-4 of a half step's 2^-4), 2^-8 of
sum_j p_j |v_j|; and by the float32 products, exponentials and sums, for which 2^-10 of that sum leaves room (scores
below about 64 in magnitude, rounded to 2^-24 of their terms' sum, plus 2^-20 of the largest query element).
The two terms have a floor: a weight w = 256 p vs_j / R (p <= 1, R the power of two not below any V scale) is hi + lo / 16
with lo's subnormals 2^-9 apart, so it is off by max(2^-8 w, 2^-9 / 16 / 2 = 2^-14); the output then by
sum_j 2^-14 (R / 256) |code_j| / l <= 2^-22 R sum_j |code_j|, since the sum l of the unrounded p has a term that is 1."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_block_reference as R
from paged_kv_cache_313_gb300 import build as pa_build
from paged_kv_cache_313_gb300 import pa
from paged_kv_cache_313_gb300 import workloads as W
from paged_kv_cache_313_gb300.runner import DeviceStep

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.lib()


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _bf16(rng, shape, gain=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * gain).astype(np.float32)).to(BF)


def _tables(rng, lens, block, spare=3, width=None):
    """Shuffled block table [S, width] for the lengths, -1 beyond, and the number of blocks of the pool."""
    n = [-(-L // block) for L in lens]
    P = sum(n) + spare
    perm = rng.permutation(P)
    t = np.full((len(lens), max(1, width or max(n, default=1))), -1, np.int32)
    at = 0
    for s, k in enumerate(n):
        t[s, :k] = perm[at:at + k]
        at += k
    return t, P


def _pools(rng, P, block, H, D, pow2=True):
    """Random codes (no NaN) and scales that differ by block and head."""
    codes = rng.integers(0, 0x7f, (P, block, H, D), dtype=np.uint8) | (rng.integers(0, 2, (P, block, H, D), dtype=np.uint8) << 7)
    # magnitudes about 1: most codes' exponents near the middle
    codes = np.where(rng.random(codes.shape) < 0.97, codes & 0x87 | (rng.integers(4, 9, codes.shape, dtype=np.uint8) << 3),
                     codes).astype(np.uint8)
    codes[(codes & 0x7f) == 0x7f] = 0x38
    scales = 2.0 ** rng.integers(-4, 2, (P, H)).astype(np.float64)
    if not pow2:
        scales *= 1 + rng.random((P, H))
    return codes, scales.astype(np.float32)


# ---------------------------------------------------------------- CPU: refusals
def test_refusals_need_no_device(lib):
    P16 = ctypes.c_void_p(16)
    w = lambda *a: lib.pa_write_kv_paged_fp8_block(*a)  # noqa: E731
    ok = [P16, P16, 4, 8, 128, P16, P16, P16, P16, 10, 16, P16, 2, 4, P16, P16, None, None, 0, None, None]
    bad = [(2, -1, 1), (3, 0, 1), (4, 0, 1), (4, 24, 2), (9, -1, 1), (10, 0, 1), (10, 1025, 2), (12, -1, 1),
           (0, None, 1), (5, None, 1), (7, None, 1), (8, None, 1), (11, None, 1), (14, None, 1), (15, None, 1),
           (0, ctypes.c_void_p(8), 2), (6, ctypes.c_void_p(24), 2), (3, 1 << 17, 2)]
    for i, value, want in bad:
        a = list(ok)
        a[i] = value
        assert w(*a) == want, (i, value)
    a = list(ok)
    a[2] = 0
    assert w(*a) == pa.PA_OK
    r_ok = [P16, P16, 4, 8, 128, pa.PA_BF16, P16, P16, P16, P16, 10, 16, P16, 2, 4, P16, P16, None, None]
    for i, value, want in [(2, -1, 1), (5, 7, 2), (4, 8, 2), (11, 0, 1), (0, None, 1), (8, None, 1), (1, ctypes.c_void_p(4), 2)]:
        a = list(r_ok)
        a[i] = value
        assert lib.pa_read_kv_paged_fp8_block(*a) == want, (i, value)
    f = ctypes.c_float(1.0)
    d_ok = [P16, P16, 2, 8, 2, 128, P16, P16, P16, P16, 10, 16, P16, 4, P16, 64, f, P16, 0, None, None]
    for i, value, want in [(2, -1, 1), (3, 7, 1), (3, 34, 2), (5, 96, 2), (11, 0, 2), (11, 2048, 2), (15, -1, 1),
                           (8, None, 1), (9, None, 1), (0, None, 1), (14, None, 1)]:
        a = list(d_ok)
        a[i] = value
        assert lib.pa_decode_fp8_block(*a) == want, (i, value)
    p_ok = [P16, P16, P16, P16, P16, 1, 4, 4, 1, 8, 2, 128, P16, P16, P16, P16, 10, 16, P16, 4, P16, 64, f, None, 0,
            None, None]
    for i, value, want in [(5, -1, 1), (6, -1, 1), (7, -1, 1), (9, 7, 1), (11, 96, 2), (17, 2048, 2), (21, -1, 1),
                           (8, 0, 1), (14, None, 1), (2, None, 1), (20, None, 1)]:
        a = list(p_ok)
        a[i] = value
        assert lib.pa_prefill_chunk_fp8_block(*a) == want, (i, value)
    assert lib.pa_write_fp8_block_workspace_size(1024, 100, 16) == 0
    assert lib.pa_write_fp8_block_workspace_size(1025, 100, 16) > 100 * 16 * 4
    assert lib.pa_write_fp8_block_workspace_size(-1, 100, 16) == 0


def test_binding_refuses_mismatched_arguments(lib):
    kc = torch.zeros(4, 16, 2, 128, dtype=torch.uint8)
    sc = torch.ones(4, 2)
    bt = torch.zeros(1, 4, dtype=torch.int32)
    i = torch.zeros(3, dtype=torch.int32)
    kn = torch.zeros(3, 2, 128, dtype=BF)
    q = torch.zeros(1, 4, 128, dtype=BF)
    with pytest.raises(ValueError):  # not CUDA tensors
        pa.pa_write_kv_paged_fp8_block(kn, kn, kc, kc, sc, sc, bt, i, i)
    with pytest.raises(TypeError):
        pa.pa_write_kv_paged_fp8_block(kn, kn, kc.to(BF), kc.to(BF), sc, sc, bt, i, i)
    with pytest.raises(ValueError, match="k_scales"):
        pa.pa_write_kv_paged_fp8_block(kn, kn, kc, kc, sc[:, :1], sc, bt, i, i)
    with pytest.raises(ValueError, match="one entry"):
        pa.pa_write_kv_paged_fp8_block(kn, kn, kc, kc, sc, sc, bt, i[:2], i)
    with pytest.raises(ValueError, match="disagree"):
        pa.pa_write_kv_paged_fp8_block(kn[:, :1], kn[:, :1], kc, kc, sc, sc, bt, i, i)
    with pytest.raises(ValueError, match="differ"):
        pa.pa_read_kv_paged_fp8_block(kc, kc, sc, sc, bt, i, i[:2])
    with pytest.raises(ValueError, match="one dtype"):
        pa.pa_read_kv_paged_fp8_block(kc, kc, sc, sc, bt, i, i, k_out=kn[:2])
    with pytest.raises(ValueError, match="head_dim"):
        pa.pa_decode_fp8_block(q[..., :64], kc, kc, sc, sc, bt, i[:1], 64, 1.0, None)
    with pytest.raises(ValueError, match="disagree"):
        pa.pa_decode_fp8_block(q, kc, kc, sc, sc, bt, i, 64, 1.0, None)
    with pytest.raises(ValueError, match="disagree"):
        pa.pa_prefill_chunk_fp8_block(q, i, i[:1], i[:1], 1, kc, kc, sc, sc, bt, i[:1], 64, 1.0)


def test_reference_codes_match_the_c_oracle():
    import oracle
    for c in range(256):
        want = oracle.e4m3_value(c)
        assert (np.isnan(want) and np.isnan(R.E4M3[c])) or want == R.E4M3[c]
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(400) * 10.0 ** rng.integers(-4, 4, 400), R.E4M3[np.isfinite(R.E4M3)],
                        [0.0, -0.0, 448.0, 464.0, 1e9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0]]).astype(np.float32)
    got = R.nearest_code(x.astype(np.float64))
    assert [int(g) for g in got] == [oracle.e4m3_encode(float(v)) for v in x]


# ---------------------------------------------------------------- GPU: write and read back
def _check_write(kn, vn, codes, scales, table, seq, pos, steps=1, ws_tokens=None):
    """The write against the reference, bit for bit: codes, scales, slots and errors."""
    P, B, H, D = codes[0].shape
    kc, vc = (torch.from_numpy(c.copy()).cuda() for c in codes)
    ks, vs = (torch.from_numpy(s.copy()).cuda() for s in scales)
    T = len(seq)
    slot = torch.full((T,), -7, dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.new_write_fp8_block_workspace(ws_tokens or T, P, B)
    for _ in range(steps):
        pa.pa_write_kv_paged_fp8_block(kn.cuda(), vn.cuda(), kc, vc, ks, vs, _i32(table), _i32(seq), _i32(pos), ws,
                                       slot_mapping=slot, error_count=err)
    want_slot, want_err = R.slots(table, seq, pos, B, P)
    assert np.array_equal(slot.cpu().numpy(), want_slot)
    assert int(err.item()) == want_err * steps
    for new, c, s, gc, gs in ((kn, codes[0], scales[0], kc, ks), (vn, codes[1], scales[1], vc, vs)):
        c, s = c.copy(), s.astype(np.float64)
        for _ in range(steps):
            R.write(new.double().numpy(), c, s, want_slot)
        assert np.array_equal(gs.cpu().numpy().astype(np.float64), s)
        got = gc.cpu().numpy()
        both_nan = ((got & 0x7f) == 0x7f) & ((c & 0x7f) == 0x7f)
        assert np.array_equal(np.where(both_nan, 0, got), np.where(both_nan, 0, c))
    if ws is not None:
        assert int(torch.count_nonzero(ws)) == 0, "the workspace is left zeroed"
    return kc, vc, ks, vs


WRITE_SHAPES = [(8, 128, 16), (1, 128, 16), (2, 64, 8), (3, 48, 5), (4, 16, 1), (2, 128, 64), (1, 32, 1024), (5, 112, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("H,D,B", WRITE_SHAPES)
@pytest.mark.parametrize("T", [1, 2, 37, 300])
def test_write_matches_reference(H, D, B, T):
    """Chunks that begin inside blocks, in shuffled order, with padding and bad indices among them."""
    rng = np.random.default_rng(100 * H + D + B + T)
    S = min(T, 4)
    first = rng.integers(0, 2 * B + 3, S)
    counts = [T // S + (i < T % S) for i in range(S)]
    lens = [int(f + c) for f, c in zip(first, counts)]
    table, P = _tables(rng, lens, B)
    seq = np.concatenate([[s] * c for s, c in enumerate(counts)]).astype(np.int32)
    pos = np.concatenate([np.arange(f, f + c) for f, c in zip(first, counts)]).astype(np.int32)
    if T >= 37:
        pos[3], seq[5], seq[6], pos[7] = -1, -1, S, 10 ** 6
        table[0, 0] = P  # no such block
    order = rng.permutation(T)
    seq, pos = seq[order], pos[order]
    codes, scales = zip(_pools(rng, P, B, H, D), _pools(rng, P, B, H, D))
    gain = 10.0 ** rng.integers(-3, 3, (T, H, 1))
    _check_write(_bf16(rng, (T, H, D), gain), _bf16(rng, (T, H, D), gain[::-1]), codes, scales, table, seq, pos)


@pytest.mark.gpu
@pytest.mark.parametrize("T,B", [(1024, 16), (1025, 16), (2500, 64), (3001, 7), (1100, 1024)])
def test_write_long_calls_match_reference(T, B):
    """Both forms around the length where the second takes over; the workspace made for more tokens."""
    rng = np.random.default_rng(T + B)
    H, D, S = 2, 128, 5
    first = rng.integers(0, 40, S)
    counts = [T // S + (i < T % S) for i in range(S)]
    table, P = _tables(rng, [int(f + c) for f, c in zip(first, counts)], B)
    seq = np.concatenate([[s] * c for s, c in enumerate(counts)]).astype(np.int32)
    pos = np.concatenate([np.arange(f, f + c) for f, c in zip(first, counts)]).astype(np.int32)
    pos[11], seq[13] = -5, 99
    order = rng.permutation(T) if B != 16 else np.arange(T)
    codes, scales = zip(_pools(rng, P, B, H, D), _pools(rng, P, B, H, D))
    _check_write(_bf16(rng, (T, H, D)), _bf16(rng, (T, H, D), 30.0), codes, scales, table, seq[order], pos[order],
                 ws_tokens=T + 500)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 1500])
def test_write_same_slot_last_token_is_stored(T):
    rng = np.random.default_rng(T)
    table, P = _tables(rng, [T], 16)
    pos = rng.integers(0, T // 3, T).astype(np.int32)
    codes, scales = zip(_pools(rng, P, 16, 2, 64), _pools(rng, P, 16, 2, 64))
    _check_write(_bf16(rng, (T, 2, 64)), _bf16(rng, (T, 2, 64)), codes, scales, table, np.zeros(T, np.int32), pos)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 1500])
def test_write_to_a_pool_without_blocks_counts_every_token(lib, T):
    """No block to store into: every token is counted and skipped, in both forms of the call."""
    H, D, B = 2, 64, 16
    x = torch.ones(T, H, D, dtype=BF, device="cuda")
    pool, sc = torch.full((B * H * D,), 7, dtype=torch.uint8, device="cuda"), torch.ones(H, device="cuda")
    bt, seq, pos = _i32([[0] * 200]), _i32([0] * T), _i32(range(T))
    need = lib.pa_write_fp8_block_workspace_size(T, 0, B)
    ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    err, slots = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for _ in range(2):
        assert lib.pa_write_kv_paged_fp8_block(
            ptr(x), ptr(x), T, H, D, ptr(pool), ptr(pool), ptr(sc), ptr(sc), 0, B, ptr(bt), 1, 200, ptr(seq), ptr(pos),
            ptr(slots), ptr(ws), need, ptr(err), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == pa.PA_OK
    assert int(err.item()) == 2 * T and bool((slots == -1).all()) and bool((pool == 7).all())
    assert int(torch.count_nonzero(ws)) == 0


@pytest.mark.gpu
def test_write_special_values():
    """Zeros, infinities, NaN, subnormals and the largest numbers; a block of zeros only; scales of 0 and old scales
    that are no power of two."""
    rng = np.random.default_rng(3)
    H, D, B, T = 4, 32, 8, 24
    table, P = _tables(rng, [T + 3], B)
    kn = _bf16(rng, (T, H, D))
    kn[0, 0, 0], kn[1, 0, 1], kn[2, 0, 2] = float("inf"), float("-inf"), float("nan")
    kn[:, 1] = 0.0
    kn[:, 2] = float("nan")
    kn[3, 3, 3] = 3e38
    kn[9, 3, :] = 1e-39  # subnormal in bf16
    vn = torch.full((T, H, D), 1.0).to(BF) * torch.tensor([448.0, 449.0, 450.0, 2.0 ** -140]).to(BF)[None, :, None]
    codes, scales = zip(_pools(rng, P, B, H, D), _pools(rng, P, B, H, D, pow2=False))
    scales[0][:, 2:] = 0.0
    _check_write(kn, vn, codes, scales, table, np.zeros(T, np.int32), np.arange(3, T + 3, dtype=np.int32))


@pytest.mark.gpu
def test_write_token_by_token_keeps_earlier_values():
    """A block that grows token by token, each larger than all before: earlier tokens keep their values up to e4m3's
    subnormals under the last scale, and a block that is used again starts anew."""
    rng = np.random.default_rng(4)
    H, D, B = 2, 64, 16
    P = 2
    kc = torch.zeros(P, B, H, D, dtype=torch.uint8, device="cuda")
    vc, ks = kc.clone(), torch.zeros(P, H, device="cuda")
    vs = ks.clone()
    table = np.array([[1]], np.int32)
    rows = _bf16(rng, (B, H, D), (2.0 ** np.arange(B) / 64)[:, None, None])
    ref_c, ref_s = np.zeros((P, B, H, D), np.uint8), np.zeros((P, H))
    first = []
    for t in list(range(B)) + [0]:  # the last one starts the block anew
        x = rows[t:t + 1]
        pa.pa_write_kv_paged_fp8_block(x.cuda(), x.cuda(), kc, vc, ks, vs, _i32(table), _i32([0]), _i32([t]))
        R.write(x.double().numpy(), ref_c, ref_s, [B + t])
        assert np.array_equal(kc.cpu().numpy(), ref_c) and np.array_equal(ks.cpu().numpy().astype(np.float64), ref_s)
        first.append(R.values(ref_c, ref_s)[1, t].copy())
        if t == B - 1:
            v = R.values(ref_c, ref_s)[1]
            step = 2.0 ** -9 * ref_s[1][None, :, None]  # the subnormals' spacing; two roundings of half of it
            for i in range(B):
                assert np.all(np.abs(v[i] - first[i]) <= step[0])
    assert float(ks[1].max()) < 1.0 and torch.equal(vc, kc) and torch.equal(vs, ks)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,B,T", [(8, 128, 16, 200), (1, 16, 1, 9), (3, 48, 5, 77), (2, 64, 64, 1), (5, 112, 1024, 1300)])
def test_read_matches_reference(H, D, B, T, dtype):
    rng = np.random.default_rng(H + D + B + T)
    lens = [T, 1, max(1, T // 2)]
    table, P = _tables(rng, lens, B)
    codes, scales = zip(_pools(rng, P, B, H, D, pow2=dtype == torch.bfloat16), _pools(rng, P, B, H, D))
    codes[0][0, 0, 0, 0] = 0x7f
    seq = rng.integers(0, 3, T).astype(np.int32)
    pos = np.array([rng.integers(0, lens[s]) for s in seq], np.int32)
    if T > 5:
        pos[1], seq[2], pos[4] = -1, 3, 10 ** 6
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    ko = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
    vo = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_read_kv_paged_fp8_block(*pools, _i32(table), _i32(seq), _i32(pos), k_out=ko, v_out=vo, error_count=err)
    slot, nerr = R.slots(table, seq, pos, B, P)
    assert int(err.item()) == nerr
    for out, c, s in ((ko, codes[0], scales[0]), (vo, codes[1], scales[1])):
        want = np.full((T, H, D), 7.0)
        ok = slot >= 0
        want[ok] = R.E4M3[c.reshape(-1, H, D)[slot[ok]]] * s.astype(np.float64)[slot[ok] // B][:, :, None]
        want = torch.from_numpy(want).float().to(dtype)  # one rounding of the exact product (float holds bf16's)
        assert torch.equal(torch.nan_to_num(out.cpu(), nan=99.0), torch.nan_to_num(want, nan=99.0))


# ---------------------------------------------------------------- GPU: attention
def _tol(out, mag, floor):
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -22 * floor + 1e-30


def _close(got, want, mag, floor):
    got = got.float().cpu().double().numpy()
    assert np.all(np.isfinite(got))
    over = np.abs(got - want) / _tol(want, mag, floor)
    assert over.max(initial=0.0) <= 1.0, f"{over.max():.2f} times the tolerance at {np.unravel_index(over.argmax(), over.shape)}"


def _poison(rng, codes, scales, table, lens, B):
    """NaN codes in every slot that holds no token, and NaN or infinite scales for blocks without any."""
    P = codes[0].shape[0]
    held = np.zeros((P, B), bool)
    for s, L in enumerate(lens):
        for j in range(L):
            if 0 <= table[s, j // B] < P:
                held[table[s, j // B], j % B] = True
    for c, s in zip(codes, scales):
        c[~held] = 0x7f
        s[~held.any(axis=1)] = np.array([np.nan, np.inf])[rng.integers(0, 2)]


def _decode_case(lens, Hq, Hkv, D, B, seed, bad=(), scale=None, gain=1.0, max_len=None, pow2=True):
    rng = np.random.default_rng(seed)
    table, P = _tables(rng, lens, B)
    codes, scales = zip(_pools(rng, P, B, Hkv, D, pow2), _pools(rng, P, B, Hkv, D, pow2))
    for s, b, value in bad:
        table[s, b] = value if value < 0 else P + value
    _poison(rng, codes, scales, table, lens, B)
    q = _bf16(rng, (len(lens), Hq, D), gain)
    scale = D ** -0.5 if scale is None else scale
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx = max_len or max(max(lens), 1)
    ws = pa.new_decode_fp8_block_workspace(len(lens), Hq, Hkv, D, B, mx)
    got = pa.pa_decode_fp8_block(q.cuda(), *pools, _i32(table), _i32(lens), mx, scale, ws, error_count=err)
    again = pa.pa_decode_fp8_block(q.cuda(), *pools, _i32(table), _i32(lens), mx, scale, ws, error_count=err)
    assert torch.equal(got, again), "the same call twice"
    s64 = [s.astype(np.float64) for s in scales]
    want, mag, floor = (np.zeros((len(lens), Hq, D)) for _ in range(3))
    for s, L in enumerate(lens):
        want[s:s + 1], mag[s:s + 1] = R.attend_rows(q[s:s + 1].double().numpy(), codes[0], s64[0], codes[1], s64[1],
                                                    table[s], [L], scale)
        floor[s:s + 1] = R.floor_rows(codes[1], s64[1], table[s], [L], Hq)
    _close(got, want, mag, floor)
    return int(err.item())


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,B", [(32, 8, 128, 16), (8, 8, 128, 16), (8, 1, 128, 32), (14, 2, 128, 64),
                                        (6, 2, 128, 8), (10, 2, 128, 128), (32, 2, 128, 16), (8, 2, 64, 16),
                                        (4, 2, 128, 5), (4, 4, 64, 100)])
def test_decode_matches_reference(Hq, Hkv, D, B):
    lens = [1, 0, B, B + 1, 63, 64, 65, 127, 128, 129, 200, 5, 333, 2]
    assert _decode_case(lens, Hq, Hkv, D, B, seed=Hq + Hkv + D + B) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B", [16, 64])
@pytest.mark.parametrize("n", [1, 3])
def test_decode_long_contexts(n, B):
    """Contexts of many partitions, merged; scales that are no powers of two."""
    assert _decode_case([2500, 1, 1025][:n], 8, 2, 128, B, seed=n + B, pow2=False) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B", [16, 100])
def test_decode_bad_pages_are_masked_and_counted(B):
    """Invalid table entries inside a context: negative, past the pool, a whole sequence without any."""
    lens = [300, 40, 16, 129]
    errors = _decode_case(lens, 4, 1, 128, B, seed=B, bad=[(0, 1, -1), (0, 2, 3), (1, 0, -9)] +
                          [(2, b, -1) for b in range(-(-16 // B))])
    assert errors > 0


@pytest.mark.gpu
def test_decode_large_and_small_queries():
    """Queries far from 1, whose scores the softmax scale brings back: the kernel's query terms are scaled by row."""
    assert _decode_case([200, 77], 8, 2, 128, 16, seed=1, gain=1e6, scale=1e-7) == 0
    assert _decode_case([200, 77], 8, 2, 128, 16, seed=2, gain=1e-6, scale=1e5) == 0
    assert _decode_case([200, 77], 8, 2, 128, 16, seed=3, scale=0.0) == 0
    assert _decode_case([200, 77], 8, 2, 128, 16, seed=4, scale=-0.1) == 0


@pytest.mark.gpu
def test_decode_contexts_beyond_the_limit_are_clamped_and_counted():
    rng = np.random.default_rng(5)
    table, P = _tables(rng, [100, 100], 16)
    codes, scales = zip(_pools(rng, P, 16, 2, 128), _pools(rng, P, 16, 2, 128))
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    q = _bf16(rng, (2, 8, 128)).cuda()
    ws = pa.new_decode_fp8_block_workspace(2, 8, 2, 128, 16, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = pa.pa_decode_fp8_block(q, *pools, _i32(table), _i32([100, 64]), 64, 0.1, ws, error_count=err)
    want = pa.pa_decode_fp8_block(q, *pools, _i32(table), _i32([64, 64]), 64, 0.1, ws)
    assert torch.equal(got, want) and int(err.item()) >= 1


def _prefill_case(chunks, Hq, Hkv, D, B, seed, extra=(), bad=(), pow2=True, gain=1.0, scale=None):
    """chunks: (offset, queries); extra: context tokens beyond each chunk's last query."""
    scale = D ** -0.5 if scale is None else scale
    rng = np.random.default_rng(seed)
    lens = [o + n + (extra[c] if c < len(extra) else 0) for c, (o, n) in enumerate(chunks)]
    table, P = _tables(rng, lens, B)
    codes, scales = zip(_pools(rng, P, B, Hkv, D, pow2), _pools(rng, P, B, Hkv, D, pow2))
    for s, b, value in bad:
        table[s, b] = value if value < 0 else P + value
    _poison(rng, codes, scales, table, lens, B)
    order = rng.permutation(len(chunks))  # sequence of chunk c
    table, ctx = table[np.argsort(order)], np.array(lens)[np.argsort(order)]
    cu = np.concatenate([[0], np.cumsum([n for _, n in chunks])])
    q = _bf16(rng, (int(cu[-1]), Hq, D), gain)
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mq, mx = max(max(n for _, n in chunks), 1), max(lens)
    ws = pa.new_prefill_fp8_block_workspace(len(chunks), int(cu[-1]), mq, Hq, Hkv, D, B, mx)
    out = torch.full(q.shape, 5.0, dtype=BF, device="cuda")
    args = (_i32(cu), _i32([o for o, _ in chunks]), _i32(order), mq, *pools, _i32(table), _i32(ctx), mx, scale, ws)
    pa.pa_prefill_chunk_fp8_block(q.cuda(), *args, out=out, error_count=err)
    first = out.clone()
    pa.pa_prefill_chunk_fp8_block(q.cuda(), *args, out=out, error_count=err)
    assert torch.equal(first, out), "the same call twice"
    s64 = [s.astype(np.float64) for s in scales]
    want, mag, floor = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    for c, (o, n) in enumerate(chunks):
        r = slice(int(cu[c]), int(cu[c + 1]))
        want[r], mag[r] = R.attend_rows(q[r].double().numpy(), codes[0], s64[0], codes[1], s64[1], table[order[c]],
                                        [o + i + 1 for i in range(n)], scale)
        floor[r] = R.floor_rows(codes[1], s64[1], table[order[c]], [o + i + 1 for i in range(n)], Hq)
    _close(out, want, mag, floor)
    return int(err.item())


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (2, 2, 128, 32), (4, 2, 128, 64), (8, 1, 128, 128), (6, 2, 128, 8),
                                        (5, 1, 128, 16), (16, 1, 128, 16), (4, 2, 64, 16), (2, 1, 128, 7)])
def test_prefill_matches_reference(Hq, Hkv, D, B):
    chunks = [(0, 1), (0, 40), (17, 33), (130, 7), (0, 0), (255, 2)]
    assert _prefill_case(chunks, Hq, Hkv, D, B, seed=Hq + Hkv + D + B) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,B", [(4, 1, 16), (8, 1, 64), (3, 1, 32)])
def test_prefill_tiles_and_long_offsets(Hq, Hkv, B):
    """Several query tiles and key tiles, a short chunk far into a context (split over keys), odd ends; scales that
    are no powers of two."""
    assert _prefill_case([(3, 200), (900, 3), (1, 129)], Hq, Hkv, 128, B, seed=Hq + B, extra=(9, 70, 0), pow2=False) == 0


@pytest.mark.gpu
def test_prefill_bad_pages_are_masked_and_counted():
    assert _prefill_case([(100, 30), (5, 20)], 4, 1, 128, 16, seed=8, bad=[(0, 0, -1), (0, 3, 2), (1, 0, -1), (1, 1, -1)]) > 0


@pytest.mark.gpu
def test_prefill_large_and_small_queries():
    """Queries far from 1; a softmax scale of 0 and a negative one; scores whose maxima grow late in single rows."""
    chunks = [(60, 70), (0, 35)]
    assert _prefill_case(chunks, 8, 2, 128, 16, seed=21, gain=1e6, scale=1e-7) == 0
    assert _prefill_case(chunks, 8, 2, 128, 16, seed=22, gain=1e-6, scale=1e5) == 0
    assert _prefill_case(chunks, 8, 2, 128, 32, seed=23, scale=0.0) == 0
    assert _prefill_case(chunks, 8, 2, 128, 64, seed=24, scale=-0.1) == 0
    assert _prefill_case([(500, 40)], 4, 1, 128, 8, seed=25, gain=np.exp(np.arange(40) / 12)[:, None, None]) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B", [16, 64])
def test_scales_far_apart(B):
    """Blocks whose scales differ by 2^60: the large ones' values rule, the small ones still count in the softmax."""
    rng = np.random.default_rng(30 + B)
    n, Hq = 400, 4
    table, P = _tables(rng, [n], B)
    codes, scales = zip(_pools(rng, P, B, 1, 128), _pools(rng, P, B, 1, 128))
    scales[1][:] = 2.0 ** rng.choice([-60.0, -3.0, 0.0], (P, 1)).astype(np.float32)
    scales[1][table[0, 1], 0] = 0.0
    scales[0][:] = 2.0 ** -5
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    s64 = [s.astype(np.float64) for s in scales]
    q = _bf16(rng, (3, Hq, 128))
    limits = [n - 2, n - 1, n]
    want, mag = R.attend_rows(q.double().numpy(), codes[0], s64[0], codes[1], s64[1], table[0], limits, 0.05)
    floor = R.floor_rows(codes[1], s64[1], table[0], limits, Hq)
    ws = pa.new_prefill_fp8_block_workspace(1, 3, 3, Hq, 1, 128, B, n)
    out = pa.pa_prefill_chunk_fp8_block(q.cuda(), _i32([0, 3]), _i32([n - 3]), _i32([0]), 3, *pools, _i32(table), _i32([n]),
                                        n, 0.05, ws)
    _close(out, want, mag, floor)
    ws = pa.new_decode_fp8_block_workspace(1, Hq, 1, 128, B, n)
    out = pa.pa_decode_fp8_block(q[2:].cuda(), *pools, _i32(table), _i32([n]), n, 0.05, ws)
    _close(out, want[2:], mag[2:], floor[2:])


@pytest.mark.gpu
@pytest.mark.parametrize("B", [8, 16, 64])
def test_larger_scales_elsewhere_cost_no_precision(B):
    """V scales 2^30 above the others, in a block of little weight and in one that only the last query sees: an output's
    floor is 2^-22 of the largest p_j vs_j among the keys that it sees (see above: the weights are relative to it)."""
    rng = np.random.default_rng(70 + B)
    n, Hq, Q, scale = 5 * 64 + 1, 4, 66, 2.0 ** -5
    table, P = _tables(rng, [n], B)
    codes, scales = zip(_pools(rng, P, B, 1, 128), _pools(rng, P, B, 1, 128))
    scales[0][:] = 2.0 ** -3
    scales[1][table[0, 1], 0] = scales[1][table[0, (n - 1) // B], 0] = 2.0 ** 30
    codes[0][table[0, 1]] = 0xb8  # -1: scores of about -50, for the queries are positive
    scales[0][table[0, 1]] = 16.0
    q = _bf16(rng, (Q, Hq, 128)).abs()
    q[-1] = 0  # every weight alike
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    K, V = (R.E4M3[c[table[0]].reshape(-1, 128)] * np.repeat(s[table[0], 0].astype(np.float64), B)[:, None]
            for c, s in zip(codes, scales))
    vs, code = np.repeat(scales[1][table[0], 0].astype(np.float64), B), np.abs(R.E4M3[codes[1][table[0]].reshape(-1, 128)])
    want, mag, floor = (np.zeros((Q, Hq, 128)) for _ in range(3))
    for i in range(Q):
        N = n - Q + 1 + i
        x = q[i].double().numpy() @ K[:N].T * scale
        w = np.exp(x - x.max(axis=1, keepdims=True))
        w /= w.sum(axis=1, keepdims=True)
        want[i], mag[i] = w @ V[:N], w @ np.abs(V[:N])
        floor[i] = (w * vs[:N]).max(axis=1)[:, None] * code[:N].sum(axis=0)
    assert floor[-2].max() < 2.0 ** 13, "the block of little weight has some after all"
    ws = pa.new_prefill_fp8_block_workspace(1, Q, Q, Hq, 1, 128, B, n)
    out = pa.pa_prefill_chunk_fp8_block(q.cuda(), _i32([0, Q]), _i32([n - Q]), _i32([0]), Q, *pools, _i32(table), _i32([n]),
                                        n, scale, ws)
    _close(out, want, mag, floor)
    for L, i in ((n - 1, Q - 2), (n, Q - 1)):
        ws = pa.new_decode_fp8_block_workspace(1, Hq, 1, 128, B, n)
        out = pa.pa_decode_fp8_block(q[i:i + 1].cuda(), *pools, _i32(table), _i32([L]), n, scale, ws)
        _close(out, want[i:i + 1], mag[i:i + 1], floor[i:i + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,B,n,Q", [(4, 16, 290, 170), (8, 64, 515, 140), (1, 32, 1500, 1400), (4, 5, 290, 170)])
def test_a_nan_reaches_the_queries_that_see_it(Hq, B, n, Q):
    """NaN codes in V of a chunk's own tokens: NaN in their columns for the queries at or after them, nothing for those
    before, whatever tile they share; a NaN code in K likewise, for every column."""
    rng = np.random.default_rng(90 + Hq)
    lens = [n, 200]
    table, P = _tables(rng, lens, B)
    codes, scales = zip(_pools(rng, P, B, 1, 128), _pools(rng, P, B, 1, 128))
    q = _bf16(rng, (Q + 150, Hq, 128))
    nan = np.zeros(q.shape, bool)
    cu, start = [0, Q, Q + 150], [n - Q, 50]
    s64 = [s.astype(np.float64) for s in scales]
    want, mag, floor = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    for c in range(2):
        r, limits = slice(cu[c], cu[c + 1]), [start[c] + i + 1 for i in range(cu[c + 1] - cu[c])]
        want[r], mag[r] = R.attend_rows(q[r].double().numpy(), codes[0], s64[0], codes[1], s64[1], table[c], limits, 0.1)
        floor[r] = R.floor_rows(codes[1], s64[1], table[c], limits, Hq)
    for c, pos, side, dims in ((0, n - 70, 1, [3, 77]), (0, n - 2, 1, [5, 127, 3]), (0, n - 1, 0, [64]), (1, 60, 1, [0]),
                               (1, 140, 1, [1]), (1, 199, 1, list(range(128)))):
        codes[side][table[c, pos // B], pos % B, 0, dims] = 0xff if pos % 2 else 0x7f
        nan[max(cu[c] + pos - start[c], cu[c]):cu[c + 1], :, dims if side else slice(None)] = True
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    for mx in (max(lens), 16384):
        ws = pa.new_prefill_fp8_block_workspace(2, Q + 150, max(Q, 150), Hq, 1, 128, B, mx)
        for _ in range(2):
            out = pa.pa_prefill_chunk_fp8_block(q.cuda(), _i32(cu), _i32(start), _i32([0, 1]), max(Q, 150), *pools,
                                                _i32(table), _i32(lens), mx, 0.1, ws).cpu()
            assert np.array_equal(torch.isnan(out).numpy(), nan)
            _close(out[~torch.from_numpy(nan)], want[~nan], mag[~nan], floor[~nan])


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,D", [(4, 128), (4, 64), (12, 128)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_queries_that_are_not_finite_give_nan(Hq, D, value):
    """The softmax of scores that are infinite or NaN is NaN: for that query and head, and for no other."""
    rng = np.random.default_rng(80 + Hq)
    n, Q, B = 300, 5, 16
    table, P = _tables(rng, [n], B)
    codes, scales = zip(_pools(rng, P, B, 1, D), _pools(rng, P, B, 1, D))
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    q = _bf16(rng, (Q, Hq, D))
    limits = [n - Q + 1 + i for i in range(Q)]
    s64 = [s.astype(np.float64) for s in scales]
    want, mag = R.attend_rows(q.double().numpy(), codes[0], s64[0], codes[1], s64[1], table[0], limits, 0.1)
    floor = R.floor_rows(codes[1], s64[1], table[0], limits, Hq)
    q[1, 2, 17] = q[4, 0, D - 1] = value
    hit = np.zeros((Q, Hq), bool)
    hit[1, 2] = hit[4, 0] = True
    for spans in (True, False):  # a limit of one key tile leaves nothing to cut
        mx = 4096 if spans else n
        ws = pa.new_prefill_fp8_block_workspace(1, Q, Q, Hq, 1, D, B, mx)
        out = pa.pa_prefill_chunk_fp8_block(q.cuda(), _i32([0, Q]), _i32([n - Q]), _i32([0]), Q, *pools, _i32(table), _i32([n]),
                                            mx, 0.1, ws)
        assert bool(torch.isnan(out.cpu()[hit]).all())
        _close(out.cpu()[~hit], want[~hit], mag[~hit], floor[~hit])
    ws = pa.new_decode_fp8_block_workspace(1, Hq, 1, D, B, n)
    out = pa.pa_decode_fp8_block(q[4:].cuda(), *pools, _i32(table), _i32([n]), n, 0.1, ws)
    assert bool(torch.isnan(out.cpu()[hit[4:]]).all())
    _close(out.cpu()[~hit[4:]], want[4:][~hit[4:]], mag[4:][~hit[4:]], floor[4:][~hit[4:]])


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,B", [(8, 16), (2, 64)])
def test_pools_beyond_32_bit_offsets(Hkv, B):
    """Blocks at the end of pools of more than 2^32 codes give what the same blocks give in a small pool, bit for bit."""
    rng = np.random.default_rng(100 + B)
    D, Hq, n = 128, 4 * Hkv, 1200
    P = (1 << 32) // (B * Hkv * D) + 200
    used = -(-n // B)
    small = torch.from_numpy(rng.permutation(used + 2)[:used].astype(np.int32)).reshape(1, -1).cuda()
    far = small + (P - used - 2)
    T = n
    k, v = _bf16(rng, (T, Hkv, D)).cuda(), _bf16(rng, (T, Hkv, D)).cuda()
    seq, pos = _i32([0] * T), _i32(range(T))
    q = _bf16(rng, (50, Hq, D)).cuda()
    got = []
    for table, blocks in ((small, used + 2), (far, P)):
        kc, vc = (torch.zeros(blocks, B, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(blocks, Hkv, device="cuda") for _ in range(2))
        for a, b in ((0, 700), (700, T)):  # both forms of the write
            pa.pa_write_kv_paged_fp8_block(k[a:b], v[a:b], kc, vc, ks, vs, table, seq[a:b], pos[a:b])
        ws = pa.new_write_fp8_block_workspace(T, blocks, B)
        pa.pa_write_kv_paged_fp8_block(k, v, kc, vc, ks, vs, table, seq, pos, ws)
        outs = list(pa.pa_read_kv_paged_fp8_block(kc, vc, ks, vs, table, seq, pos))
        ws = pa.new_decode_fp8_block_workspace(1, Hq, Hkv, D, B, n)
        outs.append(pa.pa_decode_fp8_block(q[:1], kc, vc, ks, vs, table, _i32([n]), n, 0.1, ws))
        ws = pa.new_prefill_fp8_block_workspace(1, 50, 50, Hq, Hkv, D, B, n)
        outs.append(pa.pa_prefill_chunk_fp8_block(q, _i32([0, 50]), _i32([n - 50]), _i32([0]), 50, kc, vc, ks, vs, table,
                                                  _i32([n]), n, 0.1, ws))
        got.append([o.cpu() for o in outs])
        assert int(torch.count_nonzero(ks)) == used * Hkv
        del kc, vc
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool(torch.isfinite(got[0][3]).all()) and float(got[0][3].abs().max()) > 0


# ---------------------------------------------------------------- GPU: together
@pytest.mark.gpu
def test_write_then_prefill_then_decode_then_read():
    """A prompt in two chunks, then decode steps, as a serving loop makes them; the attention sees what the read back
    gives, and every value is within e4m3's half step (2^-4) of what was written, or the scale's smallest step."""
    rng = np.random.default_rng(9)
    Hq, Hkv, D, B, n = 8, 2, 128, 16, 75
    table, P = _tables(rng, [n + 5], B)
    kc = torch.zeros(P, B, Hkv, D, dtype=torch.uint8, device="cuda")
    vc = torch.full_like(kc, 0x7f)
    ks, vs = torch.zeros(P, Hkv, device="cuda"), torch.full((P, Hkv), 1e30, device="cuda")
    bt, kn, vn, q = _i32(table), _bf16(rng, (n + 5, Hkv, D)), _bf16(rng, (n + 5, Hkv, D), 3.0), _bf16(rng, (n + 5, Hq, D))
    outs = []
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for a, b in [(0, 50), (50, n)] + [(t, t + 1) for t in range(n, n + 5)]:
        T = b - a
        pa.pa_write_kv_paged_fp8_block(kn[a:b].cuda(), vn[a:b].cuda(), kc, vc, ks, vs, bt, _i32([0] * T),
                                       _i32(np.arange(a, b)), error_count=err)
        x = q[a:b].cuda()
        if T > 1:
            ws = pa.new_prefill_fp8_block_workspace(1, T, T, Hq, Hkv, D, B, b)
            outs.append(pa.pa_prefill_chunk_fp8_block(x, _i32([0, T]), _i32([a]), _i32([0]), T, kc, vc, ks, vs, bt,
                                                      _i32([b]), b, D ** -0.5, ws, error_count=err))
        else:
            ws = pa.new_decode_fp8_block_workspace(1, Hq, Hkv, D, B, b)
            outs.append(pa.pa_decode_fp8_block(x, kc, vc, ks, vs, bt, _i32([b]), b, D ** -0.5, ws, error_count=err))
        k, v = pa.pa_read_kv_paged_fp8_block(kc, vc, ks, vs, bt, _i32([0] * b), _i32(np.arange(b)),
                                             dtype=torch.float32, error_count=err)
        k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
        want, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
        floor = R.floor_rows(vc.cpu().numpy(), vs.cpu().double().numpy(), table[0], list(range(a + 1, b + 1)), Hq)
        for i in range(T):
            for h in range(Hkv):
                g = slice(h * 4, h * 4 + 4)
                want[i, g], mag[i, g] = R.attend(q[a + i, g].double().numpy(), k[:a + i + 1, h], v[:a + i + 1, h], D ** -0.5)
        _close(outs[-1], want, mag, floor)
    assert int(err.item()) == 0
    for new, got, s in ((kn, k, ks), (vn, v, vs)):
        x = new.double().numpy()
        small = 2.0 ** -9 * s.cpu().double().numpy()[table[0, np.arange(n + 5) // B]][:, :, None]
        assert np.all(np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + small)


def _step_expected(w):
    """(slots, K codes, V codes, K scales, V scales, decode, prefill with magnitudes and floors) of a step."""
    table = w.block_tables.numpy()
    slot, err = R.slots(table, w.seq_idx.numpy(), w.pos.numpy(), w.block_size, w.num_blocks)
    assert err == 0
    pools = []
    for new, c, s in ((w.k_new, w.k_cache, w.k_scales), (w.v_new, w.v_cache, w.v_scales)):
        c, s = c.numpy().copy(), s.double().numpy()
        R.write(new.double().numpy(), c, s, slot)
        pools.append((c, s))
    (kc, ks), (vc, vs) = pools
    ctx = w.context_lens.numpy()

    def rows(q, s, limits):
        out, mag = R.attend_rows(q.double().numpy(), kc, ks, vc, vs, table[s], limits, w.scale)
        return out, mag, R.floor_rows(vc, vs, table[s], limits, w.num_q_heads)

    dec = [rows(w.q_decode[s:s + 1], s, [int(ctx[s])]) for s in range(w.num_decode)]
    pre = []
    for c in range(w.num_chunks):
        a, b, start = int(w.cu_q_lens[c]), int(w.cu_q_lens[c + 1]), int(w.q_start_pos[c])
        pre.append(rows(w.q_prefill[a:b], int(w.seq_of_chunk[c]), [start + i + 1 for i in range(b - a)]))
    cat = lambda parts: [np.concatenate(x) for x in zip(*parts)]  # noqa: E731
    return slot, kc, vc, ks, vs, cat(dec) if dec else None, cat(pre) if pre else None


def test_as_fp8_block_draws_scales_for_every_block_and_head():
    w = W.as_fp8_block(W.small("mixed_bf16"), 0)
    assert w.kv_fp8 and w.k_cache.dtype == torch.uint8 and tuple(w.k_scales.shape) == (w.num_blocks, w.num_kv_heads)
    assert w.num_chunks > 0 and w.k_scales.dtype == torch.float32 and not torch.equal(w.k_scales, w.v_scales)
    assert torch.equal(torch.exp2(torch.log2(w.v_scales).round()), w.v_scales)
    again = W.as_fp8_block(W.small("mixed_bf16"), 0)
    assert torch.equal(w.k_scales, again.k_scales) and torch.equal(w.v_cache, again.v_cache)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["eager", "graph", "host"])
def test_device_step_over_block_scaled_pools(how):
    """Write, decode and prefill as DeviceStep runs them: eagerly, as a captured graph replayed twice, and from pinned
    host memory; a continuous-batching step of decode sequences and chunks."""
    w = W.as_fp8_block(W.mixed_bf16(3, num_decode=5, num_chunks=2, chunk_len=40, max_off=200), 3)
    w.context_lens[:5] = torch.clamp(w.context_lens[:5], max=300)
    w.pos[:5] = w.context_lens[:5] - 1
    slot, kc, vc, ks, vs, dec, pre = _step_expected(w)
    st = DeviceStep(w)
    assert st.block_scales and not st.fused_decode_write
    if how == "eager":
        st.run()
    elif how == "graph":
        first = [t.clone() for t in st.run()]
        st.capture()
        for _ in range(2):
            st.out_decode.zero_()
            st.out_prefill.zero_()
            st.replay()
            assert all(torch.equal(a, b) for a, b in zip(first, (st.out_decode, st.out_prefill)))
    else:
        hin, hout = st.pinned_inputs(), st.pinned_outputs()
        st.run_from_host(hin, hout)
        torch.cuda.synchronize()
        st.capture_from_host(hin, hout)
        hout.zero_()
        st.run_from_host(hin, hout)
        torch.cuda.synchronize()
        st.out_decode, st.out_prefill = (t.cuda() for t in st.output_views(hout))
    torch.cuda.synchronize()
    assert st.errors() == 0
    assert np.array_equal(st.slots.cpu().numpy(), slot)
    assert np.array_equal(st.k_cache.cpu().numpy(), kc) and np.array_equal(st.v_cache.cpu().numpy(), vc)
    assert np.array_equal(st.k_scales.double().cpu().numpy(), ks) and np.array_equal(st.v_scales.double().cpu().numpy(), vs)
    _close(st.out_decode, *dec)
    _close(st.out_prefill, *pre)


@pytest.mark.gpu
def test_calls_on_another_stream_and_without_workspace():
    """A stream given by the caller; a workspace that is too small or absent is refused."""
    rng = np.random.default_rng(12)
    table, P = _tables(rng, [2000], 16)
    codes, scales = zip(_pools(rng, P, 16, 1, 128), _pools(rng, P, 16, 1, 128))
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    q, bt, ctx = _bf16(rng, (1, 4, 128)).cuda(), _i32(table), _i32([2000])
    ws = pa.new_decode_fp8_block_workspace(1, 4, 1, 128, 16, 2000)
    want = pa.pa_decode_fp8_block(q, *pools, bt, ctx, 2000, 0.1, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pa.pa_decode_fp8_block(q, *pools, bt, ctx, 2000, 0.1, ws, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    for bad in (None, ws[:256]):
        with pytest.raises(pa.PaError, match="workspace"):
            pa.pa_decode_fp8_block(q, *pools, bt, ctx, 2000, 0.1, bad)
    cu, z = _i32([0, 1]), _i32([0])
    pws = pa.new_prefill_fp8_block_workspace(1, 1, 1, 4, 1, 128, 16, 2000)
    assert pws is not None  # one query, 16 key tiles: cut into spans
    args = (q, cu, _i32([1999]), z, 1, *pools, bt, ctx, 2000, 0.1)
    a = pa.pa_prefill_chunk_fp8_block(*args, workspace=pws)
    assert float((a.float() - want.float()).abs().max()) <= 2.0 ** -6 * float(want.float().abs().max())
    with pytest.raises(pa.PaError, match="workspace"):
        pa.pa_prefill_chunk_fp8_block(*args)
    new = torch.zeros(1500, 1, 128, dtype=BF, device="cuda")
    with pytest.raises(pa.PaError, match="workspace"):
        pa.pa_write_kv_paged_fp8_block(new, new, *pools, bt, _i32([0] * 1500), _i32(np.arange(1500)))


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_two_streams_at_once(captured):
    """Two sequences of calls on two streams, each with its own pools and workspaces, give what they give one after the
    other, bit for bit; the same captured into a graph each and replayed at once."""
    B, Hkv, Hq, D, rounds = 16, 2, 8, 128, 6

    def job(seed):
        rng = np.random.default_rng(seed)
        lens = [1500 + seed, 40, 700]
        table, P = _tables(rng, lens, B)
        T = sum(lens)
        k, v = _bf16(rng, (T, Hkv, D)).cuda(), _bf16(rng, (T, Hkv, D)).cuda()
        seq, pos = _i32(np.repeat(range(3), lens)), _i32(np.concatenate([np.arange(L) for L in lens]))
        bt, ctx, n = _i32(table), _i32(lens), max(lens)
        q, qd = _bf16(rng, (90, Hq, D)).cuda(), _bf16(rng, (3, Hq, D)).cuda()
        kc, vc = (torch.zeros(P, B, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(P, Hkv, device="cuda") for _ in range(2))
        ww, wd = pa.new_write_fp8_block_workspace(T, P, B), pa.new_decode_fp8_block_workspace(3, Hq, Hkv, D, B, n)
        wp = pa.new_prefill_fp8_block_workspace(1, 90, 90, Hq, Hkv, D, B, n)
        cu, start, which = _i32([0, 90]), _i32([lens[0] - 90]), _i32([0])
        outs = [torch.zeros(3, Hq, D, dtype=BF, device="cuda"), torch.zeros(90, Hq, D, dtype=BF, device="cuda"),
                torch.zeros(T, Hkv, D, dtype=BF, device="cuda"), torch.zeros(T, Hkv, D, dtype=BF, device="cuda")]

        def run():
            pa.pa_write_kv_paged_fp8_block(k, v, kc, vc, ks, vs, bt, seq, pos, ww)
            pa.pa_decode_fp8_block(qd, kc, vc, ks, vs, bt, ctx, n, 0.1, wd, out=outs[0])
            pa.pa_prefill_chunk_fp8_block(q, cu, start, which, 90, kc, vc, ks, vs, bt, ctx, n, 0.1, wp, out=outs[1])
            pa.pa_read_kv_paged_fp8_block(kc, vc, ks, vs, bt, seq, pos, k_out=outs[2], v_out=outs[3])
        return run, outs

    jobs = [job(1), job(2)]
    want = []
    for run, outs in jobs:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        assert all(bool(torch.isfinite(o).all()) and int(torch.count_nonzero(o)) for o in outs)
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    if captured:
        for (run, _), st in zip(jobs, streams):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=st):
                run()
    for _ in range(rounds):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                graphs[i].replay() if captured else jobs[i][0]()
    torch.cuda.synchronize()
    for (_, outs), w in zip(jobs, want):
        for o, x in zip(outs, w):
            assert torch.equal(o, x)


@pytest.mark.gpu
def test_empty_calls():
    kc = torch.zeros(4, 16, 2, 128, dtype=torch.uint8, device="cuda")
    sc, i0 = torch.zeros(4, 2, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    bt = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, 2, 128, dtype=BF, device="cuda")
    pa.pa_write_kv_paged_fp8_block(none, none, kc, kc.clone(), sc, sc.clone(), bt, i0, i0)
    k, v = pa.pa_read_kv_paged_fp8_block(kc, kc, sc, sc, bt, i0, i0)
    assert k.shape == (0, 2, 128) and v.dtype == BF
    q = torch.zeros(0, 4, 128, dtype=BF, device="cuda")
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    assert pa.pa_decode_fp8_block(q, kc, kc, sc, sc, bt[:0], i0, 16, 1.0, ws).numel() == 0
    out = pa.pa_prefill_chunk_fp8_block(q, torch.zeros(1, dtype=torch.int32, device="cuda"), i0, i0, 0, kc, kc, sc, sc, bt,
                                        torch.ones(1, dtype=torch.int32, device="cuda"), 16, 1.0)
    assert out.numel() == 0
    # all contexts empty: zeros, whatever the pools hold
    q = torch.ones(3, 4, 128, dtype=BF, device="cuda")
    nan = torch.full_like(kc, 0x7f)
    out = pa.pa_decode_fp8_block(q, nan, nan, sc * float("nan"), sc, bt.expand(3, 4).contiguous(),
                                 torch.zeros(3, dtype=torch.int32, device="cuda"), 0, 1.0, ws)
    assert int(torch.count_nonzero(out)) == 0


@pytest.mark.gpu
def test_decode_of_more_sequences_than_one_launch_takes():
    """1100 short sequences: the call cuts the batch into launches of 512."""
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(0, 40, 1100)]
    assert _decode_case(lens, 4, 1, 128, 16, seed=14) == 0


@pytest.mark.gpu
def test_prefill_rows_outside_the_chunks_are_left():
    """Chunk descriptors that make no sense are counted, and their rows keep what they held; so do rows of no chunk."""
    rng = np.random.default_rng(15)
    table, P = _tables(rng, [64, 64], 16)
    codes, scales = zip(_pools(rng, P, 16, 1, 128), _pools(rng, P, 16, 1, 128))
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    q = _bf16(rng, (30, 4, 128)).cuda()
    out = torch.full_like(q, 5.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.new_prefill_fp8_block_workspace(3, 30, 10, 4, 1, 128, 16, 64)
    pa.pa_prefill_chunk_fp8_block(q, _i32([0, 10, 20, 25]), _i32([3, -1, 7]), _i32([0, 1, 2]), 10, *pools, _i32(table),
                                  _i32([64, 64]), 64, 0.1, ws, out=out, error_count=err)
    assert int(err.item()) >= 2  # chunk 1 starts before 0, chunk 2 names no sequence
    assert torch.all(out[10:] == 5.0) and not torch.any(torch.all((out[:10] == 5.0).flatten(1), dim=1))


@pytest.mark.gpu
def test_read_back_then_bf16_prefill_agrees():
    """The read back's rows, written into bf16 pools, give the existing prefill the values the e4m3 prefill sees."""
    rng = np.random.default_rng(16)
    n, T = 300, 50
    table, P = _tables(rng, [n], 16)
    codes, scales = zip(_pools(rng, P, 16, 2, 128), _pools(rng, P, 16, 2, 128))
    pools = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (*codes, *scales)]
    bt, seq, pos = _i32(table), _i32([0] * n), _i32(np.arange(n))
    k, v = pa.pa_read_kv_paged_fp8_block(*pools, bt, seq, pos)
    kb, vb = (torch.zeros(P, 16, 2, 128, dtype=BF, device="cuda") for _ in range(2))
    pa.pa_write_kv_paged(k, v, kb, vb, bt, seq, pos)
    q = _bf16(rng, (T, 8, 128)).cuda()
    cu, st, so, ctx = _i32([0, T]), _i32([n - T]), _i32([0]), _i32([n])
    want = pa.pa_prefill_chunk(q, cu, st, so, T, kb, vb, bt, ctx, 128 ** -0.5)
    ws = pa.new_prefill_fp8_block_workspace(1, T, T, 8, 2, 128, 16, n)
    got = pa.pa_prefill_chunk_fp8_block(q, cu, st, so, T, *pools, bt, ctx, n, 128 ** -0.5, ws)
    # the bf16 prefill takes 2^x of bf16-rounded exponents: with x up to 2^4 from the maximum, off by 2^-5 relative
    mag = float(v.float().abs().max())
    assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -4 * mag
