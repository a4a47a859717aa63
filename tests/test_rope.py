"""Rotary positions with several axes, alone and with the paged write."""
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


def _rows(rng, shape, dtype):
    return torch.tensor(rng.standard_normal(shape), dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32)


def _freq(half, theta=1e4):
    return (theta ** (-np.arange(half) / max(half, 1))).astype(np.float32)


def _near(got, want, mag, dtype):
    """cos and sin are off by less than 2^-22 (the angle's own rounding pi 2^-25, two units in the last place of sincospi),
    each of two products and their sum by 2^-24 of its size: 2^-21 of |a| + |b| together; then one rounding."""
    got = got.double().cpu().numpy()
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) + mag * 2.0 ** -21 * (1 + 2.0 ** -8)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)


# dtype, T, Hq, Hkv, D, rot, axes, interleaved
SHAPES = [
    (BF16, 1, 4, 1, 128, 128, 1, False),
    (BF16, 37, 32, 8, 128, 128, 3, False),
    (BF16, 65, 6, 2, 128, 64, 3, True),
    (F32, 9, 4, 4, 64, 64, 2, False),
    (F32, 5, 3, 1, 64, 32, 3, True),
    (BF16, 7, 3, 1, 80, 80, 3, False),   # pairs that no 16-byte piece holds
    (F32, 3, 2, 2, 10, 6, 2, True),
    (BF16, 4, 1, 1, 24, 24, 1, False),
    (BF16, 2, 2, 1, 64, 0, 1, False),    # nothing turns
    (BF16, 3, 40, 20, 256, 256, 4, False),
]


def _case(rng, dtype, T, Hq, Hkv, D, rot, axes):
    qkv = _rows(rng, (T, Hq + 2 * Hkv, D), dtype)
    pos = rng.integers(-5, 5000, (axes, T))
    pos[:, 0] = 2 ** 31 - 1 - np.arange(axes)
    if T > 1:
        pos[:, 1] = -2 ** 31
    axis = rng.integers(0, axes, rot // 2)
    return qkv, pos, _freq(rot // 2), axis


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope(shape):
    dtype, T, Hq, Hkv, D, rot, axes, inter = shape
    rng = np.random.default_rng(T)
    qkv, pos, freq, axis = _case(rng, dtype, T, Hq, Hkv, D, rot, axes)
    dev = qkv.cuda()
    q, k = dev[:, :Hq], dev[:, Hq:Hq + Hkv]
    args = (_i32(pos).cuda(), torch.tensor(freq).cuda(), _i32(axis).cuda())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = pa.pa_rope(q, k, *args, interleaved=inter, error_count=err)
    for got, x in ((qo, q), (ko, k)):
        want, mag = ref.turn(x.double().cpu().numpy(), pos, freq, axis, inter)
        _near(got, want, mag, dtype)
    assert int(err) == 0 and torch.equal(dev.cpu(), qkv)
    # in place
    qc, kc = q.contiguous(), k.contiguous()
    pa.pa_rope(qc, kc, *args, interleaved=inter, q_out=qc, k_out=kc)
    assert torch.equal(qc, qo) and torch.equal(kc, ko)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("block", [1, 16, 24])
def test_rope_write(shape, block):
    dtype, T, Hq, Hkv, D, rot, axes, inter = shape
    rng = np.random.default_rng(T + 1)
    qkv, rope_pos, freq, axis = _case(rng, dtype, T, Hq, Hkv, D, rot, axes)
    S, width, P = 3, -(-(T + 8) // block), 0
    P = S * width + 2
    table = rng.permutation(P)[:S * width].reshape(S, width)
    seq = rng.integers(0, S, T)
    pos = np.zeros(T, np.int64)
    for s in range(S):
        pos[seq == s] = rng.permutation(width * block)[:(seq == s).sum()]
    bad = []
    if T > 6:
        pos[2] = -1                 # padding
        seq[3] = S                  # no such sequence
        pos[4] = width * block + 3  # beyond the table
        table[seq[5], pos[5] // block] = P
        bad = [t for t in range(T) if t in (3, 4) or (seq[t] == seq[5] and pos[t] // block == pos[5] // block and t != 2)]
    slots, _ = _slots(table, seq, pos, block, P)
    key_w = width * block
    dev = qkv.cuda()
    kc, vc = (torch.full((P, block, Hkv, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    weights = torch.full((S, Hkv, key_w), 3.0, device="cuda")
    places = torch.full((S, Hkv, key_w), -9, dtype=torch.int32, device="cuda")
    token = rng.integers(0, 10 ** 6, T)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.full((T, Hq, D), 5.0, dtype=dtype, device="cuda")
    got_slots = torch.empty(T, dtype=torch.int64, device="cuda")
    r = pa.pa_rope_write_kv_paged(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], _i32(rope_pos).cuda(),
                                  torch.tensor(freq).cuda(), _i32(axis).cuda(), kc, vc, _i32(table).cuda(),
                                  _i32(seq).cuda(), _i32(pos).cuda(), interleaved=inter, q_out=qo, key_weights=weights,
                                  key_pos=places, token_pos=_i32(token).cuda(), slot_mapping=got_slots, error_count=err)
    assert r is qo
    x = qkv.double().numpy()
    live = pos >= 0
    want, mag = ref.turn(x, rope_pos, freq, axis, inter)
    _near(qo[torch.tensor(live)], want[live, :Hq], mag[live, :Hq], dtype)
    assert torch.all(qo[torch.tensor(~live)] == 5.0)
    assert np.array_equal(got_slots.cpu().numpy(), slots) and int(err) == len(bad)
    k, v = kc.view(-1, Hkv, D).cpu(), vc.view(-1, Hkv, D).cpu()
    w_want, p_want = np.full((S, Hkv, key_w), 3.0), np.full((S, Hkv, key_w), -9)
    stored = slots >= 0
    _near(k[slots[stored]], want[stored, Hq:Hq + Hkv], mag[stored, Hq:Hq + Hkv], dtype)
    assert torch.equal(v[slots[stored]], qkv[torch.tensor(stored), Hq + Hkv:])
    others = np.setdiff1d(np.arange(P * block), slots[stored])
    assert torch.all(k[others] == 7.0) and torch.all(v[others] == 7.0)
    for t in np.flatnonzero(stored):
        w_want[seq[t], :, pos[t]], p_want[seq[t], :, pos[t]] = 0.0, token[t]
    assert np.array_equal(weights.cpu().numpy(), w_want) and np.array_equal(places.cpu().numpy(), p_want)


def _slots(table, seq, pos, block, P):
    out, errors = [], 0
    for s, p in zip(seq, pos):
        slot = -1
        if p >= 0:
            ok = 0 <= s < table.shape[0] and p // block < table.shape[1]
            b = table[s, p // block] if ok else -1
            if 0 <= b < P:
                slot = int(b) * block + p % block
            else:
                errors += 1
        out.append(slot)
    return np.array(out, np.int64), errors


@pytest.mark.gpu
def test_rope_write_beyond_the_key_rows_is_an_invalid_index():
    rng = np.random.default_rng(3)
    qkv = _rows(rng, (2, 3, 64), BF16).cuda()
    kc, vc = (torch.zeros(2, 16, 1, 64, dtype=BF16, device="cuda") for _ in range(2))
    weights, places = torch.ones(1, 1, 8, device="cuda"), torch.ones(1, 1, 8, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_rope_write_kv_paged(qkv[:, :1], qkv[:, 1:2], qkv[:, 2:], _i32([3, 4]).cuda(), torch.ones(32).cuda(), None, kc, vc,
                              _i32([[0, 1]]).cuda(), _i32([0, 0]).cuda(), _i32([7, 8]).cuda(), key_weights=weights,
                              key_pos=places, error_count=err)
    assert int(err) == 1 and torch.all(kc[0, 8:] == 0) and bool(kc[0, 7].abs().sum() > 0)
    assert weights.cpu().tolist() == [[[1.0] * 7 + [0.0]]] and places.cpu().tolist() == [[[1] * 7 + [7]]]


@pytest.mark.gpu
def test_rope_unknown_axis_and_frequencies():
    """A pair of an unknown axis stays as it is and is counted; an infinite frequency gives NaN; a negative one turns back;
    frequencies of several turns per position, and subnormal ones, are taken as they are."""
    x = torch.randn(3, 1, 16, device="cuda")
    freq = np.array([1.0, np.inf, -0.5, 100.0, 1e-40, 3.0, np.nan, 2.5e7], np.float32)
    axis = np.array([1, 0, 0, 0, 0, 5, 0, 0])
    pos = np.array([[1, 1000, 123456], [7, 8, -9]])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, _ = pa.pa_rope(x, x, _i32(pos).cuda(), torch.tensor(freq).cuda(), _i32(axis).cuda(), error_count=err)
    assert int(err) == 3
    got = got.cpu()
    for i in (1, 6):
        assert torch.isnan(got[..., [i, 8 + i]]).all()
    assert torch.equal(got[..., [5, 13]], x.cpu()[..., [5, 13]])
    fine = [0, 2, 3, 4, 7]
    cols = fine + [8 + i for i in fine]
    want, mag = ref.turn(x.double().cpu().numpy()[..., cols], pos, freq[fine], axis[fine], False)
    # (the last frequency: 3e12 rad, of which 64 bits hold 2^-11; the library's count of turns is exact to 2^-32 of one)
    slack = np.array([0, 0, 0, 0, 1e-2] * 2) * mag
    diff = np.abs(got[..., cols].double().numpy() - want)
    assert np.all(diff <= 2.0 ** -24 * np.abs(want) + 2.0 ** -21 * mag + slack)


@pytest.mark.gpu
def test_rope_on_a_stream_and_in_a_graph():
    rng = np.random.default_rng(5)
    q, k = _rows(rng, (33, 4, 128), BF16).cuda(), _rows(rng, (33, 2, 128), BF16).cuda()
    pos, freq = _i32(rng.integers(0, 4000, (2, 33))).cuda(), torch.tensor(_freq(64)).cuda()
    axis = _i32(np.arange(64) % 2).cuda()
    want = pa.pa_rope(q, k, pos, freq, axis)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pa.pa_rope(q, k, pos, freq, axis, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = pa.pa_rope(q, k, pos, freq, axis)
    q.copy_(-q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], -want[0]) and torch.equal(got[1], want[1])


def test_rope_refusals():
    q, k = torch.zeros(2, 4, 64), torch.zeros(2, 1, 64)
    pos, freq = _i32([0, 1]), torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope(q, k, pos, freq)
    with pytest.raises(TypeError, match="unsupported dtype"):
        pa.pa_rope(q.half(), k.half(), pos, freq)
    with pytest.raises(ValueError, match="disagree"):
        pa.pa_rope(q, k[:1], pos, freq)
    with pytest.raises(ValueError, match="contiguous"):
        pa.pa_rope(q.transpose(1, 2), k, pos, freq)
    L = pa.lib()

    def rope(T=2, Hq=4, Hkv=1, D=64, dtype=pa.PA_F32, axes=1, rot=64, ptr=0):
        return L.pa_rope(ptr, ptr, ptr, ptr, T, Hq, Hkv, D, dtype, 0, 0, ptr, axes, ptr, None, rot, 0, None, None)

    assert rope(T=0) == pa.PA_OK
    assert rope() == pa.PA_ERR_INVALID_ARG  # no pointers
    for bad in (dict(T=-1), dict(rot=63), dict(rot=66), dict(axes=0), dict(D=0), dict(Hq=-1)):
        assert rope(**bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=5), dict(D=2048, rot=64), dict(Hq=1 << 20)):
        assert rope(**bad) == pa.PA_ERR_UNSUPPORTED, bad


def test_rope_write_refusals():
    L = pa.lib()

    def write(T=2, Hq=4, Hkv=1, D=64, P=2, B=16, kw=None, kp=None, width=0):
        return L.pa_rope_write_kv_paged(None, None, None, None, T, Hq, Hkv, D, pa.PA_BF16, 0, 0, 0, None, 1, None, None, D,
                                        0, None, None, P, B, None, 1, 1, None, None, kw, kp, width, None, None, None, None)

    assert write(T=0) == pa.PA_OK
    assert write() == pa.PA_ERR_INVALID_ARG
    for bad in (dict(T=0, Hkv=0), dict(T=0, B=0), dict(T=0, kw=256), dict(T=0, kw=256, kp=256), dict(T=0, width=-1)):
        assert write(**bad) == pa.PA_ERR_INVALID_ARG, bad
    q, k = torch.zeros(2, 4, 64), torch.zeros(2, 1, 64)
    pool = torch.zeros(2, 16, 1, 64)
    args = (_i32([0, 1]), torch.ones(32), None, pool, pool, _i32([[0, 1]]), _i32([0, 0]), _i32([0, 1]))
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope_write_kv_paged(q, k, k, *args)
    with pytest.raises(ValueError, match="together"):
        pa.pa_rope_write_kv_paged(q, k, k, *args, key_weights=torch.zeros(1, 1, 32))
    with pytest.raises(ValueError, match="num_kv_heads, width"):
        pa.pa_rope_write_kv_paged(q, k, k, *args, key_weights=torch.zeros(2, 1, 32),
                                  key_pos=torch.zeros(2, 1, 32, dtype=torch.int32))
    with pytest.raises(ValueError, match="rope_pos"):
        pa.pa_rope_write_kv_paged(q, k, k, _i32([0]), *args[1:])
