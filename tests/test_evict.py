"""Eviction by accumulated attention weight, and a whole serving loop with it."""
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


# dtype, Hkv, D, B, lengths, budget, keep_first, keep_recent, kind of weights
CASES = [
    (BF16, 2, 128, 16, [40, 16, 17, 0, 1, 100], 16, 2, 4, "random"),
    (BF16, 8, 128, 16, [1100, 513, 2000], 512, 4, 64, "random"),
    (BF16, 1, 64, 32, [2064] * 3, 2048, 4, 128, "random"),
    (F32, 2, 128, 8, [300], 299, 0, 0, "random"),
    (F32, 1, 4, 1, [90, 700], 1, 0, 1, "random"),
    (BF16, 1, 8, 24, [500, 450], 100, 0, 0, "equal"),     # only ties
    (BF16, 2, 64, 16, [800, 640], 320, 3, 7, "few"),      # few values, many ties across the threshold
    (BF16, 2, 64, 16, [800, 640], 320, 3, 7, "special"),  # infinities, NaN, both zeros, negatives, subnormals
    (BF16, 1, 64, 16, [100, 200], 64, 64, 0, "random"),   # all of the budget protected
    (BF16, 1, 64, 16, [100, 200], 64, 0, 64, "random"),
    (BF16, 2, 64, 16, [200, 300], 64, 10, 20, "places"),  # places that make more than the budget protected
    (BF16, 1, 64, 16, [6000, 9000], 3000, 4, 50, "few"),        # thousands of equal weights
    (BF16, 2, 64, 16, [9000, 5000], 4500, 0, 0, "special"),
    (BF16, 1, 64, 16, [1000, 1128, 1129], 1000, 2, 30, "random"),  # up to 129 moves
    (BF16, 1, 64, 64, [45000, 41000], 1000, 4, 100, "random"),  # longer than the keys held in shared memory
]


def _weights(rng, kind, shape):
    if kind == "equal":
        return np.full(shape, 0.25, np.float32)
    if kind == "few":
        return rng.integers(0, 4, shape).astype(np.float32)
    if kind == "special":
        return rng.choice(np.array([np.inf, -np.inf, np.nan, -np.nan, 0.0, -0.0, 1e-42, -1e-42, 1.5, -2.0, 3e38], np.float32),
                          shape)
    return np.exp(2 * rng.standard_normal(shape)).astype(np.float32)


def _case(case, seed=0):
    dtype, Hkv, D, B, lens, budget, first, recent, kind = case
    rng = np.random.default_rng(seed + D + len(lens) + budget)
    count = [-(-n // B) for n in lens]
    P, S, width = sum(count) + 3, len(lens), max(count) + 1
    order, at = rng.permutation(P), 0
    table = np.full((S, width), -1)
    for s in range(S):
        table[s, :count[s]] = order[at:at + count[s]]
        at += count[s]
    k, v = (torch.tensor(rng.standard_normal((P, B, Hkv, D)), dtype=torch.float32).to(dtype) for _ in range(2))
    w = _weights(rng, kind, (S, Hkv, max(lens) + 2))
    places = np.stack([np.stack([rng.permutation(2 * w.shape[2])[:w.shape[2]] for _ in range(Hkv)]) for _ in range(S)])
    nxt = np.full(S, 2 * w.shape[2])
    if kind == "places":
        places = rng.integers(0, 12, places.shape)
    return k, v, table, w, places, nxt


def _run(case, k, v, table, w, places, nxt, ws=None, **kw):
    dtype, Hkv, D, B, lens, budget, first, recent, kind = case
    dev = dict(k=k.cuda(), v=v.cuda(), w=torch.tensor(w).cuda(), p=_i32(places))
    if ws is None:
        ws = pa.new_evict_workspace(len(lens), Hkv, max(lens), budget)
        ws.fill_(255)
    lens_t = _i32(lens)
    new = pa.pa_evict_tokens(dev["k"], dev["v"], _i32(table), lens_t, max(lens), dev["w"], dev["p"], _i32(nxt), budget, first,
                             recent, ws, **kw)
    torch.cuda.synchronize()
    assert lens_t.cpu().tolist() == list(lens)
    return dev, new


def _bits(a):
    return np.ascontiguousarray(a, np.float32).view(np.uint32)


def _check(case, dev, new, k, v, table, w, places, nxt):
    dtype, Hkv, D, B, lens, budget, first, recent, kind = case
    kd, vd, w, places = k.double().numpy(), v.double().numpy(), w.copy(), places.copy()
    want = ref.evict(kd, vd, table, lens, w, places, nxt, budget, first, recent)
    assert new.cpu().tolist() == list(want)
    assert np.array_equal(dev["p"].cpu().numpy(), places)
    assert np.array_equal(_bits(dev["w"].cpu().numpy()), _bits(w))
    assert np.array_equal(dev["k"].double().cpu().numpy(), kd) and np.array_equal(dev["v"].double().cpu().numpy(), vd)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}x{c[2]}-{c[3]}-{len(c[4])}-{c[5]}-{c[8]}")
def test_evict(case):
    state = _case(case)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev, new = _run(case, *state, error_count=err)
    assert int(err) == 0
    _check(case, dev, new, *state)


@pytest.mark.gpu
def test_evict_again_changes_nothing():
    case = CASES[0]
    state = _case(case)
    dev, new = _run(case, *state)
    again = {n: t.clone() for n, t in dev.items()}
    ws = pa.new_evict_workspace(6, 2, 100, 16)
    lens = pa.pa_evict_tokens(again["k"], again["v"], _i32(state[2]), new, 100, again["w"], again["p"], _i32(state[5]), 16, 2, 4,
                              ws, new_lens=new)
    assert lens is new and new.cpu().tolist() == [16, 16, 16, 0, 1, 16]
    assert all(torch.equal(again[n], dev[n]) for n in ("k", "v", "p", "w"))


@pytest.mark.gpu
def test_evict_lengths_in_place_stream_and_graph():
    """context_lens given for new_lens; a captured eviction replayed on other weights; a workspace of a larger call."""
    case = CASES[1]
    k, v, table, w, places, nxt = _case(case)
    big = pa.new_evict_workspace(5, 8, 4000, 512)
    kc, vc, wt, pt = k.cuda(), v.cuda(), torch.tensor(w).cuda(), _i32(places)
    lens = _i32(case[4])
    args = (kc, vc, _i32(table), lens, 2000, wt, pt, _i32(nxt), 512, 4, 64, big)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pa.pa_evict_tokens(*args, new_lens=lens, stream=s)
    s.synchronize()
    _check(case, dict(k=kc, v=vc, w=wt, p=pt), lens, k, v, table, w, places, nxt)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_evict_tokens(*args, new_lens=lens)
    other = _case(case, seed=9)
    w2 = other[3]
    kc.copy_(k), vc.copy_(v), wt.copy_(torch.tensor(w2)), pt.copy_(_i32(places)), lens.copy_(_i32(case[4]))
    g.replay()
    torch.cuda.synchronize()
    _check(case, dict(k=kc, v=vc, w=wt, p=pt), lens, k, v, table, w2, places, nxt)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES[:2], ids=["few-moves", "moves"])
def test_evict_lengths_over_the_next_places(case):
    """next_pos given for new_lens: every head of a sequence sees the places from before the call."""
    state = _case(case)
    dev, want = _run(case, *state)
    again = dict(k=state[0].cuda(), v=state[1].cuda(), w=torch.tensor(state[3]).cuda(), p=_i32(state[4]))
    nxt = _i32(state[5])
    ws = pa.new_evict_workspace(len(case[4]), case[1], max(case[4]), case[5])
    got = pa.pa_evict_tokens(again["k"], again["v"], _i32(state[2]), _i32(case[4]), max(case[4]), again["w"], again["p"], nxt,
                             case[5], case[6], case[7], ws, new_lens=nxt)
    torch.cuda.synchronize()
    assert got is nxt and torch.equal(got, want)
    _check(case, again, got, *state)


@pytest.mark.gpu
def test_evict_moves_codes_of_any_bits():
    """Pools of one-byte codes, given as bf16 of half the head_dim: every pattern of bits arrives as it was."""
    case = (BF16, 2, 32, 16, [200, 90, 300], 64, 2, 8, "random")
    state = _case(case)
    rng = np.random.default_rng(5)
    codes = [torch.tensor(rng.integers(0, 256, tuple(state[0].shape[:3]) + (64,)), dtype=torch.uint8) for _ in range(2)]
    dev, new = _run(case, *(c.view(BF16) for c in codes), *state[2:])
    want = [c.numpy().astype(np.float64) for c in codes]
    w, places = state[3].copy(), state[4].copy()
    lens = ref.evict(*want, state[2], case[4], w, places, state[5], 64, 2, 8)
    assert new.cpu().tolist() == list(lens) and np.array_equal(dev["p"].cpu().numpy(), places)
    for got, exact in zip((dev["k"], dev["v"]), want):
        assert np.array_equal(got.cpu().view(torch.uint8).numpy(), exact)


@pytest.mark.gpu
def test_evict_bad_blocks_and_lengths_are_counted():
    case = (BF16, 1, 64, 16, [200, 90], 64, 0, 0, "random")
    k, v, table, w, places, nxt = _case(case)
    table[0, 1], table[0, 9] = -3, 10 ** 6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc, wt, pt = k.cuda(), v.cuda(), torch.tensor(w).cuda(), _i32(places)
    new = pa.pa_evict_tokens(kc, vc, _i32(table), _i32([200, 400]), 200, wt, pt, _i32(nxt), 64, 0, 0,
                             pa.new_evict_workspace(2, 1, 200, 64), error_count=err)
    # the second sequence counts once and is clamped to the table's 14 blocks' limit of 200 tokens
    assert int(err) > 1
    lens = [200, 200]
    kd, vd, w2, p2 = k.double().numpy(), v.double().numpy(), w.copy(), places.copy()
    want = ref.evict(kd, vd, table, lens, w2, p2, nxt, 64, 0, 0)
    assert new.cpu().tolist() == list(want) and np.array_equal(pt.cpu().numpy(), p2)
    assert np.array_equal(kc.double().cpu().numpy(), kd) and np.array_equal(vc.double().cpu().numpy(), vd)


def test_evict_refusals():
    L = pa.lib()

    def evict(B=16, Hkv=2, D=64, dtype=pa.PA_BF16, S=1, ctx=32, width=32, budget=16, first=0, recent=0, ptr=None):
        return L.pa_evict_tokens(ptr, ptr, 4, B, Hkv, D, dtype, ptr, S, 2, ptr, ctx, ptr, ptr, width, ptr, budget, first, recent,
                                 ptr, None, 0, None, None)

    assert evict(S=0) == pa.PA_OK
    for bad in (dict(), dict(B=0), dict(width=31), dict(budget=0), dict(first=-1), dict(first=8, recent=9), dict(S=-1),
                dict(first=2 ** 31 - 1, recent=2 ** 31 - 1, budget=2 ** 31 - 1)):
        assert evict(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert evict(dtype=3) == pa.PA_ERR_UNSUPPORTED
    assert evict(D=4, ptr=256) == pa.PA_ERR_UNSUPPORTED  # rows of 8 bytes
    assert L.pa_evict_workspace_size(1, 1, 10, 0) == 0
    pool, i = torch.zeros(4, 16, 2, 64), torch.zeros(1, 2, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(1, 2, 32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_evict_tokens(pool, pool, i, one, 32, w, w.int(), one, 16, 0, 0, None)
    with pytest.raises(ValueError, match="differ"):
        pa.pa_evict_tokens(pool, pool, i, one, 32, w, torch.zeros(1, 2, 31, dtype=torch.int32), one, 16, 0, 0, None)


@pytest.mark.gpu
def test_a_serving_loop_under_a_budget():
    """Prompts written with rotary positions on two axes, their weights accumulated, cut to a budget, then decode steps that go
    on at the budget with positions of their own, cut every few steps: weights, places and outputs as the same loop in numpy."""
    rng = np.random.default_rng(4)
    S, Hq, Hkv, D, B, budget, first, recent = 3, 8, 2, 128, 16, 48, 2, 8
    prompt, steps = [70, 33, 120], 12
    width_tok = 128 + 16
    blocks = width_tok // B
    P = S * blocks + 1
    table = rng.permutation(P)[:S * blocks].reshape(S, blocks)
    freq, axis = (1e4 ** (-np.arange(64) / 64)).astype(np.float32), np.arange(64) % 2
    scale = D ** -0.5
    dev = dict(k=torch.zeros(P, B, Hkv, D, dtype=BF16, device="cuda"), v=torch.zeros(P, B, Hkv, D, dtype=BF16, device="cuda"),
               w=torch.full((S, Hkv, width_tok), 9.0, device="cuda"), p=_i32(np.full((S, Hkv, width_tok), -1)))
    tb, ft, at = _i32(table), torch.tensor(freq).cuda(), _i32(axis)
    w_ref = np.full((S, Hkv, width_tok), 9.0)
    loose = [0.0]  # the largest relative error that a weight may have drawn so far
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws_p = pa.new_prefill_weights_workspace(S, sum(prompt), max(prompt), Hq, Hkv, D, B, width_tok)
    ws_d = pa.new_decode_weights_workspace(S, Hq, Hkv, D, B, width_tok)
    ws_e = pa.new_evict_workspace(S, Hkv, width_tok, budget)

    def write(seq, idx, place):
        """New rows of these tokens, turned and written; returns the turned queries."""
        qkv = torch.tensor(rng.standard_normal((len(seq), Hq + 2 * Hkv, D)), dtype=torch.float32).to(BF16).cuda()
        pos = _i32(np.stack([place, place // 3]))
        q = pa.pa_rope_write_kv_paged(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, ft, at, dev["k"], dev["v"], tb,
                                      _i32(seq), _i32(idx), key_weights=dev["w"], key_pos=dev["p"], token_pos=_i32(place),
                                      error_count=err)
        want, mag = ref.turn(qkv[:, :Hq].double().cpu().numpy(), np.stack([place, place // 3]), freq, axis, False)
        assert np.all(np.abs(q.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag)
        w_ref[seq, :, idx] = 0
        return q

    def evict(lens, nxt):
        k, v, p = (dev[n].cpu() for n in ("k", "v", "p"))
        w32 = dev["w"].cpu().numpy()
        kd, vd, pn = k.double().numpy(), v.double().numpy(), p.numpy().copy()
        ids = np.broadcast_to(np.arange(width_tok), w32.shape).copy()
        want = ref.evict(kd, vd, table, lens, w32.copy(), pn, nxt, budget, first, recent)
        for s, n in enumerate(lens):  # the float64 weights move like the library's
            for h in range(Hkv):
                if n > budget:
                    stay = ref.kept(w32[s, h], p.numpy()[s, h], n, budget, first, nxt[s] - recent)
                    src = [j for j in stay if j >= budget]
                    dst = [j for j in range(budget) if j not in set(stay)]
                    w_ref[s, h, dst] = w_ref[s, h, src]
        got = pa.pa_evict_tokens(dev["k"], dev["v"], tb, _i32(lens), width_tok, dev["w"], dev["p"], _i32(nxt), budget, first,
                                 recent, ws_e, error_count=err)
        assert got.cpu().tolist() == list(want) and np.array_equal(dev["p"].cpu().numpy(), pn)
        assert np.array_equal(dev["k"].double().cpu().numpy(), kd) and np.array_equal(dev["v"].double().cpu().numpy(), vd)
        return np.array(want)

    def check(out, want, mag, rel):
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= mag * (2.0 ** -8 + 2 * rel) * 1.01 + 2.0 ** -8 * np.abs(want))
        loose[0] = max(loose[0], rel)  # (of sums of at most 120 x 4 + 12 x 5 terms)
        assert np.all(np.abs(dev["w"].cpu().numpy() - w_ref) <= (loose[0] + 540 * 2.0 ** -24) * np.abs(w_ref))

    seq = np.repeat(np.arange(S), prompt)
    idx = np.concatenate([np.arange(n) for n in prompt])
    q = write(seq, idx, idx)
    cu = np.cumsum([0] + prompt)
    out = pa.pa_prefill_chunk_weights(q, _i32(cu), _i32([0] * S), _i32(range(S)), max(prompt), dev["k"], dev["v"], tb,
                                      _i32(prompt), max(prompt), scale, dev["w"], ws_p, error_count=err)
    kd, vd = dev["k"].double().cpu().numpy(), dev["v"].double().cpu().numpy()
    want, mag, rel = np.zeros(out.shape), np.zeros(out.shape), 0.0
    for s, n in enumerate(prompt):
        rows = slice(cu[s], cu[s + 1])
        want[rows], mag[rows], w, r = ref.attend(q[rows].double().cpu().numpy(), kd, vd, table[s], np.arange(n) + 1, scale)
        w_ref[s, :, :n] += w
        rel = max(rel, r)
    check(out, want, mag, rel)
    nxt = np.array(prompt)
    lens = evict(np.array(prompt), nxt)
    for step in range(steps):
        q = write(np.arange(S), lens, nxt)
        lens, nxt = lens + 1, nxt + 1
        out = pa.pa_decode_weights(q, dev["k"], dev["v"], tb, _i32(lens), width_tok, scale, dev["w"], ws_d, error_count=err)
        kd, vd = dev["k"].double().cpu().numpy(), dev["v"].double().cpu().numpy()
        want, mag, rel = np.zeros(out.shape), np.zeros(out.shape), 0.0
        for s in range(S):
            want[s:s + 1], mag[s:s + 1], w, r = ref.attend(q[s:s + 1].double().cpu().numpy(), kd, vd, table[s], [lens[s]], scale)
            w_ref[s, :, :lens[s]] += w
            rel = max(rel, r)
        check(out, want, mag, rel)
        if step % 5 == 4:
            lens = evict(lens, nxt)
    assert int(err) == 0
