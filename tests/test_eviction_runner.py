"""A step runner that goes on after its caches were cut: step, evict, step, evict, with the places that the tokens have in
their sequences."""
import numpy as np
import pytest
import torch

import eviction_reference as ref
from paged_kv_cache_313_gb300 import pa
from paged_kv_cache_313_gb300 import workloads as W
from paged_kv_cache_313_gb300.runner import DeviceStep


def _double(t):
    return t.double().cpu().numpy()


class _Loop:
    """What a scheduler keeps: lengths, next places, and the inputs of each step; beside it the places that every head's
    cached tokens should have."""

    def __init__(self, w, budget, first, recent, seed=0):
        self.w, self.budget, self.first, self.recent = w, budget, first, recent
        self.rng = np.random.default_rng(seed)
        self.lens = w.context_lens.numpy().copy()
        self.next = self.lens.copy()
        self.places = np.broadcast_to(np.arange(int(self.lens.max())), (len(self.lens), w.num_kv_heads, int(self.lens.max()))).copy()
        self.seq = w.seq_idx.numpy()

    def cut(self):
        self.lens = np.minimum(self.lens, self.budget)

    def inputs(self):
        """One more token for each decode sequence, one more chunk for each chunk's."""
        w, T = self.w, len(self.seq)
        count = np.bincount(self.seq, minlength=len(self.lens))
        nth = np.array([np.sum(self.seq[:t] == self.seq[t]) for t in range(T)])
        pos, token_pos = self.lens[self.seq] + nth, self.next[self.seq] + nth
        start = self.lens[w.seq_of_chunk.numpy()]
        self.lens, self.next = self.lens + count, self.next + count
        self.places[self.seq, :, pos] = token_pos[:, None]
        new = {name: torch.tensor(self.rng.standard_normal(getattr(w, name).shape), dtype=torch.float32).to(w.dtype)
               for name in ("q_decode", "q_prefill", "k_new", "v_new")}
        i32 = lambda x: torch.tensor(np.ascontiguousarray(x), dtype=torch.int32)  # noqa: E731
        return dict(new, pos=i32(pos), token_pos=i32(token_pos), q_start_pos=i32(start), context_lens=i32(self.lens),
                    next_pos=i32(self.next))

    def check_cut(self, st, before):
        """The caches after an eviction, against the reference's from what lay there `before`."""
        k, v, weights, table = before
        want = ref.evict(k, v, table, self.lens, weights, self.places, self.next, self.budget, self.first, self.recent)
        assert st.context_lens.cpu().tolist() == list(want)
        for s, n in enumerate(want):
            got = st.key_pos[s, :, :n].cpu().numpy()
            assert np.array_equal(got, self.places[s, :, :n])
            for h in range(got.shape[0]):  # the sequence's newest tokens are among those that stay
                assert set(range(int(self.next[s]) - min(self.recent, n), int(self.next[s]))) <= set(got[h].tolist())
        assert np.array_equal(_double(st.k_cache), k) and np.array_equal(_double(st.v_cache), v)


def _before(st, w):
    return _double(st.k_cache), _double(st.v_cache), st.key_weights.cpu().numpy(), w.block_tables.numpy()


def _decode_only(dtype):
    return W._decode_batch("loop", [70, 33, 120], 8, 2, 128, 16, dtype, 3)


def _mixed(dtype):
    return W.prefill_batch(4, 8, 2, 128, 16, chunk_lens=[30], offsets=[60], dtype=dtype, decode_lens=[90, 33])


# ------------------------------------------------------------------ on the CPU, the library's calls played by numpy
def _stubs(monkeypatch):
    def write(q, k_new, v_new, rope_pos, inv_freq, axis, kc, vc, table, seq, pos, key_weights=None, key_pos=None, token_pos=None,
              **kw):
        B = kc.shape[1]
        for t in range(len(seq)):
            s, i = int(seq[t]), int(pos[t])
            kc[table[s, i // B], i % B], vc[table[s, i // B], i % B] = k_new[t], v_new[t]
            key_weights[s, :, i] = 0
            key_pos[s, :, i] = int(pos[t] if token_pos is None else token_pos[t])

    def decode(q, kc, vc, table, lens, max_len, scale, weights, ws, **kw):
        for s, n in enumerate(lens.tolist()):  # early tokens draw the most
            weights[s, :, :n] += 1.0 / (1 + torch.arange(n))

    def prefill(q, cu, start, seq, max_q, kc, vc, table, lens, max_len, scale, weights, ws, **kw):
        pass

    def evict(kc, vc, table, lens, max_len, weights, places, nxt, budget, first, recent, ws, new_lens=None, **kw):
        kd, vd, w, p = _double(kc), _double(vc), weights.numpy(), places.numpy()
        new = ref.evict(kd, vd, table.numpy(), lens.numpy(), w, p, nxt.numpy(), budget, first, recent)
        kc.copy_(torch.tensor(kd)), vc.copy_(torch.tensor(vd)), new_lens.copy_(torch.tensor(new))
        return new_lens

    for name, f in (("pa_rope_write_kv_paged", write), ("pa_decode_weights", decode), ("pa_prefill_chunk_weights", prefill),
                    ("pa_evict_tokens", evict), ("pa_stage_copy", lambda dst, src, stream=None: dst.copy_(src))):
        monkeypatch.setattr(pa, name, f)
    for name in ("new_decode_workspace", "new_decode_weights_workspace", "new_prefill_weights_workspace", "new_evict_workspace"):
        monkeypatch.setattr(pa, name, lambda *a, **kw: torch.zeros(1))
    monkeypatch.setattr(pa, "pa_prefill_workspace_size", lambda *a: 0)


@pytest.mark.parametrize("make", [_decode_only, _mixed], ids=["decode", "mixed"])
def test_places_go_on_after_an_eviction(monkeypatch, make):
    _stubs(monkeypatch)
    w = make(torch.float32)
    st = DeviceStep(w, "cpu", key_weights=True)
    loop = _Loop(w, budget=60, first=2, recent=8)
    host_in, host_out = st.inbuf.clone(), torch.empty_like(st.outbuf)
    for step in range(5):
        if step:
            views = st.input_views(host_in)
            for name, t in loop.inputs().items():
                views[name].copy_(t)
        st.step_from_host(host_in, host_out)
        before = _before(st, w)
        st.evict(60, keep_first=2, keep_recent=8)
        loop.check_cut(st, before)
        loop.cut()


def test_a_step_after_an_eviction_needs_its_inputs(monkeypatch):
    _stubs(monkeypatch)
    w = _decode_only(torch.float32)
    st = DeviceStep(w, "cpu", key_weights=True)
    loop = _Loop(w, budget=60, first=2, recent=8)
    st.run()
    st.run()
    before = _before(st, w)
    st.evict(60, keep_first=2, keep_recent=8)
    loop.check_cut(st, before)
    loop.cut()
    with pytest.raises(RuntimeError, match="set_inputs"):
        st.run()
    with pytest.raises(RuntimeError, match="set_inputs"):
        st.replay()
    inputs = loop.inputs()
    with pytest.raises(ValueError, match="not one of"):
        st.set_inputs(k_cache=w.k_cache)
    with pytest.raises(ValueError, match="must be"):
        st.set_inputs(pos=inputs["pos"][:1])
    with pytest.raises(ValueError, match="must be"):
        st.set_inputs(pos=inputs["pos"].long())
    with pytest.raises(RuntimeError):
        st.run()
    st.set_inputs(**inputs)
    st.run()
    before = _before(st, w)
    st.evict(60, keep_first=2, keep_recent=8)
    loop.check_cut(st, before)


# ------------------------------------------------------------------ on the GPU
def _check_outputs(st, w, loop, inputs):
    """The step's outputs and the weights that it added, from the caches that it has left."""
    kd, vd, table = _double(st.k_cache), _double(st.v_cache), w.block_tables.numpy()
    p = 2.0 ** -8 if w.dtype == torch.bfloat16 else 0.0
    half = torch.finfo(w.dtype).eps / 2
    nd, cu = w.num_decode, w.cu_q_lens.numpy()
    rows = [(st.out_decode[s:s + 1], inputs["q_decode"][s:s + 1], s, [int(loop.lens[s])]) for s in range(nd)]
    for c in range(w.num_chunks):
        s, n = int(w.seq_of_chunk[c]), int(cu[c + 1] - cu[c])
        at = slice(int(cu[c]), int(cu[c + 1]))
        rows.append((st.out_prefill[at], inputs["q_prefill"][at], s, int(loop.lens[s]) - n + 1 + np.arange(n)))
    for got, q, s, limits in rows:
        want, mag, _, rel = ref.attend(_double(q), kd, vd, table[s], limits, w.scale)
        assert np.all(np.abs(_double(got) - want) <= mag * (p + 2 * rel) * (1 + 2.0 ** -7) + half * np.abs(want))


@pytest.mark.gpu
@pytest.mark.parametrize("make,dtype", [(_decode_only, torch.bfloat16), (_mixed, torch.bfloat16), (_mixed, torch.float32)],
                         ids=["decode", "mixed", "mixed-fp32"])
def test_device_step_goes_on_after_evictions(make, dtype):
    w = make(dtype)
    st = DeviceStep(w, key_weights=True)
    loop = _Loop(w, budget=60, first=2, recent=8)
    host_in, host_out = st.pinned_inputs(), st.pinned_outputs()
    inputs = {n: t.clone() for n, t in st.input_views(host_in).items()}
    for step in range(6):
        if step:
            inputs = loop.inputs()
            for name, t in inputs.items():
                st.input_views(host_in)[name].copy_(t)
        if step == 3:  # the same without host memory
            st.set_inputs(**inputs)
            st.run()
        else:
            st.step_from_host(host_in, host_out)
        torch.cuda.synchronize()
        if step != 3:
            dec, pre = st.output_views(host_out)
            if w.num_decode:
                st.out_decode.copy_(dec)
            if w.num_chunks:
                st.out_prefill.copy_(pre)
        _check_outputs(st, w, loop, inputs)
        before = _before(st, w)
        st.evict(60, keep_first=2, keep_recent=8)
        torch.cuda.synchronize()
        loop.check_cut(st, before)
        loop.cut()
    assert st.errors() == 0


@pytest.mark.gpu
def test_a_captured_step_with_its_eviction_goes_on():
    """One graph of copy-in, step and eviction, replayed step after step: as the same loop run eagerly."""
    w = _mixed(torch.bfloat16)
    runs = []
    for graph in (False, True):
        st = DeviceStep(w, key_weights=True)
        loop = _Loop(w, budget=60, first=2, recent=8, seed=5)
        host_in, host_out = st.pinned_inputs(), st.pinned_outputs()
        host_out.zero_()  # (the bytes between the outputs)
        trace = []

        def once():
            st.step_from_host(host_in, host_out)
            st.evict(60, keep_first=2, keep_recent=8)

        for step in range(6):
            if step:
                for name, t in loop.inputs().items():
                    st.input_views(host_in)[name].copy_(t)
            if graph and step == 1:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    once()
            if graph and step:
                g.replay()
            else:
                once()
            torch.cuda.synchronize()
            trace += [t.clone() for t in (host_out, st.key_pos, st.key_weights, st.context_lens)]
            loop.cut()
        assert st.errors() == 0 and st.context_lens.cpu().tolist() == loop.lens.tolist()
        runs.append(trace)
    for a, b in zip(*runs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ rotary positions
def test_rotary_positions_of_a_step_are_checked(monkeypatch):
    _stubs(monkeypatch)
    freq = torch.full((32,), 0.1)
    with pytest.raises(ValueError, match="key_weights=True"):
        DeviceStep(_decode_only(torch.float32), "cpu", inv_freq=freq)
    with pytest.raises(ValueError, match="axis must"):
        DeviceStep(_decode_only(torch.float32), "cpu", key_weights=True, inv_freq=freq, axis=[0] * 31)
    with pytest.raises(ValueError, match="axis must"):
        DeviceStep(_decode_only(torch.float32), "cpu", key_weights=True, inv_freq=freq, axis=[-1] * 32)
    w = _mixed(torch.float32)
    w.seq_idx = w.seq_idx.flip(0)
    with pytest.raises(ValueError, match="one for each query"):
        DeviceStep(w, "cpu", key_weights=True, inv_freq=freq)
    st = DeviceStep(_mixed(torch.float32), "cpu", key_weights=True, inv_freq=freq, axis=[0, 1] * 16)
    assert st.rope_pos_decode.tolist() == [[89, 32]] * 2 and st.rope_pos_prefill.shape == (2, 30)
    st.run()


@pytest.mark.gpu
@pytest.mark.parametrize("make,dtype,interleaved", [(_decode_only, torch.bfloat16, False), (_mixed, torch.bfloat16, True),
                                                    (_mixed, torch.float32, False)], ids=["decode", "mixed", "mixed-fp32"])
def test_device_step_turns_queries_and_keys(make, dtype, interleaved):
    """Steps with positions of their own on two axes, between evictions: the turned queries and stored keys, and the attention
    over them."""
    w = make(dtype)
    freq, axis = (1e4 ** (-np.arange(48) / 48)).astype(np.float32), np.arange(48) % 2
    st = DeviceStep(w, key_weights=True, inv_freq=torch.tensor(freq), axis=torch.tensor(axis), interleaved=interleaved)
    loop = _Loop(w, budget=60, first=2, recent=8)
    host_in, host_out = st.pinned_inputs(), st.pinned_outputs()
    inputs = {n: t.clone() for n, t in st.input_views(host_in).items()}
    nd, half = w.num_decode, torch.finfo(dtype).eps / 2
    for step in range(3):
        if step:
            inputs = loop.inputs()
            places = inputs["token_pos"]
            both = torch.stack([places, places // 3 + 1000])
            inputs["rope_pos_decode"], inputs["rope_pos_prefill"] = both[:, :nd], both[:, nd:]
            for name, t in inputs.items():
                st.input_views(host_in)[name].copy_(t)
        st.step_from_host(host_in, host_out)
        torch.cuda.synchronize()
        rope = torch.cat([inputs["rope_pos_decode"], inputs["rope_pos_prefill"]], dim=1).numpy()
        q = _double(torch.cat([inputs["q_decode"], inputs["q_prefill"]]))
        rows = w.block_tables.long()[w.seq_idx.long(), inputs["pos"].long() // 16], inputs["pos"].long() % 16
        got_q = _double(torch.cat([st.turned_q_decode, st.turned_q_prefill]))
        for got, x in ((got_q, q), (_double(st.k_cache.cpu()[rows]), _double(inputs["k_new"]))):
            want, mag = ref.turn(x, rope, freq, axis, interleaved)
            assert np.all(np.abs(got - want) <= half * np.abs(want) + 2.0 ** -20 * mag)
        assert np.array_equal(_double(st.v_cache.cpu()[rows]), _double(inputs["v_new"]))
        dec, pre = st.output_views(host_out)
        if w.num_decode:
            st.out_decode.copy_(dec)
        if w.num_chunks:
            st.out_prefill.copy_(pre)
        _check_outputs(st, w, loop, dict(q_decode=st.turned_q_decode, q_prefill=st.turned_q_prefill))
        before = _before(st, w)
        st.evict(60, keep_first=2, keep_recent=8)
        torch.cuda.synchronize()
        loop.check_cut(st, before)
        loop.cut()
    assert st.errors() == 0


@pytest.mark.gpu
def test_capturing_a_step_adds_no_weight():
    """The step that is run before a capture is not counted again."""
    w = _mixed(torch.bfloat16)
    st = DeviceStep(w, key_weights=True)
    host_in, host_out = st.pinned_inputs(), st.pinned_outputs()
    st.step_from_host(host_in, host_out)
    torch.cuda.synchronize()
    want, places = st.key_weights.clone(), st.key_pos.clone()
    assert float(want.sum()) > 0
    st.capture()
    torch.cuda.synchronize()
    assert torch.equal(st.key_weights, want) and torch.equal(st.key_pos, places)
    st.capture_from_host(host_in, host_out)
    torch.cuda.synchronize()
    assert torch.equal(st.key_weights, want) and torch.equal(st.key_pos, places)
