"""Eviction in the allocator and the step runner."""
import numpy as np
import pytest
import torch

import eviction_reference as ref
from paged_kv_cache_313_gb300 import pa
from paged_kv_cache_313_gb300 import workloads as W
from paged_kv_cache_313_gb300.allocator import BlockAllocator, NoBlocks
from paged_kv_cache_313_gb300.runner import DeviceStep


def test_truncate_frees_the_blocks_behind():
    a = BlockAllocator(10, 4)
    s = a.allocate(15)
    blocks = a.blocks(s)
    a.truncate(s, 15)
    a.truncate(s, 99)
    assert a.blocks(s) == blocks and a.seq_len(s) == 15
    a.truncate(s, 6)
    assert a.blocks(s) == blocks[:2] and a.seq_len(s) == 6 and a.num_free == 8
    a.check_invariants()
    a.append(s)
    assert a.blocks(s) == blocks[:2] and a.seq_len(s) == 7  # goes on in its tail block
    a.truncate(s, 0)
    assert a.blocks(s) == [] and a.num_free == 10
    with pytest.raises(ValueError):
        a.truncate(s, -1)
    a.check_invariants()


def test_truncate_keeps_what_others_reference():
    a = BlockAllocator(10, 4)
    s = a.allocate(12)
    t = a.fork(s)
    a.truncate(s, 4)
    assert a.num_free == 7 and a.seq_len(t) == 12
    a.check_invariants()


def test_make_private():
    a = BlockAllocator(8, 4)
    s = a.allocate(10)
    old = a.blocks(s)
    assert a.make_private(s) == []
    t = a.fork(s)
    copies = a.make_private(t)
    assert [(c.src, c.num_valid) for c in copies] == list(zip(old, (4, 4, 2))) and a.blocks(s) == old
    assert a.blocks(t) == [c.dst for c in copies] and not set(a.blocks(t)) & set(old)
    a.check_invariants()
    u = a.fork(t)
    before = a.blocks(u)
    with pytest.raises(NoBlocks):
        a.make_private(u)
    assert a.blocks(u) == before
    a.check_invariants()


def test_e4m3_pools_have_no_key_weights():
    with pytest.raises(ValueError, match="bf16 or fp32"):
        DeviceStep(W.small("decode_fp8", 0), "cpu", key_weights=True)


def _double(t):
    return t.double().cpu().numpy()


def _expect(w, st):
    """Outputs, weights drawn and bounds of one step over what is in the pools now."""
    kd, vd, bt, ctx = _double(st.k_cache), _double(st.v_cache), w.block_tables.numpy(), w.context_lens.numpy()
    add, rel = np.zeros(st.key_weights.shape), 0.0
    nd = w.num_decode
    dec, dmag = np.zeros(w.q_decode.shape), np.zeros(w.q_decode.shape)
    for s in range(nd):
        dec[s:s + 1], dmag[s:s + 1], x, r = ref.attend(_double(w.q_decode[s:s + 1]), kd, vd, bt[s], [ctx[s]], w.scale)
        add[s, :, :ctx[s]] += x
        rel = max(rel, r)
    pre, pmag = np.zeros(w.q_prefill.shape), np.zeros(w.q_prefill.shape)
    cu = w.cu_q_lens.numpy()
    for c in range(w.num_chunks):
        s, start, n = int(w.seq_of_chunk[c]), int(w.q_start_pos[c]), cu[c + 1] - cu[c]
        rows = slice(cu[c], cu[c + 1])
        pre[rows], pmag[rows], x, r = ref.attend(_double(w.q_prefill[rows]), kd, vd, bt[s], start + np.arange(n) + 1, w.scale)
        add[s, :, :start + n] += x
        rel = max(rel, r)
    return dec, dmag, pre, pmag, add, rel


def _near(got, want, mag, rel, dtype):
    p = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(_double(got) - want) <= mag * (p + 2 * rel) * 1.01 + torch.finfo(dtype).eps / 2 * np.abs(want))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["mixed_bf16", "tiny_fp32"])
def test_device_step_with_key_weights(name):
    w = W.tiny_fp32(3) if name == "tiny_fp32" else W.mixed_bf16(3, num_decode=5, num_chunks=2, chunk_len=40, max_off=90)
    st = DeviceStep(w, key_weights=True)
    st.key_weights.fill_(7.0)
    out_d, out_p = st.run()
    torch.cuda.synchronize()
    assert st.errors() == 0
    dec, dmag, pre, pmag, add, rel = _expect(w, st)
    _near(out_d, dec, dmag, rel, w.dtype)
    if w.num_chunks:
        _near(out_p, pre, pmag, rel, w.dtype)
    before = np.full(add.shape, 7.0)
    before[w.seq_idx.numpy(), :, w.pos.numpy()] = 0.0  # this step's tokens begin anew
    terms = max(1, int(w.cu_q_lens[-1])) * w.num_q_heads // w.num_kv_heads + 2
    assert np.all(np.abs(_double(st.key_weights) - before - add) <= add * rel + (before + add) * terms * 2.0 ** -24)

    # cut down, then the graph of the same step over what is left
    lens = w.context_lens.numpy().copy()
    budget = max(2, int(np.median(lens)))
    kd, vd = _double(st.k_cache), _double(st.v_cache)
    wn, pn = st.key_weights.cpu().numpy(), st.key_pos.cpu().numpy()
    new = ref.evict(kd, vd, w.block_tables.numpy(), lens, wn, pn, lens, budget, 1, 1)
    got = st.evict(budget, keep_first=1, keep_recent=1)
    torch.cuda.synchronize()
    assert got is st.context_lens and got.cpu().tolist() == list(new) and st.errors() == 0
    assert np.array_equal(_double(st.k_cache), kd) and np.array_equal(_double(st.v_cache), vd)
    assert np.array_equal(st.key_weights.cpu().numpy(), wn) and np.array_equal(st.key_pos.cpu().numpy(), pn)
    st.decode()
    torch.cuda.synchronize()
    for s in range(w.num_decode):
        want, mag, _, r = ref.attend(_double(w.q_decode[s:s + 1]), kd, vd, w.block_tables.numpy()[s], [new[s]], w.scale)
        _near(st.out_decode[s:s + 1], want, mag, r, w.dtype)


@pytest.mark.gpu
def test_device_step_with_key_weights_captured():
    w = W.mixed_bf16(4, num_decode=4, num_chunks=1, chunk_len=30, max_off=60)
    st = DeviceStep(w, key_weights=True)
    st.run()
    torch.cuda.synchronize()
    want_d, want_p = st.out_decode.clone(), st.out_prefill.clone()
    st.capture()
    st.key_weights.zero_()
    st.replay()
    torch.cuda.synchronize()
    once = st.key_weights.clone()
    assert torch.equal(st.out_decode, want_d) and torch.equal(st.out_prefill, want_p)
    st.key_weights.zero_()
    st.run()
    torch.cuda.synchronize()
    assert torch.equal(st.key_weights, once) and st.errors() == 0


def test_evictions_to_several_budgets_keep_their_workspaces(monkeypatch):
    """A workspace that a captured eviction may still use is not given up for another budget's."""
    st = DeviceStep.__new__(DeviceStep)
    st.__dict__.update(track_weights=True, w=W.tiny_fp32(3), max_any_context=40, device="cpu", evict_workspaces={}, k_cache=None,
                       v_cache=None, block_tables=None, context_lens=None, key_weights=None, key_pos=None, next_pos=None,
                       error_count=None)
    made, used = [], []
    monkeypatch.setattr("paged_kv_cache_313_gb300.pa.new_evict_workspace", lambda *a, **kw: made.append(torch.zeros(4)) or made[-1])
    monkeypatch.setattr("paged_kv_cache_313_gb300.pa.pa_evict_tokens", lambda *a, **kw: used.append(a[11]))
    for budget in (8, 16, 8):
        st.evict(budget)
    assert len(made) == 2 and used[0] is used[2] is made[0] and used[1] is made[1]
    assert any(t is made[0] for t in st.evict_workspaces.values())


def test_evict_needs_key_weights():
    class Without(DeviceStep):
        def __init__(self):
            self.track_weights = False

    with pytest.raises(ValueError, match="key_weights=True"):
        Without().evict(4)
