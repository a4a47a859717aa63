"""Calls over e4m3 pools with a scale per (block, kv head) as a serving loop makes them, and at the ends of what they take:
a captured step whose contexts grow under one limit, block sizes from 1 to 1024, lengths and positions out of range."""
import numpy as np
import pytest
import torch

from test_fp8_block_long import BF, _attend, _bf16, _close, _dev, _i32, _pools, _tables, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,B", [(32, 8, 16), (8, 1, 64), (20, 2, 16)])
def test_a_captured_step_serves_growing_contexts(Hq, Hkv, B):
    """Write and decode of one token per sequence, captured once with a limit far above the contexts and replayed as they
    grow: over the ends of blocks, stages and partitions."""
    rng = np.random.default_rng(Hq)
    N, limit, steps = 6, 4096, [1, 2, B, B + 1, 127, 128, 129, 500, 513, 1024, 1025, 2050]
    per = -(-2100 // B)
    table = rng.permutation(N * per + 3)[:N * per].reshape(N, per).astype(np.int32)
    pools = _pools(rng, N * per + 3, B, Hkv)
    kc, vc, ks, vs = dev = _dev(*pools)
    bt, lens, pos = _i32(table), _i32([1] * N), _i32([0] * N)
    seq = _i32(range(N))
    new, q = (torch.zeros(N, h, 128, dtype=BF, device="cuda") for h in (Hkv, Hq))
    out, err = torch.zeros(N, Hq, 128, dtype=BF, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.new_decode_fp8_block_workspace(N, Hq, Hkv, 128, B, limit)

    def step():
        pa.pa_write_kv_paged_fp8_block(new, new, *dev, bt, seq, pos, error_count=err)
        pa.pa_decode_fp8_block(q, *dev, bt, lens, limit, 0.1, ws, out=out, error_count=err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in steps:
        at = [max(1, n - 3 * s) for s in range(N)]
        host = _bf16(rng, (N, Hq, 128))
        q.copy_(host)
        new.copy_(_bf16(rng, (N, Hkv, 128), 3.0))
        lens.copy_(torch.tensor(at, dtype=torch.int32))
        pos.copy_(lens - 1)
        graph.replay()
        got = out.cpu()
        now = tuple(t.cpu().numpy() for t in dev)
        parts = [_attend(host[s:s + 1].double().numpy(), now, table[s], [at[s]], 0.1) for s in range(N)]
        _close(got, *(np.concatenate(x) for x in zip(*parts)))
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (16, 1)])
@pytest.mark.parametrize("B", [1, 2, 3, 256, 1024])
def test_block_sizes_of_the_cuda_cores(B, Hq, Hkv):
    rng = np.random.default_rng(B)
    lens = [700, 1, 0, 257, 2, 1025]
    table, P = _tables(rng, lens, B)
    pools = _pools(rng, P, B, Hkv)
    table[0, 0 if B > 300 else 1] = P + 7
    q, err = _bf16(rng, (len(lens), Hq, 128)), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.new_decode_fp8_block_workspace(len(lens), Hq, Hkv, 128, B, 1025)
    got = pa.pa_decode_fp8_block(q.cuda(), *_dev(*pools), _i32(table), _i32(lens), 1025, 0.1, ws, error_count=err)
    assert int(err.item()) > 0
    parts = [_attend(q[s:s + 1].double().numpy(), pools, table[s], [L], 0.1) for s, L in enumerate(lens)]
    _close(got, *(np.concatenate(x) for x in zip(*parts)))
    chunks = [(0, 690, 10), (3, 250, 7), (5, 0, 5), (1, 0, 1)]  # (sequence, offset, queries)
    cu = np.concatenate([[0], np.cumsum([n for _, _, n in chunks])])
    q = _bf16(rng, (int(cu[-1]), Hq, 128))
    got = pa.pa_prefill_chunk_fp8_block(q.cuda(), _i32(cu), _i32([o for _, o, _ in chunks]), _i32([s for s, _, _ in chunks]),
                                        10, *_dev(*pools), _i32(table), _i32(lens), 1025, 0.1)
    parts = [_attend(q[int(cu[c]):int(cu[c + 1])].double().numpy(), pools, table[s], [o + i + 1 for i in range(n)], 0.1)
             for c, (s, o, n) in enumerate(chunks)]
    _close(got, *(np.concatenate(x) for x in zip(*parts)))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,spread", [(4, 1), (4, 20), (12, 1)])
def test_prefill_positions_and_lengths_out_of_range(Hq, spread):
    """Queries behind the context, or beyond the limit, see the keys that there are, and are counted; a context of negative
    length has none (zeros); positions next to 2^31; rows and chunks that make no sense are left.  Cut into spans, not cut
    (20 copies of the chunks), and on the CUDA cores (12 query heads)."""
    rng = np.random.default_rng(5 + Hq)
    H, B, n, limit = 8, 16, 900, 800
    hq = Hq * H
    table, P = _tables(rng, [n, 40, 700], B)
    pools = _pools(rng, P, B, H)
    big = 2 ** 31 - 30
    # (sequence, start, queries, keys that query i sees)
    chunks = [(0, 780, 40, lambda i: min(780 + i + 1, limit)), (1, 30, 20, lambda i: min(30 + i + 1, 40)),
              (0, big, 25, lambda i: limit), (2, 50, 9, lambda i: 0), (1, 2 ** 31 - 1, 1, lambda i: 40)] * spread
    ctx = [n, 40, -5]
    cu = np.concatenate([[0], np.cumsum([c[2] for c in chunks])]).astype(np.int64)
    total = int(cu[-1])
    q = _bf16(rng, (total + 6, hq, 128))
    # two more chunks: one that ends behind q's rows, one of a sequence that is not there
    start, seq = [c[1] for c in chunks] + [0, 0], [c[0] for c in chunks] + [1, 3]
    cu2 = np.concatenate([cu, [total + 7, total + 5]])
    out, err = torch.full(q.shape, 5.0, dtype=BF, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.new_prefill_fp8_block_workspace(len(seq), q.shape[0], 40, hq, H, 128, B, limit)
    pa.pa_prefill_chunk_fp8_block(q.cuda(), _i32(cu2), _i32(start), _i32(seq), 40, *_dev(*pools), _i32(table), _i32(ctx),
                                  limit, 0.1, ws, out=out, error_count=err)
    assert int(err.item()) > 0 and bool((out[total:] == 5.0).all())
    parts = [_attend(q[int(cu[c]):int(cu[c + 1])].double().numpy(), pools, table[s], [sees(i) for i in range(m)], 0.1)
             for c, (s, _, m, sees) in enumerate(chunks)]
    _close(out[:total], *(np.concatenate(x) for x in zip(*parts)))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [4, 12])
def test_decode_lengths_out_of_range(Hq):
    rng = np.random.default_rng(Hq)
    H, B = 2, 16
    table, P = _tables(rng, [300, 300, 300, 300], B)
    pools = _pools(rng, P, B, H)
    lens, sees = [-1, 2 ** 31 - 1, -2 ** 31, 299], [0, 280, 0, 280]
    q, err = _bf16(rng, (4, Hq * H, 128)), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.new_decode_fp8_block_workspace(4, Hq * H, H, 128, B, 280)
    got = pa.pa_decode_fp8_block(q.cuda(), *_dev(*pools), _i32(table), _i32(lens), 280, 0.1, ws, error_count=err)
    assert int(err.item()) == 4
    parts = [_attend(q[s:s + 1].double().numpy(), pools, table[s], [n], 0.1) for s, n in enumerate(sees)]
    _close(got, *(np.concatenate(x) for x in zip(*parts)))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,chunks", [(4, 1), (4, 60), (12, 2)])
def test_prefill_of_empty_contexts_gives_zeros(Hq, chunks):
    """All of a call's contexts without a token, whatever the pools hold; rows behind the chunks are left."""
    H, B, n = 8, 16, 40
    kc = torch.full((4, B, H, 128), 0x7f, dtype=torch.uint8, device="cuda")
    sc = torch.full((4, H), float("nan"), device="cuda")
    q = torch.ones(chunks * n + 3, Hq * H, 128, dtype=BF, device="cuda")
    out, err = torch.full_like(q, 5.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.new_prefill_fp8_block_workspace(chunks, q.shape[0], n, Hq * H, H, 128, B, 4096)
    pa.pa_prefill_chunk_fp8_block(q, _i32(np.arange(chunks + 1) * n), _i32([0] * chunks), _i32([0] * chunks), n, kc, kc, sc, sc,
                                  _i32([[0, 1, 2, 3]]), _i32([0]), 4096, 0.1, ws, out=out, error_count=err)
    assert int(torch.count_nonzero(out[:chunks * n])) == 0 and bool((out[chunks * n:] == 5.0).all())
    assert int(err.item()) > 0
