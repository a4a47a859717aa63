"""One workspace of the block-scaled e4m3 attention, made for the largest call, serves every smaller one: fewer sequences
or chunks, fewer queries, shorter limits."""
import numpy as np
import pytest
import torch

from test_fp8_block_long import _attend, _bf16, _close, _dev, _i32, _pools, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,B", [(32, 8, 128, 16), (8, 1, 128, 64), (24, 2, 64, 16)])
def test_decode_workspace_serves_smaller_batches(Hq, Hkv, D, B):
    rng = np.random.default_rng(Hq)
    N, n = 64, 4096
    size = lambda a, b: pa.lib().pa_decode_fp8_block_workspace_size(a, Hq, Hkv, D, B, b)  # noqa: E731
    for limit in (4096, 3000, 2048, 1000, 129, 1):
        sizes = [size(k, limit) for k in range(1, N + 1)]
        assert sizes == sorted(sizes), limit
    for k in (64, 16, 1):
        sizes = [size(k, limit) for limit in range(1, n + 1, 31)]
        assert sizes == sorted(sizes), k
    assert size(2000, 150000) >= max(size(k, m) for k in (1, 7, 300, 2000) for m in (100, 20000, 131072, 131073, 150000))
    P = 300
    pools = _pools(rng, P, B, Hkv)
    pools = _dev(*[p[..., :D] if p.ndim == 4 else p for p in pools])
    table = _i32(rng.integers(0, P, (N, n // B)))
    q = _bf16(rng, (N, Hq, D)).cuda()
    ws = pa.new_decode_fp8_block_workspace(N, Hq, Hkv, D, B, n)
    for k in (64, 55, 33, 16, 9, 2, 1, 64):
        for limit in (4096, 2048, 700, 60):
            lens = _i32(rng.integers(0, limit + 1, k))
            args = (q[:k], *pools, table[:k], lens, limit, 0.1)
            got = pa.pa_decode_fp8_block(*args, ws)
            own = pa.new_decode_fp8_block_workspace(k, Hq, Hkv, D, B, limit)
            assert torch.equal(got, pa.pa_decode_fp8_block(*args, own)), (k, limit)


@pytest.mark.gpu
def test_prefill_workspace_serves_smaller_calls():
    """Also with rows of q behind the last chunk, as a buffer of fixed size has them; those rows are left."""
    rng = np.random.default_rng(3)
    Hq, Hkv, B, P, n = 32, 8, 16, 300, 4096
    pools = _pools(rng, P, B, Hkv)
    table = rng.integers(0, P, (4, n // B)).astype(np.int32)
    q = _bf16(rng, (2048, Hq, 128))
    ws = pa.new_prefill_fp8_block_workspace(4, 2048, 512, Hq, Hkv, 128, B, n)
    dev, bt, qd = _dev(*pools), _i32(table), q.cuda()
    for chunks, queries, limit in ((4, 512, 4096), (1, 37, 4096), (2, 100, 3000), (1, 1, 2048), (3, 1, 600), (1, 512, 4096)):
        start = [limit - queries - 3 * c for c in range(chunks)]
        cu, ctx = np.arange(chunks + 1) * queries, [limit] * 4
        want = None
        for rows in (chunks * queries, 2048):
            out = torch.full((rows, Hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
            pa.pa_prefill_chunk_fp8_block(qd[:rows], _i32(cu), _i32(start), _i32(range(chunks)), queries, *dev, bt,
                                          _i32(ctx), limit, 0.1, ws, out=out)
            if want is None:
                pick = rng.permutation(chunks * queries)[:40]
                parts = [_attend(q[i:i + 1].double().numpy(), pools, table[i // queries],
                                 [start[i // queries] + i % queries + 1], 0.1) for i in pick]
                want = [np.concatenate(x) for x in zip(*parts)]
            _close(out[torch.from_numpy(pick).cuda()], *want)
            assert bool((out[chunks * queries:] == 5.0).all())
