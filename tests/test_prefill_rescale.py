"""Chunked prefill where single rows' maxima grow by far more than the lazy rescale's threshold from one key tile to a
later one: the rescale takes the whole warp through tensor memory together, whichever of its rows needs it."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_313_gb300 import pa
from paged_kv_cache_313_gb300.workloads import storage_numpy


@pytest.mark.gpu
@pytest.mark.timeout(120)
@pytest.mark.parametrize("rows", [(5,), (0, 31, 32, 77), tuple(range(0, 100, 3))])
def test_single_rows_rescale(rows):
    """Query rows `rows` point at one late key each, so that their scores jump by about 49 (base 2) there; the other
    rows' scores stay within a few units.  Output within 2e-2: a row that sees one value rounds it to bf16, half a step
    of which is 2^-8 of |v| < 5."""
    rng = np.random.default_rng(len(rows))
    T, n, G, B, D = 100, 700, 1, 16, 128
    nblk = -(-n // B)
    table = rng.permutation(nblk + 3)[:nblk].astype(np.int32)[None]
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    kc, vc = (bf(rng.standard_normal((nblk + 3, B, 1, D))) for _ in range(2))
    q = rng.standard_normal((T, G, D))
    for i, r in enumerate(rows):
        j = 300 + 7 * i % 290  # a key of the third to fifth tile that every row sees
        q[r, 0] = 3.0 * kc[table[0, j // B], j % B, 0].double().numpy()
    q = bf(q)
    cu, start, seq, ctx = (np.array(x, np.int32) for x in ([0, T], [n - T], [0], [n]))
    want = oracle.prefill(storage_numpy(q), cu, start, seq, storage_numpy(kc), storage_numpy(vc), table, ctx,
                          1 / math.sqrt(D))
    i32 = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = pa.pa_prefill_chunk(q.cuda(), i32(cu), i32(start), i32(seq), T, kc.cuda(), vc.cuda(), i32(table), i32(ctx),
                              1 / math.sqrt(D), error_count=err)
    assert float(np.abs(got.double().cpu().numpy() - want).max()) <= 2e-2
    assert int(err.item()) == 0
