"""Copy-on-write over e4m3 pools with a scale per (block, kv head): codes by pa_copy_blocks, scales beside them."""
import numpy as np
import pytest
import torch

import fp8_block_reference as R
from test_fp8_block_long import BF, _bf16, _dev, _i32, _pools, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 3, 8])
def test_a_copied_block_goes_on_as_the_block_it_was_copied_from(H):
    """Two sequences share a partly filled block; the second's next token goes to a copy, in place of blocks whose own
    scales are larger and smaller.  Copy and original give the same values, and the same codes after the same write."""
    rng = np.random.default_rng(H)
    P, B = 8, 16
    kc, vc, ks, vs = _pools(rng, P, B, H)
    ks[5], vs[5] = 2.0 ** 20, 2.0 ** 20
    ks[6], vs[6] = 2.0 ** -30, 2.0 ** -30
    dk, dv, dks, dvs = _dev(kc, vc, ks, vs)
    src, dst, valid = [1, 2], [5, 6], [5, 16]
    pa.pa_copy_blocks(dk.view(BF), dv.view(BF), _i32(src), _i32(dst), _i32(valid))
    dks[dst], dvs[dst] = dks[src], dvs[src]
    for s, d, n in zip(src, dst, valid):
        kc[d, :n], vc[d, :n], ks[d], vs[d] = kc[s, :n], vc[s, :n], ks[s], vs[s]
    table = np.array([[1], [5], [2], [6]], np.int32)
    rows = [(q, p) for q, n in zip(range(4), [5, 5, 16, 16]) for p in range(n)]
    seq, pos = (np.array(x, np.int32) for x in zip(*rows))
    k, v = (t.cpu() for t in pa.pa_read_kv_paged_fp8_block(dk, dv, dks, dvs, _i32(table), _i32(seq), _i32(pos)))
    for t in (k, v):
        assert torch.equal(t[seq == 0], t[seq == 1]) and torch.equal(t[seq == 2], t[seq == 3])
    new = _bf16(rng, (2, H, 128), 8.0)  # the shared block's next token, and another for the copy
    pa.pa_write_kv_paged_fp8_block(new.cuda(), new.cuda(), dk, dv, dks, dvs, _i32(table), _i32([0, 1]), _i32([5, 5]))
    for codes, scales, c, s in ((kc, ks, dk, dks), (vc, vs, dv, dvs)):
        want = scales.astype(np.float64)
        R.write(new.double().numpy(), codes, want, [1 * B + 5, 5 * B + 5])
        assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(s.double().cpu().numpy(), want)
