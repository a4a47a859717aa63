"""Attention over e4m3 pools whose V scales lie as far apart as the pools allow: a block of zeros has 2^-100, a block of
the largest bf16 values 2^120, and a caller may put any finite scale there.  Keys of small V keep their weight in the
softmax's sum.  The tolerance is the one of tests/test_fp8_block_long.py, whose reference is used."""
import numpy as np
import pytest
import torch

from test_fp8_block_long import _attend, _bf16, _close, _dev, _i32, _pools, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa

ORDERS = ["zeros_first", "zeros_last", "zeros_around"]


def _mark_zeros(pools, order, blocks, exponent):
    """V of some of the context's blocks (table 0, 1, 2, ...) becomes zeros as the write stores them, of the others it gets
    scales of 2^exponent."""
    _, vc, _, vs = pools
    zero = np.zeros(blocks, bool)
    third = blocks // 3
    zero[{"zeros_first": slice(0, blocks // 2), "zeros_last": slice(blocks // 2, None),
          "zeros_around": np.r_[0:third, 2 * third:blocks]}[order]] = True
    vs[:] = np.float32(2.0 ** exponent)
    vc[:blocks][zero] = 0
    vs[:blocks][zero] = np.float32(2.0 ** -100)


def _decode(pools, table, n, rows, Hq, seed, scale):
    rng = np.random.default_rng(seed)
    P, B, H, _ = pools[0].shape
    q = _bf16(rng, (rows, Hq, 128))
    q[0] = 0  # every weight alike
    ws = pa.new_decode_fp8_block_workspace(rows, Hq, H, 128, B, n)
    got = pa.pa_decode_fp8_block(q.cuda(), *_dev(*pools), _i32(np.repeat(table, rows, 0)), _i32([n] * rows), n, scale, ws)
    _close(got, *_attend(q.double().numpy(), pools, table[0], [n] * rows, scale))


def _prefill(pools, table, n, chunks, queries, Hq, seed, scale):
    """`chunks` chunks of the last `queries` tokens of one context."""
    rng = np.random.default_rng(seed)
    P, B, H, _ = pools[0].shape
    q = _bf16(rng, (chunks * queries, Hq, 128))
    q[0] = 0
    ws = pa.new_prefill_fp8_block_workspace(chunks, chunks * queries, queries, Hq, H, 128, B, n)
    got = pa.pa_prefill_chunk_fp8_block(q.cuda(), _i32(np.arange(chunks + 1) * queries), _i32([n - queries] * chunks),
                                        _i32([0] * chunks), queries, *_dev(*pools), _i32(table), _i32([n]), n, scale, ws)
    limits = [n - queries + 1 + i for i in range(queries)] * chunks
    _close(got, *_attend(q.double().numpy(), pools, table[0], limits, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("exponent", [27, 60, 119])
@pytest.mark.parametrize("G,B,n", [(1, 16, 384), (8, 64, 384), (4, 128, 768)])
def test_decode_keeps_the_weight_of_zeros_in_other_stages(G, B, n, exponent, order):
    """Items of three to six stages: 128 sequences of 8 kv heads make partitions of 1024 tokens."""
    rng = np.random.default_rng(G + exponent)
    pools = _pools(rng, n // B + 1, B, 8)
    _mark_zeros(pools, order, n // B, exponent)
    _decode(pools, np.arange(n // B)[None], n, 128, 8 * G, exponent, 0.05)


@pytest.mark.gpu
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("exponent", [27, 60, 119])
@pytest.mark.parametrize("B", [16, 24])
def test_decode_keeps_the_weight_of_zeros_in_other_partitions(B, exponent, order):
    """One sequence: partitions of 128 tokens, joined.  (Blocks of 24 tokens are the CUDA cores'.)"""
    rng = np.random.default_rng(B + exponent)
    n = 1152
    pools = _pools(rng, n // B + 1, B, 1)
    _mark_zeros(pools, order, n // B, exponent)
    _decode(pools, np.arange(n // B)[None], n, 2, 4, exponent, 0.05)


@pytest.mark.gpu
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("exponent", [27, 60, 119])
@pytest.mark.parametrize("B,n,chunks", [(16, 1152, 20), (8, 768, 20), (64, 4224, 20), (16, 1152, 1), (8, 2304, 1)])
def test_prefill_keeps_the_weight_of_zeros_in_other_blocks(B, n, chunks, exponent, order):
    """The scales are looked at 32 blocks at a time.  20 chunks of 8 kv heads are one item each over the whole context, one
    chunk is cut into spans, joined."""
    rng = np.random.default_rng(B + exponent + chunks)
    pools = _pools(rng, n // B + 1, B, 8)
    _mark_zeros(pools, order, n // B, exponent)
    _prefill(pools, np.arange(n // B)[None], n, chunks, 16, 16, exponent, 0.05)


@pytest.mark.gpu
@pytest.mark.parametrize("exponent", [125, 126, 127])
def test_the_largest_scales(exponent):
    """V scales up to the largest powers of two that a float holds, K scales that the queries bring back; values that stay
    within bf16's range."""
    rng = np.random.default_rng(exponent)
    n, B = 640, 16
    pools = _pools(rng, n // B, B, 8)
    pools[1][:] &= 0xbf  # values below 2
    pools[2][:], pools[3][:] = np.float32(2.0 ** 100), np.float32(2.0 ** exponent)
    table = np.arange(n // B)[None]
    for rows in (1, 128):  # partitions of 128 tokens, joined, and of several stages
        _decode(pools, table, n, rows, 32, exponent, 2.0 ** -104)
    for chunks in (1, 20):
        _prefill(pools, table, n, chunks, 16, 32, exponent, 2.0 ** -104)
