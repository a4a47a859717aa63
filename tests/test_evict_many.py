"""Evictions of few moves by many CTAs at once, in each of the launch's block sizes: the moves that a CTA makes itself."""
import pytest
import torch

from test_evict import BF16, _case, _check, _i32, lib  # noqa: F401
from paged_kv_cache_313_gb300 import pa


@pytest.mark.gpu
@pytest.mark.parametrize("n,cut", [(2064, 16), (4500, 100), (17000, 128)], ids=["256", "512", "1024"])
def test_few_moves_of_many_heads_are_the_same_every_time(n, cut):
    """Every (sequence, head) has its list of moves to itself, whatever order its warps run in."""
    seqs = 160 if n < 4000 else 40
    case = (BF16, 8, 8, 64, [n - (i % 7) for i in range(seqs)], n - cut, 4, 32, "random")
    k, v, table, w, places, nxt = _case(case)
    ws = pa.new_evict_workspace(seqs, 8, n, case[5])
    tb, lens, nx = _i32(table), _i32(case[4]), _i32(nxt)
    start = dict(k=k.cuda(), v=v.cuda(), w=torch.tensor(w).cuda(), p=_i32(places))
    first = None
    for _ in range(20):
        dev = {name: t.clone() for name, t in start.items()}
        new = pa.pa_evict_tokens(dev["k"], dev["v"], tb, lens, n, dev["w"], dev["p"], nx, case[5], 4, 32, ws)
        if first is None:
            first, lens0 = dev, new
        same = [torch.equal(dev[x].view(torch.uint8), first[x].view(torch.uint8)) for x in dev]
        assert all(same) and torch.equal(new, lens0)
    # against the reference: the first sequences' heads (all of them take minutes in Python)
    few = 3
    short = (BF16, 8, 8, 64, case[4][:few], case[5], 4, 32, "random")
    kd, vd = k.clone(), v.clone()
    used = torch.as_tensor(table[:few][table[:few] >= 0])
    dev = dict(k=kd.cuda(), v=vd.cuda(), w=first["w"][:few], p=first["p"][:few])
    dev["k"][used.cuda()], dev["v"][used.cuda()] = first["k"][used.cuda()], first["v"][used.cuda()]
    _check(short, dev, lens0[:few], k, v, table[:few], w[:few], places[:few], nxt[:few])
