"""Host side of page sharing, compaction, forking and attention over shared prefixes: bookkeeping, plans, and
arguments that are refused before any device work (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from sub_bit_kv_b200 import lvq, synth
from tests._helpers import make_cfg

FAKE = 1 << 20                       # a 16-byte-aligned address that is never touched


@pytest.fixture(scope="module", autouse=True)
def built():
    from sub_bit_kv_b200 import _build
    _build.build()


def test_shared_pages_are_free_with_their_last_holder():
    pool = lvq.PagePool(6)
    assert pool.alloc(4) == [0, 1, 2, 3] and pool.holders(1) == 1 and pool.holders(4) == 0
    pool.share([0, 1])
    pool.share([1])
    assert [pool.holders(i) for i in range(4)] == [2, 3, 1, 1]
    pool.free([0, 1, 2])
    assert pool.available() == 3 and [pool.holders(i) for i in range(4)] == [1, 2, 0, 1]
    assert pool.alloc(1) == [2] and pool.holders(2) == 1
    pool.free([1])
    pool.free([0, 1])
    assert pool.available() == 4
    for bad in ([0], [6], [-1], [3, 3]):                    # free, out of range, out of range, repeated
        for call in (pool.share, pool.free):
            with pytest.raises(lvq.LvqError) as e:
                call(bad)
            assert e.value.status == lvq.LVQ_EINVAL
    assert pool.holders(3) == 1 and pool.holders(6) == -1 and pool.holders(-1) == -1


def _carry_out(plan, pages):
    """The moves of a plan as lvq_compact_pages documents them: slabs of 64 pairs, the reads of a slab before
    its writes, -1 a page's worth of memory."""
    hold = None
    moves = plan.moves.tolist()
    for s in range(0, len(moves), 64):
        slab = moves[s:s + 64]
        values = [hold if src == -1 else pages[src] for src, _ in slab]
        for (_, dst), v in zip(slab, values):
            assert v is not None
            if dst == -1:
                hold = v
            else:
                pages[dst] = v
    return pages


@pytest.mark.parametrize("n,live,seed", [(1, 1, 0), (5, 0, 0), (128, 128, 1), (129, 129, 2), (1000, 1000, 3), (1000, 400, 4), (4097, 4000, 5)])
def test_compaction_plan(n, live, seed):
    order = np.random.default_rng(seed).permutation(n)[:live].tolist()
    plan = lvq.lvq_plan_compaction(n, order + order[:live // 3])
    assert plan.n_live == live and plan.n_moves <= live + live // 2
    new = plan.new_id.tolist()
    assert [new[p] for p in order] == list(range(live)) and sum(i >= 0 for i in new) == live
    pages = _carry_out(plan, list(range(n)))
    assert pages[:live] == order
    assert all(pages[i] == i for i in range(live, n))


def test_compaction_plan_of_cycles():
    """Cycles shorter than a slab, as long, longer, and back to back."""
    sizes = [2, 3, 62, 63, 64, 65, 126, 127, 128, 129, 300, 2, 500, 1, 128]
    order, at = [], 0
    for k in sizes:
        order += [at + (i + 1) % k for i in range(k)]
        at += k
    plan = lvq.lvq_plan_compaction(at, order)
    assert _carry_out(plan, list(range(at))) == order
    assert plan.n_moves <= at - 1 + len(sizes)


def test_compaction_plan_refusals():
    for n, order in ((0, []), (4, [4]), (4, [-1]), (4, [0, 9])):
        with pytest.raises(lvq.LvqError) as e:
            lvq.lvq_plan_compaction(n, order)
        assert e.value.status == lvq.LVQ_EINVAL
    L = lvq.lib()
    k = ctypes.c_int32()
    assert L.lvq_plan_compaction(4, None, 2, FAKE, FAKE, ctypes.byref(k)) == lvq.LVQ_EINVAL
    assert L.lvq_plan_compaction(4, None, -1, FAKE, FAKE, ctypes.byref(k)) == lvq.LVQ_EINVAL


def test_pool_renumber():
    pool = lvq.PagePool(6)
    pool.alloc(5)
    pool.free([0, 3])
    pool.share([4])
    for bad in ([-1] * 6, [-1, 0, 1, -1, 1, -1], [0, 1, 2, -1, 3, -1], [-1, 0, 1, -1, 6, -1]):
        with pytest.raises(lvq.LvqError) as e:
            pool.renumber(bad)                              # a page without an id, one id twice, a free page's, out of range
        assert e.value.status == lvq.LVQ_EINVAL
    with pytest.raises(ValueError):
        pool.renumber([0, 1])
    plan = lvq.lvq_plan_compaction(6, [4, 1, 2, 4])
    pool.renumber(plan.new_id)
    assert [pool.holders(i) for i in range(6)] == [2, 1, 1, 0, 0, 0]
    assert pool.alloc(3) == [3, 4, 5]


def _call(fn, cfg, lay, *args):
    return getattr(lvq.lib(), fn)(ctypes.byref(cfg), ctypes.byref(lay), *args)


def _cfgs():
    w = synth.WORKLOADS["ouro14_tc2_64k"]
    plain = make_cfg(w, n_layers=2, max_batch=4, max_ctx=1000)
    pool = make_cfg(w, n_layers=2, max_batch=4, max_ctx=1000)
    pool.pool_pages, pool.page_table = 50, FAKE
    return (plain, lvq.lvq_cache_layout(plain)), (pool, lvq.lvq_cache_layout(pool))


def test_page_calls_check_their_arguments():
    (plain, pl), (pool, ql) = _cfgs()
    assert _call("lvq_copy_pages", plain, pl, 1, FAKE, FAKE, None, None) == lvq.LVQ_EUNSUPPORTED
    assert _call("lvq_copy_pages", pool, ql, -1, FAKE, FAKE, None, None) == lvq.LVQ_EINVAL
    assert _call("lvq_copy_pages", pool, ql, 1, FAKE + 4, FAKE, None, None) == lvq.LVQ_EINVAL
    assert _call("lvq_copy_pages", pool, ql, 1, FAKE, FAKE + 8, None, None) == lvq.LVQ_EINVAL
    assert _call("lvq_copy_pages", pool, pl, 1, FAKE, FAKE, None, None) == lvq.LVQ_EINVAL          # another layout
    assert _call("lvq_compact_pages", plain, pl, 1, FAKE, FAKE, None, FAKE, None, None) == lvq.LVQ_EUNSUPPORTED
    assert _call("lvq_compact_pages", pool, ql, 1, FAKE, FAKE, FAKE + 16, FAKE, None, None) == lvq.LVQ_EINVAL   # not its table
    assert _call("lvq_compact_pages", pool, ql, 1, FAKE, None, FAKE, FAKE, None, None) == lvq.LVQ_EINVAL
    assert _call("lvq_compact_pages", pool, ql, 1, None, FAKE, FAKE, FAKE, None, None) == lvq.LVQ_EINVAL


def test_fork_checks_its_arguments():
    (plain, pl), (pool, ql) = _cfgs()

    def fork(cfg, lay, children, tails=None, parent=0, coded=16, table=None, n=None):
        arr = lambda v: None if v is None else (ctypes.c_int32 * max(1, len(v)))(*v)  # noqa: E731
        return _call("lvq_fork_requests", cfg, lay, parent, len(children) if n is None else n, arr(children), coded, arr(tails),
                     FAKE, FAKE, FAKE, FAKE, FAKE, table, None, None)

    bad = [dict(children=[0]), dict(children=[1, 1]), dict(children=[4]), dict(children=[-1]), dict(children=[1], parent=4),
           dict(children=[1], coded=-1), dict(children=[1], coded=5000), dict(children=[1], table=FAKE), dict(children=[1], n=-1),
           dict(children=[1], tails=[3])]
    for kw in bad:
        assert fork(plain, pl, **kw) == lvq.LVQ_EINVAL, kw
    bad = [dict(children=[1]), dict(children=[1], coded=13, table=FAKE), dict(children=[1], coded=16, tails=[2], table=FAKE),
           dict(children=[1, 2], coded=13, tails=[3, 3], table=FAKE), dict(children=[1], coded=13, tails=[50], table=FAKE)]
    for kw in bad:
        assert fork(pool, ql, **kw) == lvq.LVQ_EINVAL, kw
    assert fork(plain, pl, list(range(1, 4)), n=257) == lvq.LVQ_EUNSUPPORTED
    if not torch.cuda.is_available():
        assert fork(plain, pl, [1, 3]) == lvq.LVQ_EDEVICE
        assert fork(pool, ql, [1, 3], tails=[4, 5], coded=13, table=FAKE) == lvq.LVQ_EDEVICE


def test_shared_attention_checks_its_arguments():
    (plain, pl), _ = _cfgs()

    def attend(layer=0, step=0, batch=4, q=FAKE, groups=1, gb=FAKE, sink=FAKE, ns=0, ws=FAKE, cfg=plain, lay=pl):
        return _call("lvq_decode_attention_shared", cfg, lay, layer, step, batch, q, FAKE, FAKE, groups, gb, FAKE, sink, FAKE, FAKE,
                     FAKE, FAKE, ns, ws, FAKE, FAKE, None, None)

    for kw in (dict(layer=2), dict(layer=-1), dict(step=4), dict(batch=5), dict(batch=-1), dict(q=None), dict(q=FAKE + 8),
               dict(groups=0), dict(groups=5), dict(groups=-1), dict(gb=None), dict(sink=None), dict(ns=-1), dict(ns=65), dict(ws=None)):
        assert attend(**kw) == lvq.LVQ_EINVAL, kw
    big = make_cfg(synth.WORKLOADS["tiny"], max_batch=300)
    assert attend(batch=257, cfg=big, lay=lvq.lvq_cache_layout(big)) == lvq.LVQ_EUNSUPPORTED
    if not torch.cuda.is_available():
        assert attend() == lvq.LVQ_EDEVICE
        assert attend(batch=0, groups=0, q=None) == lvq.LVQ_EDEVICE
