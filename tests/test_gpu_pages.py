"""Copying pages, compacting the pool and forking requests: every byte against plain indexing."""
import dataclasses

import numpy as np
import pytest
import torch

from sub_bit_kv_b200 import lvq, synth
from tests import _helpers as Hl
from tests import _shared as Sh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from sub_bit_kv_b200 import _build
    _build.build()
    assert torch.cuda.is_available()


# page sizes of 256 (d = 128, c = 4), 128 (c = 8), 64 (c = 16) and 128, 64 (d = 64) bytes
SHAPES = [("ouro14_g16_32k", dict(n_layers=3, n_kv_heads=2, n_q_heads=2)), ("ouro14_tc2_64k", dict(n_layers=2, n_kv_heads=3, n_q_heads=3)),
          ("ouro14_tc1_32k", dict(n_layers=1, n_kv_heads=1, n_q_heads=1)), ("tiny", {}), ("tiny", dict(G=32))]


def _cache(shape, pool, batch=3, max_ctx=2000, seed=0, **kw):
    name, over = SHAPES[shape]
    w = dataclasses.replace(synth.WORKLOADS[name], **over, **kw)
    cfg = Hl.make_cfg(w, max_batch=batch, max_ctx=max_ctx)
    cfg.pool_pages = pool
    c = lvq.CodedCache(cfg)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c.idx.random_(0, 256, generator=g)
    for t in (c.sink, c.ring):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    return w, cfg, c


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("n,pool", [(0, 4), (1, 2), (3, 50), (127, 300), (1000, 2003)])
def test_copy_pages(shape, n, pool):
    w, cfg, c = _cache(shape, pool)
    ids = torch.from_numpy(np.random.default_rng(n).permutation(pool).astype(np.int32))
    pairs = torch.stack([ids[:n], ids[n:2 * n]], dim=1).contiguous()
    ref = c.idx_view().clone()
    ref[:, :, :, :, pairs[:, 1].long()] = ref[:, :, :, :, pairs[:, 0].long()]
    lvq.lvq_copy_pages(cfg, c.lay, pairs.cuda(), c.idx, c.status)
    torch.cuda.synchronize()
    c.check_status()
    assert torch.equal(c.idx_view(), ref)


def test_copy_pages_one_source_many_times_and_bad_ids():
    w, cfg, c = _cache(0, 40)
    ref = c.idx_view().clone()
    pairs = torch.tensor([[5, 6], [5, 39], [40, 1], [2, -1], [5, 0]], dtype=torch.int32, device="cuda")
    for dst in (6, 39, 0):
        ref[:, :, :, :, dst] = ref[:, :, :, :, 5]
    lvq.lvq_copy_pages(cfg, c.lay, pairs, c.idx, c.status)
    torch.cuda.synchronize()
    assert int(c.status.item()) == lvq.LVQ_ECAPACITY      # reported, skipped, the others copied
    assert torch.equal(c.idx_view(), ref)


def _orders():
    rng = np.random.default_rng(7)
    yield 200, []
    yield 1, [0]
    yield 300, list(range(300))                                            # nothing to move
    yield 300, [(i + 1) % 300 for i in range(300)]                         # one cycle through three slabs
    yield 257, list(range(256, -1, -1))                                    # cycles of two, over slab borders
    yield 1024, rng.permutation(1024).tolist()                             # a full pool: cycles only
    yield 1500, rng.permutation(1500)[:900].tolist()                       # chains and cycles
    live = rng.permutation(700)[:300].tolist()
    yield 700, live + live[:50] + rng.permutation(live)[:40].tolist()      # shared pages, named again
    yield 2000, [1999, 5, 7]
    a = [(i + 1) % 100 for i in range(100)] + [100 + (i + 1) % 100 for i in range(100)] + [200 + (i + 1) % 200 for i in range(200)]
    yield 400, a                                                           # long cycles back to back: the hold page changes hands in a slab


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("case", range(10))
def test_compact_pages(shape, case):
    pool, order = list(_orders())[case]
    w, cfg, c = _cache(shape, pool, max_ctx=4000)
    plan = lvq.lvq_plan_compaction(pool, order)
    first = list(dict.fromkeys(order))
    ref = c.idx_view().clone()
    ref[:, :, :, :, :len(first)] = c.idx_view()[:, :, :, :, torch.tensor(first, dtype=torch.long, device="cuda")]
    rng = np.random.default_rng(case)
    table = rng.integers(-1, pool, c.page_table.numel()).astype(np.int32)
    table[3], table[9] = pool, -7                                          # not pages: they stay
    c.page_table.copy_(torch.from_numpy(table))
    new = {p: i for i, p in enumerate(first)}
    want = [new.get(int(p), -1) if 0 <= p < pool else int(p) for p in table]
    lvq.lvq_compact_pages(cfg, c.lay, plan, c.page_table, c.idx, c.status)
    torch.cuda.synchronize()
    c.check_status()
    assert torch.equal(c.idx_view(), ref)
    assert c.page_table.cpu().tolist() == want


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("coded,recent,children", [(0, 1, [1]), (8, 0, [3, 1]), (301, 3, [2, 4, 1]), (512, 8, [4]), (7, 5, [1, 2, 3])])
def test_fork_requests(shape, paged, coded, recent, children):
    w, cfg, c = _cache(shape, 120 if paged else 0, batch=6, n_recent=12, n_sink=3)
    parent, R = 5, c.lay.ring_tokens
    S = w.n_sink
    ctx = S + coded + recent
    if ctx == 0:
        ctx = 1
    c.ctx_len[parent], c.coded_len[parent] = ctx, coded
    n = len(children)
    full, tails = coded // 8, None
    refs = {k: getattr(c, k).clone() for k in ("sink", "ring", "idx", "ctx_len", "coded_len")}
    sv, rv = refs["sink"].view_as(c.sink_view()), refs["ring"].view_as(c.ring_view())
    iv = refs["idx"].view_as(c.idx_view())
    if paged:
        ids = np.random.default_rng(1).permutation(120).tolist()
        stride = c.lay.page_table_stride
        row = ids[:full + 2]                                               # the parent holds a page it has not begun
        c.page_table.copy_(torch.randint(0, 120, (c.page_table.numel(),), dtype=torch.int32))
        c.page_table[parent * stride:parent * stride + len(row)].copy_(torch.tensor(row, dtype=torch.int32))
        tails = ids[full + 2:full + 2 + n] if coded % 8 else None
        tv = c.page_table.clone().view(6, stride)
    for i, ch in enumerate(children):
        sv[:, :, :, ch] = sv[:, :, :, parent]
        for t in range(recent):
            slot = (coded + t) % R
            rv[:, :, :, ch, :, slot] = rv[:, :, :, parent, :, slot]
        refs["ctx_len"][ch], refs["coded_len"][ch] = ctx, coded
        if paged:
            tv[ch] = -1
            tv[ch, :full] = tv[parent, :full]
            if tails:
                iv[:, :, :, :, tails[i]] = iv[:, :, :, :, row[full]]
                tv[ch, full] = tails[i]
        else:
            iv[:, :, ch, :, :, :(coded + 7) // 8] = iv[:, :, parent, :, :, :(coded + 7) // 8]
    lvq.lvq_fork_requests(cfg, c.lay, parent, children, coded, tails, c.ctx_len, c.coded_len, c.sink, c.ring, c.idx,
                          c.page_table if paged else None, c.status)
    torch.cuda.synchronize()
    c.check_status()
    for k, v in refs.items():
        assert torch.equal(getattr(c, k), v), k
    if paged:
        assert torch.equal(c.page_table.view(6, stride), tv)


def test_fork_reports_a_parent_that_is_not_as_described():
    w, cfg, c = _cache(1, 50, batch=3)
    before = {k: getattr(c, k).clone() for k in ("sink", "ring", "idx", "page_table")}

    def fork(coded, tails):
        lvq.lvq_fork_requests(cfg, c.lay, 0, [1, 2], coded, tails, c.ctx_len, c.coded_len, c.sink, c.ring, c.idx, c.page_table, c.status)
        torch.cuda.synchronize()
        s = int(c.status.item())
        c.status.zero_()
        return s

    c.ctx_len[0], c.coded_len[0] = w.n_sink + 30, 13
    assert fork(12, [3, 4]) == lvq.LVQ_EINVAL              # the parent has 13 coded tokens
    assert fork(13, [3, 4]) == lvq.LVQ_ECAPACITY           # its partial page is not in the page table
    c.ctx_len[0] = cfg.max_ctx + 1
    assert fork(13, [3, 4]) == lvq.LVQ_ECAPACITY
    for k, v in before.items():
        assert torch.equal(getattr(c, k), v), k
    assert c.coded_len.cpu().tolist() == [13, 0, 0]


def test_large_pool_offsets_pass_32_bits():
    """A pool whose last pages lie past 2^32 bytes: copied, compacted and forked there."""
    w = dataclasses.replace(synth.WORKLOADS["ouro14_g16_32k"], n_layers=1, n_kv_heads=1, n_q_heads=1, n_recent=8)
    cfg = Hl.make_cfg(w, max_batch=2, max_ctx=400)
    cfg.pool_pages = 17_000_000                             # 256 B each: 4.35 GB of K pages, then as much of V
    c = lvq.CodedCache(cfg)
    last = cfg.pool_pages - 1
    g = torch.Generator(device="cuda")
    v = c.idx_view()
    v[:, :, :, :, last - 40:].random_(0, 256)
    v[:, :, :, :, :40].random_(0, 256)
    keep = v[:, :, :, :, last - 40:].clone()
    lvq.lvq_copy_pages(cfg, c.lay, torch.tensor([[last, 3], [5, last - 1]], dtype=torch.int32, device="cuda"), c.idx, c.status)
    assert torch.equal(v[:, :, :, :, 3], keep[:, :, :, :, 40]) and torch.equal(v[:, :, :, :, last - 1], v[:, :, :, :, 5])
    plan = lvq.lvq_plan_compaction(cfg.pool_pages, [last, last - 3, 0])
    first = v[:, :, :, :, 0].clone()
    lvq.lvq_compact_pages(cfg, c.lay, plan, c.page_table, c.idx, c.status)
    assert torch.equal(v[:, :, :, :, 0], keep[:, :, :, :, 40]) and torch.equal(v[:, :, :, :, 1], keep[:, :, :, :, 37])
    assert torch.equal(v[:, :, :, :, 2], first)
    c.ctx_len[0], c.coded_len[0] = w.n_sink + 13, 13
    c.page_table[:2].copy_(torch.tensor([7, last], dtype=torch.int32))
    lvq.lvq_fork_requests(cfg, c.lay, 0, [1], 13, [last - 9], c.ctx_len, c.coded_len, c.sink, c.ring, c.idx, c.page_table, c.status)
    torch.cuda.synchronize()
    c.check_status()
    assert torch.equal(v[:, :, :, :, last - 9], keep[:, :, :, :, 40])


def test_serving_with_forks():
    """A prompt is encoded, forked twice, the children go on by themselves (page encodes into pages of their
    own), a request ends, the pool is compacted: at every stage the shared attention matches
    lvq_decode_attention on the same cache, and forks of forks share what they should."""
    w = dataclasses.replace(synth.WORKLOADS["ouro14_g32_b32"], n_layers=2, n_kv_heads=2, n_q_heads=4, n_recent=16)
    cfg = Hl.make_cfg(w, max_batch=4, max_ctx=700)
    cfg.pool_pages = 150
    c = lvq.CodedCache(cfg)
    L, n0 = 2, 357                                          # a partial last page
    for layer in range(L):
        c.cb_view()[layer] = synth.codebooks(w, layer).cuda()
    lvq.lvq_pack_codebooks(cfg, c.lay, c.cb, c.cbp, c.cb_norm)
    lvq.lvq_rope_table(cfg, c.lay, c.rope)
    c.sink.copy_(torch.randn(c.sink.shape, device="cuda"))
    c.ring.copy_(torch.randn(c.ring.shape, device="cuda"))
    c.assign_pages(0, (n0 + 7) // 8)
    for layer in range(L):
        kv = synth.loop_kv(w, layer, n0).cuda()
        lvq.lvq_encode_prefill(cfg, c.lay, layer, 0, kv, 0, n0, 0, c.cb, c.idx, c.status)
    c.ctx_len[0], c.coded_len[0] = w.n_sink + n0 + w.n_recent, n0

    def attend(begin, tokens):
        B = begin[-1]
        gb, gt = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (begin, tokens))
        for layer in range(L):
            for step in (0, 3):
                q = synth.queries(w, layer, step, batch=B).cuda()
                outs = []
                for shared in (True, False):
                    out = torch.zeros(B, 4, 128, device="cuda")
                    lse = torch.zeros(B, 4, device="cuda")
                    if shared:
                        lvq.lvq_decode_attention_shared(cfg, c.lay, layer, step, B, q, c.ctx_len, c.coded_len, gb, gt, c.sink, c.ring,
                                                        c.idx, c.cbp, c.rope, 0, c.workspace, out, lse, c.status)
                    else:
                        lvq.lvq_decode_attention(cfg, c.lay, layer, step, B, q, c.ctx_len, c.coded_len, c.sink, c.ring, c.idx,
                                                 c.cbp, c.rope, 3, c.workspace, out, lse, c.status)
                    torch.cuda.synchronize()
                    c.check_status()
                    outs.append((out, lse))
                assert float((outs[0][0] - outs[1][0]).abs().max()) <= 2 * Hl.OUT_ATOL
                assert float((outs[0][1] - outs[1][1]).abs().max()) <= 2 * Hl.LSE_REL * float(outs[1][1].abs().max())

    attend([0, 1], [0])
    c.fork(0, [1, 2], n0)
    assert c.pages[1][:44] == c.pages[0][:44] and len({c.pages[i][44] for i in range(3)}) == 3
    assert c.pool.holders(c.pages[0][0]) == 3 and c.pool.available() == 150 - 47
    attend([0, 3], [n0 // 8 * 8])
    # the requests go on: eight new tokens each, then a page encode over the page border
    for b in range(3):
        c.assign_pages(b, 46)
    c.ctx_len[:3] += 8
    c.ring.copy_(torch.randn(c.ring.shape, device="cuda"))
    lvq.lvq_encode_page(cfg, c.lay, 3, c.ctx_len, c.coded_len, c.ring, c.cb, c.cb_norm, c.idx, c.status)
    attend([0, 3], [352])
    c.fork(2, [3], n0 + 8)
    attend([0, 2, 4], [352, 360])
    attend([0, 4], [352])
    # request 0 ends; its slot takes a fork of request 1; the pool is compacted
    c.release(0)
    assert c.pool.holders(c.pages[1][0]) == 3
    c.fork(1, [0], n0 + 8)
    attend([0, 4], [352])
    held = 150 - c.pool.available()
    moved = c.compact()
    assert moved > 0 and sorted({p for row in c.pages for p in row}) == list(range(held))
    assert c.pool.alloc(1) == [held]
    c.pool.free([held])
    torch.cuda.synchronize()
    c.check_status()
    attend([0, 4], [352])
    for b in range(4):
        c.release(b)
    assert c.pool.available() == 150


def test_captured_calls():
    """Copies and forks replay on what the buffers hold then; a compaction is refused and leaves the pool as it was."""
    w, cfg, c = _cache(1, 60, batch=4, n_recent=12, n_sink=3)
    other = _cache(1, 60, batch=4)[2]
    other.assign_pages(0, 3), other.assign_pages(1, 6)
    other.release(0)
    c.assign_pages(0, 6)
    c.ctx_len[0], c.coded_len[0] = w.n_sink + 43 + 4, 43
    tails = c.pool.alloc(2)
    pairs = torch.tensor([[1, 50], [2, 51]], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lvq.lvq_copy_pages(cfg, c.lay, pairs, c.idx, c.status)
        lvq.lvq_fork_requests(cfg, c.lay, 0, [2, 3], 43, tails, c.ctx_len, c.coded_len, c.sink, c.ring, c.idx,
                              c.page_table, c.status)
        with pytest.raises(RuntimeError, match="captured"):
            other.compact()
    assert other.pages[1] == list(range(3, 9)) and [other.pool.holders(p) for p in (0, 2, 3, 8, 9)] == [0, 0, 1, 1, 0]
    stride = c.lay.page_table_stride
    for seed in (1, 2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        c.idx.random_(0, 256, generator=g)
        c.ring.copy_(torch.randn(c.ring.shape, generator=g, device="cuda"))
        pairs.copy_(torch.tensor([[seed, 50], [2, 51 + seed]], dtype=torch.int32))
        c.ctx_len[2:] = 0
        ref, ring = c.idx_view().clone(), c.ring_view().clone()
        ref[:, :, :, :, 50], ref[:, :, :, :, 51 + seed] = ref[:, :, :, :, seed], ref[:, :, :, :, 2]
        for ch, p in zip((2, 3), tails):
            ref[:, :, :, :, p] = ref[:, :, :, :, 5]
            for t in range(4):
                ring[:, :, :, ch, :, (43 + t) % c.lay.ring_tokens] = ring[:, :, :, 0, :, (43 + t) % c.lay.ring_tokens]
        graph.replay()
        torch.cuda.synchronize()
        c.check_status()
        assert torch.equal(c.idx_view(), ref) and torch.equal(c.ring_view(), ring)
        assert c.ctx_len.tolist()[2:] == [w.n_sink + 47] * 2 and c.coded_len.tolist()[2:] == [43] * 2
        for ch, p in zip((2, 3), tails):
            assert c.page_table[ch * stride:ch * stride + 6].tolist() == [0, 1, 2, 3, 4, p]
