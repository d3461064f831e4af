"""Decode attention for groups of requests with shared coded prefixes, against the fp64 oracle: shapes, ragged
lengths, groupings, the page pool, its limits and refusals."""
import dataclasses

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


def _w(name, **kw):
    return dataclasses.replace(synth.WORKLOADS[name], n_layers=1, **kw)


SHAPES = [
    _w("tiny"),                                                            # d = 64, c = 4
    _w("tiny", G=32, n_kv_heads=3, n_q_heads=3),                           # d = 64, c = 8
    _w("ouro14_g16_32k", n_kv_heads=2, n_q_heads=2),                       # d = 128, c = 4
    _w("ouro14_g32_b32", n_kv_heads=2, n_q_heads=8),                       # c = 8, four query heads per KV head
    _w("ouro14_tc2_64k", n_kv_heads=1, n_q_heads=20, n_recent=31, n_sink=5),   # c = 8, two blocks, 20 query heads
    _w("ouro14_tc1_32k", n_kv_heads=2, n_q_heads=2, n_recent=8, n_sink=0),     # c = 16, four blocks, no sink
]
GROUPS = [
    [(488, [0, 5])],                                                       # a pair, one with no token of its own
    [(1000, [0, 1, 7, 8, 9, 130])],                                        # ragged
    [(7, [40, 3]), (0, [17]), (16, [0]), (333, [1, 300, 22])],             # a prefix below a page, none, a lone request
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("groups", range(len(GROUPS)))
def test_matches_oracle(shape, groups):
    w = SHAPES[shape]
    gr = GROUPS[groups]
    B = sum(len(o) for _, o in gr)
    case, begin, tokens = Sh.shared_case(w, gr, recent=[1 + (w.n_recent + 7 * b) % (w.n_recent + 7) for b in range(B)])
    pcase = Sh.to_pool(case, begin, tokens)
    for step in (0, w.T - 1):
        q = synth.queries(w, 0, step, batch=B).cuda()
        out, lse = Sh.run_shared(pcase, begin, tokens, step, q)
        heads = None if w.n_q_heads <= 8 else [0, 3, 15, 16, 19]
        Sh.check_against_oracle(case, step, q, out, lse, heads=heads)
        so, sl = Sh.run_shared(case, begin, tokens, step, q)               # the leader's stream: the same arithmetic
        assert torch.equal(out, so) and torch.equal(lse, sl)


@pytest.mark.parametrize("ns", [1, 2, 5, 64])
def test_any_number_of_parts(ns):
    w = _w("ouro14_g32_b32", n_kv_heads=2, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(515, [3, 0, 90, 4]), (64, [11, 200])], recent=[128, 1, 135, 77, 130, 2])
    q = synth.queries(w, 0, 1, batch=6).cuda()
    out, lse = Sh.run_shared(case, begin, tokens, 1, q, num_splits=ns)
    Sh.check_against_oracle(case, 1, q, out, lse)
    again = Sh.run_shared(case, begin, tokens, 1, q, num_splits=ns)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])       # a fixed order of summation


def test_many_queries_per_group():
    """More rows than one tile of queries holds, and not a multiple of it."""
    w = _w("ouro14_g32_b32", n_kv_heads=1, n_q_heads=3)
    own = [(7 * b) % 23 for b in range(41)]
    case, begin, tokens = Sh.shared_case(w, [(700, own)], recent=[1 + b % 135 for b in range(41)])
    pcase = Sh.to_pool(case, begin, tokens)
    q = synth.queries(w, 0, 2, batch=41).cuda()
    out, lse = Sh.run_shared(pcase, begin, tokens, 2, q)
    Sh.check_against_oracle(case, 2, q, out, lse, requests=[0, 1, 5, 10, 11, 21, 31, 32, 33, 39, 40])


def test_short_requests():
    """Requests with no coded token, fewer tokens than the sink, a single one."""
    w = _w("ouro14_g16_32k", n_kv_heads=2, n_q_heads=4)
    case, begin, tokens = Sh.shared_case(w, [(0, [0, 0, 0]), (8, [0])], recent=[0, 0, 3, 1], ctx=[1, 3, None, None])
    q = synth.queries(w, 0, 3, batch=4).cuda()
    out, lse = Sh.run_shared(case, begin, tokens, 3, q)
    Sh.check_against_oracle(case, 3, q, out, lse)


def test_more_shared_tokens_than_coded_are_cut():
    """group_tokens is an upper bound: whole pages, and no more than the shortest request has."""
    w = _w("ouro14_g32_b32", n_kv_heads=1, n_q_heads=2)
    case, begin, _ = Sh.shared_case(w, [(203, [0, 10])], recent=[5, 9])
    q = synth.queries(w, 0, 0, batch=2).cuda()
    ref = Sh.run_shared(case, begin, [200], 0, q)
    for t in (203, 201, 1 << 30):
        got = Sh.run_shared(case, begin, [t], 0, q)
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    none = Sh.run_shared(case, begin, [-5], 0, q)
    Sh.check_against_oracle(case, 0, q, *none)


def test_counters_outside_the_layout_are_reported():
    w = _w("ouro14_g32_b32", n_kv_heads=1, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(96, [3, 20, 8])], recent=[5, 9, 30])
    q = synth.queries(w, 0, 0, batch=3).cuda()
    for bad in (-1, 0, case.cfg.max_ctx + 1, 50):
        case.cache.ctx_len[1] = bad
        out, lse = Sh.run_shared(case, begin, tokens, 0, q, check=False)
        assert int(case.cache.status.item()) == lvq.LVQ_ECAPACITY
        case.cache.status.zero_()
        assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()     # left empty, the others as ever
        Sh.check_against_oracle(case, 0, q, out, lse, requests=[0, 2])


@pytest.mark.parametrize("begin", [[0, 2, 2], [1, 2, 3], [0, 3, 3, 2], [0, -1, 3], [0, 5, 3]])
def test_bad_groups_are_reported(begin):
    w = _w("ouro14_g32_b32", n_kv_heads=1, n_q_heads=1)
    case, _, _ = Sh.shared_case(w, [(16, [3, 0, 8])], recent=[5, 9, 30])
    q = synth.queries(w, 0, 0, batch=3).cuda()
    Sh.run_shared(case, begin, [16] * (len(begin) - 1), 0, q, check=False)
    assert int(case.cache.status.item()) == lvq.LVQ_EINVAL
    case.cache.status.zero_()
    out, lse = Sh.run_shared(case, [0, 3], [16], 0, q)
    Sh.check_against_oracle(case, 0, q, out, lse)


def test_out_of_range_page_is_reported():
    w = _w("ouro14_g32_b32", n_kv_heads=1, n_q_heads=1)
    case, begin, tokens = Sh.shared_case(w, [(160, [30, 9])], recent=[5, 9])
    pcase = Sh.to_pool(case, begin, tokens)
    q = synth.queries(w, 0, 0, batch=2).cuda()
    stride = pcase.cache.lay.page_table_stride
    for at in (3, 21, stride + 20):
        old = int(pcase.cache.page_table[at])
        for b in range(2):
            if at < 20:
                pcase.cache.page_table[b * stride + at] = pcase.cfg.pool_pages
        pcase.cache.page_table[at] = pcase.cfg.pool_pages
        Sh.run_shared(pcase, begin, tokens, 0, q, check=False)
        assert int(pcase.cache.status.item()) == lvq.LVQ_ECAPACITY
        pcase.cache.status.zero_()
        for b in range(2):
            if at < 20:
                pcase.cache.page_table[b * stride + at] = old
        pcase.cache.page_table[at] = old
    out, lse = Sh.run_shared(pcase, begin, tokens, 0, q)
    Sh.check_against_oracle(case, 0, q, out, lse)


def test_rows_that_name_other_pages_are_reported():
    w = _w("ouro14_g32_b32", n_kv_heads=2, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(160, [30, 9, 0])], recent=[5, 9, 20])
    pcase = Sh.to_pool(case, begin, tokens)
    q = synth.queries(w, 0, 0, batch=3).cuda()
    at = 2 * pcase.cache.lay.page_table_stride + 19
    old = int(pcase.cache.page_table[at])
    pcase.cache.page_table[at] = pcase.cache.pages[0][20]
    Sh.run_shared(pcase, begin, tokens, 0, q, check=False)
    assert int(pcase.cache.status.item()) == lvq.LVQ_EINVAL
    pcase.cache.status.zero_()
    pcase.cache.page_table[at] = old
    Sh.run_shared(pcase, begin, tokens, 0, q)


def test_workspace_is_shared_with_lvq_decode_attention():
    """Calls of both kinds in turn on one workspace: the merge counters stay zero, stale partials are not read."""
    w = _w("ouro14_g16_32k", n_kv_heads=2, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(900, [3, 70])], recent=[128, 130], max_splits=16)
    q = synth.queries(w, 0, 2, batch=2).cuda()
    ref, rl, _ = Hl.run_decode(case, 0, 2, q, 7, split_lse=False)
    out, lse = Sh.run_shared(case, begin, tokens, 2, q, num_splits=16)
    got, gl, _ = Hl.run_decode(case, 0, 2, q, 7, split_lse=False)
    assert torch.equal(ref, got) and torch.equal(rl, gl)
    again = Sh.run_shared(case, begin, tokens, 2, q, num_splits=3)
    Sh.check_against_oracle(case, 2, q, out, lse)
    Sh.check_against_oracle(case, 2, q, *again)


def test_graph_replay_and_another_stream():
    """Captured once and replayed while the counters move; run on a stream that is not the current one."""
    w = _w("ouro14_g32_b32", n_kv_heads=2, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(260, [3, 70, 40])], recent=[100, 101, 102])
    pcase = Sh.to_pool(case, begin, tokens)
    c = pcase.cache
    q = synth.queries(w, 0, 1, batch=3).cuda()
    gb, gt = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (begin, tokens))
    out = torch.zeros(3, 2, w.head_dim, device="cuda")
    lse = torch.zeros(3, 2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lvq.lvq_decode_attention_shared(pcase.cfg, c.lay, 0, 1, 3, q, c.ctx_len, c.coded_len, gb, gt, c.sink, c.ring, c.idx,
                                        c.cbp, c.rope, 0, c.workspace, out, lse, c.status)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.check_status()
        Sh.check_against_oracle(case, 1, q, out.cpu(), lse.cpu())
    gt.zero_()                                    # nothing shared any more: every request on its own
    graph.replay()
    torch.cuda.synchronize()
    Sh.check_against_oracle(case, 1, q, out.cpu(), lse.cpu())
    got = Sh.run_shared(pcase, begin, tokens, 1, q, stream=torch.cuda.Stream())
    Sh.check_against_oracle(case, 1, q, *got)


def test_refusals():
    w = _w("ouro14_g32_b32", n_kv_heads=1, n_q_heads=1)
    case, begin, tokens = Sh.shared_case(w, [(16, [3, 0])], recent=[5, 9], max_splits=8)
    q = synth.queries(w, 0, 0, batch=2).cuda()
    with pytest.raises(lvq.LvqError) as e:
        Sh.run_shared(case, begin, tokens, 4, q)
    assert e.value.status == lvq.LVQ_EINVAL
    with pytest.raises(lvq.LvqError):
        Sh.run_shared(case, begin, tokens, 0, q, num_splits=9)
    with pytest.raises(lvq.LvqError):
        Sh.run_shared(case, [0, 1, 1, 2], [16, 0, 0], 0, q)                # more groups than requests
    with pytest.raises(ValueError):
        Sh.run_shared(case, begin, tokens, 0, q.float())
    with pytest.raises(ValueError):
        Sh.run_shared(case, begin, tokens, 0, q[:1])


def test_empty_groups_and_one_slot():
    """Groups without requests, and a layout whose rows have room for a single part."""
    w = _w("ouro14_g32_b32", n_kv_heads=3, n_q_heads=3)
    case, begin, tokens = Sh.shared_case(w, [(300, [3, 20]), (64, [9, 0])], recent=[5, 9, 130, 1], max_splits=1)
    q = synth.queries(w, 0, 1, batch=4).cuda()
    out, lse = Sh.run_shared(case, [0, 0, 2, 4], [77] + tokens, 1, q)
    Sh.check_against_oracle(case, 1, q, out, lse)
    out, lse = Sh.run_shared(case, [0, 2, 2, 4], [tokens[0], 1 << 20, tokens[1]], 1, q)
    Sh.check_against_oracle(case, 1, q, out, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["tiny", "ouro14_g16_32k", "ouro14_g32_b32", "ouro14_tc1_32k"])
def test_nothing_is_read_from_masked_places(name, bad):
    """Entry 255 of every codebook, the window's slots without a token and the sink's tokens past a short
    context hold NaN or infinities; no token uses that entry, but the rest of the partial last pages does."""
    w = _w(name, n_kv_heads=2, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(203, [0, 13]), (40, [2]), (0, [0])], recent=[5, 1, 11, 0], ctx=[None, None, None, 2])
    c = case.cache
    for (layer, b), (ck, cv) in case.codes.items():
        for kv, codes in ((0, ck), (1, cv)):
            codes.clamp_(max=254)
            room = c.lay.max_pages * 8
            full = torch.full((codes.shape[0], room, codes.shape[2], codes.shape[3]), 255, dtype=torch.uint8)
            full[:, :codes.shape[1]] = codes
            Hl.put_codes(c, layer, b, kv, full.cuda())
    c.cb_view()[..., 255, :] = bad
    lvq.lvq_pack_codebooks(case.cfg, c.lay, c.cb, c.cbp, c.cb_norm)
    ring = c.ring_view()
    for b in range(4):
        n_rec = case.ctx[b] - min(w.n_sink, case.ctx[b]) - case.coded[b]
        dead = [s for s in range(c.lay.ring_tokens) if s not in {(case.coded[b] + i) % c.lay.ring_tokens for i in range(n_rec)}]
        ring[:, :, :, b, :, dead] = bad
    c.sink_view()[:, :, :, 3, :, 2:] = bad
    q = synth.queries(w, 0, 1, batch=4).cuda()
    for ns in (0, 1):
        out, lse = Sh.run_shared(case, begin, tokens, 1, q, num_splits=ns)
        Sh.check_against_oracle(case, 1, q, out, lse)


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 20])
def test_scale_of_the_entries(scale):
    """Keys and values far from 1: the operands' powers of two follow the head's largest entry (queries make up for
    the keys' scale, so that the softmax stays one)."""
    w = _w("ouro14_g32_b32", n_kv_heads=2, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(300, [3, 20])], recent=[70, 9])
    c = case.cache
    for t in (c.cb, c.sink, c.ring):
        t.mul_(scale)
    case.cb[0].mul_(scale)
    for d in (case.sink_kv, case.ring_kv):
        for v in d.values():
            v.mul_(scale)
    lvq.lvq_pack_codebooks(case.cfg, c.lay, c.cb, c.cbp, c.cb_norm)
    q = (synth.queries(w, 0, 1, batch=2) / scale).to(torch.bfloat16).cuda()
    out, lse = Sh.run_shared(case, begin, tokens, 1, q)
    Sh.check_against_oracle(case, 1, q, out, lse)


def test_zero_codebooks():
    """All entries zero: the bf16 tokens alone carry values."""
    w = _w("ouro14_g16_32k", n_kv_heads=1, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(96, [3, 20])], recent=[70, 9])
    case.cache.cbp.zero_()
    case.cb[0].zero_()
    q = synth.queries(w, 0, 1, batch=2).cuda()
    out, lse = Sh.run_shared(case, begin, tokens, 1, q)
    Sh.check_against_oracle(case, 1, q, out, lse)


def test_waits_are_bounded():
    """With waits cut to a single poll the call ends, with LVQ_ETIMEOUT where the entries were not there yet, and the next one
    is right."""
    w = _w("ouro14_g32_b32", n_kv_heads=2, n_q_heads=2)
    case, begin, tokens = Sh.shared_case(w, [(300, [3, 20])], recent=[70, 9])
    q = synth.queries(w, 0, 1, batch=2).cuda()
    lvq.lvq_debug_faults(1, 0)
    try:
        Sh.run_shared(case, begin, tokens, 1, q, check=False)
    finally:
        lvq.lvq_debug_faults(0, 0)
    assert int(case.cache.status.item()) in (lvq.LVQ_OK, lvq.LVQ_ETIMEOUT)
    case.cache.status.zero_()
    out, lse = Sh.run_shared(case, begin, tokens, 1, q)
    Sh.check_against_oracle(case, 1, q, out, lse)
