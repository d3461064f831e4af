"""Attention over shared prefixes at lengths where every warp's run of tiles is long (the ring of code stages refilled
again and again, the rotation taken anew every eighth tile, page ids fetched in further windows), and with as many
requests and groups as a call takes; against the fp64 oracle."""
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


def _w(name, **kw):
    return dataclasses.replace(synth.WORKLOADS[name], n_layers=1, **kw)


def _to_pool(case, begin, tokens, seed=11):
    """Sh.to_pool with a request's pages copied at once."""
    need = [(c + 7) // 8 for c in case.coded]
    cfg = lvq.lvq_config.from_buffer_copy(case.cfg)
    cfg.pool_pages = sum(need) + 9
    cfg.page_table = None
    pc = lvq.CodedCache(cfg)
    for name in ("cb", "cbp", "cb_norm", "sink", "ring", "rope", "ctx_len", "coded_len"):
        getattr(pc, name).copy_(getattr(case.cache, name))
    free = np.random.default_rng(seed).permutation(cfg.pool_pages).tolist()
    sv, dv, stride = case.cache.idx_view(), pc.idx_view(), pc.lay.page_table_stride
    for i, t in enumerate(tokens):
        common = [free.pop() for _ in range(t // 8)]
        for b in range(begin[i], begin[i + 1]):
            pages = common + [free.pop() for _ in range(need[b] - t // 8)]
            ids = torch.tensor(pages, dtype=torch.int32, device="cuda")
            dv[:, :, :, :, ids.long()] = sv[:, :, b, :, :, :len(pages)]
            pc.page_table[b * stride:b * stride + len(pages)].copy_(ids)
            pc.pages[b] = pages
    torch.cuda.synchronize()
    return dataclasses.replace(case, cfg=cfg, cache=pc)


def _check(case, step, q, out, lse, requests=None, heads=None):
    """As Sh.check_against_oracle, whose bound on a score does not count how a rotation is carried from page to page: in
    a run it turns up to 15 times by e^{i 8 theta} (7 times by e^{i 16 theta} with more channels) before it is taken from
    the tables again.  A turn rounds three times (two products of a fused sum's four, and the sum: 3 u of the pair's
    length, u = 2^-24) and repeats the table's own rounding (sqrt(2) u): 15 x 4.5 u < 2^-17.9, beside the 2^-21 there.
    Scores are then good to 2^-17.3 |q| |k| / sqrt(d) < 4 ds.  The sums: a warp's run has at most 110 tiles, two steps
    of a lane's running sum each, which with the joins stays at the 256 steps counted there; and over many values the
    roundings average out as there."""
    ob, lb = Sh.bounds(case, q.cpu())
    ds = lb - 2.0 ** -16
    ob, lb = ob + ob / (2 * ds + 2.0 ** -16) * 6 * ds, lb + 3 * ds
    num = den = 0.0
    for b in range(len(case.ctx)) if requests is None else requests:
        for hq in range(case.w.n_q_heads) if heads is None else heads:
            ro, rl, _ = Hl.oracle_decode(case, 0, step, b, hq, q.cpu())
            d = out[b, hq].numpy().astype(np.float64) - ro
            assert np.abs(d).max() <= ob, (b, hq, np.abs(d).max(), ob)
            assert abs(float(lse[b, hq]) - rl) <= lb * max(1.0, abs(rl)), (b, hq, float(lse[b, hq]), rl)
            num += (d ** 2).sum()
            den += (ro ** 2).sum()
    assert num ** 0.5 <= 2e-5 * den ** 0.5, (num / den) ** 0.5


LONG = [
    (_w("tiny"), 6011),                                                                # d = 64, c = 4
    (_w("tiny", G=32, n_kv_heads=2, n_q_heads=2, n_sink=5), 5608),                     # d = 64, c = 8
    (_w("ouro14_g16_32k", n_kv_heads=1, n_q_heads=2), 5203),                           # d = 128, c = 4
    (_w("ouro14_g32_b32", n_kv_heads=2, n_q_heads=2, n_sink=0), 6400),                 # c = 8
    (_w("ouro14_tc2_64k", n_kv_heads=1, n_q_heads=9), 5337),                           # c = 8, two blocks, 18 rows
    (_w("ouro14_tc1_32k", n_kv_heads=1, n_q_heads=1), 5999),                           # c = 16
]


@pytest.mark.parametrize("shape", range(len(LONG)))
def test_long_runs(shape):
    """One part a KV head: each of its 8 warps takes more than 40 tiles of the shared tokens; with nothing shared,
    between 80 and 110 tiles of own ones.  Shuffled pages."""
    w, prefix = LONG[shape]
    assert prefix // 16 // 8 >= 40 and 80 <= 2 * prefix // 16 // 8 and (2 * prefix + 700) // 16 // 8 + 2 <= 110
    case, begin, tokens = Sh.shared_case(w, [(prefix, [0, 211])], recent=[5, w.n_recent + 3])
    pcase = _to_pool(case, begin, tokens)
    q = synth.queries(w, 0, 1, batch=2).cuda()
    heads = None if w.n_q_heads <= 2 else [0, 7, 8]
    for shared in (tokens, [0]):
        out, lse = Sh.run_shared(pcase, begin, shared, 1, q, num_splits=1)
        _check(case, 1, q, out, lse, heads=heads)
        so, sl = Sh.run_shared(case, begin, shared, 1, q, num_splits=1)     # per-request streams: the same arithmetic
        assert torch.equal(out, so) and torch.equal(lse, sl)


def test_a_serving_batch_behind_32k():
    """32 ragged requests behind one prompt of 32636 tokens, cut as the 16-head model's heads are (9 parts): runs of 56
    shared tiles; sampled rows."""
    w = _w("ouro14_g32_b32", n_kv_heads=2, n_q_heads=2)
    own = [700 * ((b * 59 + 13) % 97) // 96 for b in range(32)]
    case, begin, tokens = Sh.shared_case(w, [(32636, own)], recent=[w.n_recent + b % 8 for b in range(32)])
    pcase = _to_pool(case, begin, tokens)
    q = synth.queries(w, 0, 2, batch=32).cuda()
    out, lse = Sh.run_shared(pcase, begin, tokens, 2, q, num_splits=9)
    _check(case, 2, q, out, lse, requests=[0, 1, 13, 15, 16, 30, 31])


@pytest.mark.parametrize("name,over", [("tiny", {}), ("ouro14_g16_32k", dict(n_recent=16)), ("ouro14_tc1_32k", dict(n_recent=16))])
@pytest.mark.parametrize("size", [1, 3, 256])
def test_as_many_requests_as_a_call_takes(name, over, size):
    """256 requests: each a group of its own, in groups of three (a last one of one), all in one."""
    w = _w(name, **over)
    w = dataclasses.replace(w, n_kv_heads=1, n_q_heads=1)
    own = [(7 * b) % 41 for b in range(256)]
    groups = [(8 * (i % 5) + i % 8 if size < 256 else 203, own[at:at + size]) for i, at in enumerate(range(0, 256, size))]
    case, begin, tokens = Sh.shared_case(w, groups, recent=[1 + b % 23 for b in range(256)])
    pcase = _to_pool(case, begin, tokens)
    assert len(tokens) == (256 + size - 1) // size
    q = synth.queries(w, 0, 1, batch=256).cuda()
    for ns in (0, 1):
        out, lse = Sh.run_shared(pcase, begin, tokens, 1, q, num_splits=ns)
        _check(case, 1, q, out, lse, requests=[*range(0, 256, 17), 127, 128, 253, 254, 255])
