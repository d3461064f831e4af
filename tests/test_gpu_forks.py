"""CodedCache.fork on the device: refused forks, and as many children as a call takes."""
import dataclasses

import pytest
import torch

from sub_bit_kv_b200 import lvq, synth
from tests import _helpers as Hl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from sub_bit_kv_b200 import _build
    _build.build()
    assert torch.cuda.is_available()


def _cache(pool, batch, n_recent=12, **kw):
    w = dataclasses.replace(synth.WORKLOADS["ouro14_tc2_64k"], n_layers=2, n_kv_heads=2, n_q_heads=2, n_recent=n_recent, n_sink=3, **kw)
    cfg = Hl.make_cfg(w, max_batch=batch, max_ctx=600)
    cfg.pool_pages = pool
    c = lvq.CodedCache(cfg)
    g = torch.Generator(device="cuda")
    g.manual_seed(batch)
    c.idx.random_(0, 256, generator=g)
    for t in (c.sink, c.ring):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    return w, c


def _held_as_named(c):
    stride = c.lay.page_table_stride
    held = [p for pages in c.pages for p in pages]
    for b, pages in enumerate(c.pages):
        row = c.page_table[b * stride:(b + 1) * stride].tolist()
        assert row[:len(pages)] == pages and set(row[len(pages):]) <= {-1}, b
    assert c.pool.available() == c.cfg.pool_pages - len(set(held))


@pytest.mark.parametrize("other_stream", [False, True])
def test_refused_fork(other_stream):
    """The parent has 43 coded tokens, the caller says 35: checked, nothing is held; not checked, releasing the
    children restores the pool.  A status that another call left does not undo a fork."""
    w, c = _cache(30, 4)
    s = torch.cuda.Stream() if other_stream else None
    c.assign_pages(0, 6)
    c.ctx_len[0], c.coded_len[0] = w.n_sink + 43 + 5, 43
    torch.cuda.synchronize()
    with pytest.raises(lvq.LvqError) as e:
        c.fork(0, [1, 3], 35, stream=s, check=True)
    assert e.value.status == lvq.LVQ_EINVAL and int(c.status.item()) == lvq.LVQ_OK
    assert c.pages[1:] == [[], [], []] and c.pool.available() == 24
    _held_as_named(c)
    c.fork(0, [1, 3], 35, stream=s)
    torch.cuda.synchronize()
    with pytest.raises(lvq.LvqError):
        c.check_status()
    for b in (1, 3):
        c.release(b)
    _held_as_named(c)
    assert [c.pool.holders(p) for p in c.pages[0]] == [1] * 6
    c.status.fill_(lvq.LVQ_ETIMEOUT)
    torch.cuda.synchronize()
    c.fork(0, [3, 1], 43, stream=s, check=True)
    _held_as_named(c)
    assert c.coded_len.tolist() == [43, 43, 0, 43] and c.pages[3][:5] == c.pages[0][:5]
    iv = c.idx_view()
    for b in (1, 3):
        assert torch.equal(iv[:, :, :, :, c.pages[b][5]], iv[:, :, :, :, c.pages[0][5]])


def test_check_is_refused_under_capture():
    w, c = _cache(30, 3)
    c.assign_pages(0, 6)
    c.ctx_len[0], c.coded_len[0] = w.n_sink + 43 + 5, 43
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            c.fork(0, [1], 43, check=True)
        c.page_table.add_(0)
    assert c.pages[1] == [] and c.pool.available() == 24


@pytest.mark.parametrize("paged", [True, False])
def test_as_many_children_as_a_call_takes(paged):
    """256 children, in no order, of a parent in the middle of the batch: windows, counters, pages, and the
    request that is no child left as it was."""
    B, parent, coded, recent = 258, 100, 21, 9
    w, c = _cache(300 if paged else 0, B, n_recent=8)
    children = [b for b in torch.randperm(B, generator=torch.Generator().manual_seed(1)).tolist() if b != parent][:256]
    spared = next(b for b in range(B) if b != parent and b not in children)
    if paged:
        c.assign_pages(parent, 3)
    c.ctx_len[parent], c.coded_len[parent] = w.n_sink + coded + recent, coded
    sv, rv, iv = c.sink_view().clone(), c.ring_view().clone(), c.idx_view().clone()
    slots = [(coded + i) % c.lay.ring_tokens for i in range(recent)]
    ch = torch.tensor(children, device="cuda")
    sv[:, :, :, ch] = sv[:, :, :, parent:parent + 1]
    for s in slots:
        rv[:, :, :, ch, :, s] = rv[:, :, :, parent:parent + 1, :, s]
    c.fork(parent, children, coded, check=True)
    if paged:
        tails = torch.tensor([c.pages[b][2] for b in children], device="cuda")
        assert len(set(tails.tolist())) == 256
        iv[:, :, :, :, tails] = iv[:, :, :, :, c.pages[parent][2]].unsqueeze(4)
        _held_as_named(c)
        assert [c.pool.holders(p) for p in c.pages[parent]] == [257, 257, 1]
    else:
        iv[:, :, ch, :, :, :3] = iv[:, :, parent:parent + 1, :, :, :3]
    assert torch.equal(c.sink_view(), sv) and torch.equal(c.ring_view(), rv) and torch.equal(c.idx_view(), iv)
    want = [0 if b == spared else coded for b in range(B)]
    assert c.coded_len.tolist() == want and c.ctx_len.tolist() == [x and x + w.n_sink + recent for x in want]
    with pytest.raises(lvq.LvqError) as e:
        lvq.lvq_fork_requests(c.cfg, c.lay, parent, [b for b in range(B) if b != parent], 24, None, c.ctx_len, c.coded_len, c.sink,
                              c.ring, c.idx, c.page_table if paged else None, c.status)
    assert e.value.status == lvq.LVQ_EUNSUPPORTED
