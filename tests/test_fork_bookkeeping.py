"""CodedCache.fork where the fork is refused, with the device's answer played by the test (no GPU needed)."""
import pytest
import torch

from sub_bit_kv_b200 import lvq, synth
from tests._helpers import make_cfg


@pytest.fixture(scope="module", autouse=True)
def built():
    from sub_bit_kv_b200 import _build
    _build.build()


@pytest.fixture
def cache(monkeypatch):
    """A cache in host memory whose forks end with `cache.answer` in the status word they are given."""
    cfg = make_cfg(synth.WORKLOADS["tiny"], max_batch=4, max_ctx=400)
    cfg.pool_pages = 20
    c = lvq.CodedCache(cfg, device="cpu")
    c.answer = lvq.LVQ_OK

    def fork(cfg, lay, parent, children, coded, tails, ctx_len, coded_len, sink, ring, idx, table, status, stream=None):
        if c.answer != lvq.LVQ_OK:
            status.fill_(c.answer)
            return
        stride = lay.page_table_stride
        for i, ch in enumerate(children):
            row = c.pages[parent][:coded // 8] + ([tails[i]] if tails else [])
            table[ch * stride:ch * stride + len(row)] = torch.tensor(row, dtype=torch.int32)
            coded_len[ch] = coded

    monkeypatch.setattr(lvq, "lvq_fork_requests", fork)
    c.assign_pages(0, 5)
    return c


def _rows_agree(c):
    for b, pages in enumerate(c.pages):
        row = c.page_table[b * c.lay.page_table_stride:(b + 1) * c.lay.page_table_stride].tolist()
        assert row[:len(pages)] == pages and set(row[len(pages):]) <= {-1}, b
    held = [p for pages in c.pages for p in pages]
    assert [c.pool.holders(p) for p in range(20)] == [held.count(p) for p in range(20)]


@pytest.mark.parametrize("coded", [32, 37])
@pytest.mark.parametrize("answer", [lvq.LVQ_EINVAL, lvq.LVQ_ECAPACITY])
def test_refused_and_checked(cache, coded, answer):
    """The lists stay as the page table is, and the slots can be used at once."""
    cache.answer = answer
    with pytest.raises(lvq.LvqError) as e:
        cache.fork(0, [1, 3], coded, check=True)
    assert e.value.status == answer and int(cache.status.item()) == lvq.LVQ_OK
    assert cache.pages[1:] == [[], [], []] and cache.pool.available() == 15
    _rows_agree(cache)
    cache.assign_pages(3, 2)
    cache.answer = lvq.LVQ_OK
    cache.status.fill_(lvq.LVQ_ETIMEOUT)                     # another call's: it does not undo this fork
    cache.fork(0, [1, 2], coded, check=True)
    _rows_agree(cache)
    assert cache.pages[1][:4] == cache.pages[0][:4] and cache.coded_len.tolist()[1:3] == [coded, coded]


@pytest.mark.parametrize("coded", [32, 37])
def test_refused_and_released(cache, coded):
    """Not checked, the status is read later: releasing the children restores the pool and the rows."""
    cache.answer = lvq.LVQ_EINVAL
    cache.fork(0, [1, 3], coded)
    with pytest.raises(lvq.LvqError):
        cache.check_status()
    for b in (1, 3):
        cache.release(b)
    assert cache.pool.available() == 15 and cache.pool.holders(0) == 1
    _rows_agree(cache)
    cache.answer = lvq.LVQ_OK
    cache.fork(0, [3, 1, 2], coded)
    cache.check_status()
    _rows_agree(cache)


def test_a_fork_that_raises_leaves_the_pool(cache, monkeypatch):
    def fail(*a, **k):
        raise lvq.LvqError(lvq.LVQ_ECUDA, "lvq_fork_requests")

    monkeypatch.setattr(lvq, "lvq_fork_requests", fail)
    for check in (False, True):
        with pytest.raises(lvq.LvqError):
            cache.fork(0, [1, 2], 37, check=check)
        assert cache.pool.available() == 15
        _rows_agree(cache)
