"""Compaction of pools with many streams, whose pages a CTA moves 128 bytes at a time (few streams: 64, as in the
other tests): every byte against plain indexing."""
import dataclasses

import numpy as np
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


# (workload, layers, KV heads): pages of 256 bytes (two CTAs side by side), 128, and 128 of d = 64
SHAPES = [("ouro14_g16_32k", 5, 16), ("ouro14_tc2_64k", 6, 16), ("tiny", 160, 1)]


def _orders():
    rng = np.random.default_rng(3)
    yield 1, [0]
    yield 300, list(range(300))                                            # nothing to move
    yield 300, [(i + 1) % 300 for i in range(300)]                         # one cycle through five slabs
    yield 257, list(range(256, -1, -1))                                    # cycles of two, over slab borders
    yield 1024, rng.permutation(1024).tolist()                             # a full pool: cycles only
    yield 1500, rng.permutation(1500)[:900].tolist()                       # chains and cycles
    sizes, order, at = [2, 3, 62, 63, 64, 65, 126, 127, 128, 129, 300, 2, 500, 1, 128], [], 0
    for k in sizes:                                                        # cycles shorter than a slab, as long, longer,
        order += [at + (i + 1) % k for i in range(k)]                      # back to back: the hold page changes hands in a slab
        at += k
    yield at, order
    yield 900, [899, 5, 7] + [i for i in range(100, 400)]                  # a few far pages, then one long chain


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("case", range(8))
def test_compact_pages(shape, case):
    name, layers, heads = SHAPES[shape]
    pool, order = list(_orders())[case]
    w = dataclasses.replace(synth.WORKLOADS[name], n_layers=layers, n_kv_heads=heads, n_q_heads=heads, n_recent=8)
    cfg = Hl.make_cfg(w, max_batch=2, max_ctx=2000)
    cfg.pool_pages = pool
    c = lvq.CodedCache(cfg)
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    streams = layers * c.lay.n_blocks * heads * 2
    assert c.lay.page_bytes >= 128 and streams * (c.lay.page_bytes // 128) >= 2 * n_sm      # (the wide kernel's rule)
    g = torch.Generator(device="cuda")
    g.manual_seed(case)
    c.idx.random_(0, 256, generator=g)
    first = list(dict.fromkeys(order))
    ref = c.idx_view().clone()
    ref[:, :, :, :, :len(first)] = c.idx_view()[:, :, :, :, torch.tensor(first, dtype=torch.long, device="cuda")]
    table = np.random.default_rng(case).integers(-1, pool, c.page_table.numel()).astype(np.int32)
    table[3], table[9] = pool, -7                                          # not pages: they stay
    c.page_table.copy_(torch.from_numpy(table))
    new = {p: i for i, p in enumerate(first)}
    want = [new.get(int(p), -1) if 0 <= p < pool else int(p) for p in table]
    plan = lvq.lvq_plan_compaction(pool, order)
    lvq.lvq_compact_pages(cfg, c.lay, plan, c.page_table, c.idx, c.status)
    torch.cuda.synchronize()
    c.check_status()
    assert torch.equal(c.idx_view(), ref)
    assert c.page_table.cpu().tolist() == want
