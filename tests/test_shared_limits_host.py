"""Refusals of attention over shared prefixes at sizes that no test runs (no GPU needed)."""
import ctypes

import pytest
import torch

from sub_bit_kv_b200 import lvq, synth
from tests._helpers import make_cfg

FAKE = 1 << 20                       # a 16-byte-aligned address that is never touched


@pytest.fixture(scope="module", autouse=True)
def built():
    from sub_bit_kv_b200 import _build
    _build.build()


def test_more_table_entries_than_a_cta_counts_are_refused():
    """Rows of 2^25 pages, 255 of them to compare with the first: one part would count 2^33 entries."""
    cfg = make_cfg(synth.WORKLOADS["tiny"], n_layers=1, max_batch=256, max_ctx=1 << 28)
    plain = lvq.lvq_cache_layout(cfg)
    cfg.pool_pages, cfg.page_table = 50, FAKE
    lay = lvq.lvq_cache_layout(cfg)

    def attend(batch, ns, c=cfg, lay=lay):
        return lvq.lib().lvq_decode_attention_shared(ctypes.byref(c), ctypes.byref(lay), 0, 0, batch, FAKE, FAKE, FAKE, 1, FAKE, FAKE,
                                                     FAKE, FAKE, FAKE, FAKE, FAKE, ns, FAKE, FAKE, FAKE, None, None)

    assert attend(256, 1) == lvq.LVQ_EUNSUPPORTED and attend(256, 7) == lvq.LVQ_EUNSUPPORTED
    assert attend(34, 1) == lvq.LVQ_EUNSUPPORTED
    if not torch.cuda.is_available():
        assert attend(256, 8) == lvq.LVQ_EDEVICE and attend(32, 1) == lvq.LVQ_EDEVICE and attend(256, 0) == lvq.LVQ_EDEVICE
        cfg.pool_pages, cfg.page_table = 0, None
        assert attend(256, 1, cfg, plain) == lvq.LVQ_EDEVICE               # no table, nothing to compare


def test_fault_bits():
    for mask in (8, 1 << 30, -1):
        with pytest.raises(lvq.LvqError) as e:
            lvq.lvq_debug_faults(0, mask)
        assert e.value.status == lvq.LVQ_EINVAL
    lvq.lvq_debug_faults(1 << 10, 7)
    lvq.lvq_debug_faults(0, 0)
