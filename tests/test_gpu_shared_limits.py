"""Attention over shared prefixes at the ends of its range: scores near the lowest float, waits that run out."""
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


@pytest.mark.parametrize("name,over", [("tiny", {}), ("ouro14_g16_32k", {}), ("ouro14_g32_b32", {}), ("ouro14_tc1_32k", {})])
@pytest.mark.parametrize("tokens,coded", [(8, 8), (0, 8), (0, 0)])         # shared tokens, own coded ones, bf16 ones
@pytest.mark.parametrize("log2_q,log2_k", [(56, 55), (63, 62)])
def test_scores_near_the_lowest_float(name, over, tokens, coded, log2_q, log2_k):
    """Queries and keys whose scores are all about -2^(q + k + 1) / sqrt(d), -3e32 or less: a softmax all the same.

    Only the slowest frequency's pair of channels is not small (it turns by less than 2^-9 over 8 positions).  All
    tokens have one and the same value, so the output is it whichever of them the rounding of such scores prefers.
    Weights are good to 2^-21 of their sum in numerator and denominator: outputs to 2^-16 of the largest value
    as elsewhere; the score to 2^-19 of its size, the logarithm of 8 equal weights is nothing beside it."""
    w = dataclasses.replace(synth.WORKLOADS[name], n_layers=1, n_kv_heads=2, n_q_heads=2, n_sink=0, n_recent=8, **over)
    n_bf16 = 8 if coded == 0 else 0
    case, begin, _ = Sh.shared_case(w, [(coded, [0, 0])], recent=[n_bf16, n_bf16])
    c, F, d = case.cache, w.head_dim // 2, w.head_dim
    ch = w.G // w.Tc
    cb = c.cb_view()                                                       # [L][kv][blk][H][group][256][Tc * c]
    for chan in (F - 1, d - 1):
        for s in range(w.Tc):
            cb[:, 0, :, :, chan // ch, :, s * ch + chan % ch] = -2.0 ** log2_k
    case.cb[0].copy_(cb[0].cpu())
    lvq.lvq_pack_codebooks(case.cfg, c.lay, c.cb, c.cbp, c.cb_norm)
    c.idx.zero_()
    for b in range(2):
        for t in case.codes[(0, b)]:
            t.zero_()
        ring = case.ring_kv[(0, b)]
        ring[0][..., [F - 1, d - 1]] = -2.0 ** log2_k
        ring[1].copy_(ring[1][:, :1].expand_as(ring[1]) if n_bf16 else ring[1])
        for i in range(n_bf16):
            c.ring_view()[0, :, :, b, :, (coded + i) % c.lay.ring_tokens, :] = ring[:, :, i].cuda()
    q = torch.zeros(2, 2, d, dtype=torch.bfloat16)
    q[..., [F - 1, d - 1]] = 2.0 ** log2_q
    for ns in (0, 1):
        out, lse = Sh.run_shared(case, begin, [tokens], 1, q.cuda(), num_splits=ns)
        for b in range(2):
            for h in range(2):
                ro, rl, _ = Hl.oracle_decode(case, 0, 1, b, h, q)
                assert rl < -2e32
                assert np.abs(out[b, h].double().numpy() - ro).max() <= 2.0 ** -16 * np.abs(ro).max()
                assert abs(float(lse[b, h]) - rl) <= 2.0 ** -18 * abs(rl)


@pytest.mark.parametrize("name,over", [("tiny", {}), ("ouro14_g16_32k", {}), ("ouro14_g32_b32", {}), ("ouro14_tc1_32k", {})])
def test_a_wait_that_runs_out(name, over):
    """Every CTA's values never come: the call ends with LVQ_ETIMEOUT and empty rows, and the same context then
    computes right results, this attention's and lvq_decode_attention's on the same workspace."""
    w = dataclasses.replace(synth.WORKLOADS[name], n_layers=1, n_kv_heads=2, n_q_heads=4, **over)
    case, begin, tokens = Sh.shared_case(w, [(300, [3, 200]), (0, [40])], recent=[7, 9, 11])
    pcase = Sh.to_pool(case, begin, tokens)
    q = synth.queries(w, 0, 1, batch=3).cuda()
    ref, rl, _ = Hl.run_decode(pcase, 0, 1, q, 5, split_lse=False)
    for ns in (0, 1, 7):
        lvq.lvq_debug_faults(16, 4)
        try:
            out, lse = Sh.run_shared(pcase, begin, tokens, 1, q, num_splits=ns, check=False)
        finally:
            lvq.lvq_debug_faults(0, 0)
        assert int(pcase.cache.status.item()) == lvq.LVQ_ETIMEOUT
        pcase.cache.status.zero_()
        assert (out == 0).all() and (lse == -float("inf")).all()
        out, lse = Sh.run_shared(pcase, begin, tokens, 1, q, num_splits=ns)
        Sh.check_against_oracle(case, 1, q, out, lse)
        got, gl, _ = Hl.run_decode(pcase, 0, 1, q, 5, split_lse=False)
        assert torch.equal(ref, got) and torch.equal(rl, gl)
