"""Test infrastructure for groups of requests that share coded prefixes: builds such caches, on per-request
streams or through the page pool, and bounds the error of an fp32 attention over them."""
import dataclasses

import numpy as np
import torch

from sub_bit_kv_b200 import lvq, synth
from tests import _helpers as Hl


def shared_case(w, groups, recent, max_splits=64, ctx=None):
    """groups: [(prefix, [own, own, ...]), ...]: each group's shared coded tokens and its requests' own ones;
    recent[b]: tokens in request b's window.  ctx: overrides context lengths (requests without coded tokens).
    Returns (case on per-request streams, group_begin, group_tokens)."""
    coded = [p + o for p, own in groups for o in own]
    begin = np.cumsum([0] + [len(own) for _, own in groups]).tolist()
    ctx = [w.n_sink + c + recent[b] if ctx is None or ctx[b] is None else ctx[b] for b, c in enumerate(coded)]
    case = Hl.build_case(w, layers=1, ctx=ctx, coded=coded, max_splits=max_splits)
    for i, (p, own) in enumerate(groups):
        lead = begin[i]
        for b in range(begin[i] + 1, begin[i + 1]):
            for kv in range(2):
                codes = case.codes[(0, b)][kv]
                codes[:, :p] = case.codes[(0, lead)][kv][:, :p]
                Hl.put_codes(case.cache, 0, b, kv, codes.cuda())
    torch.cuda.synchronize()
    return case, begin, [p for p, _ in groups]


def to_pool(case, begin, tokens, slack=37, seed=5):
    """The same cache through a page pool: a group's full shared pages once, all ids in random order."""
    need = [(c + 7) // 8 for c in case.coded]
    cfg = lvq.lvq_config.from_buffer_copy(case.cfg)
    cfg.pool_pages = sum(need) + slack
    cfg.page_table = None
    pc = lvq.CodedCache(cfg)
    for name in ("cb", "cbp", "cb_norm", "sink", "ring", "rope", "ctx_len", "coded_len"):
        getattr(pc, name).copy_(getattr(case.cache, name))
    free = np.random.default_rng(seed).permutation(cfg.pool_pages).tolist()
    sv, dv = case.cache.idx_view(), pc.idx_view()
    for i, t in enumerate(tokens):
        common = [free.pop() for _ in range(t // 8)]
        for b in range(begin[i], begin[i + 1]):
            pages = common + [free.pop() for _ in range(need[b] - t // 8)]
            for k, p in enumerate(pages):
                dv[:, :, :, :, p] = sv[:, :, b, :, :, k]
            stride = pc.lay.page_table_stride
            pc.page_table[b * stride:b * stride + len(pages)].copy_(torch.tensor(pages, dtype=torch.int32))
            pc.pages[b] = pages
    torch.cuda.synchronize()
    return dataclasses.replace(case, cfg=cfg, cache=pc)


def run_shared(case, begin, tokens, step, q, num_splits=0, layer=0, stream=None, check=True):
    c = case.cache
    B = len(case.ctx)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((B, case.w.n_q_heads, case.w.head_dim), 7.0, dtype=torch.float32, device="cuda")
    lse = torch.full((B, case.w.n_q_heads), 7.0, dtype=torch.float32, device="cuda")
    lvq.lvq_decode_attention_shared(case.cfg, c.lay, layer, step, B, q, c.ctx_len, c.coded_len, ints(begin), ints(tokens),
                                    c.sink, c.ring, c.idx, c.cbp, c.rope, num_splits, c.workspace, out, lse, c.status,
                                    stream=stream)
    torch.cuda.synchronize()
    if check:
        c.check_status("lvq_decode_attention_shared")
    return out.cpu(), lse.cpu()


def bounds(case, q):
    """(output, lse) error bounds of an fp32 evaluation, from the inputs alone.

    A score is q'.k'/sqrt(d) over rotated vectors.  Every factor is good to 2^-21 of its pair's length (the
    rotation's three fp32 roundings on each of tables, products and sums, 6 * 2^-24, and two-part fp16
    operands, 2^-22 with both), and the fp32 sum adds d / 16 * 3 roundings of 2^-24 of the running sum: in all
    below 2^-19 of |q| |k| / sqrt(d) =: A, so a score is off by at most ds = 2^-19 A.  Every weight is then off by
    exp(ds), the softmax by 2 ds of max |v|; the sums of weights and products add at most 2^-16 (256 steps
    of 2^-24, thousands of tokens being split over warps and parts)."""
    cb = Hl.f64(case.cb[0])
    step_norm = lambda x: np.sqrt((x ** 2).sum(-1))  # noqa: E731
    c = case.w.G // case.w.Tc
    e = cb[0].reshape(*cb.shape[1:-1], case.w.Tc, c)                       # [blk][H][n_g][256][Tc][c]
    kmax = np.sqrt((step_norm(e).max(axis=3) ** 2).sum(axis=2)).max()      # longest entry of every group
    vmax = np.abs(cb[1]).max()
    for b in range(len(case.ctx)):
        for t in (case.sink_kv[(0, b)], case.ring_kv[(0, b)]):
            if t.numel():
                kmax = max(kmax, step_norm(Hl.f64(t[0])).max())
                vmax = max(vmax, np.abs(Hl.f64(t[1])).max())
    ds = 2.0 ** -19 * step_norm(Hl.f64(q)).max() * kmax / np.sqrt(case.w.head_dim)
    return vmax * (2 * ds + 2.0 ** -16), ds + 2.0 ** -16


def check_against_oracle(case, step, q, out, lse, requests=None, heads=None):
    """Every (request, query head) against the fp64 oracle; the relative 2-norm over all of them as well: the
    roundings are independent, so over many values it stays within 2^-15.6 (2e-5), a tenth of the bound's size."""
    ob, lb = bounds(case, q.cpu())
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
