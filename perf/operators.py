"""Operators over a paged, coded KV cache whose requests share prefixes: their cases, their plain
forms in elementary torch operations, and the calls a user makes of them.

  attend   decode attention of one (layer, loop step) for groups of requests; the coded tokens
           that a group's requests share are read and restored once for the whole group
  fork     children start as copies of a parent request: bf16 sink and recent window, counters and
           page-table row (its full pages shared, a partial last page copied), or, outside pool
           mode, its code streams
  copy     copies pages of the pool in every (layer, block, head, K/V)
  compact  renumbers the live pages of the pool 0, 1, ... in the order given, in place, and
           rewrites the page table

Shapes are those of the repository's Ouro-shaped workloads and of its small one (`tiny`).
"""
import math

import torch

own = False

OURO = dict(H=16, Hq=16, d=128, T=4)
TINY = dict(H=1, Hq=1, d=64, T=4, Tc=4, G=16)


def listed():
    return [
        # two samples of one prompt, the small workload: a call that is all latency
        dict(name="attend tiny pair", op="attend", B=2, groups=1, prefix=424, suffix=40, S=4, W=16, **TINY),
        # eight samples of one 8K prompt (0.5 bit), ragged answers
        dict(name="attend 8 of 8K", op="attend", B=8, groups=1, prefix=8191, suffix=300, S=4, W=128, Tc=4, G=16, **OURO),
        # a serving batch behind one long system prompt (0.25 bit)
        dict(name="attend 32 of 32K", op="attend", B=32, groups=1, prefix=32636, suffix=700, S=4, W=128, Tc=4, G=32, **OURO),
        # four query heads to a KV head, two steps a block, 64K of shared document
        dict(name="attend 64K, GQA", op="attend", B=8, groups=1, prefix=65276, suffix=260, S=4, W=256, H=4, Hq=16, d=128,
             T=4, Tc=2, G=16),
        # four tenants, each with a prompt of its own and an odd length; per-step coding
        dict(name="attend 4 groups", op="attend", B=48, groups=4, prefix=12345, suffix=1111, S=4, W=128, Tc=1, G=16, **OURO),
        # one sample more of a short context, per-request streams
        dict(name="fork tiny", op="fork", L=1, children=1, coded=492, recent=16, paged=False, S=4, W=16, **TINY),
        # eight samples of one prompt: every layer's window eight times, and a partial last page
        dict(name="fork 8", op="fork", L=24, children=8, coded=8187, recent=133, paged=True, S=4, W=128, Tc=4, G=16, **OURO),
        # a beam splits in two on per-request streams: 32K of codes go along
        dict(name="fork streams", op="fork", L=24, children=1, coded=32631, recent=128, paged=False, S=4, W=128, Tc=4, G=16,
             **OURO),
        # three requests get a copy of their own of the page that they are about to write
        dict(name="copy 3 pages", op="copy", L=24, pages=3, pool=600, S=4, W=128, Tc=4, G=16, **OURO),
        # a 32K prompt is duplicated to be evicted elsewhere
        dict(name="copy 4000 pages", op="copy", L=24, pages=4000, pool=8200, S=4, W=128, Tc=4, G=32, **OURO),
        # a small pool after some traffic
        dict(name="compact tiny", op="compact", L=1, live=100, pool=256, **TINY, S=4, W=16),
        # a pool that has been served from for long: three quarters in use, in no order
        dict(name="compact 12K pages", op="compact", L=24, live=12000, pool=16000, S=4, W=128, Tc=4, G=32, **OURO),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    coding = rng.choice([dict(Tc=4, G=16), dict(Tc=4, G=32), dict(Tc=2, G=16), dict(Tc=2, G=32), dict(Tc=1, G=16)])
    op = rng.choice(["attend", "attend", "attend", "fork", "copy", "compact"])
    if op == "attend":
        if rng.random() < 0.2:
            return dict(op=op, B=rng.randint(1, 16), groups=1, prefix=_log(rng, 8, 4000), suffix=_log(rng, 1, 200), S=rng.randint(0, 9),
                        W=rng.randint(1, 40), H=rng.choice([1, 2, 5]), Hq=10, d=64, T=4, Tc=4, G=rng.choice([16, 32]))
        B = _log(rng, 1, 64)
        H = rng.choice([4, 8, 16])
        rows = 16 * B
        return dict(op=op, B=B, groups=rng.randint(1, max(1, min(4, B // 2))), prefix=min(_log(rng, 100, 65000), 16 * 32 * 32000 // rows),
                    suffix=_log(rng, 1, 1200), S=rng.choice([0, 1, 4, 8]), W=rng.choice([8, 31, 128, 256]), H=H, Hq=16, d=128, T=4, **coding)
    if op == "fork":
        paged = rng.random() < 0.7
        W = rng.choice([8, 31, 128])
        return dict(op=op, L=rng.randint(1, 24), children=rng.randint(1, 8), coded=_log(rng, 1, 8000 if paged else 4000),
                    recent=W + rng.randint(0, 7), paged=paged, S=rng.choice([0, 4, 5]), W=W, **coding, **OURO)
    if op == "copy":
        pages = _log(rng, 1, 3000)
        return dict(op=op, L=rng.randint(1, 24), pages=pages, pool=2 * pages + rng.randint(1, 500), S=4, W=16, **coding, **OURO)
    live = _log(rng, 8, 5000)
    return dict(op=op, L=rng.randint(1, 24), live=live, pool=live + rng.randint(1, 1000), S=4, W=16, **coding, **OURO)


# ------------------------------------------------------------------ lengths and layouts

def _lengths(c):
    """Shared coded tokens of each group, the groups' first requests, and each request's coded
    and context lengths: ragged, and the same for every seed."""
    ng, B = c["groups"], c["B"]
    prefix = [max(1, c["prefix"] - c["prefix"] * (3 * g % 7) // 11) for g in range(ng)]
    begin = [B * g // ng for g in range(ng + 1)]
    group = [next(g for g in range(ng) if b < begin[g + 1]) for b in range(B)]
    suffix = [c["suffix"] * ((b * 59 + 13) % 97) // 96 for b in range(B)]
    coded = [prefix[group[b]] + suffix[b] for b in range(B)]
    ctx = [c["S"] + coded[b] + c["W"] + b % 8 for b in range(B)]
    shared = [p // 8 * 8 for p in prefix]        # whole pages are shared
    return shared, begin, group, coded, ctx


def _geometry(c):
    ch = c["G"] // c["Tc"]
    return dict(c=ch, ng=c["d"] // ch, nblk=c["T"] // c["Tc"], R=c["W"] + 8)


def _rope_table(max_ctx, d, base, device):
    """Rows (cos, sin)(8 k theta_f), then (cos, sin)(r theta_f) for r < 8, in 64 bits rounded once."""
    rows = max((max_ctx + 7) // 8, 64) + 16
    pos = torch.cat([8.0 * torch.arange(rows, device=device, dtype=torch.float64), torch.arange(8, device=device, dtype=torch.float64)])
    ang = pos[:, None] * base ** (-2.0 * torch.arange(d // 2, device=device, dtype=torch.float64) / d)
    return torch.stack([ang.cos(), ang.sin()], dim=-1).float().reshape(-1).contiguous()


def _config(c, L, batch, max_ctx, pool, table):
    """The handle a user's program keeps: configuration and layout."""
    from sub_bit_kv_b200 import lvq
    cfg = lvq.make_config(L, c["H"], c["Hq"], c["d"], c["T"], c["Tc"], c["G"], c["S"], c["W"], batch, max_ctx, pool_pages=pool)
    if pool:
        cfg.page_table = table.data_ptr()
    return cfg, lvq.lvq_cache_layout(cfg)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"attend": _prepare_attend, "fork": _prepare_fork, "copy": _prepare_pages, "compact": _prepare_pages}[case["op"]](case, g)


def _bytes(shape, g):
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _prepare_attend(c, g):
    """Codebook entries and tokens with lognormal channel scales, two key channels a head eight
    times larger; codes uniform; pages in shuffled runs of 16, as after some traffic."""
    geo = _geometry(c)
    shared, begin, group, coded, ctx = _lengths(c)
    B, H, d, T = c["B"], c["H"], c["d"], c["T"]
    scale = torch.exp(0.5 * torch.randn(2, H, d, generator=g, device="cuda"))
    scale[0].scatter_(1, torch.rand(H, d, generator=g, device="cuda").argsort(1)[:, :2], 8.0)
    n_pages = [(n + 7) // 8 for n in coded]
    used = sum(s // 8 for s in shared) + sum(n_pages[b] - shared[group[b]] // 8 for b in range(B))
    pool = (used + used // 3 + 31) // 16 * 16
    runs = torch.rand(pool // 16, generator=g, device="cuda").argsort()
    ids = (16 * runs[:, None] + torch.arange(16, device="cuda")).flatten().to(torch.int32)
    max_ctx = max(ctx) + 8
    P = (max_ctx - c["S"] + 7) // 8
    table = torch.full((B, (P + 3) // 4 * 4), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, s in enumerate(shared):
        table[begin[i]:begin[i + 1], :s // 8] = ids[at:at + s // 8]
        at += s // 8
    for b in range(B):
        lo, n = shared[group[b]] // 8, n_pages[b] - shared[group[b]] // 8
        table[b, lo:lo + n] = ids[at:at + n]
        at += n
    step = T - 2
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    entries = torch.randn(2, geo["nblk"], H, c["Tc"], 256, geo["ng"], geo["c"], generator=g, device="cuda")
    entries *= scale.view(2, 1, H, 1, 1, geo["ng"], geo["c"])
    tokens = lambda n: (torch.randn(2, T, B, H, n, d, generator=g, device="cuda") * scale.view(2, 1, 1, H, 1, d)).bfloat16()[None]  # noqa: E731
    s = dict(case=c, geo=geo, step=step, pool=pool, max_ctx=max_ctx, q=_normal((B, c["Hq"], d), g), table=table,
             idx=_bytes((1, geo["nblk"], H, 2, pool, geo["ng"], 8), g), cbp=entries.bfloat16()[None], sink=tokens(c["S"]),
             ring=tokens(geo["R"]), rope=_rope_table(max_ctx, d, 10000.0, "cuda"), ctx_len=ints(ctx), coded_len=ints(coded),
             group_begin=ints(begin), group_tokens=ints(shared), group=ints(group).long(),
             place=torch.tensor([b - begin[group[b]] for b in range(B)], device="cuda"),
             most=(max(begin[i + 1] - begin[i] for i in range(len(shared))), max(shared), max(n_pages[b] - shared[group[b]] // 8 for b in range(B))))
    if own:
        s["cfg"], s["lay"] = _config(c, 1, B, max_ctx, pool, table)
        s["workspace"] = torch.zeros(s["lay"].workspace_bytes // 4, device="cuda")
        s["out"] = torch.empty(B, c["Hq"], d, device="cuda")
        s["lse"] = torch.empty(B, c["Hq"], device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _prepare_fork(c, g):
    geo = _geometry(c)
    L, H, d, T, n = c["L"], c["H"], c["d"], c["T"], c["children"]
    B = n + 2                                     # the last request is a stranger
    ctx = c["S"] + c["coded"] + c["recent"]
    max_ctx = ctx + 16
    P = (max_ctx - c["S"] + 7) // 8
    full, tail = c["coded"] // 8, c["coded"] % 8 > 0
    s = dict(case=c, geo=geo, children=list(range(1, n + 1)), sink=_normal((L, 2, T, B, H, c["S"], d), g),
             ring=_normal((L, 2, T, B, H, geo["R"], d), g), ctx_len=torch.zeros(B, dtype=torch.int32, device="cuda"),
             coded_len=torch.zeros(B, dtype=torch.int32, device="cuda"), table=None, tails=None)
    s["ctx_len"][0], s["coded_len"][0] = ctx, c["coded"]
    pool = 0
    if c["paged"]:
        pool = full + n + 8
        ids = torch.rand(pool, generator=g, device="cuda").argsort().to(torch.int32)
        s["table"] = torch.full((B, (P + 3) // 4 * 4), -1, dtype=torch.int32, device="cuda")
        s["table"][0, :full + tail] = ids[:full + tail]
        s["tails"] = ids[full + 1:full + 1 + n].tolist() if tail else None
        s["idx"] = _bytes((L, geo["nblk"], H, 2, pool, geo["ng"], 8), g)
    else:
        s["idx"] = _bytes((L, geo["nblk"], B, H, 2, P, geo["ng"], 8), g)
    if own:
        s["cfg"], s["lay"] = _config(c, L, B, max_ctx, pool, s["table"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _prepare_pages(c, g):
    """copy: pairs of pages in no order; compact: the live pages' ids in the order wanted (what the
    requests' page lists hold), and a page table that four requests share them in."""
    geo = _geometry(c)
    pool = c["pool"]
    ids = torch.rand(pool, generator=g, device="cuda").argsort().to(torch.int32)
    s = dict(case=c, geo=geo, idx=_bytes((c["L"], geo["nblk"], c["H"], 2, pool, geo["ng"], 8), g))
    if c["op"] == "copy":
        s["pairs"] = torch.stack([ids[:c["pages"]], ids[c["pages"]:2 * c["pages"]]], dim=1).contiguous()
        batch, row = 1, 64
        s["table"] = torch.full((1, row), -1, dtype=torch.int32, device="cuda")
    else:
        s["order"] = ids[:c["live"]].cpu()
        batch, row = 4, ((c["live"] + 3) // 4 + 3) // 4 * 4
        s["table"] = torch.full((4, row), -1, dtype=torch.int32, device="cuda")
        s["table"].view(-1)[:c["live"]] = ids[:c["live"]]
    if own:
        s["cfg"], s["lay"] = _config(c, c["L"], batch, c["S"] + 8 * row, pool, s["table"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _attend_own, "fork": _fork_own, "copy": _copy_own, "compact": _compact_own}[op](state)
    return {"attend": _attend_plain, "fork": _fork_plain, "copy": _copy_plain, "compact": _compact_plain}[op](state)


def _attend_own(s):
    from sub_bit_kv_b200 import lvq
    lvq.lvq_decode_attention_shared(s["cfg"], s["lay"], 0, s["step"], s["case"]["B"], s["q"], s["ctx_len"], s["coded_len"],
                                    s["group_begin"], s["group_tokens"], s["sink"], s["ring"], s["idx"], s["cbp"], s["rope"], 0,
                                    s["workspace"], s["out"], s["lse"], s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _fork_own(s):
    from sub_bit_kv_b200 import lvq
    lvq.lvq_fork_requests(s["cfg"], s["lay"], 0, s["children"], s["case"]["coded"], s["tails"], s["ctx_len"], s["coded_len"], s["sink"],
                          s["ring"], s["idx"], s["table"], s["status"])
    return _fork_outputs(s)


def _copy_own(s):
    from sub_bit_kv_b200 import lvq
    lvq.lvq_copy_pages(s["cfg"], s["lay"], s["pairs"], s["idx"], s["status"])
    return {"idx": s["idx"]}


def _compact_own(s):
    from sub_bit_kv_b200 import lvq
    plan = lvq.lvq_plan_compaction(s["case"]["pool"], s["order"])
    lvq.lvq_compact_pages(s["cfg"], s["lay"], plan, s["table"], s["idx"], s["status"])
    return {"idx": s["idx"], "table": s["table"]}


def _restore(s, rows, kv):
    """fp32 tokens [n][H][pages * 8][d] of the page ids `rows` [n][pages]: the entries' shares of the step."""
    c, geo = s["case"], s["geo"]
    blk, t = divmod(s["step"], c["Tc"])
    codes = s["idx"][0, blk, :, kv][:, rows.clamp(min=0).long()]                    # [H][n][pages][n_g][8]
    codes = codes.permute(1, 0, 2, 4, 3).reshape(rows.shape[0], c["H"], -1, geo["ng"]).long()
    at = (torch.arange(c["H"], device="cuda")[:, None, None] * 256 + codes) * geo["ng"] + torch.arange(geo["ng"], device="cuda")
    return s["cbp"][0, kv, blk, :, t].reshape(-1, geo["c"])[at].float().flatten(-2)


def _rotate(x, pos, base=10000.0):
    """RoPE of x [..., tokens, d] at positions that broadcast over [..., tokens]; angles in 64 bits."""
    half = x.shape[-1] // 2
    ang = pos[..., None].double() * base ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    cos, sin = ang.cos().float(), ang.sin().float()
    return torch.cat([x[..., :half] * cos - x[..., half:] * sin, x[..., half:] * cos + x[..., :half] * sin], dim=-1)


def _attend_plain(s):
    c, geo = s["case"], s["geo"]
    B, H, d, S, R = c["B"], c["H"], c["d"], c["S"], geo["R"]
    rep = c["Hq"] // H
    size, longest, own_pages = s["most"]
    ctx, coded, group = s["ctx_len"].long(), s["coded_len"].long(), s["group"]
    shared = s["group_tokens"].long()
    q = _rotate(s["q"].float(), (ctx - 1)[:, None]).view(B, H, rep, d) / math.sqrt(d)
    # the shared tokens, restored once a group: queries of a group are the rows of one product
    ng = shared.numel()
    rows = s["table"][s["group_begin"][:-1].long(), :longest // 8]
    n = torch.arange(longest, device="cuda")
    K = _rotate(_restore(s, rows, 0), S + n)                                         # [ng][H][N][d]
    V = _restore(s, rows, 1)
    qg = torch.zeros(ng, size, H, rep, d, device="cuda")
    qg[group, s["place"]] = q
    qg = qg.permute(0, 2, 1, 3, 4).reshape(ng, H, size * rep, d)
    S1 = (qg @ K.transpose(-1, -2)).masked_fill((n >= shared[:, None])[:, None, None], -math.inf)
    # each request's own tokens: the rest of its coded ones, the sink, the recent window
    first = shared[group] // 8
    own_rows = s["table"].gather(1, (first[:, None] + torch.arange(own_pages, device="cuda")).clamp(max=s["table"].shape[1] - 1))
    m = shared[group][:, None] + torch.arange(own_pages * 8, device="cuda")
    slot = torch.arange(R, device="cuda")
    recent = coded[:, None] + (slot - coded[:, None]) % R                            # coded-region index of each slot's token
    i = torch.arange(S, device="cuda").expand(B, S)
    pos = torch.cat([S + m, i, S + recent], dim=1)
    live = torch.cat([m < coded[:, None], i < ctx[:, None], S + recent < ctx[:, None]], dim=1)
    K2 = torch.cat([_restore(s, own_rows, 0), s["sink"][0, 0, s["step"]].float(), s["ring"][0, 0, s["step"]].float()], dim=2)
    V2 = torch.cat([_restore(s, own_rows, 1), s["sink"][0, 1, s["step"]].float(), s["ring"][0, 1, s["step"]].float()], dim=2)
    S2 = (q @ _rotate(K2, pos[:, None]).transpose(-1, -2)).masked_fill(~live[:, None, None], -math.inf)   # [B][H][rep][X]
    # one softmax over both
    S1 = S1.view(ng, H, size, rep, -1).transpose(1, 2)[group, s["place"]]            # [B][H][rep][N]
    top = torch.maximum(S1.amax(-1, keepdim=True), S2.amax(-1, keepdim=True))
    P1, P2 = torch.exp(S1 - top), torch.exp(S2 - top)
    total = P1.sum(-1, keepdim=True) + P2.sum(-1, keepdim=True)
    Pg = torch.zeros(ng, size, H, rep, longest, device="cuda")
    Pg[group, s["place"]] = P1
    O1 = (Pg.permute(0, 2, 1, 3, 4).reshape(ng, H, size * rep, longest) @ V).view(ng, H, size, rep, d).transpose(1, 2)[group, s["place"]]
    out = (O1 + P2 @ V2) / total
    return {"out": out.reshape(B, c["Hq"], d), "lse": (top + total.log()).reshape(B, c["Hq"])}


def _fork_outputs(s):
    r = {k: s[k] for k in ("sink", "ring", "idx", "ctx_len", "coded_len")}
    if s["table"] is not None:
        r["table"] = s["table"]
    return r


def _fork_plain(s):
    c, geo = s["case"], s["geo"]
    kids = slice(1, 1 + c["children"])
    s["sink"][:, :, :, kids] = s["sink"][:, :, :, :1]
    live = (c["coded"] + torch.arange(c["recent"], device="cuda")) % geo["R"]        # slots of the recent tokens
    s["ring"][:, :, :, kids].index_copy_(5, live, s["ring"][:, :, :, :1].index_select(5, live).expand(-1, -1, -1, c["children"], -1, -1, -1))
    full = c["coded"] // 8
    if c["paged"]:
        s["table"][kids] = -1
        s["table"][kids, :full] = s["table"][0, :full]
        if s["tails"]:
            tails = torch.tensor(s["tails"], device="cuda")
            s["idx"][:, :, :, :, tails] = s["idx"].index_select(4, s["table"][0, full:full + 1])
            s["table"][kids, full] = tails.to(torch.int32)
    else:
        n = (c["coded"] + 7) // 8
        s["idx"][:, :, kids, :, :, :n] = s["idx"][:, :, :1, :, :, :n]
    s["ctx_len"][kids] = s["ctx_len"][0]
    s["coded_len"][kids] = s["coded_len"][0]
    return _fork_outputs(s)


def _copy_plain(s):
    pairs = s["pairs"].long()
    s["idx"].index_copy_(4, pairs[:, 1], s["idx"].index_select(4, pairs[:, 0]))
    return {"idx": s["idx"]}


def _compact_plain(s):
    order = s["order"].cuda().long()
    s["idx"][:, :, :, :, :order.numel()] = s["idx"].index_select(4, order)
    new = torch.full((s["case"]["pool"],), -1, dtype=torch.int32, device="cuda")
    new[order] = torch.arange(order.numel(), dtype=torch.int32, device="cuda")
    table = s["table"]
    table.copy_(torch.where(table >= 0, new[table.clamp(min=0).long()], -1))
    return {"idx": s["idx"], "table": table}


def work(case):
    c, geo = case, _geometry(case)
    page = 8 * geo["ng"]
    if c["op"] == "attend":
        shared, _, group, coded, ctx = _lengths(c)
        own_tokens = [coded[b] - shared[group[b]] for b in range(c["B"])]
        bf16 = [ctx[b] - coded[b] for b in range(c["B"])]
        codes = (sum(shared) + sum(own_tokens)) * 2 * geo["ng"] * c["H"]
        entries = 2 * c["H"] * 256 * c["d"] * 2
        io = c["B"] * c["Hq"] * (c["d"] * 6 + 4)
        return {"bytes": codes + entries + sum(bf16) * 2 * c["H"] * c["d"] * 2 + io, "flops": 4 * c["Hq"] * c["d"] * sum(ctx)}
    streams = c["L"] * geo["nblk"] * c["H"] * 2
    if c["op"] == "fork":
        n = c["children"]
        window = c["L"] * 2 * c["T"] * c["H"] * (c["S"] + c["recent"]) * c["d"] * 2
        pages = (1 if c["coded"] % 8 else 0) if c["paged"] else (c["coded"] + 7) // 8
        return {"bytes": (1 + n) * (window + pages * page * streams), "flops": 0}
    return {"bytes": 2 * (c["pages"] if c["op"] == "copy" else c["live"]) * page * streams, "flops": 0}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    if case["op"] == "fork":
        s = prepare(case, seed)
        alive = [(case["coded"] + i) % s["geo"]["R"] for i in range(case["recent"])]
        sink, ring = s["sink"].double(), s["ring"].double()
        for child in s["children"]:
            sink[:, :, :, child] = sink[:, :, :, 0]
            for slot in alive:
                ring[:, :, :, child, :, slot] = ring[:, :, :, 0, :, slot]
        r = dict.fromkeys(_fork_outputs(s))
        return {**r, "sink": sink, "ring": ring}
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    c, geo = case, s["geo"]
    S, R, d, step = c["S"], geo["R"], c["d"], s["step"]
    f = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    theta = 10000.0 ** (-2.0 * f / d)

    def turn(x, p):                               # x [n][d] at positions p [n], as complex numbers
        z = torch.complex(x[:, :d // 2], x[:, d // 2:]) * torch.polar(torch.ones_like(p[:, None] * theta), p[:, None] * theta)
        return torch.cat([z.real, z.imag], dim=1)

    def decode(h, kv, pages, n):                  # the first n tokens of the pages' list, [n][d]
        codes = s["idx"][0, step // c["Tc"], h, kv][pages.long()]                    # [pages][n_g][8]
        book = s["cbp"][0, kv, step // c["Tc"], h, step % c["Tc"]]                   # [256][n_g][c]
        parts = [book[:, i][codes[:, i].reshape(-1).long()] for i in range(geo["ng"])]
        return torch.cat(parts, dim=1)[:n].double()

    shared, begin, group, coded, ctx = _lengths(c)
    out = torch.empty(c["B"], c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.empty(c["B"], c["Hq"], dtype=torch.float64, device="cuda")
    where = lambda lo, n: lo + torch.arange(n, device="cuda", dtype=torch.float64)  # noqa: E731
    for h in range(c["H"]):
        for gi, n0 in enumerate(shared):
            common = s["table"][begin[gi], :n0 // 8]
            K0, V0 = turn(decode(h, 0, common, n0), where(S, n0)), decode(h, 1, common, n0)
            for b in range(begin[gi], begin[gi + 1]):
                rest = s["table"][b, n0 // 8:(coded[b] + 7) // 8]
                n1, n2, sunk = coded[b] - n0, ctx[b] - S - coded[b], min(S, ctx[b])
                slots = (coded[b] + torch.arange(n2, device="cuda")) % R
                near = [torch.cat([s["sink"][0, kv, step, b, h, :sunk], s["ring"][0, kv, step, b, h, slots]]).double() for kv in (0, 1)]
                K = torch.cat([K0, turn(decode(h, 0, rest, n1), where(S + n0, n1)),
                               turn(near[0], torch.cat([where(0, sunk), where(S + coded[b], n2)]))])
                V = torch.cat([V0, decode(h, 1, rest, n1), near[1]])
                rep = c["Hq"] // c["H"]
                qs = turn(s["q"][b, h * rep:(h + 1) * rep].double(), torch.full((rep,), ctx[b] - 1.0, device="cuda", dtype=torch.float64))
                x = qs @ K.T / math.sqrt(d)
                lse[b, h * rep:(h + 1) * rep] = torch.logsumexp(x, dim=1)
                out[b, h * rep:(h + 1) * rep] = torch.softmax(x, dim=1) @ V
    return {"out": out, "lse": lse}
