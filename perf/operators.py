"""The paged 8-bit KV cache's operators, measured: the page plan (block tables and slot maps from
request lengths), the write that quantises new rows into pages, and the attention that reads them.

A page holds `page` consecutive tokens (or compressed entries) of one request; the codes are E4M3
[n_pages, Hkv, page, d] with one fp32 scale per page and KV head.  Where `own` is false `run`
computes the plain form with elementary torch operations in 32 bits."""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TINY = 2.0 ** -126


def listed():
    return [
        # one decode step of eight long sequences (up to a million tokens each): latency
        dict(name="plan_decode", op="plan", B=8, page=64, ctx=1048576, new=1, T=8),
        # continuous batching with short pages: many requests, some of them new prompts
        dict(name="plan_batch", op="plan", B=1024, page=16, ctx=8192, new=64, T=65536),
        # one token for each of 32 sequences, grouped heads
        dict(name="write_decode", op="write", B=32, new=1, ctx=500, page=64, Hkv=8, d=128, shared=False),
        # 4096 new tokens of a layer whose rows are both key and value
        dict(name="write_chunk_shared", op="write", B=1, new=4096, ctx=1000, page=64, Hkv=1, d=128, shared=True),
        # prompts of four sequences, grouped heads, odd ends
        dict(name="write_prompts", op="write", B=4, new=16383, ctx=100, page=64, Hkv=8, d=128, shared=False),
        # HCA decode: dense over 512 compressed entries (128 tokens each), 16 heads on one shared row
        dict(name="attn_hca_decode", op="attn", B=4, H=16, Hkv=1, d=128, page=64, shared=True, new=1, len=512,
             m=128, W=0, sink=True),
        # one token for each of 32 sequences of ragged lengths, grouped heads
        dict(name="attn_decode_gqa", op="attn", B=32, H=64, Hkv=8, d=128, page=64, shared=False, new=1, len=32768,
             m=1, W=0, sink=False),
        # a few draft tokens at once, small heads, short pages
        dict(name="attn_draft_d64", op="attn", B=61, H=32, Hkv=8, d=64, page=16, shared=False, new=4, len=5000,
             m=1, W=0, sink=False),
        # decode at long context, 128 heads on one shared row
        dict(name="attn_decode_mqa", op="attn", B=8, H=128, Hkv=1, d=128, page=128, shared=True, new=1, len=131072,
             m=1, W=0, sink=True),
        # the raw window's branch over a ragged batch of chunks
        dict(name="attn_window_chunks", op="attn", B=7, H=16, Hkv=1, d=128, page=32, shared=True, new=1025, len=5000,
             m=1, W=128, sink=False),
        # a causal chunk at the end of a long context
        dict(name="attn_chunk_long", op="attn", B=1, H=16, Hkv=1, d=128, page=64, shared=True, new=2048, len=65536,
             m=1, W=0, sink=False),
        # prompts from their start, grouped heads
        dict(name="attn_prompts_gqa", op="attn", B=4, H=32, Hkv=4, d=128, page=64, shared=False, new=4096, len=4096,
             m=1, W=0, sink=False),
    ]


def _logu(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _logu(rng, 1, 1024)
        new = 1 if rng.random() < 0.5 else _logu(rng, 2, max(2, 65536 // B))
        ctx = _logu(rng, 1, min(1048576, (4 << 20) * page // (16 * B)))
        return dict(op="plan", B=B, page=page, ctx=ctx, new=new, T=B * new + rng.randrange(0, 8))
    d = rng.choice([64, 128])
    shared = rng.random() < 0.4
    if op == "write":
        Hkv = 1 if shared else rng.choice([1, 2, 4, 8])
        B = _logu(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _logu(rng, 2, max(2, 32768 // B))
        return dict(op="write", B=B, new=new, ctx=_logu(rng, 1, 1000), page=page, Hkv=Hkv, d=d, shared=shared)
    Hkv = 1 if shared else rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16]) if Hkv > 1 else rng.choice([1, 4, 7, 8, 16, 32, 64, 128])
    B = _logu(rng, 1, 64)
    new = 1 if rng.random() < 0.5 else _logu(rng, 2, max(2, 4096 // B))
    most = min(131072, (1 << 31) // (B * Hkv * G * new), (1 << 29) // (B * Hkv * d))
    length = _logu(rng, min(new, most), max(min(new, most), most))
    m = rng.choice([1, 1, 1, 4, 128])
    W = rng.choice([0, 0, 128, 511]) if m == 1 else 0
    return dict(op="attn", B=B, H=Hkv * G, Hkv=Hkv, d=d, page=page, shared=shared, new=min(new, length), len=length,
                m=m, W=W, sink=rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------
# lengths: a spread over the batch that the case alone fixes (the seed shuffles who has which)


def _spread(n, hi, lo_frac):
    """n whole numbers from hi * lo_frac to hi; the first is hi."""
    x = [1.0 if i == 0 else lo_frac + (1 - lo_frac) * ((i * 0.6180339887498949) % 1.0) for i in range(n)]
    return [max(1, int(hi * v)) for v in x]


def _plan_lengths(case):
    seq = _spread(case["B"], case["ctx"], 0.05)
    keep, new = [], []
    fresh = case["new"] > 1
    for b, s in enumerate(seq):
        if fresh and b % 4 == 1:
            keep.append(0)              # the row has a new request: its predecessor's pages come back
        elif b % 8 == 3:
            keep.append(max(0, s - 3))  # rejected draft tokens
        else:
            keep.append(s)
    for b in range(case["B"]):
        if case["new"] == 1:
            new.append(0 if b % 16 == 9 else 1)
        else:
            new.append(case["new"] if b % 4 == 1 else 1 + (b * 7) % max(1, case["new"] // 4))
    return seq, keep, new


def _attn_lengths(case):
    """(kv_len, new, q_start) of each request: rows held (new ones among them), queries, position of the first."""
    lens = _spread(case["B"], case["len"], 0.25)
    news = [case["new"]] * case["B"]
    if case["new"] > 8:
        news = _spread(case["B"], case["new"], 0.5)
    news = [min(n, l) if case["m"] == 1 else n for n, l in zip(news, lens)]
    if case["m"] == 1:
        start = [l - n for l, n in zip(lens, news)]
    else:
        start = [max(0, l * case["m"] - n) for l, n in zip(lens, news)]
    return lens, news, start


def _visible(case, lens, start, i):
    """[lo, hi) of the rows that query i of a request sees."""
    p = start + i
    hi = min(lens, (p + 1) // case["m"])
    lo = max(0, p - case["W"] + 1) if case["W"] else 0
    return min(lo, hi), hi


def work(case):
    if case["op"] == "plan":
        seq, keep, new = _plan_lengths(case)
        pg = case["page"]
        up = lambda x: -(-x // pg)  # noqa: E731
        back = sum(up(s) - up(k) for s, k in zip(seq, keep))
        need = sum(up(k + n) - up(k) for k, n in zip(keep, new))
        return {"bytes": 16 * case["B"] + 8 * case["T"] + 8 * (back + need), "flops": 0}
    if case["op"] == "write":
        n = sum(_write_lengths(case)[1]) * case["Hkv"] * case["d"] * (1 if case["shared"] else 2)
        return {"bytes": 3 * n + 4 * sum(_write_lengths(case)[1]), "flops": 2 * n}
    lens, news, start = _attn_lengths(case)
    pairs = rows = 0
    for l, n, s in zip(lens, news, start):
        span = [_visible(case, l, s, i) for i in range(n)]
        pairs += sum(hi - lo for lo, hi in span)
        rows += max(hi for _, hi in span) - min(lo for lo, _ in span)
    T = sum(news)
    size = rows * case["Hkv"] * case["d"] * (1 if case["shared"] else 2)
    return {"bytes": size + 4 * T * case["H"] * case["d"] + 4 * T * case["H"],
            "flops": 4 * case["d"] * case["H"] * pairs}


def _write_lengths(case):
    ctx = _spread(case["B"], case["ctx"], 0.1)
    new = [case["new"]] * case["B"] if case["new"] == 1 else _spread(case["B"], case["new"], 0.6)
    return ctx, new


# ---------------------------------------------------------------------------------------------
# what a program has in hand


def _table(lens, page, gen):
    """Pages for the lengths, in random order; a few spare ones."""
    per = [-(-l // page) for l in lens]
    n = sum(per) + 5
    order = torch.randperm(n, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k]
        at += k
    return table, n


def _codes(shape, gen):
    """E4M3 codes of values as a quantised layer holds them: normal, the page's largest near the top."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16).mul_(100.0).clamp_(-448, 448)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(n, h, gen, mid):
    """Powers of two around `mid`, as the write gives them."""
    return torch.exp2(torch.randint(-1, 2, (n, h), generator=gen, device=DEV).float() + mid).contiguous()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    perm = torch.randperm(case["B"], generator=cpu).tolist()
    mix = lambda v: [v[i] for i in perm]  # noqa: E731
    if case["op"] == "plan":
        seq, keep, new = (mix(v) for v in _plan_lengths(case))
        page = case["page"]
        longest = max(max(a, k + n) for a, k, n in zip(seq, keep, new))
        held, _ = _table(seq, page, cpu)
        spare = sum(-(-(k + n) // page) for k, n in zip(keep, new))
        n_pages = int((held >= 0).sum()) + spare + 64
        order = torch.randperm(n_pages, generator=cpu).to(torch.int32)
        table = torch.full((case["B"], -(-longest // page)), -1, dtype=torch.int32)
        taken = held >= 0
        count = int(taken.sum())
        table[:, :held.shape[1]][taken] = order[:count]
        free = torch.full((n_pages,), -1, dtype=torch.int32)
        free[:n_pages - count] = order[count:]
        T = case["T"]
        empty = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
        s.update(seq_len=_i32(seq), keep=_i32(keep), new_len=_i32(new), table=table.to(DEV), free_list=free.to(DEV),
                 n_free=_i32([n_pages - count]), page=page, cu_new=empty(case["B"] + 1), pos=empty(T), slot=empty(T),
                 status=torch.zeros(1, dtype=torch.int32, device=DEV))
    elif case["op"] == "write":
        ctx, new = (mix(v) for v in _write_lengths(case))
        page, Hkv, d = case["page"], case["Hkv"], case["d"]
        # the pages that the new tokens reach: a request's last, partly filled one and those after
        first = [c // page * page for c in ctx]
        table, n_pages = _table([c + n - f for c, n, f in zip(ctx, new, first)], page, cpu)
        slot = []
        for b in range(case["B"]):
            at = torch.arange(ctx[b] - first[b], ctx[b] - first[b] + new[b])
            slot.append(table[b, at // page] * page + (at % page).to(torch.int32))
        T = sum(new)

        def rows():
            x = torch.randn(T, Hkv, d, generator=gen, device=DEV)
            return (x * torch.exp2(torch.randn(T, Hkv, 1, generator=gen, device=DEV))).to(torch.bfloat16)

        shape = (n_pages, Hkv, page, d)
        s.update(slot=torch.cat(slot).to(torch.int32).to(DEV), k_new=rows(), k=_codes(shape, gen),
                 k_scale=_scales(n_pages, Hkv, gen, -6.0), v_new=None, v=None, v_scale=None,
                 status=torch.zeros(1, dtype=torch.int32, device=DEV))
        if not case["shared"]:
            s.update(v_new=rows(), v=_codes(shape, gen), v_scale=_scales(n_pages, Hkv, gen, -6.0))
    else:
        lens, news, start = (mix(v) for v in _attn_lengths(case))
        table, n_pages = _table(lens, case["page"], cpu)
        shape = (n_pages, case["Hkv"], case["page"], case["d"])
        T = sum(news)
        cu = np.concatenate([[0], np.cumsum(news)]).tolist()
        s.update(q=torch.randn(T, case["H"], case["d"], generator=gen, device=DEV).mul_(1.5).to(torch.bfloat16),
                 cu_q=_i32(cu), q_start=_i32(start), kv_len=_i32(lens), table=table.to(DEV), k=_codes(shape, gen),
                 k_scale=_scales(n_pages, case["Hkv"], gen, -6.0), v=None, v_scale=None, max_q=max(news),
                 sink=torch.randn(case["H"], generator=gen, device=DEV) if case["sink"] else None,
                 scale=1.0 / math.sqrt(case["d"]),
                 out=torch.empty(T, case["H"], case["d"], dtype=torch.bfloat16, device=DEV),
                 lse=torch.empty(T, case["H"], dtype=torch.float32, device=DEV),
                 status=torch.zeros(1, dtype=torch.int32, device=DEV))
        if not case["shared"]:
            s.update(v=_codes(shape, gen), v_scale=_scales(n_pages, case["Hkv"], gen, -6.0))
    if own and case["op"] != "plan":
        from heavily_compressed_long_b200 import api
        s["store"] = api.PagedKV(s["k"], s["k_scale"], s["v"], s["v_scale"])
        if case["op"] == "attn":
            n = api.paged_attn_workspace_bytes(s["q"].shape[0], case["H"], case["Hkv"], case["d"])
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(s):
    op = s["case"]["op"]
    if op == "plan":
        if own:
            from heavily_compressed_long_b200 import api
            api.hcl_page_plan(s["keep"], s["new_len"], s["seq_len"], s["table"], s["free_list"], s["n_free"],
                              s["page"], s["cu_new"], s["pos"], s["slot"], status=s["status"])
        else:
            _plan_plain(s)
        return {k: s[k] for k in ("seq_len", "table", "n_free", "cu_new", "pos", "slot")}
    if op == "write":
        if own:
            from heavily_compressed_long_b200 import api
            api.hcl_paged_write(s["k_new"], s["v_new"], s["slot"], s["store"], status=s["status"])
        else:
            _write_plain(s["k_new"], s["slot"], s["k"], s["k_scale"])
            if s["v"] is not None:
                _write_plain(s["v_new"], s["slot"], s["v"], s["v_scale"])
        out = {"k": s["k"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"]}
        if s["v"] is not None:
            out.update(v=s["v"].view(torch.float8_e4m3fn), v_scale=s["v_scale"])
        return out
    if own:
        from heavily_compressed_long_b200 import api
        api.hcl_paged_attn(s["q"], s["cu_q"], s["q_start"], s["store"], s["table"], s["kv_len"], s["out"],
                           lse=s["lse"], m=s["case"]["m"], W=s["case"]["W"], max_q=s["max_q"], scale=s["scale"],
                           sink=s["sink"], ws=s["ws"], status=s["status"])
        return {"out": s["out"], "lse": s["lse"]}
    return _attn_plain(s)


def _plan_plain(s):
    page, T = s["page"], s["slot"].shape[0]
    seq, keep, new, table, free = s["seq_len"], s["keep"], s["new_len"], s["table"], s["free_list"]
    up = lambda x: torch.div(x + page - 1, page, rounding_mode="floor")  # noqa: E731
    old, kept, want = up(seq), up(keep), up(keep + new)
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    back = (j >= kept[:, None]) & (j < old[:, None])
    ids = table[back]
    top = s["n_free"] + ids.numel()
    free[(top - 1 - torch.arange(ids.numel(), device=DEV)).long()] = ids
    need = (j >= kept[:, None]) & (j < want[:, None])
    count = need.sum()
    rank = torch.cumsum(need.flatten(), 0).view_as(need) - 1
    got = free[(top - 1 - rank).clamp(0, free.numel() - 1).long()]
    table.copy_(torch.where(need, got, torch.where(back, torch.full_like(table, -1), table)))
    cu = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0)).to(torch.int32)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=seq.numel() - 1)
    pos = keep[b] + (t - cu[b])
    live = t < cu[-1]
    at = torch.where(live, pos, torch.zeros_like(pos))
    slot = table[b, torch.div(at, page, rounding_mode="floor").long()] * page + at % page
    s["pos"].copy_(torch.where(live, pos, torch.full_like(pos, -1)))
    s["slot"].copy_(torch.where(live, slot, torch.full_like(slot, -1)))
    s["cu_new"].copy_(cu)
    s["n_free"].copy_(top - count)
    seq.copy_(keep + new)


def _write_plain(x, slot, codes, scale):
    page = codes.shape[2]
    x = x.float()
    at = torch.div(slot, page, rounding_mode="floor").long()
    ids, where = torch.unique(at, return_inverse=True)
    off = (slot % page).long()
    first = torch.full((ids.numel(),), page, dtype=torch.long, device=DEV).scatter_reduce(0, where, off, "amin")
    amax = torch.zeros(ids.numel(), x.shape[1], device=DEV).index_reduce_(0, where, x.abs().amax(-1), "amax")
    mant, expo = torch.frexp(amax)                       # amax = mant * 2^expo, 0.5 <= mant < 1
    need = torch.ldexp(torch.ones_like(amax), torch.where(mant > 0.875, expo - 8, expo - 9))
    need = torch.where(amax > 0, need.clamp(min=TINY), torch.full_like(need, TINY))
    was = scale[ids]
    now = torch.where((first == 0)[:, None], need, torch.maximum(was, need))
    held = codes[ids]
    again = held.view(torch.float8_e4m3fn).float() * (was / now)[:, :, None, None]
    again = again.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    before = torch.arange(page, device=DEV)[None, :] < first[:, None]
    codes[ids] = torch.where(before[:, None, :, None], again, held)
    scale[ids] = now
    fresh = (x / now[where][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[at, :, off] = fresh


def _attn_plain(s):
    c = s["case"]
    B, H, Hkv, d, page, m, W = c["B"], c["H"], c["Hkv"], c["d"], c["page"], c["m"], c["W"]
    q, cu, lens, table = s["q"], s["cu_q"].long(), s["kv_len"].long(), s["table"].long()
    T, G, Q = q.shape[0], H // Hkv, s["max_q"]
    N = table.shape[1] * page
    pages = table.clamp(min=0)

    def rows(codes, scale):  # [B, Hkv, N, d]
        x = codes.view(torch.float8_e4m3fn)[pages.flatten()].float() * scale[pages.flatten()][:, :, None, None]
        x = x.view(B, -1, Hkv, page, d).transpose(1, 2).reshape(B, Hkv, N, d)
        return x.masked_fill_((torch.arange(N, device=DEV)[None, :] >= lens[:, None])[:, None, :, None], 0.0)

    k = rows(s["k"], s["k_scale"])
    v = k if s["v"] is None else rows(s["v"], s["v_scale"])
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[b]
    qp = torch.zeros(B, Q, H, d, device=DEV)
    qp[b, i] = q.float()
    qp = qp.view(B, Q, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, d)
    z = torch.matmul(qp, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, G, Q, N)
    p = s["q_start"].long()[:, None] + torch.arange(Q, device=DEV)[None, :]
    j = torch.arange(N, device=DEV)[None, None, :]
    seen = (j < lens[:, None, None]) & (m * (j + 1) - 1 <= p[:, :, None])
    if W:
        seen &= j > p[:, :, None] - W
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, Hkv, G, 1, 1)
        top = torch.maximum(top, sink)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    z.sub_(base).exp_()
    total = z.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - base)
    o = torch.matmul(z.view(B, Hkv, G * Q, N), v).view(B, Hkv, G, Q, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (torch.log(total) + base)[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, H, d)[b, i]
    return {"out": o.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(B, Q, H)[b, i]}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    with torch.no_grad():
        return {"plan": _plan_exact, "write": _write_exact, "attn": _attn_exact}[case["op"]](prepare(case, seed))


def _plan_exact(s):
    """The plan as a list of free pages and a loop over the requests would do it."""
    page, B, T = s["page"], s["case"]["B"], s["case"]["T"]
    seq, keep, new = s["seq_len"].tolist(), s["keep"].tolist(), s["new_len"].tolist()
    table = s["table"].cpu().numpy().copy()
    stack = s["free_list"][:s["n_free"].item()].tolist()
    held = lambda n: (n + page - 1) // page  # noqa: E731
    for b in reversed(range(B)):
        for at in reversed(range(held(keep[b]), held(seq[b]))):
            stack.append(int(table[b, at]))
            table[b, at] = -1
    cu, pos, slot = [0], [], []
    for b in range(B):
        for at in range(held(keep[b]), held(keep[b] + new[b])):
            table[b, at] = stack.pop()
        for p in range(keep[b], keep[b] + new[b]):
            pos.append(p)
            slot.append(int(table[b, p // page]) * page + p % page)
        cu.append(len(pos))
    pad = [-1] * (T - len(pos))
    t = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32)  # noqa: E731
    return {"seq_len": t([k + n for k, n in zip(keep, new)]), "table": t(table), "n_free": t([len(stack)]),
            "cu_new": t(cu), "pos": t(pos + pad), "slot": t(slot + pad)}


def _e4m3(x):
    """The nearest E4M3 value of a float64 tensor, ties to even, the largest being 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _write_exact(s):
    out = {}
    page = s["case"]["page"]
    slot = s["slot"].long()
    for name in ("k", "v"):
        if s[name] is None:
            continue
        codes = s[name].view(torch.float8_e4m3fn).double()
        scale = s[name + "_scale"].double()
        x = s[name + "_new"].double()
        n_pages, Hkv = scale.shape
        # each value of the batch in its place of a cache-shaped array, NaN where nothing is written
        put = torch.full_like(codes, math.nan)
        put[slot // page, :, slot % page] = x
        there = ~torch.isnan(put[:, 0, :, 0])                          # [n_pages, page]
        touched = there.any(1)
        amax = torch.nan_to_num(put, nan=0.0).abs().amax((2, 3))
        half, e = torch.frexp((amax / 448.0).clamp(min=TINY))           # half * 2^e, 0.5 <= half < 1
        least = torch.ldexp(torch.ones_like(half), torch.where(half == 0.5, e - 1, e))
        fresh = there[:, 0]
        now = torch.where(fresh[:, None], least, torch.maximum(scale, least))
        now = torch.where(touched[:, None], now, scale)
        ahead = (torch.cumsum(there.long(), 1) == 0) & touched[:, None]  # rows before the first new one
        moved = _e4m3(codes * (scale / now)[:, :, None, None])
        codes = torch.where(ahead[:, None, :, None], moved, codes)
        codes = torch.where(there[:, None, :, None], _e4m3(put / now[:, :, None, None]), codes)
        out[name], out[name + "_scale"] = codes, now
    return out


def _attn_exact(s):
    c = s["case"]
    H, Hkv, d, page = c["H"], c["Hkv"], c["d"], c["page"]
    G = H // Hkv
    cu, lens, start = s["cu_q"].tolist(), s["kv_len"].tolist(), s["q_start"].tolist()
    out = torch.zeros(s["q"].shape[0], H, d, dtype=torch.float64, device=DEV)
    lse = torch.full((s["q"].shape[0], H), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        L, n = lens[b], cu[b + 1] - cu[b]
        ids = s["table"][b, :-(-L // page)].long()
        j = torch.arange(L, device=DEV)
        for g in range(Hkv):
            k = (s["k"][ids, g].view(torch.float8_e4m3fn).double() * s["k_scale"][ids, g].double()[:, None, None])
            k = k.reshape(-1, d)[:L]
            v = k
            if s["v"] is not None:
                v = (s["v"][ids, g].view(torch.float8_e4m3fn).double() * s["v_scale"][ids, g].double()[:, None, None])
                v = v.reshape(-1, d)[:L]
            step = max(1, (1 << 28) // (G * max(L, 1)))
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                rows = s["q"][cu[b] + i0:cu[b] + i1, g * G:(g + 1) * G].double()
                z = torch.einsum("qhd,nd->qhn", rows, k) * s["scale"]
                p = start[b] + torch.arange(i0, i1, device=DEV)
                hide = (j[None, :] + 1) * c["m"] - 1 > p[:, None]
                if c["W"]:
                    hide |= j[None, :] <= p[:, None] - c["W"]
                z.masked_fill_(hide[:, None, :], -math.inf)
                if s["sink"] is not None:
                    z = torch.cat([z, s["sink"][g * G:(g + 1) * G].double()[None, :, None].expand(i1 - i0, G, 1)], 2)
                l = torch.logsumexp(z, 2)
                w = torch.exp(z - torch.where(l == -math.inf, torch.zeros_like(l), l)[..., None])[..., :L]
                out[cu[b] + i0:cu[b] + i1, g * G:(g + 1) * G] = torch.einsum("qhn,nd->qhd", w, v)
                lse[cu[b] + i0:cu[b] + i1, g * G:(g + 1) * G] = l
    return {"out": out, "lse": lse}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(3)]:
        print(case, work(case))
