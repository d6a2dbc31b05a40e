"""The layers over paged 8-bit caches, the merge of their parts, and the page plan's sizes."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged import PlanState, assert_attn, check_attn, held_rows, i32, make_cache, status

pytestmark = pytest.mark.gpu

DEV = "cuda"


# ------------------------------------------------------------------------------------ plan


@pytest.mark.parametrize("B", [3040, 3046, 3047, 3060, 3071, 3080, 8192])
def test_plan_many_requests(hcl, B):
    """Numbers of requests around the shared memory that a launch has without asking, and the most."""
    rng = np.random.default_rng(B)
    S = PlanState(B, 3, 2 * B, 16, 3 * B, rng)
    S.step(hcl, [0] * B, rng.integers(0, 4, B).tolist())
    S.step(hcl, [max(0, n - 1) for n in S.seq], rng.integers(0, 3, B).tolist())


def test_plan_many_requests_first_in_a_process(hcl):
    """The same where no larger call has gone before it in the process."""
    code = ("import numpy as np; from heavily_compressed_long_b200 import api; "
            "from tests.test_gpu_paged import PlanState; rng = np.random.default_rng(0); "
            "PlanState(3060, 2, 4000, 16, 9000, rng).step(api, [0] * 3060, rng.integers(0, 3, 3060).tolist())")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_plan_gives_back_two_to_the_31_entries(hcl):
    """The largest table, all of it given back though the cache has four pages: what does not fit
    the free list is refused, the table is cleared to its end."""
    B, width = 16, (1 << 27) - 1
    table = torch.full((B, width), 3, dtype=torch.int32, device=DEV)
    seq, free, n = i32([width * 16] * B), i32([0, 1, 2, 3]), i32([0])
    cu, pos, slot, st = i32([0] * (B + 1)), i32([0]), i32([0]), status()
    hcl.hcl_page_plan(i32([0] * B), i32([0] * B), seq, table, free, n, 16, cu, pos, slot, status=st)
    assert st.item() == 16 and n.item() == 4 and seq.tolist() == [0] * B and free.tolist() == [3] * 4
    assert bool((table.view(-1)[:1 << 30] == -1).all()) and bool((table.view(-1)[1 << 30:] == -1).all())


def test_batch_start_is_the_first_new_row(hcl):
    """Also where keep is out of range: the positions that the plan gives, and the start that the
    attention uses, are the same."""
    from heavily_compressed_long_b200.pipeline import PagedBatch
    b = PagedBatch(3, 16, 4, 12, 40)
    b.plan(i32([20, 5, 9]))
    b.plan(i32([1, 2, 3]), keep=i32([25, -4, 9]))
    assert b.status.item() == 16
    assert b.start.tolist() == [20, 0, 9] and b.seq_len.tolist() == [21, 2, 12]
    assert b.pos[:6].tolist() == [20, 0, 1, 9, 10, 11]
    b.status.zero_()
    b.plan(i32([1, 1, 1]), keep=torch.tensor([21, 1, 0], device=DEV))  # (any integer type)
    assert b.status.item() == 0 and b.start.tolist() == [21, 1, 0] and b.seq_len.tolist() == [22, 2, 1]


# ------------------------------------------------------------------------------------ write


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("order,written", [((3, 5, 6), 1), ((5, 3), 1), ((4, 4), 1), ((0, 0), 1), ((7, 8, 0, 1), 2),
                                           ((2, 3, 4, 6, 7), 3)])
@pytest.mark.parametrize("pad", [0, 200])
def test_write_rows_of_a_page_not_in_order(hcl, page, order, written, pad):
    """Rows of one page that are not one run of slots: the first run is written, the others are left
    out and the status says so; the pages around it are as without them."""
    gen = torch.Generator().manual_seed(page)
    n_pages, Hkv, d = 20, 3, 64
    slot = list(range(5 * page, 5 * page + min(pad, 9 * page)))
    first = len(slot)
    slot += [2 * page + o for o in order] + [3 * page, 3 * page + 1]
    x = (torch.randn(len(slot), Hkv, d, generator=gen) * torch.exp2(torch.randn(len(slot), 1, 1, generator=gen) * 4))
    x = x.to(torch.bfloat16)
    codes = (torch.randn(n_pages, Hkv, page, d, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.exp2(torch.randint(-9, 0, (n_pages, Hkv), generator=gen).float())
    c, s, st = codes.cuda(), scale.cuda(), status()
    hcl.hcl_paged_write(x.cuda(), None, i32(slot), hcl.PagedKV(c, s), status=st)
    assert st.item() == 16
    kept = np.asarray(slot)
    kept[first + written:first + len(order)] = -1
    val, want = ref.write(ref.f64(x), kept, codes.numpy(), scale.numpy())
    np.testing.assert_array_equal(ref.f64(s), want)
    np.testing.assert_array_equal(ref.decode_e4m3(c.cpu().numpy()), val)


# ------------------------------------------------------------------------------------ merge


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("G,part", [(1, 0), (2, 0), (2, 1), (3, 1)])
def test_merge_keeps_nan(hcl, G, part, sink):
    """A part whose log-sum-exp is NaN makes its row NaN, and no other row; a part that weighs
    nothing may hold anything."""
    gen = torch.Generator().manual_seed(G + part)
    rows, H, d = 8, 4, 64
    o = torch.randn(G, rows, d, generator=gen).to(torch.bfloat16)
    lse = torch.randn(G, rows, generator=gen)
    lse[part, 2] = math.nan
    lse[part, 5] = -math.inf
    o[part, 5] = math.nan
    s = torch.randn(H, generator=gen) if sink else None
    out = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
    got_l = torch.zeros(rows, device=DEV)
    hcl.hcl_lse_merge(o.view(G, 2, H, d).cuda(), lse.view(G, 2, H).cuda(), out.view(2, H, d),
                      lse_out=got_l.view(2, H), sink=None if s is None else s.cuda())
    z = lse.double()
    if sink:
        z = torch.cat([z, s.double().repeat(rows // H)[None]])
    want_l = torch.logsumexp(z, 0)
    w = torch.exp(lse.double() - torch.where(torch.isneginf(want_l), 0.0, want_l))
    want = (torch.where(w[..., None] == 0, 0.0, o.double()) * w[..., None]).sum(0)
    nan = torch.arange(rows) == 2
    assert torch.isnan(out.cpu()[nan]).all() and torch.isnan(got_l.cpu()[nan]).all()
    assert not torch.isnan(out.cpu()[~nan]).any()
    # bf16: half a step; weights by exponentials of differences below 8, a few steps of 2^-24 each
    err = (out.cpu().double() - want).abs()[~nan]
    assert bool((err <= 2.0 ** -8 * want.abs()[~nan] + 2.0 ** -18 * (w[..., None] * o.double().abs().nan_to_num()).sum(0)[~nan]).all())
    fin = ~nan & torch.isfinite(want_l)
    assert torch.equal(torch.isneginf(got_l.cpu()[~nan]), torch.isneginf(want_l[~nan]))
    assert bool(((got_l.cpu().double() - want_l).abs()[fin] <= 2.0 ** -20 * (1 + want_l.abs()[fin])).all())


def hca_layer(H, T, entries_T, n_entries, gen, sink=None, raw_rows=200):
    """A PagedHcaLayer of one request with raw rows and entries in its caches; the plan of the step
    covers the last T rows."""
    from heavily_compressed_long_b200.pipeline import PagedBatch, PagedHcaLayer
    d, mh = 128, 16
    raw, ent = PagedBatch(1, 16, 20, 24, T), PagedBatch(1, 16, 2, 4, entries_T)
    layer = PagedHcaLayer(raw, ent, 24, 4, H, d, mh=mh, W=64, sink=sink)
    at = 0
    while at < raw_rows:
        n = min(T, raw_rows - at)
        raw.plan(i32([n]))
        layer.raw_layer.write(torch.randn(T, 1, d, generator=gen).to(torch.bfloat16).cuda())
        at += n
    for _ in range(n_entries // entries_T):
        ent.plan(i32([entries_T]))
        layer.entry_layer.write(torch.randn(entries_T, 1, d, generator=gen).to(torch.bfloat16).cuda())
    return layer, raw, ent


@pytest.mark.parametrize("with_sink", [False, True])
@pytest.mark.parametrize("where", ["query", "entry", "raw"])
def test_hca_layer_keeps_nan(hcl, where, with_sink):
    """A NaN in a query, or in an entry or a raw row that the queries see, comes out as NaN."""
    gen = torch.Generator().manual_seed(3)
    H, T = 16, 4
    sink = torch.randn(H, generator=gen).cuda() if with_sink else None
    layer, raw, ent = hca_layer(H, T, 4, 8, gen, sink=sink)
    q = torch.randn(T, H, 128, generator=gen).to(torch.bfloat16)
    rows, heads = slice(None), slice(None)
    if where == "query":
        q[1, 3, 7] = math.nan
        rows, heads = slice(1, 2), slice(3, 4)
    elif where == "entry":
        layer.entry_layer.store.k[ent.table[0, 0].item(), 0, 5, 11] = 0x7F
    else:
        layer.raw_layer.store.k[raw.table[0, 190 // 16].item(), 0, 190 % 16, 11] = 0x7F
    out = torch.zeros(T, H, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(T, H, device=DEV)
    layer.attend(q.cuda(), out, lse=lse, max_q=T)
    assert raw.status.item() == 0 and ent.status.item() == 0
    want = torch.zeros(T, H, dtype=torch.bool)
    want[rows, heads] = True
    assert torch.equal(torch.isnan(lse).cpu(), want)
    assert torch.equal(torch.isnan(out).all(-1).cpu(), want) and torch.equal(torch.isnan(out).any(-1).cpu(), want)


@pytest.mark.parametrize("H,T,entries_T", [(16, 4, 1), (8, 8, 2), (64, 3, 1)])
def test_hca_layer_with_more_queries_than_new_entries(hcl, H, T, entries_T):
    """The entry batch plans fewer rows a step than the raw batch has queries: the result is that of
    a layer whose entry batch is as large."""
    got = []
    for n in (entries_T, T):
        gen = torch.Generator().manual_seed(8)
        layer, raw, ent = hca_layer(H, T, entries_T, 6, gen)
        if n != entries_T:
            from heavily_compressed_long_b200.pipeline import PagedBatch, PagedHcaLayer
            big = PagedBatch(1, 16, 2, 4, T)
            big.seq_len, big.table = ent.seq_len, ent.table
            other = PagedHcaLayer(raw, big, 24, 4, H, 128, mh=16, W=64)
            other.raw_layer.store, other.entry_layer.store = layer.raw_layer.store, layer.entry_layer.store
            layer = other
        q = torch.randn(T, H, 128, generator=gen).to(torch.bfloat16).cuda()
        got.append(layer.attend(q, torch.zeros(T, H, 128, dtype=torch.bfloat16, device=DEV), max_q=T))
        assert raw.status.item() == 0 and ent.status.item() == 0
    assert torch.isfinite(got[0]).all() and (got[0] != 0).any() and torch.equal(*got)


@pytest.mark.parametrize("H,T,n_entries,raw_rows", [(16, 4, 8, 200), (64, 40, 0, 200), (16, 40, 8, 203), (4, 1, 24, 70)])
@pytest.mark.parametrize("with_sink", [False, True])
def test_hca_layer_rounds_once(hcl, H, T, n_entries, raw_rows, with_sink):
    """The layer against one softmax over entries, window and sink in 64 bits, at the bound of the
    attention itself: the parts are not rounded before they are merged."""
    gen = torch.Generator().manual_seed(H + T)
    sink = torch.randn(H, generator=gen) if with_sink else None
    layer, raw, ent = hca_layer(H, T, 8, n_entries, gen, sink=None if sink is None else sink.cuda(), raw_rows=raw_rows)
    for _ in range(12):
        q = (torch.randn(T, H, 128, generator=gen) * 0.3).to(torch.bfloat16)
        out = torch.zeros(T, H, 128, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros(T, H, device=DEV)
        layer.attend(q.cuda(), out, lse=lse, max_q=T)
        new, start = int(raw.cu_new[1]), int(raw.start[0])
        rows = [held_rows(b, x, 0)[0][:, 0] for b, x in ((ent, layer.entry_layer), (raw, layer.raw_layer))]
        want, mass = np.zeros((new, H, 128)), np.zeros((new, H, 128))
        wl, zabs = np.zeros((new, H)), np.zeros((new, H))
        for i in range(new):
            p = start + i
            x = np.concatenate([rows[0][:(p + 1) // 16], rows[1][max(0, p - 63):p + 1]])
            z = ref.f64(q[i]) @ x.T / math.sqrt(128)
            zz = z if sink is None else np.concatenate([z, ref.f64(sink)[:, None]], 1)
            wl[i] = np.log(np.exp(zz - zz.max(1, keepdims=True)).sum(1)) + zz.max(1)
            w = np.exp(z - wl[i][:, None])
            want[i], mass[i] = w @ x, w @ np.abs(x)
            zabs[i] = (np.abs(ref.f64(q[i])) @ np.abs(x).T).max(1) / math.sqrt(128)
        assert_attn(ref.f64(out)[:new], ref.f64(lse)[:new], want, wl, mass, zabs)


# ------------------------------------------------------------------------------------ parts in fp32


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,lens,news", [(8, [1, 65, 300], [1, 1, 1]), (16, [40, 9], [1, 0]), (8, [30000], [1]),
                                         (8, [3000] * 40, [1] * 40), (128, [100, 5], [1, 1]), (64, [30000, 70], [1, 2]),
                                         (8, [200, 90], [200, 33]), (16, [9000], [300])])
def test_attn_fp32_out(hcl, d, G, lens, news):
    """The fp32 output rounds to the bf16 one, whichever kernel and merge writes it; rows behind the
    last request stay."""
    gen = torch.Generator().manual_seed(G)
    table, k, ks, v, vs = make_cache(lens, 32, 2, d, False, gen)
    T, H = sum(news) + 2, 2 * G
    q = torch.randn(T, H, d, generator=gen).to(torch.bfloat16).cuda()
    store = hcl.PagedKV(k.cuda(), ks.cuda(), v.cuda(), vs.cuda())
    args = (q, i32(np.concatenate([[0], np.cumsum(news)])), i32([a - b for a, b in zip(lens, news)]), store, i32(table),
            i32(lens))
    res = []
    for call, dtype in ((hcl.hcl_paged_attn, torch.bfloat16), (hcl.hcl_paged_attn_f32, torch.float32)):
        out, lse = torch.full((T, H, d), 7.0, dtype=dtype, device=DEV), torch.full((T, H), 7.0, device=DEV)
        call(*args, out, lse=lse, max_q=max(news))
        res.append((out, lse))
    (a, al), (b, bl) = res
    assert torch.equal(a, b.to(torch.bfloat16)) and torch.equal(al, bl)
    assert bool((b[-2:] == 7.0).all()) and torch.isfinite(b).all()
    assert not torch.equal(b[:-2], a[:-2].float())
    with pytest.raises(ValueError):
        hcl.hcl_paged_attn_f32(*args, torch.empty(T, H, d, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        hcl.hcl_lse_merge(torch.empty(1, 1, T, H, d, dtype=torch.float16, device=DEV), al[None, None], a[None])


# ------------------------------------------------------------------------------------ calls together


@pytest.mark.parametrize("graph", [False, True])
def test_attn_calls_on_streams(hcl, graph):
    """Calls in flight on several streams, each with its own workspace, whose long requests are split
    over blocks: finite, the bits of a call alone, and sampled rows against 64 bits; also captured,
    the graphs replayed side by side."""
    gen = torch.Generator().manual_seed(12)
    calls = []
    for lens, news, G, d in (([4000, 70, 900], [300, 1, 64], 8, 128), ([3000, 2500, 10], [1, 1, 1], 64, 64),
                             ([9000, 30, 700], [1, 1, 1], 8, 128), ([6000, 500], [40, 300], 16, 64)):
        table, k, ks, v, vs = make_cache(lens, 32, 2, d, False, gen)
        T = sum(news)
        q = torch.randn(T, 2 * G, d, generator=gen).to(torch.bfloat16)
        cu, start = np.concatenate([[0], np.cumsum(news)]), [a - b for a, b in zip(lens, news)]
        args = (q.cuda(), i32(cu), i32(start), hcl.PagedKV(k.cuda(), ks.cuda(), v.cuda(), vs.cuda()), i32(table), i32(lens))
        ws = torch.empty(hcl.paged_attn_workspace_bytes(T, 2 * G, 2, d), dtype=torch.uint8, device=DEV)
        out, lse = torch.empty(T, 2 * G, d, dtype=torch.bfloat16, device=DEV), torch.empty(T, 2 * G, device=DEV)
        alone = hcl.hcl_paged_attn(*args, torch.empty_like(out), max_q=max(news), ws=ws)
        torch.cuda.synchronize()
        calls.append((args, ws, max(news), out, lse, torch.cuda.Stream(), alone, (lens, news, start, cu, table, k, ks, v, vs, q)))
    graphs = []
    for args, ws, mq, out, lse, stream, _, _ in calls:
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                hcl.hcl_paged_attn(*args, out, lse=lse, max_q=mq, ws=ws, stream=stream)
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (args, ws, mq, out, lse, stream, _, _) in enumerate(calls):
            if graph:
                with torch.cuda.stream(stream):
                    graphs[i].replay()
            else:
                hcl.hcl_paged_attn(*args, out, lse=lse, max_q=mq, ws=ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, _, out, lse, _, alone, (lens, news, start, cu, table, k, ks, v, vs, q) in calls:
        assert torch.isfinite(out).all() and torch.isfinite(lse).all() and torch.equal(out, alone)
        H, d = q.shape[1], q.shape[2]
        for b in range(len(lens)):
            for i in {0, news[b] // 2, news[b] - 1}:
                for h in (0, H // 2 - 1, H - 1):
                    g, t = h // (H // 2), int(cu[b]) + i
                    w = ref.attn(ref.f64(q[t:t + 1, h:h + 1]), [0, 1], [start[b] + i], lens[b:b + 1], table[b:b + 1],
                                 k[:, g:g + 1].numpy(), ks[:, g:g + 1].numpy(), v[:, g:g + 1].numpy(),
                                 vs[:, g:g + 1].numpy(), 32, 1, 0, 1 / math.sqrt(d))
                    assert_attn(ref.f64(out[t:t + 1, h:h + 1]), ref.f64(lse[t:t + 1, h:h + 1]), *w)


@pytest.mark.parametrize("d,W,m", [(64, 0, 1), (128, 20, 1), (64, 0, 4), (64, 0, 2 ** 31 - 1)])
def test_attn_most_requests(hcl, d, W, m):
    """8192 requests in one call, decode among short chunks, some without queries or rows."""
    gen = torch.Generator().manual_seed(2)
    rng = np.random.default_rng(2)
    B = 8192
    lens = rng.integers(0, 40, B).tolist()
    news = [min(int(n), 1 + l) for n, l in zip(rng.choice([0, 1, 1, 1, 1, 1, 2, 9], B), lens)]
    case = dict(lens=lens, news=news, Hkv=1, G=4, d=d, page=16, shared=True, W=W, m=m, sink=W == 0,
                start=[min(2 ** 31 - 20, max(0, l * m - n)) for l, n in zip(lens, news)])
    assert_attn(*check_attn(hcl, case))
