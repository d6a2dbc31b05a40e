"""The paged 8-bit cache on the GPU against plain references in 64 bits: page plan, write,
attention, refusals of the binding, and a run of them together."""
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------ plan


class PlanState:
    def __init__(self, B, width, n_pages, page, T, rng):
        self.page, self.T, self.n_pages = page, T, n_pages
        self.seq = [0] * B
        self.table = np.full((B, width), -1, np.int32)
        self.stack = rng.permutation(n_pages).tolist()
        self.d_seq, self.d_table = i32(self.seq), i32(self.table)
        self.d_free, self.d_n = i32(self.stack), i32([n_pages])
        self.d_cu = i32(np.zeros(B + 1))
        self.d_pos, self.d_slot = i32(np.zeros(T)), i32(np.zeros(T))

    def step(self, hcl, keep, new, alias=False):
        want = ref.plan(keep, new, self.seq, self.table, self.stack + [-1] * (self.n_pages - len(self.stack)),
                        len(self.stack), self.page, self.T)
        st = status()
        hcl.hcl_page_plan(self.d_seq if alias else i32(keep), i32(new), self.d_seq, self.d_table, self.d_free,
                          self.d_n, self.page, self.d_cu, self.d_pos, self.d_slot, status=st)
        self.seq, self.table, self.stack = want["seq"], want["table"], want["stack"]
        assert self.d_seq.tolist() == want["seq"]
        assert np.array_equal(self.d_table.cpu().numpy(), want["table"])
        assert self.d_n.item() == len(want["stack"])
        assert self.d_free[:len(want["stack"])].tolist() == want["stack"]
        assert self.d_cu.tolist() == want["cu"]
        assert self.d_pos.tolist() == want["pos"]
        assert self.d_slot.tolist() == want["slot"]
        assert st.item() == want["status"]
        return want


@pytest.mark.parametrize("B,page,width,T", [(1, 16, 8, 40), (3, 64, 5, 130), (33, 16, 40, 6000), (300, 32, 20, 20000),
                                            (1500, 128, 3, 9000)])
def test_plan_steps(hcl, B, page, width, T):
    """Growth, rollback, replaced requests, idle requests; pages come back and go out again."""
    rng = np.random.default_rng(B)
    S = PlanState(B, width, B * width + 3, page, T, rng)
    most = min(width * page, T // B)
    S.step(hcl, [0] * B, rng.integers(0, most + 1, B).tolist())
    for _ in range(6):
        keep = [int(rng.choice([s, s, max(0, s - 2), 0, rng.integers(0, s + 1)])) for s in S.seq]
        room = [min(width * page - k, T // B) for k in keep]
        new = [int(rng.choice([0, min(1, r), rng.integers(0, r + 1)])) for r in room]
        S.step(hcl, keep, new)
        held = [p for b, s in enumerate(S.seq) for p in S.table[b, :-(-s // page)].tolist()]
        assert sorted(held + S.stack) == list(range(S.n_pages))  # every page has one owner
    S.step(hcl, S.seq, [0] * B, alias=True)
    if most > 1:
        S.step(hcl, [min(s, width * page - 1) for s in S.seq], [1] * B)


def test_plan_same_step_again(hcl):
    rng = np.random.default_rng(3)
    S = PlanState(20, 10, 150, 16, 900, rng)
    S.step(hcl, [0] * 20, rng.integers(0, 45, 20).tolist())
    keep, new = [s // 2 for s in S.seq], rng.integers(0, 40, 20).tolist()
    a = S.step(hcl, keep, new)
    b = S.step(hcl, keep, new)
    assert np.array_equal(a["table"], b["table"]) and a["stack"] == b["stack"]


def test_plan_short_of_pages(hcl):
    rng = np.random.default_rng(4)
    S = PlanState(6, 8, 10, 16, 200, rng)
    w = S.step(hcl, [0] * 6, [16, 48, 17, 64, 10, 0])      # 1 + 3 + 2 fit in 10; 4 fit; 1 does not
    assert w["status"] == 32 and w["seq"] == [16, 48, 17, 64, 0, 0]
    w = S.step(hcl, S.seq, [0, 0, 1, 0, 5, 3])             # growth inside a page needs none
    assert w["seq"][2] == 18 and w["seq"][4] == 0 and w["status"] == 32
    w = S.step(hcl, [0, 48, 18, 64, 0, 0], [0, 0, 0, 0, 5, 0])  # a released page serves another request
    assert w["seq"][4] == 5 and w["status"] == 0


def test_plan_beyond_capacity_and_width(hcl):
    rng = np.random.default_rng(5)
    S = PlanState(4, 2, 20, 16, 50, rng)
    w = S.step(hcl, [0] * 4, [20, 33, 20, 1])   # request 1 is longer than its table row; 2 and 3 end beyond T
    assert w["status"] == 32 and w["seq"] == [20, 0, 0, 0] and S.d_cu.tolist() == [0, 20, 50, 50, 50]
    w = S.step(hcl, [25, -1, 0, 0], [-3, 4, 2, 2])
    assert w["status"] == 16 and w["seq"] == [20, 4, 2, 2]


def test_plan_row_sums_beyond_every_capacity(hcl):
    """New rows that sum far past T (and past 32 bits): the requests that end there get nothing, also
    one whose own few rows would fit; no page is taken for it from an empty stack."""
    rng = np.random.default_rng(8)
    S = PlanState(5, 3, 2, 16, 40, rng)
    big = 2 ** 31 - 1
    w = S.step(hcl, [0] * 5, [10, big, 10, big, 1])
    assert w["status"] == 32 and w["seq"] == [10, 0, 0, 0, 0] and S.d_n.item() == 1
    w = S.step(hcl, S.seq, [0, 20, 2 ** 30, 20, 5])
    assert w["status"] == 32 and w["seq"] == [10, 0, 0, 0, 0]
    w = S.step(hcl, S.seq, [big, big, 0, 0, 0])
    assert w["status"] == 32 and w["seq"] == [10, 0, 0, 0, 0]


def test_plan_no_requests_no_rows(hcl):
    empty = torch.zeros(0, dtype=torch.int32, device=DEV)
    cu, pos, slot = i32([7]), i32([5, 5]), i32([5, 5])
    hcl.hcl_page_plan(empty, empty, empty, torch.zeros(0, 3, dtype=torch.int32, device=DEV), i32([1, 2]), i32([2]),
                      16, cu, pos, slot)
    assert cu.tolist() == [0] and pos.tolist() == [-1, -1] and slot.tolist() == [-1, -1]


def test_plan_captured_steps(hcl):
    """One captured decode step, replayed: the state moves on in place."""
    rng = np.random.default_rng(6)
    S = PlanState(5, 6, 40, 16, 5, rng)
    new = i32([1] * 5)

    def call():
        hcl.hcl_page_plan(S.d_seq, new, S.d_seq, S.d_table, S.d_free, S.d_n, 16, S.d_cu, S.d_pos, S.d_slot)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for n in range(35):
        g.replay()
    assert S.d_seq.tolist() == [35] * 5 and S.d_pos.tolist() == [34] * 5
    held = S.d_table[:, :3].flatten().tolist() + S.d_free[:S.d_n.item()].tolist()
    assert sorted(held) == list(range(40))


# ------------------------------------------------------------------------------------ write


def codes_of(n_pages, Hkv, page, d, gen, scale=100.0):
    x = torch.randn(n_pages, Hkv, page, d, generator=gen) * scale
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def check_write(hcl, x, slot, codes, scale, xv=None, cv=None, sv=None):
    """Runs the write on copies and compares codes and scales exactly."""
    c, s = codes.cuda(), scale.cuda()
    c2, s2 = (None, None) if cv is None else (cv.cuda(), sv.cuda())
    st = status()
    store = hcl.PagedKV(c, s, c2, s2)
    hcl.hcl_paged_write(x, xv, i32(slot), store, status=st)
    assert st.item() == 0
    for xx, c0, s0, c1, s1 in ((x, codes, scale, c, s), (xv, cv, sv, c2, s2)):
        if xx is None:
            continue
        val, want = ref.write(ref.f64(xx), slot, c0.numpy(), s0.numpy())
        np.testing.assert_array_equal(ref.f64(s1), want)
        np.testing.assert_array_equal(ref.decode_e4m3(c1.cpu().numpy()), val)
    return store


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,both", [(1, False), (2, True), (5, True)])
def test_write(hcl, d, page, Hkv, both):
    """Prompts from a page's middle and start, single rows, padding; scales that grow and do not."""
    gen = torch.Generator().manual_seed(page + d)
    n_pages = 14
    perm = torch.randperm(n_pages, generator=gen).tolist()
    slot = []
    for first, n in ((page // 2 + 1, 2 * page + 3), (0, page), (page - 1, 1), (3, 2), (0, 1)):
        own = [perm.pop() for _ in range(-(-(first + n) // page))]
        slot += [own[p // page] * page + p % page for p in range(first, first + n)]
        slot += [-1]
    T = len(slot)

    def rows():
        big = torch.exp2(torch.randn(T, Hkv, 1, generator=gen) * 3)
        return (torch.randn(T, Hkv, d, generator=gen) * big).to(torch.bfloat16).cuda()

    def scales():
        return torch.exp2(torch.randint(-9, 0, (n_pages, Hkv), generator=gen).float())

    args = (codes_of(n_pages, Hkv, page, d, gen), scales())
    more = (rows(), codes_of(n_pages, Hkv, page, d, gen), scales()) if both else ()
    check_write(hcl, rows(), slot, *args, *more)


def test_write_special_values(hcl):
    """Infinities saturate and do not set the scale, NaN stays NaN, zeros and subnormals; a scale
    that is no power of two is kept until it grows."""
    page, d = 16, 64
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(8, 1, d, generator=gen)
    x[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 448.0])
    x[1] = 0.0
    x[2] = 1e-40                  # bf16 subnormals
    x[3, 0, 0] = 3.3e38           # near the largest bf16
    x[4, 0, 0] = 1.75             # 448 * 2^-8 exactly
    x[5, 0, 0] = 1.7578125        # the next bf16 above
    x[4, 0, 1:] *= 0.01
    x[5, 0, 1:] *= 0.01
    x = x.to(torch.bfloat16).cuda()
    codes = codes_of(10, 1, page, d, gen)
    scale = torch.full((10, 1), 0.3)
    slot = [0, 16, 32, 48, 64, 80, 96 + 5, 112 + 15]
    store = check_write(hcl, x, slot, codes, scale)
    got = store.k_scale.flatten().tolist()
    assert got[1] == 2.0 ** -126 and got[4] == 2.0 ** -8 and got[5] == 2.0 ** -7
    assert got[6] == torch.tensor(0.3).item()


def test_write_rows_behind_stay(hcl):
    gen = torch.Generator().manual_seed(2)
    codes = codes_of(2, 2, 32, 128, gen)
    codes[:, :, 20:] = 0x7F
    x = (torch.randn(3, 2, 128, generator=gen) * 1000).to(torch.bfloat16).cuda()
    store = check_write(hcl, x, [32 + 17, 32 + 18, 32 + 19], codes, torch.ones(2, 2))
    assert bool((store.k[:, :, 20:] == 0x7F).all()) and torch.equal(store.k[0].cpu(), codes[0])


def test_write_slice_of_wider_rows_and_stream(hcl):
    gen = torch.Generator().manual_seed(7)
    wide = torch.randn(40, 6 * 64, generator=gen).to(torch.bfloat16).cuda()
    k, v = wide[:, 128:256].view(40, 2, 64), wide[:, 256:].view(40, 2, 64)
    codes, scale = codes_of(4, 2, 16, 64, gen), torch.ones(4, 2)
    slot = list(range(5, 45))
    side = torch.cuda.Stream()
    c, c2 = codes.cuda(), codes.cuda()
    s, s2 = scale.cuda(), scale.cuda()
    store = hcl.PagedKV(c, s, c2, s2)
    sl = i32(slot)
    side.wait_stream(torch.cuda.current_stream())
    hcl.hcl_paged_write(k, v, sl, store, stream=side)
    side.synchronize()
    for xx, c1, s1 in ((k, c, s), (v, c2, s2)):
        val, want = ref.write(ref.f64(xx), slot, codes.numpy(), scale.numpy())
        np.testing.assert_array_equal(ref.decode_e4m3(c1.cpu().numpy()), val)
        np.testing.assert_array_equal(ref.f64(s1), want)


def test_write_slot_beyond_cache(hcl):
    gen = torch.Generator().manual_seed(8)
    codes = codes_of(2, 1, 16, 64, gen)
    c, s, st = codes.cuda(), torch.ones(2, 1, device=DEV), status()
    x = torch.randn(3, 1, 64, generator=gen).to(torch.bfloat16).cuda()
    hcl.hcl_paged_write(x, None, i32([32, 2 ** 31 - 1, 16]), hcl.PagedKV(c, s), status=st)
    assert st.item() == 16
    assert torch.equal(c[0].cpu(), codes[0]) and not torch.equal(c[1, :, :1].cpu(), codes[1, :, :1])


def test_write_far_into_a_large_cache(hcl):
    """Code offsets beyond 32 bits."""
    n_pages = (1 << 32) // (128 * 128) + 8
    c = torch.zeros(n_pages, 1, 128, 128, dtype=torch.uint8, device=DEV)
    s = torch.ones(n_pages, 1, device=DEV)
    x = torch.randn(130, 1, 128, device=DEV).to(torch.bfloat16)
    last = n_pages - 2
    slot = [last * 128 + 127] + [(last + 1) * 128 + i for i in range(128)] + [0]
    hcl.hcl_paged_write(x, None, i32(slot), hcl.PagedKV(c, s))
    for row, sl in ((0, slot[0]), (64, slot[64]), (129, 0)):
        val = ref.decode_e4m3(c[sl // 128, 0, sl % 128].cpu().numpy()) * s[sl // 128, 0].item()
        np.testing.assert_allclose(val, ref.f64(x[row, 0]), rtol=2.0 ** -4, atol=s[sl // 128, 0].item() * 2.0 ** -10)
    assert int((c[1:last] != 0).sum()) == 0


# ------------------------------------------------------------------------------------ attention


def make_cache(lens, page, Hkv, d, shared, gen, spare=3, nan_tail=True):
    per = [max(0, -(-n // page)) for n in lens]
    n_pages = sum(per) + spare
    order = torch.randperm(n_pages, generator=gen).tolist()
    table = np.full((len(lens), max(per + [1]) + 1), -1, np.int32)
    for b, n in enumerate(per):
        table[b, :n] = [order.pop() for _ in range(n)]

    def plane():
        return (codes_of(n_pages, Hkv, page, d, gen),
                torch.exp2(torch.randint(-9, -4, (n_pages, Hkv), generator=gen).float()))

    k, ks = plane()
    v, vs = (None, None) if shared else plane()
    if nan_tail:  # rows behind a request's last, and pages of no request, hold NaN codes
        for b, n in enumerate(lens):
            if n % page:
                for c in (k, v):
                    if c is not None:
                        c[table[b, n // page], :, n % page:] = 0x7F
        for pg in order:
            for c in (k, v):
                if c is not None:
                    c[pg] = 0xFF
    return table, k, ks, v, vs


def tolerance(want, mass, zabs):
    """bf16 output: half a step, 2^-8 |out|.  Probabilities in 11 bits: 2^-11 of each term, so
    2^-11 mass, twice that for the smallest; scores: products of codes and bf16 are exact, their
    fp32 sum over d <= 128 terms is off by at most 128 * 2^-24 of zabs, as is the exponent's
    argument, and moves each probability by twice that."""
    return 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -15 * zabs[..., None]) * mass + 1e-30


def check_attn(hcl, case, seed=0, poison=None, **kw):
    """case: lens, news, start (None: the last queries), Hkv, G, d, page, shared, m, W, sink."""
    gen = torch.Generator().manual_seed(seed)
    lens, news, Hkv, G, d, page = (case[k] for k in ("lens", "news", "Hkv", "G", "d", "page"))
    m, W = case.get("m", 1), case.get("W", 0)
    start = case.get("start") or [l * m - n for l, n in zip(lens, news)]
    H = Hkv * G
    cu = np.concatenate([[0], np.cumsum(news)]).astype(int)
    T = int(cu[-1]) + case.get("pad", 0)
    table, k, ks, v, vs = make_cache(lens, page, Hkv, d, case.get("shared", False), gen)
    q = (torch.randn(T, H, d, generator=gen) * case.get("qs", 1.5)).to(torch.bfloat16)
    sink = torch.randn(H, generator=gen) if case.get("sink") else None
    if poison:
        poison(table, k, ks, v, vs, q)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    store = hcl.PagedKV(dev(k), dev(ks), dev(v), dev(vs))
    out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), 7.0, device=DEV)
    st = status()
    scale = case.get("scale", 1 / math.sqrt(d))
    args = (i32(cu), i32(start), store, i32(table), i32(lens))
    hcl.hcl_paged_attn(q.cuda(), *args, out, lse=lse, m=m, W=W, scale=scale, sink=dev(sink), status=st,
                       max_q=case.get("max_q", max(news + [0])), **kw)
    torch.cuda.synchronize()
    assert st.item() == case.get("status", 0)
    want, wl, mass, zabs = ref.attn(ref.f64(q), cu, start, lens, np.maximum(table, 0), k.numpy(), ks.numpy(),
                                    None if v is None else v.numpy(), None if vs is None else vs.numpy(), page, m, W,
                                    scale, sink)
    got, gl = ref.f64(out), ref.f64(lse)
    n = int(cu[-1])
    assert np.all(got[n:] == 7.0) and np.all(gl[n:] == 7.0)
    return got[:n], gl[:n], want[:n], wl[:n], mass[:n], zabs[:n]


def assert_attn(got, gl, want, wl, mass, zabs):
    assert np.array_equal(np.isneginf(wl), np.isneginf(gl)) and not np.isnan(gl).any()
    fin = np.isfinite(wl)
    assert np.all(np.abs(gl - wl)[fin] <= (2.0 ** -16 * zabs + 2.0 ** -19 * (1 + np.abs(wl)))[fin])
    assert np.all(got[~fin] == 0.0)
    bad = np.abs(got - want) > tolerance(want, mass, zabs)
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - want).max())


CASES = {
    "one_token": dict(lens=[1], news=[1], Hkv=1, G=1, d=128, page=16),
    "decode_gqa": dict(lens=[1, 63, 64, 65, 127, 200, 500], news=[1] * 7, Hkv=2, G=8, d=128, page=64),
    "decode_g5_d64": dict(lens=[3, 130, 257], news=[1] * 3, Hkv=3, G=5, d=64, page=16),
    "decode_mha": dict(lens=[40, 333], news=[1, 1], Hkv=4, G=1, d=64, page=32),
    "decode_shared16": dict(lens=[100, 513, 1], news=[1] * 3, Hkv=1, G=16, d=128, page=128, shared=True, sink=True),
    "decode_g24": dict(lens=[300, 77], news=[1] * 2, Hkv=2, G=24, d=128, page=64),
    "decode_mqa128": dict(lens=[300, 1, 129], news=[1] * 3, Hkv=1, G=128, d=128, page=64, shared=True, sink=True),
    "decode_mqa64_d64": dict(lens=[700, 15], news=[1] * 2, Hkv=1, G=64, d=64, page=16),
    "draft": dict(lens=[5, 64, 300], news=[4, 3, 4], Hkv=2, G=4, d=64, page=16),
    "draft_mqa": dict(lens=[50, 260], news=[3, 2], Hkv=1, G=64, d=128, page=32, shared=True),
    "empty_requests": dict(lens=[0, 50, 0, 20, 0], news=[1, 0, 0, 2, 1], start=[-1, 50, 0, 18, 0], Hkv=2, G=2, d=128,
                           page=16, pad=3),
    "prompt": dict(lens=[150, 31, 128], news=[150, 31, 128], Hkv=2, G=4, d=128, page=64),
    "prompt_d64": dict(lens=[150, 300], news=[150, 97], Hkv=1, G=7, d=64, page=32, sink=True),
    "chunk_shared": dict(lens=[700], news=[100], Hkv=1, G=16, d=128, page=64, shared=True),
    "mixed": dict(lens=[400, 90, 256, 10], news=[1, 90, 40, 1], Hkv=2, G=8, d=128, page=16, pad=5),
    "mixed_d64": dict(lens=[400, 90, 256, 10], news=[1, 90, 40, 1], Hkv=2, G=4, d=64, page=128, pad=1),
    "window_decode": dict(lens=[300, 5, 128, 129], news=[1] * 4, Hkv=1, G=8, d=128, page=16, W=128),
    "window_one": dict(lens=[40, 100], news=[7, 100], Hkv=1, G=4, d=128, page=16, W=1),
    "window_prompt": dict(lens=[700, 257], news=[300, 257], Hkv=1, G=16, d=128, page=32, W=128, shared=True, sink=True),
    "entries_m128": dict(lens=[5, 40], news=[300, 1], start=[100, 40 * 128 - 1], Hkv=1, G=16, d=128, page=16, m=128,
                         shared=True),
    "entries_m4": dict(lens=[64, 20], news=[70, 81], start=[186, 0], Hkv=2, G=3, d=64, page=16, m=4, sink=True),
    "rows_see_nothing": dict(lens=[30, 30], news=[40, 3], start=[-35, -2], Hkv=1, G=2, d=64, page=16),
    "held_but_ahead": dict(lens=[100, 300], news=[5, 200], start=[20, 10], Hkv=2, G=2, d=128, page=16),
    "behind_the_rows": dict(lens=[20, 200], news=[4, 60], start=[50, 190], Hkv=1, G=8, d=128, page=32, W=64),
    "window_past_all": dict(lens=[20], news=[4], start=[500], Hkv=1, G=8, d=128, page=32, W=64),
    "sharp": dict(lens=[260, 100], news=[1, 100], Hkv=1, G=8, d=128, page=64, qs=20.0),
    "loose_max_q": dict(lens=[260, 100], news=[1, 60], Hkv=1, G=8, d=128, page=64, max_q=1000),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_attn(hcl, name):
    assert_attn(*check_attn(hcl, CASES[name], seed=len(name)))


@pytest.mark.parametrize("G,new", [(8, 1), (128, 1), (8, 60)])
def test_attn_page_scales_far_apart(hcl, G, new):
    """Value scales that span 2^40: each page's weight is kept to its own precision."""
    def poison(table, k, ks, v, vs, q):
        n = vs.shape[0]
        vs[:] = torch.exp2(torch.arange(n).float() * (40.0 / n) - 30)[:, None]
        ks[:] = 0.01
    assert_attn(*check_attn(hcl, dict(lens=[300], news=[new], Hkv=1, G=G, d=128, page=16), poison=poison))


@pytest.mark.parametrize("G,new", [(8, 1), (64, 1), (8, 90)])
def test_attn_query_range(hcl, G, new):
    """Query rows from 2^-60 to 2^60 times the ordinary, with matching scales' effect; a zero row."""
    def poison(table, k, ks, v, vs, q):
        q[:, 0] *= 2.0 ** -60
        q[:, 1] = 0
        q[:, 2] *= 2.0 ** 4
    assert_attn(*check_attn(hcl, dict(lens=[200], news=[new], Hkv=1, G=G, d=128, page=32), poison=poison))
    def tiny(table, k, ks, v, vs, q):
        q *= 2.0 ** 60
        ks *= 2.0 ** -60
    assert_attn(*check_attn(hcl, dict(lens=[200], news=[new], Hkv=1, G=G, d=128, page=32), poison=tiny))


@pytest.mark.parametrize("G,news,shared", [(8, [1, 1], False), (128, [1, 1], True), (16, [60, 80], True),
                                           (8, [100, 30], False), (4, [4, 3], True), (4, [4, 3], False),
                                           (2, [4, 1], True), (1, [7, 4], False)])
def test_attn_nan_row_reaches_only_those_who_see_it(hcl, G, news, shared):
    """A NaN code in a key or value row: the queries that see the row become NaN, no others."""
    lens, page = [120, 100], 16
    at = [lens[0] - max(1, news[0] // 2), None]  # row of request 0
    case = dict(lens=lens, news=news, Hkv=1, G=G, d=128, page=page, shared=shared)

    def poison(table, k, ks, v, vs, q):
        (k if v is None else v)[table[0, at[0] // page], 0, at[0] % page, 5] = 0x7F

    got, gl, want, wl, mass, zabs = check_attn(hcl, case, poison=poison)
    sees = np.zeros(got.shape[0], bool)
    for i in range(news[0]):
        sees[i] = lens[0] - news[0] + i >= at[0]
    assert sees.any()
    assert np.isnan(got[sees][:, :, 5]).all() and not np.isnan(got[~sees]).any()
    ok = ~sees
    assert_attn(got[ok], gl[ok], want[ok], wl[ok], mass[ok], zabs[ok])


@pytest.mark.parametrize("G,new", [(8, 1), (128, 1), (8, 200)])
def test_attn_bad_page_is_left_out(hcl, G, new):
    """A page id outside the cache: its rows do not count, the status says so."""
    gen = torch.Generator().manual_seed(5)
    lens, page, d = [300], 16, 128
    table, k, ks, v, vs = make_cache(lens, page, 1, d, False, gen)
    q = torch.randn(new, G, d, generator=gen).to(torch.bfloat16)
    for bad in (-1, k.shape[0], 2 ** 31 - 1):
        t2 = table.copy()
        t2[0, 3] = bad
        out, lse, st = torch.empty(new, G, d, dtype=torch.bfloat16, device=DEV), torch.empty(new, G, device=DEV), status()
        hcl.hcl_paged_attn(q.cuda(), i32([0, new]), i32([300 - new]),
                           hcl.PagedKV(k.cuda(), ks.cuda(), v.cuda(), vs.cuda()), i32(t2), i32(lens), out, lse=lse,
                           max_q=new, status=st)
        assert st.item() == 16
        # the reference over a cache without that page's rows; queries stand behind or inside all others
        keep = [j for j in range(19) if j != 3]
        t3 = table[:, keep]
        w, wl, mass, zabs = ref.attn(ref.f64(q)[-1:], [0, 1], [300 - 16 - 1], [300 - 16], t3, k.numpy(), ks.numpy(),
                                     v.numpy(), vs.numpy(), page, 1, 0, 1 / math.sqrt(d))
        assert_attn(ref.f64(out)[-1:], ref.f64(lse)[-1:], w, wl, mass, zabs)


def test_attn_length_beyond_table(hcl):
    """kv_len beyond the table's row: the rows there are, and the status."""
    case = dict(lens=[100], news=[1], Hkv=1, G=8, d=64, page=16)
    gen = torch.Generator().manual_seed(5)
    table, k, ks, v, vs = make_cache([112], 16, 1, 64, True, gen, nan_tail=False)
    q = torch.randn(1, 8, 64, generator=gen).to(torch.bfloat16)
    out, st = torch.empty(1, 8, 64, dtype=torch.bfloat16, device=DEV), status()
    hcl.hcl_paged_attn(q.cuda(), i32([0, 1]), i32([10 ** 6]), hcl.PagedKV(k.cuda(), ks.cuda()), i32(table[:, :7]),
                       i32([10 ** 9]), out, max_q=1, status=st)
    assert st.item() == 16
    w, wl, mass, zabs = ref.attn(ref.f64(q), [0, 1], [10 ** 6], [112], table, k.numpy(), ks.numpy(), None, None, 16, 1,
                                 0, 1 / 8.0)
    assert np.all(np.abs(ref.f64(out) - w) <= tolerance(w, mass, zabs))
    del case


def test_attn_more_queries_than_max_q(hcl):
    gen = torch.Generator().manual_seed(6)
    table, k, ks, v, vs = make_cache([64, 64], 16, 1, 64, True, gen)
    q = torch.randn(6, 8, 64, generator=gen).to(torch.bfloat16).cuda()
    out, st = torch.full((6, 8, 64), 3.0, dtype=torch.bfloat16, device=DEV), status()
    hcl.hcl_paged_attn(q, i32([0, 5, 6]), i32([59, 63]), hcl.PagedKV(k.cuda(), ks.cuda()), i32(table), i32([64, 64]),
                       out, max_q=4, status=st)
    assert st.item() == 16 and bool((out[:5] == 3.0).all()) and not bool((out[5] == 3.0).all())


@pytest.mark.parametrize("G,news", [(8, [1, 1, 1]), (8, [40, 1, 60]), (32, [1, 2, 1])])
def test_attn_requests_share_pages(hcl, G, news):
    """A prefix that three requests have in common stands once, and a page may stand twice in a row."""
    def poison(table, k, ks, v, vs, q):
        table[1:, :5] = table[0, :5]
        table[2, 6] = table[2, 5]

    got = check_attn(hcl, dict(lens=[200, 150, 130], news=news, Hkv=2, G=G, d=64, page=16), poison=poison)
    assert_attn(*got)


@pytest.mark.parametrize("H", [8, 64])
def test_attn_sixteen_million_rows(hcl, H):
    """One page that stands 2^18 times in a request's table: out as over the page alone, the
    log-sum-exp larger by log 2^18.  Beside the usual tolerance, the sums over many rounds: a block has
    at most 2^18 / 148 rounds on 148 SMs, in two streams of four (row kernel: fewer) additions each,
    and an addition that truncates loses less than 2^-23 of the sum."""
    gen = torch.Generator().manual_seed(9)
    page, d, n = 64, 128, 1 << 18
    codes = torch.randn(1, 1, page, d, generator=gen).mul(100).to(torch.float8_e4m3fn).view(torch.uint8)
    ks = torch.full((1, 1), 2.0 ** -6)
    q = torch.randn(1, H, d, generator=gen).to(torch.bfloat16)
    out, lse, st = torch.empty(1, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(1, H, device=DEV), status()
    hcl.hcl_paged_attn(q.cuda(), i32([0, 1]), i32([n * page - 1]), hcl.PagedKV(codes.cuda(), ks.cuda()),
                       torch.zeros(1, n, dtype=torch.int32, device=DEV), i32([n * page]), out, lse=lse, status=st)
    assert st.item() == 0
    want, wl, mass, zabs = ref.attn(ref.f64(q), [0, 1], [page - 1], [page], np.zeros((1, 1), int), codes.numpy(),
                                    ks.numpy(), None, None, page, 1, 0, 1 / math.sqrt(d))
    wl = wl + math.log(n)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    long = 4 * (n / sms / 2 + 1) * 2.0 ** -23
    assert np.all(np.abs(ref.f64(out) - want) <= tolerance(want, mass, zabs) + 2 * long * mass)
    assert np.all(np.abs(ref.f64(lse) - wl) <= 2.0 ** -16 * zabs + 2.0 ** -19 * (1 + np.abs(wl)) + 2 * long)


def test_attn_two_calls_at_once(hcl):
    """Calls on two streams, each with its own workspace, give what each gives alone."""
    gen = torch.Generator(device=DEV).manual_seed(12)
    calls = []
    for lens, news, G, d in (([4000, 70, 900], [300, 1, 64], 8, 128), ([3000, 2500, 10], [1, 1, 1], 64, 64),
                             ([9000, 30, 700], [1, 1, 1], 8, 128)):
        per = -(-max(lens) // 32)
        k = (torch.randn(3 * per, 2, 32, d, generator=gen, device=DEV) * 100).to(torch.float8_e4m3fn).view(torch.uint8)
        store = hcl.PagedKV(k, torch.full((3 * per, 2), 2.0 ** -6, device=DEV))
        table = torch.randperm(3 * per, generator=gen, device=DEV).to(torch.int32).view(3, per)
        q = torch.randn(sum(news), 2 * G, d, generator=gen, device=DEV).to(torch.bfloat16)
        ws = torch.empty(hcl.paged_attn_workspace_bytes(sum(news), 2 * G, 2, d), dtype=torch.uint8, device=DEV)
        args = (q, i32(np.concatenate([[0], np.cumsum(news)])), i32([a - b for a, b in zip(lens, news)]), store, table,
                i32(lens))
        out = torch.empty_like(q)
        calls.append((args, ws, max(news), out, torch.cuda.Stream()))
    want = []
    for args, ws, mq, out, _ in calls:
        want.append(hcl.hcl_paged_attn(*args, torch.empty_like(out), max_q=mq, ws=ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, ws, mq, out, stream in calls:
            hcl.hcl_paged_attn(*args, out, max_q=mq, ws=ws, stream=stream)
    torch.cuda.synchronize()
    for (_, _, _, out, _), w in zip(calls, want):
        assert torch.equal(out.view(torch.int16), w.view(torch.int16))  # (bits: some codes are NaN)


@pytest.mark.parametrize("H", [8, 32])
def test_attn_max_q_of_zero(hcl, H):
    """No request may have a query then: one that has gets no output, and the status word says so."""
    gen = torch.Generator().manual_seed(6)
    table, k, ks, v, vs = make_cache([64, 64], 16, 1, 64, True, gen)
    q = torch.randn(1, H, 64, generator=gen).to(torch.bfloat16).cuda()
    out, st = torch.full((1, H, 64), 3.0, dtype=torch.bfloat16, device=DEV), status()
    hcl.hcl_paged_attn(q, i32([0, 1, 1]), i32([63, 63]), hcl.PagedKV(k.cuda(), ks.cuda()), i32(table), i32([64, 64]),
                       out, max_q=0, status=st)
    assert st.item() == 16 and bool((out == 3.0).all())


@pytest.mark.parametrize("G,d,lens,news,shared", [(8, 128, [9000, 20000, 100], [1, 1, 1], False),
                                                  (128, 128, [9000, 5000], [1, 1], True),
                                                  (4, 64, [20000], [1], False)])
def test_attn_long_split(hcl, G, d, lens, news, shared):
    """Requests long enough to be split over many blocks, and the same bits every time."""
    case = dict(lens=lens, news=news, Hkv=1, G=G, d=d, page=64, shared=shared)
    a = check_attn(hcl, case)
    assert_attn(*a)
    b = check_attn(hcl, case)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("G,news", [(8, [1, 1, 1]), (8, [1, 70, 1]), (64, [1, 1, 1])])
def test_attn_slice_of_wider_rows_stream_and_graph(hcl, G, news):
    """q as a slice of a fused projection, a side stream, then a captured call replayed with other
    lengths, another table and a used workspace."""
    gen = torch.Generator().manual_seed(9)
    lens, page, d = [200, 90, 33], 16, 128
    T = sum(news)
    cu = np.concatenate([[0], np.cumsum(news)])
    table, k, ks, v, vs = make_cache(lens, page, 1, d, False, gen)
    wide = torch.randn(T, (G + 2) * d, generator=gen).to(torch.bfloat16).cuda()
    q = wide[:, :G * d].view(T, G, d)
    store = hcl.PagedKV(k.cuda(), ks.cuda(), v.cuda(), vs.cuda())
    out, lse = torch.empty(T, G, d, dtype=torch.bfloat16, device=DEV), torch.empty(T, G, device=DEV)
    d_cu, d_start, d_len, d_table = i32(cu), i32([l - n for l, n in zip(lens, news)]), i32(lens), i32(table)
    ws = torch.full((max(16, hcl.paged_attn_workspace_bytes(T, G, 1, d)),), 0xFF, dtype=torch.uint8, device=DEV)

    def call(stream=None, ws=ws):
        hcl.hcl_paged_attn(q, d_cu, d_start, store, d_table, d_len, out, lse=lse, max_q=max(news), ws=ws,
                           stream=stream)

    def check(lens, tab):
        w, wl, mass, zabs = ref.attn(ref.f64(q), cu, [l - n for l, n in zip(lens, news)], lens, tab, k.numpy(),
                                     ks.numpy(), v.numpy(), vs.numpy(), page, 1, 0, 1 / math.sqrt(d))
        assert_attn(ref.f64(out), ref.f64(lse), w, wl, mass, zabs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    check(lens, table)
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side, ws=None)
    side.synchronize()
    check(lens, table)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens2, tab2 in (([120, 80, 20], table), ([90, 72, 33], table[[1, 0, 2]])):
        d_len.copy_(i32(lens2))
        d_start.copy_(i32([l - n for l, n in zip(lens2, news)]))
        d_table.copy_(i32(tab2))
        out.zero_()
        ws.fill_(0xA5)
        g.replay()
        torch.cuda.synchronize()
        check(lens2, tab2)


def test_attn_far_into_a_large_cache(hcl):
    """Pages whose codes lie beyond 2^32 bytes, for the row kernel and the tile kernel."""
    n_pages = (1 << 32) // (128 * 128) + 40
    c = torch.full((n_pages, 1, 128, 128), 0x7F, dtype=torch.uint8, device=DEV)
    s = torch.full((n_pages, 1), 2.0 ** -6, device=DEV)
    gen = torch.Generator().manual_seed(3)
    tail = codes_of(30, 1, 128, 128, gen)
    c[-30:] = tail.cuda()
    ids = np.arange(20, 0, -1, dtype=np.int32)[None]       # within the tail
    for G in (8, 128):
        q = torch.randn(1, G, 128, generator=gen).to(torch.bfloat16)
        out, lse = torch.empty(1, G, 128, dtype=torch.bfloat16, device=DEV), torch.empty(1, G, device=DEV)
        hcl.hcl_paged_attn(q.cuda(), i32([0, 1]), i32([2499]), hcl.PagedKV(c, s), i32(ids + n_pages - 30), i32([2500]),
                           out, lse=lse, max_q=1)
        w, wl, mass, zabs = ref.attn(ref.f64(q), [0, 1], [2499], [2500], ids, tail.numpy(),
                                     np.full((30, 1), 2.0 ** -6), None, None, 128, 1, 0, 1 / math.sqrt(128))
        assert_attn(ref.f64(out), ref.f64(lse), w, wl, mass, zabs)


# ------------------------------------------------------------------------------------ binding


def test_binding_refusals(hcl):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV)
    s = torch.ones(4, 2, device=DEV)
    with pytest.raises(ValueError):
        hcl.PagedKV(k, s, k)                       # v without its scale
    with pytest.raises(ValueError):
        hcl.PagedKV(k, s[:, :1])
    with pytest.raises(ValueError):
        hcl.PagedKV(k.float(), s)
    with pytest.raises(ValueError):
        hcl.PagedKV(k.cpu(), s.cpu())
    store = hcl.PagedKV(k, s)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    ok = dict(q=q, cu_q=i32([0, 3]), q_start=i32([0]), store=store, table=i32([[0, 1]]), kv_len=i32([3]), out=out)
    hcl.hcl_paged_attn(**ok)
    for bad in (dict(q=q.float()), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(cu_q=i32([0, 1, 3])),
                dict(cu_q=ok["cu_q"].long()), dict(kv_len=i32([3]).cpu()), dict(out=out.float()),
                dict(out=out[:2]), dict(lse=torch.empty(3, 4, dtype=torch.float64, device=DEV)),
                dict(sink=torch.zeros(3, device=DEV)), dict(W=4, m=2), dict(scale=-1.0), dict(scale=math.nan),
                dict(q=q[:, :3], out=out[:, :3].contiguous())):
        with pytest.raises((ValueError, RuntimeError)):
            hcl.hcl_paged_attn(**{**ok, **bad})
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    hcl.hcl_paged_write(x, None, i32([0, 1, 2]), store)
    for args in ((x, x, i32([0, 1, 2]), store), (x[:2], None, i32([0, 1, 2]), store),
                 (x.float(), None, i32([0, 1, 2]), store), (x[:, :1], None, i32([0, 1, 2]), store),
                 (x, None, torch.tensor([0, 1, 2], device=DEV), store)):
        with pytest.raises((ValueError, RuntimeError)):
            hcl.hcl_paged_write(*args)
    # nothing to do
    hcl.hcl_paged_write(x[:0], None, i32([]), store)
    hcl.hcl_paged_attn(q[:0], i32([0, 0]), i32([0]), store, i32([[0, 1]]), i32([3]), out[:0])


@pytest.mark.parametrize("Hkv,G,d,shared,W", [(8, 8, 128, False, 0), (8, 4, 128, True, 0), (4, 16, 128, False, 0),
                                              (8, 8, 64, False, 0), (4, 16, 64, True, 0), (2, 128, 128, True, 0),
                                              (4, 64, 64, False, 0), (8, 2, 128, False, 3000)])
def test_attn_long_rings(hcl, Hkv, G, d, shared, W):
    """Blocks that run through their rings many times and over several requests and heads: sampled
    rows against 64 bits."""
    gen = torch.Generator().manual_seed(11)
    lens = [70000, 1, 33333, 9000, 64, 50001]
    page, H, B = 64, Hkv * G, len(lens)
    table, k, ks, v, vs = make_cache(lens, page, Hkv, d, shared, gen)
    q = torch.randn(B, H, d, generator=gen).to(torch.bfloat16)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    out, lse, st = torch.empty(B, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, device=DEV), status()
    scale = 1 / math.sqrt(d)
    hcl.hcl_paged_attn(q.cuda(), i32(range(B + 1)), i32([n - 1 for n in lens]),
                       hcl.PagedKV(dev(k), dev(ks), dev(v), dev(vs)), i32(table), i32(lens), out, lse=lse, max_q=1,
                       W=W, status=st)
    assert st.item() == 0
    for b in range(B):
        for h in (0, G - 1, H // 2, H - 1):
            g = h // G
            args = (ref.f64(q[b:b + 1, h:h + 1]), [0, 1], [lens[b] - 1], lens[b:b + 1], table[b:b + 1],
                    k[:, g:g + 1].numpy(), ks[:, g:g + 1].numpy(), None if shared else v[:, g:g + 1].numpy(),
                    None if shared else vs[:, g:g + 1].numpy(), page, 1, W, scale)
            w, wl, mass, zabs = ref.attn(*args)
            assert_attn(ref.f64(out[b:b + 1, h:h + 1]), ref.f64(lse[b:b + 1, h:h + 1]), w, wl, mass, zabs)


@pytest.mark.parametrize("G,new,order", [(8, 1, "up"), (8, 1, "down"), (16, 1, "up"), (128, 1, "up"), (128, 1, "down"),
                                         (8, 60, "up"), (8, 60, "mid")])
def test_attn_zero_pages_among_others(hcl, G, new, order):
    """Pages of zero values (scale 2^-126) beside ordinary ones: their rows take their share of the
    softmax, whatever the order and however the scores lie."""
    def poison(table, k, ks, v, vs, q):
        used = table[0][:20]
        zero = {"up": used[:10], "down": used[10:19], "mid": used[5:13]}[order]
        v[zero] = 0
        vs[zero] = 2.0 ** -126
        if order != "mid":
            ks[zero] *= 8.0      # the zero rows have the sharper scores
    got, gl, want, wl, mass, zabs = check_attn(hcl, dict(lens=[319], news=[new], Hkv=1, G=G, d=128, page=16),
                                               poison=poison, seed=5)
    # Where the zero rows take all but 2^-60 of a row's sum, the reference M of the other rows'
    # weights is kept 2^59 / N above where their own largest would put it (the sum is held below
    # 2^60), and what lies 2^-29 below M is lost in fp16: terms with p * v_scale below
    # 2^-84 * N * (the largest scale), N = 319 of them: under 2^-60 of the largest value.
    lost = 2.0 ** -60 * 448 * 2.0 ** -4
    assert_attn(got, gl, np.where(np.abs(got - want) <= lost, got, want), wl, mass, zabs)


# ------------------------------------------------------------------------------------ together


def held_rows(b, layer, r):
    """The rows that the layer's cache holds for request r, as values (float64)."""
    n = b.seq_len[r].item()
    ids = b.table[r, :-(-n // b.page)].cpu().numpy()

    def plane(codes, scale):
        v = ref.decode_e4m3(codes.cpu().numpy()[ids]) * scale.cpu().numpy()[ids].astype(np.float64)[:, :, None, None]
        return v.transpose(0, 2, 1, 3).reshape(-1, v.shape[1], v.shape[3])[:n]

    s = layer.store
    return plane(s.k, s.k_scale), (None if s.v is None else plane(s.v, s.v_scale))


@pytest.mark.parametrize("page,d,Hkv,G,graph", [(16, 128, 2, 8, False), (64, 64, 1, 4, True)])
def test_serving_steps(hcl, page, d, Hkv, G, graph):
    """Prompts, decode steps (captured and replayed in the second case), rejected drafts and a
    request that takes another's place: plan, write and attention as a server calls them.  The
    cache follows the rows that were written, the attention follows the cache."""
    from heavily_compressed_long_b200.pipeline import PagedAttnLayer, PagedBatch
    gen = torch.Generator().manual_seed(page)
    B, T, H = 4, 160, Hkv * G
    b = PagedBatch(B, page, 20, 4 * 20, T)
    layer = PagedAttnLayer(b, 4 * 20, H, Hkv, d)
    rows = [np.zeros((0, 2, Hkv, d)) for _ in range(B)]  # what was written
    out, lse = torch.zeros(T, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(T, H, device=DEV)
    q, k, v = (torch.zeros(T, h, d, dtype=torch.bfloat16, device=DEV) for h in (H, Hkv, Hkv))
    d_new, d_keep = i32([0] * B), i32([0] * B)

    def calls(max_q):
        b.plan(d_new, d_keep)
        layer.step(q, k, v, out, lse=lse, max_q=max_q)

    captured = None
    steps = [([0] * 4, [40, 1, 70, 17])] + [(None, [1, 1, 1, 1])] * 4 + [(None, [3, 0, 4, 1]), ("less", [2, 1, 1, 1]),
                                                                       ("replace", [1, 30, 1, 2])]
    for keep, new in steps:
        lens = [len(r) for r in rows]
        keep_n = (list(keep) if isinstance(keep, list) else [max(0, n - 2) for n in lens] if keep == "less"
                  else [lens[0], 0, lens[2], lens[3]] if keep == "replace" else lens)
        d_new.copy_(i32(new))
        d_keep.copy_(i32(keep_n))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen).to(torch.bfloat16))
        if graph and keep is None and new == [1] * 4:
            if captured is None:
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    calls(1)
            captured.replay()
        else:
            calls(max(new))
        assert b.status.item() == 0
        at = 0
        kv = np.stack([ref.f64(k), ref.f64(v)], 1)
        for r in range(B):
            rows[r] = np.concatenate([rows[r][:keep_n[r]], kv[at:at + new[r]]])
            at += new[r]
        assert b.seq_len.tolist() == [len(r) for r in rows]
        cu = np.concatenate([[0], np.cumsum(new)])
        for r in range(B):
            kk, vv = held_rows(b, layer, r)
            # a code is within half a step of its value at the page's scale, and was rounded once
            # more at most per growth of the scale for values near the subnormals: 2^-4 of the value
            # or two subnormal half steps, 2 * 2^-10 of the scale (<= 2 * amax / 448, amax < 8)
            for got, want in ((kk, rows[r][:, 0]), (vv, rows[r][:, 1])):
                assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2 * 2.0 ** -10 * 16 / 448)
        tab = b.table.cpu().numpy()
        w, wl, mass, zabs = ref.attn(ref.f64(q), cu, keep_n, b.seq_len.tolist(), np.maximum(tab, 0),
                                     layer.store.k.cpu().numpy(), layer.store.k_scale.cpu().numpy(),
                                     layer.store.v.cpu().numpy(), layer.store.v_scale.cpu().numpy(), page, 1, 0,
                                     1 / math.sqrt(d))
        n = int(cu[-1])
        assert_attn(ref.f64(out)[:n], ref.f64(lse)[:n], w[:n], wl[:n], mass[:n], zabs[:n])


def test_paged_hca_layer_against_oracle(hcl, orc):
    """HCA over paged entries and a paged raw window: compress, plan, write, attend, merge, against
    the oracle's HCA attention over the rows that the caches hold."""
    from heavily_compressed_long_b200.pipeline import PagedBatch, PagedHcaLayer
    gen = torch.Generator().manual_seed(21)
    lens, news, H, d, mh, W = [1500, 700], [5, 1], 16, 128, 128, 128
    B, T = 2, 8
    raw, ent = PagedBatch(B, 64, 24, 50, 2200), PagedBatch(B, 16, 2, 6, 20)
    q_raw = PagedBatch(B, 64, 24, 50, T)  # the step's plan: the same state, fewer rows
    sink = torch.randn(H, generator=gen)
    kv = [torch.randn(1, n, d, generator=gen).to(torch.bfloat16).cuda() for n in lens]
    gate = [torch.randn(1, n, d, generator=gen).to(torch.bfloat16).cuda() for n in lens]
    bias = (torch.randn(mh, generator=gen) * 0.1).cuda()
    done = [n // mh for n in lens]  # completed entries
    entries = []
    for i in range(B):
        e = torch.empty(1, -(-lens[i] // mh), d, dtype=torch.bfloat16, device=DEV)
        hcl.hcl_hca_compress(kv[i], gate[i], bias, mh, e)
        entries.append(e[0, :done[i]])
    layer = PagedHcaLayer(q_raw, ent, 50, 6, H, d, mh=mh, W=W, sink=sink.cuda())
    # everything but the step's rows, then the step's rows
    raw.plan(i32([n - m for n, m in zip(lens, news)]))
    first = torch.zeros(2200, 1, d, dtype=torch.bfloat16, device=DEV)
    first[:sum(lens) - sum(news), 0] = torch.cat([x[0, :n - m] for x, n, m in zip(kv, lens, news)])
    hcl.hcl_paged_write(first, None, raw.slot, layer.raw_layer.store)
    q_raw.seq_len, q_raw.table, q_raw.free_list, q_raw.n_free = raw.seq_len, raw.table, raw.free_list, raw.n_free
    q_raw.plan(i32(news))
    step = torch.zeros(T, 1, d, dtype=torch.bfloat16, device=DEV)
    step[:sum(news), 0] = torch.cat([x[0, n - m:] for x, n, m in zip(kv, lens, news)])
    layer.raw_layer.write(step)
    ent.plan(i32(done))
    e_rows = torch.zeros(20, 1, d, dtype=torch.bfloat16, device=DEV)
    e_rows[:sum(done), 0] = torch.cat(entries)
    layer.entry_layer.write(e_rows)
    q = torch.randn(T, H, d, generator=gen).to(torch.bfloat16)
    out, lse = torch.empty(T, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, device=DEV)
    layer.attend(q.cuda(), out, lse=lse, max_q=max(news))
    assert q_raw.status.item() == 0 and ent.status.item() == 0 and raw.status.item() == 0
    at = 0
    for i in range(B):
        rr, _ = held_rows(q_raw, layer.raw_layer, i)
        ee, _ = held_rows(ent, layer.entry_layer, i)
        as16 = lambda x: torch.from_numpy(x[None, :, 0].astype(np.float32)).to(torch.bfloat16)  # noqa: E731  (exact)
        pos = torch.arange(lens[i] - news[i], lens[i], dtype=torch.int32)[None]
        o, l = orc.hca_attn(q[at:at + news[i]][None], orc.KV(0, as16(ee), done[i]), done[i], mh,
                            orc.KV(0, as16(rr), lens[i]), W, pos, sink=sink)
        # the framework's bound for attention over 8-bit rows; log-sum-exps: scores of bf16 queries
        # and exact rows
        assert np.abs(ref.f64(out)[at:at + news[i]] - o[0]).max() <= 2e-2
        assert np.abs(ref.f64(lse)[at:at + news[i]] - l[0]).max() <= 1e-3
        at += news[i]


def test_paged_hca_layer_fewer_rows_in_a_later_step(hcl):
    """Rows behind the last request's become zeros, whatever an earlier and longer step left."""
    from heavily_compressed_long_b200.pipeline import PagedBatch, PagedHcaLayer
    gen = torch.Generator().manual_seed(5)
    B, T, H, d = 2, 12, 16, 128
    raw, ent = PagedBatch(B, 16, 8, 16, T), PagedBatch(B, 16, 2, 4, T)
    layer = PagedHcaLayer(raw, ent, 16, 4, H, d, mh=128, W=128)
    ent.plan(i32([0, 0]))
    out = torch.empty(T, H, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, H, device=DEV)
    for news in ([7, 5], [1, 2]):
        raw.plan(i32(news))
        layer.raw_layer.write(torch.randn(T, 1, d, generator=gen).to(torch.bfloat16).cuda())
        layer.attend(torch.randn(T, H, d, generator=gen).to(torch.bfloat16).cuda(), out, lse=lse, max_q=max(news))
        n = sum(news)
        assert torch.isfinite(lse[:n]).all() and (out[:n] != 0).any(-1).all()
        assert (out[n:] == 0).all() and torch.isneginf(lse[n:]).all()


def test_one_row_of_any_stride(hcl):
    """A single row's token stride does not matter."""
    gen = torch.Generator().manual_seed(6)
    wide = torch.randn(1, 2 * 64 + 3, generator=gen).to(torch.bfloat16).cuda()
    x = wide[:, :128].unflatten(1, (2, 64))
    a, b = (hcl.PagedKV.empty(1, 2, 16, 64, shared=True) for _ in range(2))
    out = [torch.empty(1, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for store, rows, o in ((a, x, out[0]), (b, x.contiguous(), out[1])):
        hcl.hcl_paged_write(rows, None, i32([0]), store)
        hcl.hcl_paged_attn(rows, i32([0, 1]), i32([0]), store, i32([[0]]), i32([1]), o)
    assert torch.equal(a.k[:, :, 0], b.k[:, :, 0]) and torch.equal(*out)


@pytest.mark.parametrize("d,page,shared", [(128, 64, False), (128, 16, False), (64, 64, False), (128, 64, True)])
def test_attn_same_bits_under_load(hcl, d, page, shared):
    """Calls in flight behind one another, on caches too large to stay in L2 together: the same bits
    every time (a read that came too late once took the next rows' bytes)."""
    B, n, Hkv, G = 3, 3000, 4, 8
    gen = torch.Generator(device=DEV).manual_seed(4)
    sets = []
    for _ in range(2):
        per = -(-n // page)
        shape = (B * per, Hkv, page, d)

        def plane():
            x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16).mul_(100).clamp_(-448, 448)
            return x.to(torch.float8_e4m3fn).view(torch.uint8), torch.full((B * per, Hkv), 2.0 ** -6, device=DEV)

        k, ks = plane()
        store = hcl.PagedKV(k, ks) if shared else hcl.PagedKV(k, ks, *plane())
        table = torch.randperm(B * per, generator=gen, device=DEV).to(torch.int32).view(B, per)
        q = torch.randn(B * n, Hkv * G, d, generator=gen, device=DEV).to(torch.bfloat16)
        sets.append((q, store, table, torch.empty_like(q)))
    cu, start, lens = i32([0, n, 2 * n, 3 * n]), i32([0] * B), i32([n] * B)
    ws = [torch.empty(hcl.paged_attn_workspace_bytes(B * n, Hkv * G, Hkv, d), dtype=torch.uint8, device=DEV)
          for _ in sets]

    def call(i):
        q, store, table, out = sets[i]
        hcl.hcl_paged_attn(q, cu, start, store, table, lens, out, max_q=n, ws=ws[i])

    call(0)
    torch.cuda.synchronize()
    first = sets[0][3].clone()
    for _ in range(25):
        call(0)
        call(1)
        call(0)
        torch.cuda.synchronize()
        assert torch.equal(sets[0][3], first)
