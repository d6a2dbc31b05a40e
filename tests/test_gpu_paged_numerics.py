"""Attention over the paged 8-bit cache where the softmax weights or the pages' value scales lie far
apart: against plain references in 64 bits."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged import assert_attn, check_attn

pytestmark = pytest.mark.gpu



def assert_attn_lost(got, codes, top, rows):
    """assert_attn with what the products of weight and value scale may lose beside their 11 bits:
    half a step of fp16's subnormals, 2^-25, where the largest product is at least 2^12 (more than
    16 query rows) or 2^15: 2^-37 or 2^-40 of the largest product, which is at most the largest
    scale `top`, for each of the rows, whose codes sum to `codes` [d]."""
    out, lse, want, wl, mass, zabs = got
    lost = (2.0 ** -40 if rows <= 16 else 2.0 ** -37) * top * codes
    assert_attn(np.where(np.abs(out - want) <= lost, want, out - np.clip(out - want, -lost, lost)), lse, want, wl, mass, zabs)


# query heads per KV head and new rows: few query rows (8, 16), many on one token, a prompt
FORMS = [(8, 1), (16, 1), (4, 3), (128, 1), (8, 60)]


@pytest.mark.parametrize("G,new", FORMS)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("at", [0, 290])
@pytest.mark.parametrize("alike", [True, False])
@pytest.mark.parametrize("orders", [14.0, 20.0, 26.3, 27.6, 30.0, 44.0, 60.0])
def test_attn_tail_below_a_row_without_value(hcl, G, new, shared, at, alike, orders):
    """One row whose weight is 2^orders of any other's and whose values are zeros (where rows are both
    key and value: zeros in all dimensions but its key's one): the others make the output.  With
    scores alike, what their weights lose they lose alike, so nothing of it averages out."""
    codes = []

    def poison(table, k, ks, v, vs, q):
        ks[:] = 2.0 ** -7
        k[:, :, :, 0] = 0
        page, row = table[0, at // 16], at % 16
        k[page, :, row] = 0
        k[page, :, row, 0] = 0x70                  # 128: the key 1
        q[:] *= 0.0 if alike else 2.0 ** -6
        q[:, :, 0] = 8.0
        if v is not None:
            v &= 0x7F                              # one sign: the output is as large as its terms
            v[page, :, row] = 0
        codes.append(np.abs(np.nan_to_num(ref.decode_e4m3((k if v is None else v)[table[0, :21], 0].numpy()))).sum((0, 1)))

    scale = orders * float(np.log(2.0)) / 8.0
    got = check_attn(hcl, dict(lens=[330], news=[new], Hkv=1, G=G, d=128, page=16, shared=shared, scale=scale),
                     poison=poison, seed=3)
    assert_attn_lost(got, codes[0], 2.0 ** -5 if not shared else 2.0 ** -7, new * G)


@pytest.mark.parametrize("orders", [30.0, 60.0])
def test_attn_long_tail_over_many_blocks(hcl, orders):
    """The same over a context that many blocks share: the merge keeps what the parts hold."""
    def poison(table, k, ks, v, vs, q):
        ks[:] = 2.0 ** -7
        k[:, :, :, 0] = 0
        k[table[0, 0], :, 0] = 0
        k[table[0, 0], :, 0, 0] = 0x70
        q[:] *= 2.0 ** -6
        q[:, :, 0] = 8.0
        v &= 0x7F
        v[table[0, 0], :, 0] = 0
        codes.append(np.abs(np.nan_to_num(ref.decode_e4m3(v[table[0, :313], 0].numpy()))).sum((0, 1)))

    for G in (8, 64):
        codes = []
        got = check_attn(hcl, dict(lens=[20000], news=[1], Hkv=1, G=G, d=64, page=64,
                                   scale=orders * float(np.log(2.0)) / 8.0), poison=poison, seed=4)
        assert_attn_lost(got, codes[0], 2.0 ** -5, G)


# Which rows the queries see: a prompt from its start, drafts over a page's end, one token ahead of
# the rows held, windows that have left the first pages, chunks over entries.
VIEWS = {
    "prompt": dict(lens=[40], news=[40], start=[0]),
    "prompt_long": dict(lens=[300], news=[300], start=[0]),
    "drafts": dict(lens=[18], news=[4], start=[14]),
    "behind": dict(lens=[64], news=[1], start=[10]),
    "window": dict(lens=[100], news=[1], W=16),
    "window_chunk": dict(lens=[400], news=[90], W=40),
    "entries": dict(lens=[60], news=[4], start=[100], m=4),
}


@pytest.mark.parametrize("G", [1, 4, 8, 64])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("view", sorted(VIEWS))
@pytest.mark.parametrize("apart", [70, 120])
@pytest.mark.parametrize("large", ["first", "last", "mixed"])
def test_attn_scales_of_pages_that_a_query_does_not_see(hcl, G, shared, view, apart, large):
    """Value scales 2^apart apart: what a query sees decides its output, though pages with far larger
    scales stand beside it in the call."""
    case = dict(Hkv=1, G=G, d=64, page=16, shared=shared, **VIEWS[view])

    def poison(table, k, ks, v, vs, q):
        n = -(-case["lens"][0] // 16)
        big = {"first": np.arange(n) * 16 < (case["lens"][0] - case["news"][0]) // 16 * 16 - 16,
               "last": np.arange(n) > 0, "mixed": np.arange(n) % 3 == 1}[large]
        if view == "behind":
            big = np.arange(n) > 0
        s = ks if v is None else vs
        for i in range(n):
            s[table[0, i]] = 2.0 ** (20 if big[i] else 20 - apart)
        if v is None:                       # (a key's scale is its value's: scores of ordinary size)
            q *= 2.0 ** -22

    scales = []

    def keep(table, k, ks, v, vs, q):
        poison(table, k, ks, v, vs, q)
        scales.extend(float((ks if v is None else vs)[pg, 0]) for pg in table[0, :-(-case["lens"][0] // 16)])

    got, gl, want, wl, mass, zabs = check_attn(hcl, case, poison=keep, seed=len(view))
    # a product of weight and scale loses up to 2^-37 of the query's largest, which its mass holds for
    # codes of ordinary size, or 2^-60 of the largest scale that it sees, for each row with codes of at most 448
    m, W = case.get("m", 1), case.get("W", 0)
    for i in range(case["news"][0]):
        p = (case["start"][0] if "start" in case else case["lens"][0] - case["news"][0]) + i
        hi = min(case["lens"][0], (p + 1) // m)
        lo = max(0, p - W + 1) if W else 0
        lost = 2.0 ** -60 * max(scales[lo // 16:-(-hi // 16)]) * 448 * (hi - lo)
        diff = got[i] - want[i]
        got[i] = np.where(np.abs(diff) <= lost, want[i], got[i] - np.clip(diff, -lost, lost))
    assert_attn(got, gl, want, wl, mass, zabs)


@pytest.mark.parametrize("G,lens,news", [(8, [40, 3000], [1, 1]), (16, [200000], [1]), (128, [700], [1]), (64, [200000], [1]),
                                         (8, [90], [60]), (4, [3000, 5], [3, 3])])
@pytest.mark.parametrize("scale", [-126, -118, 119])
def test_attn_smallest_and_largest_value_scales(hcl, G, lens, news, scale):
    """Values of 2^-126 (and up to 2^119) times their codes come out with bf16's precision however
    long the sum of the weights."""
    def poison(table, k, ks, v, vs, q):
        vs[:] = 2.0 ** scale
        ks[:] = 2.0 ** -7
        v &= 0x7F

    got, gl, want, wl, mass, zabs = check_attn(hcl, dict(lens=lens, news=news, Hkv=1, G=G, d=64, page=64, qs=0.2), poison=poison)
    assert_attn(got * 2.0 ** -scale, gl, want * 2.0 ** -scale, wl, mass * 2.0 ** -scale, zabs)
