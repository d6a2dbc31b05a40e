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
