"""Host-side validation of the paged cache's entry points (no GPU), and its references."""
import ctypes

import numpy as np
import pytest
import torch

from tests import paged_ref as ref


@pytest.fixture(scope="module")
def lib():
    from heavily_compressed_long_b200 import build as b
    b.build()
    from heavily_compressed_long_b200 import _lib
    return _lib


FAKE = 1 << 20


def store(lib, page=64, n=8, Hkv=2, d=128, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE):
    return ctypes.byref(lib.hcl_paged_kv_t(page, n, Hkv, d, k, v, ks, vs))


def attn(lib, kv, q=FAKE, qs=1024, T=4, H=8, B=2, mp=4, max_q=2, m=1, W=0, scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40,
         table=FAKE):
    return lib.lib().hcl_paged_attn(q, qs, T, H, FAKE, FAKE, B, kv, table, mp, FAKE, max_q, m, W, scale, None, out,
                                    None, ws, wsb, None, None)


@pytest.mark.parametrize("change,code", [
    (dict(page=48), 2), (dict(page=256), 2), (dict(d=96), 2), (dict(d=256), 2), (dict(n=0), 1), (dict(Hkv=0), 1),
    (dict(n=1 << 25), 1), (dict(k=None), 1), (dict(vs=None), 1), (dict(v=None), 1), (dict(k=FAKE + 16), 1),
    (dict(ks=FAKE + 2), 1)])
def test_store_refused(lib, change, code):
    L = lib.lib()
    assert attn(lib, store(lib, **change)) == code
    assert L.hcl_paged_write(FAKE, 256, FAKE, 256, FAKE, 4, store(lib, **change), None, None) == code
    assert L.hcl_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(H=7), 1), (dict(H=2 * 129, qs=1 << 16), 2), (dict(B=9000), 2), (dict(m=0), 1), (dict(W=-1), 1),
    (dict(m=4, W=8), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(T=-1), 1), (dict(max_q=-1), 1), (dict(T=1 << 29), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(table=None), 1), (dict(mp=0), 1), (dict(mp=1 << 26), 1), (dict(qs=1000), 1), (dict(qs=1028), 1),
    (dict(q=FAKE + 8), 1), (dict(out=FAKE + 8), 1)])
def test_attn_refused(lib, change, code):
    assert attn(lib, store(lib), **change) == code


def test_attn_workspace_too_small(lib):
    need = lib.lib().hcl_paged_attn_workspace_bytes(4, 8, 2, 128)
    if need:
        assert attn(lib, store(lib), wsb=need - 1) == 1
        assert attn(lib, store(lib), ws=None) == 1


def test_write_refused(lib):
    L = lib.lib()
    ok = [FAKE, 256, FAKE, 256, FAKE, 4, store(lib), None, None]
    for i, bad in ((0, None), (0, FAKE + 8), (1, 255), (1, 260), (2, None), (3, 128), (4, None), (5, -1), (6, None)):
        args = list(ok)
        args[i] = bad
        assert L.hcl_paged_write(*args) == 1, i
    assert L.hcl_paged_write(FAKE, 256, FAKE, 256, FAKE, 4, store(lib, v=None, vs=None), None, None) == 1
    assert L.hcl_paged_write(None, 256, None, 256, None, 0, store(lib), None, None) == 0


def test_plan_refused(lib):
    L = lib.lib()
    ok = [FAKE, FAKE, 4, 16, FAKE, FAKE, 8, FAKE, 64, FAKE, 32, FAKE, FAKE, FAKE, None, None]
    for i, bad, code in ((0, None, 1), (1, None, 1), (2, -1, 1), (2, 8193, 2), (3, 24, 2), (4, None, 1), (5, None, 1),
                         (6, 0, 1), (6, 1 << 30, 1), (7, None, 1), (8, 1 << 28, 1), (8, -1, 1), (9, None, 1),
                         (10, -1, 1), (10, (1 << 29) + 1, 1), (11, None, 1), (12, None, 1), (13, None, 1)):
        args = list(ok)
        args[i] = bad
        assert L.hcl_page_plan(*args) == code, (i, bad)


def test_reference_e4m3_against_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.decode_e4m3(codes), want)
    x = np.random.default_rng(0).normal(size=20000) * np.exp2(np.random.default_rng(1).uniform(-12, 9, 20000))
    x = np.clip(x, -448, 448).astype(np.float32)
    np.testing.assert_array_equal(ref.round_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())
    assert ref.pow2_scale(448.0) == 1.0 and ref.pow2_scale(448.1) == 2.0 and ref.pow2_scale(0.0) == 2.0 ** -126


def test_reference_attn_against_torch():
    """The reference itself: a causal prompt equals scaled dot-product attention in 64 bits."""
    g = torch.Generator().manual_seed(0)
    page, n, d = 16, 37, 64
    k = (torch.randn(4, 1, page, d, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    ks = torch.full((4, 1), 0.01)
    table = np.array([[2, 0, 3]], np.int32)
    q = torch.randn(n, 2, d, generator=g).double()
    out, lse, _, _ = ref.attn(q.numpy(), [0, n], [0], [n], table, k.numpy(), ks.numpy(), None, None, page, 1, 0, 0.125)
    kk = torch.from_numpy(ref.decode_e4m3(k[[2, 0, 3], 0].numpy()).reshape(-1, d)[:n] * np.float64(ks[0, 0]))
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), kk[None].expand(2, -1, -1), kk[None].expand(2, -1, -1), is_causal=True, scale=0.125)
    np.testing.assert_allclose(out, want.transpose(0, 1).numpy(), atol=1e-12)
