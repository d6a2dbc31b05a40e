"""Host-side validation of the fp32 parts' entry points (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from heavily_compressed_long_b200 import build as b
    b.build()
    from heavily_compressed_long_b200 import _lib
    return _lib


FAKE = 1 << 20


@pytest.mark.parametrize("at,bad,code", [(0, None, 1), (0, FAKE + 8, 1), (1, 1000, 1), (2, -1, 1), (3, 7, 1), (6, 9000, 2),
                                         (8, None, 1), (11, -1, 1), (12, 0, 1), (13, -1, 1), (14, 0.0, 1), (16, None, 1),
                                         (16, FAKE + 8, 1), (18, None, 1)])
def test_attn_refused(lib, at, bad, code):
    kv = ctypes.byref(lib.hcl_paged_kv_t(64, 8, 2, 128, FAKE, FAKE, FAKE, FAKE))
    args = [FAKE, 1024, 4, 8, FAKE, FAKE, 2, kv, FAKE, 4, FAKE, 2, 1, 0, 0.1, None, FAKE, None, FAKE, 1 << 40, None, None]
    args[at] = bad
    if at == 18 and not lib.lib().hcl_paged_attn_workspace_bytes(4, 8, 2, 128):
        pytest.skip("no workspace without a device")
    assert lib.lib().hcl_paged_attn_f32(*args) == code
    assert lib.lib().hcl_last_error()


@pytest.mark.parametrize("at,bad", [(0, None), (0, FAKE + 4), (1, None), (2, 0), (3, -1), (4, 63), (4, 2048), (5, 0), (7, None)])
def test_merge_refused(lib, at, bad):
    args = [FAKE, FAKE, 2, 8, 64, 4, None, FAKE, None, None]
    args[at] = bad
    assert lib.lib().hcl_lse_merge_f32(*args) == 1
    args[3] = 0
    assert at != 0 or lib.lib().hcl_lse_merge_f32(*args) == 0
