"""GPU: row and page counts whose products leave 64 bits are refused as out of range, before anything is launched."""
import ctypes

import pytest
import torch

from helpers import build_all

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


@pytest.mark.parametrize("hq,hkv", [(4, 2), (8, 8), (16, 2)])
def test_counts_beyond_64_bits(hq, hkv):
    from conditional_sparse_attention_b200 import _lib, oda
    L = _lib.load()
    ctx = oda.oda_create(oda.make_config(2, hq, hkv, 3, 512))
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = ctypes.c_void_p(buf.data_ptr())
    most = (2 ** 31 - 1) // hq
    for n in (most + 1, 2 ** 31, 2 ** 32 + 4, 2 ** 62, 2 ** 64 // hq, 2 ** 64 // hq + 4, 2 ** 63 - 1, -2 ** 63, -4):
        for call in (L.oda_attend_full_prompt, L.oda_attend_local_prompt):
            assert call(ctx.handle, 1, n, p, p, p, p, hq * 128, hkv * 128, p, None) == 1, n
            assert b"n_rows out of range" in L.oda_last_error()
    limit = (2 ** 31 - 1) // (16 * hkv)
    for pages in (limit, 2 ** 31, 2 ** 60 // hkv, 2 ** 60 // hkv + 6, 2 ** 63 - 1, -2 ** 63, -1, 0):
        kv = ctypes.byref(_lib.OdaKVLayer(buf.data_ptr(), buf.data_ptr(), pages))
        assert L.oda_attend_full_tree(ctx.handle, kv, p, p, None, 4, p, p, p, p, p, p, None) == 1, pages
        assert b"n_pages out of range" in L.oda_last_error()
    torch.cuda.synchronize()
    assert oda.oda_get_error(ctx) == 0
    ctx.close()
