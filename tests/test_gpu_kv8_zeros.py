"""GPU: zeros of both signs beside other values keep their sign in fp8 pages, in every call that quantises."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle.kv_fp8 import quantize_rows

pytestmark = pytest.mark.gpu

HKV, TOKENS = 2, 16


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


def _rows():
    """bf16 rows [16, HKV, 128] whose largest values lie far below 2^-80, inside 2^-80..2^100 and above, with zeros of
    both signs and values that become codes of 0."""
    r = np.random.RandomState(1)
    scale = 2.0 ** np.array([-130, -100, -81, -80, -79, -40, -3, 0, 0, 1, 5, 60, 99, 100, 101, 126])
    x = torch.from_numpy(r.rand(TOKENS, HKV, 128) * scale[:, None, None])
    x = x * torch.from_numpy(r.choice([-1.0, 1.0], x.shape))
    at = torch.from_numpy(r.rand(*x.shape))
    x[at < 0.2] *= 0.0                                   # keeps the sign
    x[(at > 0.8)] *= 2.0 ** -14                          # codes of 0 of both signs
    return x.to(torch.bfloat16).cuda()


def _want(x):
    """Codes [HKV, 16, 128] and scales [HKV, 16] of rows [16, HKV, 128]."""
    codes, s = quantize_rows(x.float().cpu().numpy().transpose(1, 0, 2))
    return codes, s


def _read(block, which):
    """The codes [16, 128] and scales [16] that a block [4224] holds of K (0) or V (1)."""
    codes = np.empty((TOKENS, 128), np.uint8)
    for t in range(TOKENS):
        if which == 0:
            codes[t] = np.concatenate([block[128 * t + 16 * (c ^ (t & 7)):][:16] for c in range(8)])
        else:
            codes[t] = block[2048:4096].reshape(128, 16)[:, 4 * ((t & 7) >> 1) + ((t >> 3) << 1) + (t & 1)]
    return codes, block[4096 + 64 * which:][:64].view(np.float32)


def _same(page, k, v):
    """A page [HKV, 4224] against the rows it was made from."""
    page = page.cpu().numpy()
    for which, x in ((0, k), (1, v)):
        codes, scales = _want(x)
        assert (codes == 0x80).any() and (codes == 0).any()
        for h in range(HKV):
            got, s = _read(page[h], which)
            assert np.array_equal(s.astype(np.float64), scales[h])
            assert np.array_equal(got, codes[h]), (which, h, np.argwhere(got != codes[h])[:4].tolist())


def _pool():
    return torch.zeros(3, HKV, 4224, dtype=torch.uint8, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_pack_keeps_the_sign_of_zeros():
    from conditional_sparse_attention_b200 import oda
    k, v = _rows(), _rows().flip(0)
    kp, vp = (torch.zeros(3, HKV, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp[1], vp[1] = k.transpose(0, 1), v.transpose(0, 1)
    pool = _pool()
    oda.oda_kv8_pack(oda.kv_layer(kp, vp), oda.kv8_layer(pool), HKV)
    torch.cuda.synchronize()
    _same(pool[1], k, v)


@pytest.mark.parametrize("cuts", [[16], [5, 11], [1, 2, 13]])
def test_append_keeps_the_sign_of_zeros(cuts):
    """A page appended in one call, and in several that each fill a part."""
    from conditional_sparse_attention_b200 import oda
    k, v = _rows(), _rows().flip(0)
    ctx, pool, pos = oda.oda_create(oda.make_config(1, HKV, HKV, 1, 512)), _pool(), _i32([1])
    at = 0
    for n in cuts:
        oda.oda_append_fp8(ctx, [oda.kv8_layer(pool)], _i32([[1]]), pos, _i32([0, n]), None, k[None, at:at + n].contiguous(),
                           v[None, at:at + n].contiguous(), pos_next=pos)
        at += n
    assert oda.oda_get_error(ctx) == 0 and pos.item() == 17
    _same(pool[1], k, v)
    ctx.close()


def test_commit_keeps_the_sign_of_zeros():
    from conditional_sparse_attention_b200 import oda
    k, v = _rows(), _rows().flip(0)
    ctx, pool, pos = oda.oda_create(oda.make_config(1, HKV, HKV, 1, 512)), _pool(), _i32([1])
    h, h_prev = torch.zeros(1, 512, device="cuda"), torch.zeros(1, 512, device="cuda")
    for t in range(TOKENS):
        ks, vs = k[None, t:t + 1].contiguous(), v[None, t:t + 1].contiguous()
        oda.oda_commit_fp8(ctx, [oda.kv8_layer(pool)], _i32([[1]]), pos, _i32([0]), ks, vs, torch.ones_like(ks), torch.ones_like(vs),
                           h, h, h_prev)
    assert oda.oda_get_error(ctx) == 0 and pos.item() == 17
    _same(pool[1], k, v)
    ctx.close()
