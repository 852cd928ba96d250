"""GPU: rows of K and V into bf16 and fp8 pages: exact data movement and quantisation."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle import serve

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


def _setup(B, L, hkv, mp, n_stage, D=512, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    total = B * mp + 2
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    pt = perm[:B * mp].view(B, mp).contiguous().cuda()
    ks = torch.randn(L, n_stage, hkv, 128, generator=gen, device="cuda").to(torch.bfloat16)
    vs = torch.randn(L, n_stage, hkv, 128, generator=gen, device="cuda").to(torch.bfloat16)
    h = torch.randn(n_stage, D, generator=gen, device="cuda")
    return pt, total, ks, vs, h


CASES = [
    # cu, pos, rows
    ([0, 5, 5, 22], [1, 9, 16], None),
    ([0, 1], [1], None),
    ([0, 300], [17], None),
    ([0, 3, 7, 8], [14, 100, 33], [5, 5, 0, 9, 3, 2, 1, 9]),
    ([0, 0, 0], [3, 4], None),
    ([2, 6, 40], [1, 30], None),
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("case", CASES)
def test_rows_reach_their_positions(case, fmt, hkv):
    from conditional_sparse_attention_b200 import oda
    cu, pos0, rows = case
    B, L, mp = len(pos0), 3, 24
    n_stage = max(10, cu[-1]) if rows is None else 10
    pt, total, ks, vs, h = _setup(B, L, hkv, mp, n_stage)
    ctx = oda.oda_create(oda.make_config(B, hkv, hkv, mp, 512))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pos, h_prev = i32(pos0), torch.full((B, 512), -3.0, device="cuda")
    kw = dict(h_stage=h, h_prev=h_prev, pos_next=pos)
    places = serve.append_places(pos0, cu, rows, mp, n_stage)
    table = pt.cpu().numpy()
    if fmt == "bf16":
        pools = [torch.full((2, total, hkv, 16, 128), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(L)]
        want = [p.clone() for p in pools]
        oda.oda_append(ctx, [oda.kv_layer(p[0], p[1]) for p in pools], pt, pos, i32(cu), None if rows is None else i32(rows),
                       ks, vs, **kw)
        for l in range(L):
            for b, src, lp, slot in places:
                want[l][0, table[b, lp], :, slot] = ks[l, src]
                want[l][1, table[b, lp], :, slot] = vs[l, src]
    else:
        # a bf16 cache holding the same rows, packed whole, gives the expected blocks
        pools = [torch.full((total, hkv, 4224), 0x11, dtype=torch.uint8, device="cuda") for _ in range(L)]
        want = [p.clone() for p in pools]
        oda.oda_append_fp8(ctx, [oda.kv8_layer(p) for p in pools], pt, pos, i32(cu), None if rows is None else i32(rows),
                           ks, vs, **kw)
        for l in range(L):
            k = torch.zeros(total, hkv, 16, 128, dtype=torch.bfloat16, device="cuda")
            v = torch.zeros_like(k)
            full = torch.zeros(total, hkv, 4224, dtype=torch.uint8, device="cuda")
            for b, src, lp, slot in places:
                k[table[b, lp], :, slot] = ks[l, src]
                v[table[b, lp], :, slot] = vs[l, src]
            oda.oda_kv8_pack(oda.kv_layer(k, v), oda.kv8_layer(full), hkv)
            for b, src, lp, slot in places:
                pg = int(table[b, lp])
                vslot = 4 * ((slot & 7) // 2) + 2 * (slot // 8) + slot % 2
                at = torch.cat([torch.arange(128 * slot, 128 * slot + 128), 2048 + 16 * torch.arange(128) + vslot,
                                4096 + 4 * slot + torch.arange(4), 4160 + 4 * slot + torch.arange(4)]).cuda()
                want[l][pg][:, at] = full[pg][:, at]
    torch.cuda.synchronize()
    assert oda.oda_get_error(ctx) == 0
    for l in range(L):
        assert torch.equal(pools[l], want[l])
    assert pos.tolist() == [p + cu[b + 1] - cu[b] for b, p in enumerate(pos0)]
    for b in range(B):
        if cu[b + 1] > cu[b]:
            last = cu[b + 1] - 1 if rows is None else rows[cu[b + 1] - 1]
            assert torch.equal(h_prev[b], h[last])
        else:
            assert torch.all(h_prev[b] == -3.0)
    ctx.close()


def test_special_values_in_fp8_rows():
    """All-zero rows, the largest bf16, denormals: the codes oda_kv8_pack writes."""
    from conditional_sparse_attention_b200 import oda
    pt, total, ks, vs, _ = _setup(1, 1, 2, 2, 20)
    ks[0, 0] = 0.0
    ks[0, 1] = 3.3895313892515355e38
    ks[0, 2] = 9.2e-41
    vs[0, 3, :, ::2] = 0.0
    vs[0, 4] = -0.0
    ctx = oda.oda_create(oda.make_config(1, 2, 2, 2, 512))
    pool = torch.zeros(total, 2, 4224, dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    oda.oda_append_fp8(ctx, [oda.kv8_layer(pool)], pt, i32([1]), i32([0, 20]), None, ks, vs)
    k = torch.zeros(total, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    for j in range(20):
        k[pt[0, j // 16], :, j % 16] = ks[0, j]
        v[pt[0, j // 16], :, j % 16] = vs[0, j]
    full = torch.zeros_like(pool)
    oda.oda_kv8_pack(oda.kv_layer(k, v), oda.kv8_layer(full), 2)
    torch.cuda.synchronize()
    ids = pt[0].long()
    assert torch.equal(pool[ids[0]], full[ids[0]])
    assert torch.equal(pool[ids[1]][:, :512], full[ids[1]][:, :512])
    ctx.close()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_bad_data_is_reported_and_not_written(fmt):
    from conditional_sparse_attention_b200 import oda
    B, L, hkv, mp = 2, 2, 2, 2
    pt, total, ks, vs, h = _setup(B, L, hkv, mp, 40)
    ctx = oda.oda_create(oda.make_config(B, hkv, hkv, mp, 512))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(cu, pos, rows, table=pt):
        if fmt == "bf16":
            pools = [torch.zeros(2, total, hkv, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(L)]
            layers, fn = [oda.kv_layer(p[0], p[1]) for p in pools], oda.oda_append
        else:
            pools = [torch.zeros(total, hkv, 4224, dtype=torch.uint8, device="cuda") for _ in range(L)]
            layers, fn = [oda.kv8_layer(p) for p in pools], oda.oda_append_fp8
        h_prev, nxt = torch.zeros(B, 512, device="cuda"), i32([0, 0])
        fn(ctx, layers, table, i32(pos), i32(cu), None if rows is None else i32(rows), ks, vs, h_stage=h, h_prev=h_prev,
           pos_next=nxt)
        e = oda.oda_get_error(ctx)
        oda.oda_clear_error(ctx)
        touched = sorted({int(x) for p in pools for x in
                          (p.view(torch.uint8).view(2, total, -1).any(-1).any(0) if fmt == "bf16" else
                           p.view(total, -1).any(-1)).nonzero().flatten()})
        return e, touched, nxt.tolist()

    both = lambda *lps: sorted(int(pt[b, lp]) for b, lp in lps)  # noqa: E731
    assert call([0, 2, 4], [1, 1], None)[:2] == (0, both((0, 0), (1, 0)))
    # capacity is 32 positions: rows behind it are skipped
    e, t, nxt = call([0, 5, 6], [31, 1], None)
    assert e == 0x2 and t == both((0, 1), (1, 0)) and nxt == [36, 2]
    e, t, nxt = call([0, 2, 3], [0, 1], None)
    assert e == 0x2 and t == both((1, 0)) and nxt == [0, 2]
    e, t, _ = call([0, 2, 3], [2 ** 31 - 3, 1], None)
    assert e == 0x2 and t == both((1, 0))
    e, t, _ = call([0, 2, 3], [1, 1], [40, -1, 3])
    assert e == 0x8 and t == both((1, 0))
    e, t, nxt = call([0, 2, 1], [1, 1], None)
    assert e == 0x8 and t == both((0, 0)) and nxt == [3, 1]
    bad = pt.clone()
    bad[0, 0], bad[1, 0] = -1, total
    e, t, _ = call([0, 2, 20], [1, 1], None, bad)
    assert e == 0x1 and t == both((1, 1))
    ctx.close()


def test_fp8_rows_of_every_scale():
    """Rows whose largest value is 2^-133 .. 2^127: codes and scales of IEEE divisions, bit for bit."""
    from conditional_sparse_attention_b200 import oda
    n = 261
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, n, 1, 128, generator=gen, device="cuda", dtype=torch.float64)
    x = x / x.abs().amax(-1, keepdim=True) * torch.exp2(torch.arange(n, device="cuda", dtype=torch.float64).view(1, n, 1, 1) - 133)
    x[:, :, :, ::3] *= torch.exp2(-torch.arange(43, device="cuda", dtype=torch.float64) / 3)     # down to codes of 0
    ks, vs = x.to(torch.bfloat16), x.flip(1).to(torch.bfloat16)
    mp = (n + 15) // 16
    ctx = oda.oda_create(oda.make_config(1, 1, 1, mp, 512))
    pool = torch.zeros(mp, 1, 4224, dtype=torch.uint8, device="cuda")
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    oda.oda_append_fp8(ctx, [oda.kv8_layer(pool)], torch.arange(mp, **dict(dtype=torch.int32, device="cuda")).view(1, mp),
                       i32([1]), i32([0, n]), None, ks, vs)
    assert oda.oda_get_error(ctx) == 0
    got = pool.cpu().numpy()
    for which, rows in ((0, ks), (1, vs)):
        f = rows[0, :, 0].float().cpu()
        amax = f.abs().amax(-1)
        s = torch.where(amax > 0, amax / torch.tensor(448.0), torch.tensor(1.0))
        codes = (f / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        for j in range(n):
            blk, t = got[j // 16, 0], j % 16
            assert blk[4096 + 64 * which + 4 * t:][:4].tobytes() == s[j].numpy().tobytes(), (which, j)
            if which == 0:
                c = np.concatenate([blk[128 * t + 16 * (k ^ (t & 7)):][:16] for k in range(8)])
            else:
                c = blk[2048:4096].reshape(128, 16)[:, 4 * ((t & 7) >> 1) + ((t >> 3) << 1) + (t & 1)]
            assert np.array_equal(c, codes[j]), (which, j)
    ctx.close()
