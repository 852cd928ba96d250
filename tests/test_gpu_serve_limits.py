"""GPU: prompts, trees, append and sampling at offsets past 32 bits, beside rows of other calls, and at the
sizes where sampling changes its way."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle import serve
from serve_helpers import check_attention, cumulative, f64, make_pages, normal

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


def test_prompt_rows_past_32_bits():
    """q, k and v as rows 2^27 elements apart: the last rows lie more than 2^31 elements in."""
    from conditional_sparse_attention_b200 import oda
    n, hq, hkv, stride = 21, 4, 2, 1 << 27
    gen = torch.Generator(device="cuda").manual_seed(1)
    buf = torch.full(((n - 1) * stride + 4096,), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((n, hq, 128), (stride, 128, 1), 0)
    k = buf.as_strided((n, hkv, 128), (stride, 128, 1), 1024)
    v = buf.as_strided((n, hkv, 128), (stride, 128, 1), 2048)
    for x in (q, k, v):
        x.copy_(normal(gen, *x.shape))
    out = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    ctx = oda.oda_create(oda.make_config(1, hq, hkv, 4, 512))
    oda.oda_attend_full_prompt(ctx, cumulative([n]), q, k, v, out)
    assert oda.oda_get_error(ctx) == 0
    o, a = serve.prompt(f64(q), f64(k), f64(v))
    check_attention(f64(out), o, a)
    ctx.close()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_pages_past_32_bits(fmt):
    """Pages at the end of a pool of more than 2^32 bytes (bf16: 2^31 elements): appended, then read by a tree."""
    from conditional_sparse_attention_b200 import oda
    hq, hkv, n, mp = 4, 2, 40, 4
    gen = torch.Generator(device="cuda").manual_seed(2)
    ks, vs = normal(gen, 1, n, hkv, 128), normal(gen, 1, n, hkv, 128)
    ctx = oda.oda_create(oda.make_config(1, hq, hkv, mp, 512))
    pos = torch.ones(1, **I32)
    if fmt == "fp8":
        total = (1 << 32) // (hkv * 4224) + 100
        pool = torch.zeros(total, hkv, 4224, dtype=torch.uint8, device="cuda")
        layer, call = oda.kv8_layer(pool), oda.oda_append_fp8
    else:
        total = (1 << 31) // (hkv * 2048) + 100
        kp, vp = (torch.zeros(total, hkv, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        layer, call = oda.kv_layer(kp, vp), oda.oda_append
    pt = torch.tensor([[total - 1, 3, total - 2, 0]], **I32)
    call(ctx, [layer], pt, pos, cumulative([n]), None, ks, vs, pos_next=pos)
    assert oda.oda_get_error(ctx) == 0 and pos.item() == n + 1
    if fmt == "fp8":
        small = torch.zeros(4, hkv, 4224, dtype=torch.uint8, device="cuda")
        call(ctx, [oda.kv8_layer(small)], torch.tensor([[1, 3, 2, 0]], **I32), torch.ones(1, **I32), cumulative([n]), None, ks, vs)
        assert torch.equal(pool[total - 1], small[1]) and torch.equal(pool[3], small[3]) and torch.equal(pool[total - 2], small[2])
        assert not pool[4:total - 2].any()
    else:
        for i, page in enumerate((total - 1, 3, total - 2)):
            m = min(16, n - 16 * i)
            assert torch.equal(kp[page, :, :m], ks[0, 16 * i:16 * i + m].transpose(0, 1))
            assert torch.equal(vp[page, :, :m], vs[0, 16 * i:16 * i + m].transpose(0, 1))
        q, kn, vn = normal(gen, 5, hq, 128), normal(gen, 5, hkv, 128), normal(gen, 5, hkv, 128)
        out = torch.zeros(5, hq, 128, dtype=torch.bfloat16, device="cuda")
        par = [-1, 0, 0, 2, 3]
        oda.oda_attend_full_tree(ctx, layer, pt, pos, None, cumulative([5]), torch.tensor(par, **I32), q, kn, vn, out)
        assert oda.oda_get_error(ctx) == 0
        o, a = serve.tree(f64(q), f64(ks[0]), f64(vs[0]), f64(kn), f64(vn), par)
        check_attention(f64(out), o, a)
    ctx.close()


def test_sampled_rows_past_32_bits():
    from conditional_sparse_attention_b200 import oda
    n, vocab, stride = 4, 3001, (1 << 30) + 5
    gen = torch.Generator(device="cuda").manual_seed(3)
    buf = torch.empty((n - 1) * stride + vocab, device="cuda")
    logits = buf.as_strided((n, vocab), (stride, 1))
    logits.copy_(torch.randn(n, vocab, generator=gen, device="cuda") * 3)
    u = torch.rand(n, generator=gen, device="cuda")
    token = torch.zeros(n, **I32)
    ctx = oda.oda_create(oda.make_config(1, 2, 1, 4, 512))
    oda.oda_sample(ctx, logits, u, token, top_p=torch.full((n,), 0.9, device="cuda"))
    assert oda.oda_get_error(ctx) == 0
    l, uu = logits.cpu().numpy(), u.cpu().numpy()
    assert token.tolist() == [serve.sample(l[r], uu[r], top_p=np.float32(0.9))[0] for r in range(n)]
    ctx.close()


@pytest.mark.parametrize("nodes", [[3, 17], [1, 64], [33, 5]])
def test_tree_rows_behind_the_last_sequence(nodes):
    """Rows of q, k_new, v_new and out behind the last node hold NaN and stay as they were."""
    from conditional_sparse_attention_b200 import oda
    hq, hkv, lens = 4, 2, [70, 300]
    gen = torch.Generator(device="cuda").manual_seed(4)
    kp, vp, pt, caches = make_pages(lens, hkv, gen)
    N, T = sum(nodes), sum(nodes) + 7
    q, kn, vn = normal(gen, T, hq, 128), normal(gen, T, hkv, 128), normal(gen, T, hkv, 128)
    q[N:], kn[N:], vn[N:] = float("nan"), float("inf"), float("nan")
    par = [[-1] + list(range(n - 1)) for n in nodes]
    parent = torch.tensor(par[0] + par[1] + [99] * 7, **I32)
    out = torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ctx = oda.oda_create(oda.make_config(2, hq, hkv, pt.shape[1], 512))
    pos = torch.tensor([n + 1 for n in lens], **I32)
    oda.oda_attend_full_tree(ctx, oda.kv_layer(kp, vp), pt, pos, None, cumulative(nodes), parent, q, kn, vn, out)
    assert oda.oda_get_error(ctx) == 0
    at = 0
    for b, n in enumerate(nodes):
        s = slice(at, at + n)
        at += n
        o, a = serve.tree(f64(q[s]), f64(caches[b][0]), f64(caches[b][1]), f64(kn[s]), f64(vn[s]), par[b])
        check_attention(f64(out[s]), o, a, b)
    assert torch.all(out[N:] == 7.0)
    ctx.close()


@pytest.mark.parametrize("vocab", [190, 191, 192, 193, 194, 1022, 1023, 1024, 1025, 1026])
@pytest.mark.parametrize("equal", [False, True])
def test_sampling_at_the_lists_sizes(vocab, equal):
    """Rows as long as the lists that are compared in pairs and cut by bits, with many equal values too."""
    from conditional_sparse_attention_b200 import oda
    r = np.random.RandomState(vocab)
    n = 48
    l = (r.randn(n, vocab) * 2).astype(np.float32)
    if equal:
        l = np.round(l * 2) / 2
    l[r.rand(n, vocab) < 0.05] = -np.inf
    u, k = r.rand(n).astype(np.float32), r.randint(0, vocab + 3, n).astype(np.int32)
    p, m = (0.5 + 0.6 * r.rand(n)).astype(np.float32), np.where(r.rand(n) < 0.5, 0.0, 0.02 * r.rand(n)).astype(np.float32)
    cuda = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    ctx = oda.oda_create(oda.make_config(1, 2, 1, 4, 512))
    for kw in (dict(top_k=k), dict(top_p=p), dict(top_k=k, top_p=p, min_p=m)):
        token, prob = torch.zeros(n, **I32), torch.zeros(n, device="cuda")
        oda.oda_sample(ctx, cuda(l), cuda(u), token, prob=prob, **{a: cuda(x) for a, x in kw.items()})
        assert oda.oda_get_error(ctx) == 0
        for i in range(n):
            t, w = serve.sample(l[i], u[i], **{a: x[i] for a, x in kw.items()})
            assert token[i].item() == t, (i, kw.keys(), token[i].item(), t)
            assert abs(prob[i].item() - w) <= w * (2.0 ** -24 + 1e-12) + vocab * 2.0 ** -43
    ctx.close()
