"""Shared parts of the tests of prompt and tree attention, append and sampling."""
import numpy as np
import torch

BF16_HALF = 2.0 ** -8      # half a step of bf16, relative
# Error of one output element against fp64 (A = the softmax-weighted mean of |v|, o the exact output):
#   weights rounded to bf16 before the product with V:            at most 2^-8 A
#   fp32 scores: sums of 128 products, |q.k| / sqrt(128) off by at most 128 * 2^-24 * sum |q_i k_i| /
#     sqrt(128) (about 1e-4 at the tests' values), once in the weights and once in their sum; exp2 (a
#     quarter of them by a cubic, 7.5e-5) and the fp32 sums below 1e-4; together below 2^-11 = 4.9e-4 A
#   the result rounded to bf16:                                   at most 2^-8 of what is rounded,
#     2^-8 (|o| + the above)
W_SLACK = BF16_HALF + 2.0 ** -11


def attn_bound(o, a):
    """Elementwise bound on |got - o|."""
    before = W_SLACK * a
    return before + BF16_HALF * (np.abs(o) + before) + 1e-30


def check_attention(got, o, a, what=""):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - o) <= attn_bound(o, a))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(got - o))))


def normal(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def make_pages(lens, hkv, gen, mp=None, extra=0, fill=float("nan")):
    """Pools [n_pages, hkv, 16, 128] with random pages for caches of the given lengths (slots behind each
    sequence's end hold `fill`), the table, and the logical caches."""
    pages = [(n + 15) // 16 for n in lens]
    mp = mp or max(max(pages), 1)
    total = sum(pages) + 3 + extra
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(5)).to(torch.int32)
    pt = torch.full((len(lens), mp), -7, dtype=torch.int32)
    k = torch.full((total, hkv, 16, 128), fill, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, fill)
    caches, at = [], 0
    for b, n in enumerate(lens):
        pt[b, :pages[b]] = perm[at:at + pages[b]]
        ids = perm[at:at + pages[b]].long().cuda()
        at += pages[b]
        kc, vc = normal(gen, n, hkv, 128), normal(gen, n, hkv, 128)
        caches.append((kc, vc))
        for pool, c in ((k, kc), (v, vc)):
            pad = torch.full((pages[b] * 16, hkv, 128), fill, dtype=torch.bfloat16, device="cuda")
            pad[:n] = c
            pool[ids] = pad.view(pages[b], 16, hkv, 128).permute(0, 2, 1, 3)
    return k, v, pt.cuda(), caches


def cumulative(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
