"""GPU: a request's way through the calls together: prompt, append, drafted tree, sampling, append of the
accepted path, decode step; eagerly and as one replayed graph.  And the calls' refusals."""
import ctypes

import numpy as np
import pytest
import torch

from helpers import attn_close, build_all
from oracle import serve
from serve_helpers import check_attention, cumulative, f64, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


I32 = dict(dtype=torch.int32, device="cuda")


class Run:
    """Two layers, three sequences: what a server holds between the calls."""

    def __init__(self, seed=1, hq=8, hkv=2, L=2, vocab=5000):
        from conditional_sparse_attention_b200 import oda
        self.oda, self.hq, self.hkv, self.L, self.vocab = oda, hq, hkv, L, vocab
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.nodes = [37, 300, 129], [5, 9, 1]
        self.parents = [[-1, 0, 0, 1, 3], [-1, 0, 1, 1, 0, 4, 4, -1, 7], [-1]]
        B, n, N = 3, sum(self.lens), sum(self.nodes)
        self.mp = 24
        self.ctx = oda.oda_create(oda.make_config(B, hq, hkv, self.mp, hq * 128))
        self.pt = torch.randperm(B * self.mp, generator=torch.Generator().manual_seed(seed)).to(torch.int32).view(B, self.mp).cuda()
        shape = (L, B * self.mp, hkv, 16, 128)
        self.kp = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vp = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.layers = [oda.kv_layer(self.kp[i], self.vp[i]) for i in range(L)]
        self.pos = torch.ones(B, **I32)
        self.pos0 = torch.ones(B, **I32)
        self.h_prev = torch.zeros(B, hq * 128, device="cuda")
        self.cu, self.cun = cumulative(self.lens), cumulative(self.nodes)
        self.q, self.k, self.v = normal(gen, L, n, hq, 128), normal(gen, L, n, hkv, 128), normal(gen, L, n, hkv, 128)
        self.h = torch.randn(n, hq * 128, generator=gen, device="cuda")
        self.qt, self.kt, self.vt = normal(gen, L, N, hq, 128), normal(gen, L, N, hkv, 128), normal(gen, L, N, hkv, 128)
        self.ht = torch.randn(N, hq * 128, generator=gen, device="cuda")
        self.parent = torch.tensor([p for ps in self.parents for p in ps], **I32)
        self.o = torch.zeros(L, n, hq, 128, dtype=torch.bfloat16, device="cuda")
        self.ot = torch.zeros(L, N, hq, 128, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.randn(N, vocab, generator=gen, device="cuda") * 3
        self.u = torch.rand(N, generator=gen, device="cuda")
        self.top_p = torch.full((N,), 0.9, device="cuda")
        self.token = torch.zeros(N, **I32)
        # the accepted paths, as a server finds them by comparing tokens: root, a child, its child
        self.accepted = [[0, 1, 3], [5, 6], [14]]
        self.rows = torch.tensor([r for x in self.accepted for r in x], **I32)
        self.cua = cumulative([len(x) for x in self.accepted])
        self.qd, self.kd, self.vd = normal(gen, B, hq, 128), normal(gen, B, hkv, 128), normal(gen, B, hkv, 128)
        self.od = torch.zeros(B, hq, 128, device="cuda")
        self.ones = torch.ones(B, **I32)

    def issue(self, s):
        oda = self.oda
        with torch.cuda.stream(s):
            self.pos.copy_(self.pos0)
        for i in range(self.L):                # layer by layer, as the prompt's hidden states come
            call = oda.oda_attend_full_prompt if i else oda.oda_attend_local_prompt
            call(self.ctx, self.cu, self.q[i], self.k[i], self.v[i], self.o[i], stream=s)
            last = i + 1 == self.L
            oda.oda_append(self.ctx, self.layers[i:i + 1], self.pt, self.pos, self.cu, None, self.k[i:i + 1], self.v[i:i + 1],
                           h_stage=self.h if last else None, h_prev=self.h_prev if last else None,
                           pos_next=self.pos if last else None, stream=s)
        for i in range(self.L):
            oda.oda_attend_full_tree(self.ctx, self.layers[i], self.pt, self.pos, None, self.cun, self.parent, self.qt[i],
                                     self.kt[i], self.vt[i], self.ot[i], stream=s)
        oda.oda_sample(self.ctx, self.logits, self.u, self.token, top_p=self.top_p, stream=s)
        oda.oda_append(self.ctx, self.layers, self.pt, self.pos, self.cua, self.rows, self.kt, self.vt, h_stage=self.ht,
                       h_prev=self.h_prev, pos_next=self.pos, stream=s)
        oda.oda_attend_full_if(self.ctx, self.layers[0], self.pt, self.pos, self.ones, self.qd, self.kd, self.vd, self.od,
                               stream=s)

    def check(self):
        assert self.oda.oda_get_error(self.ctx) == 0
        at = ar = 0
        for b, n in enumerate(self.lens):
            s, t = slice(at, at + n), slice(ar, ar + self.nodes[b])
            at, ar = at + n, ar + self.nodes[b]
            for i in range(self.L):
                k, v = f64(self.k[i, s]), f64(self.v[i, s])
                o, a = serve.prompt(f64(self.q[i, s]), k, v, 4, None if i else 2048)
                check_attention(f64(self.o[i, s]), o, a, ("prompt", b, i))
                o, a = serve.tree(f64(self.qt[i, t]), k, v, f64(self.kt[i, t]), f64(self.vt[i, t]), self.parents[b])
                check_attention(f64(self.ot[i, t]), o, a, ("tree", b, i))
            acc = self.accepted[b]
            kc = torch.cat([self.k[0, s], self.kt[0, acc], self.kd[b:b + 1]])
            vc = torch.cat([self.v[0, s], self.vt[0, acc], self.vd[b:b + 1]])
            w = np.stack([serve._rows(f64(self.qd[b, h:h + 1]), f64(kc[:, h // 4]), f64(vc[:, h // 4]),
                                      np.ones((1, kc.shape[0]), bool))[0][0] for h in range(self.hq)])
            ok, ma, rel = attn_close(self.od[b].cpu().numpy(), w)
            assert ok, ("decode", b, ma, rel)
            assert torch.equal(self.h_prev[b], self.ht[acc[-1]])
        assert self.pos.tolist() == [1 + n + len(a) for n, a in zip(self.lens, self.accepted)]
        logits, u = self.logits.cpu().numpy(), self.u.cpu().numpy()
        for r, t in enumerate(self.token.tolist()):
            assert t == serve.sample(logits[r], u[r], top_p=np.float32(0.9))[0]


def test_calls_together_eager_and_replayed():
    from conditional_sparse_attention_b200 import oda
    run = Run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    run.issue(s)
    s.synchronize()
    run.check()
    first = [x.clone() for x in (run.o, run.ot, run.token, run.od)]
    oda.oda_graph_begin(s)
    run.issue(s)
    g = oda.oda_graph_end(s)
    for x in (run.o, run.ot, run.token, run.od, run.h_prev):
        x.zero_()
    run.kp.fill_(float("nan"))
    run.vp.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(2):
        g.launch(s)
        s.synchronize()
        run.check()
    # the prompt, tree and sampling calls repeat bit for bit (the decode call's split may not)
    for x, y in zip((run.o, run.ot, run.token), first):
        assert torch.equal(x, y)
    g.close()
    run.ctx.close()


def test_two_contexts_on_two_streams():
    """Each context has its own scratch: two at once give what each gives alone."""
    a, b = Run(seed=3), Run(seed=4)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.issue(sa)
        b.issue(sb)
    torch.cuda.synchronize()
    a.check()
    b.check()
    a.ctx.close()
    b.ctx.close()


def test_refusals():
    from conditional_sparse_attention_b200 import _lib, oda
    L = _lib.load()
    ctx = oda.oda_create(oda.make_config(2, 4, 2, 3, 512))
    h = ctx.handle
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = ctypes.c_void_p(buf.data_ptr())
    odd = ctypes.c_void_p(buf.data_ptr() + 2)
    N = None
    kv = ctypes.byref(_lib.OdaKVLayer(buf.data_ptr(), buf.data_ptr(), 1))
    prompt = lambda n_seqs=1, n=4, cu=p, q=p, k=p, v=p, qs=512, ks=256, out=p: L.oda_attend_full_prompt(  # noqa: E731
        h, n_seqs, n, cu, q, k, v, qs, ks, out, N)
    for kw in (dict(n_seqs=0), dict(n_seqs=257), dict(n=0), dict(n=-1), dict(n=1 << 31), dict(cu=N), dict(q=N), dict(k=N),
               dict(v=N), dict(out=N), dict(qs=504), dict(ks=128), dict(qs=516), dict(ks=260), dict(qs=1 << 40), dict(q=odd),
               dict(k=odd), dict(v=odd), dict(out=odd)):
        assert prompt(**kw) == 1, kw
    tree = lambda kvl=kv, pt=p, pos=p, n=4, cu=p, par=p, q=p, k=p, v=p, out=p: L.oda_attend_full_tree(  # noqa: E731
        h, kvl, pt, pos, N, n, cu, par, q, k, v, out, N)
    for kw in (dict(kvl=N), dict(pt=N), dict(pos=N), dict(n=0), dict(n=129), dict(cu=N), dict(par=N), dict(q=N), dict(k=N),
               dict(v=N), dict(out=N), dict(q=odd), dict(out=odd), dict(k=odd), dict(v=odd),
               dict(kvl=ctypes.byref(_lib.OdaKVLayer(buf.data_ptr(), buf.data_ptr(), 0))),
               dict(kvl=ctypes.byref(_lib.OdaKVLayer(buf.data_ptr() + 8, buf.data_ptr(), 1)))):
        assert tree(**kw) == 1, kw
    app = lambda kvl=kv, nl=1, pt=p, pos=p, n=2, ns=2, cu=p, rows=N, k=p, v=p, hs=N, hp=N: L.oda_append(  # noqa: E731
        h, kvl, nl, pt, pos, n, ns, cu, rows, k, v, hs, hp, N, N)
    for kw in (dict(kvl=N), dict(nl=0), dict(nl=65), dict(pt=N), dict(pos=N), dict(n=-1), dict(ns=0), dict(n=3), dict(cu=N),
               dict(k=N), dict(v=N), dict(k=odd), dict(v=odd), dict(hs=p), dict(hp=p), dict(hs=odd, hp=p),
               dict(kvl=ctypes.byref(_lib.OdaKVLayer(buf.data_ptr(), 0, 1)))):
        assert app(**kw) == 1, kw
    samp = lambda n=2, vocab=8, st=8, lg=p, u=p, tok=p, t=N: L.oda_sample(h, n, vocab, st, lg, t, N, N, N, u, tok, N, N)  # noqa: E731
    for kw in (dict(n=0), dict(n=65536), dict(vocab=0), dict(vocab=262145, st=262145), dict(st=7), dict(lg=N), dict(u=N),
               dict(tok=N), dict(lg=odd), dict(t=odd)):
        assert samp(**kw) == 1, kw
    torch.cuda.synchronize()
    assert oda.oda_get_error(ctx) == 0
    # the binding names the tensor that is wrong
    c2 = oda.oda_create(oda.make_config(2, 4, 2, 3, 512))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, **I32)  # noqa: E731
    with pytest.raises(ValueError, match="q:"):
        oda.oda_attend_full_prompt(c2, i32(2), bf(5, 2, 128), bf(5, 2, 128), bf(5, 2, 128), bf(5, 4, 128))
    with pytest.raises(ValueError, match="number of rows"):
        oda.oda_attend_full_prompt(c2, i32(2), bf(5, 4, 128), bf(6, 2, 128), bf(6, 2, 128), bf(5, 4, 128))
    with pytest.raises(ValueError, match="out"):
        oda.oda_attend_full_prompt(c2, i32(2), bf(5, 4, 128), bf(5, 2, 128), bf(5, 2, 128), bf(5, 4, 128).float())
    with pytest.raises(ValueError, match="parent"):
        oda.oda_attend_full_tree(c2, oda.kv_layer(bf(1, 2, 16, 128), bf(1, 2, 16, 128)), i32(2, 3), i32(2), None, i32(3), i32(4),
                                 bf(5, 4, 128), bf(5, 2, 128), bf(5, 2, 128), bf(5, 4, 128))
    with pytest.raises(ValueError, match="v_stage"):
        oda.oda_append(c2, [oda.kv_layer(bf(1, 2, 16, 128), bf(1, 2, 16, 128))], i32(2, 3), i32(2), i32(3), None,
                       bf(1, 5, 2, 128), bf(1, 4, 2, 128))
    with pytest.raises(ValueError, match="top_k"):
        oda.oda_sample(c2, torch.zeros(2, 9, device="cuda"), torch.zeros(2, device="cuda"), i32(2), top_k=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="contiguous rows"):
        oda.oda_sample(c2, torch.zeros(9, 2, device="cuda").T, torch.zeros(2, device="cuda"), i32(2))
    ctx.close()
    c2.close()


def test_empty_calls():
    """No rows at all: every sequence empty."""
    from conditional_sparse_attention_b200 import oda
    ctx = oda.oda_create(oda.make_config(2, 4, 2, 3, 512))
    bf = lambda *s: torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    z = torch.zeros(3, **I32)
    out = bf(5, 4, 128)
    oda.oda_attend_full_prompt(ctx, z, bf(5, 4, 128), bf(5, 2, 128), bf(5, 2, 128), out)
    oda.oda_attend_local_prompt(ctx, z, bf(5, 4, 128), bf(5, 2, 128), bf(5, 2, 128), out)
    kp = bf(6, 2, 16, 128)
    pos = torch.tensor([5, 9], **I32)
    oda.oda_attend_full_tree(ctx, oda.kv_layer(kp, kp.clone()), torch.zeros(2, 3, **I32), pos, None, z, torch.zeros(5, **I32),
                             bf(5, 4, 128), bf(5, 2, 128), bf(5, 2, 128), out)
    nxt = torch.zeros(2, **I32)
    oda.oda_append(ctx, [oda.kv_layer(kp, kp.clone())], torch.zeros(2, 3, **I32), pos, z, torch.zeros(0, **I32), bf(1, 4, 2, 128),
                   bf(1, 4, 2, 128), pos_next=nxt)
    torch.cuda.synchronize()
    assert oda.oda_get_error(ctx) == 0
    assert torch.all(out == 3.0) and torch.all(kp == 3.0) and nxt.tolist() == [5, 9]
    ctx.close()


def test_one_row_of_any_stride():
    """A single row has no stride: a view whose row stride fits no rule is taken."""
    from conditional_sparse_attention_b200 import oda
    ctx = oda.oda_create(oda.make_config(1, 2, 1, 3, 512))
    gen = torch.Generator(device="cuda").manual_seed(8)
    buf = normal(gen, 4 * 1001)
    q = buf.as_strided((1, 2, 128), (1001, 128, 1))
    k = buf.as_strided((1, 1, 128), (3, 128, 1), 1024)
    v = buf.as_strided((1, 1, 128), (1001, 128, 1), 2048)
    out = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    oda.oda_attend_full_prompt(ctx, cumulative([1]), q, k, v, out)
    logits = torch.randn(90, generator=gen, device="cuda").as_strided((1, 50), (3, 1), 7)
    token = torch.zeros(1, **I32)
    oda.oda_sample(ctx, logits, torch.zeros(1, device="cuda"), token, temperature=torch.zeros(1, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out, v.expand(1, 2, 128)) and token.item() == logits.argmax().item()
    ctx.close()
