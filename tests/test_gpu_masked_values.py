"""GPU: what a row does not see has weight 0: values of v near bf16's largest in masked places change nothing."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle import serve
from serve_helpers import check_attention, cumulative, f64, make_pages, normal

pytestmark = pytest.mark.gpu

BIG = 1e37
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 1)])
@pytest.mark.parametrize("n,first", [(40, 25), (130, 3), (300, 200), (700, 641)])
def test_later_tokens_of_a_prompt(hq, hkv, n, first):
    """Rows in front of token `first`, from which on v is huge."""
    from conditional_sparse_attention_b200 import oda
    gen = torch.Generator(device="cuda").manual_seed(n + hq)
    q, k, v = normal(gen, n, hq, 128, scale=1.5), normal(gen, n, hkv, 128), normal(gen, n, hkv, 128)
    v[first:] = BIG
    out = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    ctx = oda.oda_create(oda.make_config(1, hq, hkv, 4, 512, 4, 50))
    for call, window in ((oda.oda_attend_full_prompt, None), (oda.oda_attend_local_prompt, 50)):
        call(ctx, cumulative([n]), q, k, v, out)
        assert oda.oda_get_error(ctx) == 0
        o, a = serve.prompt(f64(q[:first]), f64(k[:first]), f64(v[:first]), 4, window)
        check_attention(f64(out[:first]), o, a, call.__name__)
    ctx.close()


@pytest.mark.parametrize("n", [200, 500])
@pytest.mark.parametrize("sinks", [0, 4, 16])
def test_tokens_the_window_has_left(n, sinks):
    """Local rows whose window has left tokens 20..79, whose v is huge and of one sign."""
    from conditional_sparse_attention_b200 import oda
    hq, hkv, window = 4, 2, 30
    gen = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = normal(gen, n, hq, 128), normal(gen, n, hkv, 128), normal(gen, n, hkv, 128)
    v[20:80] = -BIG
    out = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    ctx = oda.oda_create(oda.make_config(1, hq, hkv, 4, 512, sinks, window))
    oda.oda_attend_local_prompt(ctx, cumulative([n]), q, k, v, out)
    assert oda.oda_get_error(ctx) == 0
    o, a = serve.prompt(f64(q), f64(k), f64(v), sinks, window)
    rows = np.r_[0:20, 79 + window:n]
    check_attention(f64(out)[rows], o[rows], a[rows])
    ctx.close()


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2)])
@pytest.mark.parametrize("cached", [0, 5, 130, 1000])
def test_nodes_of_another_branch(hq, hkv, cached):
    """Two branches from the last cached token; the v of one of them is huge."""
    from conditional_sparse_attention_b200 import oda
    m = 33
    gen = torch.Generator(device="cuda").manual_seed(cached + hq)
    kp, vp, pt, caches = make_pages([cached], hkv, gen)
    parent = [-1] + [max(i - 2, -1) for i in range(1, m)]              # odd and even nodes
    q, kn, vn = normal(gen, m, hq, 128), normal(gen, m, hkv, 128), normal(gen, m, hkv, 128)
    vn[1::2] = BIG
    out = torch.zeros(m, hq, 128, dtype=torch.bfloat16, device="cuda")
    ctx = oda.oda_create(oda.make_config(1, hq, hkv, pt.shape[1], 512))
    oda.oda_attend_full_tree(ctx, oda.kv_layer(kp, vp), pt, torch.tensor([cached + 1], **I32), None, cumulative([m]),
                             torch.tensor(parent, **I32), q, kn, vn, out)
    assert oda.oda_get_error(ctx) == 0
    o, a = serve.tree(f64(q), f64(caches[0][0]), f64(caches[0][1]), f64(kn), f64(vn), parent)
    check_attention(f64(out)[::2], o[::2], a[::2])
    ctx.close()
