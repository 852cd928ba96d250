"""GPU: a tree of drafted tokens over the paged cache against fp64."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle import serve
from serve_helpers import check_attention, cumulative, f64, make_pages, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


def _parents(r, n, kind):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] * n
    return [int(r.randint(-1, i)) if i else -1 for i in range(n)]


def _case(lens, nodes, hq, hkv, kind="random", flags=None, seed=1, mp=None):
    from conditional_sparse_attention_b200 import oda
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed)
    B, N = len(lens), sum(nodes)
    kp, vp, pt, caches = make_pages(lens, hkv, gen, mp)
    q = normal(gen, N + 1, hq, 128, scale=1.5)[:N]
    kn, vn = normal(gen, N, hkv, 128), normal(gen, N, hkv, 128)
    parents = [_parents(r, n, kind) for n in nodes]
    par = torch.tensor([x for p in parents for x in p], dtype=torch.int32, device="cuda")
    out = torch.full((N, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ctx = oda.oda_create(oda.make_config(B, hq, hkv, pt.shape[1], 512))
    pos = torch.tensor([n + 1 for n in lens], dtype=torch.int32, device="cuda")
    flag = None if flags is None else torch.tensor(flags, dtype=torch.int32, device="cuda")
    args = (ctx, oda.kv_layer(kp, vp), pt, pos, flag, cumulative(nodes), par, q, kn, vn)
    oda.oda_attend_full_tree(*args, out)
    torch.cuda.synchronize()
    assert oda.oda_get_error(ctx) == 0
    at = 0
    for b, n in enumerate(nodes):
        s = slice(at, at + n)
        at += n
        if flags is not None and not flags[b]:
            assert torch.all(out[s] == 7.0)
        elif n:
            kc, vc = caches[b]
            o, a = serve.tree(f64(q[s]), f64(kc), f64(vc), f64(kn[s]), f64(vn[s]), parents[b])
            check_attention(f64(out[s]), o, a, (b, lens[b], n))
    again = torch.full_like(out, 7.0)
    oda.oda_attend_full_tree(*args, again)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    ctx.close()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 2), (5, 1), (6, 1), (7, 1), (8, 1), (16, 8)])
def test_group_sizes(hq, hkv):
    _case([300, 0, 1, 129], [64, 3, 1, 33], hq, hkv)


@pytest.mark.parametrize("lens", [[0], [1], [15], [16], [17], [127], [128], [129], [1000], [2500, 3, 640]])
@pytest.mark.parametrize("nodes", [1, 16, 64])
def test_lengths(lens, nodes):
    _case(lens, [nodes] * len(lens), 4, 2)


@pytest.mark.parametrize("kind", ["chain", "star", "random"])
def test_shapes_of_trees(kind):
    _case([500, 77, 1300], [64, 40, 7], 8, 2, kind)


def test_ragged_batch_with_empty_and_unflagged_sequences():
    _case([40, 900, 0, 256, 2000], [0, 5, 64, 17, 1], 4, 1, flags=[1, 1, 0, 1, 1])
    _case([40, 900, 0, 256, 2000], [3, 5, 64, 17, 1], 4, 1, flags=[0, 0, 0, 0, 0])


def test_many_sequences_share_ctas():
    r = np.random.RandomState(3)
    _case(r.randint(0, 300, 200).tolist(), r.randint(0, 9, 200).tolist(), 2, 2)


def test_one_long_sequence_over_all_ctas():
    _case([40000], [64], 4, 1)
    _case([40000], [6], 2, 1, "chain")


def test_one_node_is_the_decode_call():
    """A tree of one node reads the same positions as oda_attend_full_if."""
    from conditional_sparse_attention_b200 import oda
    lens, hq, hkv = [700, 33], 8, 2
    gen = torch.Generator(device="cuda").manual_seed(5)
    kp, vp, pt, _ = make_pages(lens, hkv, gen, fill=0.0)
    q, kn, vn = normal(gen, 2, hq, 128), normal(gen, 2, hkv, 128), normal(gen, 2, hkv, 128)
    ctx = oda.oda_create(oda.make_config(2, hq, hkv, pt.shape[1], 512))
    pt = pt.clamp(min=0)
    pos = torch.tensor([n + 1 for n in lens], dtype=torch.int32, device="cuda")
    a = torch.zeros(2, hq, 128, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(2, hq, 128, device="cuda")
    oda.oda_attend_full_tree(ctx, oda.kv_layer(kp, vp), pt, pos, None, cumulative([1, 1]),
                             torch.tensor([-1, -1], dtype=torch.int32, device="cuda"), q, kn, vn, a)
    oda.oda_attend_full_if(ctx, oda.kv_layer(kp, vp), pt, pos, torch.ones(2, dtype=torch.int32, device="cuda"), q, kn,
                           vn, b)
    torch.cuda.synchronize()
    # the decode call is within 2e-3 relative l2 of exact, this one within 2^-7 of it elementwise
    assert (a.float() - b).norm() <= (2e-3 + 2.0 ** -7) * b.norm()
    ctx.close()


def test_capture_replays_with_new_positions():
    from conditional_sparse_attention_b200 import oda
    lens, nodes, hq, hkv = [500, 130], [9, 20], 4, 1
    gen = torch.Generator(device="cuda").manual_seed(6)
    kp, vp, pt, caches = make_pages(lens, hkv, gen)
    N = sum(nodes)
    q, kn, vn = normal(gen, N, hq, 128), normal(gen, N, hkv, 128), normal(gen, N, hkv, 128)
    par = torch.tensor([-1] * N, dtype=torch.int32, device="cuda")
    out = torch.zeros(N, hq, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([301, 131], dtype=torch.int32, device="cuda")
    ctx = oda.oda_create(oda.make_config(2, hq, hkv, pt.shape[1], 512))
    cu = cumulative(nodes)                # the captured call keeps reading it
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    oda.oda_graph_begin(s)
    oda.oda_attend_full_tree(ctx, oda.kv_layer(kp, vp), pt, pos, None, cu, par, q, kn, vn, out, stream=s)
    g = oda.oda_graph_end(s)
    for n in (300, 500, 1):
        pos[0] = n + 1
        torch.cuda.synchronize()
        g.launch(s)
        s.synchronize()
        o, a = serve.tree(f64(q[:9]), f64(caches[0][0][:n]), f64(caches[0][1][:n]), f64(kn[:9]), f64(vn[:9]), [-1] * 9)
        check_attention(f64(out[:9]), o, a, n)
    assert oda.oda_get_error(ctx) == 0
    g.close()
    ctx.close()


def test_bad_data_is_reported():
    from conditional_sparse_attention_b200 import oda
    lens, nodes, hq, hkv = [100, 200], [4, 5], 2, 1
    gen = torch.Generator(device="cuda").manual_seed(7)
    kp, vp, pt, caches = make_pages(lens, hkv, gen)
    N = sum(nodes)
    q, kn, vn = normal(gen, N, hq, 128), normal(gen, N, hkv, 128), normal(gen, N, hkv, 128)
    good = [-1, 0, 1, 2, -1, 0, 0, 1, 1]
    ctx = oda.oda_create(oda.make_config(2, hq, hkv, pt.shape[1], 512))

    def call(pt=pt, pos=(101, 201), cu=(0, 4, 9), par=good):
        out = torch.full((N, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        oda.oda_attend_full_tree(ctx, oda.kv_layer(kp, vp), pt, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                                 None, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                 torch.tensor(par, dtype=torch.int32, device="cuda"), q, kn, vn, out)
        e = oda.oda_get_error(ctx)
        oda.oda_clear_error(ctx)
        return e, out

    def second_is_right(out):
        o, a = serve.tree(f64(q[4:]), f64(caches[1][0]), f64(caches[1][1]), f64(kn[4:]), f64(vn[4:]), good[4:])
        check_attention(f64(out[4:]), o, a)

    e, out = call()
    assert e == 0
    second_is_right(out)
    bad = pt.clone()
    bad[0, 2] = 10 ** 6
    e, out = call(pt=bad)
    assert e == 0x1
    second_is_right(out)
    for p in (0, -5, 16 * pt.shape[1] + 2, 2 ** 31 - 1):
        e, out = call(pos=(p, 201))
        assert e == 0x2 and torch.all(out[:4] == 7.0)
        second_is_right(out)
    e, out = call(par=[-1, 1, 5, -2] + good[4:])       # children of -1, all of them
    assert e == 0x8
    second_is_right(out)
    o, a = serve.tree(f64(q[:4]), f64(caches[0][0]), f64(caches[0][1]), f64(kn[:4]), f64(vn[:4]), [-1] * 4)
    check_attention(f64(out[:4]), o, a)
    e, out = call(cu=(0, 4, 10))
    assert e == 0x8 and torch.all(out[4:] == 7.0)
    e, out = call(cu=(4, 0, 9))
    assert e == 0x8 and torch.all(out[0:0] == 7.0)
    ctx.close()


@pytest.mark.parametrize("place", [6, 1000, 3000])
def test_nodes_that_see_a_nan_key_are_nan(place):
    """A NaN key in the cache reaches every node of its sequence, one of a node itself and its descendants;
    other sequences none.  Infinite keys: as in the formula."""
    from conditional_sparse_attention_b200 import oda
    hq, hkv, lens, nodes = 4, 2, [3100, 50], [24, 5]
    gen = torch.Generator(device="cuda").manual_seed(place)
    r = np.random.RandomState(place)
    kp, vp, pt, caches = make_pages(lens, hkv, gen)
    N = sum(nodes)
    q, kn, vn = normal(gen, N, hq, 128), normal(gen, N, hkv, 128), normal(gen, N, hkv, 128)
    parents = [_parents(r, n, "random") for n in nodes]
    par = torch.tensor([x for p in parents for x in p], dtype=torch.int32, device="cuda")
    ctx = oda.oda_create(oda.make_config(2, hq, hkv, pt.shape[1], 512))
    pos = torch.tensor([n + 1 for n in lens], dtype=torch.int32, device="cuda")

    def run(kp, kn):
        out = torch.zeros(N, hq, 128, dtype=torch.bfloat16, device="cuda")
        oda.oda_attend_full_tree(ctx, oda.kv_layer(kp, vp), pt, pos, None, cumulative(nodes), par, q, kn, vn, out)
        torch.cuda.synchronize()
        return f64(out)
    want = [serve.tree(f64(q[s]), *map(f64, caches[b]), f64(kn[s]), f64(vn[s]), parents[b])
            for b, s in enumerate((slice(0, 24), slice(24, 29)))]
    bad = kp.clone()
    bad[pt[0, place // 16].item(), :, place % 16, 7] = float("nan")
    got = run(bad, kn)
    assert np.isnan(got[:24]).all()
    check_attention(got[24:], *want[1])
    bad = kn.clone()
    bad[6, :, 50] = float("nan")
    got = run(kp, bad)
    sees = serve.lineage(parents[0])[:, 6]
    assert np.isnan(got[:24][sees]).all()
    check_attention(got[:24][~sees], want[0][0][~sees], want[0][1][~sees])
    check_attention(got[24:], *want[1])
    # every score of sequence 0 is -inf (cache and nodes), and a row of +inf
    q[:, :, 9] = -1.0
    kb, nb = kp.clone(), kn.clone()
    kb[pt[0, :194].long(), :, :, 9] = float("inf")
    nb[:24, :, 9] = float("inf")
    assert np.isnan(run(kb, nb)[:24]).all()
    q[:, :, 9] = 1.0
    assert np.isnan(run(kb, nb)[:24]).all()
    ctx.close()
