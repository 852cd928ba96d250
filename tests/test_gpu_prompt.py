"""GPU: causal attention over packed prompts (full and local set) against fp64."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle import serve
from serve_helpers import check_attention, cumulative, f64, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


def _ctx(hq, hkv, sinks=4, window=2048, batch=1):
    from conditional_sparse_attention_b200 import oda
    return oda.oda_create(oda.make_config(batch, hq, hkv, 4, 512, sinks, window))


def _run(ctx, local, *a, **kw):
    from conditional_sparse_attention_b200 import oda
    (oda.oda_attend_local_prompt if local else oda.oda_attend_full_prompt)(ctx, *a, **kw)


def _check(lens, hq, hkv, local=False, sinks=4, window=2048, behind=2, seed=1, qscale=1.5):
    from conditional_sparse_attention_b200 import oda
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(lens)
    T = n + behind
    q, k, v = normal(gen, T, hq, 128, scale=qscale), normal(gen, T, hkv, 128), normal(gen, T, hkv, 128)
    q[n:], k[n:], v[n:] = float("nan"), float("inf"), float("nan")   # behind the last sequence
    out = torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ctx = _ctx(hq, hkv, sinks, window)
    _run(ctx, local, cumulative(lens), q, k, v, out)
    torch.cuda.synchronize()
    assert oda.oda_get_error(ctx) == 0
    ctx.close()
    at = 0
    for i, m in enumerate(lens):
        if m:
            s = slice(at, at + m)
            o, a = serve.prompt(f64(q[s]), f64(k[s]), f64(v[s]), sinks, window if local else None)
            check_attention(f64(out[s]), o, a, (i, m))
        at += m
    assert torch.all(out[n:] == 7.0)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 2), (5, 1), (6, 1), (7, 1), (8, 1), (16, 8)])
def test_group_sizes(hq, hkv):
    _check([5, 0, 130, 1, 61], hq, hkv)


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255, 256, 257], [0, 0, 3, 0], [1] * 40,
                                  [600, 1, 300], [1300], [64, 65, 63, 512]])
def test_lengths(lens):
    _check(lens, 4, 2)


@pytest.mark.parametrize("sinks,window", [(4, 2048), (0, 1), (1, 1), (16, 128), (4, 100), (0, 300), (5, 129), (16, 700)])
@pytest.mark.parametrize("hq,hkv", [(2, 1), (6, 2)])
def test_local_set(sinks, window, hq, hkv):
    _check([3, 700, 130, 1100], hq, hkv, True, sinks, window)


def test_long_local_set_of_the_method():
    _check([2600, 2049, 2052], 2, 1, True)


def test_flat_and_peaked_weights():
    """Rows whose reference moves many times, and rows that never move it."""
    for scale in (0.0, 0.05, 8.0, 40.0):
        _check([700], 2, 1, qscale=scale, seed=3)


def test_growing_scores_move_the_reference():
    """Scores that grow by far more than the lazy step from tile to tile."""
    from conditional_sparse_attention_b200 import oda
    n = 1000
    k = torch.zeros(n, 1, 128)
    k[:, 0, 0] = torch.arange(n) / 8.0
    q = torch.zeros(n, 1, 128)
    q[:, 0, 0] = 16.0
    v = torch.randn(n, 1, 128, generator=torch.Generator().manual_seed(2))
    q, k, v = (x.to(torch.bfloat16).cuda() for x in (q, k, v))
    out = torch.zeros(n, 1, 128, dtype=torch.bfloat16, device="cuda")
    ctx = _ctx(1, 1)
    _run(ctx, False, cumulative([n]), q, k, v, out)
    torch.cuda.synchronize()
    assert oda.oda_get_error(ctx) == 0
    o, a = serve.prompt(f64(q), f64(k), f64(v))
    check_attention(f64(out), o, a)
    ctx.close()


def test_strided_rows_of_one_projection():
    """q, k and v as columns of one [n, (Hq + 2 Hkv) 128] projection output."""
    from conditional_sparse_attention_b200 import oda
    lens, hq, hkv = [300, 17, 129], 8, 2
    n = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(8)
    qkv = normal(gen, n, (hq + 2 * hkv) * 128)
    q = qkv[:, :hq * 128].view(n, hq, 128)
    k = qkv[:, hq * 128:(hq + hkv) * 128].view(n, hkv, 128)
    v = qkv[:, (hq + hkv) * 128:].view(n, hkv, 128)
    a, b = (torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx = _ctx(hq, hkv)
    _run(ctx, False, cumulative(lens), q, k, v, a)
    _run(ctx, False, cumulative(lens), q.contiguous(), k.contiguous(), v.contiguous(), b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    o, m = serve.prompt(f64(q[300:317]), f64(k[300:317]), f64(v[300:317]))
    check_attention(f64(a[300:317]), o, m)
    ctx.close()


def test_non_finite_sequence_does_not_reach_others():
    lens, hq, hkv = [130, 61, 200], 4, 2
    gen = torch.Generator(device="cuda").manual_seed(9)
    n = sum(lens)
    q, k, v = normal(gen, n, hq, 128), normal(gen, n, hkv, 128), normal(gen, n, hkv, 128)
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[130:191] = bad
    out = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    ctx = _ctx(hq, hkv)
    for local in (False, True):
        _run(ctx, local, cumulative(lens), q, k, v, out)
        torch.cuda.synchronize()
        for s in (slice(0, 130), slice(191, 391)):
            o, a = serve.prompt(f64(q[s]), f64(k[s]), f64(v[s]))
            check_attention(f64(out[s]), o, a)
    ctx.close()


def test_many_sequences():
    r = np.random.RandomState(0)
    _check(r.randint(0, 40, 256).tolist(), 2, 1)


def test_long_prompt_sampled_rows():
    """A 33000-token prompt: rows near the start, the middle and the end against fp64."""
    from conditional_sparse_attention_b200 import oda
    n, hq, hkv = 33000, 4, 1
    gen = torch.Generator(device="cuda").manual_seed(11)
    q, k, v = normal(gen, n, hq, 128, scale=2.0), normal(gen, n, hkv, 128), normal(gen, n, hkv, 128)
    out = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    ctx = _ctx(hq, hkv)
    for local in (False, True):
        _run(ctx, local, cumulative([n]), q, k, v, out)
        torch.cuda.synchronize()
        assert oda.oda_get_error(ctx) == 0
        for t in (0, 2047, 2048, 2060, 16383, 16384, 32767, 32999):
            j = torch.arange(t + 1, device="cuda")
            if local:
                j = j[(j < 4) | (j > t - 2048)]
            x = (k[j, 0].double() @ q[t].double().T).T / 128 ** 0.5
            w = torch.softmax(x, -1)
            vd = v[j, 0].double()
            check_attention(f64(out[t]), f64(w @ vd), f64(w @ vd.abs()), (local, t))
    ctx.close()


def test_equal_calls_give_equal_bits_and_capture_replays():
    from conditional_sparse_attention_b200 import oda
    lens, hq, hkv = [900, 33, 400], 8, 2
    n = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(12)
    q, k, v = normal(gen, n, hq, 128), normal(gen, n, hkv, 128), normal(gen, n, hkv, 128)
    cu = cumulative(lens)
    out = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    ctx = _ctx(hq, hkv)
    _run(ctx, False, cu, q, k, v, out)
    torch.cuda.synchronize()
    first = out.clone()
    s = torch.cuda.Stream()
    oda.oda_graph_begin(s)
    _run(ctx, False, cu, q, k, v, out, stream=s)
    g = oda.oda_graph_end(s)
    out.zero_()
    q2 = normal(gen, n, hq, 128)
    keep = q.clone()
    torch.cuda.synchronize()
    g.launch(s)
    s.synchronize()
    assert torch.equal(out, first)
    q.copy_(q2)
    torch.cuda.synchronize()
    g.launch(s)
    s.synchronize()
    again = out.clone()
    _run(ctx, False, cu, q2, k, v, out)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and not torch.equal(out, first)
    q.copy_(keep)
    g.close()
    ctx.close()


def test_bad_bounds_are_reported_and_skipped():
    from conditional_sparse_attention_b200 import oda
    gen = torch.Generator(device="cuda").manual_seed(13)
    n = 100
    q, k, v = normal(gen, n, 2, 128), normal(gen, n, 1, 128), normal(gen, n, 1, 128)
    ctx = _ctx(2, 1)
    for cu in ([0, 40, 30, 100], [-1, 40, 100], [0, 40, 101], [0, 40, 2 ** 31 - 1]):
        out = torch.full((n, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        _run(ctx, False, torch.tensor(cu, dtype=torch.int32, device="cuda"), q, k, v, out)
        assert oda.oda_get_error(ctx) == 0x8
        oda.oda_clear_error(ctx)
        for a, e in zip(cu, cu[1:]):
            if 0 <= a < e <= n and not (cu == [0, 40, 30, 100] and a == 30):
                o, m = serve.prompt(f64(q[a:e]), f64(k[a:e]), f64(v[a:e]))
                got = f64(out[a:e])
                keep = 30 if cu == [0, 40, 30, 100] else e - a   # rows 30..39 belong to two sequences there
                check_attention(got[:keep], o[:keep], m[:keep])
    ctx.close()


@pytest.mark.parametrize("j", [3, 70, 135, 263])
@pytest.mark.parametrize("local", [False, True])
def test_rows_that_see_a_nan_key_are_nan(j, local):
    """A NaN key: every row that sees it is NaN, the others are as they were.  An infinite one: NaN where
    its score is +inf; as if it were not there where the score is -inf; NaN where every score is."""
    n, hq, hkv, window = 400, 4, 2, 100
    gen = torch.Generator(device="cuda").manual_seed(j)
    q, k, v = normal(gen, n, hq, 128), normal(gen, n, hkv, 128), normal(gen, n, hkv, 128)
    q[:, 0::2, 9], q[:, 1::2, 9] = 1.0, -1.0
    ctx = _ctx(hq, hkv, 2, window)
    t = np.arange(n)
    sees = (t >= j) & ((t < j + window) | (not local))
    for bad in (float("nan"), float("inf")):
        k1 = k.clone()
        k1[j, :, 9] = bad
        out = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
        _run(ctx, local, cumulative([n]), q, k1, v, out)
        torch.cuda.synchronize()
        got, ok = f64(out), (t[None, :] <= t[:, None])
        if local:
            ok &= (t[None, :] < 2) | (t[None, :] > t[:, None] - window)
        ok[:, j] = False
        for h in range(hq):
            odd = h % 2 == 1 and bad > 0             # score -inf
            o, a = serve._rows(f64(q[:, h]), f64(k[:, h // 2]), f64(v[:, h // 2]), ok)
            rows = np.ones(n, bool) if odd else ~sees
            check_attention(got[rows, h], o[rows], a[rows], (h, bad))
            assert odd or np.isnan(got[sees, h]).all()
    k1 = k.clone()
    k1[:, :, 9] = float("inf")                       # every score of an odd head is -inf, of an even one +inf
    _run(ctx, local, cumulative([n]), q, k1, v, out)
    assert torch.isnan(out).all()
    ctx.close()
