"""GPU: tokens from logits with temperature, top-k, top-p and min-p against fp64."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle import serve

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


@pytest.fixture(scope="module")
def ctx():
    build_all()
    from conditional_sparse_attention_b200 import oda
    c = oda.oda_create(oda.make_config(1, 2, 1, 4, 512))
    yield c
    c.close()


def _run(ctx, logits, u, stream=None, **kw):
    from conditional_sparse_attention_b200 import oda
    n = logits.shape[0]
    dt = {"top_k": torch.int32}
    dev = {k: torch.as_tensor(np.asarray(v), dtype=dt.get(k, torch.float32)).cuda().expand(n).contiguous()
           for k, v in kw.items()}
    token = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((n,), -9.0, device="cuda")
    oda.oda_sample(ctx, logits, torch.as_tensor(u, dtype=torch.float32).cuda(), token, prob=prob, stream=stream, **dev)
    torch.cuda.synchronize()
    return token.cpu().numpy(), prob.cpu().numpy()


def _check(ctx, logits, u, **kw):
    """Tokens equal, probabilities within fp32's half step (2^-24) and the weights' 2^-43 steps."""
    logits = np.asarray(logits, np.float32)
    u = np.asarray(u, np.float32)
    n = logits.shape[0]
    token, prob = _run(ctx, torch.from_numpy(logits).cuda(), u, **kw)
    one = lambda k, r, d: np.broadcast_to(np.float32(kw[k]) if k in kw else d, (n,))[r] if k in kw else d  # noqa: E731
    for r in range(n):
        t, p = serve.sample(logits[r], u[r], one("temperature", r, 1.0), int(one("top_k", r, 0)), one("top_p", r, 1.0),
                            one("min_p", r, 0.0))
        assert token[r] == t, (r, token[r], t, kw)
        # a weight is off by half a step of 2^-43 and 1e-14 of itself, the sum by that for each term
        assert abs(prob[r] - p) <= p * (2.0 ** -24 + 1e-12) + logits.shape[1] * 2.0 ** -43, (r, prob[r], p)


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=40), dict(top_p=0.9), dict(top_p=0.05), dict(min_p=0.05),
            dict(temperature=1.3, top_k=200, top_p=0.95, min_p=0.01), dict(temperature=0.0), dict(top_p=0.999, temperature=2.5),
            dict(top_k=3000, top_p=0.5)]


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 1000, 5117, 5118, 32000, 50257, 151936, 262144])
@pytest.mark.parametrize("kw", SETTINGS)
def test_settings_and_sizes(ctx, vocab, kw):
    r = np.random.RandomState(vocab % 1000 + 1)
    n = 5
    _check(ctx, r.randn(n, vocab) * 3, r.rand(n), **kw)


def test_each_row_its_own_settings(ctx):
    r = np.random.RandomState(2)
    n = 64
    _check(ctx, r.randn(n, 20000) * 2.5, r.rand(n), temperature=np.where(r.rand(n) < 0.1, 0, 0.4 + r.rand(n)),
           top_k=(r.rand(n) * 300).astype(np.int32) * (r.rand(n) < 0.6), top_p=np.where(r.rand(n) < 0.5, r.rand(n), 1.0),
           min_p=np.where(r.rand(n) < 0.5, 0.1 * r.rand(n), 0.0))


@pytest.mark.parametrize("vocab", [7, 1024, 1025, 40000])
def test_ties_go_to_the_lowest_index(ctx, vocab):
    """All logits equal, and a few levels of equal ones: the cut and the draw go by index."""
    n = 6
    u = np.array([0, 0.1, 0.4999, 0.5, 0.9, 0.99999994], np.float32)
    flat = np.zeros((n, vocab), np.float32)
    for kw in (dict(), dict(top_k=5), dict(top_p=0.3), dict(top_k=vocab // 2 + 1, top_p=0.7), dict(top_k=2000),
               dict(min_p=1.0), dict(temperature=0.0)):
        _check(ctx, flat, u, **kw)
    r = np.random.RandomState(3)
    steps = r.randint(0, 4, (n, vocab)).astype(np.float32)
    for kw in (dict(), dict(top_k=vocab // 3 + 1), dict(top_p=0.8), dict(top_k=vocab // 2 + 1, top_p=0.9, temperature=0.5),
               dict(min_p=0.2), dict(top_k=3)):
        _check(ctx, steps, u, **kw)


@pytest.mark.parametrize("scale,shift", [(1e-6, 0.0), (1e-3, 5.0), (1e-4, -1e4), (300.0, 0.0), (1e30, 0.0), (1e-38, 0.0)])
def test_narrow_and_wide_ranges(ctx, scale, shift):
    """Values that share a bin of the histogram, and values that leave its range."""
    r = np.random.RandomState(4)
    x = (r.randn(4, 30000) * scale + shift).astype(np.float32)
    for kw in (dict(), dict(top_k=7), dict(top_k=5000), dict(top_p=0.6), dict(top_k=1500, top_p=0.4), dict(temperature=40.0, top_p=0.7),
               dict(temperature=1e-3, top_p=0.7)):
        _check(ctx, x, r.rand(4), **kw)


def test_masked_and_non_finite_logits(ctx):
    r = np.random.RandomState(5)
    x = (r.randn(8, 3001) * 2).astype(np.float32)
    x[0, r.rand(3001) < 0.9] = -np.inf
    x[1, r.rand(3001) < 0.5] = np.nan
    x[2] = -np.inf
    x[3] = np.nan
    x[4, [17, 1900, 2999]] = np.inf
    x[5, :] = np.finfo(np.float32).min
    x[5, 100] = 1.0
    x[6] = -np.inf
    x[6, 2500] = -3e38
    x[7] = np.finfo(np.float32).min
    u = r.rand(8)
    for kw in (dict(), dict(top_k=2), dict(top_k=2500), dict(top_p=0.5), dict(min_p=0.3), dict(temperature=0.0), dict(top_k=50, top_p=0.9)):
        _check(ctx, x, u, **kw)


def test_settings_out_of_range(ctx):
    r = np.random.RandomState(6)
    x = (r.randn(3, 500) * 2).astype(np.float32)
    u = np.array([0.3, 0.6, 0.9], np.float32)
    for kw in (dict(top_k=-3), dict(top_k=500), dict(top_k=10 ** 9), dict(top_p=0.0), dict(top_p=-1.0), dict(top_p=7.0),
               dict(min_p=-1.0), dict(min_p=3.0), dict(temperature=-2.0), dict(temperature=np.inf), dict(temperature=np.inf, top_k=4),
               dict(temperature=np.inf, top_p=0.5), dict(temperature=1e-40)):
        _check(ctx, x, u, **kw)
    nan = float("nan")
    base = _run(ctx, torch.from_numpy(x).cuda(), u)
    for kw in (dict(top_p=nan), dict(min_p=nan)):
        assert np.array_equal(_run(ctx, torch.from_numpy(x).cuda(), u, **kw)[0], base[0])
    assert np.array_equal(_run(ctx, torch.from_numpy(x).cuda(), u, temperature=nan)[0], x.argmax(1))
    for bad, same in ((nan, 0.0), (-1.0, 0.0), (5.0, 0.99999994)):
        a = _run(ctx, torch.from_numpy(x).cuda(), np.full(3, bad, np.float32))
        b = _run(ctx, torch.from_numpy(x).cuda(), np.full(3, same, np.float32))
        if same == 0.0:
            assert np.array_equal(a[0], b[0])
        else:
            assert np.all(a[0] >= b[0])      # at u = 1 the last value with any mass
    assert np.all(_run(ctx, torch.from_numpy(x).cuda(), np.zeros(3, np.float32))[0] == 0)


def test_rows_with_a_stride_and_odd_alignment(ctx):
    r = np.random.RandomState(7)
    buf = torch.from_numpy((r.randn(5, 10007) * 2).astype(np.float32)).cuda()
    u = r.rand(5).astype(np.float32)
    for off in range(5):
        view = buf[:, off:off + 10001]
        got = _run(ctx, view, u, top_p=0.9, top_k=100)
        want = _run(ctx, view.contiguous(), u, top_p=0.9, top_k=100)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        for i in range(5):
            assert got[0][i] == serve.sample(view[i].cpu().numpy(), u[i], top_p=np.float32(0.9), top_k=100)[0]


def test_equal_calls_give_equal_bits(ctx):
    r = np.random.RandomState(8)
    x = torch.from_numpy((r.randn(40, 60000)).astype(np.float32)).cuda()
    u = r.rand(40).astype(np.float32)
    a = _run(ctx, x, u, top_p=0.97)
    for _ in range(3):
        b = _run(ctx, x, u, top_p=0.97)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_frequencies_follow_the_distribution(ctx):
    """40000 draws over 6 tokens: each count within 6 standard deviations."""
    p = np.array([0.4, 0.25, 0.2, 0.1, 0.04, 0.01])
    n = 40000
    x = torch.from_numpy(np.log(p).astype(np.float32)).cuda().expand(n, 6).contiguous()
    u = np.random.RandomState(9).rand(n).astype(np.float32)
    t, _ = _run(ctx, x, u)
    for i in range(6):
        assert abs((t == i).sum() - n * p[i]) < 6 * np.sqrt(n * p[i] * (1 - p[i]))


@pytest.mark.parametrize("vocab", [50, 5000, 60000])
@pytest.mark.parametrize("kw", [dict(top_p=0.8), dict(top_k=20), dict(min_p=0.01), dict(top_k=30, top_p=0.7)])
def test_logits_whose_differences_leave_fp32(ctx, vocab, kw):
    """Logits of both signs near fp32's largest, under a temperature of their size."""
    r = np.random.RandomState(vocab)
    logits = ((r.rand(6, vocab) * 2 - 1) * 3.3e38).astype(np.float32)
    logits[1] = np.where(r.rand(vocab) < 0.5, np.float32(3.4e38), np.float32(-3.4e38))
    _check(ctx, logits, r.rand(6), temperature=1e38, **kw)


@pytest.mark.parametrize("temperature", [0.3, 0.05, 0.003, 1e-4])
@pytest.mark.parametrize("kw", [dict(top_k=50), dict(top_k=900, top_p=0.9999), dict(top_k=5000), dict(top_k=59990)])
def test_low_temperatures_with_top_k(ctx, temperature, kw):
    """A top-k that reaches far behind the maximum."""
    r = np.random.RandomState(5)
    _check(ctx, r.randn(8, 60000) * 2.5, r.rand(8), temperature=temperature, **kw)
