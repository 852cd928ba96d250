"""GPU: logits and temperatures down to fp32's subnormals, whose distances in units of the temperature are ordinary."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle import serve

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    build_all()
    from conditional_sparse_attention_b200 import oda
    c = oda.oda_create(oda.make_config(1, 2, 1, 4, 512))
    yield c
    c.close()


def _check(ctx, x, u, temperature, **kw):
    """Tokens equal to the oracle's; probabilities within fp32's half step, a weight's 1e-14 and half steps of 2^-43 of
    the largest weight for each term."""
    from conditional_sparse_attention_b200 import oda
    n, vocab = x.shape
    kw = dict(kw, temperature=np.float32(temperature))
    dev = {k: torch.full((n,), v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in kw.items()}
    dev["temperature"] = torch.from_numpy(np.full(n, kw["temperature"])).cuda()
    token, prob = torch.full((n,), -9, dtype=torch.int32, device="cuda"), torch.full((n,), -9.0, device="cuda")
    oda.oda_sample(ctx, torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda(), token, prob=prob, **dev)
    assert oda.oda_get_error(ctx) == 0
    for i in range(n):
        t, p = serve.sample(x[i], u[i], **kw)
        assert token[i].item() == t, (i, token[i].item(), t, temperature, kw)
        assert abs(prob[i].item() - p) <= p * (2.0 ** -24 + 1e-12) + vocab * 2.0 ** -43, (i, prob[i].item(), p)


@pytest.mark.parametrize("log2t", [-149, -145, -140, -133, -127, -126, -120, -101, -100, -99])
@pytest.mark.parametrize("vocab", [60, 700, 9000])
def test_temperatures_of_the_logits_size(ctx, log2t, vocab):
    """Differences of a few temperatures (top-k and top-p keep few, far and near), with and without min-p."""
    r = np.random.RandomState(vocab - log2t)
    t = 2.0 ** log2t
    x = (r.randn(6, vocab) * 2.5 * t).astype(np.float32)
    x[3] -= np.float32(40 * t)
    x[4, ::3] = -np.inf
    x[5, 1:] -= np.float32(2.0 ** 20 * t)                # far behind one value
    u = r.rand(6).astype(np.float32)
    for kw in (dict(), dict(min_p=np.float32(0.1)), dict(top_k=20, min_p=np.float32(1e-3)), dict(top_p=np.float32(0.7)),
               dict(top_k=1500, top_p=np.float32(0.8), min_p=np.float32(0.02))):
        _check(ctx, x, u, t, **kw)


@pytest.mark.parametrize("top", [3e38, 2.0 ** 68, 2.0 ** 60, 1e18, 0.0, -1e18, -2.0 ** 60, -2.0 ** 68, -3e38])
@pytest.mark.parametrize("log2t", [-149, -128, -101, -100, -60])
def test_large_logits_under_small_temperatures(ctx, top, log2t):
    """Logits of any size under such a temperature: all but the largest are infinitely far."""
    r = np.random.RandomState(7)
    for vocab in (50, 1000, 5000):
        x = (r.randn(4, vocab) * 10.0 ** r.uniform(0, 38, (4, vocab))).clip(-3.4e38, 3.4e38).astype(np.float32)
        x = np.minimum(x, np.float32(top))
        x[0, ::7] = np.float32(top)
        x[1, 3] = np.float32(top)
        u = r.rand(4).astype(np.float32)
        for kw in (dict(), dict(top_k=30), dict(top_p=np.float32(0.6)), dict(min_p=np.float32(0.5)), dict(top_k=200, top_p=np.float32(0.9))):
            _check(ctx, x, u, 2.0 ** log2t, **kw)
