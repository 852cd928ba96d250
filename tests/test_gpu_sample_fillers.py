"""GPU: rows whose masked logits are the type's lowest finite value, which counts as a logit like any other."""
import numpy as np
import pytest
import torch

from helpers import build_all
from oracle import serve

pytestmark = pytest.mark.gpu

FLOOR = np.finfo(np.float32).min


@pytest.fixture(scope="module")
def ctx():
    build_all()
    from conditional_sparse_attention_b200 import oda
    c = oda.oda_create(oda.make_config(1, 2, 1, 4, 512))
    yield c
    c.close()


def _sample(ctx, logits, u, **kw):
    """Tokens and probabilities, written over values that no row can give."""
    from conditional_sparse_attention_b200 import oda
    n = logits.shape[0]
    dev = {k: torch.as_tensor(np.broadcast_to(np.asarray(v, np.int32 if k == "top_k" else np.float32), (n,)).copy()).cuda()
           for k, v in kw.items()}
    token, prob = torch.full((n,), -9, dtype=torch.int32, device="cuda"), torch.full((n,), -9.0, device="cuda")
    oda.oda_sample(ctx, torch.from_numpy(np.asarray(logits, np.float32)).cuda(),
                   torch.from_numpy(np.asarray(u, np.float32)).cuda(), token, prob=prob, **dev)
    torch.cuda.synchronize()
    return token.cpu().numpy(), prob.cpu().numpy()


def _rows(vocab, top, few, spread, seed):
    """Rows of `vocab` with `few` ordinary logits, the largest `top`, among fillers."""
    r = np.random.RandomState(seed)
    n = len(top)
    x = np.full((n, vocab), FLOOR, np.float32)
    if spread:
        x = (-(2e38 + 1.4e38 * r.rand(n, vocab))).astype(np.float32)
    for i in range(n):
        at = r.choice(vocab, few, replace=False)
        x[i, at] = top[i] - r.rand(few) * 2
        x[i, at[0]] = top[i]
    return x, r.rand(n).astype(np.float32)


TOPS = np.float32([5, 9, 20, 40, 1.5, 3, 0.75, -2, -5])


@pytest.mark.parametrize("vocab", [193, 500, 1000, 1024])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("kw", [dict(top_k=50), dict(top_k=150, top_p=0.9)])
def test_every_row_gets_its_token(ctx, vocab, spread, kw):
    """Token and probability are written for every row: nothing of the call before stands in them."""
    x, u = _rows(vocab, TOPS, 3, spread, vocab)
    token, prob = _sample(ctx, x, u, **kw)
    assert np.all((token >= -1) & (token < vocab)), token
    assert np.all((prob >= 0) & (prob <= 1)), prob


def _check(ctx, x, u, **kw):
    """Tokens equal to the oracle's; probabilities within fp32's half step (2^-24), a weight's 1e-14 and half steps of
    2^-43 of the largest weight for each term."""
    token, prob = _sample(ctx, x, u, **kw)
    for i in range(x.shape[0]):
        t, p = serve.sample(x[i], u[i], **{k: np.broadcast_to(v, (x.shape[0],))[i] for k, v in kw.items()})
        assert token[i] == t, (i, token[i], t, kw)
        assert abs(prob[i] - p) <= p * (2.0 ** -24 + 1e-12) + x.shape[1] * 2.0 ** -43, (i, prob[i], p)


@pytest.mark.parametrize("vocab", [193, 500, 1000, 1024])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("few", [3, 100])
def test_cut_among_the_lowest_values(ctx, vocab, spread, few):
    """A top-k that reaches into the fillers, for maxima on both sides of a power of two's middle."""
    x, u = _rows(vocab, TOPS, few, spread, vocab + few)
    for k in (few + 1, few + 40, vocab - 1):
        for kw in (dict(), dict(top_p=np.float32(0.9)), dict(min_p=np.float32(0.05)), dict(temperature=np.float32(1e-3))):
            _check(ctx, x, u, top_k=k, **kw)


@pytest.mark.parametrize("vocab", [193, 700, 1024, 1500])
@pytest.mark.parametrize("spread", [False, True])
def test_fillers_that_weigh_something(ctx, vocab, spread):
    """Under a temperature of their size the lowest values have weights, and a cut by mass falls among them."""
    x, u = _rows(vocab, TOPS, 20, spread, vocab)
    for t in (np.float32(1e38), np.float32(np.inf)):
        for kw in (dict(top_p=np.float32(0.3)), dict(top_p=np.float32(0.83)), dict(top_k=vocab // 2),
                   dict(top_k=vocab // 2, top_p=np.float32(0.6))):
            _check(ctx, x, u, temperature=t, **kw)


@pytest.mark.parametrize("fillers", [200, 900, 1000])
def test_long_rows_with_some_fillers(ctx, fillers):
    """Long rows, masked but for a few ordinary values and a list's worth of fillers."""
    r = np.random.RandomState(fillers)
    x = np.full((len(TOPS), 40000), -np.inf, np.float32)
    for i, top in enumerate(TOPS):
        at = r.choice(40000, fillers + 4, replace=False)
        x[i, at] = FLOOR
        x[i, at[:4]] = top - np.float32([0, 0.5, 1, 2])
    u = r.rand(len(TOPS)).astype(np.float32)
    for kw in (dict(top_k=50), dict(top_k=190, top_p=np.float32(0.95)), dict(top_p=np.float32(0.99)),
               dict(top_k=150, temperature=np.float32(2e38))):
        _check(ctx, x, u, **kw)
