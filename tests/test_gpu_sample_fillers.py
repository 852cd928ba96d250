"""GPU: rows whose masked logits are the type's lowest finite value, which counts as a logit like any other."""
import numpy as np
import pytest
import torch

from helpers import build_all

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
