"""GPU: where top-p ends in long rows, whose far weights are summed in fp32."""
import numpy as np
import pytest
import torch

from helpers import build_all

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    build_all()
    from conditional_sparse_attention_b200 import oda
    c = oda.oda_create(oda.make_config(1, 2, 1, 4, 512))
    yield c
    c.close()


def _row(shape, n, t, r):
    """A row in falling order: ordinary logits, or one value with as much mass as all the others at one distance."""
    if shape == "normal":
        x = r.randn(n) * 2.5
    else:
        x = -(np.log(n) + r.uniform(-1, 1)) * t - 1e-3 * r.rand(n)
        x[0] = 0.0
    return np.sort(x.astype(np.float32))[::-1].copy()


@pytest.mark.parametrize("shape", ["normal", "far"])
@pytest.mark.parametrize("n", [20000, 151936, 262144])
def test_the_end_lies_where_the_mass_is(ctx, shape, n):
    """The last value kept, by the draw at the end of the mass, against fp64 sums.  An end may lie off by what the fp32
    masses beyond a distance of 3 are: for each, 4.2 d + 4 roundings of 2^-24 and half the number of a lane's terms
    (n / 8 CTAs / 512 threads); in the running mass and, times top_p, in the whole."""
    from conditional_sparse_attention_b200 import oda
    r = np.random.RandomState(n % 1000)
    for _ in range(12):
        t = np.float32(r.uniform(0.4, 1.6))
        x = _row(shape, n, float(t), r)
        d = (float(x[0]) - x.astype(np.float64)) / float(t)
        w = np.exp(-d)
        sums = np.cumsum(w)
        rows = 48
        k = np.searchsorted(sums, r.uniform(0.3, 0.99, rows) * sums[-1])
        p = (sums[k] / sums[-1] + r.randint(-40, 41, rows) * 2.0 ** -25).clip(0, 1 - 2.0 ** -24).astype(np.float32)
        cuda = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        token = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
        oda.oda_sample(ctx, cuda(x).expand(rows, n).contiguous(), cuda(np.full(rows, 1 - 2.0 ** -24, np.float32)), token,
                       temperature=cuda(np.full(rows, t)), top_p=cuda(p))
        far = (w * (4.2 * d + 4 + n / 8192))[d >= 3].sum() * 2.0 ** -24 / sums[-1]
        for i, e in enumerate(token.cpu().numpy()):
            # u is half a step of 2^-24 below 1: the draw's value may lie that far in front of the last one kept
            first = sums[e - 1] / sums[-1] if e > 0 else 0.0
            last = np.searchsorted(sums, sums[e] / (1 - 2.0 ** -23))
            assert first - 2 * far <= p[i] <= sums[min(last + 1, n - 1)] / sums[-1] + 2 * far, (i, e, p[i], far)
