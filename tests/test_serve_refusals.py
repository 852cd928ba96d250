"""CPU: the binding of prompts, trees, append and sampling refuses wrong tensors before it calls the
library, and the library refuses a missing context; the oracle's pins."""
import ctypes
import types

import numpy as np
import pytest
import torch

from conditional_sparse_attention_b200 import _lib, build, oda
from oracle import attention as OA
from oracle import serve
from oracle.sets import full_set, local_set


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_library_refuses_a_missing_context(lib):
    p = ctypes.c_void_p(4096)
    assert lib.oda_attend_full_prompt(None, 1, 1, p, p, p, p, 128, 128, p, None) == 1
    assert lib.oda_attend_local_prompt(None, 1, 1, p, p, p, p, 128, 128, p, None) == 1
    assert lib.oda_attend_full_tree(None, None, p, p, None, 1, p, p, p, p, p, p, None) == 1
    assert lib.oda_append(None, None, 1, p, p, 1, 1, p, None, p, p, None, None, None, None) == 1
    assert lib.oda_append_fp8(None, None, 1, p, p, 1, 1, p, None, p, p, None, None, None, None) == 1
    assert lib.oda_sample(None, 1, 10, 10, p, None, None, None, None, p, p, None, None) == 1
    assert b"ctx is NULL" in lib.oda_last_error()


def _ctx(batch=2, hq=4, hkv=2):
    return types.SimpleNamespace(cfg=oda.make_config(batch, hq, hkv, 3, 512), handle=None)


def test_binding_wants_cuda_tensors_of_the_right_kind():
    c = _ctx()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        oda.oda_attend_full_prompt(c, i32(2), bf(5, 4, 128), bf(5, 2, 128), bf(5, 2, 128), bf(5, 4, 128))
    with pytest.raises(ValueError, match="CUDA"):
        oda.oda_attend_full_tree(c, None, i32(2, 3), i32(2), None, i32(3), i32(5), bf(5, 4, 128), bf(5, 2, 128),
                                 bf(5, 2, 128), bf(5, 4, 128))
    with pytest.raises(ValueError, match="CUDA"):
        oda.oda_append(c, [], i32(2, 3), i32(2), i32(3), None, bf(1, 5, 2, 128), bf(1, 5, 2, 128))
    with pytest.raises(ValueError, match="CUDA"):
        oda.oda_sample(c, torch.zeros(2, 10), torch.zeros(2), i32(2))


def test_oracle_prompt_rows_are_decode_steps():
    """Row p of a prompt is the decode step at t = p + 1 over the same keys and values, both sets."""
    r = np.random.RandomState(0)
    n, hq, hkv = 40, 4, 2
    q, k, v = r.randn(n, hq, 128), r.randn(n, hkv, 128), r.randn(n, hkv, 128)
    for window in (None, 7):
        o, a = serve.prompt(q, k, v, 3, window)
        for p in (0, 1, 5, 20, 39):
            t = p + 1
            S = full_set(t) if window is None else local_set(t, 3, window)
            assert np.allclose(o[p], OA.attend(q[p], k[:t], v[:t], S), rtol=0, atol=1e-12)
            assert np.allclose(a[p], OA.attend(q[p], k[:t], np.abs(v[:t]), S), rtol=0, atol=1e-12)


def test_oracle_chain_of_nodes_is_a_prompt_continued():
    r = np.random.RandomState(1)
    n, m, hq, hkv = 9, 5, 2, 1
    q, k, v = r.randn(n + m, hq, 128), r.randn(n + m, hkv, 128), r.randn(n + m, hkv, 128)
    o, _ = serve.tree(q[n:], k[:n], v[:n], k[n:], v[n:], [-1, 0, 1, 2, 3])
    assert np.allclose(o, serve.prompt(q, k, v)[0][n:], rtol=0, atol=1e-12)
    seen = serve.lineage([-1, 0, 0, 2, -1])
    assert [list(np.nonzero(x)[0]) for x in seen] == [[0], [0, 1], [0, 2], [0, 2, 3], [4]]


def test_oracle_sampling():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    at = lambda u, **kw: serve.sample(l, u, **kw)[0]  # noqa: E731
    assert [at(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [at(u, top_k=2) for u in (0.0, 0.57, 0.58, 0.99)] == [1, 1, 3, 3]
    assert [at(u, top_p=0.65) for u in (0.0, 0.57, 0.58, 0.99)] == [1, 1, 3, 3]
    assert [at(u, top_p=0.75) for u in (0.0, 0.43, 0.45, 0.66, 0.68)] == [1, 1, 2, 2, 3]
    assert [at(u, min_p=0.6) for u in (0.0, 0.99)] == [1, 3]
    assert at(0.99, temperature=0.0) == 1 and abs(serve.sample(l, 0.2)[1] - 0.4) < 1e-12
    assert serve.sample(np.array([-np.inf, np.nan]), 0.3) == (-1, 0.0)
    assert serve.sample(np.array([0.0, 0.0, 0.0, 0.0]), 0.6, top_k=2)[0] == 1      # ties to the lowest index
    assert serve.sample(np.array([1.0, np.inf, 2.0, np.inf]), 0.6)[0] == 3


def test_oracle_append_places():
    assert serve.append_places([15, 1], [0, 3, 4], [2, 0, 9, 1], 1, 3) == [(0, 2, 0, 14), (0, 0, 0, 15), (1, 1, 0, 0)]
