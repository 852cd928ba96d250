"""GPU: the calls around the decode step refuse tensors of another device than the current one, before they launch."""
import pytest
import torch

from helpers import build_all

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _build():
    build_all()


def _bf(*s):
    return torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda")


def test_tensors_of_another_device_are_refused(monkeypatch):
    """With cuda:1 as the current device, as far as the binding can tell, cuda:0's tensors are another's."""
    from conditional_sparse_attention_b200 import oda
    ctx = oda.oda_create(oda.make_config(2, 4, 2, 3, 512))
    stream = torch.cuda.current_stream()
    i32 = lambda *s: torch.zeros(*s, **I32)  # noqa: E731
    kp, out, token, nxt = _bf(6, 2, 16, 128), _bf(5, 4, 128), i32(2) - 9, i32(2) - 9
    pages = kp.clone(), kp.clone()
    pool8 = torch.zeros(6, 2, 4224, dtype=torch.uint8, device="cuda")
    q, kn, vn = _bf(5, 4, 128), _bf(5, 2, 128), _bf(5, 2, 128)
    stage = _bf(1, 4, 2, 128), _bf(1, 4, 2, 128)
    cu, one, table, parent = torch.tensor([0, 2, 4], **I32), torch.ones(2, **I32), i32(2, 3), i32(5) - 1
    logits, u = torch.zeros(2, 9, device="cuda"), torch.zeros(2, device="cuda")
    calls = [
        lambda: oda.oda_attend_full_prompt(ctx, cu, q, kn, vn, out, stream=stream),
        lambda: oda.oda_attend_local_prompt(ctx, cu, q, kn, vn, out, stream=stream),
        lambda: oda.oda_attend_full_tree(ctx, oda.kv_layer(*pages), table, one, None, cu, parent, q, kn, vn, out, stream=stream),
        lambda: oda.oda_append(ctx, [oda.kv_layer(*pages)], table, one, cu, None, *stage, pos_next=nxt, stream=stream),
        lambda: oda.oda_append_fp8(ctx, [oda.kv8_layer(pool8)], table, one, cu, None, *stage, pos_next=nxt, stream=stream),
        lambda: oda.oda_sample(ctx, logits, u, token, stream=stream),
    ]
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        for call in calls:
            with pytest.raises(ValueError, match="current device"):
                call()
    torch.cuda.synchronize()
    assert torch.all(out == 3.0) and torch.equal(pages[0], kp) and not pool8.any()
    assert token.tolist() == [-9, -9] and nxt.tolist() == [-9, -9]
    for call in calls:
        call()
    assert oda.oda_get_error(ctx) == 0 and token.tolist() == [0, 0] and nxt.tolist() == [3, 3]
    ctx.close()
