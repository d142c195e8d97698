"""Row rotation with many heads a row: up to the limit, and refused beyond it."""
import numpy as np
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_rope import D, _gen, _handle, _rope64, _table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 40, 6])
@pytest.mark.parametrize("heads", [33, 64, 127, 1024])
def test_many_heads(style, rot, heads):
    g, n = _gen(heads + rot), 7
    table = _table(rot, 99)
    x = torch.randn(n, heads, D, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 99, (n,), generator=g, device="cuda", dtype=torch.int32)
    h, rope, y = _handle(), K.make_rope(table, style), torch.empty_like(x)
    K.kvq_rope(h, x, y, pos, rope)
    want, tol = _rope64(x.double().cpu().numpy(), pos.cpu().numpy(), table, style)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)
    assert torch.equal(y[..., rot:], x[..., rot:])
    K.kvq_rope(h, x, x, pos, rope)
    assert torch.equal(x, y)
    assert K.kvq_get_status(h) == 0


def test_too_many_heads():
    h, rope = _handle(), K.make_rope(_table(64, 10), "half")
    x = torch.zeros(1, 1025, D, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(K.KvqError) as e:
        K.kvq_rope(h, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"), rope)
    assert e.value.code == K.KVQ_EINVAL
