"""kvq_set_rotation: what it derives from R, for every KV head, and its time on the stream."""
import numpy as np
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_prefill import D, Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_rotated", [False, True])
def test_every_head(q_rotated):
    """64 KV heads: the prefill's operands of each head, and the decode's R_V^T beside them."""
    c = Paged("int2", 64, 64, [40], seed=21, q_rotated=q_rotated)
    q = c.queries(20)
    out = c.prefill(q, [0, 20])
    c.check(out, q, [20])
    ws = torch.empty(K.kvq_workspace_bytes(c.h, 1, 1), dtype=torch.uint8, device="cuda")
    one = torch.empty(1, 64, D, device="cuda")
    K.kvq_decode(c.h, c.pool, c.pages, q[19:], c.pt, c.seq_lens, one, ws, 1)
    # bf16's half step, and the two paths' operand roundings
    diff = (out[19].double() - one[0].double()).norm(dim=1)
    assert torch.all(diff <= 2.0 ** -7 * one[0].double().norm(dim=1))


def test_replaced_rotations():
    """A second call replaces every matrix of the first."""
    c = Paged("int2", 8, 4, [70], seed=22)
    q = c.queries(70)
    first = c.prefill(q, [0, 70])
    other = torch.from_numpy(np.ascontiguousarray(c.R.cpu().numpy()[:, ::-1])).cuda()
    mu = torch.zeros(4, D, device="cuda")
    K.kvq_set_rotation(c.h, other, mu)
    assert not torch.equal(c.prefill(q, [0, 70]), first)
    K.kvq_set_rotation(c.h, c.R, mu)
    assert torch.equal(c.prefill(q, [0, 70]), first)


@pytest.mark.parametrize("Hkv", [1, 64])
def test_time(Hkv):
    """Two copies and one kernel: about 12 us a call on the stream.  A kernel that walks a head's
    matrix in one CTA takes 60 us more."""
    h = K.kvq_create(K.make_layout(Hkv, Hkv))
    R, mu = torch.randn(2, Hkv, D, D, device="cuda"), torch.zeros(Hkv, D, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = float("inf")
    for _ in range(5):
        for _ in range(3):
            K.kvq_set_rotation(h, R, mu)
        torch.cuda.synchronize()
        torch.cuda._sleep(30_000_000)            # the calls queue behind it
        start.record()
        for _ in range(50):
            K.kvq_set_rotation(h, R, mu)
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) / 50 * 1e3)
    assert best < 40, best
