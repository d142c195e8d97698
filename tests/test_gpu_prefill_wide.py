"""The chunk attention over batches of more sequences than a block has threads."""
import numpy as np
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_prefill import KINDS, Paged, _cu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [511, 512, 513, 1025, 1600])
def test_many_sequences(kind, B):
    """Two to four sequences a thread of the line's setup; decode tokens, drafts, chunks and sequences
    without new tokens."""
    rng = np.random.default_rng(B)
    new = rng.choice([0, 1, 1, 1, 4, 9], B)
    new[B // 2], new[B - 1], new[0] = 150, 3, 0
    lens = [int(n + rng.integers(0, 60)) for n in new]
    c = Paged(kind, 2, 1, lens, seed=B)
    q = c.queries(int(new.sum()))
    out = c.prefill(q, _cu(new))
    at = np.r_[0, np.cumsum(new)]
    for b in [int(x) for x in np.unique(np.r_[0:40, B // 2 - 20:B // 2 + 20, B - 40:B])]:
        rows = slice(int(at[b]), int(at[b + 1]))
        _check_one(c, b, out[rows], q[rows])
    assert K.kvq_get_status(c.h) == 0


def _check_one(c, b, out, q):
    """c.check of sequence b alone."""
    at, lens, k, v, pt = sum(c.lens[:b]), c.lens, c.k, c.v, c.pt
    c.k, c.v = k[at:at + lens[b]], v[at:at + lens[b]]
    c.pt, c.lens = pt[b:b + 1].contiguous(), [lens[b]]
    try:
        c.check(out, q, [q.shape[0]])
    finally:
        c.lens, c.k, c.v, c.pt = lens, k, v, pt


@pytest.mark.parametrize("kind", KINDS)
def test_largest_batch_mostly_empty(kind):
    """65,535 sequences of which six have new tokens: the same work in the same order as a batch of the
    six, so the same bits."""
    lens, new = [40, 300, 17, 1000, 5, 64], [3, 130, 17, 1, 5, 64]
    c = Paged(kind, 4, 2, lens, seed=51)
    q = c.queries(sum(new))
    want = c.prefill(q, _cu(new))
    c.check(want, q, new)
    B, at = 65535, [0, 511, 512, 40000, 65533, 65534]
    pt = torch.full((B, c.pt.shape[1]), -1, dtype=torch.int32, device="cuda")
    pt[at] = c.pt
    seq_lens = torch.full((B,), 7, dtype=torch.int32, device="cuda")
    seq_lens[at] = c.seq_lens
    n = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    n[torch.tensor(at) + 1] = torch.tensor(new, device="cuda")
    size = (K.kvq_prefill_workspace_bytes if kind == "int2" else K.kvq_bf16_prefill_workspace_bytes)
    ws = torch.empty(size(c.h, B, q.shape[0]), dtype=torch.uint8, device="cuda")
    out = c.prefill(q, n.cumsum(0).to(torch.int32), pt=pt, seq_lens=seq_lens, ws=ws)
    assert torch.equal(out, want)
    assert K.kvq_get_status(c.h) == 0
    # beyond the limit: no workspace size
    assert size(c.h, B + 1, 1) == 0 and size(c.h, 0, 1) == 0
