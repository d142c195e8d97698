"""Contexts as long as a page table allows, and row arrays past 2^31 elements."""
import math

import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_prefill import D, KINDS, Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pages", [2 ** 20, 2 ** 26])
def test_one_page_over_and_over(kind, pages):
    """A table whose entries are all the same full page: the output is that of its 16 tokens.  Beside
    the roundings of test_gpu_prefill.py, a range's sums run over pages / 8 / ranges tiles, each adding at
    most 2^-23 (tensor-core sums may truncate)."""
    c = Paged(kind, 4, 1, [16], seed=61)
    n = 3
    q = c.queries(n)
    k, v = (x[0] for x in c.entries(0))
    pt = torch.full((1, pages), int(c.pt[0, 0]), dtype=torch.int32, device="cuda")
    seq_lens = torch.full((1,), 16 * pages, dtype=torch.int32, device="cuda")
    out = c.prefill(q, [0, n], pt=pt, seq_lens=seq_lens)
    tiles = pages / 8 / torch.cuda.get_device_properties(0).multi_processor_count
    for hh in range(4):
        qq = q[:, hh].double()
        if kind == "int2":
            qq = qq @ c.R[0, 0].double()
        p = torch.softmax(qq @ k.T / math.sqrt(D), 1)      # hiding two of 2^24 tokens is nothing
        o, mag = p @ v, (p @ v.abs()).norm(dim=1)
        if kind == "int2":
            o = o @ c.R[1, 0].double().T
            sd = (qq.square() @ k.square().T).amax(1).sqrt()
            w = 3 * 2.0 ** -11 + 2 * 6 / math.sqrt(D) * 2.0 ** -11 * math.sqrt(2 / 3) * sd
        else:
            w = 2.0 ** -8 + 2.0 ** -11
        tol = 2.0 ** -8 * o.norm(dim=1) + (w + tiles * 2.0 ** -23) * mag
        assert torch.all((out[:, hh].double() - o).norm(dim=1) <= tol)
    assert K.kvq_get_status(c.h) == 0


def test_rows_past_32_bits():
    """kvq_rope, the rotating append and the prefill at rows whose element offset is beyond 2^31."""
    Hkv, heads = 8, 32
    n, wide = 2 ** 31 // (64 * D) + 9, 64
    c = Paged("bf16", heads, Hkv, [2000], seed=62)
    qkv = torch.empty(n, wide, D, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(8, wide, D, generator=c.g, device="cuda").bfloat16()
    qkv[-8:] = tail
    table = torch.empty(2000, 128, device="cuda")
    K.kvq_rope_table(table, K.make_rope_scaling())
    rope = K.make_rope(table, "half")
    pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    pos[-8:] = torch.arange(1992, 2000, device="cuda")
    want = torch.empty(8, heads, D, dtype=torch.bfloat16, device="cuda")
    K.kvq_rope(c.h, tail[:, :heads], want, pos[-8:].clone(), rope)
    K.kvq_rope(c.h, qkv[:, :heads], qkv[:, :heads], pos, rope)      # every other row is skipped
    assert torch.equal(qkv[-8:, :heads], want)
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_POS
    seq = torch.zeros_like(pos)
    other = c.pool.clone()
    K.kvq_bf16_append_rope(c.h, c.pool, c.pages, qkv[:, heads:heads + Hkv],
                           qkv[:, heads + Hkv:heads + 2 * Hkv], seq, pos, c.pt, rope)
    K.kvq_bf16_append_rope(c.h, other, c.pages, tail[:, heads:heads + Hkv],
                           tail[:, heads + Hkv:heads + 2 * Hkv], seq[:8], pos[-8:].clone(), c.pt, rope)
    assert torch.equal(c.pool, other)
    K.kvq_get_status(c.h)
    out = torch.zeros(n, heads, D, dtype=torch.bfloat16, device="cuda")
    c.prefill(qkv[:, :heads], [n - 8, n], out=out)
    assert torch.equal(out[-8:], c.prefill(want, [0, 8]))
    assert int(out[:-8].count_nonzero()) == 0
    assert K.kvq_get_status(c.h) == 0
