"""The 16-bit roundings of the chunk attention where they matter most: one key that dwarfs a long flat
tail, and one sequence alone and in other company.

The dominant key.  Logits are g for the first token (whose values are zeros) and 0 for all others, so
the output is the mean of the others' values times n e^-g / (1 + n e^-g): an error of a tail weight is an
error of the whole output.  Relative to |o|, with weights w = e^-g of the row's reference:
  bf16 result                                      2^-8
  weights in bf16 (BF16 cache)                     2^-8, and sums 2^-11
  weights in fp16 (INT2 cache)                     2^-11, or 2^-25 / (2^7 w) where 2^7 w is below 2^-14
  values in fp16, sums, normalised output in fp16  2^-11 each
  keys and queries in fp16 (INT2)                  logit g off by up to g (2^-11 + 2^-11)
"""
import math

import numpy as np
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_prefill import KINDS, Paged

pytestmark = pytest.mark.gpu
D = 128


def _dominant(kind, n, length, gap, H=2):
    """Cache and query rows of a first key that stands `gap` nats above the rest."""
    c = Paged(kind, H, 1, [length], seed=int(100 * gap) + n)
    g = torch.Generator(device="cuda").manual_seed(n)
    signs = torch.where(torch.rand(D, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    clip = 0.96 if kind == "int2" else 1.0       # both ends of the key's range are clipped
    first = gap * math.sqrt(D) / D / clip * signs
    q = signs
    if kind == "int2":                           # two-valued in the cache's basis
        first, q = first @ c.R[0, 0].T, q @ c.R[0, 0].T
    c.k.zero_()
    c.k[0, 0] = first.bfloat16()
    c.v = (1.0 + 0.3 * torch.randn(length, 1, D, generator=g, device="cuda")).bfloat16()
    c.v[0] = 0
    c.append(c.k, c.v)
    return c, q.bfloat16().expand(n, H, D).contiguous()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,length,batch", [(200, 1500, 320), (3, 1500, 320), (200, 9000, 1),
                                            (3, 9000, 1), (1, 9000, 200)])
def test_dominant_first_key(kind, n, length, batch):
    """`batch` sequences of the same pages: enough of them that whole sequences, not single tiles,
    fall to one CTA and share the first key's reference."""
    size = (K.kvq_prefill_workspace_bytes if kind == "int2"
            else K.kvq_bf16_prefill_workspace_bytes)
    for gap in (8.0, 10.0, 12.0, 13.5, 15.0, 15.7, 16.3, 17.0, 17.5):
        c, q = _dominant(kind, n, length, gap)
        cu = torch.arange(0, n * batch + 1, n, dtype=torch.int32, device="cuda")
        out = c.prefill(q.repeat(batch, 1, 1), cu, pt=c.pt.expand(batch, -1).contiguous(),
                        seq_lens=c.seq_lens.expand(batch).contiguous(),
                        ws=torch.empty(size(c.h, batch, n * batch), dtype=torch.uint8, device="cuda"))
        out = out[:, 0].double().view(batch, n, D)
        k, v = (x[0] for x in c.entries(0))
        qq = q[0, 0].double()
        if kind == "int2":
            qq = qq @ c.R[0, 0].double()
        s = k @ qq / math.sqrt(D)
        assert abs(float(s[0]) - gap) < 0.02 * gap and float(s[1:].abs().max()) == 0
        hidden = torch.ones(n, length, device="cuda", dtype=torch.bool).triu(length - n + 1)
        o = torch.softmax(s.expand(n, length).masked_fill(hidden, -math.inf), 1) @ v
        if kind == "int2":
            o = o @ c.R[1, 0].double().T
            tol = (2.0 ** -8 + 3 * 2.0 ** -11 + gap * 2.0 ** -10
                   + max(2.0 ** -11, 2.0 ** (-32 + 1.02 * gap / math.log(2))))
        else:
            tol = 2 * 2.0 ** -8 + 2.0 ** -11
        err = float(((out - o).norm(dim=2) / o.norm(dim=1)).max())
        assert err <= tol, (gap, err, tol)
        assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_alone_and_in_company(kind):
    """A sequence gives the same bits in the same call.  In another batch or chunking its sums are taken
    in another order: a weight moves by about 2^-20 (fp32 scores of up to 16 binary orders), which
    moves its 16-bit rounding in one of 2^12 cases (bf16, by 2^-8) or 2^9 (fp16, by 2^-11): 2^-14 of
    an output at most as a root mean square.  That moves the bf16 result, by 2^-8 at most, in one case of
    2^6: 2^-11 of the output's 2-norm, and 2^-10.5 is allowed.  (Weights rounded against references that
    depend on the division differ by 2^-9 to 2^-10.)"""
    lens, n = [5000, 300, 2500, 17], 130
    c = Paged(kind, 8, 2, lens, seed=16)
    q = c.queries(n)
    one = c.prefill(q, [0, n, n, n, n])
    assert torch.equal(one, c.prefill(q, [0, n, n, n, n]))
    c.check(one, q, [n, 0, 0, 0])
    new = [n, 33, 350, 17]
    both = c.prefill(torch.cat([q, c.queries(400)]), [0, *np.cumsum(new).tolist()])[:n]
    c.check(both, q, [n])
    chunks = torch.cat([c.prefill(q[a:b], [0, b - a, b - a, b - a, b - a],
                                  seq_lens=torch.tensor([lens[0] - n + b, 300, 2500, 17],
                                                        dtype=torch.int32, device="cuda"))
                        for a, b in ((0, 1), (1, 70), (70, n))])
    c.check(chunks, q, [n])
    for other in (both, chunks):
        assert float((one.double() - other.double()).norm()) <= 2.0 ** -10.5 * float(one.double().norm())


@pytest.mark.parametrize("H,Hkv", [(4, 1), (3, 3), (16, 8)])
def test_one_visible_token_is_returned(H, Hkv):
    """BF16: rows that see one token give its values bit for bit, whatever the score: first rows of
    prompts, and single tokens."""
    new = [1] * 40 + [300, 5, 130]
    c = Paged("bf16", H, Hkv, new, seed=18)
    q = c.queries(sum(new), scale=2.0)
    out = c.prefill(q, [0, *np.cumsum(new).tolist()])
    first = torch.tensor([0, *np.cumsum(new)[:-1].tolist()], device="cuda")
    assert torch.equal(out[first], c.v[first].repeat_interleave(H // Hkv, 1))
