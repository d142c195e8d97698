"""The INT2 chunk attention with cache entries near the ends of fp16's range (bound of the error as in
test_gpu_prefill.py), and past it."""
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_prefill import D, Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [100, 5])
@pytest.mark.parametrize("kv", [(1e-6, 1.0), (1e-3, 1.0), (5e3, 1.0), (1.0, 1e-6), (1.0, 1e-4),
                                (1.0, 1.2e4), (2e3, 1e-5)])
def test_small_and_large_entries(kv, n):
    """Keys and values whose scales and zeros are near the ends of fp16 (subnormal, or entries up to
    6e4), the queries scaled the other way so that the logits stay moderate."""
    ks, vs = kv
    c = Paged("int2", 2, 1, [400], seed=15)
    c.k, c.v = (c.k.float() * ks).bfloat16(), (c.v.float() * vs).bfloat16()
    c.append(c.k, c.v)
    entries = torch.stack(c.entries(0)).abs()
    assert torch.isfinite(entries).all() and float(entries.max()) < 65504
    q = c.queries(n, scale=1 / ks)
    c.check(c.prefill(q, [0, n]), q, [n])


@pytest.mark.parametrize("which", ["k", "v"])
def test_entries_past_fp16(which):
    """A token whose scale and zero are finite but whose largest entry is not in fp16 counts as
    infinite: the rows that see it become NaN, the others are as ever."""
    n, at = 200, 77
    clean = Paged("int2", 2, 1, [n], seed=17)
    q = clean.queries(n)
    want = clean.prefill(q, [0, n])
    c = Paged("int2", 2, 1, [n], seed=17)
    turned = torch.zeros(D, device="cuda")
    turned[5] = 8e4                               # in the cache's basis: scale 2.6e4, zero 0
    getattr(c, which)[at, 0] = (turned @ c.R[0 if which == "k" else 1, 0].T).bfloat16()
    c.append(c.k, c.v)
    entry = c.entries(0)[0 if which == "k" else 1][0, at].abs()
    assert torch.isfinite(entry).all() and float(entry.max()) > 65520
    got = c.prefill(q, [0, n])
    assert torch.equal(got[:at], want[:at])
    if which == "v":
        assert torch.isnan(got[at:]).all()
    else:          # its logit is infinite: NaN where positive, weight 0 where negative
        nan = torch.isnan(got[at:]).all(2)
        assert bool(nan.any()) and bool((~nan).any())
        assert torch.isfinite(got[at:][~nan].float()).all()
    assert K.kvq_get_status(c.h) == 0
