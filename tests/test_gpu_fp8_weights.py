"""kvq_fp8_prefill: the weights' bits, and values of very different scales, element by element.

Tolerance of an element: the result's half step (2^-8 of it), and of sum_t p_t |v_td| each weight's rounding and 2^-11
for the sums.  Weights are fp16 (2^-11), in a tile of eight pages with a value scale outside 2^-21 .. 2^1 bf16 (2^-8)."""
import math

import pytest
import torch

from fp8_testlib import Cache8, D, attend, seen
from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_fp8_scales import flat_tail, outliers

pytestmark = pytest.mark.gpu


def check_prefill(c, out, q, n, window=0, sinks=0, weight=2.0 ** -8, lens=None):
    G, length = c.H // c.Hkv, c.lens[0] if lens is None else lens[0]
    keys, vals = c.entries(0, length)
    mask = seen(length, n, window, sinks)
    for h in range(c.H):
        o, mag, _ = attend(q[:, h].double(), keys[h // G], vals[h // G], mask)
        err = (out[:, h].double() - o).abs()
        tol = 2.0 ** -8 * o.abs() + (weight + 2.0 ** -11) * mag
        assert torch.all(err <= tol), (h, float((err - tol).max()))


@pytest.mark.parametrize("small,big", [(1.0, 2.0 ** 14), (1.0, 2.0 ** 40), (1.0, 2.0 ** 100), (2.0 ** -60, 2.0 ** 60),
                                       (2.0 ** -20, 1.0), (2.0 ** -40, 1.0)])
@pytest.mark.parametrize("length,at,n", [(300, (0,), 40), (300, (299,), 200), (700, (40, 330, 690), 9),
                                         (3000, (1500,), 3)])
def test_prefill_one_large_element(small, big, length, at, n):
    c = outliers([length], at, small, big)
    q = c.randn(n, 4)
    for window, sinks in ((0, 0), (150, 3)):
        check_prefill(c, c.prefill(q, [n], window, sinks), q, n, window, sinks)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("period", [16, 128])
@pytest.mark.parametrize("exponents", [(0, -30), (-30, 0, 40), (0, 12, -9), (110, 0)])
def test_prefill_scales_that_alternate(period, exponents):
    """Pages, or whole tiles, in turn on scales that fp16 holds and on others, in different elements."""
    n, length, many = 130, 1500, len(exponents)
    c = Cache8(4, 2, [length], seed=3, scale_k=0.5, fill=False)
    v = torch.zeros(length, 2, D, device="cuda")
    for p in range(length):
        j = p // period % many
        v[p, :, 30 * j:30 * j + 30] = c.v[p, :, :30].float() * 2.0 ** exponents[j]
    c.append(c.k, v.bfloat16(), [length])
    q = c.randn(n, 4)
    for window, sinks in ((0, 0), (300, 20)):
        check_prefill(c, c.prefill(q, [n], window, sinks), q, n, window, sinks)


def near_weights(sv, x, length=1024, H=4):
    """Half of the tokens with logit 0 and value sv, half with logit ln(1 + x) and value -sv: the result is the
    difference of two sums of nearly equal weights."""
    c = Cache8(H, 1, [length], seed=4, fill=False)
    c.k.zero_()
    c.v.fill_(sv)
    second = (torch.arange(length, device="cuda") // 16 % 2) == 1
    c.k[second, :, 0] = 1.0
    c.v[second] = -sv
    c.append(c.k, c.v, [length])
    q = torch.zeros(3, H, D, device="cuda")
    q[:, :, 0] = math.log(1 + x) * math.sqrt(D)
    return c, q.bfloat16()


@pytest.mark.parametrize("sv", [1.0, 2.0 ** -6, 2.0 ** 6, 448 * 2.0, 448 * 2.0 ** -21])
@pytest.mark.parametrize("x", [2.0 ** -8 * 0.98, 2.0 ** -7 * 1.5 * 0.98, 0.3, 0.711])
def test_prefill_weights_of_fp16(sv, x):
    """Weights that differ by less than bf16 tells apart."""
    c, q = near_weights(sv, x)
    check_prefill(c, c.prefill(q, [3]), q, 3, weight=2.0 ** -11)


@pytest.mark.parametrize("sv", [448 * 4.0, 448 * 2.0 ** -22, 2.0 ** 60])
def test_prefill_weights_of_bf16(sv):
    """Just outside what fp16 holds."""
    for x in (2.0 ** -8 * 0.98, 0.3):
        c, q = near_weights(sv, x)
        check_prefill(c, c.prefill(q, [3]), q, 3)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("drop", [6, 12, 18, 22])
def test_prefill_flat_tail(drop, first):
    """fp16 has 2^-10 of a weight of 2^-15, with the 2^7 that weights are taken times, left as its half step."""
    c, q = flat_tail(drop, first)
    check_prefill(c, c.prefill(q, [4]), q, 4)


@pytest.mark.parametrize("small", [2.0 ** -17, -3 * 2.0 ** -18, 2.0 ** -12 * 1.0078125])
def test_small_query_elements(small):
    """127 elements far below a row's largest: each is off by at most 2^-17 of that (half of the second part's step of
    2^-9, the largest in [128, 256)), which moves a score by scale * 2^-17 sum |k_d| and a weight, and the sum of the
    weights, by that factor."""
    length, size = 512, 200.0
    c = Cache8(2, 1, [length], seed=8, fill=False)
    second = (torch.arange(length, device="cuda") // 16 % 2) == 1
    c.k.zero_()
    c.k[second, :, 1:] = size
    c.v.fill_(1.0)
    c.v[second] = -1.0
    c.append(c.k, c.v, [length])
    q = torch.full((5, 2, D), small, device="cuda")
    q[:, :, 0] = 1.0
    q = q.bfloat16()
    moved = 2.0 ** -17 * 127 * size / math.sqrt(D)
    check_prefill(c, c.prefill(q, [5]), q, 5, weight=2.0 ** -11 + 2 * math.expm1(moved))


@pytest.mark.parametrize("sv", [1.0, 2.0 ** -40, 2.0 ** 5, 2.0 ** 60])
@pytest.mark.parametrize("H,Hkv,n", [(4, 1, 20), (2, 2, 300)])
def test_nan_values_on_any_scale(sv, H, Hkv, n):
    """Values that are not finite, in pages that are fp16 operands, and bf16 ones, with others of the tile on
    ordinary scales."""
    length, at = 500, (3, 215, 350, 490)
    c = Cache8(H, Hkv, [length], seed=9, fill=False)
    v = c.v.float()
    v[::32] *= sv               # a token of every other page
    for i, p in enumerate(at):
        v[p, 0, 5 + i] = float("nan") if i % 2 else float("inf")
    c.append(c.k, v.bfloat16(), [length])
    q = c.randn(n, H)
    for window, sinks in ((0, 0), (100, 2), (140, 5), (9, 0)):
        out = c.prefill(q, [n], window, sinks)
        mask = seen(length, n, window, sinks)
        spoiled = mask[:, list(at)].any(1)
        G = H // Hkv
        assert torch.isnan(out[spoiled, :G]).all() and not torch.isnan(out[~spoiled, :G]).any()
        assert not torch.isnan(out[:, G:]).any()
        keys, vals = c.entries(0)
        for h in range(H):
            o, mag, _ = attend(q[:, h].double(), keys[h // G], vals[h // G].nan_to_num(), mask)
            err = (out[:, h].double() - o).abs()
            fine = torch.all(err <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11) * mag, dim=1)
            assert fine[~spoiled].all() and (h < G or fine.all())
    assert K.kvq_get_status(c.h) == 0
