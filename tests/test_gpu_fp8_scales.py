"""kvq_fp8_decode over 8-bit pages of very different scales, element by element.

Element d of a head is a sum of p_t v_td; the tolerance is c sum_t p_t |v_td| with
c = 2^-17 + 4 * 2^-20 size, the terms of which test_gpu_fp8_decode.py derives for a vector's 2-norm: they are
factors on each weight, so they hold for each element too, as long as a weight's own error is one: a weight is
an fp16 number and a residual of 2^-11 of its last place, so its error is below 2^-22 of it down to 2^-13 of the
largest, and below 2^-35 of the largest everywhere (2^-29 where its page's scale is 2^-6 of its run's).  Weights
here are within 2^12 of one another, but for the flat tail's."""
import math

import pytest
import torch

from fp8_testlib import Cache8, D, attend, seen
from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu


def check_decode(c, out, q, window=0, sinks=0, lens=None, extra=0.0):
    G = c.H // c.Hkv
    for b, length in enumerate(c.lens if lens is None else lens):
        keys, vals = c.entries(b, length)
        mask = seen(length, 1, window, sinks)
        for h in range(c.H):
            o, mag, size = attend(q[b:b + 1, h].double(), keys[h // G], vals[h // G], mask)
            tol = (2.0 ** -17 + 4 * 2.0 ** -20 * float(size[0]) + extra) * mag[0]
            err = (out[b, h].double() - o[0]).abs()
            assert torch.all(err <= tol), (b, h, float((err / mag[0].clamp(min=1e-300)).max()))


def outliers(lens, at, small, big, dims=(0,), seed=0, H=4, Hkv=2):
    """Values of size `small`, but for elements `dims` of the positions `at` of each sequence, which are `big` beside
    zeros; keys that set the tokens little apart."""
    c = Cache8(H, Hkv, lens, seed=seed, scale_k=0.3, scale_v=1.0, fill=False)
    v = c.v.float() * small
    for start in [sum(lens[:b]) for b in range(len(lens))]:
        for p in at:
            v[start + p] = 0
            for d in dims:
                v[start + p, :, d] = big
    c.v = v.bfloat16()
    c.append(c.k, c.v, lens)
    return c


# Lengths and batches that give a warp several pages of an item, and those that give it one.
SPREADS = [([32], (3,), 4, 2), ([300], (0,), 4, 2), ([300] * 40, (0,), 8, 8), ([300] * 40, (299,), 8, 8),
           ([300] * 40, (40, 130, 260), 8, 8), ([60000], (30000,), 4, 2), ([60000], (0, 59999), 2, 2),
           ([5000, 33, 900] * 12, (17,), 8, 8)]


@pytest.mark.parametrize("small,big", [(1.0, 2.0 ** 14), (1.0, 2.0 ** 24), (1.0, 2.0 ** 40), (1.0, 2.0 ** 100),
                                       (2.0 ** -60, 2.0 ** 60), (2.0 ** -20, 1.0), (2.0 ** -40, 1.0),
                                       (2.0 ** -90, 2.0 ** 30), (2.0 ** -40, 2.0 ** 120), (1.0, 2.0 ** 126)])
@pytest.mark.parametrize("lens,at,H,Hkv", SPREADS)
def test_decode_one_large_element(small, big, lens, at, H, Hkv):
    """Every other element is what the pages without it make it."""
    c = outliers(lens, at, small, big, H=H, Hkv=Hkv)
    q = c.randn(len(lens), H)
    check_decode(c, c.decode(q), q)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("gap", [14, 30, 60])
def test_decode_scales_that_alternate(gap):
    """Page after page on another scale, in different elements."""
    lens = [700] * 30
    c = Cache8(8, 8, lens, seed=2, scale_k=0.3, fill=False)
    v = torch.zeros(30, 700, 8, D, device="cuda")
    for p in range(700):
        j = p // 16 % 3
        v[:, p, :, 40 * j:40 * j + 40] = c.v.view(30, 700, 8, D)[:, p, :, :40].float() * 2.0 ** (gap * (j - 1))
    c.append(c.k, v.bfloat16().view(-1, 8, D), lens)
    q = c.randn(30, 8)
    check_decode(c, c.decode(q), q)
    check_decode(c, c.decode(q, 200, 20), q, 200, 20)


def test_decode_a_hidden_token_raised_the_scale():
    """The large token is outside the window, or was cut off, and its page keeps the scale."""
    many = 60
    c = outliers([200] * many, (130,), 1.0, 2.0 ** 40, H=8, Hkv=8)
    q = c.randn(many, 8)
    check_decode(c, c.decode(q, 66, 5), q, 66, 5)        # sees 134 .. 199, and 0 .. 4
    lens = [130] * many
    check_decode(c, c.decode(q, lens=lens), q, lens=lens)
    # cut back to 130 and appended to again: the scale stays
    lens = [170] * many
    c.append(c.randn(40 * many, 8, scale=0.3), c.randn(40 * many, 8), [40] * many, lens=lens)
    check_decode(c, c.decode(q, lens=lens), q, lens=lens)


def test_decode_one_huge_value_among_many_parts():
    """Parts of one item, in many CTAs, of which one has totals in another unit."""
    c = outliers([20000], (11111,), 1.0, 2.0 ** 126, H=2, Hkv=1)
    q = c.randn(1, 2)
    check_decode(c, c.decode(q), q)


def flat_tail(drop, first, length=6000):
    """One key 2^drop times as heavy as each of the others, whose values alone are not zero."""
    c = Cache8(2, 1, [length], seed=5, fill=False)
    c.k.zero_()
    c.v = c.v.abs()
    at = 0 if first else length - 5
    c.k[at, :, 0] = 8.0
    c.v[at] = 0
    c.append(c.k, c.v, [length])
    q = torch.zeros(4, 2, D, device="cuda")
    q[:, :, 0] = drop * math.log(2) * math.sqrt(D) / 8
    return c, q.bfloat16()


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("drop", [6, 12, 18, 22])
def test_decode_flat_tail(drop, first):
    """A light weight's own error: 2^-36 of the heavy one, once more for a run's exponent."""
    c, q = flat_tail(drop, first)
    one = q[:1].contiguous()
    check_decode(c, c.decode(one), one, extra=2.0 ** (drop - 35))


@pytest.mark.parametrize("sk,sq", [(2.0 ** 124, 2.0 ** -124), (2.0 ** 124, 2.0 ** -130), (2.0 ** -90, 2.0 ** 90),
                                   (2.0 ** 116, 2.0 ** -112)])
@pytest.mark.parametrize("length", [20, 900])
def test_decode_keys_and_queries_at_the_ends_of_the_range(sk, sq, length):
    """Scores of ordinary size from keys and queries that are not, all of a score's products of one sign: no partial
    product overflows, nor do queries below the smallest normal number count as zeros."""
    c = Cache8(4, 2, [length], seed=7, fill=False)
    sign = torch.where(torch.rand(D, generator=c.g, device="cuda") < 0.5, -1.0, 1.0)
    size = 0.5 + 0.5 * torch.rand(length, 2, 1, generator=c.g, device="cuda")
    c.append((sign * sk * size).bfloat16(), c.v, [length])
    q = (sign * sq * torch.rand(1, 4, D, generator=c.g, device="cuda")).bfloat16()
    check_decode(c, c.decode(q), q)
