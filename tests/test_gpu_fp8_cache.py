"""The 8-bit cache: what kvq_fp8_append writes, bit for bit against the definition, and what
kvq_fp8_read gives back (exactly the entries)."""
import numpy as np
import pytest
import torch

from fp8_testlib import Cache8, D, Model, PAGE, REC, code_values, cu_of, encode, i32
from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu


def _np(x):
    return x.double().cpu().numpy()


def _used(c, lens=None):
    pt = c.pt.cpu().numpy()
    return sorted(int(pt[b, p]) for b, m in enumerate(lens or c.lens) for p in range((m + 15) // 16))


@pytest.mark.parametrize("hkv", [1, 2, 3, 8, 9, 17])
@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [33, 5], [1, 1, 1, 16, 31], [300]])
def test_bytes_of_one_append(hkv, lens):
    c = Cache8(hkv, hkv, lens, seed=sum(lens) + hkv)
    m = Model(c.pages, hkv)
    m.append(_np(c.k), _np(c.v), lens, lens, c.pt.cpu().numpy())
    m.check(c.pool, _used(c))
    untouched = sorted(set(range(c.pages)) - set(_used(c)))
    assert (c.pool.view(c.pages, -1)[untouched] == 255).all()
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("steps", [[1] * 20, [3, 1, 12, 1, 16, 17, 1], [40, 1, 1, 7, 30]])
def test_bytes_of_many_appends(steps):
    """Tokens of growing and shrinking size, so that pages' scales grow again and again."""
    n = sum(steps)
    c = Cache8(2, 2, [n, 2 * n], seed=n, fill=False)
    m = Model(c.pages, 2)
    done = [0, 0]
    for i, s in enumerate(steps):
        size = 2.0 ** ((5 * i) % 7 - 2)
        new = [s, 2 * s]
        k, v = c.randn(3 * s, 2, scale=size), c.randn(3 * s, 2, scale=1 / size)
        done = [a + b for a, b in zip(done, new)]
        c.append(k, v, new, lens=done)
        m.append(_np(k), _np(v), new, done, c.pt.cpu().numpy())
        m.check(c.pool, _used(c, done))
    assert K.kvq_get_status(c.h) == 0


def test_cut_back_and_reused_pages():
    """A sequence that goes on from an earlier position, in a page and at a page's border."""
    c = Cache8(1, 1, [40], seed=1)
    m = Model(c.pages, 1)
    m.append(_np(c.k), _np(c.v), [40], [40], c.pt.cpu().numpy())
    for length, n, size in ((25, 2, 0.01), (34, 1, 8.0), (33, 1, 0.5), (40, 8, 0.25)):
        k, v = c.randn(n, 1, scale=size), c.randn(n, 1, scale=size)
        c.append(k, v, [n], lens=[length])
        m.append(_np(k), _np(v), [n], [length], c.pt.cpu().numpy())
        m.check(c.pool, _used(c))


@pytest.mark.parametrize("size", [1e-38, 1e-20, 1e-3, 1e3, 1e20, 1e37])
def test_extreme_sizes(size):
    c = Cache8(1, 1, [37], seed=2, scale_k=size, scale_v=1.0, fill=False)
    c.append(c.k, c.v, [37])
    m = Model(c.pages, 1)
    m.append(_np(c.k), _np(c.v), [37], [37], c.pt.cpu().numpy())
    m.check(c.pool, _used(c))


def test_every_bf16_mantissa_and_tie():
    """All finite bf16 magnitudes of four binades beside a fixed largest one: each rounding."""
    bits = torch.arange(0x3c00, 0x3c00 + 4 * 128, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).cuda().view(-1, 1, D).repeat(1, 1, 1)
    c = Cache8(1, 1, [4], seed=3, fill=False)
    for top in (1.0, 1.75, 1.7578125, 448.0, 7.0):
        k = torch.cat([x[:3], torch.full((1, 1, D), top, dtype=torch.bfloat16, device="cuda")])
        c.append(k, -k, [4])
        m = Model(c.pages, 1)
        m.append(_np(k), _np(-k), [4], [4], c.pt.cpu().numpy())
        m.check(c.pool, _used(c))


def test_zeros_and_nonfinite():
    c = Cache8(2, 2, [20], seed=4, fill=False)
    k, v = c.k.clone(), c.v.clone()
    k[:, 0] = 0
    k[3, 1, 5], k[4, 1, 6], k[17, 1, 7] = float("nan"), float("inf"), float("-inf")
    v[19, 0, 0] = float("nan")
    c.append(k, v, [20])
    m = Model(c.pages, 2)
    m.append(_np(k), _np(v), [20], [20], c.pt.cpu().numpy())
    m.check(c.pool, _used(c))
    ko, vo = c.read([20])
    assert torch.equal(torch.isnan(ko), ~torch.isfinite(k)) and torch.equal(torch.isnan(vo), torch.isnan(v))
    # a page keeps its flag while its tokens stay, and loses it when it begins anew
    c.append(k[:1], v[:1], [1], lens=[19])
    c.append(c.k[:16], c.v[:16], [16], lens=[16])
    flags = c.pool.view(c.pages, 2, REC)[c.pt[0].long()][..., 4104].cpu()
    assert flags[0].tolist() == [0, 0] and flags[1].tolist() == [2, 1]


@pytest.mark.parametrize("hkv", [1, 3, 8, 20])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([50], [50]), ([50], [3]), ([50], [18]),
                                      ([64, 7, 40, 1], [16, 0, 25, 1]), ([700], [600])])
def test_read(hkv, lens, new):
    c = Cache8(hkv, hkv, lens, seed=sum(new))
    ko, vo = c.read(new)
    at = 0
    for b, n in enumerate(new):
        for got, want in zip((ko, vo), c.entries(b)):
            want = want[:, lens[b] - n:lens[b]].transpose(0, 1)
            assert torch.equal(got[at:at + n].double(), want)
        at += n
    # half a step of what they were: 2^-4 of the value, 2^-10 of the scale for the smallest
    if new == lens:
        s = max(float(x.abs().max()) for x in (c.k, c.v)) / 224
        for got, want in ((ko, c.k), (vo, c.v)):
            d = (got.double() - want.double()).abs()
            assert torch.all(d <= torch.clamp(want.double().abs() * 2.0 ** -4, min=s * 2.0 ** -10))
    assert K.kvq_get_status(c.h) == 0


def test_strided_rows_and_one_output():
    c = Cache8(4, 2, [70], seed=5, fill=False)
    qkv = c.randn(70, 8)
    c.append(qkv[:, 4:6], qkv[:, 6:8], [70])
    m = Model(c.pages, 2)
    m.append(_np(qkv[:, 4:6]), _np(qkv[:, 6:8]), [70], [70], c.pt.cpu().numpy())
    m.check(c.pool, _used(c))
    ko, vo = c.read([70])
    wide = torch.full((70, 5, D), 3.0, dtype=torch.bfloat16, device="cuda")
    K.kvq_fp8_read(c.h, c.pool, c.pages, wide[:, 1:3], None, cu_of([70]), c.pt, c.seq_lens)
    assert torch.equal(wide[:, 1:3], ko) and (wide[:, [0, 3, 4]] == 3).all()
    K.kvq_fp8_read(c.h, c.pool, c.pages, None, wide[:, 3:], cu_of([70]), c.pt, c.seq_lens)
    assert torch.equal(wide[:, 3:], vo) and torch.equal(wide[:, 1:3], ko)


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 500, 1025, 5000])
def test_many_sequences(batch):
    """A step of one token each, some sequences without: rows find their sequence."""
    new = [(i % 5 != 2) * 1 for i in range(batch)]
    c = Cache8(1, 1, [1 + i % 40 for i in range(batch)], seed=batch)
    before = c.pool.clone()
    k, v = c.randn(sum(new) or 1, 1, scale=0.1), c.randn(sum(new) or 1, 1, scale=0.1)
    n = sum(new)
    c.append(k[:n], v[:n], new)
    ko, vo = c.read(new)
    for b in range(0, batch, max(1, batch // 60)):
        want = c.entries(b)
        if new[b]:
            at = sum(new[:b])
            assert torch.equal(ko[at, 0].double(), want[0][0, -1])
            assert (ko[at].double() - k[at].double()).abs().max() <= 0.1 * 5 * 2.0 ** -4
        else:
            ids = c.pt[b, :(c.lens[b] + 15) // 16].long()
            assert torch.equal(c.pool.view(c.pages, -1)[ids], before.view(c.pages, -1)[ids])
    assert K.kvq_get_status(c.h) == 0


def test_bad_sequences_and_pages():
    c = Cache8(2, 2, [40, 40, 40], seed=6)
    before = c.pool.clone()
    k, v = c.randn(12, 2), c.randn(12, 2)

    def rows(cu, lens, pt=None):
        K.kvq_fp8_append(c.h, c.pool, c.pages, k, v, i32(cu), c.pt if pt is None else pt, i32(lens))
        ko = torch.full((12, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
        K.kvq_fp8_read(c.h, c.pool, c.pages, ko, None, i32(cu), c.pt if pt is None else pt, i32(lens))
        return ko

    # lengths that do not fit: skipped, zeros read; the others are as ever
    ko = rows([0, 4, 8, 12], [40, 3, 49])
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_SEQLEN
    assert (ko[4:] == 0).all() and torch.equal(ko[:4].double(), c.entries(0)[0][:, 36:40].transpose(0, 1))
    for b in (1, 2):
        ids = c.pt[b].long()
        assert torch.equal(c.pool.view(c.pages, -1)[ids], before.view(c.pages, -1)[ids])
    # rows behind the last sequence and outside every range are left as they were
    ko = rows([0, 4, 4, 6], [40, 40, 40])
    assert K.kvq_get_status(c.h) == 0 and (ko[6:] == 9).all()
    c.pool.copy_(before)
    ko = rows([0, 4, 8, 40], [40, 40, 40])
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_SEQ and (ko[8:] == 9).all()
    ids = c.pt[2].long()
    assert torch.equal(c.pool.view(c.pages, -1)[ids], before.view(c.pages, -1)[ids])
    # a page out of range
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        pt = c.pt.clone()
        pt[1, 2] = bad
        ko = rows([0, 4, 8, 12], [40, 40, 40], pt)
        assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_PAGE and (ko[4:8] == 0).all()


def test_pool_past_32_bits():
    c = Cache8(8, 8, [100], seed=7, extra=400_000)
    assert int(c.pt.max()) * 8 * REC > 2 ** 32
    m = Model(int(c.pt.max()) + 1, 8)
    m.append(_np(c.k), _np(c.v), [100], [100], c.pt.cpu().numpy())
    m.check(c.pool.view(c.pages, -1)[:int(c.pt.max()) + 1], _used(c))


def test_captured_append_and_read():
    """A step in a graph, replayed with other tokens and lengths in the same buffers."""
    c = Cache8(2, 2, [30, 30], seed=8)
    k, v = c.randn(2, 2), c.randn(2, 2)
    lens, cu = i32([31, 31]), cu_of([1, 1])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    pt = torch.cat([c.pt, torch.full((2, 1), -1, dtype=torch.int32, device="cuda")], 1)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        def step():
            K.kvq_fp8_append(c.h, c.pool, c.pages, k, v, cu, pt, lens)
            K.kvq_fp8_read(c.h, c.pool, c.pages, ko, vo, cu, pt, lens)
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for length in (31, 32):
            lens.fill_(length)
            k.copy_(c.randn(2, 2))
            graph.replay()
            stream.synchronize()
            for b in range(2):
                assert torch.equal(ko[b].double(), c.entries(b, length)[0][:, -1])
                assert torch.equal(vo[b].double(), c.entries(b, length)[1][:, -1])
    assert K.kvq_get_status(c.h) == 0
