"""kvq_fp8_decode against float64 attention over the cache's own entries.

Tolerance of a head's output (2-norm of the difference): c sum_t p_t |v_t| (its 2-norm) with
c = 2^-17 + 4 * 2^-20 size, size = the largest sum_d scale |q_d k_td| of a visible position: a score
is a sum of 128 products in fp32 (the tensor cores round towards zero, 2^-23 a step of 8 at most,
and twice more for the query's two parts and the factors: below 2^-20 of the sum of magnitudes),
moves its weight and the sum of weights by that factor each (twice for the reference), and the
weights' own parts, exponentials and sums take 2^-17 together."""
import pytest
import torch

from fp8_testlib import Cache8, D, attend, cu_of, i32, seen
from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu


def check(c, out, q, window=0, sinks=0, lens=None, drop=None, skip=()):
    G = c.H // c.Hkv
    for b in range(len(c.lens)):
        length = c.lens[b] if lens is None else lens[b]
        if b in skip:
            continue
        if length == 0:
            assert (out[b] == 0).all()
            continue
        keys, vals = c.entries(b, length)
        mask = seen(length, 1, window, sinks)
        if drop is not None and b == 0:
            mask[:, drop] = False
        for h in range(c.H):
            o, mag, size = attend(q[b:b + 1, h].double(), keys[h // G], vals[h // G].nan_to_num(), mask)
            err = (out[b, h].double() - o[0]).norm()
            tol = (2.0 ** -17 + 4 * 2.0 ** -20 * float(size[0])) * mag[0].norm()
            assert err <= tol, (b, h, float(err), float(tol))


@pytest.mark.parametrize("H,Hkv", [(4, 1), (1, 1), (2, 1), (6, 3), (8, 8), (32, 8), (20, 10)])
@pytest.mark.parametrize("lens", [[1], [2], [16], [17], [130], [700, 16, 33], [3, 0, 1, 400], [2100]])
def test_small(H, Hkv, lens):
    c = Cache8(H, Hkv, lens, seed=sum(lens) + H)
    q = c.randn(len(lens), H)
    check(c, c.decode(q), q)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 0), (16, 16), (17, 4), (64, 17),
                                          (100, 300), (129, 1), (2000, 4), (10 ** 9, 7), (0, 5),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("lens", [[1, 16, 17, 20], [130, 331, 0, 64], [1500, 5]])
def test_window(window, sinks, lens):
    c = Cache8(8, 2, lens, seed=sum(lens) + window % 97)
    q = c.randn(len(lens), 8)
    check(c, c.decode(q, window, sinks), q, window, sinks)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("lens,window", [([20000], 0), ([9001, 3], 0), ([17 * i + 1 for i in range(100)], 0),
                                         ([33 * i for i in range(64)], 300), ([40000, 1, 25000], 8192)])
def test_long_and_wide(lens, window):
    c = Cache8(8, 2, lens, seed=len(lens))
    q = c.randn(len(lens), 8)
    check(c, c.decode(q, window, 4), q, window, 4)
    assert K.kvq_get_status(c.h) == 0


def test_pages_outside_the_window_are_not_read():
    """Their ids may be anything."""
    c = Cache8(4, 2, [1000], seed=1)
    q = c.randn(1, 4)
    want = c.decode(q, 100, 20)
    pt = c.pt.clone()
    pt[0, 2:56] = -7            # sinks: pages 0, 1; window [900, 1000): pages 56 .. 62
    assert torch.equal(c.decode(q, 100, 20, pt=pt), want) and K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("sk,sv", [(1e-3, 1e-30), (8.0, 1e4), (1.5, 1e30), (1e-20, 1.0)])
def test_sizes(sk, sv):
    c = Cache8(4, 2, [300, 20], seed=2, scale_k=sk, scale_v=sv)
    q = c.randn(2, 4)
    check(c, c.decode(q), q)


def test_scales_that_differ_between_pages():
    """Values of very different size, small ones under heavy weights and the other way round."""
    for flip in (1, -1):
        c = Cache8(2, 1, [640], seed=3, fill=False)
        ramp = 2.0 ** torch.linspace(-30, 30, 640, device="cuda")[:, None, None]
        c.v = (c.v.float() * ramp).bfloat16()
        q = c.randn(1, 2)
        c.k = (c.k.float() + flip * torch.linspace(-3, 3, 640, device="cuda")[:, None, None]
               * q[0, :1].float()).bfloat16()
        c.append(c.k, c.v, [640])
        check(c, c.decode(q), q)


def test_sharp_and_rising_scores():
    c = Cache8(4, 2, [1500], seed=4, fill=False)
    c.k = (c.k.float() * torch.linspace(0.01, 4, 1500, device="cuda")[:, None, None]).bfloat16()
    c.append(c.k, c.v, [1500])
    for scale in (0.0, 1e-30, 1.0, 6.0):
        q = c.randn(1, 4, scale=scale)
        check(c, c.decode(q), q)


def test_long_accumulation():
    """One KV head whose values are all alike: the sum must not drift over 40,000 positions."""
    c = Cache8(1, 1, [40000], seed=5, fill=False)
    c.v.fill_(1.0)
    c.append(c.k, c.v, [40000])
    out = c.decode(c.randn(1, 1, scale=0.1))
    assert (out.double() - 1).abs().max() <= 2.0 ** -17


@pytest.mark.parametrize("n", [5, 200])
def test_nan_keys_and_values(n):
    """A NaN value makes NaN its element of the heads that see it; hidden ones change nothing."""
    c = Cache8(4, 2, [n, 90], seed=6, fill=False)
    k, v = c.k.clone(), c.v.clone()
    v[n // 2, 0, 7] = float("nan")
    v[n + 10, 1, 9] = float("inf")
    k[n + 50, 0, 0] = float("nan")
    c.append(k, v, [n, 90])
    q = c.randn(2, 4)
    out = c.decode(q)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, :2, 7] = True
    bad[1, 2:, 9] = True
    bad[1, :2] = True
    assert torch.equal(torch.isnan(out), bad)
    # all of them outside the window
    window = n - n // 2 - 1
    out = c.decode(q, window, 0, lens=[n, 90])
    assert not torch.isnan(out[0]).any()
    check(c, out, q, window, 0, skip=(1,))
    out = c.decode(q, 39, 10, lens=[n, 90])
    assert not torch.isnan(out[1]).any()
    # behind the end: a shorter length
    out = c.decode(q, 0, 0, lens=[n // 2, 10])
    assert not torch.isnan(out).any()
    check(c, out, q, lens=[n // 2, 10])


def test_bad_lengths_and_pages():
    c = Cache8(4, 2, [100, 100, 100], seed=7)
    q = c.randn(3, 4)
    want = c.decode(q)
    out = c.decode(q, lens=[100, -1, 113])
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_SEQLEN
    assert torch.equal(out[0], want[0]) and (out[1:] == 0).all()
    for bad in (-1, c.pages, 2 ** 31 - 1):
        pt = c.pt.clone()
        pt[0, 3] = bad
        check(c, c.decode(q, pt=pt), q, drop=slice(48, 64))
        assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_PAGE


def test_nonfinite_queries():
    c = Cache8(4, 2, [300, 300], seed=8)
    q = c.randn(2, 4)
    want = c.decode(q)
    q[0, 1, 5], q[1, 2, 77] = float("nan"), float("inf")
    out = c.decode(q)
    bad = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], want[~bad])


def test_pool_past_32_bits():
    c = Cache8(16, 8, [500], seed=9, extra=400_000)
    q = c.randn(1, 16)
    check(c, c.decode(q), q)


def test_same_bits_and_streams_and_graphs():
    """Repeats, another stream, and two graphs with a workspace each give the same bits."""
    c = Cache8(32, 8, [3000, 17, 900], seed=10)
    q = c.randn(3, 32)
    want = c.decode(q, 700, 5)
    for _ in range(3):
        assert torch.equal(c.decode(q, 700, 5), want)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        out = c.decode(q, 700, 5)
    stream.synchronize()
    assert torch.equal(out, want)
    size = K.kvq_fp8_workspace_bytes(c.h, 3)
    lens, graphs = i32(c.lens), []
    for _ in range(2):
        out, ws = torch.zeros(3, 32, D, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            K.kvq_fp8_decode(c.h, c.pool, c.pages, q, c.pt, lens, out, ws, window=700, sinks=5)
        graphs.append((graph, out, ws))
    for graph, *_ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, out, _ in graphs:
        assert torch.equal(out, want)


def test_append_then_decode_on_one_stream():
    """Step after step without waiting for the host: each sees the token before it."""
    c = Cache8(8, 2, [60, 33], seed=11)
    ws = torch.empty(K.kvq_fp8_workspace_bytes(c.h, 2), dtype=torch.uint8, device="cuda")
    pt = torch.cat([c.pt, i32([c.pages - 1, c.pages - 2])[:, None]], 1)
    pt[1, 3] = c.pages - 2
    c.pt = pt.contiguous()
    cu, outs, qs = cu_of([1, 1]), [], [c.randn(2, 8) for _ in range(8)]
    kv = [(c.randn(2, 2), c.randn(2, 2)) for _ in range(8)]
    lens = [[60 + 1 + i, 33 + 1 + i] for i in range(4)]
    for i in range(4):
        out = torch.empty(2, 8, D, device="cuda")
        at = i32(lens[i])
        K.kvq_fp8_append(c.h, c.pool, c.pages, *kv[i], cu, c.pt, at)
        K.kvq_fp8_decode(c.h, c.pool, c.pages, qs[i], c.pt, at, out, ws)
        outs.append(out)
    c.lens = lens[3]
    check(c, outs[3], qs[3])
    assert K.kvq_get_status(c.h) == 0
