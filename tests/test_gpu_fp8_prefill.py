"""kvq_fp8_prefill against float64 attention over the cache's own entries, and the operators of the
8-bit path together.

Tolerance of a row's output vector (2-norm of the difference): 2^-8 |o| + c |sum_t p_t |v_t|| with
c = 2^-8 + 2^-11: bf16's half step for the result, and for each weight, and 2^-11 for the sums (the
products' operands are exact)."""
import math

import numpy as np
import pytest
import torch

from fp8_testlib import Cache8, D, attend, cu_of, i32, seen
from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu


def check(c, out, q, new, window=0, sinks=0, lens=None, skip=(), drop=None, rows=None):
    """Every row (or `rows` of sequence 0) against float64; `drop`: positions of sequence 0 that
    no row sees."""
    G, at = c.H // c.Hkv, 0
    for b, n in enumerate(new):
        length = c.lens[b] if lens is None else lens[b]
        if n and b not in skip:
            keys, vals = c.entries(b, length)
            mask = seen(length, n, window, sinks)
            if drop is not None and b == 0:
                mask[:, drop] = False
            for h in range(c.H):
                o, mag, _ = attend(q[at:at + n, h].double(), keys[h // G], vals[h // G].nan_to_num(), mask)
                err = (out[at:at + n, h].double() - o).norm(dim=1)
                tol = 2.0 ** -8 * o.norm(dim=1) + (2.0 ** -8 + 2.0 ** -11) * mag.norm(dim=1)
                bad = err > tol
                if rows is not None and b == 0:
                    bad &= rows
                assert not bad.any(), (b, h, bad.nonzero().flatten()[:8].tolist(), float((err - tol).max()))
        at += n


@pytest.mark.parametrize("H,Hkv", [(4, 1), (1, 1), (2, 1), (6, 3), (8, 8), (32, 8)])
@pytest.mark.parametrize("new,lens", [
    ([1], [1]), ([1], [130]), ([16], [16]), ([5], [37]), ([64], [128]), ([65], [129]),
    ([129], [129]), ([300], [300]), ([257], [1000]),
    ([1, 1, 1], [700, 16, 33]), ([3, 0, 70, 1], [3, 50, 400, 2100])])
def test_small(H, Hkv, new, lens):
    c = Cache8(H, Hkv, lens, seed=sum(lens) + H)
    q = c.randn(sum(new), H)
    check(c, c.prefill(q, new), q, new)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("H,Hkv", [(4, 1), (2, 2), (4, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 0), (64, 17), (100, 300), (127, 4),
                                          (128, 128), (129, 129), (200, 130), (500, 4), (10 ** 6, 4), (0, 9),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 30, 0)])
@pytest.mark.parametrize("new,lens", [([1], [700]), ([300], [300]), ([257, 9, 0, 130], [1000, 9, 40, 2100]),
                                      ([700], [1500])])
def test_window(H, Hkv, window, sinks, new, lens):
    c = Cache8(H, Hkv, lens, seed=sum(lens) + window % 97)
    q = c.randn(sum(new), H)
    check(c, c.prefill(q, new, window, sinks), q, new, window, sinks)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("new,lens,window", [
    ([1], [20000], 0), ([33], [9001], 0), ([2000], [2000], 0), ([1500, 1, 7], [4000, 5000, 6001], 700),
    ([1] * 100, [17 * i + 1 for i in range(100)], 300), ([4] * 40, [33 * i + 4 for i in range(40)], 0),
    ([4000], [12000], 1000), ([3001], [3001], 129)])
def test_long_and_wide(new, lens, window):
    c = Cache8(8, 2, lens, seed=len(lens))
    q = c.randn(sum(new), 8)
    check(c, c.prefill(q, new, window, 4), q, new, window, 4)
    assert K.kvq_get_status(c.h) == 0


def test_sharp_rising_and_zero_scores():
    c = Cache8(4, 2, [1500], seed=3, fill=False)
    c.k = (c.k.float() * torch.linspace(0.01, 4, 1500, device="cuda")[:, None, None]).bfloat16()
    c.append(c.k, c.v, [1500])
    for scale in (0.0, 1e-30, 1.0, 6.0):
        q = c.randn(300, 4, scale=scale)
        for window in (0, 200):
            check(c, c.prefill(q, [300], window, 3), q, [300], window, 3)


@pytest.mark.parametrize("sk,sv", [(1e-3, 1e-25), (8.0, 1e4), (1.5, 1e30), (1e-20, 1.0), (1e3, 1.0)])
def test_sizes(sk, sv):
    """Scales on both sides of what one bf16 factor can hold."""
    c = Cache8(4, 2, [300, 20], seed=2, scale_k=sk, scale_v=sv)
    q = c.randn(107, 4, scale=1 / max(1.0, sk))
    check(c, c.prefill(q, [100, 7]), q, [100, 7])


def test_every_code():
    """A cache of all finite codes on scales from 2^-100 to 2^110, one visible token a row: the
    result is that token's entry, exactly.  kvq_fp8_decode: within 2^-20 of it: the weight (also the
    sum of weights) enters in two fp16 parts of 22 bits, their two products are added with at most
    2^-23 lost each, and the factor and the division round once (2^-24) each."""
    c = Cache8(1, 1, [256], seed=4)
    codes = torch.arange(256, device="cuda", dtype=torch.uint8)
    codes[(codes & 127) == 127] = 0
    rec = c.pool.view(c.pages, 1, 4112)
    q = c.randn(256, 1)
    for e in (-100, -50, -7, 0, 6, 7, 8, 50, 110):
        for p, page in enumerate(c.pt[0].tolist()):
            rec[page, 0, 2048:4096] = codes.roll(37 * p).repeat(8)
            rec[page, 0, 4100:4104] = torch.tensor([2.0 ** e], device="cuda").view(torch.uint8)
        want = c.entries(0)[1].transpose(0, 1)
        assert torch.equal(c.prefill(q, [256], 1, 0).double(), want), e
        out = c.decode(q[:1], 1, 0, lens=[201])
        assert torch.all((out[0].double() - want[200]).abs() <= 2.0 ** -20 * want[200].abs()), e


def test_pages_outside_the_window_are_not_read():
    c = Cache8(4, 2, [1000], seed=1)
    q = c.randn(20, 4)
    want = c.prefill(q, [20], 100, 20)
    pt = c.pt.clone()
    pt[0, 2:55] = -7           # sinks: pages 0, 1; the first row's window starts at 980 - 99 = 881
    assert torch.equal(c.prefill(q, [20], 100, 20, pt=pt), want) and K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("H,Hkv,n", [(4, 1, 20), (1, 1, 300), (2, 1, 130)])
@pytest.mark.parametrize("at", [0, 3, 150, 290, 310, 399])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 2), (200, 5), (33, 0)])
def test_nan_values(H, Hkv, n, at, window, sinks):
    """Rows that see the NaN are NaN, the others as without it."""
    c = Cache8(H, Hkv, [400], seed=6)
    q = c.randn(n, H)
    want = c.prefill(q, [n], window, sinks)
    k, v = c.k.clone(), c.v.clone()
    v[at, 0, 7] = float("nan")
    c.append(k, v, [400])
    # the page's scale may have been the lost element's: compare with the cache as it is now
    out = c.prefill(q, [n], window, sinks)
    spoiled = seen(400, n, window, sinks)[:, at]
    assert torch.isnan(out[spoiled]).all() and not torch.isnan(out[~spoiled]).any()
    check(c, out, q, [n], window, sinks, rows=~spoiled)
    if (v[at, 0, 7] != v[at, 0, 7]) and c.v[at, 0].abs().argmax() != 7:
        same = ~spoiled
        assert torch.equal(out[same], want[same])


def test_several_nan_values_and_keys():
    c = Cache8(2, 2, [600], seed=7)
    k, v = c.k.clone(), c.v.clone()
    for at in (5, 250, 470, 520, 599):
        v[at, 0, at % D] = float("inf")
    k[555, 1, 3] = float("nan")
    c.append(k, v, [600])
    q = c.randn(200, 2)
    for window, sinks in ((0, 0), (50, 0), (50, 6), (130, 3), (1, 0)):
        out = c.prefill(q, [200], window, sinks)
        mask = seen(600, 200, window, sinks)
        bad0, bad1 = mask[:, [5, 250, 470, 520, 599]].any(1), mask[:, 555]
        assert torch.equal(torch.isnan(out[:, 0]).all(1), bad0) and torch.equal(torch.isnan(out[:, 0]).any(1), bad0)
        assert torch.equal(torch.isnan(out[:, 1]).all(1), bad1) and torch.equal(torch.isnan(out[:, 1]).any(1), bad1)


@pytest.mark.parametrize("n", [9, 200])
def test_nonfinite_queries(n):
    """A query with a NaN or an infinity spoils its own row and head, and no other."""
    c = Cache8(4, 2, [300])
    q = c.randn(n, 4)
    want = c.prefill(q, [n])
    q[3, 1, 5], q[n - 1, 2, 77] = float("nan"), float("inf")
    out = c.prefill(q, [n])
    bad = torch.zeros(n, 4, dtype=torch.bool, device="cuda")
    bad[3, 1] = bad[n - 1, 2] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], want[~bad])


def test_queries_of_uneven_elements():
    """One element far larger than the others, against keys that cancel it: what the query's 8-bit
    parts keep of the small ones (2^-18 of the largest) enters the scores."""
    c = Cache8(2, 1, [256], seed=14, fill=False)
    c.k[:, :, 0] = 0
    c.append(c.k, c.v, [256])
    for big in (16.0, 256.0):
        q = c.randn(130, 2)
        q[:, :, 0] = big
        out = c.prefill(q, [130])
        # a score moves by at most scale * 2^-18 big sum |k_d|, its weight by that factor, twice
        k = c.entries(0)[0].abs().sum(-1).max()
        extra = 2 * 2.0 ** -18 * 2 * big * float(k) / math.sqrt(D)
        keys, vals = c.entries(0)
        mask = seen(256, 130, 0, 0)
        for h in range(2):
            o, mag, _ = attend(q[:, h].double(), keys[0], vals[0], mask)
            err = (out[:, h].double() - o).norm(dim=1)
            assert torch.all(err <= 2.0 ** -8 * o.norm(dim=1) + (2.0 ** -8 + 2.0 ** -11 + extra) * mag.norm(dim=1))


def test_pages_of_very_different_keys():
    """Keys of one page 2^20 times those of the next, in one tile: each page's scale is its own."""
    c = Cache8(2, 1, [400], seed=15, fill=False)
    size = torch.tensor([2.0 ** (20 * (i // 16 % 2) - 20) for i in range(400)], device="cuda")[:, None, None]
    c.k = (c.k.float() * size * 3).bfloat16()
    c.append(c.k, c.v, [400])
    q = c.randn(300, 2)
    check(c, c.prefill(q, [300]), q, [300])
    check(c, c.prefill(q, [300], 60, 3), q, [300], 60, 3)


def test_behind_the_end():
    """A shorter length: what lies behind it in the last page, NaN or not, is not seen."""
    c = Cache8(4, 2, [90], seed=8, fill=False)
    k, v = c.k.clone(), c.v.clone()
    v[75], k[77] = float("nan"), float("nan")
    c.append(k, v, [90])
    q = c.randn(40, 4)
    out = c.prefill(q, [40], lens=[74])
    check(c, out, q, [40], lens=[74])


def test_bad_lengths_pages_and_rows():
    c = Cache8(4, 2, [300, 300, 300], seed=9)
    q = c.randn(60, 4)
    want = c.prefill(q, [20, 20, 20], 50, 3)
    out = c.prefill(q, [20, 20, 20], 50, 3, lens=[300, 19, 305])
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_SEQLEN
    assert (out[20:] == 0).all()
    check(c, out, q, [20, 20, 20], 50, 3, skip=(1, 2))
    out = c.prefill(q, None, 50, 3, cu=i32([0, 20, 61, 61]))
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_SEQ
    assert (out[20:] == 9).all()
    out = c.prefill(q, None, 50, 3, cu=i32([0, 20, 40, 40]))
    assert K.kvq_get_status(c.h) == 0 and (out[40:] == 9).all()
    for bad in (-1, c.pages, 2 ** 31 - 1):
        pt = c.pt.clone()
        pt[0, 16] = bad
        check(c, c.prefill(q, [20, 20, 20], 50, 3, pt=pt), q, [20, 20, 20], 50, 3, drop=slice(256, 272))
        assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_PAGE
    assert torch.equal(c.prefill(q, [20, 20, 20], 50, 3), want)


@pytest.mark.parametrize("n", [3, 200])
def test_rows_that_see_nothing(n):
    """A window of one token whose page is missing leaves a row without a position: zeros."""
    c = Cache8(4, 2, [400], seed=16)
    q = c.randn(n, 4)
    want = c.prefill(q, [n], 1, 0)
    pt = c.pt.clone()
    pt[0, 24] = -1                         # positions 384 .. 399
    out = c.prefill(q, [n], 1, 0, pt=pt)
    lost = min(n, 16)
    assert (out[n - lost:] == 0).all() and torch.equal(out[:n - lost], want[:n - lost])
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_PAGE
    one = q[n - 1:].contiguous()
    assert (c.decode(one, 1, 0, pt=pt) == 0).all() and K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_PAGE
    check(c, c.prefill(q, [n], 17, 2, pt=pt), q, [n], 17, 2, drop=slice(384, 400))


def test_windows_beyond_a_c_int():
    c = Cache8(4, 2, [300], seed=17)
    q = c.randn(40, 4)
    assert torch.equal(c.prefill(q, [40], 2 ** 32, 2 ** 33), c.prefill(q, [40]))
    assert torch.equal(c.decode(q[:1], 2 ** 32), c.decode(q[:1]))
    assert torch.equal(c.prefill(q, [40], 9, 2 ** 32 + 1), c.prefill(q, [40]))


def test_calls_at_once():
    """Attention of both kinds over one cache, and reads of it, on four streams with workspaces of
    their own: the results are those of one call after the other."""
    c = Cache8(32, 8, [6000, 33, 900], seed=18)
    new = [700, 9, 100]
    cu, q, q1 = cu_of(new), c.randn(809, 32), c.randn(3, 32)
    size, size1 = K.kvq_fp8_prefill_workspace_bytes(c.h, 3, 809), K.kvq_fp8_workspace_bytes(c.h, 3)

    def calls():
        kinds = []
        for _ in range(2):
            out, ws = torch.zeros_like(q), torch.empty(size, dtype=torch.uint8, device="cuda")
            kinds.append((out, lambda o=out, w=ws: c.prefill(q, new, 500, 4, out=o, ws=w, cu=cu)))
        out, ws = torch.zeros(3, 32, D, device="cuda"), torch.empty(size1, dtype=torch.uint8, device="cuda")
        kinds.append((out, lambda o=out, w=ws: c.decode(q1, 800, 2, out=o, ws=w)))
        out = torch.zeros(809, 8, D, dtype=torch.bfloat16, device="cuda")
        kinds.append((out, lambda o=out: K.kvq_fp8_read(c.h, c.pool, c.pages, None, o, cu, c.pt, c.seq_lens)))
        return kinds

    want = calls()
    for _, run in want:
        run()
    got, streams = calls(), [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (_, run), stream in zip(got, streams):
            with torch.cuda.stream(stream):
                run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for (a, _), (b, _) in zip(got, want)) and K.kvq_get_status(c.h) == 0


def test_strided_queries_and_pool_past_32_bits():
    c = Cache8(16, 8, [400], seed=10, extra=400_000)
    assert int(c.pt.max()) * 8 * 4112 > 2 ** 32
    wide = c.randn(33, 40)
    q = wide[:, 5:21]
    check(c, c.prefill(q, [33]), q, [33])


@pytest.mark.parametrize("batch", [511, 3000])
def test_wide_batches(batch):
    new = [(i % 3 != 1) * (1 + i % 2) for i in range(batch)]
    c = Cache8(2, 1, [max(1, n) + i % 200 for i, n in enumerate(new)], seed=batch)
    q = c.randn(sum(new), 2)
    out = c.prefill(q, new, 40, 2)
    check(c, out, q, new, 40, 2, skip=[i for i in range(batch) if i % 41])


def test_agrees_with_decode():
    """A row of a chunk is kvq_fp8_decode of that query and length, in fewer bits."""
    c = Cache8(8, 2, [500], seed=11)
    q = c.randn(50, 8)
    out = c.prefill(q, [50], 90, 4)
    for i in (0, 17, 49):
        one = c.decode(q[i:i + 1].contiguous(), 90, 4, lens=[451 + i])
        d = (out[i].double() - one[0].double()).norm()
        assert d <= 2.0 ** -7 * one.double().norm() * 2


def test_same_bits_streams_graphs():
    c = Cache8(32, 8, [3000, 17, 900], seed=12)
    new = [300, 17, 1]
    q, cu = c.randn(318, 32), cu_of([300, 17, 1])
    want = c.prefill(q, new, 700, 5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        out = c.prefill(q, new, 700, 5)
    stream.synchronize()
    assert torch.equal(out, want)
    size, graphs = K.kvq_fp8_prefill_workspace_bytes(c.h, 3, 318), []
    for _ in range(2):
        out, ws = torch.zeros_like(want), torch.empty(size, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            K.kvq_fp8_prefill(c.h, c.pool, c.pages, q, cu, c.pt, c.seq_lens, out, ws, window=700, sinks=5)
        graphs.append((graph, out, ws))
    for graph, *_ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out, _ in graphs)


def _model_step(c, rope, table, w, x, k, v, positions, new, lens, window, sinks):
    """Norms and rotation, append, attention through the library."""
    n = x.shape[0]
    yq, yk = torch.empty_like(x), torch.empty_like(k)
    K.kvq_norm_rope(c.h, x, k, yq, yk, w[0], w[1], 1e-6, i32(positions), rope)
    c.append(yk, v, new, lens=lens)
    return yq, yk, c.prefill(yq, new, window, sinks, lens=lens)


@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 4)])
def test_prompt_in_chunks_then_steps(window, sinks):
    """A prompt in chunks, then single tokens by kvq_fp8_decode, as a layer of a model runs them:
    norms and rotation, append, attention; against float64 from the plain inputs on, where the
    only differences are the roundings of the rotated heads and of the cache."""
    H, Hkv, total = 8, 2, 333
    c = Cache8(H, Hkv, [total], seed=13, fill=False)
    a = torch.arange(total, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)[None]
    table = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    rope = K.make_rope(table, "half")
    w = [1 + 0.2 * torch.randn(D, generator=c.g, device="cuda") for _ in range(2)]
    x, k, v = c.randn(total, H, scale=3.0), c.randn(total, Hkv, scale=0.5), c.randn(total, Hkv)
    outs, done = [], 0
    for n in (100, 1, 130, 60):
        at = slice(done, done + n)
        done += n
        outs.append(_model_step(c, rope, table, w, x[at], k[at], v[at], range(at.start, at.stop), [n], [done],
                                window, sinks))
    yq = torch.cat([o[0] for o in outs])
    out = torch.cat([o[2] for o in outs])
    while done < total:
        one = slice(done, done + 1)
        done += 1
        q1, k1 = torch.empty_like(x[one]), torch.empty_like(k[one])
        K.kvq_norm_rope(c.h, x[one], k[one], q1, k1, w[0], w[1], 1e-6, i32([done - 1]), rope)
        c.append(k1, v[one], [1], lens=[done])
        o = c.decode(q1, window, sinks, lens=[done])
        yq, out = torch.cat([yq, q1]), torch.cat([out, o.bfloat16()])
    assert K.kvq_get_status(c.h) == 0

    def turned(y, wt):
        y = y.double()
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * wt.double()
        cs = table.double()[:, None]
        p, q = y[..., :64], y[..., 64:]
        return torch.cat([p * cs[..., :64] - q * cs[..., 64:], q * cs[..., :64] + p * cs[..., 64:]], -1)

    want_q, want_k = turned(x, w[0]), turned(k, w[1])
    assert (yq.double() - want_q).norm() <= 2.0 ** -8 * want_q.norm()
    keys, vals = c.entries(0)
    # every entry is its element within half a code's step and the rotated keys' rounding; the
    # smallest step of a page is 2^-10 of at most its largest element / 224
    for got, want in ((keys, want_k.transpose(0, 1)), (vals, v.double().transpose(0, 1))):
        assert torch.all((got - want).abs() <= want.abs() * (2.0 ** -4 + 2.0 ** -7) + want.abs().max() / 224 * 2.0 ** -9)
    mask = seen(total, total, window, sinks)
    for h in range(H):
        o, mag, _ = attend(yq[:, h].double(), keys[h // 4], vals[h // 4], mask)
        err = (out[:, h].double() - o).norm(dim=1)
        # pages' scales may have grown since a row was computed: an older entry then lost up to
        # 2^-10 of the new scale, which is at most (largest element) / 224
        late = 2.0 ** -10 / 224 * (float(vals.abs().max()) + 2 * float(keys.abs().max())
                                   * float(yq[:, h].double().abs().sum(-1).max()) / math.sqrt(D)
                                   * float(vals.abs().max())) * math.sqrt(D)
        assert torch.all(err <= 2.0 ** -8 * o.norm(dim=1) + (2.0 ** -8 + 2.0 ** -11) * mag.norm(dim=1) + late)


def test_each_call_sees_what_came_before_it():
    """Calls back to back, each on what the last one or a torch kernel has just written, eagerly and in a
    graph, give the bits that they give with the GPU idle before each."""
    total = 3000
    c = Cache8(8, 2, [total], seed=19, fill=False)
    table = torch.randn(total, D, generator=c.g, device="cuda")
    rope = K.make_rope(table, "half")
    x, k, v = c.randn(total, 8), c.randn(total, 2), c.randn(total, 2)
    pos, chunks = i32(range(total)), [(0, 1500), (1500, 1501), (1501, 2200), (2200, 3000)]
    fixed = [(cu_of([b - a]), i32([b])) for a, b in chunks]
    ws = [torch.empty(max(K.kvq_fp8_prefill_workspace_bytes(c.h, 1, total), K.kvq_fp8_workspace_bytes(c.h, 1)),
                      dtype=torch.uint8, device="cuda") for _ in range(2)]

    def chain(after=lambda: None):
        got, pool = [], torch.full_like(c.pool, 255)
        after()
        for (a, b), (cu, sl) in zip(chunks, fixed):
            n = b - a
            q0, k0 = x[a:b] * 2, k[a:b] * 0.5                      # torch kernels write what the norms read
            yq, yk = torch.empty_like(q0), torch.empty_like(k0)
            after()
            K.kvq_norm_rope(c.h, q0, k0, yq, yk, None, None, 1e-6, pos[a:b], rope)
            after()
            yk.mul_(1.5)
            after()
            K.kvq_fp8_append(c.h, pool, c.pages, yk, v[a:b], cu, c.pt, sl)
            after()
            out, one = torch.zeros_like(yq), torch.zeros(1, 8, D, device="cuda")
            back = [torch.zeros_like(yk) for _ in range(2)]
            after()
            K.kvq_fp8_read(c.h, pool, c.pages, back[0], back[1], cu, c.pt, sl)
            after()
            K.kvq_fp8_prefill(c.h, pool, c.pages, yq, cu, c.pt, sl, out, ws[0], window=800, sinks=3)
            after()
            K.kvq_fp8_decode(c.h, pool, c.pages, out[n - 1:], c.pt, sl, one, ws[1], window=90)
            after()
            got += [yq, yk, *back, out, one * 1]
        return got

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(chain(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_copies_and_other_streams(captured):
    """What a call reads comes from a copy, a memset and kernels of another stream that its own stream waits
    for; what it writes is read in another stream."""
    n = 600
    c = Cache8(8, 2, [n], seed=20, fill=False)
    rope = K.make_rope(torch.randn(n, D, generator=c.g, device="cuda"), "half")
    x, k, v = c.randn(n, 8, scale=2.0), c.randn(n, 2), c.randn(n, 2)
    pos, cu, sl = i32(range(n)), cu_of([n]), c.seq_lens
    ws = torch.empty(K.kvq_fp8_prefill_workspace_bytes(c.h, 1, n), dtype=torch.uint8, device="cuda")
    q0, v0, yq, yk, out = (torch.empty_like(t) for t in (x, v, x, k, x))
    big, res = torch.empty(1 << 26, device="cuda"), torch.empty_like(x)
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        q0.copy_(x)                                # a copy right before the norms
        K.kvq_norm_rope(c.h, q0, k, yq, yk, None, None, 1e-6, pos, rope)
        with torch.cuda.stream(side):
            big.fill_(1.0)                         # long enough for the main stream to be ahead
            v0.copy_(v * big[0])
        c.pool.zero_()                             # a memset
        main.wait_stream(side)
        K.kvq_fp8_append(c.h, c.pool, c.pages, yk, v0, cu, c.pt, sl)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            K.kvq_fp8_prefill(c.h, c.pool, c.pages, yq, cu, c.pt, sl, out, ws, window=100)
            res.copy_(out)
        main.wait_stream(side)

    run()
    torch.cuda.synchronize()
    c.pool.zero_()
    torch.cuda.synchronize()
    K.kvq_norm_rope(c.h, x, k, yq, yk, None, None, 1e-6, pos, rope)
    torch.cuda.synchronize()
    c.append(yk, v, [n])
    torch.cuda.synchronize()
    want = c.prefill(yq, [n], 100)
    torch.cuda.synchronize()
    assert torch.equal(res, want)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for _ in range(3):
        for t in (q0, v0, yq, yk, out, res):
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        assert torch.equal(res, want)
    assert K.kvq_get_status(c.h) == 0
