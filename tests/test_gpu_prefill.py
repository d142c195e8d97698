"""Attention of chunks of new tokens over the paged caches (kvq_prefill, kvq_bf16_prefill) against
float64 attention over the cache's own entries.

Tolerance of a row's output vector (2-norm of the difference):
    2^-8 |o| + c |sum_t p_t |v_t||
2^-8 is bf16's half step.  BF16 cache: the scores' operands are exact, a weight is rounded to bf16
(2^-8), the sums are fp32 (2^-11 is ample): c = 2^-8 + 2^-11.  INT2 cache: weights and values are
rounded to fp16 (2^-11 each, and 2^-11 for the sums and the fp32 rotation), keys and rotated queries
too, which moves logit t by scale * sum_d q_d k_td (e_d + f_td) with independent |e|, |f| <= 2^-11,
of standard deviation at most scale * 2^-11 sqrt(2/3) sqrt(sum_d q_d^2 k_td^2): six of these, D,
move every weight and their sum by a factor within exp(+-D) each: c = 3 * 2^-11 + 2 D.
"""
import math

import numpy as np
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu
D = 128


class Paged:
    """A cache of sequences with `lens` positions, filled through the library's append."""

    def __init__(self, kind, H, Hkv, lens, seed=0, extra=2, max_pages=None, **flags):
        self.kind, self.H, self.Hkv, self.lens = kind, H, Hkv, list(lens)
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.h = K.kvq_create(K.make_layout(H, Hkv, **flags))
        q, _ = np.linalg.qr(torch.randn(2, Hkv, D, D, generator=g, device="cuda",
                                        dtype=torch.float64).cpu().numpy())
        self.R = torch.from_numpy(np.ascontiguousarray(q, np.float32)).cuda()
        K.kvq_set_rotation(self.h, self.R, torch.zeros(Hkv, D, device="cuda"))
        need = [(c + 15) // 16 for c in lens]
        self.pages = sum(need) + extra
        perm = np.random.default_rng(seed).permutation(self.pages).astype(np.int32)
        pt = np.full((len(lens), max(max_pages or 1, max(need))), -1, np.int32)
        o = 0
        for b, m in enumerate(need):
            pt[b, :m] = perm[o:o + m]
            o += m
        self.pt = torch.from_numpy(pt).cuda()
        size = K.kvq_page_bytes(self.h) if kind == "int2" else K.kvq_bf16_page_bytes(self.h)
        # 0xFF bytes: NaN wherever nothing is appended
        self.pool = torch.full((self.pages * size,), 255, dtype=torch.uint8, device="cuda")
        n = sum(lens)
        self.k = (1.5 * torch.randn(max(n, 1), Hkv, D, generator=g, device="cuda")).bfloat16()
        self.v = torch.randn(max(n, 1), Hkv, D, generator=g, device="cuda").bfloat16()
        if n:
            self.append(self.k, self.v)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def append(self, k, v):
        seq = torch.cat([torch.full((c,), b, dtype=torch.int32) for b, c in
                         enumerate(self.lens)]).cuda()
        pos = torch.cat([torch.arange(c, dtype=torch.int32) for c in self.lens]).cuda()
        fn = K.kvq_append if self.kind == "int2" else K.kvq_bf16_append
        fn(self.h, self.pool, self.pages, k, v, seq, pos, self.pt)

    def entries(self, b):
        """float64 keys and values [Hkv, len, 128] of sequence b, in the cache's basis."""
        c = self.lens[b]
        if self.kind == "bf16":
            at = sum(self.lens[:b])
            return [x[at:at + c].double().transpose(0, 1) for x in (self.k, self.v)]
        ko = torch.empty(c, self.Hkv, D, device="cuda")
        vo = torch.empty_like(ko)
        K.kvq_dequant(self.h, self.pool, self.pages, self.pt, b, 0, c, ko, vo)
        return ko.double().transpose(0, 1), vo.double().transpose(0, 1)

    def queries(self, n, scale=1.0):
        return (scale * torch.randn(n, self.H, D, generator=self.g, device="cuda")).bfloat16()

    def prefill(self, q, cu, out=None, ws=None, seq_lens=None, pt=None):
        n, B = q.shape[0], self.pt.shape[0]
        size = (K.kvq_prefill_workspace_bytes if self.kind == "int2"
                else K.kvq_bf16_prefill_workspace_bytes)
        fn = K.kvq_prefill if self.kind == "int2" else K.kvq_bf16_prefill
        out = torch.full((n, self.H, D), 9.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        # the workspace's contents on entry do not matter: NaN bytes
        ws = torch.full((size(self.h, B, n),), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda") if isinstance(cu, list) else cu
        fn(self.h, self.pool, self.pages, q, cu, self.pt if pt is None else pt,
           self.seq_lens if seq_lens is None else seq_lens, out, ws)
        return out

    def check(self, out, q, new, lens=None, skip=(), drop=None):
        """Every row against float64; `drop`: positions of sequence 0 that no row sees."""
        at, G = 0, self.H // self.Hkv
        f = self.h.layout.flags
        for b, n in enumerate(new):
            length = self.lens[b] if lens is None else lens[b]
            if n == 0 or b in skip:
                at += n
                continue
            keys, vals = self.entries(b)
            for hh in range(self.H):
                kv = hh // G
                k, v = keys[kv, :length], vals[kv, :length]
                qq = q[at:at + n, hh].double()
                if self.kind == "int2" and not f & K.KVQ_Q_ROTATED:
                    qq = qq @ self.R[0, kv].double()
                hidden = torch.ones(n, length, device="cuda", dtype=torch.bool).triu(length - n + 1)
                if drop is not None and b == 0:
                    hidden[:, drop] = True
                scale = 1 / math.sqrt(D)
                s = (qq @ k.T * scale).masked_fill(hidden, -math.inf)
                p = torch.nan_to_num(torch.softmax(s, 1))
                o, mag = p @ v, p @ v.abs()
                if self.kind == "int2":
                    sd = (qq.square() @ k.square().T).masked_fill(hidden, 0).amax(1).sqrt()
                    c = 3 * 2.0 ** -11 + 2 * 6 * scale * 2.0 ** -11 * math.sqrt(2 / 3) * sd
                    if not f & K.KVQ_OUT_ROTATED:
                        o = o @ self.R[1, kv].double().T
                else:
                    c = 2.0 ** -8 + 2.0 ** -11
                err = (out[at:at + n, hh].double() - o).norm(dim=1)
                tol = 2.0 ** -8 * o.norm(dim=1) + c * mag.norm(dim=1)
                worst = int((err - tol).argmax())
                assert torch.all(err <= tol), (b, hh, worst, float(err[worst]), float(tol[worst]))
            at += n


def _cu(new):
    return [0] + [int(x) for x in np.cumsum(new)]


KINDS = ["bf16", "int2"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,Hkv", [(4, 1), (1, 1), (2, 1), (6, 3), (8, 8), (32, 8)])
@pytest.mark.parametrize("new,lens", [
    ([1], [1]), ([1], [130]), ([16], [16]), ([5], [37]), ([64], [128]), ([65], [129]),
    ([129], [129]), ([300], [300]), ([257], [1000]),
    ([1, 1, 1], [700, 16, 33]), ([3, 0, 70, 1], [3, 50, 400, 2100])])
def test_small(kind, H, Hkv, new, lens):
    c = Paged(kind, H, Hkv, lens, seed=sum(lens) + H)
    q = c.queries(sum(new))
    c.check(c.prefill(q, _cu(new)), q, new)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,lens", [
    ([1], [20000]), ([33], [9001]), ([2000], [2000]), ([1500, 1, 7], [4000, 5000, 6001]),
    ([1] * 100, [17 * i + 1 for i in range(100)]), ([4] * 40, [33 * i + 4 for i in range(40)])])
def test_long_and_wide(kind, new, lens):
    c = Paged(kind, 8, 2, lens, seed=len(lens))
    q = c.queries(sum(new))
    c.check(c.prefill(q, _cu(new)), q, new)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_sharp_scores(kind):
    """Large logits whose maximum keeps moving: the running maximum and the rescaling."""
    c = Paged(kind, 4, 2, [1500], seed=3)
    q = c.queries(200, scale=6.0)
    c.check(c.prefill(q, [0, 200]), q, [200])


def test_rising_maximum():
    """Keys that grow along the sequence, so that each tile's scores dwarf the last one's."""
    c = Paged("bf16", 2, 1, [900], seed=4)
    c.k = (c.k.float() * torch.linspace(0.01, 4, 900, device="cuda")[:, None, None]).bfloat16()
    c.append(c.k, c.v)
    q = c.queries(300, scale=3.0)
    c.check(c.prefill(q, [0, 300]), q, [300])


def test_tiny_and_large_values():
    """Values and keys of 1e-6 and of 3e4: fp16 operands of the INT2 path."""
    for size in (1e-4, 2e3):
        c = Paged("int2", 2, 1, [400], seed=5)
        c.v = (c.v.float() * size).bfloat16()
        c.append(c.k, c.v)
        q = c.queries(100)
        c.check(c.prefill(q, [0, 100]), q, [100])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [0.0, 1e-38, 1e-30])
def test_queries_near_zero(kind, size):
    """Rows of zeros (padding) and of next to nothing weigh what they see alike; what lies behind
    their position stays hidden, and other rows of the tile are as ever."""
    c = Paged(kind, 4, 2, [300, 70], seed=6)
    q = c.queries(130)
    q[::2] = (q[::2].float() * size).bfloat16()
    c.check(c.prefill(q, [0, 90, 130]), q, [90, 40])
    q = c.queries(5, scale=size)               # one row tile, several of the keys' tiles
    c.check(c.prefill(q, [0, 5, 5]), q, [5, 0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [9, 200])
def test_nonfinite_queries(kind, n):
    """A query with a NaN or an infinity spoils its own row and head, and no other."""
    c = Paged(kind, 4, 2, [300])
    q = c.queries(n)
    want = c.prefill(q, [0, n])
    q[3, 1, 5], q[n - 1, 2, 77] = float("nan"), float("inf")
    out = c.prefill(q, [0, n])
    bad = torch.zeros(n, 4, dtype=torch.bool, device="cuda")
    bad[3, 1] = bad[n - 1, 2] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("kind,extra", [("int2", 500_000), ("bf16", 80_000)])
def test_pool_past_32_bits(kind, extra):
    """Records beyond 4 GB, and appends to them."""
    c = Paged(kind, 16, 8, [400], seed=7, extra=extra)
    assert int(c.pt.max()) * (c.pool.numel() // c.pages) > 2 ** 32
    q = c.queries(33)
    c.check(c.prefill(q, [0, 33]), q, [33])
    rope, pos = K.make_rope(torch.ones(1, 2, device="cuda"), "half"), torch.zeros(1, dtype=torch.int32,
                                                                                  device="cuda")
    app = K.kvq_append_rope if kind == "int2" else K.kvq_bf16_append_rope
    plain = K.kvq_append if kind == "int2" else K.kvq_bf16_append
    last, seq = pos + 399, torch.zeros_like(pos)
    turned = torch.empty_like(c.k[:1])
    K.kvq_rope(c.h, c.k[:1], turned, pos, rope)
    plain(c.h, c.pool, c.pages, turned, c.v[:1], seq, last, c.pt)
    want = c.prefill(q, [0, 33])
    c.append(c.k, c.v)
    app(c.h, c.pool, c.pages, c.k[:1], c.v[:1], seq, last, c.pt, rope, rope_positions=pos)
    assert torch.equal(c.prefill(q, [0, 33]), want)


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams(kind):
    """Calls that overlap on two streams, each with its own workspace, and a call whose tensors
    were made on another stream."""
    c = Paged(kind, 8, 2, [3000, 40], seed=8)
    q = [c.queries(n) for n in (140, 60)]
    cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 120, 140], [0, 60, 60])]
    want = [c.prefill(*a) for a in zip(q, cu)]
    size = (K.kvq_prefill_workspace_bytes if kind == "int2" else K.kvq_bf16_prefill_workspace_bytes)
    ws = [torch.empty(size(c.h, 2, 140), dtype=torch.uint8, device="cuda") for _ in q]
    streams = [torch.cuda.Stream() for _ in q]
    outs = [[torch.empty_like(w) for _ in range(4)] for w in want]
    torch.cuda.synchronize()
    for r in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                c.prefill(q[i], cu[i], out=outs[i][r], ws=ws[i])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)
    assert K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("out_rotated,q_rotated", [(True, False), (False, True), (True, True)])
def test_folded_rotations(out_rotated, q_rotated):
    c = Paged("int2", 8, 2, [500, 90], out_rotated=out_rotated, q_rotated=q_rotated)
    q = c.queries(150)
    c.check(c.prefill(q, [0, 130, 150]), q, [130, 20])


@pytest.mark.parametrize("kind", KINDS)
def test_equals_decode(kind):
    """A row is what the one-token decode gives for its length.  (The decode reads a copy of the
    cache whose empty slots are zeros: it multiplies what lies behind the length by weight 0.)"""
    c = Paged(kind, 4, 1, [600])
    pool0 = torch.zeros_like(c.pool)
    full, c.pool = c.pool, pool0
    c.append(c.k, c.v)
    c.pool = full
    n = 70
    q = c.queries(n)
    got = c.prefill(q, [0, n])
    dec = K.kvq_decode if kind == "int2" else K.kvq_bf16_decode
    ws = torch.empty(K.kvq_workspace_bytes(c.h, 1, 2), dtype=torch.uint8, device="cuda")
    for r in (0, 1, 33, 69):
        want = torch.empty(1, 4, D, device="cuda")
        dec(c.h, pool0, c.pages, q[r:r + 1], c.pt,
            torch.tensor([600 - n + r + 1], dtype=torch.int32, device="cuda"), want, ws, 2)
        # bf16's half step, and the two paths' operand roundings
        assert (got[r].double() - want[0].double()).norm() <= 2.0 ** -7 * want.double().norm()


@pytest.mark.parametrize("kind", KINDS)
def test_strided_queries_and_rows_left_alone(kind):
    """q as a slice of a fused projection; rows behind the last sequence stay as they were."""
    c = Paged(kind, 8, 2, [100, 300])
    wide = torch.randn(160, 8 + 4, D, generator=c.g, device="cuda").bfloat16()
    out = torch.full((160, 8, D), 5.0, dtype=torch.bfloat16, device="cuda")
    c.prefill(wide[:, :8], [3, 40, 150], out=out)
    assert torch.all(out[:3] == 5) and torch.all(out[150:] == 5)
    c.check(out[3:150], wide[3:150, :8], [37, 110])


@pytest.mark.parametrize("kind", KINDS)
def test_invalid_sequences(kind):
    """Too many new tokens, a negative length, one beyond the table: zeros and the status bit; a
    row range outside q: skipped."""
    lens = [50, 60, 70, 80, 40]
    c = Paged(kind, 4, 2, lens)
    q = c.queries(200)
    sl = torch.tensor([50, 19, -1, 16 * c.pt.shape[1] + 1, 40], dtype=torch.int32, device="cuda")
    new = [30, 20, 3, 5, 10]
    out = c.prefill(q, _cu(new), seq_lens=sl)
    assert torch.all(out[30:58] == 0) and torch.all(out[68:] == 9)
    c.check(out, q, new, skip=(1, 2, 3))
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_SEQLEN
    out = c.prefill(q, [0, 30, 20, 500, -1, -1])        # only the first is a range of rows
    assert torch.all(out[30:] == 9)
    c.check(out, q, [30, 0, 0, 0, 0])
    assert K.kvq_get_status(c.h) & K.KVQ_STATUS_BAD_SEQ


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_are_left_out(kind):
    c = Paged(kind, 4, 2, [400, 50])
    pt = c.pt.clone()
    pt[0, 3], pt[0, 20] = -1, c.pages
    q = c.queries(150)
    out = c.prefill(q, [0, 120, 150], pt=pt)
    drop = list(range(48, 64)) + list(range(320, 336))
    c.check(out, q, [120, 30], drop=drop)
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_PAGE
    # every page bad: rows that see nothing are zero
    out = c.prefill(q, [0, 120, 150], pt=torch.full_like(pt, -1))
    assert torch.all(out == 0)
    K.kvq_get_status(c.h)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_nonfinite_tokens(kind, what):
    """A value vector with a NaN or an infinity reaches the rows that see it and no others; so
    does a key's."""
    n = 200
    for which in ("k", "v"):
        c = Paged(kind, 4, 2, [n])
        x = getattr(c, which)
        x[77, 1, 5] = what
        c.append(c.k, c.v)
        q = c.queries(n)
        clean = Paged(kind, 4, 2, [n])
        want = clean.prefill(q, [0, n])
        got = c.prefill(q, [0, n])
        assert torch.equal(got[:77], want[:77]) and torch.equal(got[:, :2], want[:, :2])
        if which == "v" or math.isnan(what):
            assert torch.all(torch.isnan(got[77:, 2:]))


def test_refusals():
    c = Paged("int2", 4, 2, [40])
    q = c.queries(10)
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    out = torch.empty(10, 4, D, dtype=torch.bfloat16, device="cuda")
    need = K.kvq_prefill_workspace_bytes(c.h, 1, 10)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(K.KvqError) as e:
        c.prefill(q, cu, ws=ws[:need - 1])
    assert e.value.code == K.KVQ_ENOSPACE
    with pytest.raises(K.KvqError) as e:
        c.prefill(q, cu, ws=ws[16:])
    assert e.value.code == K.KVQ_EINVAL
    c.prefill(q[:0], torch.zeros(2, dtype=torch.int32, device="cuda"), out=out[:0], ws=ws)
    for bad in (dict(q=q[:, :2], cu=cu), dict(q=q, cu=cu[:1]), dict(q=q, cu=cu, out=out[:9]),
                dict(q=q.transpose(1, 2), cu=cu)):
        with pytest.raises(ValueError):
            c.prefill(ws=ws, **bad)
    with pytest.raises(TypeError):
        c.prefill(q.float(), cu, ws=ws)
    with pytest.raises(TypeError):
        c.prefill(q, cu.long(), ws=ws)
    h = K.kvq_create(K.make_layout(4, 2))
    with pytest.raises(K.KvqError) as e:
        K.kvq_prefill(h, c.pool, c.pages, q, cu, c.pt, c.seq_lens, out, ws)
    assert e.value.code == K.KVQ_ENOTREADY


@pytest.mark.parametrize("kind", KINDS)
def test_repeats_and_graphs(kind):
    """The same call twice gives the same bits; a captured call replays on changed inputs, and two
    graphs may share a workspace one after the other."""
    c = Paged(kind, 8, 2, [700, 300])
    n = 90
    q = c.queries(n)
    cu = torch.tensor([0, 60, n], dtype=torch.int32, device="cuda")
    want = c.prefill(q, cu)
    size = (K.kvq_prefill_workspace_bytes if kind == "int2" else K.kvq_bf16_prefill_workspace_bytes)
    ws = torch.empty(size(c.h, 2, n), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(want) for _ in range(2)]
    c.prefill(q, cu, out=outs[0], ws=ws)
    assert torch.equal(outs[0], want)
    q2 = c.queries(n)
    qs = [q2.clone(), q2.clone()]
    graphs = []
    for i in range(2):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.prefill(qs[i], cu, out=outs[i], ws=ws)
        graphs.append(g)
    qs[0].copy_(q)
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    assert torch.equal(outs[1], c.prefill(q2, cu))


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_in_chunks_with_rotary_positions(kind):
    """The operators together: per chunk, rotate the queries, append the rotated keys and the
    values, attend; then against attention over the whole cache, and against one chunk."""
    H, Hkv, L = 8, 2, 333
    results = []
    for chunks in ([333], [100, 1, 16, 216]):
        c = Paged(kind, H, Hkv, [L], seed=11)
        g = torch.Generator(device="cuda").manual_seed(12)
        qkv = torch.randn(L, H + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
        table = torch.empty(L, 64, device="cuda")
        K.kvq_rope_table(table, K.make_rope_scaling("banded", 5e5, 8.0, 4096))
        rope = K.make_rope(table, "interleaved")
        c.pool.fill_(255)
        out = torch.empty(L, H, D, dtype=torch.bfloat16, device="cuda")
        qr = torch.empty(L, H, D, dtype=torch.bfloat16, device="cuda")
        app = K.kvq_append_rope if kind == "int2" else K.kvq_bf16_append_rope
        at = 0
        for m in chunks:
            part = qkv[at:at + m]
            pos = torch.arange(at, at + m, dtype=torch.int32, device="cuda")
            K.kvq_rope(c.h, part[:, :H], qr[at:at + m], pos, rope)
            app(c.h, c.pool, c.pages, part[:, H:H + Hkv], part[:, H + Hkv:],
                torch.zeros_like(pos), pos, c.pt, rope)
            c.prefill(qr[at:at + m], [0, m], out=out[at:at + m],
                      seq_lens=torch.tensor([at + m], dtype=torch.int32, device="cuda"))
            at += m
        kr = torch.empty(L, Hkv, D, dtype=torch.bfloat16, device="cuda")
        K.kvq_rope(c.h, qkv[:, H:H + Hkv], kr, torch.arange(L, dtype=torch.int32, device="cuda"),
                   rope)
        c.k, c.v = kr, qkv[:, H + Hkv:].contiguous()
        c.check(out, qr, [L])
        assert K.kvq_get_status(c.h) == 0
        results.append((out, c.pool))
    assert torch.equal(results[0][1], results[1][1])          # the same cache, byte for byte
