"""Rotary positions on the GPU: the table, the rotation of rows and its inverse, and the appends
that rotate keys on the way, against float64 and against the unfused calls.

Tolerances.  The rotation rounds two products and their sum to fp32 and the result to bf16:
|y - exact| <= 2^-8 |exact| + 3 * 2^-24 (|a c| + |b s|) (a half step of bf16; the second term also
covers the half step of a result that the fp32 errors moved).  The table: reducing the angle leaves
2^-32 of a turn and float64's own p f 2^-52 in the reference, converting the rest of the angle (at
most pi/4) to fp32 pi/4 2^-24, the sine and cosine of it at most 2 units in the last place of a
value below 1 (2^-23), the amplitude's product 2^-24: below 3e-7 times the amplitude together.  The appends must
equal the unfused calls byte for byte.
"""
import math

import numpy as np
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu
D = 128


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table(rot, length, base=1e4):
    t = torch.empty(length, rot, device="cuda")
    K.kvq_rope_table(t, K.make_rope_scaling(base=base))
    return t


def _handle(H=4, Hkv=1, seed=None):
    h = K.kvq_create(K.make_layout(H, Hkv))
    if seed is not None:
        g = _gen(seed)
        q, _ = np.linalg.qr(torch.randn(2, Hkv, D, D, generator=g, device="cuda",
                                        dtype=torch.float64).cpu().numpy())
        mu = torch.randn(Hkv, D, generator=g, device="cuda")
        K.kvq_set_rotation(h, torch.from_numpy(np.ascontiguousarray(q, np.float32)).cuda(), mu)
    return h


def _pairs(rot, style):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if style == "half" else (2 * i, 2 * i + 1)


# ---- the table ----------------------------------------------------------------------------------

def _freq64(rot, kind, base, factor, orig, low, high):
    i = np.arange(rot // 2)
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if kind == "linear":
        f = f / factor
    if kind == "yarn":
        a = max(math.floor(rot * math.log(orig / (high * 2 * math.pi)) / (2 * math.log(base))), 0)
        b = min(math.ceil(rot * math.log(orig / (low * 2 * math.pi)) / (2 * math.log(base))),
                rot - 1)
        r = np.clip((i - a) / max(b - a, 1e-3), 0, 1)
        f = f * (1 - r) + f / factor * r
    if kind == "banded":
        s = np.clip((orig * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = f * s + f / factor * (1 - s)
    return f


@pytest.mark.parametrize("kind,low,high", [("none", 1, 4), ("linear", 1, 4), ("ntk", 1, 4),
                                           ("yarn", 1, 32), ("yarn", 2, 20), ("banded", 1, 4)])
@pytest.mark.parametrize("rot,length", [(128, 1000), (4, 1), (6, 4097), (96, 33), (64, 1 << 20)])
def test_table(kind, low, high, rot, length):
    base, factor, orig = 5e5, 8.0, 4096
    t = torch.empty(length, rot, device="cuda")
    K.kvq_rope_table(t, K.make_rope_scaling(kind, base, factor, orig, low, high))
    f = _freq64(rot, kind, base, factor, orig, low, high)
    amp = 0.1 * math.log(factor) + 1 if kind == "yarn" else 1.0
    p = np.arange(length) if length <= 5000 else np.r_[0:100, length // 2:length // 2 + 100,
                                                       length - 100:length]
    a = np.outer(p, f)
    want = amp * np.concatenate([np.cos(a), np.sin(a)], 1)
    got = t[torch.from_numpy(p).cuda()].double().cpu().numpy()
    assert np.abs(got - want).max() <= 3e-7 * amp


def test_table_amplitude_and_refusals():
    t = torch.empty(8, 128, device="cuda")
    K.kvq_rope_table(t, K.make_rope_scaling(amplitude=2.5))
    assert torch.all(t[0, :64] == 2.5) and torch.all(t[0, 64:] == 0)
    for bad in [dict(base=1.0), dict(base=float("nan")), dict(kind="linear", factor=0.5),
                dict(kind="yarn", factor=4.0, orig_len=0), dict(amplitude=-1.0),
                dict(kind="banded", factor=4.0, orig_len=4096, low_turns=4, high_turns=4)]:
        with pytest.raises(K.KvqError) as e:
            K.kvq_rope_table(t, K.make_rope_scaling(**bad))
        assert e.value.code == K.KVQ_EINVAL
    for shape in [(8, 130), (8, 3)]:
        with pytest.raises(K.KvqError):
            K.kvq_rope_table(torch.empty(*shape, device="cuda"), K.make_rope_scaling())
    with pytest.raises(K.KvqError):
        K.kvq_rope_table(torch.empty(8, 2, device="cuda"), K.make_rope_scaling("ntk", factor=2.0))


# ---- rows ---------------------------------------------------------------------------------------

def _rope64(x, pos, table, style, inverse=False):
    """float64 rotation and the bound of its error."""
    rot = table.shape[1]
    t = table.double().cpu().numpy()[pos]
    c, s = t[:, None, :rot // 2], t[:, None, rot // 2:] * (-1 if inverse else 1)
    d0, d1 = _pairs(rot, style)
    y, slack = x.copy(), np.zeros_like(x)
    a, b = x[..., d0], x[..., d1]
    y[..., d0], y[..., d1] = a * c - b * s, b * c + a * s
    slack[..., d0] = np.abs(a * c) + np.abs(b * s)
    slack[..., d1] = np.abs(b * c) + np.abs(a * s)
    return y, 2.0 ** -8 * np.abs(y) + 3 * 2.0 ** -24 * slack


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 96, 64, 48, 24, 10, 2])
@pytest.mark.parametrize("n,heads", [(1, 1), (5, 4), (131, 3), (1030, 32)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rows(style, rot, n, heads, inverse):
    g = _gen(n + rot)
    table = _table(rot, 777)
    x = torch.randn(n, heads, D, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 777, (n,), generator=g, device="cuda", dtype=torch.int32)
    y = torch.empty_like(x)
    h, rope = _handle(), K.make_rope(table, style)
    K.kvq_rope(h, x, y, pos, rope, inverse=inverse)
    want, tol = _rope64(x.double().cpu().numpy(), pos.cpu().numpy(), table, style, inverse)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)
    assert torch.equal(y[..., rot:], x[..., rot:])
    z = x.clone()
    K.kvq_rope(h, z, z, pos, rope, inverse=inverse)      # in place
    assert torch.equal(z, y)
    wide = torch.full((n, heads + 3, D), 7.0, device="cuda", dtype=torch.bfloat16)
    wide[:, 1:1 + heads] = x                              # slices of wider rows
    K.kvq_rope(h, wide[:, 1:1 + heads], wide[:, 1:1 + heads], pos, rope, inverse=inverse)
    assert torch.equal(wide[:, 1:1 + heads], y)
    assert torch.all(wide[:, 0] == 7) and torch.all(wide[:, 1 + heads:] == 7)
    assert K.kvq_get_status(h) == 0


def test_inverse_is_the_gradient():
    """d/dx of sum(w * rope(x)) is rope(w, inverse): against differences of the linear map."""
    g = _gen(3)
    table, n = _table(128, 64), 9
    pos = torch.randint(0, 64, (n,), generator=g, device="cuda", dtype=torch.int32)
    h = _handle()
    for style in ("half", "interleaved"):
        rope = K.make_rope(table, style)
        w = torch.randn(n, 2, D, generator=g, device="cuda").bfloat16()
        grad = torch.empty_like(w)
        K.kvq_rope(h, w, grad, pos, rope, inverse=True)
        for d in (0, 1, 63, 64, 65, 127):
            e = torch.zeros(n, 2, D, device="cuda", dtype=torch.bfloat16)
            e[..., d] = 1
            col = torch.empty_like(e)
            K.kvq_rope(h, e, col, pos, rope)
            want = (w.double() * col.double()).sum(-1)
            # two terms, each |w| times a bf16-rounded cos or sin, and grad's own half step
            tol = 2.0 ** -8 * ((w.double() * col.double()).abs().sum(-1) + want.abs()) + 1e-6
            assert torch.all((grad[..., d].double() - want).abs() <= tol)


def test_bad_positions_leave_rows_alone():
    h, rope = _handle(), K.make_rope(_table(64, 10), "half")
    x = torch.ones(4, 2, D, device="cuda", dtype=torch.bfloat16)
    y = torch.full_like(x, 5.0)
    K.kvq_rope(h, x, y, torch.tensor([0, 10, -1, 9], device="cuda", dtype=torch.int32), rope)
    assert torch.all(y[1:3] == 5) and torch.equal(y[0], x[0]) and not torch.all(y[3] == 5)
    assert K.kvq_get_status(h) == K.KVQ_STATUS_BAD_POS


def test_rows_refusals():
    h, rope = _handle(), K.make_rope(_table(64, 10), "half")
    x = torch.zeros(4, 2, D, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(4, device="cuda", dtype=torch.int32)
    K.kvq_rope(h, x[:0], x[:0], pos[:0], rope)              # nothing to do
    with pytest.raises(ValueError):
        K.kvq_rope(h, x, x[:, :1], pos, rope)
    with pytest.raises(ValueError):
        K.kvq_rope(h, x, x, pos[:3], rope)
    with pytest.raises(ValueError):
        K.kvq_rope(h, x.transpose(1, 2), x.transpose(1, 2), pos, rope)
    with pytest.raises(TypeError):
        K.kvq_rope(h, x.float(), x.float(), pos, rope)
    with pytest.raises(TypeError):
        K.kvq_rope(h, x.cpu(), x.cpu(), pos, rope)
    flat = torch.zeros(4 * 2 * D + 1, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(K.KvqError):                         # not on 16 bytes
        K.kvq_rope(h, flat[1:].view(4, 2, D), x, pos, rope)
    with pytest.raises(K.KvqError):                         # rows that overlap
        K.kvq_rope(h, torch.as_strided(flat, (4, 2, D), (D, D, 1)), x, pos, rope)
    with pytest.raises(KeyError):
        K.make_rope(rope.table, "quarter")


# ---- appends --------------------------------------------------------------------------------------

def _paged(lens, extra=3, seed=0):
    need = [(c + 15) // 16 for c in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + extra).astype(np.int32)
    pt = np.full((len(lens), max(need)), -1, np.int32)
    o = 0
    for b, m in enumerate(need):
        pt[b, :m] = perm[o:o + m]
        o += m
    return torch.from_numpy(pt).cuda(), sum(need) + extra


def _tokens(new, lens):
    seq = np.concatenate([np.full(m, b, np.int32) for b, m in enumerate(new)])
    pos = np.concatenate([np.arange(c - m, c, dtype=np.int32) for m, c in zip(new, lens)])
    return torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()


def _unfused(kind, h, pool, pages, k, v, seq, pos, pt, rope, rpos=None):
    kr = torch.empty(k.shape, dtype=torch.bfloat16, device="cuda")
    K.kvq_rope(h, k, kr, pos if rpos is None else rpos, rope)
    fn = K.kvq_append if kind == "int2" else K.kvq_bf16_append
    fn(h, pool, pages, kr, v.contiguous(), seq, pos, pt)


@pytest.mark.parametrize("kind", ["int2", "bf16"])
@pytest.mark.parametrize("style,rot", [("half", 128), ("interleaved", 128), ("half", 96),
                                       ("interleaved", 40), ("half", 6)])
@pytest.mark.parametrize("Hkv,new,lens", [
    (1, [1], [1]), (8, [1] * 16, [17 * i + 1 for i in range(16)]),
    (3, [16, 1, 33], [16, 90, 40]), (8, [700, 129, 1], [705, 129, 64]),
    (5, [2049], [2051]), (1, [4000, 96], [4000, 101])])
def test_append_equals_rope_then_append(kind, style, rot, Hkv, new, lens):
    g = _gen(sum(new) + rot)
    n = sum(new)
    h = _handle(Hkv, Hkv, seed=5)
    rope = K.make_rope(_table(rot, max(lens)), style)
    pt, pages = _paged(lens)
    seq, pos = _tokens(new, lens)
    qkv = torch.randn(n, 2 * Hkv + 1, D, generator=g, device="cuda").bfloat16()
    k, v = qkv[:, 1:1 + Hkv], qkv[:, 1 + Hkv:]
    size = K.kvq_page_bytes(h) if kind == "int2" else K.kvq_bf16_page_bytes(h)
    pool = torch.randint(0, 255, (pages * size,), generator=g, device="cuda", dtype=torch.uint8)
    want = pool.clone()
    fn = K.kvq_append_rope if kind == "int2" else K.kvq_bf16_append_rope
    fn(h, pool, pages, k, v, seq, pos, pt, rope)
    _unfused(kind, h, want, pages, k, v, seq, pos, pt, rope)
    assert torch.equal(pool, want)
    # contiguous inputs, tokens in another order, angles of other positions
    order = torch.randperm(n, generator=g, device="cuda")
    rpos = ((pos * 7 + 3) % max(lens)).to(torch.int32)
    a, b = pool.clone(), pool.clone()
    args = (k[order].contiguous(), v[order].contiguous(), seq[order].contiguous(),
            pos[order].contiguous(), pt, rope, rpos[order].contiguous())
    fn(h, a, pages, *args)
    _unfused(kind, h, b, pages, *args)
    assert torch.equal(a, b)
    assert K.kvq_get_status(h) == 0


@pytest.mark.parametrize("Hkv", [8, 1])
@pytest.mark.parametrize("n", [151, 153, 161, 290, 304, 305, 620, 1215, 1217, 1300, 2431, 2433])
def test_int2_append_sizes(Hkv, n):
    """Token counts at which the tokens a warp takes, or the tiles a CTA takes, change."""
    g = _gen(n)
    h = _handle(Hkv, Hkv, seed=8)
    rope = K.make_rope(_table(128, n), "half")
    pt, pages = _paged([n])
    seq, pos = _tokens([n], [n])
    k, v = (torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    pool = torch.zeros(pages * K.kvq_page_bytes(h), device="cuda", dtype=torch.uint8)
    want = pool.clone()
    K.kvq_append_rope(h, pool, pages, k, v, seq, pos, pt, rope)
    _unfused("int2", h, want, pages, k, v, seq, pos, pt, rope)
    assert torch.equal(pool, want)


@pytest.mark.parametrize("kind", ["int2", "bf16"])
def test_append_skips_bad_tokens(kind):
    """Bad sequence, position, page and angle: the token is skipped (key and value), the bit is
    set, and the other tokens are stored."""
    Hkv, n = 2, 40
    h = _handle(Hkv, Hkv, seed=6)
    rope = K.make_rope(_table(64, 64), "half")
    pt, pages = _paged([48], extra=0)
    pt[0, 1] = pages                                       # positions 16..31: no such page
    g = _gen(1)
    k = torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16()
    v = torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16()
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    rpos = pos.clone()
    rpos[3], rpos[4] = 64, -5
    seq[5] = 1
    pos[6] = 48
    size = K.kvq_page_bytes(h) if kind == "int2" else K.kvq_bf16_page_bytes(h)
    pool = torch.full((pages * size,), 0x5A, device="cuda", dtype=torch.uint8)
    want = pool.clone()
    fn = K.kvq_append_rope if kind == "int2" else K.kvq_bf16_append_rope
    fn(h, pool, pages, k, v, seq, pos, pt, rope, rpos)
    assert K.kvq_get_status(h) == (K.KVQ_STATUS_BAD_PAGE | K.KVQ_STATUS_BAD_POS
                                   | K.KVQ_STATUS_BAD_SEQ)
    keep = torch.tensor([i for i in range(n) if i not in (3, 4, 5, 6) and not 16 <= i < 32],
                        device="cuda")
    _unfused(kind, h, want, pages, k[keep].contiguous(), v[keep].contiguous(), seq[keep],
             pos[keep], pt, rope)
    assert torch.equal(pool, want)


def test_append_refusals():
    h = _handle(2, 2)
    rope = K.make_rope(_table(64, 64), "half")
    pt, pages = _paged([48], extra=0)
    z = torch.zeros(4, 2, D, device="cuda", dtype=torch.bfloat16)
    i = torch.zeros(4, device="cuda", dtype=torch.int32)
    pool = torch.zeros(pages * K.kvq_bf16_page_bytes(h), device="cuda", dtype=torch.uint8)
    with pytest.raises(K.KvqError) as e:
        K.kvq_append_rope(h, pool, pages, z, z, i, i, pt, rope)
    assert e.value.code == K.KVQ_ENOTREADY
    K.kvq_bf16_append_rope(h, pool, pages, z[:0], z[:0], i[:0], i[:0], pt, rope)
    with pytest.raises(ValueError):
        K.kvq_bf16_append_rope(h, pool, pages, z[:, :1], z, i, i, pt, rope)
    with pytest.raises(ValueError):
        K.kvq_bf16_append_rope(h, pool, pages, z, z[:3], i, i, pt, rope)
    with pytest.raises(ValueError):
        K.kvq_bf16_append_rope(h, pool, pages, z, z, i[:3], i, pt, rope)
    with pytest.raises(ValueError):
        K.kvq_bf16_append_rope(h, pool, pages, z, z, i, i, pt, rope, i[:3])


def test_captured_and_on_another_stream():
    """Rotation and append captured into a graph, replayed on changed inputs."""
    Hkv, n = 2, 20
    h = _handle(Hkv, Hkv, seed=7)
    rope = K.make_rope(_table(128, 64), "half")
    pt, pages = _paged([n])
    seq, pos = _tokens([n], [n])
    g = _gen(9)
    k = torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16()
    v = torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16()
    y = torch.empty_like(k)
    pool = torch.zeros(pages * K.kvq_page_bytes(h), device="cuda", dtype=torch.uint8)

    def step():
        K.kvq_rope(h, k, y, pos, rope)
        K.kvq_append_rope(h, pool, pages, k, v, seq, pos, pt, rope)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    k.copy_(torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    want, wy = torch.zeros_like(pool), torch.empty_like(y)
    K.kvq_rope(h, k, wy, pos, rope)
    _unfused("int2", h, want, pages, k, v, seq, pos, pt, rope)
    assert torch.equal(y, wy) and torch.equal(pool, want)
