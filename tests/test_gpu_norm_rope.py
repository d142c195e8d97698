"""kvq_norm_rope and its backward pass against the formulas in float64.

Tolerances: a result is rounded once to bf16 (half a step: 2^-8 of it); the fp32 arithmetic before
that, a sum of 128 squares in chains of 16 and some ten more operations, stays below 2^-19 of the
magnitudes that enter it.  dw: fp32 sums, below 2^-20 + rows * 2^-24 of the sum of magnitudes."""
import math

import numpy as np
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu
D = 128


def table_of(length, rot, amplitude=1.0):
    a = torch.arange(length, dtype=torch.float64)[:, None] * 1e4 ** (
        -2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)[None]
    return (amplitude * torch.cat([a.cos(), a.sin()], 1)).float().cuda()


def parts(x, rot, style):
    half = rot // 2
    a = slice(0, half) if style == "half" else slice(0, rot, 2)
    b = slice(half, rot) if style == "half" else slice(1, rot, 2)
    return x[..., a], x[..., b], a, b


def turned(x, table, pos, style, back=False):
    """Rows turned by their positions (back: the transposed map), and the magnitudes that enter."""
    rot = table.shape[1]
    t = table.double()[pos.long()][:, None]
    c, s = t[..., :rot // 2], t[..., rot // 2:] * (-1 if back else 1)
    y, mag = x.clone(), x.abs()
    p, q, a, b = parts(x, rot, style)
    y[..., a], y[..., b] = p * c - q * s, q * c + p * s
    mag[..., a] = mag[..., b] = (p.abs() + q.abs()) * (c.abs() + s.abs())
    return y, mag


def forward(x, w, eps, table, pos, style):
    x = x.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return turned(x * r * (1.0 if w is None else w.double()), table, pos, style)


def backward(x, dy, w, eps, table, pos, style):
    x = x.double()
    w = torch.ones(D, device="cuda").double() if w is None else w.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    dn, mag = turned(dy.double(), table, pos, style, back=True)
    xh, g = x * r, dn * w
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    dmag = r * (mag * w.abs() + xh.abs() * (mag * w.abs() * xh.abs()).mean(-1, keepdim=True))
    return dx, dmag, (dn * xh).sum((0, 1)), (mag * xh.abs()).sum((0, 1))


class Case:
    def __init__(self, H, Hkv, n, rot, style, fused=False, weight=True, eps=1e-6, seed=0, size=2.0, length=500):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.h = K.kvq_create(K.make_layout(H, Hkv))
        self.H, self.Hkv, self.n, self.style, self.eps = H, Hkv, n, style, eps
        x = (size * rn(n, H + 2 * Hkv, D)).bfloat16()
        self.q, self.k = x[:, :H], x[:, H:H + Hkv]
        if not fused:
            self.q, self.k = self.q.contiguous(), self.k.contiguous()
        self.wq, self.wk = [1 + 0.3 * rn(D) if weight else None for _ in range(2)]
        self.dq, self.dk = rn(n, H, D).bfloat16(), rn(n, Hkv, D).bfloat16()
        self.table = table_of(length, rot)
        self.rope = K.make_rope(self.table, style)
        self.pos = torch.randint(0, length, (n,), generator=g, device="cuda", dtype=torch.int32)

    def forward(self, q_out=None, k_out=None, pos=None):
        q_out = torch.full((self.n, self.H, D), 9.0, dtype=torch.bfloat16, device="cuda") if q_out is None else q_out
        k_out = torch.full((self.n, self.Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda") if k_out is None else k_out
        K.kvq_norm_rope(self.h, self.q, self.k, q_out, k_out, self.wq, self.wk, self.eps,
                        self.pos if pos is None else pos, self.rope)
        return q_out, k_out

    def backward(self, pos=None, dx=None):
        out = [torch.full_like(t, 9.0) for t in (self.dq, self.dk)] if dx is None else dx
        dw = [torch.full((D,), 9.0, device="cuda") for _ in range(2)]
        ws = torch.full((K.kvq_norm_rope_backward_workspace_bytes(self.h, self.n),), 255, dtype=torch.uint8,
                        device="cuda")
        K.kvq_norm_rope_backward(self.h, self.q, self.k, self.dq, self.dk, *out, self.wq, self.wk, *dw,
                                 self.eps, self.pos if pos is None else pos, self.rope, ws)
        return out + dw

    def check(self):
        for got, x, w in zip(self.forward(), (self.q, self.k), (self.wq, self.wk)):
            want, mag = forward(x, w, self.eps, self.table, self.pos, self.style)
            r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + self.eps)
            _, mag = turned(x.double().abs() * r * (1.0 if w is None else w.double().abs()), self.table, self.pos,
                            self.style)
            assert torch.all((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * mag)
        dq, dk, dwq, dwk = self.backward()
        for got, dw, x, dy, w in ((dq, dwq, self.q, self.dq, self.wq), (dk, dwk, self.k, self.dk, self.wk)):
            want, mag, want_w, mag_w = backward(x, dy, w, self.eps, self.table, self.pos, self.style)
            assert torch.all((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * mag)
            rows = x.shape[0] * x.shape[1]
            assert torch.all((dw.double() - want_w).abs() <= (2.0 ** -20 + rows * 2.0 ** -24) * mag_w)
        assert K.kvq_get_status(self.h) == 0


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 64, 96, 16, 8, 2, 20, 126])
@pytest.mark.parametrize("H,Hkv,n", [(1, 1, 1), (4, 1, 3), (6, 3, 17), (32, 8, 5), (5, 5, 33)])
def test_small(style, rot, H, Hkv, n):
    Case(H, Hkv, n, rot, style, seed=rot + n).check()


@pytest.mark.parametrize("H,Hkv,n,rot,style", [(32, 8, 1000, 128, "half"), (8, 2, 3001, 64, "interleaved"),
                                               (1, 1, 20001, 128, "half"), (64, 64, 65, 34, "half")])
def test_large(H, Hkv, n, rot, style):
    Case(H, Hkv, n, rot, style, fused=True, seed=n).check()


@pytest.mark.parametrize("rot,style", [(128, "half"), (64, "interleaved"), (20, "half"), (2, "interleaved")])
@pytest.mark.parametrize("H,Hkv,n", [(5, 5, 700), (6, 3, 401), (10, 5, 203), (9, 9, 101)])
def test_heads_that_leave_groups_short(rot, style, H, Hkv, n):
    """Enough tokens for two rows a group, heads that are no multiple of what a warp takes."""
    Case(H, Hkv, n, rot, style, fused=True, seed=rot + n).check()


@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("size,eps", [(1e-4, 1e-6), (1e-4, 0.0), (3e4, 1e-5), (1.0, 0.5), (1e-15, 1e-6)])
def test_sizes(weight, size, eps):
    Case(4, 2, 9, 128, "half", weight=weight, eps=eps, size=size).check()


def test_the_formula_against_differences():
    """The gradients of the float64 forward by central differences (no kernel)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)
    x, dy, w = rn(3, 2, D), rn(3, 2, D), 1 + 0.3 * rn(D)
    table, pos = table_of(50, 64, 1.3), torch.tensor([0, 7, 49], device="cuda")
    dx, _, dw, _ = backward(x, dy, w, 1e-2, table, pos, "interleaved")
    f = lambda x, w: float((forward(x, w, 1e-2, table, pos, "interleaved")[0] * dy).sum())
    for at in [(0, 0, 0), (1, 1, 63), (2, 0, 64), (2, 1, 127)]:
        e = torch.zeros_like(x)
        e[at] = 1e-5
        assert abs((f(x + e, w) - f(x - e, w)) / 2e-5 - float(dx[at])) <= 1e-7
        e = torch.zeros_like(w)
        e[at[2]] = 1e-5
        assert abs((f(x, w + e) - f(x, w - e)) / 2e-5 - float(dw[at[2]])) <= 1e-7


def test_in_place_and_one_side():
    for fused in (False, True):
        c = Case(8, 2, 21, 128, "half", fused=fused)
        q, k = c.forward()
        dq, dk, dwq, dwk = c.backward()
        # queries alone, keys alone
        only = torch.empty_like(q)
        K.kvq_norm_rope(c.h, c.q, None, only, None, c.wq, None, c.eps, c.pos, c.rope)
        assert torch.equal(only, q)
        only = torch.empty_like(k)
        K.kvq_norm_rope(c.h, None, c.k, None, only, None, c.wk, c.eps, c.pos, c.rope)
        assert torch.equal(only, k)
        ws = torch.empty(K.kvq_norm_rope_backward_workspace_bytes(c.h, c.n), dtype=torch.uint8, device="cuda")
        got, gw = torch.empty_like(dk), torch.empty_like(dwk)
        K.kvq_norm_rope_backward(c.h, None, c.k, None, c.dk, None, got, None, c.wk, None, gw, c.eps, c.pos,
                                 c.rope, ws)
        assert torch.equal(got, dk) and torch.equal(gw, dwk)
        K.kvq_norm_rope_backward(c.h, c.q, None, c.dq, None, got.new_empty(dq.shape), None, c.wq, None, None, None,
                                 c.eps, c.pos, c.rope, ws)
        # gradients over their inputs, rows over theirs
        a, b = c.dq.clone(), c.dk.clone()
        c.dq, c.dk = a, b
        c.backward(dx=[a, b])
        assert torch.equal(a, dq) and torch.equal(b, dk)
        c.forward(c.q, c.k)
        assert torch.equal(c.q, q) and torch.equal(c.k, k)


def test_bad_positions():
    """Their rows stay as they were and add nothing to dw."""
    c = Case(4, 2, 9, 128, "half")
    pos = c.pos.clone()
    pos[2], pos[5] = -1, 500
    q, k = c.forward(pos=pos)
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_POS
    want = c.forward()
    keep = torch.tensor([i not in (2, 5) for i in range(9)], device="cuda")
    assert torch.equal(q[keep], want[0][keep]) and (q[~keep] == 9).all() and (k[~keep] == 9).all()
    dq, dk, dwq, dwk = c.backward(pos=pos)
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_POS and (dq[~keep] == 9).all() and (dk[~keep] == 9).all()
    _, _, want_w, mag = backward(c.q[keep], c.dq[keep], c.wq, c.eps, c.table, c.pos[keep], "half")
    assert torch.all((dwq.double() - want_w).abs() <= 2.0 ** -19 * mag)


def test_zero_rows_and_no_rows():
    c = Case(2, 1, 4, 128, "half")
    c.q[1] = 0
    q, _ = c.forward()
    assert (q[1] == 0).all()
    dq = c.backward()[0]
    want = backward(c.q, c.dq, c.wq, c.eps, c.table, c.pos, "half")[0]
    assert torch.all((dq.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * want.abs().amax())
    c = Case(2, 1, 0, 128, "half")
    c.forward()
    assert all((x == 0).all() for x in c.backward()[2:])


def test_nonfinite_rows_stay_their_own():
    c = Case(4, 2, 6, 64, "half")
    want = c.forward()
    c.q[3, 1, 100] = float("nan")
    c.k[0, 0, 0] = float("inf")
    q, k = c.forward()
    bad = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    bad[3, 1] = True
    assert torch.isnan(q[bad]).all() and torch.equal(q[~bad], want[0][~bad])
    assert torch.equal(k[1:], want[1][1:]) and torch.equal(k[0, 1], want[1][0, 1])


def test_same_bits_streams_graphs():
    c = Case(32, 8, 700, 128, "half", fused=True)
    want = [*c.forward(), *c.backward()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = [*c.forward(), *c.backward()]
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.zeros_like(t) for t in want]
    ws = torch.empty(K.kvq_norm_rope_backward_workspace_bytes(c.h, c.n), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kvq_norm_rope(c.h, c.q, c.k, out[0], out[1], c.wq, c.wk, c.eps, c.pos, c.rope)
        K.kvq_norm_rope_backward(c.h, c.q, c.k, c.dq, c.dk, out[2], out[3], c.wq, c.wk, out[4], out[5],
                                 c.eps, c.pos, c.rope, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_agrees_with_norm_then_rotation():
    """kvq_rope of the rounded norm differs by that rounding only."""
    c = Case(4, 2, 50, 128, "half")
    q, _ = c.forward()
    x = c.q.double()
    n = (x / torch.sqrt(x.square().mean(-1, keepdim=True) + c.eps) * c.wq.double()).bfloat16()
    y = torch.empty_like(n)
    K.kvq_rope(c.h, n, y, c.pos, c.rope)
    mag = turned(n.double(), c.table, c.pos, "half")[1]
    assert torch.all((q.double() - y.double()).abs() <= 2.0 ** -7 * q.double().abs() + 2.0 ** -7 * mag)
