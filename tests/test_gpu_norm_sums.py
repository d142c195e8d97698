"""The weights' gradients of kvq_norm_rope_backward over many rows.

dw_d = sum of dn_d xh_d over the rows (token, head).  A term's error: xh = x r to 2^-20 (a sum of 128 squares in
chains of 8 and four steps more, 1 / sqrt within 2^-22), dn = p c +- q s to 2^-22 of |p c| + |q s|, and two
roundings more: below 2^-19 of (|p c| + |q s|) |xh|.  The sum: a lane adds the rows of its group one after the
other (at most 64 at these sizes), then some 24 steps of trees and chains follow, each at most 2^-24 of the sum of
magnitudes: together below (64 + 24) 2^-24 < 2^-17.5.  So the tolerance is 2^-17 of that sum, far below what one
CTA's rows make of the gradients when all terms have one sign."""
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_norm_rope import Case, D, parts, turned

pytestmark = pytest.mark.gpu


def weight_gradient(x, dy, table, pos, style, eps):
    """dw and the sum of its terms' magnitudes, float64."""
    x, dy = x.double(), dy.double()
    xh = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    dn, _ = turned(dy, table, pos, style, back=True)
    rot = table.shape[1]
    t = table.double()[pos.long()][:, None]
    c, s = t[..., :rot // 2].abs(), t[..., rot // 2:].abs()
    mag = dy.abs()
    p, q, a, b = parts(dy.abs(), rot, style)
    mag[..., a], mag[..., b] = p * c + q * s, q * c + p * s
    return (dn * xh).sum((0, 1)), (mag * xh.abs()).sum((0, 1))


def along(x, table, pos, style, eps):
    """A gradient that has every term of dw positive: the rotated normalised row."""
    x = x.double()
    return turned(x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps), table, pos, style)[0].bfloat16()


SIZES = [(32, 8, 1000, 128, "half"), (8, 2, 3001, 64, "interleaved"), (1, 1, 20001, 128, "half"),
         (5, 5, 700, 20, "half"), (2, 1, 4099, 2, "interleaved"), (32, 8, 4099, 128, "half")]


@pytest.mark.parametrize("coherent", [True, False])
@pytest.mark.parametrize("H,Hkv,n,rot,style", SIZES)
def test_many_rows(H, Hkv, n, rot, style, coherent):
    c = Case(H, Hkv, n, rot, style, fused=True, seed=n + rot)
    if coherent:
        c.dq, c.dk = (along(x, c.table, c.pos, style, c.eps) for x in (c.q, c.k))
    got = c.backward()[2:]
    for dw, x, dy in ((got[0], c.q, c.dq), (got[1], c.k, c.dk)):
        want, mag = weight_gradient(x, dy, c.table, c.pos, style, c.eps)
        tol = 2.0 ** -17 * mag
        if coherent:        # what one of a thousand parts adds is far above the tolerance
            assert torch.all(want / 1000 > 50 * tol)
        assert torch.all((dw.double() - want).abs() <= tol), float(((dw.double() - want).abs() / mag).max())
    assert K.kvq_get_status(c.h) == 0


def test_a_bad_position_among_many():
    """Its rows add nothing, wherever in a group they fall."""
    c = Case(8, 2, 3001, 128, "half", fused=True, seed=1)
    c.dq, c.dk = (along(x, c.table, c.pos, "half", c.eps) for x in (c.q, c.k))
    pos = c.pos.clone()
    bad = torch.randperm(3001, generator=torch.Generator().manual_seed(3))[:40].cuda()
    pos[bad] = -1
    got = c.backward(pos=pos)[2:]
    assert K.kvq_get_status(c.h) == K.KVQ_STATUS_BAD_POS
    keep = torch.ones(3001, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for dw, x, dy in ((got[0], c.q, c.dq), (got[1], c.k, c.dk)):
        want, mag = weight_gradient(x[keep], dy[keep], c.table, c.pos[keep], "half", c.eps)
        assert torch.all((dw.double() - want).abs() <= 2.0 ** -17 * mag)


@pytest.mark.parametrize("n", [0, 5])
def test_a_missing_side_keeps_its_gradient(n):
    """Without queries (keys), the other arguments of that side are not looked at, with no tokens either."""
    c = Case(4, 2, n, 128, "half")
    ws = torch.empty(K.kvq_norm_rope_backward_workspace_bytes(c.h, n), dtype=torch.uint8, device="cuda")
    for q, k in ((None, c.k), (c.q, None)):
        dw = [torch.full((D,), 9.0, device="cuda") for _ in range(2)]
        dq, dk = (None if x is None else torch.empty_like(x) for x in (q, k))
        K.kvq_norm_rope_backward(c.h, q, k, None if q is None else c.dq, None if k is None else c.dk, dq, dk, c.wq, c.wk,
                                 *dw, c.eps, c.pos, c.rope, ws)
        assert (dw[0 if q is None else 1] == 9).all() and not (dw[1 if q is None else 0] == 9).any()
        assert n > 0 or (dw[1 if q is None else 0] == 0).all()
