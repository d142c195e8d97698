"""Calls of the 8-bit path and the norms back to back on shared workspaces: the bits of every step, not of the last
one alone, are those of a run that waits for the GPU between the calls."""
import pytest
import torch

from fp8_testlib import Cache8, D, cu_of, i32
from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu


def in_a_graph(run):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    return graph, got


def test_every_decode_sees_its_own_append():
    """Each step's append and decode, on one workspace, through a page's end and a raised scale."""
    steps = 24
    c = Cache8(8, 2, [60, 33, 16], seed=1, extra=9)
    used = set(c.pt[c.pt >= 0].tolist())
    spare = [p for p in range(c.pages) if p not in used]
    pt = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
    pt[:, :4] = c.pt
    for b in range(3):
        held = (c.lens[b] + 15) // 16
        pt[b, held:held + 2] = i32([spare.pop(), spare.pop()])
    c.pt = pt
    ws = torch.empty(K.kvq_fp8_workspace_bytes(c.h, 3), dtype=torch.uint8, device="cuda")
    cu, start = cu_of([1, 1, 1]), c.pool.clone()
    q = [c.randn(3, 8) for _ in range(steps)]
    kv = [(c.randn(3, 2, scale=1.0 + i), c.randn(3, 2, scale=1.0 + i % 7)) for i in range(steps)]
    at = [i32([x + 1 + i for x in c.lens]) for i in range(steps)]

    def run(after=lambda: None):
        c.pool.copy_(start)
        after()
        outs = []
        for i in range(steps):
            out = torch.empty(3, 8, D, device="cuda")
            after()
            K.kvq_fp8_append(c.h, c.pool, c.pages, *kv[i], cu, c.pt, at[i])
            after()
            K.kvq_fp8_decode(c.h, c.pool, c.pages, q[i], c.pt, at[i], out, ws, window=40 if i % 2 else 0, sinks=3)
            after()
            outs.append(out)
        return outs

    want = run(torch.cuda.synchronize)
    for a, b in zip(want, want[1:]):
        assert not torch.equal(a, b)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    graph, got = in_a_graph(run)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and K.kvq_get_status(c.h) == 0


@pytest.mark.parametrize("n", [3, 700])
def test_gradients_back_to_back(n):
    """Steps of forward, a torch kernel on its result, backward and an update of the weights from dw right behind
    it, which the next step reads; one workspace."""
    steps, H, Hkv = 6, 8, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    h = K.kvq_create(K.make_layout(H, Hkv))
    rope = K.make_rope(rn(n, D), "half")
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    q, k = rn(n, H, D).bfloat16(), rn(n, Hkv, D).bfloat16()
    w0 = [1 + 0.3 * rn(D) for _ in range(2)]
    ws = torch.empty(K.kvq_norm_rope_backward_workspace_bytes(h, n), dtype=torch.uint8, device="cuda")

    def run(after=lambda: None):
        got, w = [], [x.clone() for x in w0]
        dw = [torch.empty(D, device="cuda") for _ in range(2)]
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        x, y = q.clone(), k.clone()
        after()
        for _ in range(steps):
            yq, yk = torch.empty_like(q), torch.empty_like(k)
            K.kvq_norm_rope(h, x, y, yq, yk, *w, 1e-6, pos, rope)
            after()
            yq.mul_(0.5)
            yk.add_(y)
            after()
            K.kvq_norm_rope_backward(h, x, y, yq, yk, dq, dk, *w, *dw, 1e-6, pos, rope, ws)
            after()
            for a, b in zip(w, dw):
                a.sub_(b, alpha=1e-3 / n)
            after()
            x.sub_(dq, alpha=0.1)
            y.sub_(dk, alpha=0.1)
            after()
            got += [yq, yk, dq.clone(), dk.clone(), dw[0].clone(), dw[1].clone()]
            after()
        return got + w

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    graph, got = in_a_graph(run)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and K.kvq_get_status(h) == 0
