"""Refused arguments of the 8-bit cache's and the norms' calls (nothing is launched)."""
import ctypes
import math

import pytest
import torch

from fp8_testlib import Cache8, D, cu_of, i32
from rotated_int2_kv_kvq_gb300 import kvq as K

pytestmark = pytest.mark.gpu


def _args(good, **change):
    return [change.get(k, v) for k, v in good.items()]


def _refused(fn, good, cases, code=K.KVQ_EINVAL):
    assert fn(*_args(good)) == K.KVQ_OK
    for case in cases:
        assert fn(*_args(good, **case)) == code, case
    torch.cuda.synchronize()


def test_cache_calls():
    c = Cache8(4, 2, [40], seed=1)
    lib, at = K.load_library(), lambda t: t.data_ptr()
    cu, before = cu_of([40]), c.pool.clone()
    rows = dict(h=c.h.ptr, pool=at(c.pool), pages=c.pages, k=at(c.k), ks=256, v=at(c.v), vs=256, cu=at(cu),
                n=40, pt=at(c.pt), mp=c.pt.shape[1], sl=at(c.seq_lens), b=1, st=None)
    bad = [dict(pool=None), dict(pool=at(c.pool) + 8), dict(pages=0), dict(ks=255), dict(ks=252), dict(ks=128),
           dict(vs=0), dict(k=at(c.k) + 2), dict(v=at(c.v) + 8), dict(cu=None), dict(n=-1), dict(pt=None),
           dict(mp=0), dict(mp=(1 << 26) + 1), dict(sl=None), dict(b=0), dict(b=65536), dict(h=None)]
    _refused(lib.kvq_fp8_append, rows, bad + [dict(k=None), dict(v=None)])
    assert torch.equal(c.pool, before)                # the one good call stored the same tokens again
    out = torch.empty_like(c.k)
    rows.update(k=at(out), v=at(out))
    _refused(lib.kvq_fp8_read, rows, bad + [dict(k=None, v=None)])
    assert lib.kvq_fp8_append(*_args(rows, n=0, pool=None)) == K.KVQ_OK       # no rows: nothing is looked at

    q, o = c.randn(1, 4), torch.empty(1, 4, D, device="cuda")
    size = K.kvq_fp8_workspace_bytes(c.h, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    good = dict(h=c.h.ptr, pool=at(c.pool), pages=c.pages, q=at(q), pt=at(c.pt), mp=c.pt.shape[1],
                sl=at(c.seq_lens), b=1, w=0, s=0, out=at(o), ws=at(ws), size=size, st=None)
    _refused(lib.kvq_fp8_decode, good, [
        dict(pool=None), dict(pages=0), dict(q=None), dict(q=at(q) + 2), dict(pt=None), dict(mp=0), dict(sl=None),
        dict(b=0), dict(b=65536), dict(w=-1), dict(s=-1), dict(out=None), dict(out=at(o) + 2), dict(ws=None),
        dict(ws=at(ws) + 16)])
    assert lib.kvq_fp8_decode(*_args(good, size=size - 1)) == K.KVQ_ENOSPACE
    assert K.kvq_fp8_workspace_bytes(c.h, 0) == 0 and K.kvq_fp8_workspace_bytes(c.h, 65536) == 0
    assert K.kvq_get_status(c.h) == 0


def test_prefill_calls():
    c = Cache8(4, 2, [40], seed=4)
    lib, at = K.load_library(), lambda t: t.data_ptr()
    q, cu = c.randn(8, 4), cu_of([8])
    out = torch.empty_like(q)
    size = K.kvq_fp8_prefill_workspace_bytes(c.h, 1, 8)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    good = dict(h=c.h.ptr, pool=at(c.pool), pages=c.pages, q=at(q), qs=512, cu=at(cu), n=8, pt=at(c.pt),
                mp=c.pt.shape[1], sl=at(c.seq_lens), b=1, w=0, s=0, out=at(out), ws=at(ws), size=size, st=None)
    _refused(lib.kvq_fp8_prefill, good, [
        dict(h=None), dict(pool=None), dict(pool=at(c.pool) + 8), dict(pages=0), dict(q=None), dict(q=at(q) + 8),
        dict(qs=511), dict(qs=504), dict(cu=None), dict(n=-1), dict(pt=None), dict(mp=0), dict(mp=(1 << 26) + 1),
        dict(sl=None), dict(b=0), dict(b=65536), dict(w=-1), dict(s=-1), dict(out=None), dict(out=at(out) + 8),
        dict(ws=None), dict(ws=at(ws) + 64)])
    assert lib.kvq_fp8_prefill(*_args(good, size=size - 1)) == K.KVQ_ENOSPACE
    assert lib.kvq_fp8_prefill(*_args(good, n=0, pool=None)) == K.KVQ_OK      # no rows: nothing is looked at
    assert K.kvq_fp8_prefill_workspace_bytes(c.h, 0, 8) == 0 and K.kvq_fp8_prefill_workspace_bytes(c.h, 1, -1) == 0
    for bad in (dict(window=-1), dict(sinks=-2 ** 32), dict(window=-2 ** 32)):
        with pytest.raises(RuntimeError):
            c.prefill(q, [8], **bad)
        with pytest.raises(RuntimeError):
            c.decode(c.randn(1, 4), **bad)
    for bad in (dict(out=out[:7]), dict(cu=i32([0, 8, 8])), dict(q=c.randn(8, 2))):
        with pytest.raises(ValueError):
            c.prefill(bad.pop("q", q), [8], **bad)
    assert K.kvq_get_status(c.h) == 0


def test_norm_calls():
    h = K.kvq_create(K.make_layout(4, 2))
    lib, at = K.load_library(), lambda t: t.data_ptr()
    q, k = (torch.ones(3, n, D, dtype=torch.bfloat16, device="cuda") for n in (4, 2))
    yq, yk, gq, gk = (torch.empty_like(t) for t in (q, k, q, k))
    table, pos, w = torch.ones(8, 64, device="cuda"), i32([0, 1, 2]), torch.ones(D, device="cuda")
    spec = lambda **kw: ctypes.byref(K.KvqRopeSpec(kw.get("t", at(table)), kw.get("n", 8), kw.get("rot", 64),
                                                   kw.get("style", 0)))
    good = dict(h=h.ptr, q=at(q), qs=512, k=at(k), ks=256, yq=at(yq), yqs=512, yk=at(yk), yks=256, wq=at(w),
                wk=None, eps=1e-6, pos=at(pos), n=3, rope=spec(), st=None)
    bad = [dict(h=None), dict(q=None, k=None), dict(qs=504), dict(ks=257), dict(yq=None), dict(yk=at(yk) + 2),
           dict(yqs=0), dict(wq=at(w) + 2), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(pos=None),
           dict(n=-1), dict(rope=None), dict(rope=spec(rot=63)), dict(rope=spec(rot=130)), dict(rope=spec(n=0)),
           dict(rope=spec(style=2)), dict(rope=spec(t=at(table) + 4)), dict(rope=spec(t=None))]
    _refused(lib.kvq_norm_rope, good, bad)
    size = K.kvq_norm_rope_backward_workspace_bytes(h, 3)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    good = dict(h=h.ptr, q=at(q), qs=512, k=at(k), ks=256, dyq=at(yq), dyqs=512, dyk=at(yk), dyks=256, yq=at(gq),
                yqs=512, yk=at(gk), yks=256, wq=at(w), wk=None, dwq=at(w), dwk=None, eps=1e-6, pos=at(pos), n=3,
                rope=spec(), ws=at(ws), size=size, st=None)
    _refused(lib.kvq_norm_rope_backward, good, bad + [dict(dyq=None), dict(dyks=8), dict(dwq=at(w) + 1),
                                                      dict(ws=None), dict(ws=at(ws) + 64)])
    assert lib.kvq_norm_rope_backward(*_args(good, size=size - 1)) == K.KVQ_ENOSPACE
    for bad in (dict(dwq=at(w) + 2), dict(dwk=at(w) + 1)):        # no rows: the sums are written all the same
        assert lib.kvq_norm_rope_backward(*_args(good, n=0, **bad)) == K.KVQ_EINVAL
    assert K.kvq_get_status(h) == 0


def test_binding_shapes():
    c = Cache8(4, 2, [40], seed=2)
    q, o = c.randn(1, 4), torch.empty(1, 4, D, device="cuda")
    ws = torch.empty(K.kvq_fp8_workspace_bytes(c.h, 1), dtype=torch.uint8, device="cuda")
    cu, sl = cu_of([40]), c.seq_lens
    decode = lambda **kw: K.kvq_fp8_decode(*_args(dict(h=c.h, pool=c.pool, pages=c.pages, q=q, pt=c.pt, sl=sl,
                                                       out=o, ws=ws), **kw))
    append = lambda **kw: K.kvq_fp8_append(*_args(dict(h=c.h, pool=c.pool, pages=c.pages, k=c.k, v=c.v, cu=cu,
                                                       pt=c.pt, sl=sl), **kw))
    decode()
    append()
    for bad in (dict(q=q[:, :2].contiguous()), dict(out=o[:, :1].contiguous()), dict(sl=cu), dict(pt=c.pt[0]),
                dict(pages=c.pages + 1), dict(q=c.randn(2, 4))):
        with pytest.raises(ValueError):
            decode(**bad)
    for bad in (dict(k=c.randn(40, 4)), dict(v=c.v[:39]), dict(cu=sl), dict(sl=cu), dict(pages=c.pages + 1),
                dict(k=c.k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            append(**bad)
    for bad in (dict(k=c.k.float()), dict(pool=c.pool.view(torch.int8)), dict(cu=cu.long())):
        with pytest.raises(TypeError):
            append(**bad)
    assert K.kvq_get_status(c.h) == 0
