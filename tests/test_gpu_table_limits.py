"""Page tables whose rows are longer than positions can reach: every call refuses them (KVQ_EINVAL)
before it launches anything, and the appends and kvq_dequant take a row of the greatest length.  Only
the length is passed; the calls that run read the first entry of a table and no more."""
import ctypes

import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_rope import D, _handle, _table

pytestmark = pytest.mark.gpu
LONGEST = 2 ** 27 - 1


def _calls(n):
    """name -> call(max_pages) with n tokens or rows, over one small set of buffers."""
    h, lib = _handle(1, 1, seed=41), K.load_library()
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    x = torch.zeros(4, 1, D, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    rope = K.make_rope(_table(64, 8), "half")
    p, X, I = (ctypes.c_void_p(t.data_ptr()) for t in (buf, x, i))
    size = 1 << 20
    calls = {}
    for a in ("kvq_append", "kvq_bf16_append"):
        calls[a] = lambda m, a=a: getattr(lib, a)(h.ptr, p, 1, X, X, I, I, n, I, 1, m, None)
    for a in ("kvq_append_rope", "kvq_bf16_append_rope"):
        calls[a] = lambda m, a=a: getattr(lib, a)(h.ptr, p, 1, X, D, X, D, I, I, n, I, 1, m, rope,
                                                  None, None)
    for a in ("kvq_decode", "kvq_bf16_decode"):
        calls[a] = lambda m, a=a: getattr(lib, a)(h.ptr, p, 1, X, I, m, I, 1, p, p, size, 1, None)
    calls["kvq_append_decode"] = lambda m: lib.kvq_append_decode(
        h.ptr, p, 1, X, X, X, I, m, I, 1, p, p, size, 1, None)
    calls["kvq_dequant"] = lambda m: lib.kvq_dequant(h.ptr, p, 1, I, m, 0, 0, n, p, p, None)
    return h, calls, (buf, x, i, rope)


def test_too_long_rows_are_refused():
    h, calls, _keep = _calls(1)
    for name, call in calls.items():
        for m in (0, LONGEST + 1, 2 ** 28 + 1, 2 ** 31 - 1):
            assert call(m) == K.KVQ_EINVAL, (name, m)
    assert K.kvq_get_status(h) == 0


def test_longest_rows_are_taken():
    """One token at position 0."""
    h, calls, (buf, x, _i, _rope) = _calls(1)
    for name in ("kvq_append", "kvq_append_rope", "kvq_bf16_append", "kvq_bf16_append_rope",
                 "kvq_dequant"):
        x.fill_(1.5)
        buf.zero_()
        assert calls[name](LONGEST) == K.KVQ_OK, name
        if name != "kvq_dequant":
            assert int(buf.count_nonzero()) > 0, name
    assert K.kvq_get_status(h) == 0
