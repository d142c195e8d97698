"""Refusals of the rotary-position and rotating-append entry points that need no GPU: every check
below comes before the first CUDA call."""
import ctypes

import pytest
import torch

from rotated_int2_kv_kvq_gb300 import build, kvq as K


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(K.LIB_PATH):
        build.build()
    return K.load_library()


def test_structs_match_header(lib):
    assert ctypes.sizeof(K.KvqRopeSpec) == 24
    assert ctypes.sizeof(K.KvqRopeScaling) == 56


def test_table_refusals(lib):
    """Bad frequencies, sizes and pointers (0x1000 is never read: the call is refused before)."""
    good = dict(kind="none", base=1e4)
    at = ctypes.c_void_p(0x1000)

    def call(ptr=at, n=8, rot=128, sc=good):
        s = None if sc is None else ctypes.byref(K.make_rope_scaling(**sc))
        return lib.kvq_rope_table(ptr, n, rot, s, None)

    assert call(ptr=None) == K.KVQ_EINVAL
    assert call(ptr=ctypes.c_void_p(0x1004)) == K.KVQ_EINVAL
    assert call(sc=None) == K.KVQ_EINVAL
    for n in (0, -1):
        assert call(n=n) == K.KVQ_EINVAL
    for rot in (0, -2, 1, 127, 130):
        assert call(rot=rot) == K.KVQ_EINVAL
    nan = float("nan")
    for bad in [dict(base=1.0), dict(base=nan), dict(base=float("inf")),
                dict(kind="linear", factor=0.5), dict(kind="linear", factor=nan),
                dict(amplitude=-1.0), dict(amplitude=nan),
                dict(kind="yarn", factor=4.0, orig_len=0.0),
                dict(kind="yarn", factor=4.0, orig_len=4096.0, low_turns=0.0),
                dict(kind="banded", factor=4.0, orig_len=4096.0, low_turns=4.0, high_turns=4.0)]:
        assert call(sc=bad) == K.KVQ_EINVAL, bad
    assert call(rot=2, sc=dict(kind="ntk", factor=2.0)) == K.KVQ_EINVAL
    s = K.make_rope_scaling()
    for kind in (-1, 5):
        s.kind = kind
        assert lib.kvq_rope_table(at, 8, 128, ctypes.byref(s), None) == K.KVQ_EINVAL


def test_null_handles(lib):
    spec = K.KvqRopeSpec(0x1000, 8, 128, 0)
    at = ctypes.c_void_p(0x1000)
    assert lib.kvq_rope(None, at, 128, at, 128, 1, at, 1, ctypes.byref(spec), 0, None) == 1
    for fn in (lib.kvq_append_rope, lib.kvq_bf16_append_rope):
        assert fn(None, at, 1, at, 128, at, 128, at, at, 1, at, 1, 1, ctypes.byref(spec), None,
                  None) == 1


def test_binding_refuses_cpu_tensors(lib):
    t = torch.zeros(8, 128)
    with pytest.raises(TypeError):
        K.make_rope(t)
    with pytest.raises(ValueError):
        K.make_rope(t[0])
    with pytest.raises(KeyError):
        K.make_rope_scaling("spiral")
