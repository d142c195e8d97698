"""Refusals of the 8-bit cache's and the norms' entry points that need no GPU: null handles, and
the binding's own checks."""
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


def test_constants_match_header(lib):
    import re

    with open(f"{build.INCLUDE}/kvq.h") as f:
        m = re.search(r"#define\s+KVQ_FP8_RECORD_BYTES\s+(\d+)", f.read())
    assert int(m.group(1)) == K.FP8_RECORD_BYTES == 4112


def test_null_handles(lib):
    at, spec = ctypes.c_void_p(0x1000), ctypes.byref(K.KvqRopeSpec(0x1000, 8, 128, 0))
    assert lib.kvq_fp8_page_bytes(None) == 0
    assert lib.kvq_fp8_workspace_bytes(None, 1) == 0
    assert lib.kvq_norm_rope_backward_workspace_bytes(None, 1) == 0
    assert lib.kvq_norm_rope(None, at, 128, at, 128, at, 128, at, 128, None, None, 1e-6, at, 1, spec,
                             None) == K.KVQ_EINVAL
    assert lib.kvq_norm_rope_backward(None, at, 128, at, 128, at, 128, at, 128, at, 128, at, 128, None,
                                      None, None, None, 1e-6, at, 1, spec, at, 1 << 20,
                                      None) == K.KVQ_EINVAL
    for fn in (lib.kvq_fp8_append, lib.kvq_fp8_read):
        assert fn(None, at, 1, at, 128, at, 128, at, 1, at, 1, at, 1, None) == K.KVQ_EINVAL
    assert lib.kvq_fp8_decode(None, at, 1, at, at, 1, at, 1, 0, 0, at, at, 1 << 30,
                              None) == K.KVQ_EINVAL
    assert lib.kvq_fp8_prefill_workspace_bytes(None, 1, 1) == 0
    assert lib.kvq_fp8_prefill(None, at, 1, at, 512, at, 1, at, 1, at, 1, 0, 0, at, at, 1 << 30,
                               None) == K.KVQ_EINVAL


def test_window_and_sinks_fit_a_c_int():
    most = 2 ** 31 - 1
    assert K._span(7, 3) == [7, 3] and K._span(0, 0) == [0, 0] and K._span(most, most) == [most, most]
    assert K._span(2 ** 32, 2 ** 40) == [most, most]         # not 0, as the low bits say
    assert K._span(-2 ** 32, -5) == [-1, -1]                 # refused by the call


class _Handle:
    """What the binding reads of a handle (no call reaches the library)."""
    ptr, device = None, 0

    def __init__(self, H=4, Hkv=2):
        self.layout = K.make_layout(H, Hkv)


def test_binding_refuses_cpu_tensors(lib):
    h, rows, i = _Handle(), torch.zeros(3, 2, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    pt, buf = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    for fn in (K.kvq_fp8_append, K.kvq_fp8_read):
        with pytest.raises(TypeError):
            fn(h, buf, 1, rows, rows, i, pt, i)
    with pytest.raises(TypeError):
        K.kvq_fp8_decode(h, buf, 1, rows, pt, i, rows.float(), buf)
    with pytest.raises(TypeError):
        K.kvq_fp8_prefill(h, buf, 1, rows, i, pt, i, rows, buf)
    with pytest.raises(TypeError):
        K.kvq_norm_rope(h, rows, rows, rows, rows, None, None, 1e-6, i, None)
    with pytest.raises(ValueError):
        K.kvq_norm_rope(h, None, None, None, None, None, None, 1e-6, i, None)
    with pytest.raises(ValueError):
        K.kvq_norm_rope_backward(h, None, None, None, None, None, None, None, None, None, None, 1e-6, i,
                                 None, buf)
    with pytest.raises(ValueError):
        K.kvq_fp8_read(h, buf, 1, None, None, i, pt, i)
