"""Refusals of the prefill entry points that need no GPU: every check below comes before the first
CUDA call (a handle of its own is needed for the rest, which test_gpu_prefill.py has)."""
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


@pytest.mark.parametrize("name", ["kvq_prefill", "kvq_bf16_prefill"])
@pytest.mark.parametrize("n", [0, 1])
def test_no_handle(lib, name, n):
    at = ctypes.c_void_p(0x1000)            # never read
    assert getattr(lib, name)(None, at, 1, at, 512, at, n, at, 1, at, 1, at, at, 1 << 30,
                              None) == K.KVQ_EINVAL


@pytest.mark.parametrize("name", ["kvq_prefill_workspace_bytes", "kvq_bf16_prefill_workspace_bytes"])
def test_workspace_without_handle(lib, name):
    assert getattr(lib, name)(None, 1, 1) == 0


@pytest.mark.parametrize("fn", [K.kvq_prefill, K.kvq_bf16_prefill])
def test_tensors_on_the_cpu(fn):
    """The binding refuses a CPU tensor before the library is asked."""
    h = K.Handle(None, K.make_layout(4, 2))
    h.device = 0
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        fn(h, torch.zeros(1, dtype=torch.uint8), 1, q, i, i[None], i[:1], q, q)


@pytest.mark.parametrize("fn", [K.kvq_rope, K.kvq_append_rope, K.kvq_bf16_append_rope])
def test_rotary_tensors_on_the_cpu(fn):
    h = K.Handle(None, K.make_layout(4, 2))
    h.device = 0
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    args = (x, x, i, None) if fn is K.kvq_rope else (i, 1, x, x, i, i, i[None], None)
    with pytest.raises(TypeError):
        fn(h, *args)
