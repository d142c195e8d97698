"""The INT2 append's division of tokens into rounds and shares: one call stores what calls of a few
tokens each store, byte for byte, at counts around the borders of rounds, shares and tiles."""
import pytest
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K
from test_gpu_rope import D, _gen, _handle, _paged, _tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv,counts", [
    (1, (1, 7, 8, 9, 1215, 1216, 1217, 2431, 2432, 2433, 2440, 19457)),
    (3, (405, 406, 811, 3264, 3265, 3271, 6529)),
    (8, (1, 8, 9, 152, 153, 160, 1208, 1216, 1217, 1224, 1225, 2367, 2432, 2433)),
    (64, (1, 8, 19, 20, 27, 152, 192, 193, 200, 383, 385, 577))])
def test_one_call_equals_many(Hkv, counts):
    h = _handle(Hkv, Hkv, seed=31)
    size = K.kvq_page_bytes(h)
    for n in counts:
        g = _gen(n)
        pt, pages = _paged([n])
        seq, pos = _tokens([n], [n])
        k, v = (torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        pools = [torch.full((pages * size,), 0x5A, device="cuda", dtype=torch.uint8) for _ in range(2)]
        K.kvq_append(h, pools[0], pages, k, v, seq, pos, pt)
        for a in range(0, n, 61):
            part = slice(a, min(a + 61, n))
            K.kvq_append(h, pools[1], pages, k[part], v[part], seq[part], pos[part], pt)
        assert torch.equal(*pools), n
    assert K.kvq_get_status(h) == 0
