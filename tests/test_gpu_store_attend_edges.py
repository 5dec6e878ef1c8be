"""Attention over stores (fathom_store_attend, _batched, _partial) at its edges: a query that is not a number."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from bit_plane_key_b200 import fathom as F  # noqa: E402
from test_gpu_store_attend import make_store, queries  # noqa: E402

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,Hkv,d,G", [(40, 2, 128, 4), (900, 2, 64, 2), (4096, 1, 128, 1), (3000, 2, 256, 8), (9300, 4, 128, 8),
                                       (60000, 1, 64, 4), (50000, 8, 128, 4)])
def test_a_nan_query_shows_whatever_the_split(n, Hkv, d, G, dtype):
    """Rows of one CTA, of a cluster and of several CTAs end alike: NaN for the head whose query holds one, the same bits
    as without it for every other head."""
    ks, vs = make_store(n, Hkv, d, n), make_store(n, Hkv, d, n + 1)
    q = queries((Hkv * G, d), d, dtype)
    want = F.store_attend(ks, vs, q)
    sick = q.clone()
    h = Hkv * G - 1
    sick[h, d // 3] = math.nan
    out = F.store_attend(ks, vs, sick)
    assert out[h].isnan().all()
    assert torch.equal(out[:h], want[:h])
    parts = F.store_attend_partial(ks, vs, sick, n)
    assert parts[h, :d].isnan().all() and parts[h, d + 1].isnan() and torch.isfinite(parts[:h]).all()
    both = F.store_attend_batched([ks, ks], [vs, vs], torch.stack([q, sick])[:, None])
    assert both[1, 0, h].isnan().all() and torch.isfinite(both[0]).all() and torch.isfinite(both[1, 0, :h]).all()


def test_a_nan_query_that_sees_no_key_gets_zero():
    ks, vs = make_store(2, 1, 64, 1), make_store(2, 1, 64, 2)
    q = queries((5, 2, 64), 3)
    q[0] = math.nan
    assert (F.store_attend(ks, vs, q)[:3] == 0).all()
