"""fathom_append_rows on long inputs: the CTAs that take groups of 16 blocks, which serve prompts, against a pack of
the same rows, bit for bit.  The launch takes them from 296 CTAs of 16 blocks on; every case here has more."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from bit_plane_key_b200 import fathom as F  # noqa: E402
from test_gpu_rows import _row_cache, _same  # noqa: E402

DEV = torch.device("cuda:0")


def _ctas(Hkv, d, n_old, n_new, sides):
    """CTAs of 16 blocks that the call has work for."""
    groups = (-(-n_new // 64) + 15) // 16 - n_old // 64 // 16
    return groups * Hkv * sides * (d // (64 if d % 64 == 0 else 32))


def _store(Hkv, d, capacity):
    """A store whose every bit tells whether it was written."""
    st = F.Store.empty(Hkv, d, capacity, device=DEV)
    st.planes.fill_(0x5A5A5A5A), st.scales.fill_(0x1234)
    return st


def _untouched(st, blk0, blk1):
    """Nothing outside blocks [blk0, blk1) was written."""
    for lo, hi in ((0, blk0), (blk1, None)):
        assert (st.planes[..., 2 * lo:2 * hi if hi is not None else None] == 0x5A5A5A5A).all()
        assert (st.scales[..., lo:hi] == 0x1234).all()


@pytest.mark.parametrize("paired", [True, False])
@pytest.mark.parametrize("Hkv,d,n", [(8, 128, 20011), (8, 96, 30000), (8, 64, 40001), (16, 32, 20033), (4, 256, 20480),
                                     (3, 224, 20015), (8, 128, 19457)])
def test_a_prompt_into_empty_stores(Hkv, d, n, paired):
    assert _ctas(Hkv, d, 0, n, 2) >= 296
    Kr, Vr = _row_cache(Hkv, n, d, paired, d + n)
    ks, vs = _store(Hkv, d, n), _store(Hkv, d, n + 3000)
    F.append_rows(ks, vs, Kr, Vr, n)
    for st, rows in ((ks, Kr), (vs, Vr)):
        assert st.n == n
        _same(st, rows, n)
        _untouched(st, 0, -(-n // 64))
    assert F.last_device_status() == 0


@pytest.mark.parametrize("paired", [True, False])
@pytest.mark.parametrize("Hkv,d,n_old,n_new", [(8, 128, 5003, 20011), (8, 96, 1023, 30000), (8, 128, 64, 20011),
                                               (8, 64, 65 * 64, 40001), (16, 32, 1024, 30001), (4, 256, 960, 20481),
                                               (8, 160, 4999, 20000)])
def test_a_long_chunk_behind_earlier_keys(Hkv, d, n_old, n_new, paired):
    """Starts inside a group of 16 blocks, inside a block, and on a group's border."""
    assert _ctas(Hkv, d, n_old, n_new, 2) >= 296
    Kr, Vr = _row_cache(Hkv, n_new, d, paired, d + n_old)
    ks, vs = _store(Hkv, d, n_new + 1500), _store(Hkv, d, n_new)
    for st in (ks, vs):
        st.n = st._c.n = n_old           # its earlier blocks hold other bits, which must stay
    F.append_rows(ks, vs, Kr, Vr, n_new)
    blk0, blk1 = n_old // 64, -(-n_new // 64)
    for st, rows in ((ks, Kr), (vs, Vr)):
        want = F.pack_bitplanes(rows[:, :n_new].contiguous())
        assert torch.equal(st.planes[..., 2 * blk0:2 * blk1], want.planes[..., 2 * blk0:2 * blk1])
        assert torch.equal(st.scales[..., blk0:blk1], want.scales[..., blk0:blk1])
        _untouched(st, blk0, blk1)
    assert F.last_device_status() == 0


@pytest.mark.parametrize("Hkv,d", [(16, 128), (16, 96)])
def test_a_long_key_store_alone(Hkv, d):
    n = 20011
    assert _ctas(Hkv, d, 0, n, 1) >= 296
    Kr, _ = _row_cache(Hkv, n, d, True, 77)
    st = _store(Hkv, d, n)
    F.append_rows(st, None, Kr, None, n)
    _same(st, Kr, n)
    _untouched(st, 0, -(-n // 64))
