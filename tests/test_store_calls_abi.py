"""Host-side refusals of the row and store-attention calls; needs no GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def libpath():
    from bit_plane_key_b200 import build
    return build.build()


def test_row_and_store_attention_calls_reject_bad_arguments(libpath):
    """Null pointers and impossible sizes are turned down on the host, before any pointer is looked at."""
    from bit_plane_key_b200 import fathom as F
    L = F.lib()
    fake = ctypes.c_void_p(1 << 12)

    def rope(**k):
        a = dict(qkv=fake, dtype=1, stride=12 * 64, T=3, Hq=8, Hkv=2, d=64, wq=None, wk=None, wdt=0, eps=1e-6, pos=None,
                 inv=fake, rot=64, inter=0, q=fake, K=fake, V=fake, rs=64, host=0, rows=10, row0=0)
        a.update(k)
        return L.fathom_qk_norm_rope(*a.values(), None)

    for bad in (dict(qkv=None), dict(q=None), dict(K=None), dict(V=None), dict(dtype=2), dict(T=0), dict(Hq=0),
                dict(Hq=7), dict(Hkv=0), dict(d=48), dict(d=288), dict(stride=11 * 64), dict(stride=12 * 64 + 4),
                dict(wq=fake), dict(wk=fake), dict(wq=fake, wk=fake, wdt=5), dict(eps=-1.0), dict(eps=float("nan")),
                dict(inv=None), dict(rot=72), dict(rot=80), dict(rot=-16), dict(rows=2), dict(row0=8), dict(row0=-1),
                dict(row0=1 << 62, rows=1 << 62), dict(rows=1 << 40, row0=(1 << 31)), dict(qkv=ctypes.c_void_p(8 + 4096)),
                dict(rs=60), dict(rs=68), dict(K=ctypes.c_void_p(4096 + 2)), dict(pos=ctypes.c_void_p(4096 + 2)),
                dict(inv=ctypes.c_void_p(4096 + 1))):
        assert rope(**bad) == F.EINVAL, bad

    def store(n=100, n_pad=1024, Hkv=2, d=64, host=0, planes=1 << 12, scales=1 << 13):
        return F.fathom_store(Hkv, d, n, n_pad, host, 0, planes, scales)

    def append(K, V, **k):
        a = dict(Kr=fake, Vr=fake, rs=64, host=0, rows=2000, n_new=200)
        a.update(k)
        return L.fathom_append_rows(ctypes.byref(K) if K else None, ctypes.byref(V) if V else None, *a.values(), None)

    assert append(None, None) == F.EINVAL
    for K in (store(planes=None), store(scales=None), store(n=-1), store(n_pad=1000), store(n_pad=0), store(d=40),
              store(Hkv=0), store(planes=4096 + 8), store(scales=4096 + 8)):
        assert append(K, store()) == F.EINVAL
    assert append(store(), store(), n_new=1025) == F.EINVAL          # capacity
    assert append(store(), store(), n_new=100) == F.EINVAL           # nothing to add

    for S, T, Hq, Hkv, d in ((0, 1, 8, 2, 128), (65, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 4097, 8, 2, 128),
                             (1, 1, 6, 2, 128), (1, 1, 8, 0, 128), (1, 1, 8, 2, 100)):
        assert L.fathom_store_attend_workspace_bytes(S, T, Hq, Hkv, d) == 0
    nb = L.fathom_store_attend_workspace_bytes(1, 1, 8, 2, 64)
    assert nb > 0 and nb % 256 == 0
    assert L.fathom_store_attend_workspace_bytes(64, 9, 8, 2, 64) > nb

    def attend(K, V, **k):
        a = dict(q=fake, qdt=1, T=1, Hq=8, causal=1, out=fake, ws=fake, nb=nb)
        a.update(k)
        return L.fathom_store_attend(ctypes.byref(K) if K else None, ctypes.byref(V) if V else None, *a.values(), None)

    ok = store()
    assert attend(None, ok) == F.EINVAL and attend(ok, None) == F.EINVAL
    for bad in (dict(q=None), dict(out=None), dict(ws=None), dict(qdt=3), dict(T=0), dict(T=4097), dict(Hq=6),
                dict(Hq=0), dict(ws=ctypes.c_void_p(4096 + 16))):
        assert attend(ok, ok, **bad) == F.EINVAL, bad
    assert attend(ok, ok, nb=nb - 1) == F.ENOMEM
    assert attend(store(d=96), store(d=96), nb=1 << 30) == F.EUNSUPPORTED
    for V in (store(n=99), store(Hkv=1), store(d=128), store(n=-1)):
        assert attend(ok, V) == F.EINVAL
    assert attend(store(n=1 << 31, n_pad=1 << 31), store(n=1 << 31, n_pad=1 << 31)) == F.EINVAL
    assert L.fathom_store_attend_partial(ctypes.byref(ok), ctypes.byref(ok), fake, 1, 1, 8, 100, None, fake, nb,
                                         None) == F.EINVAL
    two = (F.fathom_store * 2)(store(), store(Hkv=4))
    assert L.fathom_store_attend_batched(two, two, 2, fake, 1, 1, 8, 1, fake, fake, 1 << 30, None) == F.EINVAL
    assert L.fathom_store_attend_batched(two, two, 0, fake, 1, 1, 8, 1, fake, fake, 1 << 30, None) == F.EINVAL
