"""Norms with rotation into the row cache (fathom_qk_norm_rope), stores grown
from it (fathom_append_rows), and a run of them with the attention over stores.

Tolerances of qk_norm_rope.  In fp32: the sum of squares, its root and the
quotient are off by at most (16 + 4) steps of 2^-24 relative (16 products a lane,
4 levels of sums at most, their halves cancel in the root), weight and rotation
add 5 roundings, the sine and cosine are off by 2^-23 absolute; so an output is
off by at most 32 * 2^-24 (|a| + |b|) of its pair before the rotation.  A bf16
output adds half a step, 2^-8 |y|.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from bit_plane_key_b200 import fathom as F  # noqa: E402
from test_gpu_store_attend import check, reference  # noqa: E402

DEV = torch.device("cuda:0")


def rope_ref(qkv, Hq, Hkv, inv_freq, pos, wq, wk, eps, interleaved):
    """f64 heads [T][Hq + 2 Hkv][d] after norm and rotation, and the pairs' magnitudes."""
    x = qkv.double().cpu().numpy().copy()
    T, H, d = x.shape
    if wq is not None:
        for sl, w in ((slice(0, Hq), wq), (slice(Hq, Hq + Hkv), wk)):
            x[:, sl] = x[:, sl] / np.sqrt((x[:, sl] ** 2).mean(-1, keepdims=True) + eps) * w.double().cpu().numpy()
    mag = np.abs(x)
    if inv_freq is not None:
        f = inv_freq.double().cpu().numpy()
        r = 2 * f.size
        i = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
        j = i + 1 if interleaved else i + r // 2
        ang = pos.astype(np.float64)[:, None, None] * f
        a, b = x[:, :Hq + Hkv, i].copy(), x[:, :Hq + Hkv, j].copy()
        x[:, :Hq + Hkv, i] = a * np.cos(ang) - b * np.sin(ang)
        x[:, :Hq + Hkv, j] = b * np.cos(ang) + a * np.sin(ang)
        mag[:, :Hq + Hkv, i] = mag[:, :Hq + Hkv, j] = np.abs(a) + np.abs(b)
    return x, mag


def near(got, ref, mag, dtype):
    tol = 32 * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) + 1e-38 if dtype == torch.bfloat16 else 0)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err - tol).max()


def freqs(rot, base=1e6):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float32, device=DEV)


@pytest.mark.parametrize("paired", [True, False])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,norm,dtype,wdtype", [
    (1, 32, 8, 128, 128, False, True, torch.bfloat16, torch.bfloat16),
    (1, 1, 1, 32, 16, True, False, torch.float32, None),
    (7, 4, 2, 64, 64, False, True, torch.float32, torch.float32),
    (33, 6, 2, 96, 96, False, True, torch.bfloat16, torch.float32),
    (65, 16, 2, 256, 64, True, True, torch.bfloat16, torch.bfloat16),
    (300, 8, 8, 128, 32, False, False, torch.bfloat16, None),
    (2000, 12, 4, 160, 80, False, True, torch.float32, torch.bfloat16),
    (5, 3, 1, 224, 0, False, True, torch.bfloat16, torch.bfloat16),
    (1300, 32, 8, 128, 128, True, True, torch.bfloat16, torch.bfloat16),
])
def test_norm_and_rotation(T, Hq, Hkv, d, rot, inter, norm, dtype, wdtype, paired):
    g = torch.Generator(device=DEV).manual_seed(T + d)
    qkv = (torch.randn(T, Hq + 2 * Hkv, d, device=DEV, generator=g) * 3).to(dtype)
    wq = wk = None
    if norm:
        wq = torch.randn(d, device=DEV, generator=g).to(wdtype)
        wk = torch.randn(d, device=DEV, generator=g).to(wdtype)
    inv = freqs(rot) if rot else None
    row0, rows = 11, T + 20
    if paired:
        Kr, Vr = F.kv_rows(Hkv, rows, d, device=DEV)
    else:
        Kr, Vr = torch.empty(2, Hkv, rows, d, dtype=torch.bfloat16, device=DEV).unbind(0)
    Kr.fill_(3.0), Vr.fill_(4.0)
    q = F.qk_norm_rope(qkv, Hq, Hkv, inv, Kr, Vr, row0, wq, wk, eps=1e-5, interleaved=inter)
    ref, mag = rope_ref(qkv, Hq, Hkv, inv, np.arange(row0, row0 + T), wq, wk, 1e-5, inter)
    near(q, ref[:, :Hq], mag[:, :Hq], dtype)
    k, v = Kr[:, row0:row0 + T].transpose(0, 1), Vr[:, row0:row0 + T].transpose(0, 1)
    near(k, ref[:, Hq:Hq + Hkv], mag[:, Hq:Hq + Hkv], torch.bfloat16)
    assert torch.equal(v, qkv[:, Hq + Hkv:].to(torch.bfloat16))
    for rows_, fill in ((Kr, 3.0), (Vr, 4.0)):       # the rows around are left alone
        assert (rows_[:, :row0] == fill).all() and (rows_[:, row0 + T:] == fill).all()


def test_far_and_given_positions():
    """Positions near 2^31 and below zero, out of order, the same twice."""
    pos = torch.tensor([0, 1, 1, 1 << 20, (1 << 31) - 1, -5, -(1 << 31), 123456789], dtype=torch.int32, device=DEV)
    T = pos.numel()
    qkv = torch.randn(T, 4, 128, device=DEV)
    inv = freqs(128, 1e4)
    Kr, Vr = F.kv_rows(1, T, 128, device=DEV)
    q = F.qk_norm_rope(qkv, 2, 1, inv, Kr, Vr, 0, positions=pos)
    ref, mag = rope_ref(qkv, 2, 1, inv, pos.cpu().numpy(), None, None, 0, False)
    near(q, ref[:, :2], mag[:, :2], torch.float32)


def test_strided_tokens_host_rows_graph_and_zero_rows():
    big = torch.randn(9, 20, 64, device=DEV)
    qkv = big[:, 4:12]                                # a token's heads lie inside a wider row
    qkv[3] = 0                                        # a zero head: eps keeps the norm finite
    w = torch.ones(64, device=DEV)
    Kr, Vr = F.kv_rows(2, 9, 64, pin_memory=True)
    out = torch.empty(9, 4, 64, device=DEV)
    inv = freqs(64)
    F.qk_norm_rope(qkv, 4, 2, inv, Kr, Vr, 0, w, w, out=out)
    torch.cuda.synchronize()
    ref, mag = rope_ref(qkv, 4, 2, inv, np.arange(9), w, w, 1e-6, False)
    near(out, ref[:, :4], mag[:, :4], torch.float32)
    near(Kr.transpose(0, 1), ref[:, 4:6], mag[:, 4:6], torch.bfloat16)
    g = torch.cuda.CUDAGraph()
    first, rows = out.clone(), Kr.clone()
    with torch.cuda.graph(g):
        F.qk_norm_rope(qkv, 4, 2, inv, Kr, Vr, 0, w, w, out=out)
    out.zero_()
    Kr.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(Kr, rows)


def test_rope_refusals():
    qkv = torch.randn(3, 4, 64, device=DEV)
    Kr, Vr = F.kv_rows(1, 3, 64, device=DEV)
    inv, w = freqs(64), torch.ones(64, device=DEV)
    ok = lambda **k: F.qk_norm_rope(**dict(dict(qkv=qkv, n_q_heads=2, n_kv_heads=1, inv_freq=inv, K_rows=Kr, V_rows=Vr,
                                                row0=0), **k))
    ok()
    for bad in (dict(row0=1), dict(row0=-1), dict(q_weight=w), dict(inv_freq=freqs(24)), dict(inv_freq=freqs(80)),
                dict(eps=-1.0), dict(eps=math.nan), dict(qkv=qkv.cpu())):
        with pytest.raises(F.FathomError):
            ok(**bad)
    with pytest.raises((ValueError, AttributeError)):
        ok(k_weight=w)
    for bad in (dict(n_q_heads=3), dict(inv_freq=inv.double()), dict(positions=torch.zeros(3, device=DEV)),
                dict(positions=torch.zeros(2, device=DEV, dtype=torch.int32)), dict(K_rows=Kr[:, :, :32]),
                dict(qkv=qkv.transpose(1, 2)), dict(V_rows=Vr.contiguous())):
        with pytest.raises(ValueError):
            ok(**bad)
    for bad in (dict(qkv=qkv.half()), dict(K_rows=Kr.float(), V_rows=Vr.float())):
        with pytest.raises(TypeError):
            ok(**bad)
    off = torch.empty(3 * 4 * 64 + 1, device=DEV)[1:].view(3, 4, 64)
    with pytest.raises(F.FathomError):
        ok(qkv=off)                                   # not on a 16-byte boundary


def _row_cache(Hkv, n, d, paired, seed, host=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(2, Hkv, n, d, device=DEV, generator=g)
    x *= torch.exp(torch.randn(2, Hkv, 1, d, device=DEV, generator=g))
    if paired:
        Kr, Vr = F.kv_rows(Hkv, n, d, device=None if host else DEV, pin_memory=host)
    else:
        b = torch.empty(2, Hkv, n, d, dtype=torch.bfloat16, device=None if host else DEV, pin_memory=host)
        Kr, Vr = b[0], b[1]
    Kr.copy_(x[0]), Vr.copy_(x[1])
    torch.cuda.synchronize()
    return Kr, Vr


def _same(st, rows, n):
    """The store equals a pack of the first n rows, over the blocks that hold keys."""
    want = F.pack_bitplanes(rows[:, :n].to(DEV).contiguous())
    nb = -(-n // 64)
    assert torch.equal(st.planes[..., :2 * nb].to(DEV), want.planes[..., :2 * nb])
    assert torch.equal(st.scales[..., :nb].to(DEV), want.scales[..., :nb])


@pytest.mark.parametrize("paired", [True, False])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 192, 256])
def test_append_rows_equals_packing(d, paired):
    Kr, Vr = _row_cache(2, 3000, d, paired, d)
    ks, vs = F.Store.empty(2, d, 3000, device=DEV), F.Store.empty(2, d, 5000, device=DEV)
    for n in (1, 2, 63, 64, 65, 128, 200, 255, 256, 257, 700, 1024, 1025, 2999, 3000):
        before = ks.planes.clone()
        blk = ks.n // 64
        F.append_rows(ks, vs, Kr, Vr, n)
        assert ks.n == vs.n == n
        _same(ks, Kr, n)
        _same(vs, Vr, n)
        assert torch.equal(ks.planes[..., :2 * blk], before[..., :2 * blk])
        nb = -(-n // 64)
        assert not ks.planes[..., 2 * nb:].any() and not ks.scales[..., nb:].any()    # behind the last block: untouched
    assert F.last_device_status() == 0


@pytest.mark.parametrize("host_rows,host_store", [(True, False), (False, True), (True, True)])
def test_append_rows_host_memory_and_key_store_alone(host_rows, host_store):
    Kr, Vr = _row_cache(2, 600, 128, True, 3, host=host_rows)
    ks = F.Store.empty(2, 128, 600, device=DEV, host_resident=host_store)
    vs = F.Store.empty(2, 128, 600, device=DEV, host_resident=host_store)
    for n in (100, 101, 600):
        F.append_rows(ks, vs, Kr, Vr, n)
        torch.cuda.synchronize()
        _same(ks, Kr, n)
        _same(vs, Vr, n)
    alone = F.Store.empty(2, 128, 600, device=DEV)
    F.append_rows(alone, None, Kr, None, 555)
    _same(alone, Kr, 555)


def test_append_rows_cell_borders_and_magnitudes(ref):
    """Values on exact cell borders, just beside them, zeros, subnormals and blocks of every magnitude that a scale can have."""
    rng = np.random.default_rng(5)
    n, d = 64 * 60, 128
    x = rng.standard_normal((1, n, d)).astype(np.float32)
    for b in range(60):
        x[0, 64 * b:64 * b + 64] *= np.float32(2.0) ** (rng.integers(-40, 16) if b % 2 else rng.integers(-24, -8))
    kb = torch.from_numpy(x).to(torch.bfloat16)
    # multiples of the block's own scale, where bf16 holds them, and their neighbours
    u = kb.view(torch.int16).clone()
    amax = kb.float().abs().view(1, 60, 64, d).amax(2)
    step = (amax / 8).half().float()
    for j in range(-8, 9):
        cell = (step * j).to(torch.bfloat16).view(torch.int16)
        pos = 3 * (j + 8)
        u.view(1, 60, 64, d)[:, :, pos] = cell
        u.view(1, 60, 64, d)[:, :, pos + 1] = torch.where(cell == 0, cell, cell + 1)
        u.view(1, 60, 64, d)[:, :, pos + 2] = torch.where((cell & 0x7FFF) == 0, torch.tensor(-32767, dtype=torch.int16),
                                                          cell - 1)
    u.view(1, 60, 64, d)[:, :5, 60:] = 0
    u.view(1, 60, 64, d)[:, 6] = 0
    rows = u.view(torch.bfloat16)
    Kr, Vr = F.kv_rows(1, n, d, device=DEV)
    Kr.copy_(rows), Vr.copy_(rows)
    ks, vs = F.Store.empty(1, d, n, device=DEV), F.Store.empty(1, d, n, device=DEV)
    F.append_rows(ks, vs, Kr, Vr, n)
    planes, scales = ref.pack(rows.float().numpy())
    for st in (ks, vs):
        assert np.array_equal(st.scales.cpu().numpy().view(np.uint16), scales)
        assert np.array_equal(st.planes.cpu().numpy().view(np.uint32), planes)


def test_append_rows_graph_replays_a_step():
    Kr, Vr = _row_cache(2, 400, 128, True, 9)
    ks, vs = F.Store.empty(2, 128, 400, device=DEV), F.Store.empty(2, 128, 400, device=DEV)
    F.append_rows(ks, vs, Kr, Vr, 300)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.append_rows(ks, vs, Kr, Vr, 301)
    Kr.neg_()
    g.replay()
    torch.cuda.synchronize()
    want = F.pack_bitplanes(torch.cat([-Kr[:, :256], Kr[:, 256:301]], 1))
    assert torch.equal(ks.planes[..., :10], want.planes[..., :10])


def test_append_rows_refusals():
    Kr, Vr = _row_cache(2, 3000, 64, True, 1)
    mk = lambda n=2048, h=2, d=64: F.Store.empty(h, d, n, device=DEV)
    ks, vs = mk(), mk()
    F.append_rows(ks, vs, Kr, Vr, 1000)
    for args in ((ks, vs, Kr, Vr, 1000), (ks, vs, Kr, Vr, 2049), (ks, ks, Kr, Vr, 1001), (ks, mk(), Kr, Vr, 1001),
                 (mk(4096), mk(4096), Kr, Vr, 3001)):
        with pytest.raises(F.FathomError):
            F.append_rows(*args)
    for args in ((ks, None, Kr, Vr, 1001), (mk(h=1), mk(h=1), Kr, Vr, 10), (mk(d=32), mk(d=32), Kr, Vr, 10)):
        with pytest.raises(ValueError):
            F.append_rows(*args)
    with pytest.raises(TypeError):
        F.append_rows(ks, vs, Kr.float(), Vr.float(), 1001)
    assert ks.n == vs.n == 1000
    F.append_rows(ks, vs, Kr, Vr, 1001)
    _same(ks, Kr, 1001)


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_layers_steps_together(interleaved):
    """A prompt, then decoded and drafted tokens: projection rows -> norm and rotation -> row cache -> stores ->
    attention over the stores, every step against the definition on the rows written so far; then the sparse decode
    step runs on the same store, queries and rows."""
    Hq, Hkv, d, cap = 8, 2, 128, 2000
    g = torch.Generator(device=DEV).manual_seed(17)
    wq = (1 + 0.3 * torch.randn(d, device=DEV, generator=g)).bfloat16()
    wk = (1 + 0.3 * torch.randn(d, device=DEV, generator=g)).bfloat16()
    inv = freqs(d)
    Kr, Vr = F.kv_rows(Hkv, cap, d, device=DEV)
    Kr.zero_(), Vr.zero_()
    ks, vs = F.Store.empty(Hkv, d, cap, device=DEV), F.Store.empty(Hkv, d, cap, device=DEV)
    n = 0
    for T in (1001, 1, 1, 5, 1, 64, 3, 1):
        qkv = torch.randn(T, Hq + 2 * Hkv, d, device=DEV, generator=g).bfloat16()
        q = F.qk_norm_rope(qkv, Hq, Hkv, inv, Kr, Vr, n, wq, wk, interleaved=interleaved)
        pos = np.arange(n, n + T)
        y, mag = rope_ref(qkv, Hq, Hkv, inv, pos, wq, wk, 1e-6, interleaved)
        near(q, y[:, :Hq], mag[:, :Hq], torch.bfloat16)
        F.append_rows(ks, vs, Kr, Vr, n + T)
        n += T
        _same(ks, Kr, n)
        _same(vs, Vr, n)
        if T <= 64:
            out = F.store_attend(ks, vs, q)
            want, tol, _, _ = reference(ks, vs, q, n - T + 1)
            check(out, want, tol)
    s2 = Kr[:, :n].float().pow(2).mean(1)
    _, idx, _, out = F.decode_step(ks, q[0], s2, 92, 256, Kr, Vr)
    assert (idx >= 0).all() and (idx < n).all() and torch.isfinite(out).all()
    assert F.last_device_status() == 0


def test_calls_behind_copies_memsets_and_other_streams():
    """The calls follow whatever the stream holds, run or captured: a copy, a memset, a kernel of another library, work
    joined from another stream."""
    Hq, Hkv, d, n = 8, 2, 128, 700
    g = torch.Generator(device=DEV).manual_seed(3)
    qkv = torch.randn(3, Hq + 2 * Hkv, d, device=DEV, generator=g)
    Kr, Vr = _row_cache(Hkv, n, d, True, 31)
    inv = freqs(d)
    K0, V0 = Kr.clone(), Vr.clone()
    src = qkv.clone()

    def step(side):
        ks, vs = F.Store.empty(Hkv, d, n, device=DEV), F.Store.empty(Hkv, d, n, device=DEV)
        buf = torch.empty_like(src)
        buf.copy_(src)                                       # a copy, then the rotation
        q = F.qk_norm_rope(buf, Hq, Hkv, inv, Kr, Vr, n - 3)
        ks.planes.zero_(), vs.planes.zero_()                 # memsets, then the append
        F.append_rows(ks, vs, Kr, Vr, n)
        out = torch.empty(3, Hq, d, device=DEV)
        ev = torch.cuda.Event()
        ev.record()
        with torch.cuda.stream(side):
            ev.wait()
            out.fill_(7.0)                                   # on the other stream, joined before the attention
            ev2 = torch.cuda.Event()
            ev2.record()
        ev2.wait()
        F.store_attend(ks, vs, q, out=out)
        return q, ks, vs, out * 1.0                          # and another library's kernel behind it

    side = torch.cuda.Stream()
    q, ks, vs, out = step(side)
    torch.cuda.synchronize()
    assert torch.equal(Kr[:, :n - 3], K0[:, :n - 3]) and torch.equal(Vr[:, :n - 3], V0[:, :n - 3])
    _same(ks, Kr, n)
    _same(vs, Vr, n)
    want, tol, _, _ = reference(ks, vs, q, n - 2)
    check(out, want, tol)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q2, ks2, vs2, out2 = step(side)
    for _ in range(3):
        Kr[:, n - 3:] = 0
        out2.zero_(), q2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, out) and torch.equal(q2, q) and torch.equal(ks2.planes, ks.planes)


def test_offsets_beyond_32_bits():
    """A small cache and the same keys in arrays whose later heads lie beyond 2^32 bytes and 2^31 elements: same bits."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    Hkv, Hq, d, T, n = 4, 8, 256, 900, 900
    g = torch.Generator(device=DEV).manual_seed(23)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, device=DEV, generator=g).bfloat16()
    got = []
    for rows_n, cap in ((1024, 1024), (1 << 22, 1 << 24)):
        rows = torch.empty(2, Hkv, rows_n, d, dtype=torch.bfloat16, device=DEV)
        stores = []
        for _ in range(2):
            stores.append(F.Store(torch.empty(Hkv, d, 4, cap // 32, dtype=torch.int32, device=DEV),
                                  torch.empty(Hkv, d, cap // 64, dtype=torch.int16, device=DEV), 0))
        ks, vs = stores
        q = F.qk_norm_rope(qkv, Hq, Hkv, freqs(d), rows[0], rows[1], 0)
        F.append_rows(ks, vs, rows[0], rows[1], n)
        out = F.store_attend(ks, vs, q[-1])
        several = F.store_attend_batched([ks, ks], [vs, vs], q[-4:].reshape(2, 2, Hq, d))
        got.append((q, rows[:, :, :n].clone(), *(st.planes[..., :30].clone() for st in stores), out, several))
        assert torch.isfinite(out).all() and out.abs().max() > 0
        torch.cuda.synchronize()
        del rows, stores, ks, vs
    for a, b in zip(*got):
        assert torch.equal(a, b)
    torch.cuda.empty_cache()
