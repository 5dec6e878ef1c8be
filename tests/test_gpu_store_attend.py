"""Attention over the 4-bit stores (fathom_store_attend, _partial, _batched)
against the definition in 64 bits.

Tolerance, as the sum of
- logits.  Sums over d channels of q Delta code, offsets included, so their
  rounding is relative to A = 15 sum_c |q_c| Delta_c / sqrt(d) of the block.  Sixteen
  channels enter per accumulation step with at most two units of the last place of
  the partial sum (2^-23 A), the split of q Delta into two halves leaves 2^-22, the
  scaling of the result 2 roundings: (d/16 + 6) 2^-23 A; and each channel's low half at
  least a rounding of 2^-25 of max |q| max Delta, so 15 sqrt(d) 2^-25 times that more.
  A logit is off by at most e, the sum of both; the largest A and Delta of any
  visible block serve for all.  The weights move by a factor of at most exp(2e).
- weights.  exp2 is off by 2^-22; its argument, below 64 in magnitude where the weight
  counts, is rounded by 2^-19; in numerator and sum: 2^-17 with room.  A weight's low half is
  rounded to 2^-23 of the largest weight in its block of 64 keys, or, as a fp16
  subnormal, to 2^-36 of the largest of all.
- sums over keys.  A warp adds two blocks a tile, then 8 warps and the partials are
  added: at most n/512 + 24 steps of two roundings (2^-24) and one rescaling (2^-22), in
  numerator and sum.
All act on sum_i p_i 15 Delta_i,c, the last but one on its own weights.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from bit_plane_key_b200 import fathom as F  # noqa: E402

DEV = torch.device("cuda:0")


def make_store(n, Hkv, d, seed, spread=1.0, capacity=None, host=False, garbage=False):
    """A store packed from random rows; with `garbage`, everything behind its last block is filled with other bits."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(Hkv, max(n, 1), d, device=DEV, generator=g)
    x *= torch.exp(spread * torch.randn(Hkv, 1, d, device=DEV, generator=g))
    st = F.Store.empty(Hkv, d, capacity or max(n, 1), device=DEV)
    if garbage:
        st.planes.random_(generator=g)
        st.scales.fill_(0x7E00)      # NaN
    if n:
        F.append_keys(st, x, n)
    if host:
        torch.cuda.synchronize()
        st = F.Store(st.planes.cpu().pin_memory(), st.scales.cpu().pin_memory(), n, host_resident=True)
    return st


def values(st):
    """The store's values f64 [Hkv][n][d] and their scales f64 [Hkv][n][d]."""
    n = st.n
    bits = np.unpackbits(st.planes.cpu().numpy().view(np.uint8), axis=-1, bitorder="little")[..., :n]
    code = (bits * np.array([8, 4, 2, 1])[:, None]).sum(2)
    sc = st.scales.cpu().numpy().view(np.float16).astype(np.float64)
    sc = np.repeat(sc, 64, axis=-1)[..., :n]
    return ((code - 7.5) * sc).transpose(0, 2, 1), sc.transpose(0, 2, 1)


def reference(ks, vs, q, visible):
    """f64 out [T][Hq][d], the tolerance of every element, and the maxima and sums (log2 units)."""
    q = q.double().cpu().numpy()
    T, Hq, d = q.shape
    Hkv = ks.n_kv_heads
    G = Hq // Hkv
    n = ks.n
    K, Kd = values(ks)
    V, Vd = values(vs)
    out, tol = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    M, L = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for t in range(T):
        see = max(0, min(n, visible + t))
        if see == 0:
            continue
        for h in range(Hq):
            g = h // G
            s = K[g, :see] @ q[t, h] / math.sqrt(d)
            p = np.exp(s - s.max())
            M[t, h], L[t, h] = s.max() / math.log(2), p.sum()
            p /= p.sum()
            out[t, h] = p @ V[g, :see]
            A = 15 * (Kd[g, :see] @ np.abs(q[t, h])).max() / math.sqrt(d)
            e = (d / 16 + 6) * 2.0 ** -23 * A
            e += 15 * math.sqrt(d) * 2.0 ** -25 * np.abs(q[t, h]).max() * Kd[g, :see].max()
            pV = p @ Vd[g, :see]
            tol[t, h] = (np.expm1(2 * e) + 2.0 ** -17 + 1.5 * (n / 512 + 24) * 2.0 ** -22) * 15 * pV
            top = np.repeat([p[i:i + 64].max() for i in range(0, see, 64)], 64)[:see] * 2.0 ** -23 + 2.0 ** -35 * p.max()
            tol[t, h] += 15 * (top @ Vd[g, :see]) + 7.5 * top.sum() * pV
    return out, tol, M, L


def check(got, ref, tol):
    got = got.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref)[bad][:5], tol[bad][:5])


def queries(shape, seed, dtype=torch.bfloat16, mult=1.0):
    g = torch.Generator(device=DEV).manual_seed(1000 + seed)
    return (torch.randn(*shape, device=DEV, generator=g) * mult).to(dtype)


def vis(n, T, causal):
    return n - T + 1 if causal else n


@pytest.mark.parametrize("n", [1, 31, 32, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1000, 4097, 20011])
def test_lengths(n):
    ks, vs = make_store(n, 2, 128, n), make_store(n, 2, 128, n + 1)
    q = queries((8, 128), n)
    ref, tol, _, _ = reference(ks, vs, q[None], n)
    check(F.store_attend(ks, vs, q), ref, tol)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_heads_and_dims(d, G, dtype):
    n = 1500 + d
    ks, vs = make_store(n, 3, d, d + G), make_store(n, 3, d, d - G)
    q = queries((3 * G, d), d + G, dtype)
    ref, tol, _, _ = reference(ks, vs, q[None], n)
    check(F.store_attend(ks, vs, q), ref, tol)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T,G,d", [(2, 4, 128), (3, 1, 64), (5, 4, 128), (7, 8, 64), (9, 2, 256), (4, 8, 256), (33, 4, 128),
                                   (70, 1, 32)])
def test_tokens(T, G, d, causal):
    n = 777
    ks, vs = make_store(n, 2, d, T), make_store(n, 2, d, T + 1)
    q = queries((T, 2 * G, d), T)
    ref, tol, _, _ = reference(ks, vs, q, vis(n, T, causal))
    check(F.store_attend(ks, vs, q, causal=causal), ref, tol)


@pytest.mark.parametrize("n,T", [(1, 1), (2, 5), (3, 3), (64, 70), (130, 129), (520, 600)])
def test_tokens_that_see_no_key_get_zero(n, T):
    """More tokens than keys: the first tokens see none."""
    ks, vs = make_store(n, 1, 64, n), make_store(n, 1, 64, T)
    q = queries((T, 2, 64), T)
    ref, tol, _, _ = reference(ks, vs, q, n - T + 1)
    out = F.store_attend(ks, vs, q)
    check(out, ref, tol)
    assert (out[:max(0, T - n)] == 0).all()


def test_empty_store():
    ks, vs = make_store(0, 2, 128, 0, garbage=True), make_store(0, 2, 128, 1, garbage=True)
    assert ks.n == 0
    out = torch.full((3, 8, 128), 7.0, device=DEV)
    F.store_attend(ks, vs, queries((3, 8, 128), 0), out=out)
    assert (out == 0).all()
    parts = F.store_attend_partial(ks, vs, queries((3, 8, 128), 0), 5)
    assert (parts[..., 128] == -math.inf).all() and (parts[..., 129] == 0).all()


@pytest.mark.parametrize("n", [1, 40, 700, 1025])
def test_nothing_behind_the_last_block_is_used(n):
    """Spare capacity, rows behind n: other bits and NaN scales there change nothing."""
    q = queries((2, 8, 128), n)
    a = F.store_attend(make_store(n, 2, 128, 5, capacity=5000), make_store(n, 2, 128, 6, capacity=3000), q)
    b = F.store_attend(make_store(n, 2, 128, 5, capacity=5000, garbage=True),
                       make_store(n, 2, 128, 6, capacity=3000, garbage=True), q)
    ks = make_store(n, 2, 128, 5, capacity=5000)
    # keys of the last block behind n: any code
    tail = n % 64
    if tail:
        w = (n // 64) * 2
        P = ks.planes.cpu().numpy().view(np.uint32)
        for i in range(tail, 64):
            P[..., w + i // 32] |= np.uint32(1 << (i % 32))
        ks.planes.copy_(torch.from_numpy(P.view(np.int32)).to(DEV))
    c = F.store_attend(ks, make_store(n, 2, 128, 6, capacity=3000), q)
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("spread,mult", [(3.0, 1.0), (0.5, 30.0), (4.0, 1e-3)])
def test_wide_channel_scales_and_sharp_weights(spread, mult):
    n = 3000
    ks, vs = make_store(n, 2, 128, 9, spread=spread), make_store(n, 2, 128, 10)
    q = queries((8, 128), 3, torch.float32, mult)
    ref, tol, _, _ = reference(ks, vs, q[None], n)
    check(F.store_attend(ks, vs, q), ref, tol)


def test_block_scales_from_zero_to_the_largest():
    """Blocks whose scales are 0, subnormal, ordinary and near the largest f16, in one row of keys."""
    n, d = 64 * 40, 64
    ks, vs = make_store(n, 1, d, 20), make_store(n, 1, d, 21)
    f = torch.tensor([0.0, 6e-8, 1e-6, 1e-3, 1.0, 300.0, 65504.0, 2.0], device=DEV)
    ks.scales.view(torch.float16)[0, :, :40] = f[torch.arange(40, device=DEV) % 8][None]
    q = queries((4, d), 1, torch.float32, 1e-4)
    ref, tol, _, _ = reference(ks, vs, q[None], n)
    check(F.store_attend(ks, vs, q), ref, tol)
    vs.scales.view(torch.float16)[0, :, :40] = f[torch.arange(40, device=DEV) * 3 % 8][None]
    ref, tol, _, _ = reference(ks, vs, q[None], n)
    check(F.store_attend(ks, vs, q), ref, tol)


@pytest.mark.parametrize("mult", [0.0, 1e-30, 1e30])
def test_query_magnitudes(mult):
    """Zero queries weigh every key alike; huge ones choose one key (equal logits share)."""
    n = 900
    ks, vs = make_store(n, 2, 128, 30), make_store(n, 2, 128, 31)
    q = queries((4, 128), 2, torch.float32) * mult
    out = F.store_attend(ks, vs, q).double().cpu().numpy()
    if mult == 1e30:
        K, _ = values(ks)
        V, _ = values(vs)
        qn = q.double().cpu().numpy()
        for h in range(4):
            s = np.sort(K[h // 2] @ qn[h])
            assert s[-1] - s[-2] > 1e-4 * abs(s[-1])       # one winner, beyond rounding
            i = int(np.argmax(K[h // 2] @ qn[h]))
            assert np.abs(out[h] - V[h // 2, i]).max() <= 64 * 2.0 ** -22 * 15 * np.abs(V[h // 2, i]).max()
    else:
        ref, tol, _, _ = reference(ks, vs, q[None], n)
        check(torch.from_numpy(out), ref, tol)


def test_partials_of_ranges_merge_to_the_whole():
    n, T, G = 3000, 3, 4
    ks, vs = make_store(n, 2, 128, 40), make_store(n, 2, 128, 41)
    q = queries((T, 2 * G, 128), 4)
    ref, tol, M, L = reference(ks, vs, q, n - T + 1)
    cuts = [0, 1024, 2048, 2048, n]
    parts = []
    for a, b in zip(cuts, cuts[1:]):
        m = max(1, -(-(b - a) // 1024)) * 1024
        def sub(st):
            P = torch.zeros(2, 128, 4, m // 32, dtype=torch.int32, device=DEV)
            S = torch.zeros(2, 128, m // 64, dtype=torch.int16, device=DEV)
            P[..., :(b - a + 31) // 32] = st.planes[..., a // 32:(b + 31) // 32]
            S[..., :(b - a + 63) // 64] = st.scales[..., a // 64:(b + 63) // 64]
            return F.Store(P, S, b - a)
        parts.append(F.store_attend_partial(sub(ks), sub(vs), q, n - T + 1 - a))
    merged = F.attend_merge(torch.stack(parts).view(len(parts), T * 2 * G, 130))
    check(merged, ref, tol)
    whole = F.store_attend_partial(ks, vs, q, n - T + 1).double().cpu().numpy()
    m, l = whole[..., 128], whole[..., 129]
    # o is relative to 2^m, l alike
    o = whole[..., :128] / l[..., None]
    assert (np.abs(o - ref) <= tol).all()
    assert np.allclose(m + np.log2(l), M + np.log2(L), rtol=0, atol=1e-3)


def test_partial_of_a_store_merges_with_a_partial_of_rows():
    """Old keys in 4 bits, the newest in bf16: the two kinds of partials share their units."""
    n, Hkv, G, d = 1024, 2, 2, 128
    ks, vs = make_store(n, Hkv, d, 50), make_store(n, Hkv, d, 51)
    q = queries((Hkv * G, d), 5)
    Kr, Vr = F.kv_rows(Hkv, 50, d, device=DEV)
    Kr.copy_(torch.randn(Hkv, 50, d, device=DEV))
    Vr.copy_(torch.randn(Hkv, 50, d, device=DEV))
    idx = torch.arange(50, dtype=torch.int32, device=DEV).repeat(Hkv * G, 1)
    p = torch.stack([F.store_attend_partial(ks, vs, q, n), F.sparse_attend_partial(q, Kr, Vr, idx, 0)])
    out = F.attend_merge(p).double().cpu().numpy()
    K = np.concatenate([values(ks)[0], Kr.double().cpu().numpy()], 1)
    V = np.concatenate([values(vs)[0], Vr.double().cpu().numpy()], 1)
    qn = q.double().cpu().numpy()
    for h in range(Hkv * G):
        s = K[h // G] @ qn[h] / math.sqrt(d)
        w = np.exp(s - s.max())
        o = (w / w.sum()) @ V[h // G]
        assert np.linalg.norm(out[h] - o) <= 1e-3 * np.linalg.norm(o)


@pytest.mark.parametrize("T", [1, 3])
def test_batched_sessions(T):
    lens = [1, 5000, 0, 64, 513, 2, 12000, 1024, 77]
    ks = [make_store(n, 2, 128, 60 + i, capacity=n + 100 * i) for i, n in enumerate(lens)]
    vs = [make_store(n, 2, 128, 160 + i) for i, n in enumerate(lens)]
    ks[3] = ks[3].to_host()
    vs[6] = vs[6].to_host()
    q = queries((len(lens), T, 8, 128), 6)
    out = F.store_attend_batched(ks, vs, q)
    full = F.store_attend_batched(ks, vs, q, causal=False)
    for s, n in enumerate(lens):
        for o, causal in ((out, True), (full, False)):
            ref, tol, _, _ = reference(ks[s], vs[s], q[s], vis(n, T, causal))
            check(o[s], ref, tol)


def test_sixty_four_sessions():
    ks = [make_store(1 + 37 * i, 1, 64, i) for i in range(64)]
    vs = [make_store(1 + 37 * i, 1, 64, 100 + i) for i in range(64)]
    q = queries((64, 1, 8, 64), 7)
    out = F.store_attend_batched(ks, vs, q)
    for s in range(64):
        ref, tol, _, _ = reference(ks[s], vs[s], q[s], ks[s].n)
        check(out[s], ref, tol)


def test_host_resident_stores_give_the_same_bits():
    ks, vs = make_store(2500, 2, 128, 70), make_store(2500, 2, 128, 71)
    q = queries((2, 8, 128), 8)
    a = F.store_attend(ks, vs, q)
    assert torch.equal(a, F.store_attend(ks.to_host(), vs.to_host(), q))
    assert torch.equal(a, F.store_attend(ks, vs.to_host(), q))


def test_same_bits_on_every_call_and_from_a_dirty_workspace():
    ks, vs = make_store(50000, 4, 128, 80), make_store(50000, 4, 128, 81)
    q = queries((16, 128), 9)
    ws = torch.empty(F.store_attend_workspace_bytes(ks, 1, 1, 16), dtype=torch.uint8, device=DEV)
    first = F.store_attend(ks, vs, q, workspace=ws)
    for b in (0, 255, 127):
        ws.fill_(b)
        assert torch.equal(first, F.store_attend(ks, vs, q, workspace=ws))
    sub = F.store_attend(ks, vs, q[:4].repeat(4, 1).contiguous())
    assert sub.shape == first.shape


def test_streams_and_graphs():
    """Two streams with a workspace each, and two captured graphs replayed in turn after the stores have grown."""
    n = 3000
    ks, vs = make_store(n, 2, 128, 90), make_store(n, 2, 128, 91)
    qa, qb = queries((8, 128), 10), queries((8, 128), 11)
    a, b = F.store_attend(ks, vs, qa), F.store_attend(ks, vs, qb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a1 = F.store_attend(ks, vs, qa)
        with torch.cuda.stream(s2):
            b1 = F.store_attend(ks, vs, qb)
        torch.cuda.synchronize()
        assert torch.equal(a, a1) and torch.equal(b, b1)
    ws = torch.empty(F.store_attend_workspace_bytes(ks, 1, 1, 8), dtype=torch.uint8, device=DEV)
    oa, ob = torch.empty_like(a), torch.empty_like(b)
    graphs = []
    for q, o in ((qa, oa), (qb, ob)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            F.store_attend(ks, vs, q, out=o, workspace=ws)     # the two share a workspace: replayed one after the other
        graphs.append(g)
    for _ in range(3):
        oa.zero_(), ob.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(a, oa) and torch.equal(b, ob)
    other = make_store(n, 2, 128, 95)
    ks.planes.copy_(other.planes)
    ks.scales.copy_(other.scales)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, F.store_attend(ks, vs, qa))


def test_long_row_over_many_ctas():
    """One KV head over 300000 keys: its tiles spread over the whole GPU."""
    n = 300001
    ks, vs = make_store(n, 1, 64, 99), make_store(n, 1, 64, 98)
    q = queries((1, 4, 64), 12)
    ref, tol, _, _ = reference(ks, vs, q, n)
    check(F.store_attend(ks, vs, q), ref, tol)


def test_refusals():
    ks, vs = make_store(100, 2, 64, 1), make_store(100, 2, 64, 2)
    q = queries((8, 64), 0)
    with pytest.raises(F.FathomError):
        F.store_attend(ks, make_store(101, 2, 64, 3), q)           # lengths differ
    with pytest.raises(F.FathomError):
        F.store_attend(ks, make_store(100, 1, 64, 3), q)           # heads differ
    with pytest.raises(F.FathomError):
        F.store_attend(ks, vs, queries((6, 64), 0))                # three heads to a KV head
    with pytest.raises(F.FathomError) as e:
        F.store_attend(make_store(10, 1, 96, 1), make_store(10, 1, 96, 2), queries((1, 96), 0))
    assert e.value.status == F.EUNSUPPORTED
    with pytest.raises(F.FathomError) as e:
        F.store_attend(ks, vs, q, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == F.ENOMEM
    ws = torch.empty(F.store_attend_workspace_bytes(ks, 1, 1, 8) + 256, dtype=torch.uint8, device=DEV)
    with pytest.raises(F.FathomError):
        F.store_attend(ks, vs, q, workspace=ws[1:])                # misaligned
    with pytest.raises(F.FathomError):
        F.store_attend(ks, vs, q.cpu())
    with pytest.raises(F.FathomError):
        F.store_attend(F.Store(ks.planes.cpu(), ks.scales.cpu(), 100, host_resident=True), vs, q)   # not page-locked
    with pytest.raises(TypeError):
        F.store_attend(ks, vs, q.half())
    with pytest.raises(ValueError):
        F.store_attend(ks, vs, queries((64, 8), 0).t())
    with pytest.raises(ValueError):
        F.store_attend(ks, vs, q, out=torch.empty(8, 64, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        F.store_attend_batched([ks], [vs, vs], q[None, None])
    with pytest.raises(F.FathomError):
        F.store_attend_batched([ks] * 65, [vs] * 65, q[None, None].repeat(65, 1, 1, 1))


@pytest.mark.parametrize("d,G,T,dtype", [(32, 2, 1, torch.float32), (64, 8, 1, torch.bfloat16), (128, 4, 1, torch.bfloat16),
                                         (128, 1, 6, torch.float32), (256, 4, 1, torch.bfloat16),
                                         (256, 8, 1, torch.float32), (64, 4, 3, torch.bfloat16)])
def test_keys_for_the_whole_gpu(d, G, T, dtype):
    """More 1024-key tiles than SMs: the long tiles, runs that end inside a row, rows of several CTAs."""
    n, Hkv = 20000 + d, 8
    ks, vs = make_store(n, Hkv, d, d + T), make_store(n, Hkv, d, d + 1)
    q = queries((T, Hkv * G, d), d, dtype)
    ref, tol, _, _ = reference(ks, vs, q, n - T + 1)
    check(F.store_attend(ks, vs, q), ref, tol)


@pytest.mark.parametrize("d,G,T,dtype", [(32, 1, 1, torch.bfloat16), (64, 8, 2, torch.float32), (128, 8, 1, torch.bfloat16),
                                         (256, 2, 3, torch.bfloat16), (256, 4, 1, torch.float32)])
def test_batched_shapes(d, G, T, dtype):
    """Short sessions beside longer ones, in the batched call's tiles: ends of blocks, of warps' shares and of tiles."""
    lens = [63, 1, 1000, 0, 65, 1025, 128, 2049, 3]
    ks = [make_store(n, 2, d, 200 + i) for i, n in enumerate(lens)]
    vs = [make_store(n, 2, d, 300 + i, capacity=n + 2000, garbage=True) for i, n in enumerate(lens)]
    q = queries((len(lens), T, 2 * G, d), d, dtype)
    out = F.store_attend_batched(ks, vs, q)
    for s, n in enumerate(lens):
        ref, tol, _, _ = reference(ks[s], vs[s], q[s], n - T + 1)
        check(out[s], ref, tol)


def test_back_to_back_calls_in_one_workspace():
    """Calls of different shapes that follow each other in a stream share a workspace: each waits for the one before."""
    shapes = [(300001, 1, 64, 4), (900, 2, 128, 4), (20000, 8, 128, 8), (100, 1, 256, 1)]
    items = []
    for i, (n, Hkv, d, G) in enumerate(shapes):
        ks, vs, q = make_store(n, Hkv, d, 400 + i), make_store(n, Hkv, d, 500 + i), queries((Hkv * G, d), 400 + i)
        items.append((ks, vs, q, F.store_attend(ks, vs, q)))
    torch.cuda.synchronize()
    nb = max(F.store_attend_workspace_bytes(k, 1, 1, q.shape[0]) for k, _, q, _ in items)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    for _ in range(10):
        got = [F.store_attend(k, v, q, workspace=ws) for k, v, q, _ in items]
        torch.cuda.synchronize()
        for g, (_, _, _, want) in zip(got, items):
            assert torch.equal(g, want)
    assert F.last_device_status() == 0



def test_calls_on_a_stream_of_their_own_leave_their_memory_to_it():
    """Temporaries of calls on another stream are not handed to the current stream while those calls run."""
    ks, vs = make_store(60000, 1, 64, 1), make_store(60000, 1, 64, 2)
    q = queries((4, 64), 3)
    want = F.store_attend(ks, vs, q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    nb = F.store_attend_workspace_bytes(ks, 1, 1, 4)
    got = []
    for _ in range(20):
        got.append(F.store_attend(ks, vs, q, stream=side))
        torch.empty(nb, dtype=torch.uint8, device=DEV).fill_(255)     # would be the workspace of the call before
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_misaligned_pointers_and_empty_batches_are_refused():
    ks, vs = make_store(100, 2, 64, 1), make_store(100, 2, 64, 2)
    ws = torch.empty(F.store_attend_workspace_bytes(ks, 1, 1, 8), dtype=torch.uint8, device=DEV)
    buf, out = torch.zeros(8 * 64 * 4 + 16, dtype=torch.uint8, device=DEV), torch.zeros(8 * 64 + 4, device=DEV)
    L, p, o = F.lib(), buf.data_ptr(), out.data_ptr()
    for at, dt, dst in ((p + 2, F.F32, o), (p + 1, F.BF16, o), (p, F.BF16, o + 2)):
        assert L.fathom_store_attend(ks.c, vs.c, at, dt, 1, 8, 1, dst, ws.data_ptr(), ws.numel(), None) == F.EINVAL
    assert L.fathom_store_attend(ks.c, vs.c, p + 2, F.BF16, 1, 8, 1, o + 4, ws.data_ptr(), ws.numel(), None) == F.OK
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        F.store_attend_batched([], [], torch.zeros(0, 1, 8, 64, device=DEV))


@pytest.mark.parametrize("n,d,G", [(131072, 64, 4), (60000, 128, 8), (4000, 256, 2)])
def test_long_sums_are_not_biased(n, d, G):
    """Flat weights over many keys: outputs are small beside the values, so an error that every block makes alike would show.
    The errors of the weights are independent and of both signs: of a logit, 2^-21 / sqrt(12) (qmax Delta_max <= 1.5) in
    each of d channels times codes of rms 3.3, over sqrt(d): 4e-7 rms; exp2 and the rounding of F S - m less than that.  The
    sums of a warp and of the partials are fp32, their rounding 2^-24 times the root of some hundred steps: 6e-7.  Bound: 2^-18,
    five times their sum in squares."""
    ks, vs = make_store(n, 1, d, n, spread=0.0), make_store(n, 1, d, n + 1, spread=0.0)
    q = queries((1, G, d), n % 97)
    ref, _, _, _ = reference(ks, vs, q, n)
    out = F.store_attend(ks, vs, q).double().cpu().numpy()
    assert np.linalg.norm(out - ref) <= 2.0 ** -18 * np.linalg.norm(ref)
    assert abs((out - ref).mean()) <= 2.0 ** -18 * np.abs(ref).mean()


@pytest.mark.parametrize("G,T,d,dtype", [(1, 1, 128, torch.float32), (4, 1, 32, torch.bfloat16), (8, 1, 128, torch.bfloat16),
                                         (8, 1, 256, torch.float32), (2, 5, 64, torch.bfloat16)])
@pytest.mark.parametrize("n", [513, 1024, 1025, 1537, 2049, 2561, 3584, 3585, 4096, 4097])
def test_short_rows_of_one_cluster(n, G, T, d, dtype):
    """2 to 8 half tiles to a row, some of a cluster's CTAs without any; and the row's partials."""
    ks, vs = make_store(n, 2, d, n, garbage=True), make_store(n, 2, d, n + 1, garbage=True)
    q = queries((T, 2 * G, d), n % 89, dtype)
    ref, tol, M, L = reference(ks, vs, q, n - T + 1)
    check(F.store_attend(ks, vs, q), ref, tol)
    parts = F.store_attend_partial(ks, vs, q, n - T + 1).double().cpu().numpy()
    assert (parts[..., d] >= M - 1e-4).all() and (parts[..., d] < M + 1 + 1e-4).all()
    check(torch.from_numpy(parts[..., :d] / parts[..., d + 1:]), ref, tol)


@pytest.mark.parametrize("T", [600, 1500])
def test_short_rows_whose_tokens_see_few_tiles(T):
    """Sets of tokens before the first key, in its tile, and behind: CTAs of a cluster that see nothing."""
    n = 1400
    ks, vs = make_store(n, 1, 32, T), make_store(n, 1, 32, T + 1)
    q = queries((T, 1, 32), T)
    ref, tol, _, _ = reference(ks, vs, q, n - T + 1)
    check(F.store_attend(ks, vs, q), ref, tol)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sets_of_eight_in_half_tiles(d, dtype):
    n = 9300
    ks, vs = make_store(n, 4, d, d), make_store(n, 4, d, d + 1)
    q = queries((32, d), d, dtype)
    ref, tol, _, _ = reference(ks, vs, q[None], n)
    check(F.store_attend(ks, vs, q), ref, tol)


def test_calls_from_several_threads():
    """Host threads with a stream each, short and long rows at once."""
    from concurrent.futures import ThreadPoolExecutor
    work = []
    for i, n in enumerate((700, 3000, 9000, 60000)):
        ks, vs = make_store(n, 2, 64, i), make_store(n, 2, 64, i + 10)
        q = queries((16, 64), i)
        work.append((ks, vs, q, F.store_attend(ks, vs, q), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def go(w):
        ks, vs, q, _, stream = w
        with torch.cuda.device(DEV):
            outs = [F.store_attend(ks, vs, q, stream=stream) for _ in range(50)]
            stream.synchronize()
        return outs

    with ThreadPoolExecutor(4) as pool:
        for w, outs in zip(work, pool.map(go, work)):
            assert all(torch.equal(o, w[3]) for o in outs)
    assert F.last_device_status() == 0
