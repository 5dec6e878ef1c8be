"""Attention over stores (fathom_store_attend, _batched) where a CTA takes several tiles: runs that end inside a row,
pass into the next row, KV head and session, and wrap the ring of copies, against the definition in 64 bits.

Bound of the error's norm relative to the output's, head by head: 2^-17.  The stores' channels have one magnitude, so
the weights are flat and the errors below are independent from key to key, as the summed values themselves are:
- logits.  A product q Delta is held to 2^-22 of itself or 2^-25 of max |q| max Delta (at most 6 and 1: 2^-22.4),
  uniform, times a code offset of at most 7.5 (rms 3.3), over d channels and sqrt(d): at most 2^-22 3.3 / sqrt(3) < 2^-21 rms.
  The fp32 sums behind it: sqrt(d/16 + 6) roundings of 2^-23 of a logit's magnitude, at most 16 where the weight
  counts: 2^-23 16 sqrt(22) < 2^-16.7 for a single logit of that size, for the weights' mean (|logit| about 1) 2^-20.7.
- weights.  A low half is rounded to 2^-23 of the block's largest weight, which is e^3 of the mean at most, against
  weights whose root mean square is e^1 of it: 2^-23 e^2 / sqrt(3) < 2^-20.8.
- sums.  fp32, at most some hundred steps of a random walk: sqrt(100) 2^-25 < 2^-21.6.
Their root sum of squares is below 2^-19.5; 2^-17 leaves a factor of five.  A tile that is missing, counted twice or taken
from another row changes the output by 1/sqrt(tiles), 2^-6 at the least.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from bit_plane_key_b200 import fathom as F  # noqa: E402
from test_gpu_store_attend import make_store, queries  # noqa: E402

DEV = torch.device("cuda:0")


def head_values(st, g):
    """The values f64 [n][d] of KV head g, on the GPU."""
    n = st.n
    P, S = st.planes[g], st.scales[g].view(torch.float16).double()
    bits = torch.arange(32, device=DEV, dtype=torch.int32)
    code = sum((((P[:, j].unsqueeze(-1) >> bits) & 1) << (3 - j)) for j in range(4)).flatten(1)[:, :n]
    return ((code.double() - 7.5) * S.repeat_interleave(64, 1)[:, :n]).t()


def check_runs(out, ks, vs, q, causal=True):
    """out and q [T][Hq][d] of one session."""
    T, Hq, d = q.shape
    n, G = ks.n, Hq // ks.n_kv_heads
    for g in range(ks.n_kv_heads):
        if n == 0:
            assert (out == 0).all()
            return
        K, V = head_values(ks, g), head_values(vs, g)
        for t in range(T):
            see = max(0, min(n, n - T + 1 + t)) if causal else n
            got = out[t, g * G:(g + 1) * G].double()
            if see == 0:
                assert (got == 0).all()
                continue
            w = torch.softmax(q[t, g * G:(g + 1) * G].double() @ K[:see].t() / math.sqrt(d), -1)
            want = w @ V[:see]
            err = ((got - want).norm(dim=-1) / want.norm(dim=-1)).max().item()
            assert err <= 2.0 ** -17, (g, t, err)


def units(lens, Hkv, G, T, pairs):
    return sum(-(-n // 1024) for n in lens) * Hkv * -(-(T * G) // pairs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,G,T,n", [(32, 4, 1, 132100), (64, 4, 1, 132100), (128, 4, 1, 132100), (256, 4, 1, 60001),
                                     (32, 8, 1, 60001), (64, 8, 1, 60001), (128, 8, 1, 132100), (256, 8, 1, 60001),
                                     (128, 4, 3, 60001), (64, 1, 2, 132100)])
def test_runs_of_one_session(d, G, T, n, dtype):
    Hkv = 8
    pairs = 4 if T * G <= 4 else 8
    resident = 296 if pairs == 4 and d <= 128 else 148
    U = units([n], Hkv, G, T, pairs)
    assert U >= 3 * resident and U % resident and -(-n // 1024) % (U // resident)   # several tiles each, run ends inside rows
    ks, vs = make_store(n, Hkv, d, d, spread=0.0), make_store(n, Hkv, d, d + 1, spread=0.0, capacity=n + 5000)
    q = queries((T, Hkv * G, d), d + G, dtype)
    check_runs(F.store_attend(ks, vs, q), ks, vs, q)
    assert F.last_device_status() == 0


def test_ten_tiles_to_a_cta():
    n, Hkv, d = 400001, 8, 128
    ks, vs = make_store(n, Hkv, d, 1, spread=0.0), make_store(n, Hkv, d, 2, spread=0.0)
    q = queries((1, 4 * Hkv, d), 5)
    check_runs(F.store_attend(ks, vs, q), ks, vs, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,G,T", [(32, 4, 1), (64, 4, 1), (64, 8, 3), (128, 4, 1), (128, 8, 1), (128, 4, 3), (256, 4, 1), (256, 8, 3)])
def test_runs_over_sessions(d, G, T, dtype):
    """Long sessions, and short and empty ones inside runs: copies ahead that change tensor maps, rows and lengths."""
    Hkv, lens = 8, [1, 0, 60000, 65, 0, 100001, 1024, 3, 2049, 0]
    pairs = 4 if T * G <= 4 else 8
    assert units(lens, Hkv, G, T, pairs) > 4 * (296 if pairs == 4 and d <= 128 else 148)
    ks = [make_store(n, Hkv, d, 10 + i, spread=0.0, capacity=n + 700 * i, garbage=True) for i, n in enumerate(lens)]
    vs = [make_store(n, Hkv, d, 50 + i, spread=0.0, garbage=True) for i, n in enumerate(lens)]
    q = queries((len(lens), T, Hkv * G, d), d + T, dtype)
    out = F.store_attend_batched(ks, vs, q)
    full = F.store_attend_batched(ks, vs, q, causal=False)
    for s in range(len(lens)):
        check_runs(out[s], ks[s], vs[s], q[s])
        check_runs(full[s], ks[s], vs[s], q[s], causal=False)
    assert F.last_device_status() == 0


def test_runs_over_two_groups_of_sessions():
    """More sessions than a launch takes, each with rows of several tiles: two launches that share a workspace."""
    Hkv, d = 4, 64
    lens = [1024 * (i % 7) + 37 * i for i in range(40)]
    ks = [make_store(n, Hkv, d, 10 + i, spread=0.0) for i, n in enumerate(lens)]
    vs = [make_store(n, Hkv, d, 90 + i, spread=0.0) for i, n in enumerate(lens)]
    q = queries((len(lens), 1, Hkv * 4, d), 3)
    out = F.store_attend_batched(ks, vs, q)
    for s in range(len(lens)):
        check_runs(out[s], ks[s], vs[s], q[s])


def test_repeated_queries_repeat_their_outputs():
    """Sixteen heads that repeat four: against the definition, and the same bits for the same queries of a KV head."""
    n, Hkv, d = 50000, 4, 128
    ks, vs = make_store(n, Hkv, d, 80, spread=0.0), make_store(n, Hkv, d, 81, spread=0.0)
    q = queries((4, d), 9).repeat(4, 1)[:, None].expand(16, 2, d).reshape(1, 32, d).contiguous()
    out = F.store_attend(ks, vs, q)
    check_runs(out, ks, vs, q)
    assert torch.equal(out[0, 0::2], out[0, 1::2])
