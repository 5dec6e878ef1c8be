// Attention over the 4-bit stores themselves: every key of a K store and the
// values of a V store, both in bit planes.
//
//   s_i = q . K_i / sqrt(d),  K_ic = Delta_c,b(i) (code_ic - 7.5),  V likewise,
//   out = sum_i exp(s_i) V_i / sum_i exp(s_i)
//
// over the keys a query may see, in one pass with a running maximum and sum.
//
// The keys of a (session, KV head, set of queries) are a row of tiles of
// kTile keys.  All rows' tiles form one list, cut into equal runs, one per
// CTA; a run may end in the middle of a row, so every (CTA, row) pair leaves a
// partial (o, m, l), and a second launch adds a row's partials in order.
// CTA p's partial of row r lies in slot p + r: a run that passes into the next
// row raises r, a row that passes into the next CTA raises p, so no two meet.
#include "fathom_internal.cuh"

namespace fathom {
namespace {

constexpr int kTile = 512;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPairs = 4;   // (query token, head of the group) pairs per set

// unit range of CTA p of P over U units, and the CTA of a unit
__device__ __forceinline__ int64_t run_start(int64_t p, int64_t U, int64_t P) { return p * U / P; }
__device__ __forceinline__ int64_t cta_of(int64_t u, int64_t U, int64_t P) { return ((u + 1) * P - 1) / U; }

// a row's place: session, KV head, set, and its first unit
struct RowAt {
    int s, g, set;
    int64_t row, unit0;
};
__device__ __forceinline__ int session_of_unit(const AttendMap& m, int64_t u) {
    int lo = 0, hi = m.nsess;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (m.unit0[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
store_attend_kernel(const __grid_constant__ AttendMap map, const void* __restrict__ q, int q_dtype, int T, int Hq, int Hkv, int sets,
                    float* __restrict__ slots) {
    __shared__ float s_q[kPairs][D];
    __shared__ float s_p[kPairs][kTile];
    __shared__ float s_o[kPairs][D];
    __shared__ float s_red[kWarps];
    const int64_t U = map.unit0[map.nsess], P = gridDim.x;
    const int64_t u0 = run_start(blockIdx.x, U, P), u1 = run_start(blockIdx.x + 1, U, P);
    const int G = Hq / Hkv, C = T * G;
    const float scale = 1.4426950408889634f / sqrtf((float)D);
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;

    int64_t u = u0;
    while (u < u1) {
        const int s = session_of_unit(map, u);
        const int tiles = map.tiles[s];
        const int64_t in = u - map.unit0[s];
        const int rl = (int)(in / tiles);
        const int g = rl / sets, set = rl % sets;
        const int64_t row = (int64_t)s * Hkv * sets + rl;
        const int64_t row_end = map.unit0[s] + (int64_t)(rl + 1) * tiles;
        const int64_t ue = row_end < u1 ? row_end : u1;
        __syncthreads();
        for (int e = threadIdx.x; e < kPairs * D; e += kThreads) {
            const int x = e / D, c = e % D, pr = set * kPairs + x;
            s_q[x][c] = pr < C ? load_q(q, q_dtype, (((int64_t)s * T + pr / G) * Hq + g * G + pr % G) * D + c) * scale : 0.0f;
            s_o[x][c] = 0.0f;
        }
        float m[kPairs], l[kPairs];
        for (int x = 0; x < kPairs; ++x) m[x] = -INFINITY, l[x] = 0.0f;
        const int64_t kw = map.k_pad[s] / 32, vw = map.v_pad[s] / 32;
        const uint32_t* Kp = map.k_planes[s] + (int64_t)g * D * 4 * kw;
        const uint16_t* Ks = map.k_scales[s] + (int64_t)g * D * (kw / 2);
        const uint32_t* Vp = map.v_planes[s] + (int64_t)g * D * 4 * vw;
        const uint16_t* Vs = map.v_scales[s] + (int64_t)g * D * (vw / 2);
        for (; u < ue; ++u) {
            const int64_t i0 = (u - (row_end - tiles)) * kTile;
            __syncthreads();
            for (int e = threadIdx.x; e < kTile; e += kThreads) {
                const int64_t i = i0 + e;
                float acc[kPairs] = {};
                if (i < map.n[s]) {
                    for (int c = 0; c < D; ++c) {
                        int code = 0;
                        for (int j = 0; j < 4; ++j) code |= ((Kp[(c * 4 + j) * kw + i / 32] >> (i & 31)) & 1) << (3 - j);
                        const float k = __half2float(__ushort_as_half(Ks[c * (kw / 2) + i / kBlock])) * ((float)code - 7.5f);
                        for (int x = 0; x < kPairs; ++x) acc[x] = fmaf(s_q[x][c], k, acc[x]);
                    }
                }
                for (int x = 0; x < kPairs; ++x) {
                    const int pr = set * kPairs + x;
                    const bool see = pr < C && i < map.n[s] && i < map.visible[s] + pr / G;
                    s_p[x][e] = see ? acc[x] : -INFINITY;
                }
            }
            for (int x = 0; x < kPairs; ++x) {
                __syncthreads();
                float mx = fmaxf(s_p[x][threadIdx.x], s_p[x][threadIdx.x + kThreads]);
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (lane == 0) s_red[wp] = mx;
                __syncthreads();
                float mn = m[x];
                for (int w = 0; w < kWarps; ++w) mn = fmaxf(mn, s_red[w]);
                const float base = mn == -INFINITY ? 0.0f : mn;
                __syncthreads();
                float sum = 0.0f;
                for (int e = threadIdx.x; e < kTile; e += kThreads) {
                    const float p = exp2f(s_p[x][e] - base);
                    s_p[x][e] = p;
                    sum += p;
                }
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) s_red[wp] = sum;
                __syncthreads();
                const float f = exp2f(m[x] - base);   // 0 while nothing has been seen
                l[x] *= f;
                for (int w = 0; w < kWarps; ++w) l[x] += s_red[w];
                for (int c = threadIdx.x; c < D; c += kThreads) s_o[x][c] *= f;
                m[x] = mn;
            }
            __syncthreads();
            const int nk = (int)(map.n[s] - i0 < kTile ? map.n[s] - i0 : kTile);
            for (int c = threadIdx.x; c < D; c += kThreads) {
                float acc[kPairs] = {};
                for (int e = 0; e < nk; ++e) {
                    const int64_t i = i0 + e;
                    int code = 0;
                    for (int j = 0; j < 4; ++j) code |= ((Vp[(c * 4 + j) * vw + i / 32] >> (i & 31)) & 1) << (3 - j);
                    const float v = __half2float(__ushort_as_half(Vs[c * (vw / 2) + i / kBlock])) * ((float)code - 7.5f);
                    for (int x = 0; x < kPairs; ++x) acc[x] = fmaf(s_p[x][e], v, acc[x]);
                }
                for (int x = 0; x < kPairs; ++x) s_o[x][c] += acc[x];
            }
        }
        float* slot = slots + (blockIdx.x + row) * kPairs * (D + 2);
        __syncthreads();
        for (int e = threadIdx.x; e < kPairs * D; e += kThreads) slot[e / D * (D + 2) + e % D] = s_o[e / D][e % D];
        if (threadIdx.x == 0)
            for (int x = 0; x < kPairs; ++x) {
                slot[x * (D + 2) + D] = m[x];
                slot[x * (D + 2) + D + 1] = l[x];
            }
    }
}

// One CTA per (row, pair): the row's partials in order, normalised into out, or
// left as (o, m, l) in parts.
__global__ void __launch_bounds__(128)
store_attend_merge_kernel(const __grid_constant__ AttendMap map, const float* __restrict__ slots, int T, int Hq, int Hkv, int sets, int D,
                          int P, float* __restrict__ out, float* __restrict__ parts) {
    pdl_wait();
    const int G = Hq / Hkv, C = T * G;
    const int64_t row = blockIdx.x / kPairs;
    const int x = blockIdx.x % kPairs;
    const int s = (int)(row / (Hkv * sets)), rl = (int)(row % (Hkv * sets));
    const int g = rl / sets, pr = rl % sets * kPairs + x;
    if (pr >= C) return;
    const int64_t U = map.unit0[map.nsess];
    const int64_t ub = map.unit0[s] + (int64_t)rl * map.tiles[s], ue = ub + map.tiles[s];
    int64_t p0 = 0, p1 = 0;
    if (ue > ub) p0 = cta_of(ub, U, P), p1 = cta_of(ue - 1, U, P) + 1;
    const int64_t st = (int64_t)kPairs * (D + 2);
    const float* base = slots + row * st + x * (D + 2);
    float M = -INFINITY, L = 0.0f;
    for (int64_t p = p0; p < p1; ++p) M = fmaxf(M, base[p * st + D]);
    const float Mb = M == -INFINITY ? 0.0f : M;
    for (int64_t p = p0; p < p1; ++p) L = fmaf(base[p * st + D + 1], exp2f(base[p * st + D] - Mb), L);
    const int64_t h = ((int64_t)s * T + pr / G) * Hq + g * G + pr % G;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float O = 0.0f;
        for (int64_t p = p0; p < p1; ++p) O = fmaf(base[p * st + c], exp2f(base[p * st + D] - Mb), O);
        if (parts) parts[h * (D + 2) + c] = O;
        else out[h * D + c] = L > 0.0f ? O / L : 0.0f;
    }
    if (parts && threadIdx.x == 0) {
        parts[h * (D + 2) + D] = M;
        parts[h * (D + 2) + D + 1] = L;
    }
}

}  // namespace

int64_t store_attend_tiles(int64_t keys) { return (keys + kTile - 1) / kTile; }

namespace {
constexpr int kMaxCtas = 592;   // 148 SMs, four CTAs each
inline int64_t n_sets(int T, int Hq, int Hkv) { return ((int64_t)T * (Hq / Hkv) + kPairs - 1) / kPairs; }
}  // namespace

size_t store_attend_workspace_bytes(int S, int T, int Hq, int Hkv, int d) {
    const size_t slots = (size_t)S * Hkv * (size_t)n_sets(T, Hq, Hkv) + kMaxCtas;
    return (slots * kPairs * (d + 2) * sizeof(float) + 255) & ~size_t(255);
}

cudaError_t launch_store_attend(AttendMap& map, int Hkv, int d, const void* q, int q_dtype, int T, int Hq, float* out,
                                float* parts, void* ws, cudaStream_t stream) {
    const int sets = (int)n_sets(T, Hq, Hkv);
    int64_t U = 0;
    for (int s = 0; s < map.nsess; ++s) {
        const int64_t last = map.visible[s] + T - 1;   // keys that the last token sees
        const int64_t keys = last < map.n[s] ? (last > 0 ? last : 0) : map.n[s];
        map.unit0[s] = U;
        map.tiles[s] = (int)store_attend_tiles(keys);
        U += (int64_t)map.tiles[s] * Hkv * sets;
    }
    map.unit0[map.nsess] = U;
    float* slots = static_cast<float*>(ws);
    const int P = (int)(U < kMaxCtas ? U : kMaxCtas);
    if (U > 0) {
        auto go = [&](auto kern) {
            return launch_ex(kern, dim3(P), dim3(kThreads), 0, stream, false, 1, map, q, q_dtype, T, Hq, Hkv, sets,
                             slots);
        };
        cudaError_t e;
        switch (d) {
            case 32: e = go(store_attend_kernel<32>); break;
            case 64: e = go(store_attend_kernel<64>); break;
            case 128: e = go(store_attend_kernel<128>); break;
            case 256: e = go(store_attend_kernel<256>); break;
            default: return cudaErrorInvalidValue;
        }
        if (e != cudaSuccess) return e;
    }
    return launch_ex(store_attend_merge_kernel, dim3((unsigned)((int64_t)map.nsess * Hkv * sets * kPairs)), dim3(128), 0,
                     stream, U > 0, 1, map, slots, T, Hq, Hkv, sets, d, P, out, parts);
}

}  // namespace fathom
