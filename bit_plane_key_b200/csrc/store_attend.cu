// Attention over the 4-bit stores themselves: every key of a K store and the
// values of a V store, both in bit planes.
//
//   s_i = q . K_i / sqrt(d),  K_ic = Delta_c,b(i) (code_ic - 7.5),  V likewise,
//   out = sum_i exp(s_i) V_i / sum_i exp(s_i)
//
// over the keys a query may see, in one pass with a running maximum and sum.
//
// Work split.  The keys of a (session, KV head, set of queries) are a row of
// tiles of kTile keys.  All rows' tiles form one list, cut into equal runs,
// one per CTA; a run may end in the middle of a row, so every (CTA, row) pair
// leaves a partial (o, m, l), and a second launch adds a row's partials in
// order.  CTA p's partial of row r lies in slot p + r: a run that passes into
// the next row raises r, a row that passes into the next CTA raises p, so no
// two meet.
//
// A tile.  The CTA's warps turn the plane words of 8 blocks of 64 keys into
// words of 4-bit codes in shared memory, laid out so that one 16-byte load is
// a lane's share of a matrix operand; then each warp takes one block through
// both products, m16n8k16 on fp16 with fp32 sums:
//   S (64 keys x columns) = codes . Q',  Q'_c = q_c Delta_c of this block,
//   O (d x columns) += Delta_c (codes . P).
// A code needs no conversion: the bits 0..15 of an fp16 are the subnormal
// code 2^-24, exactly, and shifted by 4 bits 16 times that, so one AND makes
// two operand values; the factors are undone in the scaling of S and P, and
// the offset 7.5 by one more product with a constant 15.
// Q' and P are split into two fp16 halves of 11 bits each, which sit in
// neighbouring columns, so that a column pair of the 8 is one query in 22
// bits: the products lose no more than fp32 arithmetic would.  Scores never
// leave the warp: a transposing move of 8x8 matrices makes the P operand of
// the S accumulators.
#include "fathom_internal.cuh"

namespace fathom {
namespace {

constexpr int kTileBlocks = 8;                  // one per warp
constexpr int kTile = kTileBlocks * kBlock;
constexpr int kThreads = 32 * kTileBlocks;
constexpr int kTilePairs = 4;                   // queries per 8 columns
constexpr int kMaxCtas = 592;                   // bound for the workspace: 148 SMs, four CTAs each

template <int D, int NT>
struct Shape {
    static constexpr int kPairs = kTilePairs * NT;          // (token, head of the group) pairs of a set
    static constexpr int kBlkWords = D * 8 + 4;             // code words of a block, 4 of padding against bank conflicts
    static constexpr int kCodes = kTileBlocks * kBlkWords;  // of K, and of V
    static constexpr int kScaleHalves = kTileBlocks * D;
    static constexpr size_t kSmem = 4 * (size_t)(2 * kCodes) + 2 * 2 * kScaleHalves + 4 * (size_t)(kPairs * D) +
                                    4 * (size_t)(2 * kTileBlocks * kPairs + kPairs);
    static constexpr int kCtasPerSm = (D == 256 || NT == 4) ? 1 : 2;
    // the warps' partial outputs reuse the code words
    static_assert(kTileBlocks * kPairs * D <= 2 * kCodes, "partial outputs fit");
};

// first unit of run p of P over U units, and the run of a unit
__device__ __forceinline__ int64_t run_start(int64_t p, int64_t U, int64_t P) { return p * U / P; }
__device__ __forceinline__ int64_t run_of(int64_t u, int64_t U, int64_t P) { return ((u + 1) * P - 1) / U; }

__device__ __forceinline__ int session_of_unit(const AttendMap& m, int64_t u) {
    int lo = 0, hi = m.nsess;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (m.unit0[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void mma(float* c, const uint32_t* a, const uint32_t* b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (low, high) as two fp16
__device__ __forceinline__ uint32_t half2_of(float low, float high) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(high), "f"(low));
    return r;
}
// the leading 11 significant bits
__device__ __forceinline__ float leading11(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFFE000u); }

// plane words W[j] of 32 keys -> N[r]: nibble m = code of key 4 m + r
__device__ __forceinline__ void planes_to_nibbles(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t* N) {
    const uint32_t E = ((w0 << 1) & 0xAAAAAAAAu) | (w1 & 0x55555555u), O = (w0 & 0xAAAAAAAAu) | ((w1 >> 1) & 0x55555555u);
    const uint32_t F = ((w2 << 1) & 0xAAAAAAAAu) | (w3 & 0x55555555u), H = (w2 & 0xAAAAAAAAu) | ((w3 >> 1) & 0x55555555u);
    N[0] = ((E << 2) & 0xCCCCCCCCu) | (F & 0x33333333u);
    N[2] = (E & 0xCCCCCCCCu) | ((F >> 2) & 0x33333333u);
    N[1] = ((O << 2) & 0xCCCCCCCCu) | (H & 0x33333333u);
    N[3] = (O & 0xCCCCCCCCu) | ((H >> 2) & 0x33333333u);
}

// operand value pairs p = 0..3 of a word of codes (odd p: 16 times the code)
__device__ __forceinline__ void operand(const uint4& raw, int p, uint32_t* a) {
    const uint32_t mask = (p & 1) ? 0x00F000F0u : 0x000F000Fu;
    const int sh = (p & 2) ? 8 : 0;
    a[0] = (raw.x >> sh) & mask;
    a[1] = (raw.y >> sh) & mask;
    a[2] = (raw.z >> sh) & mask;
    a[3] = (raw.w >> sh) & mask;
}

// Where the keys of a tile lie in the operands (block b = its warp): key
// 32 w + 4 (p + 4 k4) + r of the block is nibble p of half k4 of N[r] of word w.
//   S: row g = 2 r + k4 (w = 0) or that plus 8 (w = 1) of m-tile p; a lane's
//      columns k are the channels 16 ks + 4 t + 0..3.
//   O: row g is channel 16 mt + 2 g, row g + 8 the next; k-step p, column
//      pair t is r = t, k4 = 0 and 1, w = 0 then w = 1.
// Both orders meet: the transposed S accumulators of rows g = 2 t, 2 t + 1 are
// the P operand's k columns 2 t, 2 t + 1.

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kCtasPerSm)
store_attend_kernel(const __grid_constant__ AttendMap map, const void* __restrict__ q, int q_dtype, int T, int Hq,
                    int Hkv, int sets, float* __restrict__ slots, float* __restrict__ out, float* __restrict__ parts) {
    using Sh = Shape<D, NT>;
    constexpr int KS = D / 16;        // 16-channel steps
    constexpr int kPairs = Sh::kPairs;
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t* s_k = smem;                               // [block][ks][lane][4] code words
    uint32_t* s_v = s_k + Sh::kCodes;                   // [block][mt][lane][4]
    uint16_t* s_ks = reinterpret_cast<uint16_t*>(s_v + Sh::kCodes);   // [block][D] scales
    uint16_t* s_vs = s_ks + Sh::kScaleHalves;
    float* s_q = reinterpret_cast<float*>(s_vs + Sh::kScaleHalves);   // [NT][ks][4 pairs][16 channels]
    float* s_m = s_q + kPairs * D;                      // [warp][pair]
    float* s_l = s_m + kTileBlocks * kPairs;
    float* s_f = s_l + kTileBlocks * kPairs;            // [pair] 1 / the query's normalisation

    const int64_t U = map.unit0[map.nsess], P = gridDim.x;
    const int64_t u1 = run_start(blockIdx.x + 1, U, P);
    int64_t u = run_start(blockIdx.x, U, P);
    const int G = Hq / Hkv, C = T * G;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int lg = lane >> 2, lt = lane & 3;            // g and t of the operand layouts
    const bool low = lg & 1;                            // this lane's column is the low half of its query

    while (u < u1) {
        const int s = session_of_unit(map, u);
        const int tiles = map.tiles[s];
        const int rl = (int)((u - map.unit0[s]) / tiles);
        const int g = rl / sets, set = rl % sets;
        const int64_t row = (int64_t)s * Hkv * sets + rl;
        const int64_t row0 = map.unit0[s] + (int64_t)rl * tiles, row1 = row0 + tiles;
        const int64_t ue = row1 < u1 ? row1 : u1;
        const bool whole = u == row0 && ue == row1;     // no other CTA has a share of this row
        const int64_t kw = map.k_pad[s] / 32, vw = map.v_pad[s] / 32;
        const uint32_t* Kp = map.k_planes[s] + (int64_t)g * D * 4 * kw;
        const uint16_t* Ks = map.k_scales[s] + (int64_t)g * D * (kw / 2);
        const uint32_t* Vp = map.v_planes[s] + (int64_t)g * D * 4 * vw;
        const uint16_t* Vs = map.v_scales[s] + (int64_t)g * D * (vw / 2);
        const int n = (int)map.n[s];

        // the set's queries, each divided by a power of two to at most 1 to 2 in magnitude
        __syncthreads();
        for (int x = wp; x < kPairs; x += kTileBlocks) {
            const int pr = set * kPairs + x;
            float v[(D + 31) / 32];
            float mx = 0.0f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                v[e] = pr < C ? load_q(q, q_dtype, (((int64_t)s * T + pr / G) * Hq + g * G + pr % G) * D + 32 * e + lane) : 0.0f;
                mx = fmaxf(mx, fabsf(v[e]));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            int ex = 0;
            if (mx > 0.0f) ex = ilogbf(mx);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const int c = 32 * e + lane;
                s_q[(((x >> 2) * KS + (c >> 4)) * 4 + (x & 3)) * 16 + (c & 15)] = ldexpf(v[e], -ex);
            }
            // logits in log2 units = sums of products * this * 2^24 / the block's factor;
            // never 0, which a masked score of -inf would turn into NaN
            if (lane == 0) s_f[x] = fmaxf(ldexpf(1.4426950408889634f / sqrtf((float)D), ex), 1.17549435e-38f);
        }

        float O[NT][KS][2], m[NT], l[NT];
        int limit[NT], least = n;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt] = -INFINITY;
            l[nt] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) O[nt][mt][0] = O[nt][mt][1] = 0.0f;
            const int64_t see = map.visible[s] + (set * kPairs + nt * kTilePairs + lt) / G;
            limit[nt] = (int)(see < n ? (see > 0 ? see : 0) : n);
        }
        {   // the set's first pair sees the fewest keys
            const int64_t see = map.visible[s] + set * kPairs / G;
            if (see < n) least = (int)(see > 0 ? see : 0);
        }

        for (; u < ue; ++u) {
            const int i0 = (int)(u - row0) * kTile;
            __syncthreads();                            // the tile before has been read
            // ---- codes and scales of the tile into shared memory
            {
                const int b = lane & 7;                 // a lane's block; its channels: four in a row
#pragma unroll
                for (int st = wp; st < 2 * KS; st += kTileBlocks) {
                    const bool isk = st < KS;
                    const int quad = (isk ? st : st - KS) * 4 + (lane >> 3);
                    const int64_t words = isk ? kw : vw;
                    const uint32_t* src = (isk ? Kp : Vp) + (int64_t)quad * 16 * words + i0 / 32 + 2 * b;
                    uint2 W[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j) W[e][j] = __ldg(reinterpret_cast<const uint2*>(src + (e * 4 + j) * words));
                    uint32_t N[4][2][4];                // [channel][word][r]
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        planes_to_nibbles(W[e][0].x, W[e][1].x, W[e][2].x, W[e][3].x, N[e][0]);
                        planes_to_nibbles(W[e][0].y, W[e][1].y, W[e][2].y, W[e][3].y, N[e][1]);
                    }
                    if (isk) {
                        uint4* dst = reinterpret_cast<uint4*>(s_k + b * Sh::kBlkWords + (quad >> 2) * 128) + (quad & 3);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int k4 = 0; k4 < 2; ++k4) {
                                const uint32_t sel = k4 ? 0x7632u : 0x5410u;
                                dst[(2 * r + k4) * 4] =
                                    make_uint4(__byte_perm(N[0][0][r], N[1][0][r], sel), __byte_perm(N[0][1][r], N[1][1][r], sel),
                                               __byte_perm(N[2][0][r], N[3][0][r], sel), __byte_perm(N[2][1][r], N[3][1][r], sel));
                            }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(s_v + b * Sh::kBlkWords + (quad >> 2) * 128) + (quad & 3) * 8;
#pragma unroll
                        for (int gi = 0; gi < 2; ++gi)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                dst[gi * 4 + r] = make_uint4(N[2 * gi][0][r], N[2 * gi + 1][0][r], N[2 * gi][1][r], N[2 * gi + 1][1][r]);
                    }
                }
                for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
                    const bool isk = c < D;
                    const int ch = isk ? c : c - D;
                    const uint16_t* src = isk ? Ks + (int64_t)ch * (kw / 2) : Vs + (int64_t)ch * (vw / 2);
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + i0 / kBlock));
                    uint16_t* dst = (isk ? s_ks : s_vs) + ch;
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dst[(2 * e) * D] = (uint16_t)w[e];
                        dst[(2 * e + 1) * D] = (uint16_t)(w[e] >> 16);
                    }
                }
            }
            __syncthreads();
            const int k0 = i0 + wp * kBlock;            // this warp's block
            int most = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) most = limit[nt] > most ? limit[nt] : most;
            if (!__any_sync(0xffffffffu, k0 < most)) continue;

            // ---- S = codes . Q'
            const uint16_t* bs = s_ks + wp * D;
            // the block's largest scale sets a power of two that keeps Q' inside fp16
            float sc, back;   // back = 2^24 / sc
            {
                __half2 mh = __float2half2_rn(0.0f);
#pragma unroll
                for (int e = 0; e < (D + 63) / 64; ++e)
                    if (D >= 64 || lane < D / 2)
                        mh = __hmax2(mh, *reinterpret_cast<const __half2*>(bs + 2 * lane + 64 * e));
                float dm = fmaxf(__low2float(mh), __high2float(mh));
#pragma unroll
                for (int o = 16; o; o >>= 1) dm = fmaxf(dm, __shfl_xor_sync(0xffffffffu, dm, o));
                // dm * sc in [2^12, 2^13); an f16 is at least 2^-24
                const int ex = dm > 0.0f ? (int)(__float_as_uint(dm) >> 23) : 127;
                sc = __uint_as_float((uint32_t)(266 - ex) << 23);
                back = __uint_as_float((uint32_t)(ex + 12) << 23);
            }
            float S[NT][4][4], B15[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    B15[nt][e] = 0.0f;
#pragma unroll
                    for (int p = 0; p < 4; ++p) S[nt][p][e] = 0.0f;
                }
            const uint32_t a15[4] = {0x000F000Fu, 0x000F000Fu, 0x000F000Fu, 0x000F000Fu};
            const uint4* kc = reinterpret_cast<const uint4*>(s_k + wp * Sh::kBlkWords) + lane;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint4 raw = kc[ks * 32];
                const uint2 d4 = *reinterpret_cast<const uint2*>(bs + 16 * ks + 4 * lt);
                const float2 da = __half22float2(*reinterpret_cast<const __half2*>(&d4.x));
                const float2 db = __half22float2(*reinterpret_cast<const __half2*>(&d4.y));
                const float dl[4] = {da.x * sc, da.y * sc, db.x * sc, db.y * sc};
                uint32_t bq[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float4 q4 = *reinterpret_cast<const float4*>(s_q + ((nt * KS + ks) * 4 + (lg >> 1)) * 16 + 4 * lt);
                    const float v[4] = {q4.x * dl[0], q4.y * dl[1], q4.z * dl[2], q4.w * dl[3]};
                    float z[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float h = leading11(v[e]);
                        z[e] = low ? v[e] - h : h;
                    }
                    bq[nt][0] = half2_of(z[0], z[1]);
                    bq[nt][1] = half2_of(z[2], z[3]);
                    mma(B15[nt], a15, bq[nt]);
                }
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    uint32_t a[4];
                    operand(raw, p, a);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma(S[nt][p], a, bq[nt]);
                }
            }

            // ---- weights: lane (g, t) holds query t of the tile, 8 keys
            uint32_t Pb[NT][4][2];
            const bool cut = k0 + kBlock > least;       // some query of the set does not see the whole block
            float shift[NT];
            bool moved = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float off = -0.5f * (B15[nt][0] + B15[nt][1]);
                float mx = -INFINITY;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float f = (p & 1) ? 0.0625f : 1.0f;
                    S[nt][p][0] = fmaf(S[nt][p][0] + S[nt][p][1], f, off);
                    S[nt][p][2] = fmaf(S[nt][p][2] + S[nt][p][3], f, off);
                    if (cut) {
                        const int key = k0 + 4 * (p + 4 * (lg & 1)) + (lg >> 1);
                        if (key >= limit[nt]) S[nt][p][0] = -INFINITY;
                        if (key + 32 >= limit[nt]) S[nt][p][2] = -INFINITY;
                    }
                    mx = fmaxf(mx, fmaxf(S[nt][p][0], S[nt][p][2]));
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                float F = s_f[nt * kTilePairs + lt] * back;
                const float mn = fmaxf(m[nt], mx * F);
                const float base = mn == -INFINITY ? 0.0f : mn;
                // S F - base is rounded once; where the product's own rounding exceeds
                // the exponents that matter, both are rounded alike instead
                if (fabsf(base) > 1048576.0f) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        S[nt][p][0] *= F;
                        S[nt][p][2] *= F;
                    }
                    F = 1.0f;
                }
                shift[nt] = ex2(m[nt] - base);          // 0 while nothing has been seen
                moved |= mn != m[nt];
                m[nt] = mn;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    // weights times 2^15, or 2^11 where the codes come 16 times as large
                    const float up = (p & 1) ? 2048.0f : 32768.0f;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const float v = ex2(fmaf(S[nt][p][2 * w], F, -base)) * up;
                        const float h = leading11(v);
                        Pb[nt][p][w] = transpose8x8(half2_of(h, v - h));
                    }
                }
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    l[nt] *= shift[nt];
#pragma unroll
                    for (int mt = 0; mt < KS; ++mt) {
                        O[nt][mt][0] *= shift[nt];
                        O[nt][mt][1] *= shift[nt];
                    }
                }
            }
            // ---- 15 sum P: the offset of the codes, and the weights' sum
            float neg[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    uint32_t a[4];
                    operand(make_uint4(~0u, ~0u, ~0u, ~0u), p, a);
                    mma(c, a, Pb[nt][p]);
                }
                const float sum = c[0] + c[1];
                neg[nt] = -0.5f * sum;
                l[nt] = fmaf(sum, 512.0f / 15.0f, l[nt]);   // 2^24 / 2^15
            }
            // ---- O += Delta (codes - 7.5) . P
            const uint4* vc = reinterpret_cast<const uint4*>(s_v + wp * Sh::kBlkWords) + lane;
            const uint16_t* vs = s_vs + wp * D + 2 * lg;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                const uint4 raw = vc[mt * 32];
                const float2 dv = __half22float2(*reinterpret_cast<const __half2*>(vs + 16 * mt));
                float c[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][2] = neg[nt], c[nt][1] = c[nt][3] = 0.0f;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    uint32_t a[4];
                    operand(raw, p, a);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma(c[nt], a, Pb[nt][p]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    O[nt][mt][0] = fmaf(c[nt][0] + c[nt][1], dv.x, O[nt][mt][0]);
                    O[nt][mt][1] = fmaf(c[nt][2] + c[nt][3], dv.y, O[nt][mt][1]);
                }
            }
        }

        // ---- the warps' partials: merged here, o in units of 2^-9
        __syncthreads();
        float* s_o = reinterpret_cast<float*>(smem);    // [warp][pair][D]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int x = nt * kTilePairs + lt;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt)
                *reinterpret_cast<float2*>(s_o + (wp * kPairs + x) * D + 16 * mt + 2 * lg) = make_float2(O[nt][mt][0], O[nt][mt][1]);
            if (lg == 0) {
                s_m[wp * kPairs + x] = m[nt];
                s_l[wp * kPairs + x] = l[nt];
            }
        }
        __syncthreads();
        float* slot = slots + (blockIdx.x + row) * (kPairs * (D + 2));
        for (int e = threadIdx.x; e < kPairs * D; e += kThreads) {
            const int x = e / D, c = e % D, pr = set * kPairs + x;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kTileBlocks; ++w) M = fmaxf(M, s_m[w * kPairs + x]);
            const float Mb = M == -INFINITY ? 0.0f : M;
            float L = 0.0f, o = 0.0f;
#pragma unroll
            for (int w = 0; w < kTileBlocks; ++w) {
                const float f = ex2(s_m[w * kPairs + x] - Mb);
                L = fmaf(s_l[w * kPairs + x], f, L);
                o = fmaf(s_o[(w * kPairs + x) * D + c], f, o);
            }
            o *= 512.0f;
            if (!whole) {
                slot[e] = o;
                if (c == 0) slot[kPairs * D + x] = M, slot[kPairs * (D + 1) + x] = L;
            } else if (pr < C) {
                const int64_t h = ((int64_t)s * T + pr / G) * Hq + g * G + pr % G;
                if (parts) {
                    parts[h * (D + 2) + c] = o;
                    if (c == 0) parts[h * (D + 2) + D] = M, parts[h * (D + 2) + D + 1] = L;
                } else {
                    out[h * D + c] = L > 0.0f ? o / L : 0.0f;
                }
            }
        }
    }
}

// One CTA per (row, pair) whose keys were shared by several CTAs, or that has
// none: the row's partials, in an order that depends on their number alone.
constexpr int kMergeThreads = 256;
__global__ void __launch_bounds__(kMergeThreads)
store_attend_merge_kernel(const __grid_constant__ AttendMap map, const float* __restrict__ slots, int T, int Hq, int Hkv,
                          int sets, int pairs, int D, int P, float* __restrict__ out, float* __restrict__ parts) {
    __shared__ float s_w[kMaxCtas];
    __shared__ float s_red[2][kMergeThreads / 32];
    __shared__ float4 s_o[kMergeThreads];
    pdl_wait();
    const int G = Hq / Hkv, C = T * G;
    const int64_t row = blockIdx.x / pairs;
    const int x = blockIdx.x % pairs;
    const int s = (int)(row / (Hkv * sets)), rl = (int)(row % (Hkv * sets));
    const int g = rl / sets, pr = rl % sets * pairs + x;
    if (pr >= C) return;
    const int64_t U = map.unit0[map.nsess];
    const int64_t ub = map.unit0[s] + (int64_t)rl * map.tiles[s], ue = ub + map.tiles[s];
    int64_t p0 = 0;
    int np = 0;
    if (ue > ub) {
        p0 = run_of(ub, U, P);
        np = (int)(run_of(ue - 1, U, P) - p0) + 1;
        if (np == 1) return;                     // written by its CTA
    }
    const int64_t st = (int64_t)pairs * (D + 2);
    const float* base = slots + (p0 + row) * st;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    float M = -INFINITY;
    for (int p = threadIdx.x; p < np; p += kMergeThreads) {
        const float v = base[p * st + pairs * D + x];
        s_w[p] = v;
        M = fmaxf(M, v);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) s_red[0][wp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) M = fmaxf(M, s_red[0][w]);
    const float Mb = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    for (int p = threadIdx.x; p < np; p += kMergeThreads) {
        const float f = ex2(s_w[p] - Mb);
        s_w[p] = f;
        L = fmaf(base[p * st + pairs * (D + 1) + x], f, L);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) s_red[1][wp] = L;
    __syncthreads();
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) L += s_red[1][w];
    // D/4 threads take a partial's channels, the others further partials
    const int cl = D / 4, c4 = threadIdx.x % cl, grp = threadIdx.x / cl, ng = kMergeThreads / cl;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p = grp; p < np; p += ng) {
        const float4 v = *reinterpret_cast<const float4*>(base + p * st + x * D + 4 * c4);
        const float f = s_w[p];
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
    }
    s_o[threadIdx.x] = o;
    __syncthreads();
    if (grp) return;
    for (int e = 1; e < ng; ++e) {
        const float4 v = s_o[e * cl + c4];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    const int64_t h = ((int64_t)s * T + pr / G) * Hq + g * G + pr % G;
    if (parts) {
        float* dst = parts + h * (D + 2) + 4 * c4;
        dst[0] = o.x, dst[1] = o.y, dst[2] = o.z, dst[3] = o.w;
        if (c4 == 0) parts[h * (D + 2) + D] = M, parts[h * (D + 2) + D + 1] = L;
    } else {
        float* dst = out + h * D + 4 * c4;
        const float r = L > 0.0f ? L : 1.0f;     // no key: o is 0
        dst[0] = o.x / r, dst[1] = o.y / r, dst[2] = o.z / r, dst[3] = o.w / r;
    }
}

// 8-column tiles of a set: as many as the pairs fill, up to four (16 pairs)
inline int tiles_of_set(int64_t C) { return C <= kTilePairs ? 1 : (C <= 2 * kTilePairs ? 2 : 4); }

}  // namespace

size_t store_attend_workspace_bytes(int S, int T, int Hq, int Hkv, int d) {
    const int64_t C = (int64_t)T * (Hq / Hkv);
    const int pairs = tiles_of_set(C) * kTilePairs;
    const size_t rows = (size_t)S * Hkv * (size_t)((C + pairs - 1) / pairs);
    return ((rows + kMaxCtas) * pairs * (d + 2) * sizeof(float) + 255) & ~size_t(255);
}

namespace {

template <int D, int NT>
cudaError_t launch_tiles(const AttendMap& map, int P0, const void* q, int q_dtype, int T, int Hq, int Hkv, int sets,
                         float* slots, float* out, float* parts, cudaStream_t stream, int* P) {
    using Sh = Shape<D, NT>;
    static_assert(Sh::kSmem * Sh::kCtasPerSm <= kMaxSmem, "the CTAs of an SM fit");
    auto kern = store_attend_kernel<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sh::kSmem);
    if (e != cudaSuccess) return e;
    *P = P0 < 148 * Sh::kCtasPerSm ? P0 : 148 * Sh::kCtasPerSm;
    return launch_ex(kern, dim3(*P), dim3(kThreads), Sh::kSmem, stream, false, 1, map, q, q_dtype, T, Hq, Hkv, sets,
                     slots, out, parts);
}

template <int D>
cudaError_t launch_dim(int nt, const AttendMap& map, int P0, const void* q, int q_dtype, int T, int Hq, int Hkv, int sets,
                       float* slots, float* out, float* parts, cudaStream_t stream, int* P) {
    if (nt == 1) return launch_tiles<D, 1>(map, P0, q, q_dtype, T, Hq, Hkv, sets, slots, out, parts, stream, P);
    if (nt == 2) return launch_tiles<D, 2>(map, P0, q, q_dtype, T, Hq, Hkv, sets, slots, out, parts, stream, P);
    return launch_tiles<D, 4>(map, P0, q, q_dtype, T, Hq, Hkv, sets, slots, out, parts, stream, P);
}

}  // namespace

cudaError_t launch_store_attend(AttendMap& map, int Hkv, int d, const void* q, int q_dtype, int T, int Hq, float* out,
                                float* parts, void* ws, cudaStream_t stream) {
    const int64_t C = (int64_t)T * (Hq / Hkv);
    const int nt = tiles_of_set(C), pairs = nt * kTilePairs;
    const int sets = (int)((C + pairs - 1) / pairs);
    int64_t U = 0;
    bool shared = false;   // some row's keys may be shared by several CTAs, or a row has none
    for (int s = 0; s < map.nsess; ++s) {
        const int64_t last = map.visible[s] + T - 1;   // keys that the last token sees
        const int64_t keys = last < map.n[s] ? (last > 0 ? last : 0) : map.n[s];
        map.unit0[s] = U;
        map.tiles[s] = (int)((keys + kTile - 1) / kTile);
        U += (int64_t)map.tiles[s] * Hkv * sets;
        shared = shared || map.tiles[s] != 1;
    }
    map.unit0[map.nsess] = U;
    float* slots = static_cast<float*>(ws);
    int P = 0;
    if (U > 0) {
        const int P0 = (int)(U < kMaxCtas ? U : kMaxCtas);
        cudaError_t e;
        switch (d) {
            case 32: e = launch_dim<32>(nt, map, P0, q, q_dtype, T, Hq, Hkv, sets, slots, out, parts, stream, &P); break;
            case 64: e = launch_dim<64>(nt, map, P0, q, q_dtype, T, Hq, Hkv, sets, slots, out, parts, stream, &P); break;
            case 128: e = launch_dim<128>(nt, map, P0, q, q_dtype, T, Hq, Hkv, sets, slots, out, parts, stream, &P); break;
            case 256: e = launch_dim<256>(nt, map, P0, q, q_dtype, T, Hq, Hkv, sets, slots, out, parts, stream, &P); break;
            default: return cudaErrorInvalidValue;
        }
        if (e != cudaSuccess || !shared) return e;
    }
    return launch_ex(store_attend_merge_kernel, dim3((unsigned)((int64_t)map.nsess * Hkv * sets * pairs)),
                     dim3(kMergeThreads), 0, stream, U > 0, 1, map, slots, T, Hq, Hkv, sets, pairs, d, P, out, parts);
}

}  // namespace fathom
