// Attention over the 4-bit stores themselves: every key of a K store and the
// values of a V store, both in bit planes.
//
//   s_i = q . K_i / sqrt(d),  K_ic = Delta_c,b(i) (code_ic - 7.5),  V likewise,
//   out = sum_i exp(s_i) V_i / sum_i exp(s_i)
//
// over the keys a query may see, in one pass with a running maximum and sum.
//
// Work split.  The keys of a (session, KV head, set of 4 or 8 (token, head of the
// group) pairs) are a row of tiles of 1024 keys (512 where a call is short).  All
// rows' tiles form one list, cut into equal runs, one per CTA, at most as many as
// are resident; a run may end in the middle of a row, so every (CTA, row) pair
// leaves a partial (o, m, l), and a second launch adds a row's partials in
// order (those of a short row are added in its cluster's shared memory).  CTA p's partial of row r lies in slot p + r: a run that passes into
// the next row raises r, a row that passes into the next CTA raises p, so no
// two meet.
//
// A tile.  Its planes arrive 64 channels at a time, K's then V's, by one tensor copy
// each into a ring of two buffers: 128 bytes of every plane row, a
// whole line (pieces of 64 bytes end at 3 TB/s, of 32 at 1.6).  Eight warps have
// two blocks of 64 keys each, and no step of theirs waits for another warp
// but the copy that reuses a buffer, which they issue in turn.  A warp turns the
// plane words of its blocks into words of 4-bit codes in its own shared memory,
// laid out so that one 16-byte load is a lane's share of a matrix operand, and
// takes them through both products, m16n8k16 on fp16 with fp32 sums:
//   S (64 keys x columns) = codes . Q',  Q'_c = q_c Delta_c of this block,
//   O (d x columns) += Delta_c (codes . P).
// A code needs no conversion: the bits 0..15 of an fp16 are the subnormal
// code 2^-24, exactly, and shifted by 4 bits 16 times that, so one AND makes
// two operand values; the factors are undone in the scaling of S and P.  The
// offset 7.5 is half of one more product, with a constant 15.
// Scores never leave the warp: a transposing move of 8x8 matrices makes the P
// operand of the S accumulators.
//
// Precision.  Q' and P are split into a high and a low fp16 half, which sit in
// neighbouring columns, so that a column pair of the 8 is one query in some 22
// bits.  The matrix unit cuts every addend off at 2^-23 of the largest, always
// toward zero: with codes that are all positive, sums over n keys drift
// from the true one, by 1e-4 of the output at 131072 keys.  So the high halves are
// multiples of a power of two that is large enough for their sums to be exact, as
// the offset is; what is cut off the low halves' sums is 2^-10 smaller.  The running
// maximum is rounded up to a whole number of binary orders: what was summed
// is rescaled exactly.  Against 64 bits: 2e-7 to 1e-6 of the output (fp32 arithmetic: 2e-7
// to 4e-6; 4096 keys 2.4e-7 against 1.8e-7, 131072 4.5e-7 against 1.9e-6).  The
// halves are fixed point: their last place is that of the head's largest |q|
// times the block's largest Delta (2^-24 of it), so where those two do not meet in one
// channel, logits lose bits that fp32 would keep.
//
// What bounds it: the instructions around the products, ALU and issue slots, not the
// memory: 0.27 us per 64-key block and SM where the copies alone take 0.20; and
// 13 us of launches, first copies and merge.  1048576 keys (8 heads of 128, 4 queries
// each): 264 us, 4.3 TB/s; 131072: 46 us; 4096 keys of 1 head: 8.0 us.
#include <cuda.h>

#include <atomic>

#include "barrier.cuh"
#include "fathom_internal.cuh"

namespace fathom {
namespace {

constexpr int kTilePairs = 4;                   // queries per 8 columns
constexpr int kMaxCtas = 296;                   // two CTAs per SM

constexpr int kMaxCluster = 8;                  // CTAs
constexpr int kWarps = 8;                       // of a CTA
constexpr int kThreads = 32 * kWarps;

// NB: blocks of a warp
template <int D, int NT, bool F32, int NB>
struct Shape {
    static constexpr int kTileBlocks = kWarps * NB, kTile = kTileBlocks * kBlock;
    static constexpr int kRow = kTileBlocks * 2;            // words of a plane row of the tile: 128 bytes, or 64
    static constexpr int kCtas = (NT * NB <= 2 && D <= 128) ? 2 : 1;   // per SM
    static constexpr int kPairs = kTilePairs * NT;          // (token, head of the group) pairs of a set
    static constexpr int KS = D / 16;                       // 16-channel steps
    // a chunk: the tile's planes of CH channels of one operand; channels l and
    // l + HP of it are a pair
    static constexpr int CH = 32, CK = CH / 16, NC = D / CH, HP = CH / 2;
    // a copy: one chunk or two
    static constexpr int PER = D < 64 ? 1 : 2, CC = PER * CH, NCC = D / CC;
    static constexpr int kRaw = CC * 4 * kRow;              // words of a copy's planes
    static constexpr int kRawScales = D * kTileBlocks;      // halves of a tile's scales, of K or V
    static constexpr int kRing = 4 / PER;
    static constexpr int kCodes = NB * CH * 8;              // words of a warp's codes of a chunk
    static constexpr int kOwn = kCodes > kPairs * D ? kCodes : kPairs * D;   // or of its partial outputs
    static constexpr int kScales = 2 * NB * D;              // halves: K, V; block; channels, pair by pair
    static constexpr int kQWords = NT * KS * 32 * 4;        // a lane's share of the queries
    static constexpr int kQ2Words = F32 ? kQWords / 2 : 0;
    static constexpr size_t kBytes = 4 * (size_t)(kRing * kRaw + kWarps * kOwn) + 2 * (size_t)(kWarps * kScales + 2 * kRawScales) +
                                     4 * (size_t)(kQWords + kQ2Words) + 4 * (size_t)(2 * kWarps * kPairs + kPairs) +
                                     8 * 2 * (kRing + 1);
    static constexpr size_t kSmem = kBytes + 1024;          // the planes start on a 1024-byte boundary
    static_assert(NB == 1 || NB == 2, "");
};

// where channel c of D lies when channels are listed pair by pair
template <int CH>
__device__ __forceinline__ int paired(int c) {
    const int l = c % CH;
    return c - l + 2 * (l % (CH / 2)) + l / (CH / 2);
}

// What the kernels know of the sessions of a launch, up to S of them: the part that
// every warp reads first, then the tensor maps of planes and scales.  One session
// has a type of its own: a launch copies its parameters, and reads them cold.
struct Span {
    int n, visible;     // query token t sees the keys below min(n, visible + t)
    int unit0, tiles;   // its first unit; tiles of a row
};
template <int S>
struct Spans {
    int nsess;
    int each, more;     // units of a CTA, and CTAs with one more
    int cluster;        // above 1: a row's tiles, one to a CTA of a cluster of this many
    Span span[S];
};
template <int S>
struct Sessions {
    Spans<S> at;
    alignas(64) CUtensorMap k[S], ks[S], v[S], vs[S];
};

// units are cut into runs: the first `more` of each + 1, the others of each
template <class M>
__device__ __forceinline__ int run_start(const M& m, int p) { return p * m.each + (p < m.more ? p : m.more); }
template <class M>
__device__ __forceinline__ int run_of(const M& m, int u) {
    const int big = m.more * (m.each + 1);
    return u < big ? u / (m.each + 1) : m.more + (u - big) / m.each;
}

__device__ __forceinline__ void mma(float* c, const uint32_t* a, const uint32_t* b) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// with the operand B's bits in floats
__device__ __forceinline__ void mma_p(float* c, const uint32_t* a, const float* b) {
    const uint32_t bits[2] = {__float_as_uint(b[0]), __float_as_uint(b[1])};
    mma(c, a, bits);
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
__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
// (low, high) as two fp16
__device__ __forceinline__ uint32_t half2_of(float low, float high) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(high), "f"(low));
    return r;
}
// Two values v = q Delta below 2^14, q = q1 + q2, as a column's operand.  Even column:
// the high half h, v to a multiple of 1/2 or more (the sum with 1536 of an fp16 below
// 2^14 has no finer bits).  Odd column: q1 Delta - h, rounded once, + q2 Delta, of at
// most 2^-11 of v or 1/2.  Sums of the high halves' products with codes are multiples
// of 1/2, too, and exact up to 2^23 of them.
__device__ __forceinline__ uint32_t half_of_product(uint32_t q1, uint32_t own, uint32_t q2, uint32_t delta, __half2 sign, bool f32) {
    const __half2 d = as_half2(delta), big = __float2half2_rn(1536.0f);
    const __half2 h = __hadd2_rn(__hfma2(as_half2(q1), d, big), __hneg2(big));
    __half2 z = __hfma2(as_half2(own), d, __hmul2_rn(h, sign));
    if (f32) z = __hfma2(as_half2(q2), d, z);
    return *reinterpret_cast<const uint32_t*>(&z);
}

// x where mask has a bit, else y; one instruction, where the expression takes two
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t y, uint32_t mask) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(x), "r"(y), "r"(mask));
    return r;
}

// The ring of raw planes: a buffer's bytes arrive by one asynchronous tensor copy.
__device__ __forceinline__ void copy_planes(void* dst, const CUtensorMap* tm, int word, int channel, uint64_t* b) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(tm), "r"(word), "r"(channel), "r"(0), "r"(smem_addr(b))
        : "memory");
}
__device__ __forceinline__ void copy_scales(void* dst, const CUtensorMap* tm, int block, int channel, uint64_t* b) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(tm), "r"(block), "r"(channel), "r"(smem_addr(b))
        : "memory");
}
// a float of the same place in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ float peer_float(const float* p, uint32_t rank) {
    uint32_t at;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// plane words W[j] of 32 keys -> N[r]: nibble m = code of key 4 m + r
__device__ __forceinline__ void planes_to_nibbles(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t* N) {
    const uint32_t E = pick(w0 << 1, w1, 0xAAAAAAAAu), O = pick(w0, w1 >> 1, 0xAAAAAAAAu);
    const uint32_t F = pick(w2 << 1, w3, 0xAAAAAAAAu), H = pick(w2, w3 >> 1, 0xAAAAAAAAu);
    N[0] = pick(E << 2, F, 0xCCCCCCCCu);
    N[2] = pick(E, F >> 2, 0xCCCCCCCCu);
    N[1] = pick(O << 2, H, 0xCCCCCCCCu);
    N[3] = pick(O, H >> 2, 0xCCCCCCCCu);
}

// operand value pairs p = 0..3 of a word of codes (odd p: 16 times the code).  The
// last two are bytes 1 and 3 as they are less their upper nibbles: an exact
// subtraction of subnormals, on another pipe than the ANDs
__device__ __forceinline__ void operands(const uint4& raw, uint32_t a[4][4]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a[0][e] = w[e] & 0x000F000Fu;
        a[1][e] = w[e] & 0x00F000F0u;
        const uint32_t y = __byte_perm(w[e], 0u, 0x4341);
        a[3][e] = y & 0x00F000F0u;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(a[2][e]) : "r"(y), "r"(a[3][e]));
    }
}

// Where the keys of a block lie in the operands: key 32 w + 4 (p + 4 k4) + r is
// nibble p of half k4 of N[r] of word w.
//   S: row g = 2 r + k4 (w = 0) or that plus 8 (w = 1) of m-tile p; a lane's
//      columns k are the channel pairs 8 ks + 2 t and the one behind it.
//   O: row g is the first channel of pair 8 mt + g, row g + 8 the second; k-step
//      p, column pair t is r = t, k4 = 0 and 1, w = 0 then w = 1.
// Both orders meet: the transposed S accumulators of rows g = 2 t, 2 t + 1 are
// the P operand's k columns 2 t, 2 t + 1.

// A row of tiles: one KV head of one session, for one set of queries.
struct Row {
    int s, g, set, row;
    int u0, u1;   // its units
};
template <int S>
__device__ __noinline__ Row row_of(const Spans<S>& m, int u, int Hkv, int sets) {
    int lo = 0, hi = m.nsess;   // the last session that starts at or before u: empty ones start where the next does
    while (S > 1 && hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (m.span[mid].unit0 <= u) lo = mid;
        else hi = mid;
    }
    const Span& sp = m.span[lo];
    Row r;
    r.s = lo;
    const int rl = (u - sp.unit0) / sp.tiles;
    r.g = rl / sets;
    r.set = rl - r.g * sets;
    r.row = lo * Hkv * sets + rl;
    r.u0 = sp.unit0 + rl * sp.tiles;
    r.u1 = r.u0 + sp.tiles;
    return r;
}

template <int D, int NT, bool F32, int NS, int NB>
__global__ void __launch_bounds__(kThreads, (Shape<D, NT, F32, NB>::kCtas))
store_attend_kernel(const __grid_constant__ Sessions<NS> map, const void* __restrict__ q, int q_dtype, int T, int Hq,
                    int Hkv, int sets, float* __restrict__ slots, float* __restrict__ out, float* __restrict__ parts,
                    unsigned int* status) {
    using Sh = Shape<D, NT, F32, NB>;
    constexpr int kTile = Sh::kTile;
    constexpr int KS = Sh::KS, CH = Sh::CH, CK = Sh::CK, NC = Sh::NC, HP = Sh::HP, PER = Sh::PER, CC = Sh::CC, NCC = Sh::NCC, kPairs = Sh::kPairs, kRing = Sh::kRing;
    extern __shared__ uint32_t smem_raw[];
    uint32_t* s_raw = smem_raw + ((0u - smem_addr(smem_raw)) & 1023u) / 4;   // the next 1024-byte boundary
    // [ring][plane][channel][row of the tile], 16-byte pieces swizzled by the channel
    uint32_t* s_codes = s_raw + kRing * Sh::kRaw;       // [warp][block][ks][lane][4] code words
    // [K, V][D][blocks of the tile] scales, the 16-byte pieces of 32 swizzled by the channel's bit 2
    uint16_t* s_rs = reinterpret_cast<uint16_t*>(s_codes + kWarps * Sh::kOwn);
    uint16_t* s_sc = s_rs + 2 * Sh::kRawScales;         // [warp][K, V][block][D] scales, K's times the block's factor
    uint32_t* s_q = reinterpret_cast<uint32_t*>(s_sc + kWarps * Sh::kScales);      // [NT][ks][lane][4]
    uint32_t* s_q2 = s_q + Sh::kQWords;                 // [NT][ks][lane][2], f32 queries only
    float* s_m = reinterpret_cast<float*>(s_q2 + Sh::kQ2Words);   // [warp][pair]
    float* s_l = s_m + kWarps * kPairs;
    float* s_f = s_l + kWarps * kPairs;                 // [pair] the query's part of the logits' factor
    uint64_t* s_full = reinterpret_cast<uint64_t*>(s_f + kPairs);   // [ring] the copy has arrived; then the scales
    uint64_t* s_read = s_full + kRing + 1;              // every warp has read it

    const int ub = run_start(map.at, blockIdx.x);
    const int units = run_start(map.at, blockIdx.x + 1) - ub, copies = units * (2 * NCC);
    const int G = Hq / Hkv, C = T * G;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int lg = lane >> 2, lt = lane & 3;            // g and t of the operand layouts

    // issues copy c of a unit (NCC of K, then NCC of V) of row r to ring buffer i
    auto copy = [&](const Row& r, int unit, int c, int i) {
        barrier_expect(s_full + i, 4 * Sh::kRaw);
        copy_planes(s_raw + i * Sh::kRaw, c < NCC ? &map.k[r.s] : &map.v[r.s], (unit - r.u0) * (kTile / 32),
                    r.g * D + (c < NCC ? c : c - NCC) * CC, s_full + i);
    };
    auto copy_scale = [&](const Row& r, int unit) {
        const int b = (unit - r.u0) * (kTile / kBlock);
        barrier_expect(s_full + kRing, 2 * 2 * Sh::kRawScales);
        copy_scales(s_rs, &map.ks[r.s], b, r.g * D, s_full + kRing);
        copy_scales(s_rs + Sh::kRawScales, &map.vs[r.s], b, r.g * D, s_full + kRing);
    };
    Row rw = row_of(map.at, ub, Hkv, sets);
    // the merge, or the next call's kernel, may be scheduled as this grid's CTAs leave (they are all resident from
    // the start, clusters too)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (wp == kWarps - 1) {                             // the first queries go to other warps
        if (lane <= kRing) {
            barrier_init(s_full + lane, 1);
            barrier_init(s_read + lane, kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
        pdl_wait();
        if (lane == kRing) {
            copy_scale(rw, ub);
        } else if (lane < kRing && lane < copies) {
            const int unit = ub + lane / (2 * NCC);
            copy(unit < rw.u1 ? rw : row_of(map.at, unit, Hkv, sets), unit, lane % (2 * NCC), lane);
        }
    }

    pdl_wait();
    bool stuck = false;
    uint32_t* codes = s_codes + wp * Sh::kOwn;
    uint16_t *k_scales = s_sc + wp * Sh::kScales, *v_scales = k_scales + NB * D;
    const __half2 sign = __float2half2_rn((lg & 1) ? -1.0f : 1.0f);   // of Q's high half in this lane's column
    int u = 0, j = 0;
    while (u < units) {
        const int s = rw.s;
        const int left = rw.u1 - ub, re = left < units ? left : units;
        const bool whole = ub + u == rw.u0 && left <= units;   // no other CTA has a share of this row
        const int n = map.at.span[s].n, visible = map.at.span[s].visible;

        // the set's queries in fp16, each scaled by a power of two to at most 2^6 to 2^7
        // in magnitude (so that the least fp16 is 2^-31 of it): q1 = the value's first
        // 11 bits, for f32 queries q2 = the next 11
        for (int x = wp; x < kPairs; x += kWarps) {
            const int pr = rw.set * kPairs + x;
            float v[D / 32];
            float mx = 0.0f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                v[e] = pr < C ? load_q(q, q_dtype, (((int64_t)s * T + pr / G) * Hq + rw.g * G + pr % G) * D + 32 * e + lane) : 0.0f;
                mx = fmaxf(mx, fabsf(v[e]));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // 2^-120 and below count as 0
            const int ex = max((int)(__float_as_uint(mx) >> 23) - 133, -126);
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const int c = paired<CH>(32 * e + lane);
                const float vn = v[e] * down;
                const __half q1 = __float2half_rn(vn), none = __float2half_rn(0.0f);
                // columns 2x and 2x + 1 of the 8: q1 of both, then what the column's operand is made of, none and q1
                const int base = ((x >> 2) * KS + (c >> 4)) * 32 + (x & 3) * 8 + ((c >> 2) & 3);   // lane of column 2x
                __half* h0 = reinterpret_cast<__half*>(s_q + base * 4) + (c & 3);
                __half* h1 = h0 + 4 * 8;
                h0[0] = h1[0] = h1[4] = q1;
                h0[4] = none;
                if (F32) {
                    __half* g0 = reinterpret_cast<__half*>(s_q2 + base * 2) + (c & 3);
                    g0[0] = none;
                    g0[4 * 4] = __float2half_rn(vn - __half2float(q1));
                }
            }
            // logits in log2 units = sums of products * this * 2^24 / the block's factor;
            // never 0, which a masked score of -inf would turn into NaN
            if (lane == 0) s_f[x] = fmaxf(1.4426950408889634f / sqrtf((float)D) * __uint_as_float((uint32_t)(127 + ex) << 23), 1.17549435e-38f);
        }

        float O[NT][KS][2], m[NT], l[NT];
        int limit[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt] = -INFINITY;
            l[nt] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) O[nt][mt][0] = O[nt][mt][1] = 0.0f;
            limit[nt] = min(max(visible + (rw.set * kPairs + nt * kTilePairs + lt) / G, 0), n);
        }
        // the set's first pair sees the fewest keys, its last the most
        const int least = min(max(visible + rw.set * kPairs / G, 0), n);
        const int most = min(max(visible + (rw.set * kPairs + kPairs - 1) / G, 0), n);
        __syncthreads();                                // the queries are in place

        for (; u < re; ++u) {
            const int k0 = (ub + u - rw.u0) * kTile + NB * wp * kBlock;   // the warp's first block
            const bool act = k0 < most;
            // ---- the blocks' scales: 0 behind the last block that is seen, where memory may hold anything
            float back[NB];
            __syncwarp();
            {
                const uint32_t keep = act ? (NB == 2 && k0 + kBlock < most ? 0xFFFFFFFFu : 0xFFFFu) : 0u;
                __half2 mh = __float2half2_rn(0.0f);
                barrier_wait(s_full + kRing, u & 1, stuck);
                uint32_t sw[2 * D / 32];                // of the warp's blocks: K's channels, then V's
#pragma unroll
                for (int i = 0; i < 2 * D / 32; ++i) {
                    const int word = (NB * wp / 2) ^ (NB == 2 ? lane & 4 : 0);
                    sw[i] = reinterpret_cast<const uint32_t*>(s_rs)[(32 * i + lane) * (Sh::kTileBlocks / 2) + word];
                    if (NB == 1 && (wp & 1)) sw[i] >>= 16;
                }
                barrier_arrive(s_read + kRing);
#pragma unroll
                for (int i = 0; i < 2 * D / 32; ++i) {
                    sw[i] &= keep;
                    if (i < D / 32) mh = __hmax2(mh, as_half2(sw[i]));
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&mh), o);
                    mh = __hmax2(mh, as_half2(other));
                }
                // a power of two sc brings the block's largest scale to [2^6, 2^7), so that |q Delta| < 2^14
                // (an f16 is 0 or at least 2^-24)
                float sc[2] = {1.0f, 1.0f};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float dm = b ? __high2float(mh) : __low2float(mh);
                    const int ex = max((int)(__float_as_uint(dm) >> 23), 103);
                    sc[b] = __uint_as_float((uint32_t)(260 - ex) << 23);
                    back[b] = __uint_as_float((uint32_t)(ex + 18) << 23);   // 2^24 / sc
                }
#pragma unroll
                for (int i = 0; i < 2 * D / 32; ++i) {
                    __half2 v = as_half2(sw[i]);
                    if (i < D / 32) v = __floats2half2_rn(__low2float(v) * sc[0], __high2float(v) * sc[1]);
                    __half* dst = reinterpret_cast<__half*>(i < D / 32 ? k_scales : v_scales) + paired<CH>(32 * (i % (D / 32)) + lane);
                    dst[0] = __low2half(v);
                    if (NB == 2) dst[D] = __high2half(v);
                }
            }
            // scores of 16-key tiles p; then, in [p][0] and [p][1], the bits of their weights as operands
            float S[NB][NT][4][4], B15[NB][NT][4], neg[NB][NT][2];
            // the lane's channel pair, and its block (of two) or word (of one block)
            const int pl = NB == 2 ? (lane & 7) + 8 * (lane >> 4) : lane >> 1, part = NB == 2 ? (lane >> 3) & 1 : lane & 1;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    neg[b][nt][0] = neg[b][nt][1] = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        B15[b][nt][e] = 0.0f;
#pragma unroll
                        for (int p = 0; p < 4; ++p) S[b][nt][p][e] = 0.0f;
                    }
                }
            // chunk c of the tile, of K or of V: its planes of the warp's blocks to registers, as codes to the
            // warp's own memory
            auto stage = [&](bool isk, int chunk) {
                const int c = chunk / PER, part_of = chunk % PER;   // its copy, and where in it
                const int rj = (2 * NCC) % kRing == 0 ? c % kRing : j % kRing;
                const uint32_t turn = (uint32_t)((2 * NCC) % (2 * kRing) == 0 ? c / kRing : j / kRing) & 1;
                if (part_of == 0) barrier_wait(s_full + rj, turn, stuck);
                // pieces of 16 bytes: a warp's two blocks of 128 keys, or the two warps' of 64 that share one
                const uint32_t* src = s_raw + rj * Sh::kRaw + (part_of * CH + pl) * Sh::kRow;
                const int piece = NB == 2 ? wp : wp / 2, swizzle = NB == 2 ? pl & 7 : (pl >> 1) & 3;
                src += (piece ^ swizzle) * 4 + (NB == 2 ? 2 * part : 2 * (wp & 1) + part);
                // both code layouts keep the lanes of a write, and of a read, on different banks
                if (NB == 2) {
                    uint2 P[2][4];                      // [channel of the pair][plane]
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int k = 0; k < 4; ++k) P[e][k] = *reinterpret_cast<const uint2*>(src + (k * CC + e * HP) * Sh::kRow);
                    if (part_of == PER - 1) barrier_arrive(s_read + rj);
                    uint32_t N[2][2][4];                // [channel][word][r]
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        planes_to_nibbles(P[e][0].x, P[e][1].x, P[e][2].x, P[e][3].x, N[e][0]);
                        planes_to_nibbles(P[e][0].y, P[e][1].y, P[e][2].y, P[e][3].y, N[e][1]);
                    }
                    uint32_t* dst = codes + part * (Sh::kCodes / 2) + (pl >> 3) * 128;
                    if (isk) {
                        // row g of the second block lies where row g ^ 1 would
                        uint2* d2 = reinterpret_cast<uint2*>(dst) + (pl & 7);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int k4 = 0; k4 < 2; ++k4) {
                                const uint32_t sel = k4 ? 0x7632u : 0x5410u;
                                d2[(2 * r + (k4 ^ part)) * 8] = make_uint2(__byte_perm(N[0][0][r], N[1][0][r], sel),
                                                                           __byte_perm(N[0][1][r], N[1][1][r], sel));
                            }
                    } else {
                        // column pair t of row g lies where t ^ (g / 2) would
                        uint4* d4 = reinterpret_cast<uint4*>(dst) + (pl & 7) * 4;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            d4[r ^ ((pl >> 1) & 3)] = make_uint4(N[0][0][r], N[1][0][r], N[0][1][r], N[1][1][r]);
                    }
                } else {
                    uint32_t P[2][4], N[2][4];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int k = 0; k < 4; ++k) P[e][k] = src[(k * CC + e * HP) * Sh::kRow];
                    if (part_of == PER - 1) barrier_arrive(s_read + rj);
#pragma unroll
                    for (int e = 0; e < 2; ++e) planes_to_nibbles(P[e][0], P[e][1], P[e][2], P[e][3], N[e]);
                    uint32_t* dst = codes + (pl >> 3) * 128;
                    if (isk) {
                        // row g of an odd 16-channel step lies where row g ^ 1 would
                        dst += (pl & 7) * 2 + part;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int k4 = 0; k4 < 2; ++k4)
                                dst[(2 * r + (k4 ^ (pl >> 3))) * 16] = __byte_perm(N[0][r], N[1][r], k4 ? 0x7632u : 0x5410u);
                    } else {
                        uint2* d2 = reinterpret_cast<uint2*>(dst) + (pl & 7) * 8 + part;
#pragma unroll
                        for (int r = 0; r < 4; ++r) d2[(r ^ ((pl >> 1) & 3)) * 2] = make_uint2(N[0][r], N[1][r]);
                    }
                }
                // warps take turns at the buffer's next copy, once every warp has read this one
                if (part_of == PER - 1 && wp == j % kWarps && j + kRing < copies) {
                    barrier_wait(s_read + rj, turn, stuck);
                    const int cn = c + kRing, un = u + cn / (2 * NCC);
                    if (lane == 0 && !stuck) {
                        if (un < re) copy(rw, ub + un, cn % (2 * NCC), rj);
                        else copy(row_of(map.at, ub + un, Hkv, sets), ub + un, cn % (2 * NCC), rj);
                    }
                }
                if (part_of == PER - 1) ++j;
                __syncwarp();
            };
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
                stage(true, c);
                if (act) {
                    // ---- S += codes . Q' of this chunk's channels
                    const uint32_t a15[4] = {0x000F000Fu, 0x000F000Fu, 0x000F000Fu, 0x000F000Fu};
                    const uint4* kc = reinterpret_cast<const uint4*>(codes);
#pragma unroll
                    for (int k = 0; k < CK; ++k) {
                        const int ks = c * CK + k;
                        uint32_t bq[NB][NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 q4 = *reinterpret_cast<const uint4*>(s_q + ((nt * KS + ks) * 32 + lane) * 4);
                            uint2 q2 = make_uint2(0u, 0u);
                            if (F32) q2 = *reinterpret_cast<const uint2*>(s_q2 + ((nt * KS + ks) * 32 + lane) * 2);
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                const uint2 d4 = *reinterpret_cast<const uint2*>(k_scales + b * D + 16 * ks + 4 * lt);
                                bq[b][nt][0] = half_of_product(q4.x, q4.z, q2.x, d4.x, sign, F32);
                                bq[b][nt][1] = half_of_product(q4.y, q4.w, q2.y, d4.y, sign, F32);
                                mma(B15[b][nt], a15, bq[b][nt]);
                            }
                        }
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            uint32_t a[4][4];
                            operands(kc[b * (Sh::kCodes / (4 * NB)) + k * 32 + (lane ^ (NB == 2 ? b * 4 : (k & 1) * 4))], a);
#pragma unroll
                            for (int p = 0; p < 4; ++p)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma(S[b][nt][p], a[p], bq[b][nt]);
                        }
                    }
                    __syncwarp();
                }
            }
            if (act) {
                // ---- weights: lane (g, t) holds query t of the tile, 8 keys of each block
                const bool cut = k0 + NB * kBlock > least;   // some query of the set does not see all keys
                float shift[NT];
                bool moved = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float f = s_f[nt * kTilePairs + lt];
                    float F[NB], top[NB];
                    float mn = m[nt];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const float un = (p & 1) ? 0.0625f : 1.0f;
                            float* v = S[b][nt][p];
                            // the high halves' sums, and their offset, are exact
                            v[0] = fmaf(v[0], un, -0.5f * B15[b][nt][0]) + fmaf(v[1], un, -0.5f * B15[b][nt][1]);
                            v[2] = fmaf(v[2], un, -0.5f * B15[b][nt][0]) + fmaf(v[3], un, -0.5f * B15[b][nt][1]);
                            if (cut) {
                                const int key = k0 + b * kBlock + 4 * (p + 4 * (lg & 1)) + (lg >> 1);
                                if (key >= limit[nt]) v[0] = -INFINITY;
                                if (key + 32 >= limit[nt]) v[2] = -INFINITY;
                            }
                            mx = fmaxf(mx, fmaxf(v[0], v[2]));
                        }
                        F[b] = f * back[b];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        top[b] = mx * F[b];
                        // a whole number: what was summed so far is rescaled by powers of two, exactly
                        mn = fmaxf(mn, ceilf(top[b]));
                    }
                    const float base = mn == -INFINITY ? 0.0f : mn;
                    // S F - base is rounded once; where the product's own rounding exceeds
                    // the exponents that matter, both are rounded alike instead
                    if (fabsf(base) > 1048576.0f) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                S[b][nt][p][0] *= F[b];
                                S[b][nt][p][2] *= F[b];
                            }
                            F[b] = 1.0f;
                        }
                    }
                    shift[nt] = ex2(m[nt] - base);      // 0 while nothing has been seen
                    moved |= mn != m[nt];
                    m[nt] = mn;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        // the high halves of a block's weights are multiples of 2^-11 of (the power of two above)
                        // the largest: P + round is rounded to one
                        const float round = __uint_as_float(__float_as_uint(ex2(top[b] - base)) & 0x7F800000u) * 0x1.8p28f;
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            // weights times 2^15, or 2^11 where the codes come 16 times as large
                            const float up = (p & 1) ? 2048.0f : 32768.0f, r = (p & 1) ? round * 0.0625f : round;
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                const float v = ex2(fmaf(S[b][nt][p][2 * w], F[b], -base)) * up;
                                const float h = __fadd_rn(__fadd_rn(v, r), -r);
                                S[b][nt][p][w] = __uint_as_float(transpose8x8(half2_of(h, v - h)));
                            }
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
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float c4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const uint32_t v15 = (p & 1) ? 0x00F000F0u : 0x000F000Fu, a[4] = {v15, v15, v15, v15};
                            mma_p(c4, a, S[b][nt][p]);
                        }
                        neg[b][nt][0] = -0.5f * c4[0];
                        neg[b][nt][1] = -0.5f * c4[1];
                        l[nt] = fmaf(c4[0] + c4[1], 512.0f / 15.0f, l[nt]);   // 2^24 / 2^15
                    }
            }
            // a warp has its turn at the copy of the next tile's scales
            if (wp == u % kWarps && u + 1 < units) {
                barrier_wait(s_read + kRing, u & 1, stuck);
                if (lane == 0 && !stuck) copy_scale(u + 1 < re ? rw : row_of(map.at, ub + u + 1, Hkv, sets), ub + u + 1);
            }
#pragma unroll
            for (int cv = 0; cv < NC; ++cv) {
                stage(false, NC + cv);
                if (act) {
                    // ---- O += Delta (codes - 7.5) . P
                    const uint4* vc = reinterpret_cast<const uint4*>(codes) + (lane ^ ((lane >> 3) & 3));
#pragma unroll
                    for (int k = 0; k < CK; ++k) {
                        const int mt = cv * CK + k;
                        float acc[NB][NT][4];
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            uint32_t a[4][4];
                            operands(vc[b * (Sh::kCodes / (4 * NB)) + k * 32], a);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) acc[b][nt][0] = acc[b][nt][2] = neg[b][nt][0], acc[b][nt][1] = acc[b][nt][3] = neg[b][nt][1];
#pragma unroll
                            for (int p = 0; p < 4; ++p)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_p(acc[b][nt], a[p], S[b][nt][p]);
                        }
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const float2 dv = __half22float2(*reinterpret_cast<const __half2*>(v_scales + b * D + 16 * mt + 2 * lg));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                O[nt][mt][0] = fmaf(acc[b][nt][0] + acc[b][nt][1], dv.x, O[nt][mt][0]);
                                O[nt][mt][1] = fmaf(acc[b][nt][2] + acc[b][nt][3], dv.y, O[nt][mt][1]);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }

        // ---- the warps' partials: merged here, o in units of 2^-9; a warp's codes make room
        __syncwarp();
        float* s_o = reinterpret_cast<float*>(codes);   // [pair][D], channels pair by pair
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int x = nt * kTilePairs + lt;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt)
                *reinterpret_cast<float2*>(s_o + x * D + 16 * mt + 2 * lg) = make_float2(O[nt][mt][0], O[nt][mt][1]);
            if (lg == 0) {
                s_m[wp * kPairs + x] = m[nt];
                s_l[wp * kPairs + x] = l[nt];
            }
        }
        __syncthreads();
        float* part = slots + (int64_t)(blockIdx.x + rw.row) * (kPairs * (D + 2));
        // a cluster's partials stay in shared memory, where the planes were
        const bool together = NS == 1 && NB == 1 && map.at.cluster > 1;
        if (together) part = reinterpret_cast<float*>(s_raw);
        auto result = [&](int x, int c, float o, float M, float L) {
            const int pr = rw.set * kPairs + x;
            if (pr >= C) return;
            const int64_t h = ((int64_t)s * T + pr / G) * Hq + rw.g * G + pr % G;
            if (parts) {
                parts[h * (D + 2) + c] = o;
                if (c == 0) parts[h * (D + 2) + D] = M, parts[h * (D + 2) + D + 1] = L;
            } else {
                out[h * D + c] = o / (L > 0.0f ? L : 1.0f);   // no key: o is 0; a query with a NaN: o is one
            }
        };
        for (int e = threadIdx.x; e < kPairs * D; e += kThreads) {
            const int x = e / D, c = e % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w * kPairs + x]);
            const float Mb = M == -INFINITY ? 0.0f : M;
            float L = 0.0f, o = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(s_m[w * kPairs + x] - Mb);
                L = fmaf(s_l[w * kPairs + x], f, L);
                o = fmaf(reinterpret_cast<const float*>(s_codes + w * Sh::kOwn)[x * D + paired<CH>(c)], f, o);
            }
            o *= 512.0f;
            if (!whole) {
                part[e] = o;
                if (c == 0) part[kPairs * D + x] = M, part[kPairs * (D + 1) + x] = L;
            } else {
                result(x, c, o, M, L);
            }
        }
        if (together) {
            cluster_sync();
            const int cl = map.at.cluster;
            for (int e = (blockIdx.x % cl) * kThreads + threadIdx.x; e < kPairs * D; e += cl * kThreads) {
                const int x = e / D;
                float mp[kMaxCluster], lp[kMaxCluster], op[kMaxCluster], M = -INFINITY;
#pragma unroll
                for (int i = 0; i < kMaxCluster; ++i) {
                    const bool in = i < cl;
                    op[i] = in ? peer_float(part + e, i) : 0.0f;
                    mp[i] = in ? peer_float(part + kPairs * D + x, i) : -INFINITY;
                    lp[i] = in ? peer_float(part + kPairs * (D + 1) + x, i) : 0.0f;
                    M = fmaxf(M, mp[i]);
                }
                const float Mb = M == -INFINITY ? 0.0f : M;
                float L = 0.0f, o = 0.0f;
#pragma unroll
                for (int i = 0; i < kMaxCluster; ++i) {
                    const float f = ex2(mp[i] - Mb);
                    L = fmaf(lp[i], f, L);
                    o = fmaf(op[i], f, o);
                }
                result(x, e % D, o, M, L);
            }
            cluster_sync();                             // until the others have read this CTA's
        }
        __syncthreads();                                // before the next row's queries and codes
        if (u < units) rw = row_of(map.at, ub + u, Hkv, sets);
    }
    barrier_report(stuck, status);
}

// One CTA per (row, pair) whose keys were shared by several CTAs, or that has
// none: the row's partials, in an order that depends on their number alone.
constexpr int kMergeThreads = 256;
__global__ void __launch_bounds__(kMergeThreads)
store_attend_merge_kernel(const __grid_constant__ Spans<kAttendSets> map, const float* __restrict__ slots, int T, int Hq, int Hkv,
                          int sets, int pairs, int D, float* __restrict__ out, float* __restrict__ parts) {
    __shared__ float s_w[kMaxCtas];
    __shared__ float s_red[2][kMergeThreads / 32];
    __shared__ float4 s_o[kMergeThreads];
    constexpr int kFirst = 8;   // partials that a thread loads before it knows their weights
    const int G = Hq / Hkv, C = T * G;
    const int row = blockIdx.x / pairs, x = blockIdx.x % pairs;
    const int s = row / (Hkv * sets), rl = row % (Hkv * sets);
    const int g = rl / sets, pr = rl % sets * pairs + x;
    // (every CTA waits for the kernel before it, so that this one is not over sooner)
    if (pr >= C) {
        pdl_wait();
        return;
    }
    const int ub = map.span[s].unit0 + rl * map.span[s].tiles, ue = ub + map.span[s].tiles;
    int p0 = 0, np = 0;
    if (ue > ub) {
        p0 = run_of(map, ub);
        np = run_of(map, ue - 1) - p0 + 1;
        if (np == 1) {                           // written by its CTA
            pdl_wait();
            return;
        }
    }
    const int64_t st = (int64_t)pairs * (D + 2);
    const float* base = slots + (int64_t)(p0 + row) * st;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    // D/4 threads take a partial's channels, the others further partials
    const int cl = D / 4, c4 = threadIdx.x % cl, grp = threadIdx.x / cl, ng = kMergeThreads / cl;
    const float* mine = base + x * D + 4 * c4;
    pdl_wait();
    float4 v[kFirst];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
        const int p = grp + i * ng;
        v[i] = p < np ? *reinterpret_cast<const float4*>(mine + p * st) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    float M = -INFINITY, mp[(kMaxCtas + kMergeThreads - 1) / kMergeThreads], lp[(kMaxCtas + kMergeThreads - 1) / kMergeThreads];
#pragma unroll
    for (int i = 0; i < (kMaxCtas + kMergeThreads - 1) / kMergeThreads; ++i) {
        const int p = threadIdx.x + i * kMergeThreads;
        mp[i] = p < np ? base[p * st + pairs * D + x] : -INFINITY;
        lp[i] = p < np ? base[p * st + pairs * (D + 1) + x] : 0.0f;
        M = fmaxf(M, mp[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) s_red[0][wp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) M = fmaxf(M, s_red[0][w]);
    const float Mb = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
#pragma unroll
    for (int i = 0; i < (kMaxCtas + kMergeThreads - 1) / kMergeThreads; ++i) {
        const int p = threadIdx.x + i * kMergeThreads;
        if (p < np) {
            const float f = ex2(mp[i] - Mb);
            s_w[p] = f;
            L = fmaf(lp[i], f, L);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) s_red[1][wp] = L;
    __syncthreads();
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) L += s_red[1][w];
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto take = [&](const float4& e, float f) {
        o.x = fmaf(e.x, f, o.x);
        o.y = fmaf(e.y, f, o.y);
        o.z = fmaf(e.z, f, o.z);
        o.w = fmaf(e.w, f, o.w);
    };
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
        if (grp + i * ng < np) take(v[i], s_w[grp + i * ng]);
    for (int p = grp + kFirst * ng; p < np; p += ng) take(*reinterpret_cast<const float4*>(mine + p * st), s_w[p]);
    s_o[threadIdx.x] = o;
    __syncthreads();
    if (grp) return;
    for (int e = 1; e < ng; ++e) {
        const float4 w = s_o[e * cl + c4];
        o.x += w.x, o.y += w.y, o.z += w.z, o.w += w.w;
    }
    const int64_t h = ((int64_t)s * T + pr / G) * Hq + g * G + pr % G;
    if (parts) {
        float* dst = parts + h * (D + 2) + 4 * c4;
        dst[0] = o.x, dst[1] = o.y, dst[2] = o.z, dst[3] = o.w;
        if (c4 == 0) parts[h * (D + 2) + D] = M, parts[h * (D + 2) + D + 1] = L;
    } else {
        float* dst = out + h * D + 4 * c4;
        const float r = L > 0.0f ? L : 1.0f;     // as in the attention kernel
        dst[0] = o.x / r, dst[1] = o.y / r, dst[2] = o.z / r, dst[3] = o.w / r;
    }
}

// 8-column tiles of a set: one or two (8 pairs)
inline int tiles_of_set(int64_t C) { return C <= kTilePairs ? 1 : 2; }

}  // namespace

bool store_attend_fits(const AttendMap& map, int Hkv, int T, int Hq) {
    const int64_t C = (int64_t)T * (Hq / Hkv);
    const int pairs = tiles_of_set(C) * kTilePairs;
    const int64_t rows = Hkv * ((C + pairs - 1) / pairs);   // of a session
    int64_t units = 0;
    for (int s = 0; s < map.nsess; ++s) units += (map.n[s] + 1023) / 1024 * rows;
    return units <= INT32_MAX / 32 && map.nsess * rows * pairs <= INT32_MAX;
}

size_t store_attend_workspace_bytes(int S, int T, int Hq, int Hkv, int d) {
    const int64_t C = (int64_t)T * (Hq / Hkv);
    const int pairs = tiles_of_set(C) * kTilePairs;
    const size_t rows = (size_t)S * Hkv * (size_t)((C + pairs - 1) / pairs);
    return ((rows + kMaxCtas) * pairs * (d + 2) * sizeof(float) + 255) & ~size_t(255);
}

namespace {

struct Call {
    const AttendMap& map;
    const void* q;
    int q_dtype, T, Hq, Hkv, sets;
    float *slots, *out, *parts;
    cudaStream_t stream;
    Spans<kAttendSets> at;
    int P;
    int pairs;     // of a set
    bool shared;   // some row's keys may be shared by several CTAs, or a row has none

    // tiles of a row of session s
    int tiles(int s, int tile) const {
        const int64_t last = map.visible[s] + T - 1;   // keys that the last token sees
        const int64_t keys = last < map.n[s] ? (last > 0 ? last : 0) : map.n[s];
        return (int)((keys + tile - 1) / tile);
    }
};

// The tensor maps of a store: planes as words, channels of all heads, planes, a box
// being a tile's 128 bytes of a copy's channels and all planes, 16-byte pieces
// of each row swizzled by the row number; scales as blocks, channels of all
// heads, a box being a tile's blocks of a head's channels.
bool tensor_maps(CUtensorMap* tm, CUtensorMap* stm, const uint32_t* planes, const uint16_t* scales, int channels, int d,
                 int64_t n_pad, int tile) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t row = (cuuint64_t)(n_pad / 8);
    const cuuint64_t dims[3] = {row / 4, (cuuint64_t)channels, 4}, strides[2] = {4 * row, row};
    const cuuint32_t box[3] = {(cuuint32_t)tile / 32, (cuuint32_t)(d < 64 ? 32 : 64), 4}, step[3] = {1, 1, 1};
    const cuuint64_t sdims[2] = {(cuuint64_t)(n_pad / kBlock), (cuuint64_t)channels}, sstrides[1] = {(cuuint64_t)(n_pad / kBlock) * 2};
    const cuuint32_t sbox[2] = {(cuuint32_t)tile / kBlock, (cuuint32_t)d};
    return encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint32_t*>(planes), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, tile == 1024 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
           encode(stm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<uint16_t*>(scales), sdims, sstrides, sbox, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, tile == 1024 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Lays the sessions out in tiles, each row's number a multiple of `granule`; the number of units.
int lay_out(Call& a, int tile, int granule) {
    int64_t U = 0;
    for (int s = 0; s < a.map.nsess; ++s) {
        Span& sp = a.at.span[s];
        sp.n = (int)a.map.n[s];
        sp.visible = (int)a.map.visible[s];
        sp.unit0 = (int)U;
        sp.tiles = (a.tiles(s, tile) + granule - 1) / granule * granule;
        U += (int64_t)sp.tiles * a.Hkv * a.sets;
        a.shared = a.shared || sp.tiles != 1;
    }
    return (int)U;
}

// Clusters of 2, 4 or 8 CTAs of the half tiles' kernel that the current device holds at once, or (alone) holds with an
// SM for each CTA.  A GPU's groups of SMs need not be whole clusters: on B200 it is 148, 71 and 33 at two CTAs to an
// SM, and 74, 33 and 15 at one.  A device is asked once.
template <int D, int NT, bool F32>
int resident_clusters(int cluster, bool alone) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[2][kDevices][kMaxCluster + 1];   // the number and 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
    std::atomic<int>& at = known[alone][dev][cluster];
    int held = at.load(std::memory_order_relaxed) - 1;
    if (held < 0) {
        constexpr size_t kHalf = kMaxSmem / 2 + 1024;   // an SM has no room for two of these
        constexpr size_t kSmem = Shape<D, NT, F32, 1>::kSmem;
        const size_t smem = alone && kSmem < kHalf ? kHalf : kSmem;
        auto kern = store_attend_kernel<D, NT, F32, 1, 1>;
        cudaLaunchAttribute size;
        size.id = cudaLaunchAttributeClusterDimension;
        size.val.clusterDim.x = (unsigned)cluster;
        size.val.clusterDim.y = size.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(cluster);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &size;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSmem > kHalf ? kSmem : kHalf)) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&held, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        at.store(held + 1, std::memory_order_relaxed);
    }
    return held;
}

// CTAs of the cluster that takes a row of 2 to 8 half tiles and adds its partials itself, or 1: each tile by itself
// and a second launch, which costs 0.5 to 1.2 us.  Clusters that are not all resident take a second turn (2049 keys,
// 40 heads of 128: 18.2 us against 11.9; 16 heads of 256: 25.4 against 14.1).  With heads of 128 two of a cluster's CTAs
// on an SM cost more than the second launch where that would leave an SM to each tile (4096 keys, between two small
// kernels and with them: 12 heads 11.3 us against 11.9, 16 heads 13.1 against 12.4, 20 heads, 160 tiles, 13.8 against
// 14.2); with narrower heads they do not (16 heads of 32 8.2 against 9.1, 24 of 64, 1500 keys, 8 queries: 10.0 against 11.2).
template <int D, int NT, bool F32>
int cluster_of(const Call& a) {
    const int tiles = a.tiles(0, Shape<D, NT, F32, 1>::kTile), rows = a.Hkv * a.sets;
    if (tiles < 2 || tiles > kMaxCluster) return 1;
    int cluster = 2;
    while (cluster < tiles) cluster *= 2;
    if (D >= 128 && (int64_t)rows * tiles <= 148 && rows > resident_clusters<D, NT, F32>(cluster, true)) return 1;
    return rows <= resident_clusters<D, NT, F32>(cluster, false) ? cluster : 1;
}

template <int D, int NT, bool F32, int NS, int NB>
cudaError_t launch_shape(Call& a) {
    using Sh = Shape<D, NT, F32, NB>;
    static_assert(Sh::kCtas * (Sh::kSmem + 1024) <= kMaxSmem + 1024, "the CTAs of an SM fit");
    int cluster = 1;
    if constexpr (NS == 1 && NB == 1) cluster = cluster_of<D, NT, F32>(a);
    a.shared = false;
    const int U = lay_out(a, Sh::kTile, cluster);
    a.P = U < 148 * Sh::kCtas || cluster > 1 ? U : 148 * Sh::kCtas;
    a.at.each = U / a.P;
    a.at.more = U % a.P;
    Sessions<NS> m;
    m.at.nsess = a.at.nsess;
    m.at.each = a.at.each;
    m.at.more = a.at.more;
    m.at.cluster = cluster;
    a.shared = a.shared && cluster == 1;
    for (int s = 0; s < a.at.nsess; ++s) {
        m.at.span[s] = a.at.span[s];
        if (!tensor_maps(&m.k[s], &m.ks[s], a.map.k_planes[s], a.map.k_scales[s], a.Hkv * D, D, a.map.k_pad[s], Sh::kTile) ||
            !tensor_maps(&m.v[s], &m.vs[s], a.map.v_planes[s], a.map.v_scales[s], a.Hkv * D, D, a.map.v_pad[s], Sh::kTile))
            return cudaErrorInvalidValue;
    }
    auto kern = store_attend_kernel<D, NT, F32, NS, NB>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sh::kSmem);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3(a.P), dim3(kThreads), Sh::kSmem, a.stream, true, cluster, m, a.q, a.q_dtype, a.T, a.Hq, a.Hkv,
                     a.sets, a.slots, a.out, a.parts, device_status_ptr());
}

template <int D, int NT, bool F32>
cudaError_t launch_type(Call& a, int units) {
    if (a.at.nsess > 1) return launch_shape<D, NT, F32, kAttendSets, 2>(a);
    // few keys: half as long tiles, as long as all run at once (1 head of 128, 4096 keys: 9.0 us against
    // 11.4; 2 heads of 256, 8 queries each, 70001 keys, whose half tiles would not: 36 us against 27)
    if (2 * units <= 148 * Shape<D, NT, F32, 1>::kCtas) return launch_shape<D, NT, F32, 1, 1>(a);
    return launch_shape<D, NT, F32, 1, 2>(a);
}

template <int D, bool F32>
cudaError_t launch_dim(Call& a) {
    const int64_t C = (int64_t)a.T * (a.Hq / a.Hkv);
    a.pairs = kTilePairs;
    a.sets = (int)((C + kTilePairs - 1) / kTilePairs);
    int units = lay_out(a, 1024, 1);
    if (tiles_of_set(C) == 2) {
        // few keys and many queries: sets of 4, while each half tile has an SM of its own, or half of one in the
        // cluster of a short row (1 head of 128, 8 queries, 4096 keys: 8.0 us against 10.3; 16 heads: 11.0
        // against 14.2; 8 heads, 9000 keys, where two would share an SM: 13.9 against 12.6; 24 heads, 3000 keys,
        // whose clusters would not all be resident: 14.7 against 13.3)
        const bool alone = 2 * units <= 148 || (D <= 128 && (int64_t)a.Hkv * a.sets * a.tiles(0, 512) <= 148);
        const bool together = D <= 128 && 2 * units <= 2 * 148 && (a.tiles(0, 512) == 1 || cluster_of<D, 1, F32>(a) > 1);
        if (a.map.nsess > 1 || (!alone && !together)) {
            a.pairs = 2 * kTilePairs;
            a.sets = (int)((C + a.pairs - 1) / a.pairs);
            units = lay_out(a, 1024, 1);
        }
    }
    if (units == 0) return cudaSuccess;
    return a.pairs == kTilePairs ? launch_type<D, 1, F32>(a, units) : launch_type<D, 2, F32>(a, units);
}

}  // namespace

cudaError_t launch_store_attend(const AttendMap& map, int Hkv, int d, const void* q, int q_dtype, int T, int Hq, float* out,
                                float* parts, void* ws, cudaStream_t stream) {
    Call a{map, q, q_dtype, T, Hq, Hkv, 0, static_cast<float*>(ws), out, parts, stream, {}, 0, 0, true};
    a.at.nsess = map.nsess;
    const bool f32 = q_dtype == FATHOM_F32;
    cudaError_t e;
    switch (d) {
        case 32: e = f32 ? launch_dim<32, true>(a) : launch_dim<32, false>(a); break;
        case 64: e = f32 ? launch_dim<64, true>(a) : launch_dim<64, false>(a); break;
        case 128: e = f32 ? launch_dim<128, true>(a) : launch_dim<128, false>(a); break;
        case 256: e = f32 ? launch_dim<256, true>(a) : launch_dim<256, false>(a); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess || !a.shared) return e;
    return launch_ex(store_attend_merge_kernel, dim3((unsigned)((int64_t)map.nsess * Hkv * a.sets * a.pairs)),
                     dim3(kMergeThreads), 0, stream, a.P > 0, 1, a.at, a.slots, T, Hq, Hkv, a.sets, a.pairs, d, out, parts);
}

}  // namespace fathom
