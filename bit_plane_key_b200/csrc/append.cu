// The K store and the V store of a layer grow from its row cache: the bf16
// rows of the new keys, and of the last partial 64-token block, packed into
// bit planes where they lie, both stores in one launch.  Codes, scales and
// planes as pack_kernel writes them, bit for bit.
//
// One CTA per (16 aligned 64-token blocks, 64 or 32 channels of a KV head,
// store): 16 blocks are 128 bytes of every plane row, one line, and leave as one
// write; a warp's load reads 128 (or 64) contiguous bytes of a row.  What bounds the
// kernel is the number of pieces that memory moves: with 4 blocks to a CTA, its
// planes written in pieces of 32 bytes, 131072 keys of 8 heads (d = 128), K and V,
// took 155 us where this takes 130 (5.2 TB/s
// of the 6.6 that a copy reaches).
// A thread holds two channels x 64 keys of one block in registers, so the
// block's largest magnitude needs no exchange.
//
// floor(x / Delta) without a division: with c = 2^23 + 8 and i = 1/Delta
// rounded, fma.rd(x + |x| 2^-21, i, c) is c plus the product rounded down to
// an integer; the low bits are the code.  The three roundings leave a product
// above x/Delta, by a relative 2^-20.5 at most, so a quotient that is an
// integer keeps its cell and a tiny negative x still falls below c.  No
// other quotient in (-9, 9) crosses: it is at least 1/2047 from an integer m != 0.
// (x = X u, |X| <= 255, Delta = D v, D <= 2047, u and v powers of two: for
// u >= v, x - m Delta is a multiple of v and 1/D of Delta or more; for u < v it
// is a multiple of u, and Delta <= 2 |x| <= 510 u.)
// The codes' clamp to [0, 15] is one of x, two channels at a time, to the bf16
// nearest to +-8 Delta from inside: its quotient is in [-8, -7.9] or [7.9, 8).
#include "fathom_internal.cuh"

namespace fathom {
namespace {

constexpr int kGroup = 16;   // blocks per CTA: 1024 keys, a 128-byte line of a plane row
constexpr int kSmall = 4;    // the same of few keys

struct AppendSide {
    const uint16_t* rows;   // row of key i of head g at (g * rows_n + i) * row_stride
    uint32_t* planes;
    uint16_t* scales;
    int64_t n_pad;
};

// nibble words N[r] (nibble m = code of key 4 m + r) -> plane words W[j] (bit i = bit 3 - j of key i's code)
__device__ __forceinline__ void nibbles_to_planes(const uint32_t* N, uint32_t* W) {
    // bits (3,2) of keys 2m + r in P[r], bits (1,0) in Q[r]
    const uint32_t P0 = ((N[0] >> 2) & 0x33333333u) | (N[2] & 0xCCCCCCCCu);
    const uint32_t P1 = ((N[1] >> 2) & 0x33333333u) | (N[3] & 0xCCCCCCCCu);
    const uint32_t Q0 = (N[0] & 0x33333333u) | ((N[2] << 2) & 0xCCCCCCCCu);
    const uint32_t Q1 = (N[1] & 0x33333333u) | ((N[3] << 2) & 0xCCCCCCCCu);
    W[0] = ((P0 >> 1) & 0x55555555u) | (P1 & 0xAAAAAAAAu);
    W[1] = (P0 & 0x55555555u) | ((P1 << 1) & 0xAAAAAAAAu);
    W[2] = ((Q0 >> 1) & 0x55555555u) | (Q1 & 0xAAAAAAAAu);
    W[3] = (Q0 & 0x55555555u) | ((Q1 << 1) & 0xAAAAAAAAu);
}

// the bf16 next to +-8 Delta inside (-8 Delta may be reached, 8 Delta not), as bits
__device__ __forceinline__ uint32_t low_bound(float delta) { return __float_as_uint(-8.0f * delta) >> 16; }
__device__ __forceinline__ uint32_t high_bound(float delta) {
    const uint32_t b = __float_as_uint(8.0f * delta);
    return b == 0u ? 0u : (b - 1u) >> 16;   // the bits below 8 Delta, cut to bf16
}

// One block of a channel pair: x[i] = key i's two bf16 values, FULL: all 64 keys are there.
template <bool FULL>
__device__ __forceinline__ void pack_pair(const uint16_t* __restrict__ p, int64_t row_stride, int keys, uint32_t* __restrict__ s_w, int plane_ld, int ld,
                                          uint16_t* __restrict__ s_scale, int scale_ld) {
    uint32_t x[kBlock];
    __nv_bfloat162 mx = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kBlock; ++i) x[i] = FULL || i < keys ? *reinterpret_cast<const uint32_t*>(p + i * row_stride) : 0u;
#pragma unroll
    for (int i = 0; i < kBlock; ++i) mx = __hmax2(mx, __habs2(*reinterpret_cast<__nv_bfloat162*>(&x[i])));
    const __half d0 = __float2half_rn(__low2float(mx) * 0.125f), d1 = __float2half_rn(__high2float(mx) * 0.125f);
    s_scale[0] = __half_as_ushort(d0);
    s_scale[scale_ld] = __half_as_ushort(d1);
    const float delta[2] = {__half2float(d0), __half2float(d1)};
    const uint32_t lo = low_bound(delta[0]) | low_bound(delta[1]) << 16, hi = high_bound(delta[0]) | high_bound(delta[1]) << 16;
#pragma unroll
    for (int i = 0; i < kBlock; ++i) {
        const __nv_bfloat162 v = __hmin2(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), *reinterpret_cast<const __nv_bfloat162*>(&lo)),
                                         *reinterpret_cast<const __nv_bfloat162*>(&hi));
        x[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float inv = delta[e] > 0.0f ? __frcp_rn(delta[e]) : 0.0f;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint32_t N[4], W[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // the floats 2^23 + code, shifted and added as they are, less their exponents
                N[r] = 0u - 0x4B000000u * 0x11111111u;
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    const int i = 32 * w + 4 * m + r;
                    const float v = __uint_as_float(e ? (x[i] & 0xFFFF0000u) : (x[i] << 16));
                    const float u = __fmaf_rd(fmaf(fabsf(v), 4.76837158203125e-7f, v), inv, 8388616.0f);
                    N[r] += (FULL || i < keys ? __float_as_uint(u) : 0x4B000000u) * (1u << (4 * m));
                }
            }
            nibbles_to_planes(N, W);
#pragma unroll
            for (int j = 0; j < 4; ++j) s_w[j * plane_ld + w * ld + e] = W[j];
        }
    }
}

// PAIRS channel pairs and GROUP blocks to a CTA
template <int PAIRS, int GROUP>
constexpr int threads_of() { return PAIRS * (GROUP < 8 ? GROUP : 256 / PAIRS); }
template <int PAIRS, int GROUP>
__global__ void __launch_bounds__((threads_of<PAIRS, GROUP>()), 512 / threads_of<PAIRS, GROUP>())
append_rows_kernel(AppendSide ks, AppendSide vs, int64_t rows_n, int64_t row_stride, int64_t blk0, int64_t n, int d) {
    constexpr int kThreads = threads_of<PAIRS, GROUP>(), kBlocks = kThreads / PAIRS;   // blocks at a time
    constexpr int kLd = 2 * PAIRS + 1, kScaleLd = GROUP + 2, kWords = 2 * GROUP;
    __shared__ uint32_t s_w[4 * kWords * kLd];             // [plane][word of the group][channel]
    __shared__ uint16_t s_sc[2 * PAIRS * kScaleLd];        // [channel][block]
    pdl_wait();
    const int tiles = d / (2 * PAIRS), c0 = blockIdx.z % tiles * 2 * PAIRS;
    const AppendSide& sd = (int)blockIdx.z < tiles ? ks : vs;
    const int64_t g = blockIdx.y, group = (blk0 / GROUP + blockIdx.x) * GROUP;   // head, first block of the group
    const int64_t words = sd.n_pad / 32, blocks = sd.n_pad / kBlock;
    const int cp = threadIdx.x % PAIRS;
#pragma unroll 1
    for (int b = threadIdx.x / PAIRS; b < GROUP; b += kBlocks) {
        const int64_t blk = group + b, rem = n - blk * kBlock;
        if (blk < blk0 || rem <= 0) continue;
        const uint16_t* p = sd.rows + (g * rows_n + blk * kBlock) * row_stride + c0 + 2 * cp;
        uint32_t* w = s_w + 2 * b * kLd + 2 * cp;
        uint16_t* sc = s_sc + 2 * cp * kScaleLd + b;
        if (rem >= kBlock) pack_pair<true>(p, row_stride, kBlock, w, kWords * kLd, kLd, sc, kScaleLd);
        else pack_pair<false>(p, row_stride, (int)rem, w, kWords * kLd, kLd, sc, kScaleLd);
    }
    __syncthreads();
    // the plane rows' words and the scales of the blocks that were packed
    const int wl = threadIdx.x % kWords;
    if (group + wl / 2 >= blk0 && (group + wl / 2) * kBlock < n) {
        uint32_t* o = sd.planes + (g * d + c0) * 4 * words + group * 2 + wl;
        for (int row = threadIdx.x / kWords; row < 8 * PAIRS; row += kThreads / kWords)
            o[row * words] = s_w[((row & 3) * kWords + wl) * kLd + (row >> 2)];
    }
    const int bl = threadIdx.x % GROUP;
    if (group + bl >= blk0 && (group + bl) * kBlock < n) {
        uint16_t* o = sd.scales + (g * d + c0) * blocks + group + bl;
        for (int c = threadIdx.x / GROUP; c < 2 * PAIRS; c += kThreads / GROUP) o[c * blocks] = s_sc[c * kScaleLd + bl];
    }
}

}  // namespace

cudaError_t launch_append_rows(const uint16_t* K_rows, uint32_t* k_planes, uint16_t* k_scales, int64_t k_pad,
                               const uint16_t* V_rows, uint32_t* v_planes, uint16_t* v_scales, int64_t v_pad, int Hkv,
                               int d, int64_t rows_n, int64_t row_stride, int64_t blk0, int64_t n,
                               cudaStream_t stream) {
    const AppendSide ks{K_rows, k_planes, k_scales, k_pad}, vs{V_rows, v_planes, v_scales, v_pad};
    const int pairs = d % 64 == 0 ? 32 : 16, z = (V_rows ? 2 : 1) * (d / (2 * pairs));
    const int64_t last = (n + kBlock - 1) / kBlock;   // blocks
    auto groups = [&](int group) { return (last + group - 1) / group - blk0 / group; };
    auto go = [&](auto kern, int group, int threads) {
        return launch_ex(kern, dim3((unsigned)groups(group), (unsigned)Hkv, (unsigned)z), dim3(threads), 0, stream, true, 1,
                         ks, vs, rows_n, row_stride, blk0, n, d);
    };
    // few keys: more CTAs of fewer blocks, rather than whole lines from CTAs that leave SMs idle
    // (4097 keys, 2 heads of 64: 4.1 us against 6.6; 131072 keys, 8 heads of 128: 155 against 130)
    if (groups(kGroup) * Hkv * z < 2 * 148) {
        return pairs == 32 ? go(append_rows_kernel<32, kSmall>, kSmall, threads_of<32, kSmall>())
                           : go(append_rows_kernel<16, kSmall>, kSmall, threads_of<16, kSmall>());
    }
    return pairs == 32 ? go(append_rows_kernel<32, kGroup>, kGroup, threads_of<32, kGroup>())
                       : go(append_rows_kernel<16, kGroup>, kGroup, threads_of<16, kGroup>());
}

}  // namespace fathom
