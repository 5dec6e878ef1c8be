// The K store and the V store of a layer grow from its row cache: the bf16
// rows of the new keys, and of the last partial 64-token block, packed into
// bit planes where they lie, both stores in one launch.  Codes, scales and
// planes as pack_kernel writes them, bit for bit.
//
// One CTA per (four aligned 64-token blocks, KV head, store): four blocks
// are 32 bytes of every plane row, one memory sector, so the planes leave as
// whole sectors.  A thread holds two channels x 64 keys of one block in
// registers (a warp's load reads 128 contiguous bytes of a row), so the
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

constexpr int kGroup = 4;   // blocks per CTA: 256 keys, a 32-byte sector of a plane row

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
__device__ __forceinline__ void pack_pair(const uint16_t* __restrict__ p, int64_t row_stride, int keys, uint32_t* __restrict__ s_w,
                                          uint16_t* __restrict__ scale0, uint16_t* __restrict__ scale1) {
    uint32_t x[kBlock];
    __nv_bfloat162 mx = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kBlock; ++i) x[i] = FULL || i < keys ? *reinterpret_cast<const uint32_t*>(p + i * row_stride) : 0u;
#pragma unroll
    for (int i = 0; i < kBlock; ++i) mx = __hmax2(mx, __habs2(*reinterpret_cast<__nv_bfloat162*>(&x[i])));
    const __half d0 = __float2half_rn(__low2float(mx) * 0.125f), d1 = __float2half_rn(__high2float(mx) * 0.125f);
    *scale0 = __half_as_ushort(d0);
    *scale1 = __half_as_ushort(d1);
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
            for (int j = 0; j < 4; ++j) s_w[e * 33 + j * 8 + w] = W[j];
        }
    }
}

__global__ void __launch_bounds__(2 * kMaxD)
append_rows_kernel(AppendSide ks, AppendSide vs, int Hkv, int64_t rows_n, int64_t row_stride, int64_t blk0, int64_t n,
                   int d) {
    pdl_wait();
    extern __shared__ uint32_t s_w[];   // [d][33]: channel's plane words [4][8], padded
    const int half = d / 2;
    const int b = threadIdx.x / half, cp = threadIdx.x - b * half;   // block of the group, channel pair
    const int g = blockIdx.y % Hkv;
    const AppendSide& sd = blockIdx.y < Hkv ? ks : vs;
    const int64_t group = (blk0 / kGroup + blockIdx.x) * kGroup;     // first block of the group
    const int64_t blk = group + b;
    const int64_t rem = n - blk * kBlock;
    const int64_t words = sd.n_pad / 32;

    if (blk >= blk0 && rem > 0) {
        const uint16_t* p = sd.rows + ((int64_t)g * rows_n + blk * kBlock) * row_stride + 2 * cp;
        uint16_t* sc = sd.scales + ((int64_t)g * d + 2 * cp) * (sd.n_pad / kBlock) + blk;
        uint32_t* w = s_w + 2 * cp * 33 + 2 * b;
        if (rem >= kBlock) pack_pair<true>(p, row_stride, kBlock, w, sc, sc + sd.n_pad / kBlock);
        else pack_pair<false>(p, row_stride, (int)rem, w, sc, sc + sd.n_pad / kBlock);
    }
    __syncthreads();
    // the group's words of every plane row: a whole sector, or the blocks that were packed
    const int64_t last = (n + kBlock - 1) / kBlock;
    const int lo = blk0 > group ? (int)(blk0 - group) : 0;
    const int hi = last - group < kGroup ? (int)(last - group) : kGroup;
    for (int row = threadIdx.x; row < 4 * d; row += blockDim.x) {
        const uint32_t* s = s_w + (row >> 2) * 33 + (row & 3) * 8;
        uint32_t* o = sd.planes + ((int64_t)g * d * 4 + row) * words + group * 2;
        if (lo == 0 && hi == kGroup) {
            reinterpret_cast<uint4*>(o)[0] = make_uint4(s[0], s[1], s[2], s[3]);
            reinterpret_cast<uint4*>(o)[1] = make_uint4(s[4], s[5], s[6], s[7]);
        } else {
            for (int e = lo; e < hi; ++e) reinterpret_cast<uint2*>(o)[e] = make_uint2(s[2 * e], s[2 * e + 1]);
        }
    }
}

}  // namespace

cudaError_t launch_append_rows(const uint16_t* K_rows, uint32_t* k_planes, uint16_t* k_scales, int64_t k_pad,
                               const uint16_t* V_rows, uint32_t* v_planes, uint16_t* v_scales, int64_t v_pad, int Hkv,
                               int d, int64_t rows_n, int64_t row_stride, int64_t blk0, int64_t n,
                               cudaStream_t stream) {
    const AppendSide ks{K_rows, k_planes, k_scales, k_pad}, vs{V_rows, v_planes, v_scales, v_pad};
    const int64_t groups = ((n + kBlock - 1) / kBlock + kGroup - 1) / kGroup - blk0 / kGroup;
    dim3 grid((unsigned)groups, (unsigned)(V_rows ? 2 * Hkv : Hkv));
    return launch_ex(append_rows_kernel, grid, dim3(2 * d), sizeof(uint32_t) * 33 * d, stream, true, 1, ks, vs, Hkv,
                     rows_n, row_stride, blk0, n, d);
}

}  // namespace fathom
