// Norms of query and key heads with the rotation by position, in one pass
// over the rows of a layer's fused projection, written where the decode path
// reads them: queries to their own array, keys (rotated) and values (as they
// are) to the layer's row cache.
//
//   y = x / sqrt(mean_c x_c^2 + eps) * w               (heads with a weight)
//   (a, b) <- (a cos f - b sin f, b cos f + a sin f)    for the pairs (a, b) of
//   the first rot_dim channels, f = position * inv_freq[pair]
//
// in fp32, rounded once to the output type.  The angle is reduced in fp64 (at
// position 10^6 an fp32 product has lost 0.03 rad): r = 4 f / 2 pi less its
// nearest integer k lies in [-1/2, 1/2], so rounding r to fp32 costs at most
// 2^-26 * pi / 2 = 2.3e-8 rad, less than the rounding of the sine itself.
//
// One CTA per token and set of heads: the token's sines and cosines are
// computed once, a lane keeps those of its pairs in registers, and groups of
// lanes take a head each, the next head's channels on their way meanwhile.
// A lane holds 16 channels of its head as two 8-channel pieces; for pairs
// (i, i + rot_dim / 2) the two pieces are the two sides of the same 8 pairs,
// so the rotation needs no exchange between lanes.
#include <type_traits>

#include "fathom_internal.cuh"

namespace fathom {
namespace {

constexpr int kThreads = 128;

// eight channels as they lie in memory
template <bool F32>
struct Raw {
    uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(const void* p, int64_t i) {
    Raw<F32> r;
    const uint4* v = F32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i)
                         : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    r.w[0] = v[0];
    if (F32) r.w[F32 ? 1 : 0] = v[1];
    return r;
}
template <bool F32>
__device__ __forceinline__ void floats_of(const Raw<F32>& r, float* x) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (F32) {
            x[e] = __uint_as_float(w[e]);
        } else {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    if (F32) {
        const uint4 v = r.w[F32 ? 1 : 0];
        x[4] = __uint_as_float(v.x), x[5] = __uint_as_float(v.y), x[6] = __uint_as_float(v.z), x[7] = __uint_as_float(v.w);
    }
}

__device__ __forceinline__ void store8(void* p, int dtype, int64_t i, const float* x) {
    if (dtype == FATHOM_BF16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// sin and cos of position * inv_freq
__device__ __forceinline__ float2 sin_cos(int position, float inv_freq) {
    const double quarter = (double)position * (double)inv_freq * 0.63661977236758134308;   // 2 / pi
    const double k = rint(quarter);
    const float r = (float)(quarter - k);
    float s, c;
    sincospif(0.5f * r, &s, &c);
    const int q = (int)((long long)k & 3);
    const float s1 = (q & 1) ? c : s, c1 = (q & 1) ? s : c;
    return make_float2((q & 2) ? -s1 : s1, (q == 1 || q == 2) ? -c1 : c1);
}

// LPR = lanes per head: d/16 rounded up to a power of two; F32, W32: type of the
// rows and queries, and of the weights
template <int LPR, bool F32, bool W32>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const void* __restrict__ qkv, int64_t token_stride, int Hq, int Hkv, int d, const void* __restrict__ q_weight,
            const void* __restrict__ k_weight, float eps, const int32_t* __restrict__ positions,
            const float* __restrict__ inv_freq, int rot, int interleaved, void* __restrict__ q_out,
            uint16_t* __restrict__ K_rows, uint16_t* __restrict__ V_rows, int64_t row_stride, int64_t rows_n, int64_t row0) {
    __shared__ float2 s_sc[kMaxD / 2];   // (sin, cos) of the token's pairs
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int H = Hq + 2 * Hkv;
    const int j = threadIdx.x % LPR;
    const bool on = j < d / 16;
    // the lane's two pieces: of a rotated head the two sides of 8 pairs, then the channels behind
    const int rl = rot / 16;   // lanes that hold rotated channels
    const bool split = !interleaved && j < rl;
    const int c0 = split ? 8 * j : 16 * j, c1 = split ? rot / 2 + 8 * j : c0 + 8;
    constexpr int kHeads = kThreads / LPR;
    const int step = gridDim.y * kHeads;
    int h = blockIdx.y * kHeads + threadIdx.x / LPR;

    const Raw<F32> zero{};
    Raw<F32> ra = zero, rb = zero;
    if (on && h < H) {
        ra = load_raw<F32>(qkv, t * token_stride + (int64_t)h * d + c0);
        rb = load_raw<F32>(qkv, t * token_stride + (int64_t)h * d + c1);
    }
    const int position = positions ? positions[t] : (int)(row0 + t);
    for (int i = threadIdx.x; i < rot / 2; i += kThreads) s_sc[i] = sin_cos(position, inv_freq[i]);
    __syncthreads();
    float2 f[8];
    if (j < rl) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = s_sc[8 * j + e];
    }

    // every warp takes as many turns as its first lane group needs: its sums take all lanes
    for (int base = blockIdx.y * kHeads; base < H; base += step, h += step) {
        float a[8], b[8];
        floats_of<F32>(ra, a);
        floats_of<F32>(rb, b);
        ra = rb = zero;
        if (on && h + step < H) {
            ra = load_raw<F32>(qkv, t * token_stride + (int64_t)(h + step) * d + c0);
            rb = load_raw<F32>(qkv, t * token_stride + (int64_t)(h + step) * d + c1);
        }
        const bool act = on && h < H;
        if (q_weight) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (act && h < Hq + Hkv) {
                const void* w = h < Hq ? q_weight : k_weight;
                const float r = 1.0f / sqrtf(ss / (float)d + eps);
                float wa[8], wb[8];
                floats_of<W32>(load_raw<W32>(w, c0), wa);
                floats_of<W32>(load_raw<W32>(w, c1), wb);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    a[e] *= r * wa[e];
                    b[e] *= r * wb[e];
                }
            }
        }
        if (!act) continue;
        if (h < Hq + Hkv && j < rl) {
            if (interleaved) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 fa = f[e / 2], fb = f[4 + e / 2];
                    const float a0 = a[e], b0 = b[e];
                    a[e] = a0 * fa.y - a[e + 1] * fa.x;
                    a[e + 1] = a[e + 1] * fa.y + a0 * fa.x;
                    b[e] = b0 * fb.y - b[e + 1] * fb.x;
                    b[e + 1] = b[e + 1] * fb.y + b0 * fb.x;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a0 = a[e];
                    a[e] = a0 * f[e].y - b[e] * f[e].x;
                    b[e] = b[e] * f[e].y + a0 * f[e].x;
                }
            }
        }
        if (h < Hq) {
            const int64_t at = (t * Hq + h) * d;
            store8(q_out, F32 ? FATHOM_F32 : FATHOM_BF16, at + c0, a);
            store8(q_out, F32 ? FATHOM_F32 : FATHOM_BF16, at + c1, b);
        } else {
            const bool key = h < Hq + Hkv;
            const int g = key ? h - Hq : h - Hq - Hkv;
            const int64_t at = ((int64_t)g * rows_n + row0 + t) * row_stride;
            store8(key ? K_rows : V_rows, FATHOM_BF16, at + c0, a);
            store8(key ? K_rows : V_rows, FATHOM_BF16, at + c1, b);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const void* qkv, int dtype, int64_t token_stride, int n_tokens, int Hq, int Hkv, int d,
                        const void* q_weight, const void* k_weight, int w_dtype, float eps, const int32_t* positions,
                        const float* inv_freq, int rot, int interleaved, void* q_out, uint16_t* K_rows,
                        uint16_t* V_rows, int64_t row_stride, int64_t rows_n, int64_t row0, cudaStream_t stream) {
    auto go = [&](auto kern, int lpr) {
        const int per_cta = kThreads / lpr, sets = (Hq + 2 * Hkv + per_cta - 1) / per_cta;
        // many tokens: a CTA takes all heads of its token and computes the sines
        // once; few tokens: the heads spread over CTAs
        const int want = (1184 + n_tokens - 1) / n_tokens;
        dim3 grid((unsigned)n_tokens, (unsigned)(want < sets ? want : sets));
        return launch_ex(kern, grid, dim3(kThreads), 0, stream, true, 1, qkv, token_stride, Hq, Hkv, d, q_weight, k_weight,
                         eps, positions, inv_freq, rot, interleaved, q_out, K_rows, V_rows, row_stride, rows_n, row0);
    };
    const bool f32 = dtype == FATHOM_F32, w32 = q_weight && w_dtype == FATHOM_F32;
    auto types = [&](auto lpr) {
        constexpr int L = decltype(lpr)::value;
        if (f32) return w32 ? go(rope_kernel<L, true, true>, L) : go(rope_kernel<L, true, false>, L);
        return w32 ? go(rope_kernel<L, false, true>, L) : go(rope_kernel<L, false, false>, L);
    };
    if (d <= 32) return types(std::integral_constant<int, 2>{});
    if (d <= 64) return types(std::integral_constant<int, 4>{});
    if (d <= 128) return types(std::integral_constant<int, 8>{});
    return types(std::integral_constant<int, 16>{});
}

}  // namespace fathom
