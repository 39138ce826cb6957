// Norms of queries and keys for each head with the position rotation in the same pass, and
// its gradients.
//
// For one head row x of d channels (w optional, R = the first `rotary` channels):
//   xh = x r,  r = 1 / max(||x||, 1e-12) (L2), 1 / sqrt(mean x^2 + eps) (RMS) or 1 (none)
//   z  = w (.) xh,   y = s Rot(z),   s = q_scale for queries, 1 for keys
// Rot turns channel pair p by the angle pos * inv_freq[p] (times rope_scale in length); pairs
// are (p, p + R/2) in the half layout and (2p, 2p + 1) in the interleaved one. Backward:
//   dz = s Rot^T dy,  dw = sum dz (.) xh,  dxh = w (.) dz,
//   dx = r (dxh - xh <dxh, xh> c)      c = 1 (L2), 1/d (RMS), 0 (none, or a norm at its floor)
//
// HBM-bound: each row is read once and written once, everything between in fp32 registers, one
// rounding at the store. The angle is formed and reduced to one turn in 64 bits (a position of
// a million turns an fp32 angle by 0.06 rad), once per token and pair, shared by all heads
// through shared memory. Vector path: G lanes per row, 16 bytes each, UR rows per thread in
// flight; a rotated pair's other half comes from a lane R/16 away. Rows of other sizes or
// alignments take the scalar path, one warp per row through a row buffer.
#pragma once
#include "gated_common.cuh"

namespace ckda {
namespace gated {

enum { kNormNone = 0, kNormL2 = 1, kNormRms = 2 };

struct PrepArgs {
    const void* x[2];              // q, k
    const void* dy[2];             // backward: cotangents
    void* out[2];                  // forward: y; backward: dx
    const float* w[2];             // per-channel weights or NULL
    long long stride[2];           // elements from token to token of x
    int heads[2];
    const void* pos;               // int32 or int64 positions, or NULL: token % period
    const double* inv_freq;        // [rotary / 2]
    int pos64, period, tokens, d, rotary, norm, interleaved;
    float eps, q_scale, rope_scale;
    float* partial;                // backward: [blocks][2][d] sums of dw, or NULL
};

__device__ __forceinline__ float2 turn(const PrepArgs& a, int token, int p) {
    const double pos = a.pos == nullptr ? (double)(token % a.period)
                       : a.pos64 ? (double)__ldg(static_cast<const long long*>(a.pos) + token)
                                 : (double)__ldg(static_cast<const int*>(a.pos) + token);
    double t = pos * __ldg(a.inv_freq + p) * 0.15915494309189533577;    // turns
    t -= rint(t);
    float s, c;
    sincospif(2.f * (float)t, &s, &c);
    return make_float2(c * a.rope_scale, s * a.rope_scale);
}

__device__ __forceinline__ float norm_factor(const PrepArgs& a, float ss, float& coef) {
    if (a.norm == kNormL2) {
        const float n = sqrtf(ss);
        coef = n > 1e-12f ? 1.f : 0.f;
        return 1.f / fmaxf(n, 1e-12f);
    }
    if (a.norm == kNormRms) {
        coef = 1.f / (float)a.d;
        return 1.f / sqrtf(ss / (float)a.d + a.eps);
    }
    coef = 0.f;
    return 1.f;
}

template <typename T> struct Vec8 { float4 lo, hi; };           // 8 elements as loaded
template <> struct Vec8<__nv_bfloat16> { uint4 raw; };

__device__ __forceinline__ Vec8<float> ld8(const float* p) {
    return {*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4)};
}
__device__ __forceinline__ Vec8<__nv_bfloat16> ld8(const __nv_bfloat16* p) {
    return {*reinterpret_cast<const uint4*>(p)};
}
__device__ __forceinline__ void unpack8(const Vec8<float>& v, float (&x)[8]) {
    x[0] = v.lo.x; x[1] = v.lo.y; x[2] = v.lo.z; x[3] = v.lo.w;
    x[4] = v.hi.x; x[5] = v.hi.y; x[6] = v.hi.z; x[7] = v.hi.w;
}
__device__ __forceinline__ void unpack8(const Vec8<__nv_bfloat16>& v, float (&x)[8]) {
    const uint32_t u[4] = {v.raw.x, v.raw.y, v.raw.z, v.raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void st8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// Turn the 8 channels at e0 (all lanes of the warp take part). sign = -1 turns back.
template <int G>
__device__ __forceinline__ void rotate8(float (&x)[8], const PrepArgs& a, const float2* cs, int e0, float sign) {
    const int R = a.rotary;
    if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e0 + 2 * i < R) {
                const float2 t = cs[e0 / 2 + i];
                const float s = sign * t.y, u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = u * t.x - v * s;
                x[2 * i + 1] = v * t.x + u * s;
            }
        return;
    }
    const int half = R / 2, lane = threadIdx.x & 31, away = half / 8;
    const bool first = e0 < half, in = e0 < R;
    const int other = in ? (first ? lane + away : lane - away) : lane;
    const int p0 = in ? (first ? e0 : e0 - half) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[i], other);
        if (in) {
            const float2 t = cs[p0 + i];
            const float s = sign * t.y;
            x[i] = first ? x[i] * t.x - y * s : x[i] * t.x + y * s;
        }
    }
}

// Vector path: d a multiple of 8, rows 16-byte aligned, half layout with R a multiple of 16.
// A block takes `tpb` tokens at a time (all their heads), grid-stride over the tokens.
template <typename TIn, int G, int UR, bool kBack>
__global__ void __launch_bounds__(256)
prep_vec_kernel(const PrepArgs a, int tpb) {
    extern __shared__ __align__(16) float smf[];
    constexpr int GROUPS = 256 / G;
    const int half = a.rotary / 2, H = a.heads[0] + a.heads[1];
    float2* cs = reinterpret_cast<float2*>(smf);                // [tpb][half]
    float* sw = smf + 2 * tpb * half;                           // [2][d] weights, then the dw reduction
    const int lane = threadIdx.x % G, grp = threadIdx.x / G, e0 = 8 * lane;
    const bool live = e0 < a.d;
    for (int i = threadIdx.x; i < 2 * a.d; i += 256) {
        const float* w = a.w[i / a.d];
        sw[i] = w ? w[i % a.d] : 1.f;
    }
    float acc[2][8];
    if constexpr (kBack) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
    }
    for (int t0 = blockIdx.x * tpb; t0 < a.tokens; t0 += gridDim.x * tpb) {
        const int rows = min(tpb, a.tokens - t0) * H;
        for (int r0 = 0; r0 < rows; r0 += GROUPS * UR) {
            Vec8<TIn> vx[UR], vd[kBack ? UR : 1];
#pragma unroll
            for (int j = 0; j < UR; ++j) {                      // all loads of the pass in flight
                const int r = r0 + j * GROUPS + grp;
                if (r < rows && live) {
                    const int tok = t0 + r / H, h = r % H, which = h >= a.heads[0], hh = which ? h - a.heads[0] : h;
                    vx[j] = ld8(static_cast<const TIn*>(a.x[which]) + tok * a.stride[which] + (long long)hh * a.d + e0);
                    if constexpr (kBack)
                        vd[j] = ld8(static_cast<const TIn*>(a.dy[which]) + ((long long)tok * a.heads[which] + hh) * a.d + e0);
                }
            }
            if (r0 == 0) {
                __syncthreads();                                // the tokens before are done with cs
                for (int i = threadIdx.x; i < min(tpb, a.tokens - t0) * half; i += 256)
                    cs[i] = turn(a, t0 + i / half, i % half);
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < UR; ++j) {
                const int r = r0 + j * GROUPS + grp;
                if (r0 + j * GROUPS >= rows) break;             // uniform in the block
                const bool on = r < rows && live;
                const int rr = r < rows ? r : rows - 1;
                const int lt = rr / H, h = rr % H, which = h >= a.heads[0], hh = which ? h - a.heads[0] : h;
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
                if (on) unpack8(vx[j], x);
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int off = G / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                float coef;
                const float f = norm_factor(a, ss, coef);
                const float scale = which ? 1.f : a.q_scale;
                const float* w = sw + which * a.d + (live ? e0 : 0);
                const float2* c = cs + lt * half;
                if constexpr (!kBack) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = x[i] * f * w[i] * scale;
                    if (half) rotate8<G>(x, a, c, e0, 1.f);
                } else {
                    float z[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[i] = 0.f;
                    if (on) unpack8(vd[j], z);
                    if (half) rotate8<G>(z, a, c, e0, -1.f);
                    float dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] *= f;
                        z[i] *= scale;
                        const float dw = z[i] * x[i];
                        if (which) acc[1][i] += dw; else acc[0][i] += dw;
                        z[i] *= w[i];
                        dot = fmaf(z[i], x[i], dot);
                    }
#pragma unroll
                    for (int off = G / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = f * (z[i] - x[i] * (dot * coef));
                }
                if (on) st8(static_cast<TIn*>(a.out[which]) + ((long long)(t0 + lt) * a.heads[which] + hh) * a.d + e0, x);
            }
        }
    }
    if constexpr (kBack) {
        if (a.partial == nullptr) return;
        for (int s = 0; s < 2; ++s) {                           // groups in turn: one order of the sum
            __syncthreads();
            float* red = smf;                                   // [GROUPS][d], over the angles
            if (live)
#pragma unroll
                for (int i = 0; i < 8; ++i) red[grp * a.d + e0 + i] = s ? acc[1][i] : acc[0][i];
            __syncthreads();
            for (int c = threadIdx.x; c < a.d; c += 256) {
                float sum = 0.f;
                for (int gi = 0; gi < GROUPS; ++gi) sum += red[gi * a.d + c];
                a.partial[((size_t)blockIdx.x * 2 + s) * a.d + c] = sum;
            }
        }
    }
}

// Scalar path: one warp per row, d <= 256, any even R and any alignment.
template <typename TIn, bool kBack>
__global__ void __launch_bounds__(256)
prep_row_kernel(const PrepArgs a) {
    __shared__ float2 cs[128];
    __shared__ float buf[8][256];
    __shared__ float red[8][256];
    const int half = a.rotary / 2, H = a.heads[0] + a.heads[1], warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float acc[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
    auto rotated = [&](int e, float sign) {                     // channel e of the turned row in buf
        const float x = buf[warp][e];
        if (e >= a.rotary) return x;
        const int p = a.interleaved ? e / 2 : (e < half ? e : e - half);
        const bool first = a.interleaved ? (e & 1) == 0 : e < half;
        const int o = a.interleaved ? (e ^ 1) : (first ? e + half : e - half);
        const float y = buf[warp][o], s = sign * cs[p].y;
        return first ? x * cs[p].x - y * s : x * cs[p].x + y * s;
    };
    for (int t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        __syncthreads();
        for (int p = threadIdx.x; p < half; p += 256) cs[p] = turn(a, t, p);
        __syncthreads();
        for (int h = warp; h < H; h += 8) {
            const int which = h >= a.heads[0], hh = which ? h - a.heads[0] : h;
            const TIn* xp = static_cast<const TIn*>(a.x[which]) + t * a.stride[which] + (long long)hh * a.d;
            const long long row = ((long long)t * a.heads[which] + hh) * a.d;
            const float* w = a.w[which];
            const float scale = which ? 1.f : a.q_scale;
            float x[8], z[8], ss = 0.f, coef;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = lane + 32 * i;
                x[i] = e < a.d ? to_f32(xp[e]) : 0.f;
                ss = fmaf(x[i], x[i], ss);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float f = norm_factor(a, ss, coef);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = lane + 32 * i;
                if (e >= a.d) continue;
                if constexpr (kBack) buf[warp][e] = to_f32(static_cast<const TIn*>(a.dy[which])[row + e]);
                else buf[warp][e] = x[i] * f * (w ? w[e] : 1.f) * scale;
            }
            __syncwarp();
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = lane + 32 * i;
                z[i] = e < a.d ? rotated(e, kBack ? -1.f : 1.f) : 0.f;
                if constexpr (kBack) {
                    x[i] *= f;
                    z[i] *= scale;
                    const float dw = z[i] * x[i];
                    if (which) acc[1][i] += dw; else acc[0][i] += dw;
                    if (w && e < a.d) z[i] *= w[e];
                    dot = fmaf(z[i], x[i], dot);
                }
            }
            if constexpr (kBack) {
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = lane + 32 * i;
                if (e >= a.d) continue;
                const float y = kBack ? f * (z[i] - x[i] * (dot * coef)) : z[i];
                static_cast<TIn*>(a.out[which])[row + e] = from_f32<TIn>(y);
            }
        }
    }
    if constexpr (kBack) {
        if (a.partial == nullptr) return;
        for (int s = 0; s < 2; ++s) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) red[warp][lane + 32 * i] = s ? acc[1][i] : acc[0][i];
            __syncthreads();
            for (int c = threadIdx.x; c < a.d; c += 256) {
                float sum = 0.f;
                for (int gi = 0; gi < 8; ++gi) sum += red[gi][c];
                a.partial[((size_t)blockIdx.x * 2 + s) * a.d + c] = sum;
            }
        }
    }
}

// dw of q (columns 0 .. d-1) and k (d .. 2d-1): the blocks' partial sums in a fixed order, one
// block of 256 threads per 32 columns (8 strands of blocks, then the strands).
__global__ void __launch_bounds__(256)
prep_weight_kernel(const float* __restrict__ partial, int blocks, int d, float* __restrict__ dwq, float* __restrict__ dwk) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < 2 * d)
        for (int b = strand; b < blocks; b += 8) sum += partial[(size_t)b * 2 * d + c];
    red[strand][lane] = sum;
    __syncthreads();
    if (strand == 0 && c < 2 * d) {
        float s = 0.f;
        for (int i = 0; i < 8; ++i) s += red[i][lane];
        float* out = c < d ? dwq : dwk;
        if (out) out[c < d ? c : c - d] = s;
    }
}

}  // namespace gated
}  // namespace ckda
