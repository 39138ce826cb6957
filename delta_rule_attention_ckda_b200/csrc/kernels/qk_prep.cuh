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
// a million turns an fp32 angle by 0.06 rad), once per token and pair.
//
// Vector path: a warp takes a token (several warps where tokens are few), G lanes a head row, 16
// bytes each, UR rows in work and UR more on their way. Blocks stay for all their tokens, so
// loads also run under the next token's angles. What a lane does to a channel is the same for
// every head of the token, out = r (x A + x' B) with x' the pair's other channel (from a lane
// R/16 away, or the neighbour in the same register), so weight, cosine, sine and scale are folded
// into A and B once per token. Warps share nothing and meet at no barrier. Rows of other sizes or
// distances take the scalar path, one warp per row through a row buffer (tensors start on 16 bytes for
// either path): 32768 tokens of 16 + 16 heads of 100 channels take 440 us, backward 950, in either type
// (14 to 29% of the copy bandwidth, backward 10 to 20%).
//
// Measured: 32768 tokens of 16 + 16 heads of 128, 537 MB: 107 us, 77% of the copy bandwidth (without
// the rows on their way 8% slower; with 4 blocks an SM, which spill, 18%; the pair layout chosen
// in the kernel instead of by instance 10%: the issue slots are 70% busy). Backward, 16383 tokens
// of 16 + 8 heads, 302 MB: 76 us and 4 for the weights' sums, 61%; two row loads of 16 bytes a
// lane for each of x and dy in work and as many on their way fill the registers of two blocks an
// SM (with three or with four rows they spill: 33% and 8% slower).
#pragma once
#include "gated_mma.cuh"

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
    float eps, inv_d, q_scale, rope_scale;
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

// r, and the coefficient c of the gradient's projection (0 where the norm is at its floor).
__device__ __forceinline__ float norm_factor(const PrepArgs& a, float ss, float& coef) {
    if (a.norm == kNormL2) {
        const bool above = ss > 1e-24f;
        coef = above ? 1.f : 0.f;
        return above ? rsqrtf(ss) : 1e12f;
    }
    if (a.norm == kNormRms) {
        coef = a.inv_d;
        return rsqrtf(fmaf(ss, a.inv_d, a.eps));
    }
    coef = 0.f;
    return 1.f;
}

// 8 channels of a row as loaded.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint32_t r[4];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
    }
    __device__ __forceinline__ void zero() { r[0] = r[1] = r[2] = r[3] = 0u; }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = lo_of(r[i]);
            x[2 * i + 1] = hi_of(r[i]);
        }
    }
    __device__ __forceinline__ Raw8 swapped() const {
        Raw8 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o.r[i] = __byte_perm(r[i], r[i], 0x1032);
        return o;
    }
    __device__ __forceinline__ Raw8 from_lane(int lane, bool use) const {
        Raw8 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.r[i] = __shfl_sync(0xffffffffu, r[i], lane);
            if (!use) o.r[i] = 0u;
        }
        return o;
    }
    __device__ static __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    }
};
template <> struct Raw8<float> {
    float r[8];
    __device__ __forceinline__ void load(const float* p) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w; r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = 0.f;
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = r[i];
    }
    __device__ __forceinline__ Raw8 swapped() const {
        Raw8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o.r[i] = r[i ^ 1];
        return o;
    }
    __device__ __forceinline__ Raw8 from_lane(int lane, bool use) const {
        Raw8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o.r[i] = __shfl_sync(0xffffffffu, r[i], lane);
            if (!use) o.r[i] = 0.f;
        }
        return o;
    }
    __device__ static __forceinline__ void store(float* p, const float (&x)[8]) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Vector path: d a multiple of 8, rows 16-byte aligned, R a multiple of 16 (half) or 8 (interleaved).
// `wpt` warps share a token's heads.
template <typename TIn, int G, int UR, bool kBack, bool kInter>
__global__ void __launch_bounds__(256, kBack ? 2 : 3)
prep_vec_kernel(const PrepArgs a, int wpt) {
    extern __shared__ __align__(16) float smf[];
    constexpr int GP = 32 / G;                                  // rows a warp takes at once
    const int half = a.rotary / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G, e0 = 8 * l;
    float2* cs = reinterpret_cast<float2*>(smf) + warp * half;
    const bool live = e0 < a.d, in = e0 < a.rotary, first = kInter || e0 < half;
    const int other = in && !kInter ? (first ? lane + half / 8 : lane - half / 8) : lane;
    const int eo = in && !kInter ? (first ? e0 + half : e0 - half) : e0;      // the partners' channels
    const int p0 = kInter ? e0 / 2 : (first ? e0 : e0 - half);
    float acc[2][8];
    if constexpr (kBack) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
    }
    const int per = 8 / wpt, step = wpt * GP * UR, h0 = (warp % wpt) * GP;      // tokens a block takes at once; heads a warp does
    // Rows on their way: batches of UR rows a lane group, over heads, then keys, then the next token.
    struct Batch {
        Raw8<TIn> x[UR], d[kBack ? UR : 1];
    };
    auto fetch = [&](Batch& b, long long t, int which, int hb) {
        const int h = hb + lane / G, hop = wpt * GP * a.d, left = live && t < a.tokens ? a.heads[which] - h : 0;
        const TIn* xp = static_cast<const TIn*>(a.x[which]) + t * a.stride[which] + (long long)h * a.d + e0;
        const TIn* dp = kBack ? static_cast<const TIn*>(a.dy[which]) + (t * a.heads[which] + h) * a.d + e0 : nullptr;
#pragma unroll
        for (int j = 0; j < UR; ++j) {
            b.x[j].zero();
            if (j * wpt * GP < left) b.x[j].load(xp + j * hop);
            if constexpr (kBack) {
                b.d[j].zero();
                if (j * wpt * GP < left) b.d[j].load(dp + j * hop);
            }
        }
    };
    Batch now, next;
    const long long t0 = (long long)blockIdx.x * per + warp / wpt, hop = (long long)gridDim.x * per;
    const int q0 = h0 < a.heads[0] ? 0 : 1;
    fetch(now, t0, q0, h0);
    for (long long t = t0; t < a.tokens; t += hop) {
        if (half) {
            __syncwarp();
            for (int p = lane; p < half; p += 32) cs[p] = turn(a, (int)t, p);
            __syncwarp();
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (h0 >= a.heads[which]) continue;
            const float scale = which ? 1.f : a.q_scale;
            const float* w = a.w[which];
            TIn* op = static_cast<TIn*>(a.out[which]) + t * a.heads[which] * a.d + e0;
            // forward: A, B with the weights of the channel and of its partner; backward: of dy, without
            float A[8], B[8], wt[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float we = w && live ? __ldg(w + e0 + i) : 1.f;
                const float wo = kBack ? 1.f : (w && live ? __ldg(w + (kInter ? (e0 + i) ^ 1 : eo + i)) : 1.f);
                const float own = kBack ? scale : we * scale;
                A[i] = own;
                B[i] = 0.f;
                if constexpr (kBack) wt[i] = we;
                if (in) {
                    const float2 c = cs[kInter ? p0 + i / 2 : p0 + i];
                    const bool plus = kInter ? (i & 1) : !first;              // the sine's sign, turned back in reverse
                    A[i] = own * c.x;
                    B[i] = wo * scale * (plus != kBack ? c.y : -c.y);
                }
            }
#pragma unroll 1
            for (int hb = h0; hb < a.heads[which]; hb += step) {
                if (hb + step < a.heads[which]) fetch(next, t, which, hb + step);
                else if (which == 0 && h0 < a.heads[1]) fetch(next, t, 1, h0);
                else fetch(next, t + hop, q0, h0);
#pragma unroll
                for (int j = 0; j < UR; ++j) {
                    if (hb + j * wpt * GP >= a.heads[which]) break;                  // the warp's rows are done
                    const int h = hb + j * wpt * GP + lane / G;
                    float x[8], y[8];
                    now.x[j].unpack(x);
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; i += 2) fma2(s0, s1, x[i], x[i + 1], x[i], x[i + 1]);
                    float coef;
                    float f = norm_factor(a, group_sum<G>(s0 + s1), coef);
                    // lanes behind the last head hold zeros, whose RMS factor without eps is infinite: their 0 f
                    // would be a NaN in the weights' sums
                    if (kBack && h >= a.heads[which]) f = 0.f;
                    const Raw8<TIn>& turned = kBack ? now.d[kBack ? j : 0] : now.x[j];
                    (kInter ? turned.swapped() : turned.from_lane(other, in)).unpack(y);
                    if (kInter && !in) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = 0.f;
                    }
                    if constexpr (!kBack) {
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            mul2(x[i], x[i + 1], A[i], A[i + 1]);
                            fma2(x[i], x[i + 1], y[i], y[i + 1], B[i], B[i + 1]);
                            mul2(x[i], x[i + 1], f, f);
                        }
                    } else {
                        float z[8], d0 = 0.f, d1 = 0.f;
                        now.d[j].unpack(z);
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            mul2(z[i], z[i + 1], A[i], A[i + 1]);
                            fma2(z[i], z[i + 1], y[i], y[i + 1], B[i], B[i + 1]);
                            mul2(x[i], x[i + 1], f, f);                              // xh
                            fma2(acc[which][i], acc[which][i + 1], z[i], z[i + 1], x[i], x[i + 1]);
                            mul2(z[i], z[i + 1], wt[i], wt[i + 1]);
                            fma2(d0, d1, z[i], z[i + 1], x[i], x[i + 1]);
                        }
                        const float c = -coef * group_sum<G>(d0 + d1);
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            fma2(z[i], z[i + 1], x[i], x[i + 1], c, c);
                            x[i] = z[i];
                            x[i + 1] = z[i + 1];
                            mul2(x[i], x[i + 1], f, f);
                        }
                    }
                    if (live && h < a.heads[which]) Raw8<TIn>::store(op + (long long)h * a.d, x);
                }
                now = next;
            }
        }
    }
    if constexpr (kBack) {
        if (a.partial == nullptr) return;
        constexpr int GROUPS = 8 * GP;
        float* red = smf;                                       // [GROUPS][d], over the angles
#pragma unroll
        for (int s = 0; s < 2; ++s) {                           // groups in turn: one order of the sum
            __syncthreads();
            if (live)
#pragma unroll
                for (int i = 0; i < 8; ++i) red[(threadIdx.x / G) * a.d + e0 + i] = acc[s][i];
            __syncthreads();
            for (int c = threadIdx.x; c < a.d; c += 256) {
                float sum = 0.f;
                for (int gi = 0; gi < GROUPS; ++gi) sum += red[gi * a.d + c];
                a.partial[((size_t)blockIdx.x * 2 + s) * a.d + c] = sum;
            }
        }
    }
}

// Scalar path: one warp per row, d <= 256, any even R, any distance between tokens.
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
    for (long long t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        __syncthreads();
        for (int p = threadIdx.x; p < half; p += 256) cs[p] = turn(a, (int)t, p);
        __syncthreads();
        for (int h = warp; h < H; h += 8) {
            const int which = h >= a.heads[0], hh = which ? h - a.heads[0] : h;
            const TIn* xp = static_cast<const TIn*>(a.x[which]) + t * a.stride[which] + (long long)hh * a.d;
            const long long row = (t * a.heads[which] + hh) * a.d;
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
// block of 1024 threads per 32 columns: 32 strands of blocks, each with its loads in flight, then
// the strands.
__global__ void __launch_bounds__(1024)
prep_weight_kernel(const float* __restrict__ partial, int blocks, int d, float* __restrict__ dwq, float* __restrict__ dwk) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < 2 * d) {
#pragma unroll 8
        for (int b = strand; b < blocks; b += 32) sum += partial[(size_t)b * 2 * d + c];
    }
    red[strand][lane] = sum;
    __syncthreads();
    if (strand == 0 && c < 2 * d) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += red[i][lane];
        float* out = c < d ? dwq : dwk;
        if (out) out[c < d ? c : c - d] = s;
    }
}

}  // namespace gated
}  // namespace ckda
