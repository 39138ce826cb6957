// Chunked gated delta rule, part 1: what a 64-token chunk holds before any state is known, all
// chunks side by side. With G the in-chunk cumulated log gate and D_ij = e^{G_i - G_j}:
//   P = tril(D (.) Q K^T),   A = tril(D (.) K K^T, -1),   Z = -(I + A diag(beta))^{-1} A
// Z serves both passes: W = X + Z (beta X) solves the chunk's triangular system forward, and
// y = dU + Z^T (beta dU) its adjoint, without a division by beta.
//
// One CTA of four warps per (chunk, key head); the value heads that share the key head reuse
// the raw products. G is summed in fp64 and kept as hi + lo, so that differences of far-down
// sums stay exact to fp32. The solve: 16 x 16 diagonal blocks by substitution (a thread per
// column), then the blocks below level by level,
//   R = A_IJ + sum_M (A beta)_IM Z_MJ,   Z_IJ = -(R + Z_II beta_I R),
// a warp per block, on tf32 products in three passes (operands to 2^-21).
#pragma once
#include "gated_mma.cuh"

namespace ckda {
namespace gated {

constexpr int LDF = 68;                        // floats in a row of the fp32 matrices

__host__ __device__ constexpr size_t intra_region(int DK) {
    return (size_t)(2 * 64 * ld_bytes(DK)) > (size_t)(2 * 64 * LDF * 4) ? (size_t)(2 * 64 * ld_bytes(DK)) : (size_t)(2 * 64 * LDF * 4);
}
__host__ __device__ constexpr size_t intra_smem(int DK) {
    return intra_region(DK) + 2 * 64 * LD64 + 64 * 4 * 4;
}

// acc += X Y for 16 x 16 fp32 blocks in shared memory (rows of LDF floats), Y's rows times sc if
// given, both split into tf32 high and remainder.
template <bool kScale>
__device__ __forceinline__ void block_product(float (&acc)[2][4], const float* X, const float* Y, const float* sc) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    auto high = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); };
#pragma unroll
    for (int ks = 0; ks < 16; ks += 8) {
        float a[4] = {X[g * LDF + ks + t], X[(g + 8) * LDF + ks + t], X[g * LDF + ks + t + 4], X[(g + 8) * LDF + ks + t + 4]};
        float ah[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ah[i] = high(a[i]);
            al[i] = a[i] - ah[i];
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float b[2] = {Y[(ks + t) * LDF + 8 * n + g], Y[(ks + t + 4) * LDF + 8 * n + g]};
            if constexpr (kScale) {
                b[0] *= sc[ks + t];
                b[1] *= sc[ks + t + 4];
            }
            float bh[2], bl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                bh[i] = high(b[i]);
                bl[i] = b[i] - bh[i];
            }
            mma_tf32(acc[n], ah, bl);
            mma_tf32(acc[n], al, bh);
            mma_tf32(acc[n], ah, bh);
        }
    }
}

template <int DK>
__global__ void __launch_bounds__(128, 4)
intra_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k, const float* __restrict__ g,
             const float* __restrict__ beta, ChunkWs ws, Seqs seqs, int Hk, int Hv, int dk, long long qs, long long ks) {
    extern __shared__ __align__(16) unsigned char sm[];
    const int slot = blockIdx.x, hk = blockIdx.y, rep = Hv / Hk, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = seqs.find(slot);
    int start, len;
    bool ok;
    seqs.get(n, start, len, ok);
    const int c = slot - seqs.first_slot(n, start);
    if (c < 0 || (long long)c * C >= len) return;
    const int nt = min(C, len - c * C);
    const size_t tok0 = (size_t)start + (size_t)c * C;
    const uint32_t sk = s32(sm), sq = sk + 64 * ld_bytes(DK);
    float* sa = reinterpret_cast<float*>(sm);                          // over K and Q once those are used
    float* sz = sa + 64 * LDF;
    unsigned char* sp = sm + intra_region(DK);                         // P terms, padded bf16 rows
    float* sv = reinterpret_cast<float*>(sp + 2 * 64 * LD64);   // G hi, G lo, beta
    load_rows<DK, 128>(sk, k + tok0 * ks + (size_t)hk * dk, ks, nt, dk);
    load_rows<DK, 128>(sq, q + tok0 * qs + (size_t)hk * dk, qs, nt, dk);
    cp_commit();
    float gn[2] = {0.f, 0.f}, bn[2] = {0.f, 0.f};                      // warp 0: the next head's gates, in flight
    auto gates = [&](int h) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * lane + i < nt) {
                gn[i] = g[(tok0 + 2 * lane + i) * Hv + h];
                bn[i] = beta[(tok0 + 2 * lane + i) * Hv + h];
            }
    };
    if (warp == 0) gates(hk * rep);
    cp_wait<0>();
    __syncthreads();
    // rows 16 warp .. + 15 of K K^T and Q K^T, columns up to the diagonal block
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = 0.f;
#pragma unroll
    for (int d = 0; d < DK; d += 16) {
        uint32_t ak[4], aq[4];
        ldm4(ak, sk + ofs_a(ld_bytes(DK)) + at(16 * warp, d, ld_bytes(DK)));
        ldm4(aq, sq + ofs_a(ld_bytes(DK)) + at(16 * warp, d, ld_bytes(DK)));
#pragma unroll
        for (int jp = 0; jp < 4; ++jp)
            if (jp <= warp) {
                uint32_t b[4];
                ldm4(b, sk + ofs_n(ld_bytes(DK)) + at(16 * jp, d, ld_bytes(DK)));
                mma(kk[2 * jp], ak, b[0], b[1]);
                mma(kk[2 * jp + 1], ak, b[2], b[3]);
                mma(qk[2 * jp], aq, b[0], b[1]);
                mma(qk[2 * jp + 1], aq, b[2], b[3]);
            }
    }
    const int gi = lane >> 2, t2 = 2 * (lane & 3);
    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        const size_t wh = (size_t)slot * Hv + h;
        __syncthreads();                                               // K, Q (or the head before) are done with
        if (warp == 0) {
            const double x[2] = {(double)gate_in(gn[0]), (double)gate_in(gn[1])};
            const float bt[2] = {bn[0], bn[1]};
            if (r + 1 < rep) gates(h + 1);
            double sum = x[0] + x[1];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += y;
            }
            const double end = __shfl_sync(0xffffffffu, sum, 31);
            const double G[2] = {sum - x[1], sum};
            float* out = ws.vec + wh * VEC;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tt = 2 * lane + i;
                const float hi = (float)G[i], lo = (float)(G[i] - (double)hi);
                sv[tt] = hi;
                sv[64 + tt] = lo;
                sv[128 + tt] = bt[i];
                const float rest = (float)(end - G[i]), rlo = (float)(end - G[i] - (double)rest), e = expf(hi), f = expf(rest);
                out[VEC_EG + tt] = fmaf(e, lo, e);                 // e^(hi + lo)
                out[VEC_DEC + tt] = fmaf(f, rlo, f);
                out[VEC_BETA + tt] = bt[i];
                out[VEC_GHI + tt] = hi;
                out[VEC_GLO + tt] = lo;
            }
        }
        __syncthreads();
        // P to its staging tile, A beta to sa, A to sz, where Z takes its place
#pragma unroll
        for (int nn = 0; nn < 8; ++nn) {
            if (nn / 2 > warp) continue;
            const float ghj[2] = {sv[8 * nn + t2], sv[8 * nn + t2 + 1]}, glj[2] = {sv[64 + 8 * nn + t2], sv[64 + 8 * nn + t2 + 1]};
            const float bj[2] = {sv[128 + 8 * nn + t2], sv[128 + 8 * nn + t2 + 1]};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = 16 * warp + gi + 8 * half;
                const float ghi = sv[i], gli = sv[64 + i];
                float p[2], a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 8 * nn + t2 + e;
                    const float d = j <= i ? expf((ghi - ghj[e]) + (gli - glj[e])) : 0.f;
                    p[e] = j <= i ? d * qk[nn][2 * half + e] : 0.f;
                    a[e] = j < i ? d * kk[nn][2 * half + e] : 0.f;
                }
                uint32_t hi, lo;
                split2(p[0], p[1], hi, lo);
                *reinterpret_cast<uint32_t*>(sp + i * LD64 + (8 * nn + t2) * 2) = hi;
                *reinterpret_cast<uint32_t*>(sp + 64 * LD64 + i * LD64 + (8 * nn + t2) * 2) = lo;
                *reinterpret_cast<float2*>(sa + i * LDF + 8 * nn + t2) = make_float2(a[0] * bj[0], a[1] * bj[1]);
                *reinterpret_cast<float2*>(sz + i * LDF + 8 * nn + t2) = make_float2(a[0], a[1]);
            }
        }
        __syncthreads();
        if (tid < 64) {                                                // diagonal blocks: a thread per column
            const int b0 = tid & 48, j = tid & 15;
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float u = sz[(b0 + i) * LDF + b0 + j], v = 0.f;
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(sa + (b0 + i) * LDF + b0 + m);
                    u = fmaf(a.x, z[m], u);
                    if (m + 1 < i) v = fmaf(a.y, z[m + 1], v);
                    if (m + 2 < i) u = fmaf(a.z, z[m + 2], u);
                    if (m + 3 < i) v = fmaf(a.w, z[m + 3], v);
                }
                z[i] = i > j ? -(u + v) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) sz[(b0 + i) * LDF + b0 + j] = z[i];
        } else {                                                       // meanwhile: P to the workspace
            for (int e = tid - 64; e < 1024; e += 64) {
                const int term = e / 512, rr = (e % 512) / 8, p = e % 8;
                if (p / 2 <= rr / 16)
                    *reinterpret_cast<uint4*>((term ? ws.plo : ws.phi) + wh * 4096 + rr * 64 + p * 8) =
                        *reinterpret_cast<const uint4*>(sp + term * 64 * LD64 + rr * LD64 + p * 16);
            }
        }
        __syncthreads();
#pragma unroll
        for (int level = 1; level < 4; ++level) {
            if (warp < 4 - level) {
                const int J = warp, I = warp + level;
                float acc[2][4];
                float* dst = sz + 16 * I * LDF + 16 * J;
                auto frag = [&](float (&x)[2][4], const float* m) {
#pragma unroll
                    for (int nn = 0; nn < 2; ++nn) {
                        const float2 u = *reinterpret_cast<const float2*>(m + gi * LDF + 8 * nn + t2);
                        const float2 v = *reinterpret_cast<const float2*>(m + (gi + 8) * LDF + 8 * nn + t2);
                        x[nn][0] = u.x; x[nn][1] = u.y; x[nn][2] = v.x; x[nn][3] = v.y;
                    }
                };
                auto put = [&](float sign) {
#pragma unroll
                    for (int nn = 0; nn < 2; ++nn) {
                        *reinterpret_cast<float2*>(dst + gi * LDF + 8 * nn + t2) = make_float2(sign * acc[nn][0], sign * acc[nn][1]);
                        *reinterpret_cast<float2*>(dst + (gi + 8) * LDF + 8 * nn + t2) = make_float2(sign * acc[nn][2], sign * acc[nn][3]);
                    }
                };
                frag(acc, dst);
#pragma unroll
                for (int m = 0; m < level; ++m)
                    block_product<false>(acc, sa + 16 * I * LDF + 16 * (J + m), sz + 16 * (J + m) * LDF + 16 * J, nullptr);
                put(1.f);
                __syncwarp();
                block_product<true>(acc, sz + 16 * I * LDF + 16 * I, dst, sv + 128 + 16 * I);
                __syncwarp();
                put(-1.f);
            }
            __syncthreads();
        }
        for (int e = tid; e < 512; e += 128) {                         // Z to the workspace in two terms
            const int rr = e / 8, p = e % 8;
            if (p / 2 > rr / 16) continue;
            const float* z = sz + rr * LDF + p * 8;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split2(z[2 * i], z[2 * i + 1], hi[i], lo[i]);
            *reinterpret_cast<uint4*>(ws.zhi + wh * 4096 + rr * 64 + p * 8) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(ws.zlo + wh * 4096 + rr * 64 + p * 8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

}  // namespace gated
}  // namespace ckda
