// Chunked gated delta rule, part 1: what a 64-token chunk holds before any state is known, all
// chunks side by side. With G the in-chunk cumulated log gate and D_ij = e^{G_i - G_j}:
//   P = tril(D (.) Q K^T),   A = tril(D (.) K K^T, -1),   Z = -(I + A diag(beta))^{-1} A
// For the backward pass (kApart) P's diagonal lies in a vector of its own and P holds zeros there.
// Z serves both passes: W = X + Z (beta X) solves the chunk's triangular system forward, and
// y = dU + Z^T (beta dU) its adjoint, without a division by beta.
//
// One CTA of four warps per (chunk, key head); the value heads that share the key head reuse
// the raw products. G is summed in fp64 while the tiles load and kept as hi + lo, so that
// differences of far-down sums stay exact to fp32. The solve: 16 x 16 diagonal blocks by
// substitution (a thread per column: each value found updates the sums below it, so the chain is
// one fused multiply-add a row), then the blocks below them doubling, 16 and then 32 wide,
//   R = A_IJ + sum_M (A beta)_IM Z_MJ,   Z_IJ = -(R_IJ + sum_M Z_IM beta_M R_MJ),
// on tf32 products in three passes (operands to 2^-21).
//
// Measured, 8192 chunks of 128 channels (436 MB): 158 us, 42% of the copy bandwidth (164 with P's diagonal
// apart). Phases between block barriers with few products each: the issue slots are 37% busy, shared memory 51%. Four
// CTAs an SM by registers and shared memory; with P stored straight from registers five fit,
// which is no faster, nor is the substitution on four warps in place of two. With row copies instead of tensor copies and three doubling levels: 182 us.
#pragma once
#include "gated_mma.cuh"

namespace ckda {
namespace gated {

constexpr int LDF = 68;                        // floats in a row of the fp32 matrices

__host__ __device__ constexpr size_t intra_region(int DK) {
    return (size_t)(2 * 64 * 2 * DK) > (size_t)(2 * 64 * LDF * 4) ? (size_t)(2 * 64 * 2 * DK) : (size_t)(2 * 64 * LDF * 4);
}
__host__ __device__ constexpr size_t intra_smem(int DK) {
    return intra_region(DK) + 2 * 64 * LD64 + 64 * 4 * 4 + 1024;
}

// acc += X Y for 16 x 16 fp32 blocks in shared memory (rows of LDF and LDY floats), Y's rows times
// sc if given, both split into tf32 high and remainder.
template <bool kScale, int LDY>
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
            float b[2] = {Y[(ks + t) * LDY + 8 * n + g], Y[(ks + t + 4) * LDY + 8 * n + g]};
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

template <int DK, bool kApart>
__global__ void __launch_bounds__(128, 4)
intra_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const ChainIn in,
             const float* __restrict__ g, const float* __restrict__ beta, ChunkWs ws, Seqs seqs, int Hk, int Hv, int dk) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full;
    next_may_start();
    const int slot = blockIdx.x, hk = blockIdx.y, rep = Hv / Hk, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = seqs.find(slot);
    int start, len;
    bool ok;
    if (slot == 0 && hk == 0 && seqs.cu != nullptr)                    // every sequence's offsets: out of order, find() may not meet them all
        for (int m = tid; m < seqs.N; m += 128) {
            seqs.get(m, start, len, ok);
            if (!ok) report_index_error();
        }
    seqs.get(n, start, len, ok);
    const int c = slot - seqs.first_slot(n, start);
    if (c < 0 || (long long)c * C >= len) return;
    const int nt = min(C, len - c * C);
    const size_t tok0 = (size_t)start + (size_t)c * C;
    const uint32_t sk = s32(sm), sq = sk + 64 * 2 * DK;
    float* sa = reinterpret_cast<float*>(sm);                          // over K and Q once those are used
    float* sz = sa + 64 * LDF;
    unsigned char* sp = sm + intra_region(DK);                         // P terms, padded bf16 rows
    float* sr = sa + 32;                                               // R: the blocks of sa right of the diagonal, which hold nothing
    float* sv = reinterpret_cast<float*>(sp + 2 * 64 * LD64);          // G hi, G lo, beta
    const bool tiles = in.maps && nt == C;
    if (tid == 0) {
        tc::mbar_init(&full, 1);
        tc::fence_mbar_init();
        if (tiles) {
            tc::mbar_arrive_expect_tx(&full, 2 * 64 * 2 * DK);
#pragma unroll
            for (int x = 0; x < DK / 64; ++x) {
                tma_rows(sk + x * 8192, &mk, &full, 64 * x, hk, (int)tok0);
                tma_rows(sq + x * 8192, &mq, &full, 64 * x, hk, (int)tok0);
            }
        }
    }
    if (!tiles) {
        tile_rows<128>(sk, in.k + tok0 * in.ks + (size_t)hk * dk, in.ks, nt, dk, DK, tid);
        tile_rows<128>(sq, in.q + tok0 * in.qs + (size_t)hk * dk, in.qs, nt, dk, DK, tid);
        cp_commit();
    }
    // warp 0: a head's gates to sv and the workspace (the first head's while the tiles load)
    float gn[2] = {0.f, 0.f}, bn[2] = {0.f, 0.f};
    auto gates = [&](int h) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * lane + i < nt) {
                gn[i] = g[(tok0 + 2 * lane + i) * Hv + h];
                bn[i] = beta[(tok0 + 2 * lane + i) * Hv + h];
            }
    };
    auto sums = [&](int h) {
        const double x[2] = {(double)gate_in(gn[0]), (double)gate_in(gn[1])};
        double sum = x[0] + x[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += y;
        }
        const double end = __shfl_sync(0xffffffffu, sum, 31);
        const double G[2] = {sum - x[1], sum};
        float* out = ws.vec + ((size_t)slot * Hv + h) * VEC;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tt = 2 * lane + i;
            const float hi = (float)G[i], lo = (float)(G[i] - (double)hi);
            const float rest = (float)(end - G[i]), rlo = (float)(end - G[i] - (double)rest), e = expf(hi), f = expf(rest);
            sv[tt] = hi;
            sv[64 + tt] = lo;
            sv[128 + tt] = bn[i];
            out[VEC_EG + tt] = fmaf(e, lo, e);                         // e^(hi + lo)
            out[VEC_DEC + tt] = fmaf(f, rlo, f);
            out[VEC_BETA + tt] = bn[i];
            out[VEC_GHI + tt] = hi;
            out[VEC_GLO + tt] = lo;
        }
    };
    if (warp == 0) {
        gates(hk * rep);
        sums(hk * rep);
        if (rep > 1) gates(hk * rep + 1);
    }
    __syncthreads();                                                   // the barrier is set up
    if (tiles) tc::mbar_wait(&full, 0);
    else cp_wait<0>();
    __syncthreads();
    // rows 16 warp .. + 15 of K K^T and Q K^T, columns up to the diagonal block
    const uint32_t ln = swz_lane(true), lk = swz_lane(false);          // as ofs_n, as ofs_a
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = 0.f;
#pragma unroll
    for (int d = 0; d < DK; d += 16) {
        uint32_t ak[4], aq[4];
        ldm4(ak, sk + frag(lk, 16 * warp, d));
        ldm4(aq, sq + frag(lk, 16 * warp, d));
#pragma unroll
        for (int jp = 0; jp < 4; ++jp)
            if (jp <= warp) {
                uint32_t b[4];
                ldm4(b, sk + frag(ln, 16 * jp, d));
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
        if (r > 0) {
            if (warp == 0) {
                sums(h);
                if (r + 1 < rep) gates(h + 1);
            }
            __syncthreads();
        }
        // P to its staging tile, A beta to sa (diagonal blocks transposed), A to sz, where Z takes its place
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
                    if (kApart && nn / 2 == warp && j == i) {                             // the backward pass takes the diagonal by itself
                        ws.vec[wh * VEC + VEC_PD + i] = p[e];
                        p[e] = 0.f;
                    }
                }
                uint32_t hi, lo;
                split2(p[0], p[1], hi, lo);
                *reinterpret_cast<uint32_t*>(sp + i * LD64 + (8 * nn + t2) * 2) = hi;
                *reinterpret_cast<uint32_t*>(sp + 64 * LD64 + i * LD64 + (8 * nn + t2) * 2) = lo;
                if (nn / 2 == warp) {
                    sa[(8 * nn + t2) * LDF + i] = a[0] * bj[0];
                    sa[(8 * nn + t2 + 1) * LDF + i] = a[1] * bj[1];
                } else {
                    *reinterpret_cast<float2*>(sa + i * LDF + 8 * nn + t2) = make_float2(a[0] * bj[0], a[1] * bj[1]);
                }
                *reinterpret_cast<float2*>(sz + i * LDF + 8 * nn + t2) = make_float2(a[0], a[1]);
            }
        }
        __syncthreads();
        if (tid < 64) {                                                // diagonal blocks: a thread per column
            const int b0 = tid & 48, j = tid & 15;
            float z[16];                                               // minus the sums so far, then Z
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = -sz[(b0 + i) * LDF + b0 + j];
#pragma unroll
            for (int m = 0; m < 15; ++m) {
#pragma unroll
                for (int i = m / 4 * 4; i < 16; i += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(sa + (b0 + m) * LDF + b0 + i);
                    if (i > m) z[i] = fmaf(-a.x, z[m], z[i]);
                    if (i + 1 > m) z[i + 1] = fmaf(-a.y, z[m], z[i + 1]);
                    if (i + 2 > m) z[i + 2] = fmaf(-a.z, z[m], z[i + 2]);
                    if (i + 3 > m) z[i + 3] = fmaf(-a.w, z[m], z[i + 3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) sz[(b0 + i) * LDF + b0 + j] = z[i];
        }
        __syncthreads();
        auto get = [&](float (&x)[2][4], const float* m, int ld) {
#pragma unroll
            for (int nn = 0; nn < 2; ++nn) {
                const float2 u = *reinterpret_cast<const float2*>(m + gi * ld + 8 * nn + t2);
                const float2 v = *reinterpret_cast<const float2*>(m + (gi + 8) * ld + 8 * nn + t2);
                x[nn][0] = u.x; x[nn][1] = u.y; x[nn][2] = v.x; x[nn][3] = v.y;
            }
        };
        auto put = [&](const float (&x)[2][4], float* m, int ld, float sign) {
#pragma unroll
            for (int nn = 0; nn < 2; ++nn) {
                *reinterpret_cast<float2*>(m + gi * ld + 8 * nn + t2) = make_float2(sign * x[nn][0], sign * x[nn][1]);
                *reinterpret_cast<float2*>(m + (gi + 8) * ld + 8 * nn + t2) = make_float2(sign * x[nn][2], sign * x[nn][3]);
            }
        };
        auto zb = [&](int I, int J) { return sz + 16 * I * LDF + 16 * J; };
        auto ab = [&](int I, int J) { return sa + 16 * I * LDF + 16 * J; };
        const float* bt = sv + 128;
        float acc[2][4];
        if (warp < 2) {                                                // blocks (1, 0) and (3, 2)
            const int J = 2 * warp, I = J + 1;
            get(acc, zb(I, J), LDF);
            block_product<false, LDF>(acc, ab(I, J), zb(J, J), nullptr);
            put(acc, zb(I, J), LDF, 1.f);
            __syncwarp();
            block_product<true, LDF>(acc, zb(I, I), zb(I, J), bt + 16 * I);
            __syncwarp();
            put(acc, zb(I, J), LDF, -1.f);
        }
        __syncthreads();
        const int I = 2 + (warp >> 1), J = warp & 1;                   // the 32 x 32 block below: a warp a quarter
        get(acc, zb(I, J), LDF);
        block_product<false, LDF>(acc, ab(I, 1), zb(1, J), nullptr);
        if (J == 0) block_product<false, LDF>(acc, ab(I, 0), zb(0, 0), nullptr);
        put(acc, sr + 16 * (I - 2) * LDF + 16 * J, LDF, 1.f);
        __syncthreads();
        block_product<true, LDF>(acc, zb(I, 2), sr + 16 * J, bt + 32);
        if (I == 3) block_product<true, LDF>(acc, zb(3, 3), sr + 16 * LDF + 16 * J, bt + 48);
        put(acc, zb(I, J), LDF, -1.f);
        __syncthreads();
        // P and Z to the workspace, the blocks on and below the diagonal; Z in two terms
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + 128 * i, rr = e / 8, p = e % 8;
            if (p / 2 > rr / 16) continue;
            const size_t to = wh * 4096 + rr * 64 + p * 8;
            *reinterpret_cast<uint4*>(ws.phi + to) = *reinterpret_cast<const uint4*>(sp + rr * LD64 + p * 16);
            *reinterpret_cast<uint4*>(ws.plo + to) = *reinterpret_cast<const uint4*>(sp + (64 + rr) * LD64 + p * 16);
            const float4 x = *reinterpret_cast<const float4*>(sz + rr * LDF + p * 8), y = *reinterpret_cast<const float4*>(sz + rr * LDF + p * 8 + 4);
            uint32_t hi[4], lo[4];
            split2(x.x, x.y, hi[0], lo[0]);
            split2(x.z, x.w, hi[1], lo[1]);
            split2(y.x, y.y, hi[2], lo[2]);
            split2(y.z, y.w, hi[3], lo[3]);
            *reinterpret_cast<uint4*>(ws.zhi + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(ws.zlo + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

}  // namespace gated
}  // namespace ckda
