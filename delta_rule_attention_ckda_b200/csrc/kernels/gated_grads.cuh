// Chunked gated delta rule, part 3: the gradients of q, k, g and beta, all chunks side by side,
// from what the two chains left (S the entering state, dS the cotangent of the leaving one,
// U, dV, and sums per token):
//   Dw = tril(D (.) dO U^T),   Da = -tril(D (.) dV U^T, -1)
//   dQ = e^G (.) dO S^T + Dw K
//   dK = -e^G (.) dV S^T + e^{G_C - G} (.) U dS^T + Dw^T Q + Da K + Da^T K
//   dbeta_t = <w_t, y_t>,   dg_t = sum_{i >= t} e_i + <S_C, dS_C>,   e_i = <dO_i, o_i> - <dV_i, v_i>
// dg: scaling the state of one moment scales what every later term takes of it, so the later
// terms' own products with their cotangents sum to the derivative by the log gate. The same
// number counted from the chunk's start is <S_0, dS_0> - sum_{i < t} e_i; each e_i is off by its
// products' rounding, so the two are weighted by the other's number of terms, (n - t) and t of n,
// which cuts the error of the sum to a half of the one-sided one (1.04e-5 to 6e-6 of dg's norm).
//
// dQ and dK are rounded to bf16 at the end, so their operands go in one bf16 term; dg and
// dbeta come from the chains' fp32 sums. One CTA of four warps per (chunk, key head, 64
// channels of d_k), two CTAs an SM so that one's loads run under the other's products; a warp
// owns 16 tokens. Value heads that share the key head are summed in the accumulators, in
// head order.
#pragma once
#include "gated_mma.cuh"

namespace ckda {
namespace gated {

template <int DV>
struct GradSmem {
    static constexpr int LDV = ld_bytes(DV);
    static constexpr int DO = 0, U = DO + 64 * LDV, DVV = U + 64 * LDV, S = DVV + 64 * LDV, DS = S + DV * LD64,
                         K = DS + DV * LD64, Q = K + 64 * LD64, VECS = Q + 64 * LD64, BYTES = VECS + VEC * 4;
};

template <int DV>
__global__ void __launch_bounds__(128, 2)
grad_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ grad_o,
            const __nv_bfloat16* __restrict__ grad_v, __nv_bfloat16* __restrict__ grad_q, __nv_bfloat16* __restrict__ grad_k,
            float* __restrict__ grad_g, float* __restrict__ grad_beta, ChunkWs ws, Seqs seqs, int Hk, int Hv, int dk, int dv,
            long long qs, long long ks) {
    using L = GradSmem<DV>;
    constexpr int LDV = L::LDV;
    extern __shared__ __align__(16) unsigned char sm[];
    const uint32_t base = s32(sm);
    const int slot = blockIdx.x, hk = blockIdx.y, d0 = blockIdx.z * 64, rep = Hv / Hk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, t2 = 2 * (lane & 3);
    const int n = seqs.find(slot);
    int start, len;
    bool ok;
    seqs.get(n, start, len, ok);
    const int c = slot - seqs.first_slot(n, start);
    if (c < 0 || (long long)c * C >= len) return;
    const int nt = min(C, len - c * C), strips = (dv + 31) / 32;
    const size_t tok = (size_t)start + (size_t)c * C, mat = (size_t)dk * dv;
    const float* vec = reinterpret_cast<const float*>(sm + L::VECS);
    load_rows<64, 128>(base + L::K, k + tok * ks + (size_t)hk * dk + d0, ks, nt, dk - d0);
    load_rows<64, 128>(base + L::Q, q + tok * qs + (size_t)hk * dk + d0, qs, nt, dk - d0);
    float gq[8][4], gk[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) gq[i][e] = gk[i][e] = 0.f;
#pragma unroll 1
    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        const size_t wh = (size_t)slot * Hv + h;
        if (r > 0) __syncthreads();
        load_rows<DV, 128>(base + L::DO, grad_o + (tok * Hv + h) * dv, (long long)Hv * dv, nt, dv);
        load_rows<DV, 128>(base + L::U, ws.u + wh * 64 * dv, dv, 64, dv);
        load_rows<DV, 128>(base + L::DVV, grad_v + (tok * Hv + h) * dv, (long long)Hv * dv, nt, dv);
        for (int e = tid; e < VEC / 4; e += 128) cp16(base + L::VECS + e * 16, ws.vec + wh * VEC + e * 4, true);
        cp_commit();
#pragma unroll
        for (int e = tid; e < DV * 8; e += 128) {
            const int row = e % DV, p = e / DV;
            const bool in = row < dv && d0 + p * 8 < dk;
            const size_t from = wh * mat + (in ? ((size_t)(d0 / 8 + p) * dv + row) * 8 : 0);
            cp16(base + L::S + row * LD64 + p * 16, ws.shi + from, in);
            cp16(base + L::DS + row * LD64 + p * 16, ws.dshi + from, in);
        }
        cp_commit();
        if (blockIdx.z == 0 && warp == 3) {    // dg and dbeta: two tokens a lane, summed from the end
            const float* part = ws.parts + wh * strips * PARTS;
            // <S, dS> at the chunk's end, and at its start: the end of the chunk before, or SDS0
            const float* before = c > 0 ? part - (size_t)Hv * strips * PARTS + PART_SDS : part + PART_SDS0;
            double x[2];
            float db[2] = {0.f, 0.f}, end = 0.f, begin = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float a = 0.f, b = 0.f;
                for (int sidx = 0; sidx < strips; ++sidx) {
                    const float* p = part + (size_t)sidx * PARTS + 2 * lane + i;
                    a += p[PART_DOO];
                    b += p[PART_DVV];
                    db[i] += p[PART_DB];
                }
                x[i] = (double)a - (double)b;
            }
            for (int sidx = 0; sidx < strips; ++sidx) {
                end += part[(size_t)sidx * PARTS + PART_SDS] + part[(size_t)sidx * PARTS + PART_SDS + 1];
                begin += before[(size_t)sidx * PARTS] + before[(size_t)sidx * PARTS + 1];
            }
            double sum = x[0] + x[1];                              // of this lane's tokens and all later ones
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_down_sync(0xffffffffu, sum, off);
                if (lane + off < 32) sum += y;
            }
            const double all = __shfl_sync(0xffffffffu, sum, 0), from[2] = {sum, sum - x[0]};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                if (t < nt) {
                    const double f = (double)t / nt;
                    grad_g[(tok + t) * Hv + h] = (float)(f * (from[i] + end) + (1.0 - f) * (begin - (all - from[i])));
                    grad_beta[(tok + t) * Hv + h] = db[i];
                }
            }
        }
        cp_wait<1>();
        __syncthreads();
        // Dw, Da: rows 16 warp .. + 15, as the operands of the next products
        uint32_t aw[4][4], aa[4][4];
        {
            float w[8][4], a[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[i][e] = a[i][e] = 0.f;
#pragma unroll
            for (int d = 0; d < DV; d += 16) {
                uint32_t fo[4], fv[4];
                ldm4(fo, base + L::DO + ofs_a(LDV) + at(16 * warp, d, LDV));
                ldm4(fv, base + L::DVV + ofs_a(LDV) + at(16 * warp, d, LDV));
#pragma unroll
                for (int jp = 0; jp < 4; ++jp)
                    if (jp <= warp) {
                        uint32_t b[4];
                        ldm4(b, base + L::U + ofs_n(LDV) + at(16 * jp, d, LDV));
                        mma(w[2 * jp], fo, b[0], b[1]);
                        mma(w[2 * jp + 1], fo, b[2], b[3]);
                        mma(a[2 * jp], fv, b[0], b[1]);
                        mma(a[2 * jp + 1], fv, b[2], b[3]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j0 = 8 * i + t2;
                const float2 gh = *reinterpret_cast<const float2*>(vec + VEC_GHI + j0), gl = *reinterpret_cast<const float2*>(vec + VEC_GLO + j0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 16 * warp + gi + 8 * (e >> 1), j = j0 + (e & 1);
                    const float hj = (e & 1) ? gh.y : gh.x, lj = (e & 1) ? gl.y : gl.x;
                    const float D = j <= row ? expf((vec[VEC_GHI + row] - hj) + (vec[VEC_GLO + row] - lj)) : 0.f;
                    w[i][e] = j <= row ? D * w[i][e] : 0.f;
                    a[i][e] = j < row ? -D * a[i][e] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                operand(w[2 * j], w[2 * j + 1], aw[j]);
                operand(a[2 * j], a[2 * j + 1], aa[j]);
            }
        }
        cp_wait<0>();
        __syncthreads();
        // rows times states: acc = X M for X a [64][DV] tile and M a [DV][64] one
        const float eg[2] = {vec[VEC_EG + 16 * warp + gi], vec[VEC_EG + 16 * warp + gi + 8]};
        const float dc[2] = {vec[VEC_DEC + 16 * warp + gi], vec[VEC_DEC + 16 * warp + gi + 8]};
        auto times = [&](int X, int M, float (&acc)[8][4]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
            for (int d = 0; d < DV; d += 16) {
                uint32_t f[4];
                ldm4(f, base + X + ofs_a(LDV) + at(16 * warp, d, LDV));
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) {
                    uint32_t b[4];
                    ldm4t(b, base + M + ofs_k(LD64) + at(d, 16 * jp, LD64));
                    mma(acc[2 * jp], f, b[0], b[1]);
                    mma(acc[2 * jp + 1], f, b[2], b[3]);
                }
            }
        };
        {
            float acc[8][4];
            times(L::DO, L::S, acc);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) gq[i][e] = fmaf(eg[e >> 1], acc[i][e], gq[i][e]);
            times(L::DVV, L::S, acc);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) gk[i][e] = fmaf(-eg[e >> 1], acc[i][e], gk[i][e]);
            times(L::U, L::DS, acc);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) gk[i][e] = fmaf(dc[e >> 1], acc[i][e], gk[i][e]);
        }
        // Dw K, Da K
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= warp) {
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) {
                    uint32_t b[4];
                    ldm4t(b, base + L::K + ofs_k(LD64) + at(16 * j, 16 * jp, LD64));
                    mma(gq[2 * jp], aw[j], b[0], b[1]);
                    mma(gq[2 * jp + 1], aw[j], b[2], b[3]);
                    mma(gk[2 * jp], aa[j], b[0], b[1]);
                    mma(gk[2 * jp + 1], aa[j], b[2], b[3]);
                }
            }
        // Dw^T Q, Da^T K: through the tiles of dO and dV, which are done with
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= warp) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int off = (16 * warp + gi + 8 * (e & 1)) * LD64 + (16 * j + 8 * (e >> 1) + t2) * 2;
                    *reinterpret_cast<uint32_t*>(sm + L::DO + off) = aw[j][e];
                    *reinterpret_cast<uint32_t*>(sm + L::DVV + off) = aa[j][e];
                }
            }
        __syncthreads();
#pragma unroll
        for (int ip = 0; ip < 4; ++ip)
            if (ip >= warp) {
                uint32_t fw[4], fa[4];
                ldm4t(fw, base + L::DO + ofs_at(LD64) + at(16 * ip, 16 * warp, LD64));
                ldm4t(fa, base + L::DVV + ofs_at(LD64) + at(16 * ip, 16 * warp, LD64));
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) {
                    uint32_t b[4];
                    ldm4t(b, base + L::Q + ofs_k(LD64) + at(16 * ip, 16 * jp, LD64));
                    mma(gk[2 * jp], fw, b[0], b[1]);
                    mma(gk[2 * jp + 1], fw, b[2], b[3]);
                    ldm4t(b, base + L::K + ofs_k(LD64) + at(16 * ip, 16 * jp, LD64));
                    mma(gk[2 * jp], fa, b[0], b[1]);
                    mma(gk[2 * jp + 1], fa, b[2], b[3]);
                }
            }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = 16 * warp + gi + 8 * half, d = d0 + 8 * i + t2;
            if (row < nt && d < dk) {
                const size_t to = ((tok + row) * Hk + hk) * dk + d;
                *reinterpret_cast<uint32_t*>(grad_q + to) = pack2(gq[i][2 * half], gq[i][2 * half + 1]);
                *reinterpret_cast<uint32_t*>(grad_k + to) = pack2(gk[i][2 * half], gk[i][2 * half + 1]);
            }
        }
}

}  // namespace gated
}  // namespace ckda
