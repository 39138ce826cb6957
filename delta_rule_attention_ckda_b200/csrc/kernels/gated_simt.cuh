// The gated delta rule with one decay per head, token by token on CUDA cores in fp32: every
// type and size the operator accepts (any d_k, d_v <= 128).
//
//   S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t
//
// in delta form: R = e^g S; w = v - R^T k; S = R + k (beta w)^T; o = S^T q.
//
// Forward: one thread per state column (columns never mix), the column in registers, the
// tokens' q and k staged 16 at a time. Also the single-token step of sizes that have no
// kernel of their own (state indexed by `slots`).
//
// Backward (cotangent dS of S_t, reverse order):
//   dS += q dO^T; dq = S dO; du = dS^T k; dbeta = du.w; dv = beta du;
//   dk = dS (beta w) - R (beta du); dS -= k (beta du)^T; dg = <dS, R>; dS *= e^g.
// One CTA per (sequence, head): column phases (thread = column) and row phases (thread =
// row) over dS and R in padded shared memory. The forward states come from checkpoints every
// KB tokens, recomputed KB at a time into a scratch of the workspace.
//
// What bounds it is the chain of tokens (one step after the other, a few block barriers each going
// backward); it serves the types and sizes that the tensor-core kernels do not take. Measured, 8 sequences
// of 1024 tokens, 16 heads of 128, fp32: forward 1.8 ms (1.8 us a token), backward 39 ms (39 us a token);
// bytes alone would take 42 and 73 us.
#pragma once
#include "gated_common.cuh"

namespace ckda {
namespace gated {

// The slot rules of the single-token step: a negative slot is a padding row; a slot beyond the
// pool or one that an earlier row names too is reported and skipped. All threads of the block.
__device__ __forceinline__ bool slot_usable(const int* slots, int n, int pool, long long& state) {
    if (slots == nullptr) {
        state = n;
        return true;
    }
    const int s = __ldg(slots + n);
    state = s;
    if (s < 0) return false;
    bool twice = false;
    for (int m = threadIdx.x; m < n; m += blockDim.x) twice |= __ldg(slots + m) == s;
    const bool bad = __syncthreads_or(twice) != 0 || s >= pool;
    if (bad && threadIdx.x == 0) report_index_error();
    return !bad;
}

template <int DK, typename TIn>
__global__ void __launch_bounds__(128)
simt_fwd_kernel(const TIn* __restrict__ q, const TIn* __restrict__ k, const TIn* __restrict__ v,
                const float* __restrict__ g, const float* __restrict__ beta, const float* S0, TIn* __restrict__ o,
                float* ST, Seqs seqs, const int* __restrict__ slots, int pool, int Hk, int Hv, int dk, int dv,
                long long qs, long long ks, long long vs) {
    constexpr int TB = 16;
    __shared__ float sk[TB][DK], sq[TB][DK], sv[TB][128], sa[TB], sb[TB];
    const int n = blockIdx.x / Hv, h = blockIdx.x % Hv, hk = h / (Hv / Hk);
    int start, len;
    bool ok;
    seqs.get(n, start, len, ok);
    if (!ok && h == 0 && blockIdx.y == 0 && threadIdx.x == 0) report_index_error();
    long long state;
    if (!slot_usable(slots, n, pool, state)) return;
    const int j = blockIdx.y * blockDim.x + threadIdx.x;
    const bool active = j < dv;
    const size_t base = ((size_t)state * Hv + h) * dk * dv;
    float s[DK];
#pragma unroll
    for (int i = 0; i < DK; ++i) s[i] = (active && S0 != nullptr && i < dk) ? S0[base + (size_t)i * dv + j] : 0.f;
    for (int t0 = 0; t0 < len; t0 += TB) {
        const int nt = min(TB, len - t0);
        __syncthreads();
        for (int idx = threadIdx.x; idx < nt * DK; idx += blockDim.x) {
            const int tt = idx / DK, i = idx % DK;
            const size_t tok = (size_t)start + t0 + tt;
            sk[tt][i] = i < dk ? to_f32(k[tok * ks + (size_t)hk * dk + i]) : 0.f;
            sq[tt][i] = i < dk ? to_f32(q[tok * qs + (size_t)hk * dk + i]) : 0.f;
        }
        if (threadIdx.x < nt) {
            const size_t tok = (size_t)start + t0 + threadIdx.x;
            sa[threadIdx.x] = expf(gate_in(g[tok * Hv + h]));
            sb[threadIdx.x] = beta[tok * Hv + h];
        }
        for (int tt = 0; tt < nt; ++tt)
            sv[tt][threadIdx.x] = active ? to_f32(v[((size_t)start + t0 + tt) * vs + (size_t)h * dv + j]) : 0.f;
        __syncthreads();
#pragma unroll 1
        for (int tt = 0; tt < nt; ++tt) {
            const float a = sa[tt];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < DK; ++i) {
                s[i] *= a;
                y = fmaf(s[i], sk[tt][i], y);
            }
            const float u = sb[tt] * (sv[tt][threadIdx.x] - y);
            float acc = 0.f;
#pragma unroll
            for (int i = 0; i < DK; ++i) {
                s[i] = fmaf(sk[tt][i], u, s[i]);
                acc = fmaf(s[i], sq[tt][i], acc);
            }
            if (active) o[(((size_t)start + t0 + tt) * Hv + h) * dv + j] = from_f32<TIn>(acc);
        }
    }
    if (active && ST != nullptr) {
#pragma unroll
        for (int i = 0; i < DK; ++i)
            if (i < dk) ST[base + (size_t)i * dv + j] = s[i];
    }
}

constexpr int KB = 8;                          // tokens between checkpoints
constexpr int NTB = 128;                       // threads of the backward kernel
constexpr int LDS_ = 129;                      // padded row of the shared-memory matrices
constexpr size_t kSimtBwdSmem = (size_t)(2 * 128 * LDS_ + KB * 128 + 8 * 128 + 64) * sizeof(float);

// Sum of x over the block's 128 threads, the same value in every thread.
__device__ __forceinline__ float block_sum(float x, float* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// ckpt: [slot of KB tokens][Hv][dk][dv] states before every KB-th token, placed by `Seqs` as
// chunks are, C / KB to a chunk; scratch: [N * Hv][KB][dk][dv]; pq, pk: [total][Hv][dk].
template <typename TIn>
__global__ void __launch_bounds__(NTB)
simt_bwd_kernel(const TIn* __restrict__ q, const TIn* __restrict__ k, const TIn* __restrict__ v,
                const float* __restrict__ g, const float* __restrict__ beta, const float* __restrict__ S0,
                const TIn* __restrict__ grad_o, const float* __restrict__ dST, float* ckpt, float* scratch,
                float* __restrict__ pq, float* __restrict__ pk, TIn* __restrict__ grad_v, float* __restrict__ grad_g,
                float* __restrict__ grad_beta, float* grad_S0, Seqs seqs, int Hk, int Hv, int dk, int dv, long long qs,
                long long ks, long long vs) {
    extern __shared__ float smf[];
    float* D = smf;                            // [128][LDS_] the cotangent dS
    float* R = D + 128 * LDS_;                 // [128][LDS_] the running state, then e^g S_{t-1}
    float* W = R + 128 * LDS_;                 // [KB][128] w of the recomputed tokens
    float* sq = W + KB * 128;
    float* sk = sq + 128;
    float* sdo = sk + 128;
    float* sbu = sdo + 128;                    // beta w
    float* sbd = sbu + 128;                    // beta du
    float* red = sbd + 128;
    const int n = blockIdx.x / Hv, h = blockIdx.x % Hv, hk = h / (Hv / Hk), x = threadIdx.x;
    int start, len;
    bool ok;
    seqs.get(n, start, len, ok);
    if (!ok && h == 0 && x == 0) report_index_error();
    const size_t nh = (size_t)n * Hv + h, mat = (size_t)dk * dv;
    float* mine = scratch + nh * KB * mat;
    const size_t ck0 = (size_t)seqs.first_slot(n, start) * (C / KB);
    auto ck = [&](int blk) { return ckpt + ((ck0 + blk) * Hv + h) * mat; };
    const bool col = x < dv, row = x < dk;
    // one token of the recurrence on R (thread = column): returns w of the column
    auto step = [&](int t) {
        const size_t tok = (size_t)start + t;
        __syncthreads();
        if (row) sk[x] = to_f32(k[tok * ks + (size_t)hk * dk + x]);
        __syncthreads();
        float w = 0.f;
        if (col) {
            const float a = expf(gate_in(g[tok * Hv + h])), b = beta[tok * Hv + h];
            float y = 0.f;
            for (int i = 0; i < dk; ++i) {
                const float r = R[i * LDS_ + x] * a;
                R[i * LDS_ + x] = r;
                y = fmaf(r, sk[i], y);
            }
            w = to_f32(v[tok * vs + (size_t)h * dv + x]) - y;
            for (int i = 0; i < dk; ++i) R[i * LDS_ + x] = fmaf(sk[i], b * w, R[i * LDS_ + x]);
        }
        return w;
    };
    if (col)
        for (int i = 0; i < dk; ++i) {
            R[i * LDS_ + x] = S0 ? S0[nh * mat + (size_t)i * dv + x] : 0.f;
            D[i * LDS_ + x] = dST ? dST[nh * mat + (size_t)i * dv + x] : 0.f;
        }
    const int nblk = (len + KB - 1) / KB;
    for (int blk = 0; blk < nblk; ++blk) {
        if (col)
            for (int i = 0; i < dk; ++i) ck(blk)[(size_t)i * dv + x] = R[i * LDS_ + x];
        for (int t = blk * KB; t < min(len, blk * KB + KB); ++t) step(t);
    }
    for (int blk = nblk - 1; blk >= 0; --blk) {
        const int t0 = blk * KB, nt = min(KB, len - t0);
        if (col)
            for (int i = 0; i < dk; ++i) R[i * LDS_ + x] = ck(blk)[(size_t)i * dv + x];
        for (int tt = 0; tt < nt; ++tt) {      // mine[tt] = S before token t0 + tt
            if (col)
                for (int i = 0; i < dk; ++i) mine[tt * mat + (size_t)i * dv + x] = R[i * LDS_ + x];
            const float w = step(t0 + tt);
            W[tt * 128 + x] = w;
        }
        for (int tt = nt - 1; tt >= 0; --tt) {
            const size_t tok = (size_t)start + t0 + tt;
            const float a = expf(gate_in(g[tok * Hv + h])), b = beta[tok * Hv + h];
            __syncthreads();
            if (row) {
                sq[x] = to_f32(q[tok * qs + (size_t)hk * dk + x]);
                sk[x] = to_f32(k[tok * ks + (size_t)hk * dk + x]);
            }
            if (col) sdo[x] = to_f32(grad_o[(tok * Hv + h) * dv + x]);
            __syncthreads();
            float db = 0.f, udo = 0.f;
            if (col) {
                const float w = W[tt * 128 + x], dox = sdo[x];
                float du = 0.f;
                for (int i = 0; i < dk; ++i) {
                    const float d = fmaf(sq[i], dox, D[i * LDS_ + x]);
                    D[i * LDS_ + x] = d;
                    du = fmaf(d, sk[i], du);
                    R[i * LDS_ + x] = a * mine[tt * mat + (size_t)i * dv + x];
                }
                sbu[x] = b * w;
                sbd[x] = b * du;
                db = du * w;
                udo = b * w * dox;
                grad_v[(tok * Hv + h) * dv + x] = from_f32<TIn>(b * du);
            }
            db = block_sum(db, red);
            udo = block_sum(udo, red);
            if (row) {
                float dq = 0.f, dkk = 0.f;
                for (int j = 0; j < dv; ++j) {
                    const float r = R[x * LDS_ + j];
                    dq = fmaf(r, sdo[j], dq);
                    dkk = fmaf(D[x * LDS_ + j], sbu[j], dkk);
                    dkk = fmaf(-r, sbd[j], dkk);
                }
                pq[(tok * Hv + h) * dk + x] = fmaf(sk[x], udo, dq);
                pk[(tok * Hv + h) * dk + x] = dkk;
            }
            __syncthreads();
            float dg = 0.f;
            if (col) {
                const float bd = sbd[x];
                for (int i = 0; i < dk; ++i) {
                    const float d = fmaf(-sk[i], bd, D[i * LDS_ + x]);
                    dg = fmaf(d, R[i * LDS_ + x], dg);
                    D[i * LDS_ + x] = a * d;
                }
            }
            dg = block_sum(dg, red);
            if (x == 0) {
                grad_g[tok * Hv + h] = dg;
                grad_beta[tok * Hv + h] = db;
            }
        }
        __syncthreads();
    }
    if (col && grad_S0)
        for (int i = 0; i < dk; ++i) grad_S0[nh * mat + (size_t)i * dv + x] = D[i * LDS_ + x];
}

// Gradients of shared key heads: the sum over the value heads that read each, in head order.
// Rows behind the last sequence stay as they were.
template <typename TIn>
__global__ void __launch_bounds__(256)
simt_share_kernel(const float* __restrict__ pq, const float* __restrict__ pk, TIn* __restrict__ grad_q,
                  TIn* __restrict__ grad_k, Seqs seqs, int Hk, int Hv, int dk) {
    const int rep = Hv / Hk;
    const int first = seqs.cu ? min(max(__ldg(seqs.cu), 0), seqs.total) : 0;
    const int last = seqs.cu ? min(max(__ldg(seqs.cu + seqs.N), 0), seqs.total) : seqs.total;
    const size_t end = (size_t)last * Hk * dk;
    for (size_t e = (size_t)first * Hk * dk + blockIdx.x * 256ull + threadIdx.x; e < end; e += gridDim.x * 256ull) {
        const size_t th = e / dk, i = e % dk;               // token * Hk + key head
        float a = 0.f, b = 0.f;
        for (int r = 0; r < rep; ++r) {
            const size_t at = (th * rep + r) * dk + i;       // token * Hv + hk * rep + r
            a += pq[at];
            b += pk[at];
        }
        grad_q[e] = from_f32<TIn>(a);
        grad_k[e] = from_f32<TIn>(b);
    }
}

}  // namespace gated
}  // namespace ckda
