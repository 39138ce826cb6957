// Single-token step of the gated delta rule on a pool of states (d_k in {64, 128}, d_v a
// multiple of 32), HBM-bound: every state element is read once and written once.
//
// For one (row n, value head h), with a = e^g and S the row's state:
//   y = a S^T k,  z = a S^T q,  u = beta (v - y),  S' = a S + k u^T,  o = S'^T q = z + u (k.q)
// so one pass over the state in registers serves the read, the update and the output.
//
// A CTA of 256 threads owns CW columns of one state: CW / 4 lanes across a row (float4 each),
// 1024 / CW rows at a time, RPT rows per thread, all loads issued before the inputs are looked
// at. Column sums go over a thread's rows, then over the lanes of a warp that share columns,
// then over the 8 warps in shared memory. Narrow slabs (CW = 32) give few rows enough CTAs to
// fill the GPU; wide ones (CW = 128) cost fewer reductions per byte.
//
// Measured, 256 rows of 16 heads of 128 x 128 (541 MB): 94 us, 88% of the copy bandwidth, at two
// blocks an SM, which keep a whole state of 64 KB each in flight; left to three, the loads of
// a thread are split and it takes 119. 3 rows: 5 us, the launch and one trip to memory and back.
#pragma once
#include "gated_simt.cuh"

namespace ckda {
namespace gated {

template <int DK, int CW, typename TIn>
__global__ void __launch_bounds__(256, 2)
decode_kernel(const TIn* __restrict__ q, const TIn* __restrict__ k, const TIn* __restrict__ v,
              const float* __restrict__ g, const float* __restrict__ beta, float* __restrict__ S, TIn* __restrict__ o,
              const int* __restrict__ slots, int pool, int Hk, int Hv, int dv, long long qs, long long ks, long long vs) {
    constexpr int LX = CW / 4;                 // lanes across a row
    constexpr int RG = 256 / LX;               // rows at a time
    constexpr int RPT = DK / RG;               // rows per thread
    static_assert(RPT >= 1 && LX <= 32, "slab shape");
    __shared__ float sk[DK], sq[DK];
    __shared__ float4 ry[8][LX], rz[8][LX];
    __shared__ float s_kq;
    const int n = blockIdx.x / Hv, h = blockIdx.x % Hv, hk = h / (Hv / Hk);
    const int tid = threadIdx.x, warp = tid >> 5, lx = tid % LX, rg = tid / LX;
    const int col = blockIdx.y * CW + 4 * lx;
    const int slot = slots ? __ldg(slots + n) : n;
    if (slot < 0) return;
    const bool inside = slots == nullptr || slot < pool;
    float4* Sp = reinterpret_cast<float4*>(S + (((size_t)(inside ? slot : 0) * Hv + h) * DK) * dv + col);
    float4 st[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) st[r] = __ldcs(&Sp[(size_t)(rg + r * RG) * (dv / 4)]);
    if (tid < DK) {
        sk[tid] = to_f32(k[n * ks + (size_t)hk * DK + tid]);
        sq[tid] = to_f32(q[n * qs + (size_t)hk * DK + tid]);
    }
    const float a = expf(gate_in(__ldg(g + (size_t)n * Hv + h))), b = __ldg(beta + (size_t)n * Hv + h);
    const TIn* vp = v + n * vs + (size_t)h * dv + col;
    const float4 vv = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
    long long state;
    if (!slot_usable(slots, n, pool, state)) return;   // nothing was written yet
    __syncthreads();
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const float ki = sk[rg + r * RG], qi = sq[rg + r * RG];
        st[r].x *= a; st[r].y *= a; st[r].z *= a; st[r].w *= a;
        y.x = fmaf(st[r].x, ki, y.x); y.y = fmaf(st[r].y, ki, y.y);
        y.z = fmaf(st[r].z, ki, y.z); y.w = fmaf(st[r].w, ki, y.w);
        z.x = fmaf(st[r].x, qi, z.x); z.y = fmaf(st[r].y, qi, z.y);
        z.z = fmaf(st[r].z, qi, z.z); z.w = fmaf(st[r].w, qi, z.w);
    }
#pragma unroll
    for (int off = LX; off < 32; off <<= 1) {
        y.x += __shfl_xor_sync(0xffffffffu, y.x, off); y.y += __shfl_xor_sync(0xffffffffu, y.y, off);
        y.z += __shfl_xor_sync(0xffffffffu, y.z, off); y.w += __shfl_xor_sync(0xffffffffu, y.w, off);
        z.x += __shfl_xor_sync(0xffffffffu, z.x, off); z.y += __shfl_xor_sync(0xffffffffu, z.y, off);
        z.z += __shfl_xor_sync(0xffffffffu, z.z, off); z.w += __shfl_xor_sync(0xffffffffu, z.w, off);
    }
    if ((tid & 31) < LX) {
        ry[warp][lx] = y;
        rz[warp][lx] = z;
    }
    if (warp == 0) {
        float p = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) p = fmaf(sk[tid + 32 * i], sq[tid + 32 * i], p);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) p += __shfl_xor_sync(0xffffffffu, p, off);
        if (tid == 0) s_kq = p;
    }
    __syncthreads();
    float4 Y = ry[0][lx], Z = rz[0][lx];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
        const float4 c = ry[w][lx], d = rz[w][lx];
        Y.x += c.x; Y.y += c.y; Y.z += c.z; Y.w += c.w;
        Z.x += d.x; Z.y += d.y; Z.z += d.z; Z.w += d.w;
    }
    const float4 u = make_float4(b * (vv.x - Y.x), b * (vv.y - Y.y), b * (vv.z - Y.z), b * (vv.w - Y.w));
    if (tid < LX) {
        const float kq = s_kq;
        TIn* op = o + ((size_t)n * Hv + h) * dv + col;
        op[0] = from_f32<TIn>(fmaf(u.x, kq, Z.x));
        op[1] = from_f32<TIn>(fmaf(u.y, kq, Z.y));
        op[2] = from_f32<TIn>(fmaf(u.z, kq, Z.z));
        op[3] = from_f32<TIn>(fmaf(u.w, kq, Z.w));
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const float ki = sk[rg + r * RG];
        __stcs(&Sp[(size_t)(rg + r * RG) * (dv / 4)],
               make_float4(fmaf(ki, u.x, st[r].x), fmaf(ki, u.y, st[r].y), fmaf(ki, u.z, st[r].z), fmaf(ki, u.w, st[r].w)));
    }
}

}  // namespace gated
}  // namespace ckda
