// Chunked gated delta rule, part 3: the gradients of q, k, g and beta, all chunks side by side,
// from what the two chains left (S the entering state, dS the cotangent of the leaving one,
// U, dV, and sums per token):
//   Dw = tril(D (.) dO U^T),   Da = -tril(D (.) dV U^T, -1)
//   dQ = e^G (.) dO S^T + Dw K
//   dK = -e^G (.) dV S^T + e^{G_C - G} (.) U dS^T + Dw^T Q + Da K + Da^T K
//   dbeta_t = <w_t, y_t>,   dg_t = sum_{i >= t} e_i + <S_C, dS_C>,   e_i = <dO_i, o_i> - <dV_i, v_i>
// dg: scaling the state of one moment scales what every later term takes of it, so the later
// terms' own products with their cotangents sum to the derivative by the log gate. The same
// number counted from the chunk's start is <S_0, dS_0> - sum_{i < t} e_i; each term is off by its
// products' rounding, a like part of it, so the two are weighted by the squares of the other's terms. Where
// terms are alike that cuts the error to a half of the one-sided one; a sequence's dS_T, which no gate has
// damped yet, then has no say in gates that damp it.
// In e_i a token's own update meets its own output, p_i dO_i.u_i with p_i = q_i.k_i, on both sides
// and cancels: o_i = o'_i + p_i u_i, y_i = y'_i + p_i dO_i, v_i = w_i + d_i give
//   e_i = <dO_i, o'_i> - beta_i (<y_i, d_i> + <w_i, y'_i>),
// in which o' and d (what the past gives) and y' (what the future asks for) fall with the decay as dg
// does. So the chains form those three without the own part, never as differences, and dg keeps its digits
// under strong gates.
//
// dQ and dK are rounded to bf16 at the end, so their operands go in one bf16 term; dg and
// dbeta come from the chains' fp32 sums. Per chunk and head 157 KB are read (states
// and cotangents 64, the rest tokens) for 2500 warp products. One CTA of eight warps an SM walks
// over (chunk, key head) pairs; every tile of the next pair is asked for as soon as the products
// that read its place are done, so about 100 KB are always on their way. The tiles come by bulk
// and tensor copies: the same loop on cp.async, 16 bytes a thread, spent 40% of its time issuing
// them. A chunk that ends inside comes row by row, with zeros behind its end. Dw and Da are
// formed by four warps each and pass through shared memory, where they serve as left operands
// straight and transposed; then a warp owns 16 tokens and half of the channels. Value heads
// that share a key head are summed in the accumulators, in head order.
//
// Measured, 8192 chunks of 128 x 128 (1.3 GB): 487 us, 41% of the copy bandwidth; 714 before the bulk
// copies. What bounds it now is the warps' own products and fragment loads between barriers (issue
// 22%, tensor pipe 30%, shared memory 32%) with one CTA an SM by shared memory; sixteen warps
// spill and are slower.
#pragma once
#include "gated_chain.cuh"

namespace ckda {
namespace gated {

// Shared memory (bytes from a 1024-aligned base): token tiles twice, states and keys once. Token
// tiles are blocks of [64][64] with the 128-byte swizzle; states lie as in the workspace.
template <int DK, int DV>
struct GradSmem {
    static constexpr int TILE = DV / 64 * 8192, KTILE = DK / 64 * 8192;
    static constexpr int DO = 0, U = DO + TILE, DVV = U + TILE, VECS = DVV + TILE, TOKENS = VECS + 2048;
    static constexpr int S = 2 * TOKENS, DS = S + DK * DV * 2, K = DS + DK * DV * 2, Q = K + KTILE, DW = Q + KTILE,
                         DA = DW + 64 * LD64, BYTES = DA + 64 * LD64 + 1024;
};
static_assert(GradSmem<128, 128>::BYTES <= 232448, "more shared memory than an SM has");

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

struct GradBars {
    uint64_t tokens[2], s, ds, kq;
    int dead;
};
__device__ __forceinline__ void grad_wait(GradBars& b, uint64_t* bar, uint32_t phase) {
    if (tc::mbar_try_wait(bar, phase)) return;
    if (*reinterpret_cast<volatile int*>(&b.dead)) return;
    if (!tc::mbar_wait(bar, phase)) *reinterpret_cast<volatile int*>(&b.dead) = 1;
}

// One (chunk, value head): where its rows lie.
struct GradUnit {
    int item, r, c, nt;
    size_t tok, wh;
};

template <int DK, int DV>
__global__ void __launch_bounds__(256, 1)
grad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mo,
            const __grid_constant__ CUtensorMap mgv, const __grid_constant__ CUtensorMap mu, const ChainIn in,
            const __nv_bfloat16* __restrict__ grad_v, __nv_bfloat16* __restrict__ grad_q, __nv_bfloat16* __restrict__ grad_k,
            float* __restrict__ grad_g, float* __restrict__ grad_beta, ChunkWs ws, Seqs seqs, int slots, int Hk, int Hv, int dk, int dv) {
    using L = GradSmem<DK, DV>;
    constexpr int NH = DK / 16;                                         // tiles of 8 channels a warp owns
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ GradBars bars;
    const uint32_t base = s32(sm);
    const int rep = Hv / Hk, items = slots * Hk, strips = (dv + 31) / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, t2 = 2 * (lane & 3);
    const int rb = warp & 3, part2 = warp >> 2, d0 = part2 * (DK / 2);  // row block, half of the channels
    const size_t mat = (size_t)dk * dv;

    // the next unit: the next head of the item, else the next item that names a chunk
    auto advance = [&](GradUnit& u) {
        if (u.item >= 0 && u.item < items && u.r + 1 < rep) {
            ++u.r;
            ++u.wh;
            return;
        }
        u.r = 0;
        while (true) {
            u.item = u.item < 0 ? (int)blockIdx.x : u.item + (int)gridDim.x;
            if (u.item >= items) return;
            const int slot = u.item / Hk, n = seqs.find(slot);
            int start, len;
            bool ok;
            seqs.get(n, start, len, ok);
            u.c = slot - seqs.first_slot(n, start);
            if (u.c < 0 || (long long)u.c * C >= len) continue;
            u.nt = min(C, len - u.c * C);
            u.tok = (size_t)start + (size_t)u.c * C;
            u.wh = (size_t)slot * Hv + (u.item % Hk) * rep;
            return;
        }
    };
    auto load_tokens = [&](const GradUnit& u, int b) {
        const uint32_t to = base + b * L::TOKENS;
        const int h = (u.item % Hk) * rep + u.r;
        const bool tiles = in.maps && u.nt == C;
        if (tid == 0) {
            tc::fence_proxy_async_smem();
            tc::mbar_arrive_expect_tx(&bars.tokens[b], VEC * 4 + (tiles ? 3 * L::TILE : 0));
            bulk_copy(to + L::VECS, ws.vec + u.wh * VEC, VEC * 4, &bars.tokens[b]);
            if (tiles) {
#pragma unroll
                for (int x = 0; x < DV / 64; ++x) {
                    tma_rows(to + L::DO + x * 8192, &mo, &bars.tokens[b], 64 * x, h, (int)u.tok);
                    tma_rows(to + L::U + x * 8192, &mu, &bars.tokens[b], 64 * x, 0, (int)(u.wh * 64));
                    tma_rows(to + L::DVV + x * 8192, &mgv, &bars.tokens[b], 64 * x, h, (int)u.tok);
                }
            }
        }
        if (!tiles) {
            tile_rows<256>(to + L::DO, in.dO + (u.tok * Hv + h) * dv, (long long)Hv * dv, u.nt, dv, DV, tid);
            tile_rows<256>(to + L::U, ws.u + u.wh * 64 * dv, dv, 64, dv, DV, tid);
            tile_rows<256>(to + L::DVV, grad_v + (u.tok * Hv + h) * dv, (long long)Hv * dv, u.nt, dv, DV, tid);
        }
        cp_commit();
    };
    auto load_keys = [&](const GradUnit& u) {
        const int hk = u.item % Hk;
        const bool tiles = in.maps && u.nt == C;
        if (tid == 0) {
            tc::fence_proxy_async_smem();
            tc::mbar_arrive_expect_tx(&bars.kq, tiles ? 2 * L::KTILE : 0);
            if (tiles) {
#pragma unroll
                for (int x = 0; x < DK / 64; ++x) {
                    tma_rows(base + L::K + x * 8192, &mk, &bars.kq, 64 * x, hk, (int)u.tok);
                    tma_rows(base + L::Q + x * 8192, &mq, &bars.kq, 64 * x, hk, (int)u.tok);
                }
            }
        }
        if (!tiles) {
            tile_rows<256>(base + L::K, in.k + u.tok * in.ks + (size_t)hk * dk, in.ks, u.nt, dk, DK, tid);
            tile_rows<256>(base + L::Q, in.q + u.tok * in.qs + (size_t)hk * dk, in.qs, u.nt, dk, DK, tid);
        }
        cp_commit();
    };
    // a state as it lies in the workspace, [dk / 8][dv][8]: group p of 8 channels at p * dv * 16 bytes
    auto load_state = [&](const GradUnit& u, int to, const __nv_bfloat16* from, uint64_t* bar) {
        if (tid != 0) return;
        tc::fence_proxy_async_smem();
        tc::mbar_arrive_expect_tx(bar, (uint32_t)(mat * 2));
        bulk_copy(base + to, from + u.wh * mat, (uint32_t)(mat * 2), bar);
    };
    if (tid == 0) {
        for (uint64_t* e : {&bars.tokens[0], &bars.tokens[1], &bars.s, &bars.ds, &bars.kq}) tc::mbar_init(e, 1);
        bars.dead = 0;
        tc::fence_mbar_init();
    }
    for (int i = tid; i < (L::BYTES - 1024) / 16; i += 256) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    previous_done();
    const uint32_t ln = swz_lane(true), lk = swz_lane(false);           // as ofs_n / ofs_at, as ofs_k / ofs_a
    // rows of a state tile as the right operand's k: this lane's row and group of channels
    const uint32_t ls = (uint32_t)(((lane & 7) + ((lane >> 3) & 1) * 8) * 16 + ((lane >> 4) & 1) * dv * 16);

    float gq[NH][4], gk[NH][4];
    GradUnit u{-1, 0, 0, 0, 0, 0};
    advance(u);
    if (u.item < items) {
        load_tokens(u, 0);
        load_state(u, L::S, ws.shi, &bars.s);
        load_state(u, L::DS, ws.dshi, &bars.ds);
    }
#pragma unroll 1
    for (int it = 0; u.item < items; ++it) {
        const int hk = u.item % Hk, h = hk * rep + u.r, b = it & 1;
        const bool tiles = in.maps && u.nt == C;                        // else its rows come by cp.async
        const uint32_t tk = base + b * L::TOKENS;
        const float* vec = reinterpret_cast<const float*>(sm + b * L::TOKENS + L::VECS);
        grad_wait(bars, &bars.tokens[b], (it >> 1) & 1);
        if (!tiles) cp_wait<0>();
        __syncthreads();                       // the tokens are in; the last products of the unit before are done
        load_keys(u);
        if (u.r == 0) {
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) gq[i][e] = gk[i][e] = 0.f;
        }
        // warp 0: the sums that dg and dbeta come from, in flight (two tokens a lane; lanes 0 .. 7 the
        // parts of <S, dS> at the chunk's end, 8 .. 15 those at its start: the end of the chunk before,
        // or SDS0)
        float2 past[4], fut[4], wy[4];
        float edge = 0.f;
        if (warp == 0) {
            const float* part = ws.parts + u.wh * strips * PARTS;
            const float* before = u.c > 0 ? part - (size_t)Hv * strips * PARTS + PART_SDS : part + PART_SDS0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2* p = reinterpret_cast<const float2*>(part + (size_t)i * PARTS) + lane;
                const bool in = i < strips;
                past[i] = in ? p[PART_PAST / 2] : make_float2(0.f, 0.f);
                fut[i] = in ? p[PART_FUTURE / 2] : make_float2(0.f, 0.f);
                wy[i] = in ? p[PART_DB / 2] : make_float2(0.f, 0.f);
            }
            const int i = (lane & 7) / 2;
            if (lane < 16 && i < strips) edge = (lane < 8 ? part + PART_SDS : before)[(size_t)i * PARTS + (lane & 1)];
        }
        {                                      // Dw (warps 0 .. 3) and Da (4 .. 7): 16 rows, columns to the diagonal
            float w[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[i][e] = 0.f;
            const uint32_t left = tk + (part2 ? L::DVV : L::DO);
#pragma unroll
            for (int d = 0; d < DV; d += 16) {
                uint32_t f[4];
                ldm4(f, left + frag(lk, 16 * rb, d));
#pragma unroll
                for (int jp = 0; jp < 4; ++jp)
                    if (jp <= rb) {
                        uint32_t x[4];
                        ldm4(x, tk + L::U + frag(ln, 16 * jp, d));
                        mma(w[2 * jp], f, x[0], x[1]);
                        mma(w[2 * jp + 1], f, x[2], x[3]);
                    }
            }
            unsigned char* out = sm + (part2 ? L::DA : L::DW);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i / 2 > rb) continue;
                const int j0 = 8 * i + t2;
                const float2 gh = *reinterpret_cast<const float2*>(vec + VEC_GHI + j0), gl = *reinterpret_cast<const float2*>(vec + VEC_GLO + j0);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = 16 * rb + gi + 8 * half;
                    const float rh = vec[VEC_GHI + row], rl = vec[VEC_GLO + row];
                    float x[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = j0 + e;
                        const float D = expf((rh - (e ? gh.y : gh.x)) + (rl - (e ? gl.y : gl.x)));
                        x[e] = part2 ? (j < row ? -D * w[i][2 * half + e] : 0.f) : (j <= row ? D * w[i][2 * half + e] : 0.f);
                    }
                    *reinterpret_cast<uint32_t*>(out + row * LD64 + j0 * 2) = pack2(x[0], x[1]);
                }
            }
        }
        GradUnit next = u;
        advance(next);
        const bool more = next.item < items;
        if (more) load_tokens(next, b ^ 1);
        if (warp == 0) {                       // dg and dbeta
            float a[2] = {0.f, 0.f}, e[2] = {0.f, 0.f}, db[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[0] += past[i].x; a[1] += past[i].y;
                e[0] += fut[i].x; e[1] += fut[i].y;
                db[0] += wy[i].x; db[1] += wy[i].y;
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) edge += __shfl_xor_sync(0xffffffffu, edge, off);
            const double end = __shfl_sync(0xffffffffu, edge, 0), begin = __shfl_sync(0xffffffffu, edge, 8);
            const double x[2] = {(double)a[0] - (double)e[0], (double)a[1] - (double)e[1]};
            const double s[2] = {(double)a[0] * a[0] + (double)e[0] * e[0], (double)a[1] * a[1] + (double)e[1] * e[1]};
            double sum = x[0] + x[1], squares = s[0] + s[1];       // of this lane's tokens and all later ones
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_down_sync(0xffffffffu, sum, off), z = __shfl_down_sync(0xffffffffu, squares, off);
                if (lane + off < 32) {
                    sum += y;
                    squares += z;
                }
            }
            const double all = __shfl_sync(0xffffffffu, sum, 0), from[2] = {sum, sum - x[0]};
            const double every = __shfl_sync(0xffffffffu, squares, 0), later[2] = {squares, squares - s[0]};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                if (t < u.nt) {
                    const double earlier = begin * begin + (every - later[i]), both = begin * begin + every + end * end;
                    const double f = both > 0.0 ? earlier / both : 0.0;
                    grad_g[(u.tok + t) * Hv + h] = (float)(f * (from[i] + end) + (1.0 - f) * (begin - (all - from[i])));
                    grad_beta[(u.tok + t) * Hv + h] = db[i];
                }
            }
        }
        grad_wait(bars, &bars.s, it & 1);
        __syncthreads();                       // S is in; Dw and Da are written
        const float eg[2] = {vec[VEC_EG + 16 * rb + gi], vec[VEC_EG + 16 * rb + gi + 8]};
        const float dc[2] = {vec[VEC_DEC + 16 * rb + gi], vec[VEC_DEC + 16 * rb + gi + 8]};
        // rows times states: acc = X M, X a [64][DV] tile, M [DV][this warp's channels]
        auto times = [&](int X, int M, float (&acc)[NH][4]) {
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
            for (int d = 0; d < DV; d += 16) {
                uint32_t f[4];
                ldm4(f, tk + X + frag(lk, 16 * rb, d));
#pragma unroll
                for (int jp = 0; jp < NH / 2; ++jp) {
                    uint32_t x[4];
                    ldm4t(x, base + M + ls + (uint32_t)(((d0 + 16 * jp) / 8 * dv + d) * 16));
                    mma(acc[2 * jp], f, x[0], x[1]);
                    mma(acc[2 * jp + 1], f, x[2], x[3]);
                }
            }
        };
        {
            float acc[NH][4];
            times(L::DO, L::S, acc);
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) gq[i][e] = fmaf(eg[e >> 1], acc[i][e], gq[i][e]);
            times(L::DVV, L::S, acc);
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) gk[i][e] = fmaf(-eg[e >> 1], acc[i][e], gk[i][e]);
            grad_wait(bars, &bars.ds, it & 1);
            __syncthreads();                   // dS is in; S is done with
            if (more) load_state(next, L::S, ws.shi, &bars.s);
            times(L::U, L::DS, acc);
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) gk[i][e] = fmaf(dc[e >> 1], acc[i][e], gk[i][e]);
        }
        grad_wait(bars, &bars.kq, it & 1);
        if (!tiles) cp_wait<0>();
        __syncthreads();                       // K and Q are in; dS is done with
        if (more) load_state(next, L::DS, ws.dshi, &bars.ds);
#pragma unroll 1
        for (int j = 0; j <= rb; ++j) {        // Dw K, Da K
            uint32_t fw[4], fa[4];
            ldm4(fw, base + L::DW + ofs_a(LD64) + at(16 * rb, 16 * j, LD64));
            ldm4(fa, base + L::DA + ofs_a(LD64) + at(16 * rb, 16 * j, LD64));
#pragma unroll
            for (int jp = 0; jp < NH / 2; ++jp) {
                uint32_t x[4];
                ldm4t(x, base + L::K + frag(lk, 16 * j, d0 + 16 * jp));
                mma(gq[2 * jp], fw, x[0], x[1]);
                mma(gq[2 * jp + 1], fw, x[2], x[3]);
                mma(gk[2 * jp], fa, x[0], x[1]);
                mma(gk[2 * jp + 1], fa, x[2], x[3]);
            }
        }
#pragma unroll 1
        for (int ip = rb; ip < 4; ++ip) {      // Dw^T Q, Da^T K
            uint32_t fw[4], fa[4];
            ldm4t(fw, base + L::DW + ofs_at(LD64) + at(16 * ip, 16 * rb, LD64));
            ldm4t(fa, base + L::DA + ofs_at(LD64) + at(16 * ip, 16 * rb, LD64));
#pragma unroll
            for (int jp = 0; jp < NH / 2; ++jp) {
                uint32_t x[4];
                ldm4t(x, base + L::Q + frag(lk, 16 * ip, d0 + 16 * jp));
                mma(gk[2 * jp], fw, x[0], x[1]);
                mma(gk[2 * jp + 1], fw, x[2], x[3]);
                ldm4t(x, base + L::K + frag(lk, 16 * ip, d0 + 16 * jp));
                mma(gk[2 * jp], fa, x[0], x[1]);
                mma(gk[2 * jp + 1], fa, x[2], x[3]);
            }
        }
        if (u.r == rep - 1) {
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = 16 * rb + gi + 8 * half, d = d0 + 8 * i + t2;
                    if (row < u.nt && d < dk) {
                        const size_t to = ((u.tok + row) * Hk + hk) * dk + d;
                        *reinterpret_cast<uint32_t*>(grad_q + to) = pack2(gq[i][2 * half], gq[i][2 * half + 1]);
                        *reinterpret_cast<uint32_t*>(grad_k + to) = pack2(gk[i][2 * half], gk[i][2 * half + 1]);
                    }
                }
        }
        u = next;
    }
}

}  // namespace gated
}  // namespace ckda
