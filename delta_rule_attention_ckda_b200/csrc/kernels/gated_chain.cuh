// Chunked gated delta rule, part 2: the state from chunk to chunk (see gated_intra.cuh for Z, P).
// Per chunk, S the state entering it:
//   X = V - e^G (.) K S,   W = X + Z (beta X),   U = beta W
//   O = e^G (.) Q S + P U,  S' = e^{G_C} S + K^T (e^{G_C - G} (.) U)
//
// Three products follow one another in every chunk, so the time is a chain of latencies: an
// operand written, a product, its result read. One CTA per (sequence, value head) walks the
// chunks; everything is held transposed, d_v on the 128 TMEM lanes, so that an epilogue thread
// has one column of the state and each product's result, split into bf16 terms, is written
// back to TMEM as the left operand of the next without crossing threads. Eight epilogue warps
// (two per lane quarter, half of the channels or tokens each; sixteen with half the registers
// measured 7 to 20% slower) keep S in fp32 registers; four warps form the output; one thread
// issues the products; three warps load the next chunk's tiles, by tensor copies, or row by row
// where a chunk ends inside (zeros behind a packed sequence's end, where a tile copy would
// bring the next sequence's rows).
//
// The state is split 32 channels at a time, and its product starts on the first (2 to 3% of the
// time).
//
// Measured, 8 x 16 sequences of 4096 tokens: 266 us, 4.2 us a chunk (7500 cycles) of which the
// products are 2000, the tensor pipe 25% busy; with the states, V - W and U for the backward pass
// 385 us (100 more while the out warps, which sum <dO, o>, held the whole stage). A chunk's tiles brought
// to L2 ahead gain 1%: memory is not what it waits for.
//
// What hides what: the output's products (P U), its epilogue and its store run under the next
// chunk's state split; loads run a chunk ahead. A product of N = 64 takes as long as one of
// N = 128, so pairs share one: [K; Q] S, and both terms of Z side by side.
//
// Rounding: raw K, Q, V are exact; every other operand (S, beta X, Z, U, P) is two bf16 terms
// (2.7e-6 of a value at RMS), o is rounded once at its store. Sums are fp32; S' is formed in
// registers. Backward: U in three terms, and the adjoint's operands of the state too, because dg
// is a difference of sums (a model of this arithmetic in fp64: dg off by 4e-6 in place of 2.1e-5 where the
// states are large, by 1.3e-6 in place of 1.4e-5 elsewhere).
#pragma once
#include "gated_mma.cuh"
#include "tc_primitives.cuh"

namespace ckda {
namespace gated {

// Warps by role; every role is whole warpgroups, so that registers can be moved between them.
constexpr int kEpiWarps = 8, kOutWarps = 4, kMmaWarp = 12, kLoadWarps = 3;
constexpr int kChainThreads = 512;
// Registers a thread: 128 at launch; the epilogue warps hold half a state column each, the out
// warps a row of the output.
constexpr int kRegLaunch = 128, kRegEpi = 168, kRegOut = 112, kRegOther = 64;
static_assert(256 * kRegEpi + 128 * kRegOut + 128 * kRegOther <= kChainThreads * kRegLaunch,
              "a register split larger than the launch's waits forever");

// Tensor memory columns
constexpr uint32_t TM_ACC = 0;      // [K S | Q S]; backward: K dS | y
constexpr uint32_t TM_S = 128;      // the state's operand (per 32 channels: hi, lo), then its update
constexpr uint32_t TM_UZ = 256;     // the products with both terms of Z; then the operands U' and U (e^G dV)
constexpr uint32_t TM_X = 384;      // beta X (per half of the tokens: hi, lo); then U' third term
constexpr uint32_t TM_PU = 448;     // P U; backward: P^T dO
constexpr uint32_t TM_COLS = 512;

// A stage of shared memory (bytes from a 1024-aligned base), rows of 128 bytes, 128-byte swizzle
template <int DK, bool kDO>
struct ChainStage {
    static constexpr uint32_t KQ = 0;                              // per 64 channels: [64 rows of K | 64 of Q]
    static constexpr uint32_t V = KQ + (DK / 64) * 16384;          // 2 x [64][64]
    static constexpr uint32_t DO = V + 16384;                      // 2 x [64][64]
    static constexpr uint32_t Z = DO + (kDO ? 16384 : 0);          // [hi | lo]
    static constexpr uint32_t P = Z + 16384;
    static constexpr uint32_t VECS = P + 16384;
    static constexpr uint32_t BYTES = VECS + 1024;
    static constexpr uint32_t OUT = 2 * BYTES;                     // [64][128] rows on their way out
    static constexpr size_t SMEM = OUT + 16384 + 1024;
};
static_assert(ChainStage<128, true>::SMEM <= 232448, "more shared memory than an SM has");

struct ChainBars {
    uint64_t full[2], empty[2], do_full[2], do_empty[2], s[2], m1, x, m2, d, u, uo, m3, o, out, qs;
    uint32_t tmem;
    int dead;                       // a bounded wait ran out: nothing waits any more, the loops run off
};

__device__ __forceinline__ void chain_wait(ChainBars& b, uint64_t* bar, uint32_t phase) {
    if (tc::mbar_try_wait(bar, phase)) return;
    if (*reinterpret_cast<volatile int*>(&b.dead)) return;
    if (!tc::mbar_wait(bar, phase)) *reinterpret_cast<volatile int*>(&b.dead) = 1;
}
// A value the compiler takes as new, so that what it computes from it (a chunk's operand
// descriptors) is computed there and not kept in registers across the loop.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
    asm volatile("" : "+r"(x));
    return x;
}
// A warp's registers from here on, above or below those of the launch (each has its own instruction).
template <int R>
__device__ __forceinline__ void set_regs() {
    if constexpr (R > kRegLaunch) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
    else if constexpr (R < kRegLaunch) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Element (token, channel) of a tile of 64-channel blocks, read by the thread that owns the channel.
__device__ __forceinline__ float tile_value(const unsigned char* tile, int token, int ch) {
    const uint16_t x = *reinterpret_cast<const uint16_t*>(tile + (ch / 64) * 8192 + swz(token, (ch % 64) / 8) + (ch % 8) * 2);
    return __uint_as_float((uint32_t)x << 16);
}

// One lane of a warp that walks together: it issues the products, with operands the whole warp holds.
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Long sequences on few heads run as segments of `cps` chunks side by side. A segment acts on the
// state entering it as S -> M S + N; pass kSegMaps builds every segment's N (from zero, the first
// from S0) and M (from the identity, with v = 0) at once, segment_scan_kernel chains them into the
// state behind every segment, and pass kSegRun runs the segments again from those. The adjoint acts
// as dS -> M^T dS + N' on the same maps: its pass kSegMaps builds every N' (the last from dS_T),
// segment_scan_kernel chains them, and its pass kSegRun runs. Segment j of
// sequence n has place start / (cps C) + n + j of its own, as chunks have. 65536 tokens of 16
// heads: maps 0.60 ms, scan 0.01, run 0.69, against 4.2 whole.
enum { kSegWhole = 0, kSegMaps = 1, kSegRun = 2 };
struct SegArgs {
    int mode, cps;
    int longest_first;              // whole sequences of several lengths in more CTAs than SMs: see by_length
    int apart;                      // results go to segments' places: S_T is S0 (or dS_0 is dS_T), which others still read
    float* states;                  // [place][Hv][dk][dv] fp32: N, then the state behind the segment
    float* maps;                    // [place][Hv][dk][dk] fp32: M, transposed
    float* dstates;                 // backward: [place][Hv][dk][dv] fp32: the cotangent entering a segment from zero, then of the state before it
    __host__ __device__ static size_t places(int N, int total, int cps) { return (size_t)total / ((size_t)cps * C) + (size_t)N; }
    __device__ __forceinline__ int first_place(int n, int start) const { return start / (cps * C) + n; }
    __device__ __forceinline__ int find(const Seqs& seqs, int place) const {
        int lo = 0, hi = seqs.N - 1;
        while (lo < hi) {
            const int m = (lo + hi + 1) / 2;
            const int start = seqs.cu == nullptr ? m * seqs.T : min(max(__ldg(seqs.cu + m), 0), seqs.total);
            if (first_place(m, start) <= place) lo = m; else hi = m - 1;
        }
        return lo;
    }
};

// The sequence of rank `place` by length, longest first (equal ones in order): started last, a long one
// runs on alone (13 sequences of 234 to 1536 tokens, 16 heads: 138 us in order, 107 so). The block together;
// `lens`: memory for N <= kMaxRanked lengths.
constexpr int kMaxRanked = 256;
__device__ __forceinline__ int by_length(const Seqs& seqs, int place, int* lens) {
    __shared__ int found;
    for (int m = threadIdx.x; m < seqs.N; m += blockDim.x) {
        int start;
        bool ok;
        seqs.get(m, start, lens[m], ok);
    }
    __syncthreads();
    if (threadIdx.x < seqs.N) {
        const int mine = lens[threadIdx.x];
        int rank = 0;
        for (int m = 0; m < seqs.N; ++m) rank += lens[m] > mine || (lens[m] == mine && m < (int)threadIdx.x);
        if (rank == place) found = threadIdx.x;
    }
    __syncthreads();
    return found;
}

// The loading warps' share (thread x) of a chunk into stage `st`, completing on `full`: k, q, v (kDO: dO too)
// by tensor copies where the chunk is whole, else by rows with zeros behind the sequence's end;
// the lower blocks of Z and P (those above the block diagonal stay the zeros the kernel starts
// with); the vectors.
template <typename L, int DK, bool kDO>
__device__ __forceinline__ void chain_load(uint32_t st, uint64_t* full, int x, const ChainIn& in, const CUtensorMap* mq, const CUtensorMap* mk,
                                           const CUtensorMap* mv, const CUtensorMap* mo, const ChunkWs& ws, size_t wh, int tok, int nt,
                                           int h, int hk, int Hv, int dk, int dv) {
    constexpr int NT = 32 * kLoadWarps, PK = DK / 8;
    const bool tiles = in.maps && nt == C;
    if (x == 0) {
        tc::mbar_arrive_expect_tx(full, tiles ? (DK / 64) * 16384 + 16384 + (kDO ? 16384 : 0) : 0);
        if (tiles) {
#pragma unroll
            for (int b = 0; b < DK / 64; ++b) {
                tma_rows(st + L::KQ + b * 16384, mk, full, 64 * b, hk, tok);
                tma_rows(st + L::KQ + b * 16384 + 8192, mq, full, 64 * b, hk, tok);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                tma_rows(st + L::V + b * 8192, mv, full, 64 * b, h, tok);
                if constexpr (kDO) tma_rows(st + L::DO + b * 8192, mo, full, 64 * b, h, tok);
            }
        }
    }
    const size_t w0 = wh * 4096;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = x; e < 32 * (i + 1); e += NT) {
            const int r = 16 * i + e / (2 * (i + 1)), p = e % (2 * (i + 1));
            const size_t from = w0 + r * 64 + p * 8;
            const uint32_t to = st + swz(r, p);
            cp16(to + L::Z, ws.zhi + from, true);
            cp16(to + L::Z + 8192, ws.zlo + from, true);
            cp16(to + L::P, ws.phi + from, true);
            cp16(to + L::P + 8192, ws.plo + from, true);
        }
    if (x < (kDO ? 64 : 48)) cp16(st + L::VECS + x * 16, ws.vec + wh * VEC + x * 4, true);
    if (!tiles) {
        const __nv_bfloat16 *q = in.q + tok * in.qs + (size_t)hk * dk, *k = in.k + tok * in.ks + (size_t)hk * dk,
                            *v = in.v + tok * in.vs + (size_t)h * dv, *dO = kDO ? in.dO + ((size_t)tok * Hv + h) * dv : nullptr;
#pragma unroll 2
        for (int e = x; e < 64 * PK; e += NT) {
            const int r = e / PK, p = e % PK;
            const bool is = r < nt && p * 8 < dk;
            const uint32_t to = st + L::KQ + (p / 8) * 16384 + swz(r, p & 7);
            cp16(to, is ? k + r * in.ks + p * 8 : k, is);
            cp16(to + 8192, is ? q + r * in.qs + p * 8 : q, is);
        }
#pragma unroll 2
        for (int e = x; e < 64 * 16; e += NT) {
            const int r = e / 16, p = e % 16;
            const bool is = r < nt && p * 8 < dv;
            const uint32_t to = (p / 8) * 8192 + swz(r, p & 7);
            cp16(st + L::V + to, is ? v + r * in.vs + p * 8 : v, is);
            if constexpr (kDO) cp16(st + L::DO + to, is ? dO + (size_t)r * Hv * dv + p * 8 : dO, is);
        }
    }
    cp_commit();
    cp_wait<0>();
    tc::fence_proxy_async_smem();
    tc::mbar_arrive(full);
}

// The tile of dO alone, completing on `full`: the forward chain's out warps read it last, and nothing
// else should wait for them.
template <typename L>
__device__ __forceinline__ void chain_load_do(uint32_t st, uint64_t* full, int x, const ChainIn& in, const CUtensorMap* mo, int tok, int nt,
                                              int h, int Hv, int dv) {
    const bool tiles = in.maps && nt == C;
    if (x == 0) {
        tc::mbar_arrive_expect_tx(full, tiles ? 16384 : 0);
        if (tiles) {
#pragma unroll
            for (int b = 0; b < 2; ++b) tma_rows(st + L::DO + b * 8192, mo, full, 64 * b, h, tok);
        }
    }
    if (!tiles) {
        tile_rows<32 * kLoadWarps>(st + L::DO, in.dO + ((size_t)tok * Hv + h) * dv, (long long)Hv * dv, nt, dv, 128, x);
        cp_commit();
        cp_wait<0>();
        tc::fence_proxy_async_smem();
    }
    tc::mbar_arrive(full);
}

// The out warps' [64][128] tile of bf16 rows in shared memory to global rows, 16 bytes a lane.
__device__ __forceinline__ void rows_out(const unsigned char* tile, int x, __nv_bfloat16* dst, long long stride, int rows, int cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = x + 128 * i, r = e / 16, p = e % 16;
        if (r < rows && p * 8 < cols) *reinterpret_cast<uint4*>(dst + r * stride + p * 8) = *reinterpret_cast<const uint4*>(tile + r * 256 + p * 16);
    }
}
__device__ __forceinline__ void out_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// 32 fp32 values as bf16 terms to TMEM operand columns: hi at `to`, then 16 columns a term.
template <int TERMS>
__device__ __forceinline__ void put_terms(const float* x, const uint32_t (&to)[TERMS]) {
#pragma unroll
    for (int k = 0; k < 16; k += 8) {
        uint32_t h[8], m[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = 2 * (k + i);
            if constexpr (TERMS == 3) split3(x[j], x[j + 1], h[i], m[i], l[i]);
            else split2(x[j], x[j + 1], h[i], m[i]);
        }
        tc::tmem_st32<8>(to[0] + k, h);
        tc::tmem_st32<8>(to[1] + k, m);
        if constexpr (TERMS == 3) tc::tmem_st32<8>(to[TERMS - 1] + k, l);
    }
}

// A thread's half column of the state: s <- whole s + the update's columns (kFirst: as it is), and, where
// another chunk follows, s as the next product's operand. 32 channels at a time, each with a
// barrier of its own, so that the product over the first runs while the second are split; N
// columns at a time as registers allow. A third term lies in the columns of beta X, which is
// written after that product.
template <int TERMS, int H, int N>
__device__ __forceinline__ void next_state(float (&s)[H], float whole, bool first, bool more, uint32_t tl, int wg, ChainBars& bars) {
#pragma unroll
    for (int i = 0; i < H; i += 32) {
        const uint32_t at = tl + TM_S + wg * H + i;
        if (!first) {
#pragma unroll
            for (int k = 0; k < 32; k += N) {
                float d[N];
                tc::tmem_ld32<N>(at + k, d);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    fma2(d[e], d[e + 1], s[i + k + e], s[i + k + e + 1], whole, whole);
                    s[i + k + e] = d[e];
                    s[i + k + e + 1] = d[e + 1];
                }
            }
        }
        if (more) {
            uint32_t to[TERMS];
            to[0] = at;
            to[1] = at + 16;
            if constexpr (TERMS == 3) to[TERMS - 1] = tl + TM_X + wg * (H / 2) + i / 2;
            put_terms<TERMS>(s + i, to);
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.s[i / 32]);
        }
    }
}

// Sum over the lanes of each of 32 values: lane i returns the sum of v[i].
__device__ __forceinline__ float lane_sums(float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const bool up = lane & off;
            const float keep = up ? v[i + off] : v[i], send = up ? v[i] : v[i + off];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    return v[0];
}

// HD channels of a state column in 4 bytes a value: the fp32 bits, rounded half up to their
// upper 16 (a bf16 value, `hi`) and the signed rest: bits = (hi << 16) + lo. `step`: elements
// between groups of 8 channels (see ChunkWs).
template <int HD>
__device__ __forceinline__ void put_state(const float* s, __nv_bfloat16* hi, __nv_bfloat16* lo, size_t step, int left) {
#pragma unroll
    for (int i = 0; i < HD; i += 8) {
        if (i >= left) break;
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = __float_as_uint(s[i + 2 * j]), b = __float_as_uint(s[i + 2 * j + 1]);
            h[j] = __byte_perm(a + 0x8000u, b + 0x8000u, 0x7632);
            l[j] = __byte_perm(a, b, 0x5410);
        }
        *reinterpret_cast<uint4*>(hi + i / 8 * step) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo + i / 8 * step) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}
__device__ __forceinline__ float state_lo(uint32_t h, uint32_t l) {
    return __uint_as_float((h << 16) + (uint32_t)(int)(short)(l & 0xffffu));
}
__device__ __forceinline__ float state_hi(uint32_t h, uint32_t l) {
    return __uint_as_float((h & 0xffff0000u) + (uint32_t)((int)l >> 16));
}

// What both chains set up and take down.
__device__ __forceinline__ void chain_begin(ChainBars& b, unsigned char* stages, uint32_t bytes, int out_warps) {
    if (threadIdx.x / 32 == kMmaWarp) tc::tmem_alloc(&b.tmem, TM_COLS);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&b.full[i], 32 * kLoadWarps + 1);
            tc::mbar_init(&b.empty[i], 1 + kEpiWarps + out_warps);
            tc::mbar_init(&b.do_full[i], 32 * kLoadWarps + 1);
            tc::mbar_init(&b.do_empty[i], kOutWarps);
        }
        for (uint64_t* e : {&b.s[0], &b.s[1], &b.x, &b.u, &b.uo}) tc::mbar_init(e, 32 * kEpiWarps);
        for (uint64_t* e : {&b.d, &b.out, &b.qs}) tc::mbar_init(e, 32 * kOutWarps);
        for (uint64_t* e : {&b.m1, &b.m2, &b.m3, &b.o}) tc::mbar_init(e, 1);
        b.dead = 0;
        tc::fence_mbar_init();
    }
    for (uint32_t i = threadIdx.x; i < bytes / 16; i += kChainThreads) reinterpret_cast<uint4*>(stages)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    previous_done();
}
__device__ __forceinline__ void chain_end(ChainBars& b) {
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (threadIdx.x / 32 == kMmaWarp) {
        tc::tmem_dealloc(b.tmem, TM_COLS);
        tc::tmem_relinquish();
    }
}

template <int DK, bool kBack>
__global__ void __launch_bounds__(kChainThreads, 1)
chain_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                 const __grid_constant__ CUtensorMap mo, const ChainIn in, const float* S0, __nv_bfloat16* __restrict__ o, float* ST,
                 ChunkWs ws, Seqs seqs, SegArgs sg, int Hk, int Hv, int dk, int dv) {
    using L = ChainStage<DK, kBack>;
    constexpr int H = DK / 2;                  // channels of an epilogue thread
    next_may_start();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ ChainBars bars;
    const int h = blockIdx.x % Hv, hk = h / (Hv / Hk), place = blockIdx.x / Hv;
    const int n = sg.mode ? sg.find(seqs, place) : (sg.longest_first ? by_length(seqs, place, reinterpret_cast<int*>(sm)) : place);
    const bool maps = !kBack && sg.mode == kSegMaps, transition = maps && blockIdx.y == 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int start, len;
    bool ok;
    seqs.get(n, start, len, ok);
    int slot0 = seqs.first_slot(n, start);
    const int strips = (dv + 31) / 32;
    const size_t mat = (size_t)dk * dv, sbase = ((size_t)n * Hv + h) * mat;
    const float* from = S0 == nullptr ? nullptr : S0 + sbase;          // the entering state
    float* to = ST == nullptr ? nullptr : ST + sbase;                  // where the leaving state goes
    bool last = true;
    if (sg.mode) {                             // this segment's chunks, as a sequence of their own
        const int j = place - sg.first_place(n, start), skip = j * sg.cps;
        last = (long long)(skip + sg.cps) * C >= len;
        if (j < 0 || (j > 0 && (long long)skip * C >= len) || (maps && (last || (transition && j == 0)))) return previous_done();
        const size_t own = (size_t)place * Hv + h;
        if (maps) {
            if (j > 0) from = nullptr;
            to = transition ? sg.maps + own * dk * dk : sg.states + own * mat;
        } else {
            if (j > 0) from = sg.states + (own - Hv) * mat;
            if (!last) to = nullptr;
            else if (sg.apart) to = sg.states + own * mat;
        }
        slot0 += skip;
        start += skip * C;
        len = last ? len - skip * C : sg.cps * C;
    }
    const int chunks = (len + C - 1) / C, cols = transition ? dk : dv;  // columns of the state
    chain_begin(bars, sm, 2 * L::BYTES, maps ? 0 : kOutWarps);
    const uint32_t tm = bars.tmem, base = s32(sm);

    if (warp >= kMmaWarp) {
        set_regs<kRegOther>();
        if (warp > kMmaWarp) {                 // ------------------------------------------ loads
            const int x = threadIdx.x - 32 * (kMmaWarp + 1);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                if (c >= 2) chain_wait(bars, &bars.empty[c & 1], ((c >> 1) - 1) & 1);
                chain_load<L, DK, false>(base + (c & 1) * L::BYTES, &bars.full[c & 1], x, in, &mq, &mk, &mv, &mo, ws,
                                         (size_t)(slot0 + c) * Hv + h, start + c * C, min(C, len - c * C), h, hk, Hv, dk, dv);
                if constexpr (kBack) {
                    if (c >= 2) chain_wait(bars, &bars.do_empty[c & 1], ((c >> 1) - 1) & 1);
                    chain_load_do<L>(base + (c & 1) * L::BYTES, &bars.do_full[c & 1], x, in, &mo, start + c * C, min(C, len - c * C), h, Hv, dv);
                }
            }
        } else {                               // ------------------------------------------ products
            constexpr uint32_t i128 = tc::idesc_bf16(128, 128, 0, 0), i64 = tc::idesc_bf16(128, 64, 0, 0),
                               iS = tc::idesc_bf16(128, DK, 0, 1);
            // The output's product of a chunk is issued behind the next chunk's first one: it runs under the
            // epilogue that follows that one.
            auto output = [&](int c) {
                const uint32_t st = fresh(base + (c & 1) * L::BYTES);
                if (c > 0) chain_wait(bars, &bars.out, (c - 1) & 1);   // P U of the chunk before is read
                chain_wait(bars, &bars.uo, c & 1);
                tc::tc_fence_after();
                if (elected()) {
#pragma unroll
                    for (int term = 0; term < 3; ++term)               // P U: hi lo, lo hi, hi hi
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            tc::mma_ts(tm + TM_PU, tm + TM_UZ + 64 + (j / 2) * 32 + (term == 1 ? 16 : 0) + (j % 2) * 8,
                                       tc::sdesc(st + L::P + (term == 0 ? 8192 : 0) + j * 32, 16, 1024), i64, (term | j) != 0);
                    tc::mma_commit(&bars.o);
                    tc::mma_commit(&bars.empty[c & 1]);
                }
            };
            if (chunks > 0) chain_wait(bars, &bars.full[0], 0);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const uint32_t st = fresh(base + (c & 1) * L::BYTES), ph = c & 1;
                if (c > 0 && !maps) chain_wait(bars, &bars.qs, (c - 1) & 1);    // Q S of the chunk before is read
#pragma unroll
                for (int b = 0; b < H / 32; ++b) {                     // [K S | Q S], 32 channels of either half at a time
                    chain_wait(bars, &bars.s[b], ph);
                    tc::tc_fence_after();
                    if (elected()) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {                  // term, half, 16 channels
                            const int term = e / 4, half = (e / 2) % 2, ch = half * H + 32 * b + 16 * (e % 2);
                            tc::mma_ts(tm + TM_ACC, tm + TM_S + half * H + 32 * b + 16 * term + 8 * (e % 2),
                                       tc::sdesc(st + L::KQ + (ch / 64) * 16384 + (ch % 64) * 2, 16, 1024), i128, (b | e) != 0);
                        }
                        if (b == H / 32 - 1) tc::mma_commit(&bars.m1);
                    }
                }
                if (c > 0 && !maps) output(c - 1);
                chain_wait(bars, &bars.x, ph);
                tc::tc_fence_after();
                if (elected()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)                        // beta X [Z_hi | Z_lo]
                        tc::mma_ts(tm + TM_UZ, tm + TM_X + (j / 2) * 32 + (j % 2) * 8, tc::sdesc(st + L::Z + j * 32, 16, 1024), i128, j != 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tc::mma_ts(tm + TM_UZ, tm + TM_X + (j / 2) * 32 + 16 + (j % 2) * 8, tc::sdesc(st + L::Z + j * 32, 16, 1024), i64, 1);
                    tc::mma_commit(&bars.m2);
                }
                chain_wait(bars, &bars.u, ph);
                tc::tc_fence_after();
                if (elected()) {
#pragma unroll
                    for (int term = 0; term < (kBack ? 3 : 2); ++term) // the state's update
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t a = term < 2 ? TM_UZ + (j / 2) * 32 + term * 16 + (j % 2) * 8 : TM_X + (j / 2) * 32 + (j % 2) * 8;
                            tc::mma_ts(tm + TM_S, tm + a, tc::sdesc(st + L::KQ + j * 2048, 16384, 1024), iS, (term | j) != 0);
                        }
                    tc::mma_commit(&bars.m3);
                    if (maps) tc::mma_commit(&bars.empty[c & 1]);
                }
                if (c + 1 < chunks) chain_wait(bars, &bars.full[(c + 1) & 1], ((c + 1) >> 1) & 1);
            }
            if (chunks > 0) {                  // nothing in flight past this point
                if (!maps) output(chunks - 1);
                chain_wait(bars, maps ? &bars.m3 : &bars.o, (chunks - 1) & 1);
            }
        }
    } else if (warp >= kEpiWarps) {            // ------------------------------------------ output
        set_regs<kRegOut>();
        const int quarter = warp & 3, row = 32 * quarter + lane, x = threadIdx.x - 32 * kEpiWarps;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        unsigned char* tile = sm + L::OUT;
#pragma unroll 1
        for (int c = 0; c < (maps ? 0 : chunks); ++c) {
            const unsigned char* st = sm + (c & 1) * L::BYTES;
            const float* eg = reinterpret_cast<const float*>(st + L::VECS) + VEC_EG;
            const int tok = start + c * C, nt = min(C, len - c * C);
            float r[64];
            chain_wait(bars, &bars.full[c & 1], (c >> 1) & 1);
            chain_wait(bars, &bars.m1, c & 1);
            tc::tc_fence_after();
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
                float a[32];
                tc::tmem_ld32<32>(tl + TM_ACC + 64 + i, a);
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) r[i + j] = a[j];
            }
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.qs);
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
                const float4 e = *reinterpret_cast<const float4*>(eg + i);
                r[i] *= e.x; r[i + 1] *= e.y; r[i + 2] *= e.z; r[i + 3] *= e.w;
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars.empty[c & 1]);        // of the stage only dO is read from here on
            chain_wait(bars, &bars.o, c & 1);
            tc::tc_fence_after();
#pragma unroll
            for (int i = 0; i < 64; i += 16) {
                float a[16];
                tc::tmem_ld32<16>(tl + TM_PU + i, a);
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) r[i + j] += a[j];
            }
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.out);
            if constexpr (kBack) chain_wait(bars, &bars.do_full[c & 1], (c >> 1) & 1);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if constexpr (kBack) {
                    float t[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) t[i] = r[32 * half + i] * tile_value(st + L::DO, 32 * half + i, row);
                    const float sum = lane_sums(t);
                    if (quarter < strips)
                        ws.parts[(((size_t)(slot0 + c) * Hv + h) * strips + quarter) * PARTS + PART_PAST + 32 * half + lane] = sum;
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        *reinterpret_cast<__nv_bfloat16*>(tile + (32 * half + i) * 256 + 2 * row) = __float2bfloat16_rn(r[32 * half + i]);
                }
            }
            if constexpr (kBack) {
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.do_empty[c & 1]);
            } else {
                out_sync();
                rows_out(tile, x, o + ((size_t)tok * Hv + h) * dv, (long long)Hv * dv, nt, dv);
                out_sync();
            }
        }
    } else {                                   // ------------------------------------------ epilogues of the chain
        set_regs<kRegEpi>();
        const int quarter = warp & 3, wg = warp >> 2, row = 32 * quarter + lane;
        const bool live = row < cols;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        float s[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int d = wg * H + i;
            s[i] = (from != nullptr && live && d < dk) ? from[(size_t)d * dv + row] : 0.f;
            if (transition && d == row && live) s[i] = 1.f;
        }
#pragma unroll 1
        for (int c = 0; c <= chunks; ++c) {
            if (c > 0) {                       // S <- e^{G_C} S + update
                const float whole = reinterpret_cast<const float*>(sm + ((c - 1) & 1) * L::BYTES + L::VECS)[VEC_EG + 63];
                chain_wait(bars, &bars.m3, (c - 1) & 1);
                tc::tc_fence_after();
                next_state<2, H, 32>(s, whole, false, c < chunks, tl, wg, bars);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.empty[(c - 1) & 1]);
            } else {
                next_state<2, H, 32>(s, 1.f, true, c < chunks, tl, wg, bars);
            }
            if constexpr (kBack) {             // the entering (behind the last chunk: the final) state for the backward kernels
                if (live && (c < chunks || last)) {
                    const size_t to = ((size_t)(slot0 + c) * Hv + h) * mat + ((size_t)(wg * H / 8) * dv + row) * 8;
                    put_state<H>(s, ws.shi + to, ws.slo + to, (size_t)dv * 8, dk - wg * H);
                }
            }
            if (c == chunks) break;
            // X = V - e^G K S, and beta X as an operand; x holds X, with kBack e^G K S
            const unsigned char* st = sm + (c & 1) * L::BYTES;
            const float* vec = reinterpret_cast<const float*>(st + L::VECS) + 32 * wg;
            float x[32], y[32];
            chain_wait(bars, &bars.full[c & 1], (c >> 1) & 1);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = tile_value(st + L::V, 32 * wg + i, row);
            if (transition) {
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = 0.f;
            }
            chain_wait(bars, &bars.m1, c & 1);
            tc::tc_fence_after();
            tc::tmem_ld32<32>(tl + TM_ACC + 32 * wg, x);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 eg = *reinterpret_cast<const float4*>(vec + VEC_EG + i), bt = *reinterpret_cast<const float4*>(vec + VEC_BETA + i);
                fma2(y[i], y[i + 1], x[i], x[i + 1], -eg.x, -eg.y);
                fma2(y[i + 2], y[i + 3], x[i + 2], x[i + 3], -eg.z, -eg.w);
                if constexpr (kBack) {
                    mul2(x[i], x[i + 1], eg.x, eg.y);
                    mul2(x[i + 2], x[i + 3], eg.z, eg.w);
                } else {
                    x[i] = y[i]; x[i + 1] = y[i + 1]; x[i + 2] = y[i + 2]; x[i + 3] = y[i + 3];
                }
                mul2(y[i], y[i + 1], bt.x, bt.y);
                mul2(y[i + 2], y[i + 3], bt.z, bt.w);
            }
            {
                const uint32_t to[2] = {tl + TM_X + 32 * wg, tl + TM_X + 32 * wg + 16};
                put_terms<2>(y, to);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.x);
            // W, U; the operands U' = e^{G_C - G} U and U. For the backward pass d = V - W is formed first, from
            // what it consists of: it falls with the decay, and a difference of V and W would keep V's rounding.
            chain_wait(bars, &bars.m2, c & 1);
            tc::tc_fence_after();
#pragma unroll
            for (int k = 0; k < 128; k += 64) {
                tc::tmem_ld32<32>(tl + TM_UZ + k + 32 * wg, y);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    if constexpr (kBack) fma2(x[i], x[i + 1], y[i], y[i + 1], -1.f, -1.f);
                    else add2(x[i], x[i + 1], y[i], y[i + 1]);
                }
            }
            const size_t wh = (size_t)(slot0 + c) * Hv + h;
            if constexpr (kBack) {
                if (live) {
                    float4* dp = reinterpret_cast<float4*>(ws.d + wh * 64 * dv) + (size_t)(8 * wg) * dv + row;
#pragma unroll
                    for (int i = 0; i < 8; ++i) dp[i * dv] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float w0 = tile_value(st + L::V, 32 * wg + i, row), w1 = tile_value(st + L::V, 32 * wg + i + 1, row);
                    fma2(w0, w1, x[i], x[i + 1], -1.f, -1.f);
                    x[i] = w0;
                    x[i + 1] = w1;
                }
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 bt = *reinterpret_cast<const float4*>(vec + VEC_BETA + i), dc = *reinterpret_cast<const float4*>(vec + VEC_DEC + i);
                mul2(x[i], x[i + 1], bt.x, bt.y);
                mul2(x[i + 2], x[i + 3], bt.z, bt.w);
                y[i] = x[i]; y[i + 1] = x[i + 1]; y[i + 2] = x[i + 2]; y[i + 3] = x[i + 3];
                mul2(y[i], y[i + 1], dc.x, dc.y);
                mul2(y[i + 2], y[i + 3], dc.z, dc.w);
            }
            if constexpr (kBack) {
                const uint32_t to[3] = {tl + TM_UZ + 32 * wg, tl + TM_UZ + 32 * wg + 16, tl + TM_X + 32 * wg};
                put_terms<3>(y, to);
            } else {
                const uint32_t to[2] = {tl + TM_UZ + 32 * wg, tl + TM_UZ + 32 * wg + 16};
                put_terms<2>(y, to);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.u);
            {
                const uint32_t to[2] = {tl + TM_UZ + 64 + 32 * wg, tl + TM_UZ + 64 + 32 * wg + 16};
                put_terms<2>(x, to);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.uo);
            if constexpr (kBack) {
                if (live) {
                    __nv_bfloat16* up = ws.u + wh * 64 * dv + (size_t)(32 * wg) * dv + row;
#pragma unroll
                    for (int i = 0; i < 32; ++i) up[i * dv] = __float2bfloat16_rn(x[i]);
                }
            }
        }
        if constexpr (!kBack) {
            if (to != nullptr && live) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int d = wg * H + i;
                    if (d < dk) to[transition ? (size_t)row * dk + d : (size_t)d * dv + row] = s[i];
                }
            }
        }
    }
    chain_end(bars);
}

// The states between segments from their maps, fp32, one segment after the other.
// Prefix: the state behind every segment but the last, S_j = M_j S_{j-1} + N_j, in place of N_j.
// Suffix: the cotangent of the state before every segment but the first, D_j = M_j^T D_{j+1} + N'_j, in
// place of N'_j. A CTA of 256 threads takes 16 columns of one (sequence, head), a thread one row and
// 8 columns; the next map comes while one is multiplied (2 us a segment; read in the loop it was 10).
constexpr int kScanLd = 132;                   // floats in a row of a map: 16-byte reads of 8 rows side by side meet no bank twice
constexpr size_t kScanSmem = (2 * 128 * kScanLd + 128 * 16) * sizeof(float);
template <bool kSuffix>
__global__ void __launch_bounds__(256)
segment_scan_kernel(SegArgs sg, Seqs seqs, int Hv, int dk, int dv) {
    extern __shared__ __align__(16) float scan[];
    float* S = scan + 2 * 128 * kScanLd;       // [128][16]
    const int n = blockIdx.x / Hv, h = blockIdx.x % Hv, i = threadIdx.x & 127, j0 = (threadIdx.x >> 7) * 8, c0 = blockIdx.y * 16 + j0;
    int start, len;
    bool ok;
    seqs.get(n, start, len, ok);
    const int first = sg.first_place(n, start), count = (len + sg.cps * C - 1) / (sg.cps * C);
    const size_t mat = (size_t)dk * dv;
    float* places = kSuffix ? sg.dstates : sg.states;
    next_may_start();
    previous_done();
    auto own = [&](int step) { return (size_t)(first + (kSuffix ? count - 1 - step : step)) * Hv + h; };
    auto fetch = [&](int step) {
        const float* from = sg.maps + own(step) * dk * dk;
        const uint32_t to = s32(scan + (step & 1) * 128 * kScanLd);
        for (int e = threadIdx.x; e < dk * (dk / 4); e += 256) {
            const int r = e / (dk / 4), x = e % (dk / 4);
            cp16(to + (r * kScanLd + 4 * x) * 4, from + (size_t)r * dk + 4 * x, true);
        }
    };
    for (int step = 0; step < count - 1; ++step) {
        float* st = places + own(step) * mat + (size_t)i * dv + c0;
        const bool live = i < dk && c0 < dv;   // dv is a multiple of 8
        float4 add[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) add[j] = live ? reinterpret_cast<const float4*>(st)[j] : make_float4(0.f, 0.f, 0.f, 0.f);
        if (step + 1 < count - 1) fetch(step + 1);
        cp_commit();
        float acc[8] = {};
        if (step > 0) {                        // the first has its state already
            cp_wait<1>();
            __syncthreads();
            const float* M = scan + (step & 1) * 128 * kScanLd;
#pragma unroll 4
            for (int d = 0; d < dk; d += 4) {
                float m[4];
                if constexpr (kSuffix) {
                    const float4 x = *reinterpret_cast<const float4*>(M + i * kScanLd + d);
                    m[0] = x.x; m[1] = x.y; m[2] = x.z; m[3] = x.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[e] = M[(d + e) * kScanLd + i];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(S + (d + e) * 16 + j0 + j);
                        fma2(acc[j], acc[j + 1], m[e], m[e], x.x, x.y);
                        fma2(acc[j + 2], acc[j + 3], m[e], m[e], x.z, x.w);
                    }
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 x = make_float4(acc[4 * j] + add[j].x, acc[4 * j + 1] + add[j].y, acc[4 * j + 2] + add[j].z, acc[4 * j + 3] + add[j].w);
            *reinterpret_cast<float4*>(S + i * 16 + j0 + 4 * j) = x;
            if (step > 0 && live) reinterpret_cast<float4*>(st)[j] = x;
        }
        __syncthreads();
    }
    cp_wait<0>();
}

// Results from the last (or first) segments' places to where they belong.
__global__ void __launch_bounds__(256)
segment_result_kernel(SegArgs sg, Seqs seqs, const float* __restrict__ places, bool first, float* __restrict__ result, int Hv, int mat) {
    const int n = blockIdx.x / Hv, h = blockIdx.x % Hv;
    int start, len;
    bool ok;
    seqs.get(n, start, len, ok);
    const int place = sg.first_place(n, start) + (first ? 0 : max((len + sg.cps * C - 1) / (sg.cps * C) - 1, 0));
    previous_done();
    const float4* from = reinterpret_cast<const float4*>(places + ((size_t)place * Hv + h) * mat);
    float4* to = reinterpret_cast<float4*>(result + (size_t)blockIdx.x * mat);
    for (int i = threadIdx.x; i < mat / 4; i += 256) to[i] = from[i];
}

// The adjoint chain, chunks last to first, dS the cotangent of the state leaving a chunk:
//   dU = P^T dO + e^{G_C - G} (.) K dS,   y = dU + Z^T (beta dU),   dV = beta y
//   dS <- e^{G_C} dS + Q^T (e^G (.) dO) - K^T (e^G (.) dV)
// and the sums that the gradients of beta and g need (see gated_grads.cuh): w.y and what a token's
// future takes from it, <S', dS> per chunk. P comes without its diagonal, whose part of dU and y,
// q_i.k_i dO_i, is added where the whole is needed. The layout and roles of the forward chain; the out
// warps prepare the operand e^G dO and take y from TMEM for dV and the sums. The products that do not
// wait for dS (P^T dO, Q^T dO) run under the epilogues; the operands of the update carry three terms.
// Measured as the forward chain: 592 us (541 with the own part inside y, which left dg without digits under
// strong gates); the out warps' operand, rows and sums over lanes take all of a chunk's 17000 cycles, and
// 1.9 GB of states and sums are moved (44% of the bandwidth).
template <int DK>
__global__ void __launch_bounds__(kChainThreads, 1)
chain_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                 const __grid_constant__ CUtensorMap mo, const ChainIn in, const float* dST, __nv_bfloat16* __restrict__ grad_v,
                 float* grad_S0, ChunkWs ws, Seqs seqs, SegArgs sg, int Hk, int Hv, int dk, int dv) {
    using L = ChainStage<DK, true>;
    constexpr int H = DK / 2;
    next_may_start();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ ChainBars bars;
    const int h = blockIdx.x % Hv, hk = h / (Hv / Hk), place = blockIdx.x / Hv;
    const int n = sg.mode ? sg.find(seqs, place) : (sg.longest_first ? by_length(seqs, place, reinterpret_cast<int*>(sm)) : place);
    const bool maps = sg.mode == kSegMaps;     // the cotangent alone
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int start, len;
    bool ok;
    seqs.get(n, start, len, ok);
    int slot0 = seqs.first_slot(n, start);
    const int strips = (dv + 31) / 32;
    const size_t mat = (size_t)dk * dv, sbase = ((size_t)n * Hv + h) * mat;
    const float* from = dST == nullptr ? nullptr : dST + sbase;        // the cotangent of the leaving state
    float* to = grad_S0 == nullptr ? nullptr : grad_S0 + sbase;        // where that of the entering state goes
    if (sg.mode) {                             // this segment's chunks, as a sequence of their own
        const int j = place - sg.first_place(n, start), skip = j * sg.cps;
        if (j < 0 || (j > 0 && (long long)skip * C >= len) || (maps && j == 0)) return previous_done();
        const bool last = (long long)(skip + sg.cps) * C >= len;
        const size_t own = (size_t)place * Hv + h;
        if (!last) from = maps ? nullptr : sg.dstates + (own + Hv) * mat;
        if (maps || (j == 0 && sg.apart)) to = sg.dstates + own * mat;
        else if (j > 0) to = nullptr;
        slot0 += skip;
        start += skip * C;
        len = last ? len - skip * C : sg.cps * C;
    }
    const int chunks = (len + C - 1) / C;
    chain_begin(bars, sm, 2 * L::BYTES, kOutWarps);
    const uint32_t tm = bars.tmem, base = s32(sm);

    if (warp >= kMmaWarp) {
        set_regs<kRegOther>();
        if (warp > kMmaWarp) {                 // ------------------------------------------ loads
            const int x = threadIdx.x - 32 * (kMmaWarp + 1);
#pragma unroll 1
            for (int it = 0; it < chunks; ++it) {
                const int c = chunks - 1 - it;
                if (x == 32 && !maps) {        // what the epilogues read straight from memory, into L2
                    const size_t wh = (size_t)(slot0 + c) * Hv + h;
                    tc::prefetch_l2_bulk(ws.shi + (wh + (it ? 0 : Hv)) * mat, (uint32_t)(mat * 2));
                    tc::prefetch_l2_bulk(ws.slo + (wh + (it ? 0 : Hv)) * mat, (uint32_t)(mat * 2));
                    tc::prefetch_l2_bulk(ws.d + wh * 64 * dv, (uint32_t)(64 * dv * 4));
                }
                if (it >= 2) chain_wait(bars, &bars.empty[it & 1], ((it >> 1) - 1) & 1);
                chain_load<L, DK, true>(base + (it & 1) * L::BYTES, &bars.full[it & 1], x, in, &mq, &mk, &mv, &mo, ws,
                                     (size_t)(slot0 + c) * Hv + h, start + c * C, min(C, len - c * C), h, hk, Hv, dk, dv);
            }
        } else {                               // ------------------------------------------ products
            constexpr uint32_t iE = tc::idesc_bf16(128, 64, 1, 1), iK = tc::idesc_bf16(128, 64, 0, 0),
                               iZ = tc::idesc_bf16(128, 128, 0, 1), iZ64 = tc::idesc_bf16(128, 64, 0, 1),
                               iS = tc::idesc_bf16(128, DK, 0, 1);
#pragma unroll 1
            for (int it = 0; it < chunks; ++it) {
                const uint32_t st = fresh(base + (it & 1) * L::BYTES), ph = it & 1;
                chain_wait(bars, &bars.full[it & 1], (it >> 1) & 1);
                if (it > 0) chain_wait(bars, &bars.m3, (it - 1) & 1);
                tc::tc_fence_after();
                if (elected()) {
#pragma unroll
                    for (int term = 1; term >= 0; --term)              // P^T dO, both terms of P
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            tc::mma_ss(tm + TM_PU, tc::sdesc(st + L::DO + j * 2048, 8192, 1024),
                                       tc::sdesc(st + L::P + term * 8192 + j * 2048, 8192, 1024), iE, term == 0 || j != 0);
                }
#pragma unroll
                for (int b = 0; b < H / 32; ++b) {                     // K dS, 32 channels of either half at a time
                    chain_wait(bars, &bars.s[b], ph);
                    tc::tc_fence_after();
                    if (elected()) {
#pragma unroll
                        for (int e = 0; e < 12; ++e) {                 // term, half, 16 channels
                            const int term = e / 4, half = (e / 2) % 2, ch = half * H + 32 * b + 16 * (e % 2);
                            const uint32_t a = term < 2 ? TM_S + half * H + 32 * b + 16 * term : TM_X + half * (H / 2) + 16 * b;
                            tc::mma_ts(tm + TM_ACC, tm + a + 8 * (e % 2), tc::sdesc(st + L::KQ + (ch / 64) * 16384 + (ch % 64) * 2, 16, 1024),
                                       iK, (b | e) != 0);
                        }
                        if (b == H / 32 - 1) tc::mma_commit(&bars.m1);
                    }
                }
                if (it > 0) chain_wait(bars, &bars.out, (it - 1) & 1);   // y of the chunk before is read
                chain_wait(bars, &bars.x, ph);
                tc::tc_fence_after();
                if (elected()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)                        // beta dU [Z_hi | Z_lo], transposed
                        tc::mma_ts(tm + TM_UZ, tm + TM_X + (j / 2) * 32 + (j % 2) * 8, tc::sdesc(st + L::Z + j * 2048, 8192, 1024), iZ, j != 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tc::mma_ts(tm + TM_UZ, tm + TM_X + (j / 2) * 32 + 16 + (j % 2) * 8, tc::sdesc(st + L::Z + j * 2048, 8192, 1024), iZ64, 1);
                    tc::mma_commit(&bars.m2);
                }
                chain_wait(bars, &bars.d, ph);
                tc::tc_fence_after();
                if (elected()) {
#pragma unroll
                    for (int term = 0; term < 3; ++term)               // Q^T (e^G dO)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t a = (term < 2 ? TM_ACC + term * 16 : TM_PU) + (j / 2) * 32 + (j % 2) * 8;
                            tc::mma_ts(tm + TM_S, tm + a, tc::sdesc(st + L::KQ + 8192 + j * 2048, 16384, 1024), iS, (term | j) != 0);
                        }
                }
                chain_wait(bars, &bars.u, ph);
                tc::tc_fence_after();
                if (elected()) {
#pragma unroll
                    for (int term = 0; term < 3; ++term)               // - K^T (e^G dV)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t a = TM_UZ + (term < 2 ? term * 16 : 64) + (j / 2) * 32 + (j % 2) * 8;
                            tc::mma_ts(tm + TM_S, tm + a, tc::sdesc(st + L::KQ + j * 2048, 16384, 1024), iS, 1);
                        }
                    tc::mma_commit(&bars.m3);
                    tc::mma_commit(&bars.empty[it & 1]);
                }
            }
            if (chunks > 0) chain_wait(bars, &bars.m3, (chunks - 1) & 1);
        }
    } else if (warp >= kEpiWarps) {            // ------------------------------------------ e^G dO; dV and sums over y
        set_regs<kRegOut>();
        const int quarter = warp & 3, row = 32 * quarter + lane, x = threadIdx.x - 32 * kEpiWarps;
        const bool live = row < dv;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        unsigned char* tile = sm + L::OUT;
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            const int c = chunks - 1 - it, tok = start + c * C, nt = min(C, len - c * C);
            const unsigned char* st = sm + (it & 1) * L::BYTES;
            const float* vec = reinterpret_cast<const float*>(st + L::VECS);
            const size_t wh = (size_t)(slot0 + c) * Hv + h;
            float* part = ws.parts + (wh * strips + quarter) * PARTS;
            chain_wait(bars, &bars.full[it & 1], (it >> 1) & 1);
            chain_wait(bars, &bars.x, it & 1);                     // K dS and P^T dO are read: their columns are free
            tc::tc_fence_after();
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                float e[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 eg = *reinterpret_cast<const float4*>(vec + VEC_EG + 32 * half + i);
                    e[i] = eg.x * tile_value(st + L::DO, 32 * half + i, row);
                    e[i + 1] = eg.y * tile_value(st + L::DO, 32 * half + i + 1, row);
                    e[i + 2] = eg.z * tile_value(st + L::DO, 32 * half + i + 2, row);
                    e[i + 3] = eg.w * tile_value(st + L::DO, 32 * half + i + 3, row);
                }
                const uint32_t to[3] = {tl + TM_ACC + 32 * half, tl + TM_ACC + 32 * half + 16, tl + TM_PU + 32 * half};
                put_terms<3>(e, to);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.d);
            if (maps) {                                            // nobody reads y
                chain_wait(bars, &bars.u, it & 1);
                tc::mbar_arrive(&bars.out);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.empty[it & 1]);
                continue;
            }
            float d[32];
            const float4* dp = reinterpret_cast<const float4*>(ws.d + wh * 64 * dv) + (live ? row : 0);
            auto load_d = [&](int half) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 a = live ? dp[(size_t)(8 * half + i) * dv] : make_float4(0.f, 0.f, 0.f, 0.f);
                    d[4 * i] = a.x; d[4 * i + 1] = a.y; d[4 * i + 2] = a.z; d[4 * i + 3] = a.w;
                }
            };
            load_d(0);
            chain_wait(bars, &bars.u, it & 1);
            tc::tc_fence_after();
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                float y[32];
                tc::tmem_ld32<32>(tl + TM_ACC + 64 + 32 * half, y);
                tc::tmem_ld_wait();
                if (half == 1) {
                    tc::tc_fence_before();
                    tc::mbar_arrive(&bars.out);
                }
                // y arrives without the token's own dO; w = V - d
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const int t = 32 * half + i;
                    const float2 b = *reinterpret_cast<const float2*>(vec + VEC_BETA + t), p = *reinterpret_cast<const float2*>(vec + VEC_PD + t);
                    float w0 = tile_value(st + L::V, t, row), w1 = tile_value(st + L::V, t + 1, row), a0 = y[i], a1 = y[i + 1];
                    fma2(w0, w1, d[i], d[i + 1], -1.f, -1.f);
                    fma2(a0, a1, p.x, p.y, tile_value(st + L::DO, t, row), tile_value(st + L::DO, t + 1, row));
                    *reinterpret_cast<__nv_bfloat16*>(tile + t * 256 + 2 * row) = __float2bfloat16_rn(b.x * a0);
                    *reinterpret_cast<__nv_bfloat16*>(tile + (t + 1) * 256 + 2 * row) = __float2bfloat16_rn(b.y * a1);
                    mul2(y[i], y[i + 1], w0, w1);
                    fma2(y[i], y[i + 1], a0, a1, d[i], d[i + 1]);
                    mul2(a0, a1, w0, w1);
                    d[i] = a0;
                    d[i + 1] = a1;
                }
                const float db = lane_sums(d);
                if (quarter < strips) part[PART_DB + 32 * half + lane] = db;
                if (half == 0) load_d(1);
                const float future = vec[VEC_BETA + 32 * half + lane] * lane_sums(y);
                if (quarter < strips) part[PART_FUTURE + 32 * half + lane] = future;
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars.empty[it & 1]);
            out_sync();
            rows_out(tile, x, grad_v + ((size_t)tok * Hv + h) * dv, (long long)Hv * dv, nt, dv);
            out_sync();
        }
    } else {                                   // ------------------------------------------ epilogues of the chain
        set_regs<kRegEpi>();
        const int quarter = warp & 3, wg = warp >> 2, row = 32 * quarter + lane;
        const bool live = row < dv;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        float s[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int d = wg * H + i;
            s[i] = (from != nullptr && live && d < dk) ? from[(size_t)d * dv + row] : 0.f;
        }
#pragma unroll 1
        for (int it = 0; it <= chunks; ++it) {
            const int c = chunks - 1 - it;
            // the state behind the chunk (after the first chunk: before it), asked for while the update's
            // product runs
            uint4 sh[H / 8], sl[H / 8];
            const size_t next = ((size_t)(slot0 + c + 1) * Hv + h) * mat + ((size_t)(wg * H / 8) * dv + row) * 8;
#pragma unroll
            for (int i = 0; i < H / 8; ++i) {
                const bool in = live && chunks > 0 && !maps && wg * H + 8 * i < dk;
                sh[i] = in ? *reinterpret_cast<const uint4*>(ws.shi + next + (size_t)i * dv * 8) : make_uint4(0, 0, 0, 0);
                sl[i] = in ? *reinterpret_cast<const uint4*>(ws.slo + next + (size_t)i * dv * 8) : make_uint4(0, 0, 0, 0);
            }
            if (it > 0) {                      // dS <- e^{G_C} dS + update
                const float whole = reinterpret_cast<const float*>(sm + ((it - 1) & 1) * L::BYTES + L::VECS)[VEC_EG + 63];
                chain_wait(bars, &bars.m3, (it - 1) & 1);
                tc::tc_fence_after();
                next_state<3, H, 16>(s, whole, false, it < chunks, tl, wg, bars);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.empty[(it - 1) & 1]);
            } else {
                next_state<3, H, 16>(s, 1.f, true, it < chunks, tl, wg, bars);
            }
            // <S', dS>, and dS itself for the gradients of k
            if (quarter < strips && chunks > 0 && !maps) {
                float dot0 = 0.f, dot1 = 0.f;
#pragma unroll
                for (int i = 0; i < H / 8; ++i) {
                    const uint32_t hi[4] = {sh[i].x, sh[i].y, sh[i].z, sh[i].w}, lo[4] = {sl[i].x, sl[i].y, sl[i].z, sl[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        fma2(dot0, dot1, state_lo(hi[j], lo[j]), state_hi(hi[j], lo[j]), s[8 * i + 2 * j], s[8 * i + 2 * j + 1]);
                    if (it < chunks && live && wg * H + 8 * i < dk)
                        *reinterpret_cast<uint4*>(ws.dshi + next - Hv * mat + (size_t)i * dv * 8) =
                            make_uint4(pack2(s[8 * i], s[8 * i + 1]), pack2(s[8 * i + 2], s[8 * i + 3]), pack2(s[8 * i + 4], s[8 * i + 5]),
                                       pack2(s[8 * i + 6], s[8 * i + 7]));
                }
                float dot = dot0 + dot1;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
                if (lane == 0)
                    ws.parts[((((size_t)slot0 + max(c, 0)) * Hv + h) * strips + quarter) * PARTS + (it < chunks ? PART_SDS : PART_SDS0) + wg] = dot;
            }
            if (it == chunks) break;
            // dU without the token's own dO (P here has no diagonal) in x, and beta dU as an operand
            const unsigned char* st = sm + (it & 1) * L::BYTES;
            const float* vec = reinterpret_cast<const float*>(st + L::VECS) + 32 * wg;
            float x[32], y[32];
            auto add_own = [&](const unsigned char* stage, int i, float& z0, float& z1) {      // tokens i and i + 1
                const float2 p = *reinterpret_cast<const float2*>(stage + L::VECS + 4 * (32 * wg + VEC_PD + i));
                fma2(z0, z1, p.x, p.y, tile_value(stage + L::DO, 32 * wg + i, row), tile_value(stage + L::DO, 32 * wg + i + 1, row));
            };
            chain_wait(bars, &bars.full[it & 1], (it >> 1) & 1);
            chain_wait(bars, &bars.m1, it & 1);
            tc::tc_fence_after();
            tc::tmem_ld32<32>(tl + TM_ACC + 32 * wg, x);
            tc::tmem_ld32<32>(tl + TM_PU + 32 * wg, y);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 dc = *reinterpret_cast<const float4*>(vec + VEC_DEC + i), bt = *reinterpret_cast<const float4*>(vec + VEC_BETA + i);
                fma2(y[i], y[i + 1], dc.x, dc.y, x[i], x[i + 1]);
                fma2(y[i + 2], y[i + 3], dc.z, dc.w, x[i + 2], x[i + 3]);
                x[i] = y[i]; x[i + 1] = y[i + 1]; x[i + 2] = y[i + 2]; x[i + 3] = y[i + 3];
                add_own(st, i, y[i], y[i + 1]);
                add_own(st, i + 2, y[i + 2], y[i + 3]);
                mul2(y[i], y[i + 1], bt.x, bt.y);
                mul2(y[i + 2], y[i + 3], bt.z, bt.w);
            }
            {
                const uint32_t to[2] = {tl + TM_X + 32 * wg, tl + TM_X + 32 * wg + 16};
                put_terms<2>(y, to);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.x);
            // y without the token's own dO (to TMEM for the out warps), and - e^G dV as an operand
            chain_wait(bars, &bars.m2, it & 1);
            tc::tc_fence_after();
            st = sm + fresh((it & 1) * L::BYTES);  // the own parts are read again: kept from above they would spill
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                float e[8], z[8];
                uint32_t r[8];
                tc::tmem_ld32<8>(tl + TM_UZ + 32 * wg + k, e);
                tc::tmem_ld32<8>(tl + TM_UZ + 64 + 32 * wg + k, z);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[k + i] += e[i] + z[i];
                    r[i] = __float_as_uint(x[k + i]);
                }
                tc::tmem_st32<8>(tl + TM_ACC + 64 + 32 * wg + k, r);
#pragma unroll
                for (int i = k; i < k + 8; i += 4) {
                    const float4 bt = *reinterpret_cast<const float4*>(vec + VEC_BETA + i), eg = *reinterpret_cast<const float4*>(vec + VEC_EG + i);
                    add_own(st, i, x[i], x[i + 1]);
                    add_own(st, i + 2, x[i + 2], x[i + 3]);
                    mul2(x[i], x[i + 1], -eg.x * bt.x, -eg.y * bt.y);
                    mul2(x[i + 2], x[i + 3], -eg.z * bt.z, -eg.w * bt.w);
                }
            }
            {
                const uint32_t to[3] = {tl + TM_UZ + 32 * wg, tl + TM_UZ + 32 * wg + 16, tl + TM_UZ + 64 + 32 * wg};
                put_terms<3>(x, to);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars.u);
        }
        if (to != nullptr && live) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int d = wg * H + i;
                if (d < dk) to[(size_t)d * dv + row] = s[i];
            }
        }
    }
    chain_end(bars);
}

}  // namespace gated
}  // namespace ckda
