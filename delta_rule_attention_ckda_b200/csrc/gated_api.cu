// Host side of the scalar-gate operators of the C ABI (see include/ckda.h): the gated delta
// rule with one decay per head (chunked forward, backward, single-token step on a pool of
// states), the preparation of queries and keys, and copies of states within a pool.
// Argument validation, path selection, workspace layout and launches.
#include "ckda.h"

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "kernels/gated_common.cuh"
#include "kernels/gated_simt.cuh"
#include "kernels/gated_decode.cuh"
#include "kernels/gated_intra.cuh"
#include "kernels/gated_chain.cuh"
#include "kernels/gated_grads.cuh"
#include "kernels/tc_host.cuh"
#include "kernels/qk_prep.cuh"
#include "kernels/state_copy.cuh"

namespace {

using namespace ckda::gated;
typedef __nv_bfloat16 bf16;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }   // indexes, gates
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline ckda_status_t launch_status() { return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA; }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

int sm_count() {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kDevices) {
        n = known[dev].load(std::memory_order_relaxed);
        if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) known[dev].store(n);
    }
    if (n > 0) return n;
    cudaGetLastError();                        // no device: plan for a B200
    return 148;
}

// Opt in to more than 48 KB of dynamic shared memory, once per kernel and device (a kernel asks for
// the same size every time, or for the most it can use). regs != 0: the registers a thread that
// the kernel has to have been compiled to.
template <typename K>
cudaError_t kernel_ready(K kernel, size_t bytes, int regs = 0) {
    constexpr int kDevices = 64;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    struct Entry { const void* f; std::atomic<bool> done[kDevices]; };
    static Entry entries[64] = {};
    static std::mutex mu;
    const void* f = reinterpret_cast<const void*>(kernel);
    Entry* at = nullptr;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (Entry& x : entries)
            if (x.f == f || x.f == nullptr) {
                x.f = f;
                at = &x;
                break;
            }
    }
    if (at && dev >= 0 && dev < kDevices && at->done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    if (regs != 0) {
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, f);
        if (e != cudaSuccess) return e;
        if (a.numRegs != regs) return cudaErrorInvalidConfiguration;
    }
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && at && dev >= 0 && dev < kDevices) at->done[dev].store(true, std::memory_order_release);
    return e;
}

// A launch; `close`: it may begin before the kernel ahead of it in the stream has ended (see
// previous_done).
template <typename... P, typename... A>
cudaError_t launch_kernel(bool close, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A&&... a) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t how{};
    how.gridDim = grid;
    how.blockDim = dim3(threads);
    how.dynamicSmemBytes = smem;
    how.stream = st;
    how.attrs = &early;
    how.numAttrs = close ? 1 : 0;
    return cudaLaunchKernelEx(&how, kernel, static_cast<P>(a)...);
}

struct Shape {
    int N, T, total, Hk, Hv, dk, dv;
    ckda_dtype_t dt;
};

ckda_status_t check_shape(const Shape& s, bool packed) {
    if (s.N < 0 || s.T < 0 || s.total < 0 || s.Hk < 1 || s.Hv < 1) return CKDA_ERR_INVALID_ARG;
    if (s.dk < 1 || s.dk > CKDA_MAX_D || s.dv < 1 || s.dv > CKDA_MAX_D) return CKDA_ERR_INVALID_ARG;
    if (s.dt != CKDA_F32 && s.dt != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
    if (s.Hv % s.Hk != 0) return CKDA_ERR_INVALID_ARG;
    if (!packed && (long long)s.N * s.T != s.total) return CKDA_ERR_INVALID_ARG;
    if ((long long)s.N * s.Hv > 0x7fffffffLL || (long long)s.total + (long long)s.N * C > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
    return CKDA_OK;
}

// Token strides cover at least one token's heads.
bool strides_ok(const Shape& s, long long qs, long long ks, long long vs) {
    return qs >= (long long)s.Hk * s.dk && ks >= (long long)s.Hk * s.dk && vs >= (long long)s.Hv * s.dv;
}

ckda_status_t clear_or_copy(const float* from, float* to, size_t n, cudaStream_t st) {
    if (to == nullptr || to == from || n == 0) return CKDA_OK;
    cudaError_t e = from ? cudaMemcpyAsync(to, from, n * sizeof(float), cudaMemcpyDeviceToDevice, st)
                         : cudaMemsetAsync(to, 0, n * sizeof(float), st);
    return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

template <typename TIn>
ckda_status_t simt_fwd(const Shape& s, const void* q, const void* k, const void* v, const float* g, const float* beta,
                       const float* S0, void* o, float* ST, const Seqs& seqs, const int* slots, int pool, long long qs,
                       long long ks, long long vs, cudaStream_t st) {
    const int cols = s.dv <= 32 ? 32 : (s.dv <= 64 ? 64 : 128);
    const dim3 grid((unsigned)(s.N * s.Hv), (unsigned)((s.dv + cols - 1) / cols));
#define GATED_SIMT(D)                                                                                                \
    simt_fwd_kernel<D, TIn><<<grid, cols, 0, st>>>(static_cast<const TIn*>(q), static_cast<const TIn*>(k),            \
                                                   static_cast<const TIn*>(v), g, beta, S0, static_cast<TIn*>(o), ST, \
                                                   seqs, slots, pool, s.Hk, s.Hv, s.dk, s.dv, qs, ks, vs)
    if (s.dk <= 16) GATED_SIMT(16);
    else if (s.dk <= 32) GATED_SIMT(32);
    else if (s.dk <= 64) GATED_SIMT(64);
    else GATED_SIMT(128);
#undef GATED_SIMT
    return launch_status();
}

// Workspace of the CUDA-core backward.
struct SimtBwdLayout {
    size_t ckpt, scratch, pq, pk, total;
};
SimtBwdLayout simt_bwd_layout(const Shape& s) {
    SimtBwdLayout l;
    const size_t mat = (size_t)s.dk * s.dv * sizeof(float);
    l.ckpt = 0;
    l.scratch = up256(l.ckpt + Seqs::slots(s.N, s.total) * (C / KB) * s.Hv * mat);
    l.pq = up256(l.scratch + (size_t)s.N * s.Hv * KB * mat);
    l.pk = up256(l.pq + (size_t)s.total * s.Hv * s.dk * sizeof(float));
    l.total = up256(l.pk + (size_t)s.total * s.Hv * s.dk * sizeof(float));
    return l;
}

template <typename TIn>
ckda_status_t simt_bwd(const Shape& s, const void* q, const void* k, const void* v, const float* g, const float* beta,
                       const float* S0, const void* grad_o, const float* dST, void* gq, void* gk, void* gv, float* gg,
                       float* gb, float* gS0, const Seqs& seqs, long long qs, long long ks, long long vs, char* ws,
                       cudaStream_t st) {
    const SimtBwdLayout l = simt_bwd_layout(s);
    auto F = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    if (kernel_ready(simt_bwd_kernel<TIn>, kSimtBwdSmem) != cudaSuccess) return CKDA_ERR_CUDA;
    simt_bwd_kernel<TIn><<<(unsigned)(s.N * s.Hv), NTB, kSimtBwdSmem, st>>>(
        static_cast<const TIn*>(q), static_cast<const TIn*>(k), static_cast<const TIn*>(v), g, beta, S0,
        static_cast<const TIn*>(grad_o), dST, F(l.ckpt), F(l.scratch), F(l.pq), F(l.pk), static_cast<TIn*>(gv), gg, gb,
        gS0, seqs, s.Hk, s.Hv, s.dk, s.dv, qs, ks, vs);
    if (cudaPeekAtLastError() != cudaSuccess) return launch_status();
    const size_t n = (size_t)s.total * s.Hk * s.dk;
    simt_share_kernel<TIn><<<(unsigned)std::min<size_t>((n + 255) / 256, 148 * 16), 256, 0, st>>>(
        F(l.pq), F(l.pk), static_cast<TIn*>(gq), static_cast<TIn*>(gk), seqs, s.Hk, s.Hv, s.dk);
    return launch_status();
}

// ---------------------------------------------------------------- the chunked kernels

// They take bf16 with heads of a multiple of 8 channels, whose rows have to start on 16 bytes;
// channels are padded to 64 or 128 in shared memory.
bool chunked(const Shape& s) { return s.dt == CKDA_BF16 && s.dk % 8 == 0 && s.dv % 8 == 0; }
bool rows_aligned(const Shape& s, long long qs, long long ks, long long vs) {
    return !chunked(s) || (qs % 8 == 0 && ks % 8 == 0 && vs % 8 == 0);
}
// Whether grids and row numbers of the chunked kernels hold the call.
bool chunked_fits(const Shape& s) { return s.Hk <= 65535 && (long long)Seqs::slots(s.N, s.total) * s.Hv * C <= 0x7fffffffLL; }

// Chunks in a segment (0: whole sequences run), for a call's sizes alone. Time is counted in chunks of the
// forward chain one after the other (4 us): a pass takes its waves of CTAs times a segment's chunks
// and 5 or 6 more for its start, a scan a quarter per segment; going back, the chain that keeps its
// states counts 7/4, the adjoint's two passes 6/4 and 8/4. The longest sequence is not known
// on the host: the average is taken, back, where segments pay sooner, a quarter more. A batch of one long
// and many short sequences is therefore run whole, as long as its longest takes alone. Segments have
// to gain an eighth. B200, us, whole and in segments: one sequence of 2048 tokens and 16 heads of 128,
// forward 140 and 112, backward 521 and 306; of 65536, forward 4200 and 1570; 2 of 4096, forward 290
// and 245, backward 1086 and 740; 1 of 1024, forward 83 and 89 (not taken), backward 257 and 208.
int segment_chunks(const Shape& s, bool back) {
    if (s.N == 0) return 0;
    const long long rows = (long long)s.N * s.Hv, sms = sm_count(), each = (long long)s.N * C, start = back ? 5 : 6;
    const long long average = (s.total + each - 1) / each, longest = back ? (5 * average + 3) / 4 : average;
    auto waves = [&](long long per) { return (std::max(per, 1LL) * rows + sms - 1) / sms; };
    long long best = 0, time = waves(1) * (longest + start) * (back ? 15 : 4) * 7 / 8;      // quarters of a chunk
    for (long long n = 3; n <= 32 && n * 2 <= longest; ++n) {
        const long long cps = (longest + n - 1) / n, per = (average + cps - 1) / cps;
        const long long maps = waves(2 * per - 3), run = waves(per), adjoint = waves(per - 1);
        const long long t = back ? (4 * maps + 15 * run + 6 * adjoint) * (cps + start) + 2 * n : 4 * (maps + run) * (cps + start) + n;
        if (t < time) {
            time = t;
            best = cps;
        }
    }
    return (int)best;
}

struct ChunkLayout {
    size_t zhi, zlo, phi, plo, vec, shi, slo, dshi, u, d, parts, states, maps, dstates, total;
    int cps;
};
ChunkLayout chunk_layout(const Shape& s, bool back) {
    ChunkLayout l{};
    const size_t n = Seqs::slots(s.N, s.total) * s.Hv, strips = (s.dv + 31) / 32;
    size_t at = 0;
    auto take = [&](size_t each) {
        const size_t here = at;
        at = up256(at + n * each);
        return here;
    };
    l.zhi = take(8192);
    l.zlo = take(8192);
    l.phi = take(8192);
    l.plo = take(8192);
    l.vec = take(VEC * 4);
    if (back) {
        l.shi = take((size_t)s.dk * s.dv * 2);
        l.slo = take((size_t)s.dk * s.dv * 2);
        l.dshi = take((size_t)s.dk * s.dv * 2);
        l.u = take((size_t)64 * s.dv * 2);
        l.d = take((size_t)s.dv * 64 * 4);
        l.parts = take(strips * PARTS * 4);
    }
    l.cps = segment_chunks(s, back);
    if (l.cps > 0) {
        const size_t places = SegArgs::places(s.N, s.total, l.cps) * s.Hv;
        l.states = at;
        l.maps = l.states + up256(places * s.dk * s.dv * 4);
        l.dstates = l.maps + up256(places * s.dk * s.dk * 4);
        at = l.dstates + (back ? up256(places * s.dk * s.dv * 4) : 0);
    }
    l.total = at;
    return l;
}
ChunkWs chunk_ws(const ChunkLayout& l, void* base) {
    char* b = static_cast<char*>(base);
    auto H = [&](size_t at) { return reinterpret_cast<bf16*>(b + at); };
    auto F = [&](size_t at) { return reinterpret_cast<float*>(b + at); };
    return ChunkWs{H(l.zhi), H(l.zlo), H(l.phi), H(l.plo), F(l.vec), H(l.shi), H(l.slo), H(l.dshi), H(l.u), F(l.d), F(l.parts)};
}

SegArgs segments(const ChunkLayout& l, void* base, const Shape& s, bool packed) {
    char* b = static_cast<char*>(base);
    auto F = [&](size_t at) { return reinterpret_cast<float*>(b + at); };
    const int ranked = packed && l.cps == 0 && s.N <= kMaxRanked && (long long)s.N * s.Hv > sm_count();
    return SegArgs{kSegWhole, l.cps, ranked, 0, F(l.states), F(l.maps), F(l.dstates)};
}

struct Call {
    Shape s;
    Seqs seqs;
    const bf16 *q, *k, *v, *grad_o;
    const float *g, *beta, *S0, *dST;
    bf16 *o, *gq, *gk, *gv;
    float *ST, *gg, *gb, *gS0;
    long long qs, ks, vs;
    ChunkWs ws;
    SegArgs seg;
    cudaStream_t st;
};

// Tensor map over [tokens][heads][channels] rows a token stride apart, boxes of 64 channels of one
// head of 64 tokens, 128-byte swizzle; channels beyond the head read as zeros.
bool rows_map(CUtensorMap* map, const bf16* base, long long tokens, int heads, int d, long long stride) {
    auto fn = ckda::tc::encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64u, 1u, 64u}, each[3] = {1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16*>(base), dims, strides, box, each,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap q, k, v, o;
};

template <int DK, bool kBack>
cudaError_t run_intra(const Call& c, const Maps& m, const ChainIn& in) {
    constexpr size_t smem = intra_smem(DK);
    cudaError_t e = kernel_ready(intra_kernel<DK, kBack>, smem);
    if (e != cudaSuccess) return e;
    intra_kernel<DK, kBack><<<dim3((unsigned)Seqs::slots(c.s.N, c.s.total), (unsigned)c.s.Hk), 128, smem, c.st>>>(
        m.q, m.k, in, c.g, c.beta, c.ws, c.seqs, c.s.Hk, c.s.Hv, c.s.dk);
    return cudaPeekAtLastError();
}

// Short calls, whose kernels are about as long as the gaps between them, are launched closely: up to two
// chunks an SM. 2777 tokens of 4 heads back 169 us apart and 154 so, 512 of 4 forward 50 and 46; 1024
// of 16 as long; 8 x 4096 of 16 436 and 448, the chains' blocks lying where others ended first.
bool close(const Shape& s) { return (long long)Seqs::slots(s.N, s.total) * s.Hv <= 2LL * sm_count(); }

template <bool kSuffix>
cudaError_t run_scan(const Call& c, const SegArgs& sg) {
    cudaError_t e = kernel_ready(segment_scan_kernel<kSuffix>, kScanSmem);
    if (e != cudaSuccess) return e;
    return launch_kernel(close(c.s), segment_scan_kernel<kSuffix>, dim3((unsigned)(c.s.N * c.s.Hv), (unsigned)((c.s.dv + 15) / 16)), 256, kScanSmem, c.st,
                        sg, c.seqs, c.s.Hv, c.s.dk, c.s.dv);
}

template <int DK, bool kBack>
cudaError_t run_chain_fwd(const Call& c, const Maps& m, const ChainIn& in) {
    constexpr size_t smem = ChainStage<DK, kBack>::SMEM;
    // the register split between warps adds up only against the count it was compiled to
    cudaError_t e = kernel_ready(chain_fwd_kernel<DK, kBack>, smem, kRegLaunch);
    if (e != cudaSuccess) return e;
    SegArgs sg = c.seg;
    const unsigned seqs = (unsigned)(c.s.N * c.s.Hv);
    auto run = [&](unsigned grid) {
        return launch_kernel(close(c.s), chain_fwd_kernel<DK, kBack>, grid, kChainThreads, smem, c.st, m.q, m.k, m.v, m.o, in, c.S0, c.o, c.ST, c.ws,
                            c.seqs, sg, c.s.Hk, c.s.Hv, c.s.dk, c.s.dv);
    };
    if (sg.cps == 0) return run(seqs);
    const unsigned places = (unsigned)(SegArgs::places(c.s.N, c.s.total, sg.cps) * c.s.Hv);
    constexpr size_t maps_smem = ChainStage<DK, false>::SMEM;
    e = kernel_ready(chain_fwd_kernel<DK, false>, maps_smem, kRegLaunch);
    if (e != cudaSuccess) return e;
    sg.mode = kSegMaps;
    e = launch_kernel(close(c.s), chain_fwd_kernel<DK, false>, dim3(places, 2), kChainThreads, maps_smem, c.st, m.q, m.k, m.v, m.o, in, c.S0, c.o, c.ST,
                     c.ws, c.seqs, sg, c.s.Hk, c.s.Hv, c.s.dk, c.s.dv);
    if (e == cudaSuccess) e = run_scan<false>(c, sg);
    if (e != cudaSuccess) return e;
    sg.mode = kSegRun;
    sg.apart = c.ST != nullptr && c.ST == c.S0;
    e = run(places);
    if (e != cudaSuccess || !sg.apart) return e;
    return launch_kernel(close(c.s), segment_result_kernel, seqs, 256, 0, c.st, sg, c.seqs, sg.states, false, c.ST, c.s.Hv, c.s.dk * c.s.dv);
}
template <int DK>
cudaError_t run_chain_bwd(const Call& c, const Maps& m, const ChainIn& in) {
    constexpr size_t smem = ChainStage<DK, true>::SMEM;
    cudaError_t e = kernel_ready(chain_bwd_kernel<DK>, smem, kRegLaunch);
    if (e != cudaSuccess) return e;
    SegArgs sg = c.seg;
    const unsigned seqs = (unsigned)(c.s.N * c.s.Hv);
    auto run = [&](unsigned grid) {
        return launch_kernel(close(c.s), chain_bwd_kernel<DK>, grid, kChainThreads, smem, c.st, m.q, m.k, m.v, m.o, in, c.dST, c.gv, c.gS0, c.ws, c.seqs,
                            sg, c.s.Hk, c.s.Hv, c.s.dk, c.s.dv);
    };
    if (sg.cps == 0) return run(seqs);
    const unsigned places = (unsigned)(SegArgs::places(c.s.N, c.s.total, sg.cps) * c.s.Hv);
    sg.mode = kSegMaps;
    e = run(places);
    if (e != cudaSuccess) return e;
    e = run_scan<true>(c, sg);
    if (e != cudaSuccess) return e;
    sg.mode = kSegRun;
    sg.apart = c.gS0 != nullptr && c.gS0 == c.dST;
    e = run(places);
    if (e != cudaSuccess || !sg.apart) return e;
    return launch_kernel(close(c.s), segment_result_kernel, seqs, 256, 0, c.st, sg, c.seqs, sg.dstates, true, c.gS0, c.s.Hv, c.s.dk * c.s.dv);
}
template <int DK, int DV>
cudaError_t run_grads(const Call& c, const Maps& m, const ChainIn& in) {
    constexpr size_t smem = GradSmem<DK, DV>::BYTES;
    cudaError_t e = kernel_ready(grad_kernel<DK, DV>, smem);
    if (e != cudaSuccess) return e;
    const long long slots = (long long)Seqs::slots(c.s.N, c.s.total), items = slots * c.s.Hk;
    CUtensorMap gv{}, u{};
    if (in.maps && !(rows_map(&gv, c.gv, c.s.total, c.s.Hv, c.s.dv, (long long)c.s.Hv * c.s.dv) &&
                     rows_map(&u, c.ws.u, slots * c.s.Hv * C, 1, c.s.dv, c.s.dv)))
        return cudaErrorInvalidValue;
    return launch_kernel(close(c.s), grad_kernel<DK, DV>, (unsigned)std::min<long long>(items, sm_count()), 256, smem, c.st, m.q, m.k, m.o, gv, u, in, c.gv,
                        c.gq, c.gk, c.gg, c.gb, c.ws, c.seqs, (int)slots, c.s.Hk, c.s.Hv, c.s.dk, c.s.dv);
}

template <int DK, bool kBack>
cudaError_t run_chunked(const Call& c) {
    ChainIn in{c.q, c.k, c.v, c.grad_o, c.qs, c.ks, c.vs, c.s.dk >= 64 && c.s.dv >= 64};
    Maps m{};
    if (in.maps) {
        const bool ok = rows_map(&m.q, c.q, c.s.total, c.s.Hk, c.s.dk, c.qs) && rows_map(&m.k, c.k, c.s.total, c.s.Hk, c.s.dk, c.ks) &&
                        rows_map(&m.v, c.v, c.s.total, c.s.Hv, c.s.dv, c.vs) &&
                        (!kBack || rows_map(&m.o, c.grad_o, c.s.total, c.s.Hv, c.s.dv, (long long)c.s.Hv * c.s.dv));
        if (!ok) return cudaErrorInvalidValue;
    }
    cudaError_t e = run_intra<DK, kBack>(c, m, in);
    if (e == cudaSuccess) e = run_chain_fwd<DK, kBack>(c, m, in);
    if constexpr (kBack) {
        if (e == cudaSuccess) e = run_chain_bwd<DK>(c, m, in);
        if (e == cudaSuccess) e = c.s.dv <= 64 ? run_grads<DK, 64>(c, m, in) : run_grads<DK, 128>(c, m, in);
    }
    return e;
}

}  // namespace

extern "C" {

// Reads and clears the error word of this file's kernels (for ckda_get_device_error, after it
// synchronised the stream). Not part of the ABI.
cudaError_t ckda_gated_take_error(unsigned int* word) {
    const unsigned int zero = 0;
    unsigned int wait = 0;                     // bit 0: a bounded wait of this file's kernels ran out
    cudaError_t e = cudaMemcpyFromSymbol(word, g_gated_error_word, sizeof(*word));
    if (e == cudaSuccess && *word != 0) e = cudaMemcpyToSymbol(g_gated_error_word, &zero, sizeof(zero));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&wait, ckda::g_error_word, sizeof(wait));
    if (e == cudaSuccess && wait != 0) e = cudaMemcpyToSymbol(ckda::g_error_word, &zero, sizeof(zero));
    *word |= wait;
    return e;
}

size_t ckda_gated_fwd_workspace_bytes(int N, int total, int Hk, int Hv, int dk, int dv, ckda_dtype_t dt) {
    const Shape s{N, 0, total, Hk, Hv, dk, dv, dt};
    if (check_shape(s, true) != CKDA_OK || N == 0 || total == 0 || !chunked(s)) return 0;
    return chunk_layout(s, false).total;
}

int ckda_gated_fwd_segment_tokens(int N, int total, int Hk, int Hv, int dk, int dv, ckda_dtype_t dt) {
    const Shape s{N, 0, total, Hk, Hv, dk, dv, dt};
    if (check_shape(s, true) != CKDA_OK || N == 0 || total == 0 || !chunked(s)) return 0;
    return segment_chunks(s, false) * C;
}

ckda_status_t ckda_gated_fwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                             const float* S0, void* o, float* S_T, const int* cu_seqlens, int N, int T, int total, int Hk,
                             int Hv, int dk, int dv, long long q_stride, long long k_stride, long long v_stride,
                             ckda_dtype_t dt, void* workspace, size_t workspace_bytes, void* stream) {
    const Shape s{N, T, total, Hk, Hv, dk, dv, dt};
    ckda_status_t c = check_shape(s, cu_seqlens != nullptr);
    if (c != CKDA_OK) return c;
    if (total > 0 && (!q || !k || !v || !g || !beta || !o)) return CKDA_ERR_INVALID_ARG;
    if (!strides_ok(s, q_stride, k_stride, v_stride)) return CKDA_ERR_INVALID_ARG;
    if (!rows_aligned(s, q_stride, k_stride, v_stride)) return CKDA_ERR_MISALIGNED;
    if (chunked(s) && !chunked_fits(s)) return CKDA_ERR_UNSUPPORTED;
    const void* ptrs[] = {q, k, v, S0, o, S_T, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return CKDA_ERR_MISALIGNED;
    if (!aligned4(cu_seqlens) || !aligned4(g) || !aligned4(beta)) return CKDA_ERR_MISALIGNED;
    const size_t need = ckda_gated_fwd_workspace_bytes(N, total, Hk, Hv, dk, dv, dt);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return CKDA_ERR_WORKSPACE;
    cudaStream_t st = as_stream(stream);
    if (N == 0) return CKDA_OK;
    if (total == 0) return clear_or_copy(S0, S_T, (size_t)N * Hv * dk * dv, st);
    const Seqs seqs{cu_seqlens, N, T, total};
    if (chunked(s)) {
        Call a{};
        a.s = s;
        a.seqs = seqs;
        a.q = static_cast<const bf16*>(q); a.k = static_cast<const bf16*>(k); a.v = static_cast<const bf16*>(v);
        a.g = g; a.beta = beta; a.S0 = S0;
        a.o = static_cast<bf16*>(o); a.ST = S_T;
        a.qs = q_stride; a.ks = k_stride; a.vs = v_stride;
        const ChunkLayout l = chunk_layout(s, false);
        a.ws = chunk_ws(l, workspace);
        a.seg = segments(l, workspace, s, cu_seqlens != nullptr);
        a.st = st;
        const cudaError_t e = dk <= 64 ? run_chunked<64, false>(a) : run_chunked<128, false>(a);
        return e == cudaSuccess ? launch_status() : (cudaGetLastError(), CKDA_ERR_CUDA);
    }
    if (dt == CKDA_BF16) return simt_fwd<bf16>(s, q, k, v, g, beta, S0, o, S_T, seqs, nullptr, N, q_stride, k_stride, v_stride, st);
    return simt_fwd<float>(s, q, k, v, g, beta, S0, o, S_T, seqs, nullptr, N, q_stride, k_stride, v_stride, st);
}

size_t ckda_gated_bwd_workspace_bytes(int N, int total, int Hk, int Hv, int dk, int dv, ckda_dtype_t dt) {
    const Shape s{N, 0, total, Hk, Hv, dk, dv, dt};
    if (check_shape(s, true) != CKDA_OK || N == 0 || total == 0) return 0;
    return chunked(s) ? chunk_layout(s, true).total : simt_bwd_layout(s).total;
}

int ckda_gated_bwd_segment_tokens(int N, int total, int Hk, int Hv, int dk, int dv, ckda_dtype_t dt) {
    const Shape s{N, 0, total, Hk, Hv, dk, dv, dt};
    if (check_shape(s, true) != CKDA_OK || N == 0 || total == 0 || !chunked(s)) return 0;
    return segment_chunks(s, true) * C;
}

ckda_status_t ckda_gated_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                             const float* S0, const void* grad_o, const float* grad_S_T, void* grad_q, void* grad_k,
                             void* grad_v, float* grad_g, float* grad_beta, float* grad_S0, const int* cu_seqlens, int N,
                             int T, int total, int Hk, int Hv, int dk, int dv, long long q_stride, long long k_stride,
                             long long v_stride, ckda_dtype_t dt, void* workspace, size_t workspace_bytes, void* stream) {
    const Shape s{N, T, total, Hk, Hv, dk, dv, dt};
    ckda_status_t c = check_shape(s, cu_seqlens != nullptr);
    if (c != CKDA_OK) return c;
    if (total > 0 && (!q || !k || !v || !g || !beta || !grad_o || !grad_q || !grad_k || !grad_v || !grad_g || !grad_beta))
        return CKDA_ERR_INVALID_ARG;
    if (!strides_ok(s, q_stride, k_stride, v_stride)) return CKDA_ERR_INVALID_ARG;
    if (!rows_aligned(s, q_stride, k_stride, v_stride)) return CKDA_ERR_MISALIGNED;
    if (chunked(s) && !chunked_fits(s)) return CKDA_ERR_UNSUPPORTED;
    const void* ptrs[] = {q, k, v, S0, grad_o, grad_S_T, grad_q, grad_k, grad_v, grad_S0, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return CKDA_ERR_MISALIGNED;
    const void* words[] = {cu_seqlens, g, beta, grad_g, grad_beta};
    for (const void* p : words)
        if (!aligned4(p)) return CKDA_ERR_MISALIGNED;
    const size_t need = ckda_gated_bwd_workspace_bytes(N, total, Hk, Hv, dk, dv, dt);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return CKDA_ERR_WORKSPACE;
    cudaStream_t st = as_stream(stream);
    if (N == 0) return CKDA_OK;
    if (total == 0) return clear_or_copy(grad_S_T, grad_S0, (size_t)N * Hv * dk * dv, st);
    const Seqs seqs{cu_seqlens, N, T, total};
    char* ws = static_cast<char*>(workspace);
    if (chunked(s)) {
        Call a{};
        a.s = s;
        a.seqs = seqs;
        a.q = static_cast<const bf16*>(q); a.k = static_cast<const bf16*>(k); a.v = static_cast<const bf16*>(v);
        a.grad_o = static_cast<const bf16*>(grad_o);
        a.g = g; a.beta = beta; a.S0 = S0; a.dST = grad_S_T;
        a.gq = static_cast<bf16*>(grad_q); a.gk = static_cast<bf16*>(grad_k); a.gv = static_cast<bf16*>(grad_v);
        a.gg = grad_g; a.gb = grad_beta; a.gS0 = grad_S0;
        a.qs = q_stride; a.ks = k_stride; a.vs = v_stride;
        const ChunkLayout l = chunk_layout(s, true);
        a.ws = chunk_ws(l, ws);
        a.seg = segments(l, ws, s, cu_seqlens != nullptr);
        a.st = st;
        const cudaError_t e = dk <= 64 ? run_chunked<64, true>(a) : run_chunked<128, true>(a);
        return e == cudaSuccess ? launch_status() : (cudaGetLastError(), CKDA_ERR_CUDA);
    }
    if (dt == CKDA_BF16)
        return simt_bwd<bf16>(s, q, k, v, g, beta, S0, grad_o, grad_S_T, grad_q, grad_k, grad_v, grad_g, grad_beta, grad_S0,
                              seqs, q_stride, k_stride, v_stride, ws, st);
    return simt_bwd<float>(s, q, k, v, g, beta, S0, grad_o, grad_S_T, grad_q, grad_k, grad_v, grad_g, grad_beta, grad_S0,
                           seqs, q_stride, k_stride, v_stride, ws, st);
}

ckda_status_t ckda_gated_decode_step(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                     float* S, void* o, const int* slots, int N, int pool, int Hk, int Hv, int dk, int dv,
                                     long long q_stride, long long k_stride, long long v_stride, ckda_dtype_t dt,
                                     void* stream) {
    const Shape s{N, 1, N, Hk, Hv, dk, dv, dt};
    ckda_status_t c = check_shape(s, false);
    if (c != CKDA_OK) return c;
    if (pool < 0 || (slots == nullptr && pool < N)) return CKDA_ERR_INVALID_ARG;
    if (N == 0) return CKDA_OK;
    if (!q || !k || !v || !g || !beta || !o || !S || pool == 0) return CKDA_ERR_INVALID_ARG;
    if (!strides_ok(s, q_stride, k_stride, v_stride)) return CKDA_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, S, o};
    for (const void* p : ptrs)
        if (!aligned16(p)) return CKDA_ERR_MISALIGNED;
    if (!aligned4(slots) || !aligned4(g) || !aligned4(beta)) return CKDA_ERR_MISALIGNED;
    cudaStream_t st = as_stream(stream);
    // Column slab of a CTA: the widest that still gives two CTAs per SM.
    if ((dk == 64 || dk == 128) && dv % 32 == 0) {
        const long long want = 2LL * sm_count(), rows = (long long)N * Hv;
        int cw = 32;
        if (dv % 128 == 0 && rows * (dv / 128) >= want) cw = 128;
        else if (dv % 64 == 0 && rows * (dv / 64) >= want) cw = 64;
        const dim3 grid((unsigned)rows, (unsigned)(dv / cw));
#define GATED_DECODE(D, W, TIN)                                                                                     \
    decode_kernel<D, W, TIN><<<grid, 256, 0, st>>>(static_cast<const TIN*>(q), static_cast<const TIN*>(k),           \
                                                   static_cast<const TIN*>(v), g, beta, S, static_cast<TIN*>(o),     \
                                                   slots, pool, Hk, Hv, dv, q_stride, k_stride, v_stride)
#define GATED_DECODE2(D, TIN)                                                                                       \
    do {                                                                                                            \
        if (cw == 128) GATED_DECODE(D, 128, TIN);                                                                   \
        else if (cw == 64) GATED_DECODE(D, 64, TIN);                                                                \
        else GATED_DECODE(D, 32, TIN);                                                                              \
    } while (0)
        if (dk == 128) {
            if (dt == CKDA_BF16) GATED_DECODE2(128, bf16);
            else GATED_DECODE2(128, float);
        } else {
            if (dt == CKDA_BF16) GATED_DECODE2(64, bf16);
            else GATED_DECODE2(64, float);
        }
#undef GATED_DECODE2
#undef GATED_DECODE
        return launch_status();
    }
    const Seqs seqs{nullptr, N, 1, N};
    if (dt == CKDA_BF16) return simt_fwd<bf16>(s, q, k, v, g, beta, S, o, S, seqs, slots, pool, q_stride, k_stride, v_stride, st);
    return simt_fwd<float>(s, q, k, v, g, beta, S, o, S, seqs, slots, pool, q_stride, k_stride, v_stride, st);
}

}  // extern "C"

namespace {

// Blocks of the backward pass, which each leave a partial sum of the weights' gradients: fixed by
// the sizes and the device's number of SMs, so those sums have one order on it.
constexpr int kPrepMaxBlocks = 148 * 2;
int prep_blocks(long long units) { return (int)std::max(1LL, std::min(units, (long long)kPrepMaxBlocks)); }

ckda_status_t prep_args(PrepArgs& a, const void* q, const void* k, const float* qw, const float* kw, const void* pos,
                        int pos64, const double* inv_freq, int tokens, int period, int Hq, int Hk, int d, int rotary,
                        long long qs, long long ks, ckda_dtype_t dt, int norm, int interleaved, float eps, float q_scale,
                        float rope_scale) {
    if (tokens < 0 || Hq < 1 || Hk < 0 || d < 1 || d > CKDA_PREP_MAX_D || rotary < 0 || rotary > d || rotary % 2 != 0)
        return CKDA_ERR_INVALID_ARG;
    if (dt != CKDA_F32 && dt != CKDA_BF16) return CKDA_ERR_INVALID_ARG;
    if (norm < kNormNone || norm > kNormRms || interleaved < 0 || interleaved > 1 || pos64 < 0 || pos64 > 1)
        return CKDA_ERR_INVALID_ARG;
    if (qs < (long long)Hq * d || (Hk > 0 && ks < (long long)Hk * d)) return CKDA_ERR_INVALID_ARG;
    if (rotary > 0 && !inv_freq) return CKDA_ERR_INVALID_ARG;
    if (rotary > 0 && !pos && period < 1) return CKDA_ERR_INVALID_ARG;
    if (tokens > 0 && (!q || (Hk > 0 && !k))) return CKDA_ERR_INVALID_ARG;
    if ((long long)Hq + Hk > 4096) return CKDA_ERR_UNSUPPORTED;
    a = PrepArgs{};
    a.x[0] = q; a.x[1] = k;
    a.w[0] = qw; a.w[1] = kw;
    a.stride[0] = qs; a.stride[1] = ks;
    a.heads[0] = Hq; a.heads[1] = Hk;
    a.pos = rotary > 0 ? pos : nullptr;
    a.inv_freq = inv_freq;
    a.pos64 = pos64;
    a.period = std::max(period, 1);
    a.tokens = tokens; a.d = d; a.rotary = rotary; a.norm = norm; a.interleaved = interleaved;
    a.inv_d = 1.f / (float)d;
    a.eps = eps; a.q_scale = q_scale; a.rope_scale = rope_scale;
    const void* ptrs[] = {q, k, qw, kw};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return CKDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(pos) & (pos64 ? 7u : 3u)) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
        return CKDA_ERR_MISALIGNED;
    return CKDA_OK;
}

// Whether rows can be read 16 bytes a lane (see qk_prep.cuh).
bool prep_vector(const PrepArgs& a, ckda_dtype_t dt) {
    const int per16 = dt == CKDA_BF16 ? 8 : 4;
    if (a.d % 8 != 0 || a.stride[0] % per16 != 0 || (a.heads[1] > 0 && a.stride[1] % per16 != 0)) return false;
    return a.rotary % (a.interleaved ? 8 : 16) == 0;
}

template <typename TIn, bool kBack>
ckda_status_t prep_launch(const PrepArgs& a, ckda_dtype_t dt, int* blocks_out, cudaStream_t st) {
    constexpr int UR = kBack ? 2 : 4;
    if (prep_vector(a, dt)) {
        const int G = a.d <= 64 ? 8 : (a.d <= 128 ? 16 : 32), gp = 32 / G;
        // Warps to a token: one, more while tokens are too few to give every SM two blocks and the
        // heads still give each warp a row.
        int wpt = 1;
        while (wpt < 8 && (long long)a.tokens * wpt < 16LL * sm_count() && wpt * gp < a.heads[0] + a.heads[1]) wpt *= 2;
        const long long units = ((long long)a.tokens * wpt + 7) / 8;
        const int blocks = kBack ? prep_blocks(units) : (int)std::min<long long>(units, (long long)sm_count() * 3);
        size_t smem = (size_t)8 * a.rotary * sizeof(float);
        if (kBack) smem = std::max(smem, (size_t)8 * gp * a.d * sizeof(float));
        *blocks_out = blocks;
        auto go = [&](auto kernel) { kernel<<<blocks, 256, smem, st>>>(a, wpt); };
        if (G == 8) a.interleaved ? go(prep_vec_kernel<TIn, 8, UR, kBack, true>) : go(prep_vec_kernel<TIn, 8, UR, kBack, false>);
        else if (G == 16) a.interleaved ? go(prep_vec_kernel<TIn, 16, UR, kBack, true>) : go(prep_vec_kernel<TIn, 16, UR, kBack, false>);
        else a.interleaved ? go(prep_vec_kernel<TIn, 32, UR, kBack, true>) : go(prep_vec_kernel<TIn, 32, UR, kBack, false>);
    } else {
        *blocks_out = kBack ? prep_blocks(a.tokens) : std::min(a.tokens, 148 * 8);
        prep_row_kernel<TIn, kBack><<<*blocks_out, 256, 0, st>>>(a);
    }
    return launch_status();
}

}  // namespace

extern "C" {

ckda_status_t ckda_qk_prep(const void* q, const void* k, void* q_out, void* k_out, const float* q_weight,
                           const float* k_weight, const void* positions, int positions64, const double* inv_freq,
                           int tokens, int period, int Hq, int Hk, int d, int rotary, long long q_stride,
                           long long k_stride, ckda_dtype_t dt, int norm, int interleaved, float eps, float q_scale,
                           float rope_scale, void* stream) {
    PrepArgs a;
    ckda_status_t c = prep_args(a, q, k, q_weight, k_weight, positions, positions64, inv_freq, tokens, period, Hq, Hk, d,
                                rotary, q_stride, k_stride, dt, norm, interleaved, eps, q_scale, rope_scale);
    if (c != CKDA_OK) return c;
    if (tokens == 0) return CKDA_OK;
    if (!q_out || (Hk > 0 && !k_out)) return CKDA_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(k_out)) return CKDA_ERR_MISALIGNED;
    a.out[0] = q_out;
    a.out[1] = k_out;
    int blocks;
    return dt == CKDA_BF16 ? prep_launch<bf16, false>(a, dt, &blocks, as_stream(stream))
                           : prep_launch<float, false>(a, dt, &blocks, as_stream(stream));
}

size_t ckda_qk_prep_bwd_workspace_bytes(int d) {
    return d < 1 || d > CKDA_PREP_MAX_D ? 0 : (size_t)kPrepMaxBlocks * 2 * d * sizeof(float);
}

ckda_status_t ckda_qk_prep_bwd(const void* q, const void* k, const void* grad_q_out, const void* grad_k_out, void* grad_q,
                               void* grad_k, float* grad_q_weight, float* grad_k_weight, const float* q_weight,
                               const float* k_weight, const void* positions, int positions64, const double* inv_freq,
                               int tokens, int period, int Hq, int Hk, int d, int rotary, long long q_stride,
                               long long k_stride, ckda_dtype_t dt, int norm, int interleaved, float eps, float q_scale,
                               float rope_scale, void* workspace, size_t workspace_bytes, void* stream) {
    PrepArgs a;
    ckda_status_t c = prep_args(a, q, k, q_weight, k_weight, positions, positions64, inv_freq, tokens, period, Hq, Hk, d,
                                rotary, q_stride, k_stride, dt, norm, interleaved, eps, q_scale, rope_scale);
    if (c != CKDA_OK) return c;
    const bool weights = grad_q_weight || grad_k_weight;
    if (tokens > 0 && (!grad_q_out || !grad_q || (Hk > 0 && (!grad_k_out || !grad_k)))) return CKDA_ERR_INVALID_ARG;
    const void* ptrs[] = {grad_q_out, grad_k_out, grad_q, grad_k, grad_q_weight, grad_k_weight, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return CKDA_ERR_MISALIGNED;
    if (weights && tokens > 0 && (!workspace || workspace_bytes < ckda_qk_prep_bwd_workspace_bytes(d))) return CKDA_ERR_WORKSPACE;
    cudaStream_t st = as_stream(stream);
    if (tokens == 0) {
        for (float* w : {grad_q_weight, grad_k_weight})
            if (w && cudaMemsetAsync(w, 0, d * sizeof(float), st) != cudaSuccess) return CKDA_ERR_CUDA;
        return CKDA_OK;
    }
    a.dy[0] = grad_q_out;
    a.dy[1] = grad_k_out;
    a.out[0] = grad_q;
    a.out[1] = grad_k;
    a.partial = weights ? static_cast<float*>(workspace) : nullptr;
    int blocks = 0;
    c = dt == CKDA_BF16 ? prep_launch<bf16, true>(a, dt, &blocks, st) : prep_launch<float, true>(a, dt, &blocks, st);
    if (c != CKDA_OK || !weights) return c;
    prep_weight_kernel<<<(unsigned)((2 * d + 31) / 32), 1024, 0, st>>>(a.partial, blocks, d, grad_q_weight, grad_k_weight);
    return launch_status();
}

ckda_status_t ckda_state_copy(float* S, const int* src, const int* dst, int pairs, int layers, int slots,
                              long long state_floats, void* stream) {
    if (pairs < 0 || layers < 0 || slots < 0 || state_floats < 0) return CKDA_ERR_INVALID_ARG;
    if (pairs == 0 || layers == 0 || state_floats == 0) return CKDA_OK;
    if (!src || !dst || !S || slots == 0) return CKDA_ERR_INVALID_ARG;
    if (!aligned16(S) || !aligned4(src) || !aligned4(dst)) return CKDA_ERR_MISALIGNED;
    if (pairs > kCopyMaxPairs || state_floats % 4 != 0 || layers > 65535) return CKDA_ERR_UNSUPPORTED;
    const long long pieces = state_floats / 4;
    // Slice: about 32 KB of states a CTA (several CTAs per SM overlap their reads and writes), narrower
    // while that leaves SMs without work, 128 bytes at least, and whole sectors of 32 bytes, so that no two CTAs
    // write parts of one.
    int width = std::max(8, std::min(256, 2048 / pairs) & ~1);
    while (width > 8 && ((pieces + width - 1) / width) * layers < 2LL * sm_count()) width = std::max(8, width / 2 & ~1);
    if (pieces < width) width = (int)pieces;
    const long long slices = (pieces + width - 1) / width;
    if (slices > 0x7fffffffLL) return CKDA_ERR_UNSUPPORTED;
    const int table = copy_table(pairs);
    const size_t smem = (size_t)pairs * width * 16 + (size_t)(2 * table + 2 * pairs) * sizeof(int);
    if (smem > 48 * 1024 && kernel_ready(state_copy_kernel, kCopyMaxSmem) != cudaSuccess) return CKDA_ERR_CUDA;
    state_copy_kernel<<<dim3((unsigned)slices, (unsigned)layers), kCopyThreads, smem, as_stream(stream)>>>(
        reinterpret_cast<uint4*>(S), src, dst, pairs, slots, pieces, width, table);
    return launch_status();
}

}  // extern "C"
