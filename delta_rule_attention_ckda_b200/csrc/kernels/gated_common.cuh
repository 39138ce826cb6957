// Shared by the kernels of the scalar-gate operators (gated delta rule, q/k preparation,
// state copies): the device error word, packed-sequence addressing, typed loads and stores.
#pragma once
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

namespace ckda {
namespace gated {

// Device error word of this GPU for these operators (read and cleared by
// ckda_get_device_error). Bit 1: an index read on the device (a sequence offset or a pool
// slot) was out of range or named twice, and the work it named was skipped.
__device__ unsigned int g_gated_error_word = 0;
constexpr unsigned int kErrIndex = 2u;

__device__ __forceinline__ void report_index_error() { atomicOr(&g_gated_error_word, kErrIndex); }

constexpr int C = 64;                          // tokens in a chunk
constexpr float kGateFloor = -128.f;           // e^-128 is 0 in fp32: a smaller log gate decays as much

// A gate below the floor (or -inf) is taken at the floor: e^g is 0 in fp32 either way, and
// differences of sums of finite gates never become inf - inf. NaN stays NaN.
__device__ __forceinline__ float gate_in(float g) { return g < kGateFloor ? kGateFloor : g; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Kernels of one short call follow one another closely: each lets the next begin once all its own blocks
// run (what the next sets up then runs beside the last of them), and waits for the one before
// it, complete and visible, ahead of anything that one wrote. Every block waits, also one without
// work: a kernel has ended only when the one before it has.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The sequences of a call. Dense (cu == nullptr): N sequences of T tokens, one after the
// other. Packed: sequence n is tokens cu[n] .. cu[n+1] - 1 of `total`.
struct Seqs {
    const int* cu;
    int N, T, total;
    // First token and length of sequence n; offsets outside the tensors or out of order are
    // cut to them (ok = false).
    __device__ __forceinline__ void get(int n, int& start, int& len, bool& ok) const {
        if (cu == nullptr) {
            start = n * T;
            len = T;
            ok = true;
            return;
        }
        const int a = __ldg(cu + n), b = __ldg(cu + n + 1);
        start = min(max(a, 0), total);
        const int end = min(max(b, start), total);
        len = end - start;
        ok = start == a && end == b;
    }
    // Every sequence has places of its own among slots() workspace slots, one for each chunk and
    // one for the state behind the last: ceil(len / C) + 1 places of a sequence that starts at
    // token s end before (s + len) / C + 2 (n + 1), where the next one's begin.
    __host__ __device__ static size_t slots(int N, int total) { return (size_t)total / C + 2 * (size_t)N; }
    __device__ __forceinline__ int first_slot(int n, int start) const { return start / C + 2 * n; }
    // The sequence whose places hold slot s: the last n with first_slot(n) <= s.
    __device__ __forceinline__ int find(int s) const {
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int m = (lo + hi + 1) / 2;
            const int start = cu == nullptr ? m * T : min(max(__ldg(cu + m), 0), total);
            if (first_slot(m, start) <= s) lo = m; else hi = m - 1;
        }
        return lo;
    }
};

}  // namespace gated
}  // namespace ckda
