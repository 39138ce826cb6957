// Copies of whole states within a pool: pair i takes the state of slot src[i] to slot dst[i],
// as if every source were read before any destination is written (so forks, chains, swaps and
// compaction need no order), and clears dst[i] where src[i] is negative. A negative dst[i]
// names no slot; of pairs that name the same destination the last one counts.
//
// HBM-bound: every source is read once and every destination written once. A state is cut
// into slices of `width` 16-byte pieces; one CTA holds one slice of EVERY pair in shared
// memory, so nothing outside it touches the bytes that it reads and writes, and the order
// "all reads, then all writes" needs one block barrier and no staging memory. Which pair
// counts for a destination comes from a small hash table of (destination, last pair).
//
// Measured, 96 pairs of 16 states of 128 x 128 (201 MB): 34 us, 91% of the copy bandwidth; 12 layers
// of two pairs: 5 us, a launch.
#pragma once
#include "gated_common.cuh"

namespace ckda {
namespace gated {

constexpr int kCopyMaxPairs = 1024;
constexpr int kCopyThreads = 256;
constexpr size_t kCopyMaxSmem = 1024 * 8 * 16 + (2 * 2048 + 2 * 1024) * 4;     // the narrowest slice of the most pairs, and its table

__host__ __device__ inline int copy_table(int pairs) {
    int n = 2;
    while (n < 2 * pairs) n *= 2;
    return n;
}

__global__ void __launch_bounds__(kCopyThreads)
state_copy_kernel(uint4* __restrict__ S, const int* __restrict__ src, const int* __restrict__ dst, int pairs, int slots,
                  long long pieces, int width, int table) {
    extern __shared__ __align__(16) uint4 hold[];              // [pairs][width]
    int* keys = reinterpret_cast<int*>(hold + (size_t)pairs * width);
    int* last = keys + table;
    int* from = last + table;                                  // [pairs] source slot, -1 clear, -2 not copied
    int* to = from + pairs;
    const int tid = threadIdx.x;
    uint4* base = S + (long long)blockIdx.y * slots * pieces;  // one layer's pool
    const long long p0 = (long long)blockIdx.x * width;
    const int w = (int)min((long long)width, pieces - p0);
    for (int i = tid; i < table; i += kCopyThreads) {
        keys[i] = -1;
        last[i] = -1;
    }
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < pairs; i += kCopyThreads) {
        const int a = __ldg(src + i), b = __ldg(dst + i);
        const bool out = a >= slots || b >= slots;
        bad |= out;
        from[i] = out || b < 0 ? -2 : (a < 0 ? -1 : a);
        to[i] = b;
        if (!out && b >= 0) {
            unsigned at = ((unsigned)b * 2654435761u) & (unsigned)(table - 1);
            while (true) {                                     // the table has twice as many places as pairs
                const int seen = atomicCAS(keys + at, -1, b);
                if (seen == -1 || seen == b) break;
                at = (at + 1) & (unsigned)(table - 1);
            }
            atomicMax(last + at, i);
        }
    }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) report_index_error();
    __syncthreads();
    for (int i = tid; i < pairs; i += kCopyThreads) {
        if (from[i] == -2) continue;
        unsigned at = ((unsigned)to[i] * 2654435761u) & (unsigned)(table - 1);
        while (keys[at] != to[i]) at = (at + 1) & (unsigned)(table - 1);
        if (last[at] != i) from[i] = -2;
    }
    __syncthreads();
    const int all = pairs * w;
    for (int e = tid; e < all; e += kCopyThreads) {
        const int i = e / w, x = e % w;
        if (from[i] >= 0) {
            const uint32_t sm = static_cast<uint32_t>(__cvta_generic_to_shared(hold + (size_t)i * width + x));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm), "l"(base + from[i] * pieces + p0 + x)
                         : "memory");
        }
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    for (int e = tid; e < all; e += kCopyThreads) {
        const int i = e / w, x = e % w, f = from[i];
        if (f != -2) base[to[i] * pieces + p0 + x] = f < 0 ? make_uint4(0u, 0u, 0u, 0u) : hold[(size_t)i * width + x];
    }
}

}  // namespace gated
}  // namespace ckda
