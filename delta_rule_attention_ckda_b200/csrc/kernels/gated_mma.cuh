// Warp-level matrix building blocks of the chunked gated delta rule: bf16 tiles in padded
// shared memory, fragment loads, products with fp32 accumulation, and splits of fp32 values
// into bf16 terms.
//
#pragma once
#include "gated_common.cuh"
#include "tc_primitives.cuh"

namespace ckda {
namespace gated {

constexpr int LD64 = 144;                      // bytes of a padded row of 64 bf16 (9 x 16: conflict-free ldmatrix)

__device__ __forceinline__ uint32_t s32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
// c += a b, 16 x 8 x 16
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += a b in tf32, 16 x 8 x 8
__device__ __forceinline__ void mma_tf32(float (&c)[4], const float (&a)[4], const float (&b)[2]) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                   "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b[0])), "r"(__float_as_uint(b[1])));
}

// Byte offset of this lane's ldmatrix row in a tile with rows of `ld` bytes, for the fragment at
// (row r0, column c0):
//   ofs_n: rows are the operand's n (or an accumulator's transposed rows), columns its k
//   ofs_k: rows are k, columns n (loaded with .trans)
//   ofs_a: rows are the left operand's m, columns its k; ofs_at: rows k, columns m (.trans)
__device__ __forceinline__ uint32_t ofs_n(int ld) {
    const int l = threadIdx.x & 31;
    return (uint32_t)(((l & 7) + ((l >> 4) & 1) * 8) * ld + ((l >> 3) & 1) * 16);
}
__device__ __forceinline__ uint32_t ofs_k(int ld) {
    const int l = threadIdx.x & 31;
    return (uint32_t)(((l & 7) + ((l >> 3) & 1) * 8) * ld + ((l >> 4) & 1) * 16);
}
__device__ __forceinline__ uint32_t ofs_a(int ld) { return ofs_k(ld); }
__device__ __forceinline__ uint32_t ofs_at(int ld) { return ofs_n(ld); }
__device__ __forceinline__ uint32_t at(int row, int col, int ld) { return (uint32_t)(row * ld + col * 2); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_of(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_of(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Two fp32 operations in one instruction (sm_100 packed arithmetic).
__device__ __forceinline__ unsigned long long pair(float x, float y) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(unsigned long long p, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p)); }
// (x, y) <- (a, b) * (c, d) + (x, y)
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float c, float d) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a, b)), "l"(pair(c, d)), "l"(pair(x, y)));
    unpair(r, x, y);
}
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(x, y)), "l"(pair(a, b)));
    unpair(r, x, y);
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(x, y)), "l"(pair(a, b)));
    unpair(r, x, y);
}

// Two fp32 values as bf16 terms, each the rounded remainder of those before: hi + mid is within
// 2^-16 of a value (2.7e-6 at RMS), hi + mid + lo within 2^-23. Only hi goes through the
// conversion instruction, which is the scarce one; mid is rounded half up and lo cut in
// integer arithmetic. A NaN or an infinity stays in hi (its remainder, NaN, rounds to zero in mid).
__device__ __forceinline__ uint32_t upper2(uint32_t x, uint32_t y) { return __byte_perm(x, y, 0x7632); }
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& mid) {
    hi = pack2(x, y);
    fma2(x, y, lo_of(hi), hi_of(hi), -1.f, -1.f);
    mid = upper2(__float_as_uint(x) + 0x8000u, __float_as_uint(y) + 0x8000u);
}
__device__ __forceinline__ void split3(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack2(x, y);
    fma2(x, y, lo_of(hi), hi_of(hi), -1.f, -1.f);
    mid = upper2(__float_as_uint(x) + 0x8000u, __float_as_uint(y) + 0x8000u);
    fma2(x, y, lo_of(mid), hi_of(mid), -1.f, -1.f);
    lo = upper2(__float_as_uint(x), __float_as_uint(y));
}

// Tiles of 64 tokens as tensor copies write them: blocks of [64 rows][64 channels], rows of 128
// bytes, the 16-byte pieces of a row exchanged by its number (the 128-byte swizzle).
__device__ __forceinline__ uint32_t swz(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); }
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int head, int token) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(c0), "r"(head), "r"(token)
                 : "memory");
}

// What the chunked kernels read by rows: tensor maps over [tokens][heads][channels] (boxes of 64
// tokens of one head's 64 channels), and plain pointers for the rows at a sequence's end.
struct ChainIn {
    const __nv_bfloat16 *q, *k, *v, *dO;
    long long qs, ks, vs;
    int maps;                       // whether the maps are usable (heads of at least 64 channels)
};

// Rows of a tensor into such a tile of `width` channels, zeros behind the chunk's end (nt) and the
// head's channels (d); thread x of NT.
template <int NT>
__device__ __forceinline__ void tile_rows(uint32_t to, const __nv_bfloat16* from, long long stride, int nt, int d, int width, int x) {
#pragma unroll 1
    for (int e = x; e < 8 * width; e += NT) {
        const int r = e / (width / 8), p = e % (width / 8);
        const bool is = r < nt && p * 8 < d;
        cp16(to + (p / 8) * 8192 + swz(r, p & 7), is ? from + r * stride + p * 8 : from, is);
    }
}
// This lane's part of an ldmatrix address in a swizzled tile: rows as ofs_n or ofs_k; the fragment's
// column c0 (a multiple of 16) enters by frag().
__device__ __forceinline__ uint32_t swz_lane(bool rows_by_bit4) {
    const int l = threadIdx.x & 31, hi = (l >> 4) & 1, lo = (l >> 3) & 1;
    const int row = (l & 7) + (rows_by_bit4 ? hi : lo) * 8, piece = rows_by_bit4 ? lo : hi;
    return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint32_t frag(uint32_t lane, int r0, int c0) {
    return (lane ^ (uint32_t)((c0 % 64) * 2)) + (uint32_t)(r0 * 128 + (c0 / 64) * 8192);
}

// ---------------------------------------------------------------- workspace of the chunked kernels

// Per chunk and value head, floats: e^G, e^{G_C - G}, beta, P's diagonal q_i.k_i (backward only), then G in
// two parts (G = hi + lo).
enum { VEC_EG = 0, VEC_DEC = 64, VEC_BETA = 128, VEC_PD = 192, VEC_GHI = 256, VEC_GLO = 320, VEC = 384 };

// Per chunk slot and value head (each pointer is that of slot 0, head 0). What a thread per state
// column reads and writes lies with its columns side by side, 16 bytes each: states as
// [dk / 8][dv][8], w as [16][dv][4 tokens].
struct ChunkWs {
    __nv_bfloat16 *zhi, *zlo, *phi, *plo;      // [64][64]: Z and the decayed q.k, two bf16 terms each
    float* vec;                                // [VEC]
    __nv_bfloat16 *shi, *slo;                  // backward: entering state, [dk / 8][dv][8] (see put_state)
    __nv_bfloat16* dshi;                       // backward: cotangent of the leaving state, [dk / 8][dv][8]
    __nv_bfloat16* u;                          // backward: updates [64][dv]
    float* d;                                  // backward: v - w, [16][dv][4]
    float* parts;                              // backward: [dv / 32][PARTS] sums over 32 columns (SDS: two halves)
};
// PAST <dO, o> without a token's own update, FUTURE what is taken from it (see gated_grads.cuh), DB <w, y> per
// token; SDS <S', dS> of the leaving state, SDS0 (a sequence's first chunk) of the entering one
enum { PART_PAST = 0, PART_FUTURE = 64, PART_DB = 128, PART_SDS = 192, PART_SDS0 = 194, PARTS = 208 };

}  // namespace gated
}  // namespace ckda
