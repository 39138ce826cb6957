// Warp-level matrix building blocks of the chunked gated delta rule: bf16 tiles in padded
// shared memory, fragment loads, products with fp32 accumulation, and splits of fp32 values
// into bf16 terms.
//
#pragma once
#include "gated_common.cuh"

namespace ckda {
namespace gated {

constexpr int LD64 = 144;                      // bytes of a padded row of 64 bf16 (9 x 16: conflict-free ldmatrix)
__host__ __device__ constexpr int ld_bytes(int cols) { return cols * 2 + 16; }

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

// The left operand of a k-step (16 wide) from two accumulator tiles of the product before.
__device__ __forceinline__ void operand(const float (&u)[4], const float (&v)[4], uint32_t (&a)[4]) {
    a[0] = pack2(u[0], u[1]);
    a[1] = pack2(u[2], u[3]);
    a[2] = pack2(v[0], v[1]);
    a[3] = pack2(v[2], v[3]);
}

// Rows of a [tokens][...] tensor into a padded tile: `rows` of 64 rows present, `cols` of COLS
// columns present (both padded with zeros). cols is a multiple of 8.
template <int COLS, int NT>
__device__ __forceinline__ void load_rows(uint32_t dst, const __nv_bfloat16* src, long long stride, int rows, int cols) {
    constexpr int P = COLS / 8;
#pragma unroll
    for (int e = threadIdx.x; e < 64 * P; e += NT) {
        const int r = e / P, p = e % P;
        const bool in = r < rows && p * 8 < cols;
        cp16(dst + r * ld_bytes(COLS) + p * 16, in ? src + r * stride + p * 8 : src, in);
    }
}
// ---------------------------------------------------------------- workspace of the chunked kernels

// Per chunk and value head, floats: e^G, e^{G_C - G}, beta, then G in two parts (G = hi + lo).
enum { VEC_EG = 0, VEC_DEC = 64, VEC_BETA = 128, VEC_GHI = 192, VEC_GLO = 256, VEC = 320 };

// Per chunk slot and value head (each pointer is that of slot 0, head 0). What a thread per state
// column reads and writes lies with its columns side by side, 16 bytes each: states as
// [dk / 8][dv][8], w as [16][dv][4 tokens].
struct ChunkWs {
    __nv_bfloat16 *zhi, *zlo, *phi, *plo;      // [64][64]: Z and the decayed q.k, two bf16 terms each
    float* vec;                                // [VEC]
    __nv_bfloat16 *shi, *slo;                  // backward: entering state, [dk / 8][dv][8] (see put_state)
    __nv_bfloat16* dshi;                       // backward: cotangent of the leaving state, [dk / 8][dv][8]
    __nv_bfloat16* u;                          // backward: updates [64][dv]
    float* w;                                  // backward: w, [16][dv][4]
    float* parts;                              // backward: [dv / 32][PARTS] sums over 32 columns (SDS: two halves)
};
// DOO <dO, o>, DVV <dV, v>, DB <w, y> per token; SDS <S', dS> of the leaving state, SDS0 (a
// sequence's first chunk) of the entering one
enum { PART_DOO = 0, PART_DVV = 64, PART_DB = 128, PART_SDS = 192, PART_SDS0 = 194, PARTS = 208 };

}  // namespace gated
}  // namespace ckda
