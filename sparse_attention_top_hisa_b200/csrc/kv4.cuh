// The 4-bit cache format and the register-level pieces its readers share.
//
// A group of 16 dimensions shares a scale s; a value is q * s with a whole q of -7..7
// stored as the nibble u = q + 8, low nibble first.  s is an unsigned e5m3 number kept
// in one byte: bits 14..7 of its fp16 pattern.  s has 4 significant bits and q has 3, so
// q * s is exact in fp16 and in bf16.  s is at most 896 (byte 198), or 255 in a group that is
// not a number.
//
// Four bits per value were taken as whole numbers rather than as a 4-bit float (e2m1)
// because their error on Gaussian rows is smaller at this group size (about 8.5% rms of
// a value's spread against 10.5%) and because a nibble turns into an fp16 pair with one
// logic operation and one FMA (below), where the float needs its sign moved apart.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace hisa {

constexpr int KV4_DIM = HISA_ATT_DIM;              // 128
constexpr int KV4_HALF = KV4_DIM / 2;              // bytes of a key's (or value's) nibbles
constexpr int KV4_ROW = HISA_KV4_ROW_BYTES;        // key nibbles, then value nibbles
constexpr int KV4_NS = HISA_KV4_ROW_SCALES;        // scale bytes of a row: 8 key, 8 value
constexpr int KV4_GROUP = HISA_KV4_GROUP;          // 16
constexpr uint32_t KV4_MAX_SCALE = 198;            // the byte of 896
static_assert(KV4_DIM == 128 && KV4_GROUP == 16 && KV4_ROW == 128 && KV4_NS == 16,
              "the fragment layouts below take these sizes");

// find_seq for a row that a whole warp asks for: 32 offsets are looked at together, where
// a lone thread would wait for one after another (16 sequences: 1 wait instead of 5).
// Without a way out in the middle: after one the compiler no longer takes the warp to be
// together (561 us became 645 for 8192 attention rows of 2048 tokens).
__device__ __forceinline__ int find_seq_warp(const int32_t *cu_q, int S, int row, int lane) {
  int lo = 0, hi = S - 1;  // the last s of lo .. hi with cu_q[s] <= row (lo itself counts)
  while (hi - lo > 128) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu_q + mid) <= row) lo = mid; else hi = mid - 1;
  }
  int n = 0;  // of the offsets behind lo, those at or before the row (they never fall)
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int s = lo + 1 + 32 * i + lane;
    n += __popc(__ballot_sync(0xffffffffu, s <= hi && __ldg(cu_q + s) <= row));
  }
  return lo + n;
}

// The region of the keys of a query row, for a warp: no tokens for a row outside every
// sequence (behind the last one of a padded batch), so that it adds nothing to one.
struct Region {
  int base, tokens;
};
__device__ __forceinline__ Region region_of(const int32_t *cu_q, const int32_t *cu_k, int S,
                                            int row, int lane) {
  const int rows = __ldg(cu_q + S);  // beside the search, not after it
  const int s = find_seq_warp(cu_q, S, row, lane);
  // the end's address is chosen, not the count (8192 rows of 2048 tokens: 551 us against 561)
  const int base = __ldg(cu_k + s), end = __ldg(cu_k + s + (row < rows));
  return {base, end - base};
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) {
  return *reinterpret_cast<const __half2 *>(&w);
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) {
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Nibbles at bits 4..7 of both halves of w as fp16 values times the scale pair s:
// 0x5400 is 64 and its low mantissa bit 1/16, so or-ing the nibble into bits 4..7 gives
// 64 + u, and (64 + u) * s - 72 * s = (u - 8) * s, rounded once and exact.
// c72 = -72 * s (72 has 4 significant bits, so it is exact too, and finite for s <= 896; of a
// larger scale, which is none of the format's, it is -inf and so are the values.  Making them
// NaN takes one operation more for each c72: 545 us instead of 537 for 8192 attention rows).
// The magic number comes from a register that the compiler does not see through: of two
// constants it would make two logic operations.
__device__ __forceinline__ uint32_t kv4_magic() {
  uint32_t m;
  asm("mov.b32 %0, 0x54005400;" : "=r"(m));
  return m;
}
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, uint32_t magic, __half2 s, __half2 c72) {
  uint32_t t;  // (w & 0x00F000F0) | magic
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(t) : "r"(w), "r"(magic));
  return as_u32(__hfma2(as_half2(t), s, c72));
}

__device__ __forceinline__ __half2 kv4_c72(__half2 s) {
  return __hmul2(s, as_half2(0xD480D480u));  // -72
}

// D += A (16 x 16, row) * B (16 x 8, col), fp16 in, fp32 out.  The matrix instruction
// whose operands are registers: the 4-bit rows are turned into fragments where they are
// used, where the one that reads shared memory would need every row written back there in
// 16 bits (4x the bytes that arrived) before it could start.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A * B
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                              uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 2^x (the hardware approximation: relative error about 2^-22, 2^-inf = 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace hisa
