// Storing rows in the 4-bit cache and reading them back (hisa_kv4_store, hisa_kv4_load).
//
// Per group of 16 dimensions, with a = max |x|:
//   s = a / 7 rounded to nearest even in e5m3, at most 896;   q = x / s rounded to nearest
//   even, clamped to -7..7.
// Every decision is the exact one.  a and x have 8 significant bits, and a tie of a / 7
// lies at 7 * (a 5-bit number) and one of x / s at s * (a 4-bit number): both are 8-bit
// numbers, so a quotient that is not a tie is at least 2^-8 (relative) from one.  The
// products with the rounded reciprocals of 7 and s are off by a few 2^-23; rounding them
// to 12 bits (a / 7) and to a multiple of 2^-12 (x / s, in the FMA that adds 1.5 * 2^11) puts
// ties back where they belong and moves nothing else across one, and a second rounding
// decides.
//
// A sequence whose region or length does not fit, or with fewer live tokens than query
// rows, is skipped whole.  Rows behind the last sequence, in a padded batch, have no place in
// the cache and are no error.
//
// One thread per group (16 per row, 8 of the key and 8 of the value): a store reads 512
// bytes per row and writes 144, a load the reverse, so both are bound by memory (86 MB each
// for 131072 rows; a plain copy of the card moves 6.0 TB/s at this size).  A warp takes 2
// rows, or 4 where there are rows enough for every SM, whose loads are in flight together.
#include <cuda_bf16.h>
#include <limits.h>

#include "kv4.cuh"
#include "prof.cuh"

namespace hisa {

constexpr int KVS_THREADS = 128, KVS_WARPS = KVS_THREADS / 32;

// e5m3 byte of amax / 7 (amax >= 0, finite, bf16), rounded to nearest even, at most 896
__device__ __forceinline__ uint32_t e5m3_seventh(float amax) {
  // 12 significant bits: ties of the quotient are exact again
  const uint32_t u = (__float_as_uint(amax * (1.f / 7.f)) + 0x800u) & 0xFFFFF000u;
  const float t = __uint_as_float(u);
  const uint32_t normal = ((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
  const uint32_t tiny = (uint32_t)__float2int_rn(t * 0x1p17f);  // multiples of 2^-17; 8 is 2^-14
  return min(t < 0x1p-14f ? tiny : normal, KV4_MAX_SCALE);
}

__device__ __forceinline__ float reciprocal(float s) {  // of a normal s, off by an ulp or two
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Eight values (pairs of bf16) times r as nibbles q + 8; CLAMP: q may pass 7.
template <bool CLAMP>
__device__ __forceinline__ uint32_t nibbles(const uint32_t *w, float r) {
  uint32_t sum = 0;
#pragma unroll
  for (int j = 7; j >= 0; j--) {
    float t = fmaf((j & 1) ? bf_hi(w[j >> 1]) : bf_lo(w[j >> 1]), r, 0x1.8p11f);
    if (CLAMP) t = fminf(fmaxf(t, 0x1.8p11f - 7.f), 0x1.8p11f + 7.f);
    // 1.5 * 2^23 + 8 + q: rounds to a whole number, whose bits are a constant and q + 8
    t += 0x1.8p23f + 8.f - 0x1.8p11f;
    sum = sum * 16u + __float_as_uint(t);
  }
  return sum - 0x11111111u * 0x4B400000u;
}

__device__ __forceinline__ float e5m3_value(uint32_t b) {
  return __half2float(__ushort_as_half((unsigned short)(b << 7)));
}

// The cache rows of R query rows, `row`, `row` + 2, ... (row is a warp's first for its lanes
// 0-15 and the one after for the others): -1 where the sequence is skipped or there is none.
template <int R>
__device__ __forceinline__ void cache_rows(const int32_t *cu_q, const int32_t *cu_k,
                                           const int32_t *seqlens, int S, int row, int total_q,
                                           int *status, long long (&at)[R]) {
  const int lane = threadIdx.x & 31, first = __shfl_sync(0xffffffffu, row, 0);
  const int rows = __ldg(cu_q + S);  // of the sequences; beside the search, not before it
  int q0 = 0, q1 = 0;
  long long base = -1;  // the cache row of query row q0, -1: the sequence is skipped
  auto look = [&](int r) {
    const int s = find_seq_warp(cu_q, S, r, lane);
    q0 = __ldg(cu_q + s);
    q1 = __ldg(cu_q + s + 1);
    const int k0 = __ldg(cu_k + s), cap = __ldg(cu_k + s + 1) - k0;
    const int len = seqlens ? __ldg(seqlens + s) : cap;
    base = (long long)k0 + len - (q1 - q0);
    if (r >= rows) {  // and all that come after it
      base = -1;
      q1 = INT_MAX;
    } else if (k0 % BLK != 0) {
      raise_status(status, HISA_ERR_UNALIGNED);
      base = -1;
    } else if (len < 0 || len > cap || len < q1 - q0 || r < q0 || r >= q1) {
      raise_status(status, HISA_ERR_INVALID_ARG);
      base = -1;
      q1 = r + 1;  // the next row looks for itself
    }
  };
  look(min(first, total_q - 1));
  if (first + 2 * R <= q1 && first + 2 * R <= total_q) {  // all of one sequence
#pragma unroll
    for (int i = 0; i < R; i++) at[i] = base < 0 ? -1 : base + (row + 2 * i - q0);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2 * R; i++) {  // the warp's rows in order
    const int r = first + i;
    if (r < total_q && r >= q1) look(r);
    if (lane / 16 == i % 2) at[i / 2] = r < total_q && base >= 0 ? base + (r - q0) : -1;
  }
}

template <int R>
__global__ void __launch_bounds__(KVS_THREADS)
kv4_store_kernel(const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new,
                 const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k,
                 const int32_t *__restrict__ seqlens, int S, int total_q,
                 uint8_t *__restrict__ kv4, uint8_t *__restrict__ kv4_scale, int *status) {
  const int lane = threadIdx.x & 31, g = lane % KV4_NS;
  const int row = (blockIdx.x * KVS_WARPS + threadIdx.x / 32) * 2 * R + lane / 16;
  const uint4 *from = reinterpret_cast<const uint4 *>((g < 8 ? k_new : v_new) +
                                                      (size_t)row * KV4_DIM + (g & 7) * KV4_GROUP);
  uint4 x[R][2];
#pragma unroll
  for (int i = 0; i < R; i++) {
    x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (row + 2 * i < total_q) {
      x[i][0] = __ldg(from + (size_t)i * 2 * (KV4_DIM / 8));
      x[i][1] = __ldg(from + (size_t)i * 2 * (KV4_DIM / 8) + 1);
    }
  }
  long long dst[R];
  cache_rows<R>(cu_q, cu_k, seqlens, S, row, total_q, status, dst);
#pragma unroll
  for (int i = 0; i < R; i++) {
    if (dst[i] < 0) continue;
    const uint4 a = x[i][0], b = x[i][1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) mx = __vmaxu2(mx, w[j] & 0x7FFF7FFFu);
    mx = max(mx & 0xFFFFu, mx >> 16);
    uint32_t byte, c[2] = {0x88888888u, 0x88888888u};
    if (mx >= 0x7F80u) {  // an infinity or a NaN: the group reads back as NaN
      byte = 255u;
      raise_status(status, HISA_ERR_INVALID_ARG);
    } else {
      byte = e5m3_seventh(__uint_as_float(mx << 16));
      const float s = e5m3_value(byte);
      const float r = s > 0.f ? reciprocal(s) : 0.f;
      // |x / s| < 7.5 by the choice of s, but for the largest and the subnormal scales
      if (byte < 8u || byte == KV4_MAX_SCALE) {
        c[0] = nibbles<true>(w, r);
        c[1] = nibbles<true>(w + 4, r);
      } else {
        c[0] = nibbles<false>(w, r);
        c[1] = nibbles<false>(w + 4, r);
      }
    }
    *reinterpret_cast<uint2 *>(kv4 + (size_t)dst[i] * KV4_ROW + g * 8) = make_uint2(c[0], c[1]);
    kv4_scale[(size_t)dst[i] * KV4_NS + g] = (uint8_t)byte;
  }
}

template <int R>
__global__ void __launch_bounds__(KVS_THREADS)
kv4_load_kernel(const uint8_t *__restrict__ kv4, const uint8_t *__restrict__ kv4_scale,
                const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k,
                const int32_t *__restrict__ seqlens, int S, int total_q,
                uint16_t *__restrict__ k_out, uint16_t *__restrict__ v_out, int *status) {
  const int lane = threadIdx.x & 31, g = lane % KV4_NS;
  const int row = (blockIdx.x * KVS_WARPS + threadIdx.x / 32) * 2 * R + lane / 16;
  long long src[R];
  cache_rows<R>(cu_q, cu_k, seqlens, S, row, total_q, status, src);
  uint2 c[R];
  uint32_t b[R];
#pragma unroll
  for (int i = 0; i < R; i++) {
    c[i] = make_uint2(0x88888888u, 0x88888888u);  // zeros
    b[i] = 0;
    if (src[i] >= 0) {
      c[i] = __ldg(reinterpret_cast<const uint2 *>(kv4 + (size_t)src[i] * KV4_ROW + g * 8));
      b[i] = __ldg(kv4_scale + (size_t)src[i] * KV4_NS + g);
    }
  }
  uint4 *to = reinterpret_cast<uint4 *>((g < 8 ? k_out : v_out) + (size_t)row * KV4_DIM +
                                        (g & 7) * KV4_GROUP);
#pragma unroll
  for (int i = 0; i < R; i++) {
    if (row + 2 * i >= total_q) continue;
    const __nv_bfloat162 s = __float2bfloat162_rn(e5m3_value(b[i] > KV4_MAX_SCALE ? 255u : b[i]));
    uint32_t o[8];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      // nibbles j and j + 4 of the word as 128 + u in bf16; minus 136 and times s, both exact
      uint32_t e[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const uint32_t t = (((h ? c[i].y : c[i].x) >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
        const __nv_bfloat162 v =
            __hmul2(__hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&t),
                            __float2bfloat162_rn(-136.f)), s);
        e[j] = *reinterpret_cast<const uint32_t *>(&v);
      }
      o[4 * h] = __byte_perm(e[0], e[1], 0x5410);
      o[4 * h + 1] = __byte_perm(e[2], e[3], 0x5410);
      o[4 * h + 2] = __byte_perm(e[0], e[1], 0x7632);
      o[4 * h + 3] = __byte_perm(e[2], e[3], 0x7632);
    }
    to[(size_t)i * 2 * (KV4_DIM / 8)] = make_uint4(o[0], o[1], o[2], o[3]);
    to[(size_t)i * 2 * (KV4_DIM / 8) + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// Rows of a warp: 4 once that still leaves two CTAs for every SM (16 rows of a CTA).  Stored
// and read back, 131072 rows take 37 us with 2, 34 with 4 and 37 with 8; 16 rows 4.9 with 2,
// 6.2 with 4 and 8.5 with 8.
static int rows_per_unit(int total_q, int num_sms) { return total_q >= 32 * num_sms ? 2 : 1; }
static int store_grid(int total_q, int r) {
  const int per = KVS_WARPS * 2 * r;
  return (total_q + per - 1) / per;
}

cudaError_t launch_kv4_store(const uint16_t *k_new, const uint16_t *v_new, const int32_t *cu_q,
                             const int32_t *cu_k, const int32_t *seqlens, int S, int total_q,
                             uint8_t *kv4, uint8_t *kv4_scale, int num_sms, int *status,
                             cudaStream_t st) {
  const int r = rows_per_unit(total_q, num_sms);
  ProfScope ps(K_KV4_STORE, st);
  const auto fn = r == 2 ? kv4_store_kernel<2> : kv4_store_kernel<1>;
  fn<<<store_grid(total_q, r), KVS_THREADS, 0, st>>>(k_new, v_new, cu_q, cu_k, seqlens, S, total_q,
                                                     kv4, kv4_scale, status);
  return cudaGetLastError();
}

cudaError_t launch_kv4_load(const uint8_t *kv4, const uint8_t *kv4_scale, const int32_t *cu_q,
                            const int32_t *cu_k, const int32_t *seqlens, int S, int total_q,
                            uint16_t *k_out, uint16_t *v_out, int num_sms, int *status,
                            cudaStream_t st) {
  const int r = rows_per_unit(total_q, num_sms);
  ProfScope ps(K_KV4_LOAD, st);
  const auto fn = r == 2 ? kv4_load_kernel<2> : kv4_load_kernel<1>;
  fn<<<store_grid(total_q, r), KVS_THREADS, 0, st>>>(kv4, kv4_scale, cu_q, cu_k, seqlens, S,
                                                     total_q, k_out, v_out, status);
  return cudaGetLastError();
}

}  // namespace hisa
