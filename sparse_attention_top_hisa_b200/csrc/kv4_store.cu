// Storing rows in the 4-bit cache and reading them back (hisa_kv4_store, hisa_kv4_load).
//
// Per group of 16 dimensions, with a = max |x|:
//   s = a / 7 rounded to nearest even in e5m3, at most 896;   q = x / s rounded to nearest
//   even, clamped to -7..7.
// Every decision is the exact one.  a and x have 8 significant bits, and a tie of a / 7
// lies at 7 * (a 5-bit number) and one of x / s at s * (a 4-bit number): both are 8-bit
// numbers, so a quotient that is not a tie is at least 2^-8 (relative) from one, and the
// correctly rounded fp32 quotient falls on the right side.  For x / s the product with
// the rounded reciprocal of s is taken instead and rounded to a multiple of 2^-12 first,
// which puts ties back where they belong and moves nothing else across one.
//
// A sequence with fewer live tokens than query rows is skipped whole, like one whose
// region or length does not fit (locate).
//
// One thread per group (16 per row, 8 of the key and 8 of the value): a store reads 512
// bytes per row and writes 144, a load the reverse, so both are bound by memory.
#include <cuda_bf16.h>

#include "kv4.cuh"
#include "prof.cuh"

namespace hisa {

constexpr int KVS_THREADS = 256;
constexpr int KVS_ROWS = KVS_THREADS / KV4_NS;  // rows of a CTA

// e5m3 byte of t >= 0 (finite), rounded to nearest even, at most 896 (byte 198)
__device__ __forceinline__ uint32_t e5m3_round(float t) {
  uint32_t b;
  if (t < 0x1p-14f) {
    b = (uint32_t)__float2int_rn(t * 0x1p17f);  // multiples of 2^-17; 8 is 2^-14
  } else {
    uint32_t u = __float_as_uint(t);
    u += 0x7FFFFu + ((u >> 20) & 1u);
    b = (u >> 20) - ((127u - 15u) << 3);
  }
  return min(b, 198u);
}

__device__ __forceinline__ float e5m3_value(uint32_t b) {
  return __half2float(__ushort_as_half((unsigned short)(b << 7)));
}

__device__ __forceinline__ QueryInfo locate_new(const int32_t *cu_q, const int32_t *cu_k,
                                                const int32_t *seqlens, int S, int row,
                                                int *status) {
  QueryInfo r = locate(cu_q, cu_k, seqlens, S, row, status);
  if (r.ok && r.len < __ldg(cu_q + r.seq + 1) - __ldg(cu_q + r.seq)) {
    raise_status(status, HISA_ERR_INVALID_ARG);
    r.ok = false;
  }
  return r;
}

__global__ void __launch_bounds__(KVS_THREADS)
kv4_store_kernel(const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new,
                 const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k,
                 const int32_t *__restrict__ seqlens, int S, int total_q,
                 uint8_t *__restrict__ kv4, uint8_t *__restrict__ kv4_scale, int *status) {
  const int row = blockIdx.x * KVS_ROWS + threadIdx.x / KV4_NS, g = threadIdx.x % KV4_NS;
  if (row >= total_q) return;
  const QueryInfo qi = locate_new(cu_q, cu_k, seqlens, S, row, status);
  if (!qi.ok) return;
  const uint4 *src = reinterpret_cast<const uint4 *>(
      (g < 8 ? k_new : v_new) + (size_t)row * KV4_DIM + (g & 7) * KV4_GROUP);
  const uint4 a = __ldg(src), b = __ldg(src + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) mx = __vmaxu2(mx, w[i] & 0x7FFF7FFFu);
  mx = max(mx & 0xFFFFu, mx >> 16);
  const size_t dst = (size_t)(qi.kbase + qi.pos);
  uint32_t byte, lo = 0x88888888u, hi = 0x88888888u;
  if (mx >= 0x7F80u) {  // an infinity or a NaN: the group reads back as NaN
    byte = 255u;
    raise_status(status, HISA_ERR_INVALID_ARG);
  } else {
    byte = e5m3_round(__fdiv_rn(__uint_as_float(mx << 16), 7.f));
    const float s = e5m3_value(byte);
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const float x = (i & 1) ? bf_hi(w[i >> 1]) : bf_lo(w[i >> 1]);
      float t = fmaf(x, r, 3072.f) - 3072.f;  // multiples of 2^-12
      t = fminf(fmaxf(t, -7.f), 7.f) + 12582912.f;  // 1.5 * 2^23: rounds to a whole number
      c[i >> 3] |= ((__float_as_uint(t) + 8u) & 15u) << (4 * (i & 7));
    }
    lo = c[0];
    hi = c[1];
  }
  *reinterpret_cast<uint2 *>(kv4 + dst * KV4_ROW + g * 8) = make_uint2(lo, hi);
  kv4_scale[dst * KV4_NS + g] = (uint8_t)byte;
}

__global__ void __launch_bounds__(KVS_THREADS)
kv4_load_kernel(const uint8_t *__restrict__ kv4, const uint8_t *__restrict__ kv4_scale,
                const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k,
                const int32_t *__restrict__ seqlens, int S, int total_q,
                uint16_t *__restrict__ k_out, uint16_t *__restrict__ v_out, int *status) {
  const int row = blockIdx.x * KVS_ROWS + threadIdx.x / KV4_NS, g = threadIdx.x % KV4_NS;
  if (row >= total_q) return;
  const QueryInfo qi = locate_new(cu_q, cu_k, seqlens, S, row, status);
  uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  if (qi.ok) {
    const size_t src = (size_t)(qi.kbase + qi.pos);
    const uint2 c = __ldg(reinterpret_cast<const uint2 *>(kv4 + src * KV4_ROW + g * 8));
    const float s = e5m3_value(__ldg(kv4_scale + src * KV4_NS + g));
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t w = (i < 4 ? c.x : c.y) >> (8 * (i & 3));
      const float x = (float)((int)(w & 15u) - 8) * s, y = (float)((int)((w >> 4) & 15u) - 8) * s;
      const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
      o[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
  }
  uint4 *dst = reinterpret_cast<uint4 *>((g < 8 ? k_out : v_out) + (size_t)row * KV4_DIM +
                                         (g & 7) * KV4_GROUP);
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

cudaError_t launch_kv4_store(const uint16_t *k_new, const uint16_t *v_new, const int32_t *cu_q,
                             const int32_t *cu_k, const int32_t *seqlens, int S, int total_q,
                             uint8_t *kv4, uint8_t *kv4_scale, int *status, cudaStream_t st) {
  const int grid = (total_q + KVS_ROWS - 1) / KVS_ROWS;
  ProfScope ps(K_KV4_STORE, st);
  kv4_store_kernel<<<grid, KVS_THREADS, 0, st>>>(k_new, v_new, cu_q, cu_k, seqlens, S, total_q,
                                                 kv4, kv4_scale, status);
  return cudaGetLastError();
}

cudaError_t launch_kv4_load(const uint8_t *kv4, const uint8_t *kv4_scale, const int32_t *cu_q,
                            const int32_t *cu_k, const int32_t *seqlens, int S, int total_q,
                            uint16_t *k_out, uint16_t *v_out, int *status, cudaStream_t st) {
  const int grid = (total_q + KVS_ROWS - 1) / KVS_ROWS;
  ProfScope ps(K_KV4_LOAD, st);
  kv4_load_kernel<<<grid, KVS_THREADS, 0, st>>>(kv4, kv4_scale, cu_q, cu_k, seqlens, S, total_q,
                                                k_out, v_out, status);
  return cudaGetLastError();
}

}  // namespace hisa
