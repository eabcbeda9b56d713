// Sparse attention over the 4-bit cache, and the attention weight of every token
// (hisa_sparse_attention_kv4, hisa_token_weights).
//
//   s_j = scale * q[i][h] . k_j,   out[i][h] = sum_j softmax(s)_j v_j,
//   weight[j] += sum_h softmax(s)_j
//
// over the entries j >= 0 of the index row.  One warp takes 32 selected tokens at a time
// and does everything to them: it copies their rows (144 bytes each) into a ring of its
// own, turns the key nibbles into fp16 fragments, multiplies, keeps the running maximum
// and sum of its share, turns the value nibbles into fragments and multiplies again.  With
// many rows a warp has a row to itself; with few, the warps of a CTA and the CTAs of a
// cluster share one and are merged by their maxima and sums.
//
// The fragments' dimensions are assigned so that no value moves between lanes.  With
// g = lane / 4 and c = lane % 4, in m16n8k16:
//   scores   rows = heads, columns n = tokens, k = dimensions.  Lane (g, c) supplies
//            token g with dimensions 32c .. 32c + 31: 16 bytes of nibbles, 2 scales.
//   output   rows = heads, k = tokens, columns n = dimensions.  The score fragment's
//            tokens (columns 2c, 2c + 1 of two tiles) are already where the weights are
//            needed; lane (g, c) supplies those four tokens with dimensions 16g .. 16g +
//            15: 8 bytes of nibbles and one scale of each.
// A register with the nibbles of dimensions d and d + 4 (scores) or of two tokens
// (output) becomes an fp16 pair by one logic operation and one FMA (kv4.cuh).
//
// Precision: q (bf16) is held as fp16 times a power of two per head, exact over 29 binades
// below the head's largest value; the products are exact and summed in fp32; maxima and
// sums are fp32; the softmax weights enter the value product as fp16.  They are taken
// against a reference 2^7 below a maximum that later ones pass by 2^8 at most, so that they
// use fp16's whole range: at most 2^15, and the largest of a share at least 2^7.  A weight of
// 2^-21 of that one and more is off by at most 2^-11 of itself (an eighth of the bf16
// output's own rounding); a smaller one by half the smallest fp16 number, 2^-25, which is
// 2^-32 of it.  n selected tokens are so off by at most n 2^-32 of the largest value.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "kv4.cuh"
#include "prof.cuh"
#include "tc.cuh"

namespace cg = cooperative_groups;

namespace hisa {

constexpr int A4_STEP = 32;                                   // tokens of a warp's step
constexpr int A4_CODES = A4_STEP * KV4_ROW;                   // 4096 bytes
constexpr int A4_STAGE = A4_CODES + A4_STEP * KV4_NS;         // 4608
constexpr int A4_MAX_CLUSTER = 8;
// A head's reference: this many powers of two below its maximum when it was last raised, and
// how far a score may pass the reference before it is raised again.
constexpr float A4_BELOW = 7.f, A4_TOP = A4_BELOW + 8.f;
constexpr int A4_OSTRIDE = KV4_DIM + 4;                       // padded row of partial outputs
constexpr float LOG2E = 1.4426950408889634f, LOG2E_LO = 1.92596303e-8f, LN2 = 0.6931471805599453f;

constexpr int A4_WARPS = 4, A4_THREADS = A4_WARPS * 32;
__host__ __device__ constexpr int a4_stages(int MT) { return MT == 1 ? 2 : 4; }
// CTAs of an SM: one or two 16-head tiles in up to 168 or 255 registers per thread
__host__ __device__ constexpr int a4_ctas(int MT) { return MT == 1 ? 3 : 2; }
// a warp's ring, which later holds its partial output
__host__ __device__ constexpr int a4_ring(int MT) { return a4_stages(MT) * A4_STAGE; }
static_assert(16 * A4_OSTRIDE * 4 <= a4_ring(1) && 32 * A4_OSTRIDE * 4 <= a4_ring(2),
              "a warp's partial output fits its ring");

// 16-byte chunk of token t's 128-byte row: the key chunks of two neighbouring tokens, and
// the value chunks of every second token, fall into different banks
__device__ __forceinline__ int a4_chunk(int t, int chunk) {
  return chunk ^ (((t >> 1) & 3) << 1) ^ ((t & 1) << 2);
}

// What bounds it: no unit alone.  A step of 32 tokens and 16 heads takes about 645
// instructions, its 64 matrix instructions among them (352 turn 8192 nibbles into fp16), on
// three warps per scheduler: issue slots are 58% full, ALU and matrix pipe 47% and 45%, and the
// warps wait for a pipe, for the instruction before or for dispatch.  The gather (160 bytes of
// L2 sectors per token, 5.0 TB/s of the 17 the same copies reach alone) and DRAM are idle
// beside it.  8192 queries x 2048 tokens x 16 heads: 537 us, 256 TFLOP/s; 4096 queries of 32
// heads: 454 us, 302 TFLOP/s (two warps per scheduler, matrix pipe 54%).  Measured and left
// out: the value product of one step written between the scores of the next (658
// against 637 us at the time), four CTAs per SM of 128 registers (697, spills), and the
// same products on the tensor core that reads shared memory, with the tokens as its rows: it
// takes about 85 cycles for each 128 tokens x 16 dimensions whatever the number of heads up
// to 32, so the scores alone would cost 170 cycles of a step's 290.

// 16 bytes global -> shared; zeros when !ok
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
// the warp's number, told to the compiler as one that all its lanes share
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
}

// A load from shared memory by its 32-bit address: the walks below keep such addresses, at
// half the registers of pointers.
template <typename T>
__device__ __forceinline__ T lds(uint32_t at) {
  return *reinterpret_cast<const T *>(__cvta_shared_to_generic(at));
}

// p + j * KV4_ROW in one multiply-add
__device__ __forceinline__ const uint8_t *row_of(const uint8_t *p, int j) {
  uint64_t r;
  asm("mad.wide.u32 %0, %1, %2, %3;"
      : "=l"(r)
      : "r"(j), "r"(KV4_ROW), "l"(reinterpret_cast<uint64_t>(p)));
  return reinterpret_cast<const uint8_t *>(r);
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Power of two that brings a head's largest |q| (as bf16 bits) to [2^14, 2^15), and what
// undoes it.  1 for a head of zeros or with an infinity or NaN.
__device__ __forceinline__ void q_shift(uint32_t max_bits, float &up, float &down) {
  const int e = (int)(max_bits >> 7);  // biased exponent
  up = down = 1.f;
  if (max_bits == 0u || e == 255) return;
  const int sh = min(126, max(-126, 127 + 14 - max(e, 1)));
  up = __uint_as_float((uint32_t)(127 + sh) << 23);
  down = __uint_as_float((uint32_t)(127 - sh) << 23);
}

// The query fragments, in shared memory as [mt][ks][lane] of 16 bytes: fragment ks = 2w +
// half of a 16-head tile holds the dimension pairs (d, d + 4) of word w (32c + 8w ..), d = 0
// and 1 (half 0) or 2 and 3; heads >= H are zeros.  In registers (32 for 16 heads) they
// left the compiler too few to overlap its work: 663 us instead of 637 for 8192 queries of
// 16 heads on 2048 tokens each.
// Each of the W warps that share a query looks at all of it (QueryRaw), since it needs the
// heads' powers of two (f: what takes its raw scores, of heads g and g + 8, to exponents of
// two), and converts its part; the caller synchronises them.
template <int MT>
struct QueryRaw {
  uint4 w[MT][2][4];  // dimensions 32c .. 32c + 31 of heads g and g + 8
  __device__ __forceinline__ void load(const uint16_t *__restrict__ q, size_t row, int H,
                                       int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int r = 0; r < 2; r++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int h = 16 * mt + g + 8 * r;
          w[mt][r][i] = make_uint4(0u, 0u, 0u, 0u);
          if (h < H)
            w[mt][r][i] =
                __ldg(reinterpret_cast<const uint4 *>(q + (row * H + h) * KV4_DIM + 32 * c) + i);
        }
  }
};
template <int MT, int W>
__device__ __forceinline__ void convert_query(const QueryRaw<MT> &raw, float scale, uint4 *qs,
                                              int lane, int warp, float (&f)[MT][2]) {
#pragma unroll
  for (int mt = 0; mt < MT; mt++) {
    const auto &w = raw.w[mt];
    float up[2];
#pragma unroll
    for (int r = 0; r < 2; r++) {
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint4 v = w[r][i];
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                   __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
      }
      mx = max(mx & 0xFFFFu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      float down;
      q_shift(mx, up[r], down);
      f[mt][r] = down * (scale * LOG2E);
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
      if ((4 * mt + i) % W == warp % W) {
        uint32_t t[2][4];  // [r][pair]
#pragma unroll
        for (int r = 0; r < 2; r++) {
          const uint4 v = w[r][i];
          // dimensions 0..7 of the word: pairs (0,4) (1,5) (2,6) (3,7)
          t[r][0] = as_u32(__floats2half2_rn(bf_lo(v.x) * up[r], bf_lo(v.z) * up[r]));
          t[r][1] = as_u32(__floats2half2_rn(bf_hi(v.x) * up[r], bf_hi(v.z) * up[r]));
          t[r][2] = as_u32(__floats2half2_rn(bf_lo(v.y) * up[r], bf_lo(v.w) * up[r]));
          t[r][3] = as_u32(__floats2half2_rn(bf_hi(v.y) * up[r], bf_hi(v.w) * up[r]));
        }
        uint4 *d = qs + (mt * 8 + 2 * i) * 32 + lane;
        d[0] = make_uint4(t[0][0], t[1][0], t[0][1], t[1][1]);
        d[32] = make_uint4(t[0][2], t[1][2], t[0][3], t[1][3]);
      }
  }
}

// A lane's places in a ring stage: the swizzle of a token's row depends on the token modulo
// 8 only, so every other token is a constant distance away.  Rows without their value half
// (VALUES false) need no swizzle: two of them fill the banks.
template <bool VALUES>
struct LanePlaces {
  static constexpr int ROW = VALUES ? KV4_ROW : KV4_HALF, CODES = A4_STEP * ROW;
  static constexpr int STAGE = CODES + A4_STEP * KV4_NS;
  uint32_t kc, ks;        // token g: the lane's 16 key bytes, its two key scales
  uint32_t v0, v1;        // tokens 2c and 2c + 1: the lane's 8 value bytes
  uint32_t s0;            // token 2c: its value scale
  uint32_t d0, d1;        // copies: chunks lane % 4 and lane % 4 + 4 of token lane / 4
  __device__ __forceinline__ explicit LanePlaces(int lane) {
    const int g = lane >> 2, c = lane & 3, t = 2 * c;
    kc = g * ROW + ((VALUES ? a4_chunk(g, c) : c) << 4);
    ks = CODES + g * KV4_NS + 2 * c;
    d0 = kc;
    d1 = g * KV4_ROW + (a4_chunk(g, c + 4) << 4);
    v0 = t * KV4_ROW + (a4_chunk(t, 4 + (g >> 1)) << 4) + (g & 1) * 8;
    v1 = (t + 1) * KV4_ROW + (a4_chunk(t + 1, 4 + (g >> 1)) << 4) + (g & 1) * 8;
    s0 = CODES + t * KV4_NS + 8 + g;
  }
};

// Raw scores of the tokens 8j0 .. 8(j0 + J) - 1 of a ring stage: s[mt] are their score
// fragments.  qs: the query fragments at this lane's place (shared address).  J octets of
// tokens side by side share the query's loads and give the matrix unit independent sums (8192
// queries of 2048 tokens: 541 us by twos, 552 one by one or by fours; 32 heads, 2.5 M entries:
// 188 us against 238, the registers being fewer too).
template <int J, int MT, typename LP>
__device__ __forceinline__ void kv4_scores(uint32_t stage, int j0, const LP &lp, uint32_t qs,
                                           uint32_t magic, float (&s)[MT][4][4]) {
  uint32_t w[J][4], sb[J];
#pragma unroll
  for (int j = 0; j < J; j++) {
    const uint4 kw = lds<uint4>(stage + lp.kc + (j0 + j) * 8 * LP::ROW);
    w[j][0] = kw.x;
    w[j][1] = kw.y;
    w[j][2] = kw.z;
    w[j][3] = kw.w;
    sb[j] = lds<uint16_t>(stage + lp.ks + (j0 + j) * 8 * KV4_NS);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    uint32_t b[J][4];
#pragma unroll
    for (int j = 0; j < J; j++) {
      // both halves of the scale pair: byte 0 (words 0, 1) or byte 1 (words 2, 3)
      const __half2 sc = as_half2(__byte_perm(sb[j], 0u, i < 2 ? 0x4040 : 0x4141) << 7);
      const __half2 c72 = kv4_c72(sc);
      b[j][0] = kv4_pair(w[j][i] << 4, magic, sc, c72);
      b[j][1] = kv4_pair(w[j][i], magic, sc, c72);
      b[j][2] = kv4_pair(w[j][i] >> 4, magic, sc, c72);
      b[j][3] = kv4_pair(w[j][i] >> 8, magic, sc, c72);
    }
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      const uint4 qa = lds<uint4>(qs + (mt * 8 + 2 * i) * 512);
      const uint4 qb = lds<uint4>(qs + (mt * 8 + 2 * i + 1) * 512);
#pragma unroll
      for (int j = 0; j < J; j++)
        if (i == 0)
          mma_f16_first(s[mt][j0 + j], qa.x, qa.y, qa.z, qa.w, b[j][0], b[j][1]);
        else
          mma_f16(s[mt][j0 + j], qa.x, qa.y, qa.z, qa.w, b[j][0], b[j][1]);
#pragma unroll
      for (int j = 0; j < J; j++)
        mma_f16(s[mt][j0 + j], qb.x, qb.y, qb.z, qb.w, b[j][2], b[j][3]);
    }
  }
}

// The value fragments' raw material of 16 tokens (half i of a stage).
struct ValueRaw {
  uint2 v[4];              // nibbles of the tokens 2c, 2c + 1, 2c + 8, 2c + 9
  __half2 s0, s1, k0, k1;  // their scales in pairs, and -72 times them
  __device__ __forceinline__ void load(uint32_t stage, int i, const LanePlaces<true> &lp) {
    uint32_t sb[4];
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int t = 16 * i + 8 * (u >> 1);
      v[u] = lds<uint2>(stage + ((u & 1) ? lp.v1 : lp.v0) + t * KV4_ROW);
      sb[u] = lds<uint8_t>(stage + lp.s0 + (t + (u & 1)) * KV4_NS);
    }
    s0 = as_half2(__byte_perm(sb[0], sb[1], 0x5410) << 7);
    s1 = as_half2(__byte_perm(sb[2], sb[3], 0x5410) << 7);
    k0 = kv4_c72(s0);
    k1 = kv4_c72(s1);
  }
};

// o += weights p (of 16 tokens: half i) times dimensions 8b .. 8b + 7 of every group
template <int MT>
__device__ __forceinline__ void kv4_values(const ValueRaw &r, int i, int b,
                                           const uint32_t (&p)[MT][4][2], uint32_t magic,
                                           float (&o)[MT][16][4]) {
#pragma unroll
  for (int w = 2 * b; w < 2 * b + 2; w++) {  // dimensions 4w .. 4w + 3
    const uint32_t sel = (w & 1) ? 0x7632 : 0x5410;
    const uint32_t r0 =
        b ? __byte_perm(r.v[0].y, r.v[1].y, sel) : __byte_perm(r.v[0].x, r.v[1].x, sel);
    const uint32_t r1 =
        b ? __byte_perm(r.v[2].y, r.v[3].y, sel) : __byte_perm(r.v[2].x, r.v[3].x, sel);
#pragma unroll
    for (int d = 0; d < 4; d++) {
      const uint32_t b0 = kv4_pair(d == 0 ? r0 << 4 : r0 >> (4 * d - 4), magic, r.s0, r.k0);
      const uint32_t b1 = kv4_pair(d == 0 ? r1 << 4 : r1 >> (4 * d - 4), magic, r.s1, r.k1);
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
        mma_f16(o[mt][4 * w + d], p[mt][2 * i][0], p[mt][2 * i][1], p[mt][2 * i + 1][0],
                p[mt][2 * i + 1][1], b0, b1);
    }
  }
}

// A warp's walk over its steps: the token ids are read one step ahead of the copies, the
// copies run AHEAD = NST - 1 steps ahead of the products, over NST stages.
// VALUES: the value halves of the rows are copied too.
template <int NST, int AHEAD, bool VALUES>
struct Ring {
  using LP = LanePlaces<VALUES>;
  const int32_t *irow;
  int e1, nsteps, next_e, stride;   // this lane's entry of the next step to read, up to e1
  int first_e;                      // and of the first
  int kcap;
  const uint8_t *codes, *scales;    // the region's first row; codes at this lane's chunk
  uint32_t ring, slot, fill;        // shared address; bytes to the stage of the next step, and copy
  int next_tok;                     // this lane's token of the next step to copy (-1 = none)
  uint32_t mask[AHEAD];             // valid tokens of the steps in flight, oldest first
  bool bad;

  // steps first, first + stride, ... of the entries [e0, e1)
  __device__ __forceinline__ void init(const int32_t *row, int e0, int end, int first, int step,
                                       int kbase, int cap, const uint8_t *kv4,
                                       const uint8_t *kv4_scale, uint8_t *mem, int lane) {
    entries(row, e0, end, first, step, lane);
    region(kbase, cap, kv4, kv4_scale, mem, lane);
  }
  __device__ __forceinline__ void entries(const int32_t *row, int e0, int end, int first, int step,
                                          int lane) {
    irow = row;
    e1 = end;
    const int steps = end > e0 ? (end - e0 + A4_STEP - 1) / A4_STEP : 0;
    nsteps = steps > first ? (steps - first + step - 1) / step : 0;
    first_e = next_e = e0 + first * A4_STEP + lane;
    stride = step * A4_STEP;
    bad = false;
    read();
  }
  __device__ __forceinline__ void region(int kbase, int cap, const uint8_t *kv4,
                                         const uint8_t *kv4_scale, uint8_t *mem, int lane) {
    kcap = cap;
    codes = kv4 + (size_t)kbase * KV4_ROW + (lane & 3) * 16;
    scales = kv4_scale + (size_t)kbase * KV4_NS;
    ring = smem_u32(mem);
    slot = fill = 0;
  }
  __device__ __forceinline__ void read() {
    next_tok = next_e < e1 ? __ldg(irow + next_e) : -1;
    next_e += stride;
  }
  static __device__ __forceinline__ uint32_t after(uint32_t at) {
    return at == (NST - 1) * LP::STAGE ? 0 : at + LP::STAGE;
  }
  // start the copy of the next step; the valid tokens in it
  __device__ __forceinline__ uint32_t copy(const LP &lp, int lane) {
    int j = next_tok;
    read();
    if (j >= kcap) {
      bad = true;
      j = -1;
    }
    const uint32_t valid = __ballot_sync(0xffffffffu, j >= 0);
    const uint32_t dst = ring + fill;
    fill = after(fill);
    const uint32_t a0 = dst + lp.d0, a1 = dst + lp.d1;
    // four lanes copy 64 bytes of a token together, eight tokens at a time
    if (valid == 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint8_t *src = row_of(codes, __shfl_sync(0xffffffffu, j, 8 * i + (lane >> 2)));
        cp_async_16(a0 + i * 8 * LP::ROW, src);
        if (VALUES) cp_async_16(a1 + i * 8 * KV4_ROW, src + 64);
      }
      cp_async_16(dst + LP::CODES + lane * KV4_NS, scales + (size_t)(uint32_t)j * KV4_NS);
    } else if (valid) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int jt = __shfl_sync(0xffffffffu, j, 8 * i + (lane >> 2));
        const uint8_t *src = row_of(codes, max(jt, 0));
        cp_async_16_or_zero(a0 + i * 8 * LP::ROW, src, jt >= 0);
        if (VALUES) cp_async_16_or_zero(a1 + i * 8 * KV4_ROW, src + 64, jt >= 0);
      }
      cp_async_16_or_zero(dst + LP::CODES + lane * KV4_NS,
                          scales + (size_t)(uint32_t)max(j, 0) * KV4_NS, j >= 0);
    }
    cp_async_commit();
    return valid;
  }
  __device__ __forceinline__ void start(const LP &lp, int lane) {
#pragma unroll
    for (int n = 0; n < AHEAD; n++) mask[n] = copy(lp, lane);
  }
  // start one more copy, wait for the next step; its stage and the mask of its valid tokens
  __device__ __forceinline__ uint32_t arrive(const LP &lp, int lane, uint32_t &valid) {
    __syncwarp();  // every lane has read the stage that is filled now
    const uint32_t more = copy(lp, lane);
    valid = mask[0];
#pragma unroll
    for (int i = 0; i + 1 < AHEAD; i++) mask[i] = mask[i + 1];
    mask[AHEAD - 1] = more;
    cp_async_wait_group<AHEAD>();
    __syncwarp();  // the step has landed for every lane
    const uint32_t stage = ring + slot;
    slot = after(slot);
    return stage;
  }
};

// Sum over the 8 lanes g of a column c: v[i] (i = 0..7) -> the sum of v[g].
__device__ __forceinline__ float column_sum(float (&v)[8], int g) {
#pragma unroll
  for (int st = 0; st < 3; st++) {
    const int half = 4 >> st, o = 16 >> st;
    const bool up = (g & half) != 0;
#pragma unroll
    for (int i = 0; i < half; i++) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

// Adds the weights of a step's 32 tokens (tok: lane t's is token t, -1 = none).  v[i] = this
// lane's heads' sum for column i & 1 of tile i >> 1.
__device__ __forceinline__ void add_weights(float (&v)[8], int tok, unsigned long long *weights,
                                            int lane, int *status) {
  const float w = column_sum(v, lane >> 2);
  // lane (g, c) holds value g of column pair c: token 8 (g / 2) + 2c + g % 2
  const int g = lane >> 2, c = lane & 3;
  const int j = __shfl_sync(0xffffffffu, tok, 8 * (g >> 1) + 2 * c + (g & 1));
  if (j < 0) return;
  if (!(w < 4096.f)) {  // NaN or beyond any softmax
    raise_status(status, HISA_ERR_INVALID_ARG);
    return;
  }
  const unsigned long long fx = __float2ull_rn(w * 4294967296.f);
  if (fx) atomicAdd(weights + j, fx);
}

// Factor of a share with reference m and sum l in a merge whose largest is mx: 0 for a share
// of no score; a share that holds a NaN keeps it whatever its maximum says.
__device__ __forceinline__ float share_factor(float m, float l, float mx) {
  return l != l ? l : m == -__int_as_float(0x7f800000) ? 0.f : ex2(m - mx);
}

__device__ __forceinline__ void add_share(float4 &acc, float a, const float4 &v) {
  acc.x = fmaf(a, v.x, acc.x);
  acc.y = fmaf(a, v.y, acc.y);
  acc.z = fmaf(a, v.z, acc.z);
  acc.w = fmaf(a, v.w, acc.w);
}

// four values of head h's partial output, summed over W warps
template <int W>
__device__ __forceinline__ float4 sum_shares(const uint8_t *smem, int ring, const float *factor,
                                             int NH, int h, int at) {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < W; w++)
    add_share(acc, factor[w * NH + h],
              *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w * ring) +
                                                at));
  return acc;
}

__device__ __forceinline__ void store_out(uint16_t *dst, const float4 &v, float by) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * by, v.y * by);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.z * by, v.w * by);
  *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}

// A warp's running state over its tokens: unnormalised outputs, references (in exponents of
// two) and sums of its 16-head tiles.
template <int MT>
struct Running {
  float o[MT][16][4];
  float m[MT][2];   // -inf before the first step, and only then
  float2 l[MT][2];  // sums of the even and of the odd columns
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int t = 0; t < 16; t++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[mt][t][e] = 0.f;
#pragma unroll
      for (int r = 0; r < 2; r++) {
        m[mt][r] = -__int_as_float(0x7f800000);
        l[mt][r] = make_float2(0.f, 0.f);
      }
    }
  }
  // the sum of a head over the quad's columns
  __device__ __forceinline__ float total(int mt, int r) const {
    float sum = l[mt][r].x + l[mt][r].y;
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    return sum + __shfl_xor_sync(0xffffffffu, sum, 2);
  }
};

// All steps of a warp's ring.
template <int MT, typename R>
__device__ __forceinline__ void attend(R &ring, const LanePlaces<true> &lp, uint32_t qf,
                                       const float (&f)[MT][2], int lane, Running<MT> &st) {
  const float NEG = -__int_as_float(0x7f800000);
  const int c = lane & 3;
  const uint32_t magic = kv4_magic();
  auto &o = st.o;
  auto &m = st.m;
  auto &l = st.l;
  for (int n = 0; n < ring.nsteps; n++) {
    uint32_t valid;
    const uint32_t stage = ring.arrive(lp, lane, valid);
    if (!valid) continue;
    float x[MT][4][4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) kv4_scores<2>(stage, j, lp, qf, magic, x);
    // exponents against the references; -inf where there is no token
    float top = NEG;
    float y[MT][4][4];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
          const float2 t = fma2(make_float2(x[mt][j][2 * r], x[mt][j][2 * r + 1]), f[mt][r],
                                -m[mt][r]);
          y[mt][j][2 * r] = t.x;
          y[mt][j][2 * r + 1] = t.y;
        }
    if (valid != 0xffffffffu) {
      const uint32_t v = valid >> (2 * c);
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (!((v >> (8 * j + (e & 1))) & 1u)) y[mt][j][e] = NEG;
    }
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) top = fmaxf(top, y[mt][j][e]);
    // the references rise (and sums and outputs are rescaled) only where a score passes one
    // by 2^A4_TOP; a first score always does
    if (__any_sync(0xffffffffu, top > A4_TOP)) {
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
          float mx = NEG;
#pragma unroll
          for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 2 * r; e < 2 * r + 2; e++)
              if (y[mt][j][e] != NEG) mx = fmaxf(mx, x[mt][j][e] * f[mt][r]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mx = fmaxf(m[mt][r], mx - A4_BELOW);
          const float a = mx == NEG ? 1.f : ex2(m[mt][r] - mx);
          m[mt][r] = mx;
          l[mt][r].x *= a;
          l[mt][r].y *= a;
#pragma unroll
          for (int t = 0; t < 16; t++) {
            o[mt][t][2 * r] *= a;
            o[mt][t][2 * r + 1] *= a;
          }
#pragma unroll
          for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 2 * r; e < 2 * r + 2; e++)
              if (y[mt][j][e] != NEG) y[mt][j][e] = fmaf(x[mt][j][e], f[mt][r], -mx);
        }
    }
    uint32_t p[MT][4][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int r = 0; r < 2; r++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float2 pp = make_float2(ex2(y[mt][j][2 * r]), ex2(y[mt][j][2 * r + 1]));
          l[mt][r] = add2(l[mt][r], pp);
          p[mt][j][r] = as_u32(__floats2half2_rn(pp.x, pp.y));
        }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      ValueRaw r;
      r.load(stage, i, lp);
      kv4_values<MT>(r, i, 0, p, magic, o);
      kv4_values<MT>(r, i, 1, p, magic, o);
    }
  }
  cp_async_wait_all();
  __syncwarp();  // the ring is free
}

// Heads past the last, and those of a row without tokens, have no weights.
template <int MT>
__device__ __forceinline__ void dead_heads(int H, int g, float (&f)[MT][2], float (&m)[MT][2],
                                           float (&inv)[MT][2]) {
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int r = 0; r < 2; r++)
      if (16 * mt + g + 8 * r >= H || m[mt][r] == -__int_as_float(0x7f800000))
        f[mt][r] = m[mt][r] = inv[mt][r] = 0.f;
}

// v += sum over the lane's heads of 2^(x f - m) / l of a step's scores
template <int MT>
__device__ __forceinline__ void weigh_step(int mt, int j, const float4 &t, const float (&f)[MT][2],
                                           const float (&m)[MT][2], const float (&inv)[MT][2],
                                           float (&v)[8]) {
  v[2 * j] = fmaf(ex2(fmaf(t.x, f[mt][0], -m[mt][0])), inv[mt][0], v[2 * j]);
  v[2 * j + 1] = fmaf(ex2(fmaf(t.y, f[mt][0], -m[mt][0])), inv[mt][0], v[2 * j + 1]);
  v[2 * j] = fmaf(ex2(fmaf(t.z, f[mt][1], -m[mt][1])), inv[mt][1], v[2 * j]);
  v[2 * j + 1] = fmaf(ex2(fmaf(t.w, f[mt][1], -m[mt][1])), inv[mt][1], v[2 * j + 1]);
}

// The weights of a warp's tokens from a second look at their keys; m, inv: the row's
// references and inverse sums.
template <int MT, typename R>
__device__ __forceinline__ void weigh_again(R &ring, uint32_t qf,
                                            const float (&f)[MT][2], const float (&m)[MT][2],
                                            const float (&inv)[MT][2], int lane,
                                            unsigned long long *weights, int *status) {
  const uint32_t magic = kv4_magic();
  const typename R::LP lp(lane);
  ring.start(lp, lane);
  const int32_t *entry = ring.irow + ring.first_e;
  for (int n = 0; n < ring.nsteps; n++) {
    uint32_t valid;
    const uint32_t stage = ring.arrive(lp, lane, valid);
    if (!valid) continue;
    const int tok = (valid >> lane) & 1u ? __ldg(entry + (size_t)n * ring.stride) : -1;
    float x[MT][4][4], v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += 2) {
      kv4_scores<2>(stage, j0, lp, qf, magic, x);
#pragma unroll
      for (int j = j0; j < j0 + 2; j++)
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
          weigh_step<MT>(mt, j, make_float4(x[mt][j][0], x[mt][j][1], x[mt][j][2], x[mt][j][3]), f,
                         m, inv, v);
    }
    add_weights(v, tok, weights, lane, status);
  }
  cp_async_wait_all();
}

// A warp's partial output to its ring, [head][dimension] with the 4-value pieces of a
// 32-dimension block turned by the block so that the lanes' stores spread over the banks;
// its references and sums to wm and wl.
template <int MT>
__device__ __forceinline__ void store_share(const Running<MT> &st, uint8_t *ring, float *wm,
                                            float *wl, int lane) {
  const int g = lane >> 2, c = lane & 3;
  float *po = reinterpret_cast<float *>(ring);
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int r = 0; r < 2; r++) {
      const float sum = st.total(mt, r);
      const int h = 16 * mt + g + 8 * r;
      if (c == 0) {
        wm[h] = st.m[mt][r];
        wl[h] = sum;
      }
#pragma unroll
      for (int u = 0; u < 8; u++) {
        // piece u of dimensions 32c ..: tiles 4 (u & 3) .., column 2c + (u >> 2)
        const int e = 2 * r + (u >> 2), t = 4 * (u & 3);
        *reinterpret_cast<float4 *>(po + h * A4_OSTRIDE + 32 * c + 4 * (u ^ (2 * c))) =
            make_float4(st.o[mt][t][e], st.o[mt][t + 1][e], st.o[mt][t + 2][e],
                        st.o[mt][t + 3][e]);
      }
    }
}

// References and sums of W warps' shares of head h: their factors replace the references in wm.
template <int W>
__device__ __forceinline__ void join_shares(float *wm, const float *wl, int NH, int h, float &mx,
                                            float &sum) {
  mx = -__int_as_float(0x7f800000);
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < W; w++) mx = fmaxf(mx, wm[w * NH + h]);
#pragma unroll
  for (int w = 0; w < W; w++) {
    const float lw = wl[w * NH + h], a = share_factor(wm[w * NH + h], lw, mx);
    wm[w * NH + h] = a;
    sum += lw != lw ? lw : a * lw;
  }
}

__device__ __forceinline__ float inverse_sum(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float lse_of(float mx, float sum) {
  return sum == 0.f ? -__int_as_float(0x7f800000) : (mx + log2f(sum)) * LN2;
}

// ---------------------------------------------------------------------------
// Many rows: a row is one warp's, so that its start and end (about 3000 cycles of latency)
// hide behind the other warps of the SM and nothing is merged.

// WT: with weights (a kernel of its own: what the second look needs would cost the first
// one registers, 561 us against 639 at the time for 8192 rows of 2048 tokens and 16 heads).
template <int MT, bool WT>
__global__ void __launch_bounds__(A4_THREADS, a4_ctas(MT))
attn_kv4_rows_kernel(const uint16_t *__restrict__ q, const uint8_t *__restrict__ kv4,
                     const uint8_t *__restrict__ kv4_scale, const int32_t *__restrict__ idx,
                     const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int S,
                     int total_q, int H, int topk, float scale, uint16_t *__restrict__ out,
                     float *__restrict__ lse, unsigned long long *__restrict__ weights,
                     int *status) {
  extern __shared__ __align__(16) uint8_t a4_smem[];
  constexpr int NST = a4_stages(MT), RING = a4_ring(MT);
  const int lane = threadIdx.x & 31, warp = warp_index();
  const int row = blockIdx.x * A4_WARPS + warp;
  if (row >= total_q) return;  // the whole warp; the others do not wait for it
  const int g = lane >> 2, c = lane & 3;
  uint4 *qs = reinterpret_cast<uint4 *>(a4_smem + A4_WARPS * RING + warp * MT * 4096);
  uint8_t *mem = a4_smem + warp * RING;

  const Region rg = region_of(cu_q, cu_k, S, row, lane);
  const int kbase = rg.base, kcap = rg.tokens;
  const LanePlaces<true> lp(lane);
  const int32_t *irow = idx + (size_t)row * topk;
  Ring<NST, NST - 1, true> ring;
  ring.init(irow, 0, topk, 0, 1, kbase, kcap, kv4, kv4_scale, mem, lane);
  ring.start(lp, lane);
  float f[MT][2];
  QueryRaw<MT> raw;
  raw.load(q, (size_t)row, H, lane);
  convert_query<MT, 1>(raw, scale, qs, lane, 0, f);
  __syncwarp();
  const uint32_t qf = smem_u32(qs + lane);
  Running<MT> st;
  st.clear();
  attend<MT>(ring, lp, qf, f, lane, st);
  if (__any_sync(0xffffffffu, ring.bad) && lane == 0) raise_status(status, HISA_ERR_INVALID_ARG);

  float mx[MT][2], inv[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int r = 0; r < 2; r++) {
      const int h = 16 * mt + g + 8 * r;
      const float sum = st.total(mt, r);
      mx[mt][r] = st.m[mt][r];
      inv[mt][r] = inverse_sum(sum);
      if (h >= H) continue;
      if (c == 0 && lse) lse[(size_t)row * H + h] = lse_of(mx[mt][r], sum);
      // the lane's 32 dimensions: 16 of column 2c, 16 of column 2c + 1
      uint4 *dst = reinterpret_cast<uint4 *>(out + ((size_t)row * H + h) * KV4_DIM + 32 * c);
#pragma unroll
      for (int u = 0; u < 4; u++) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int t = 8 * (u & 1) + 2 * i, e = 2 * r + (u >> 1);
          const __nv_bfloat162 b = __floats2bfloat162_rn(st.o[mt][t][e] * inv[mt][r],
                                                         st.o[mt][t + 1][e] * inv[mt][r]);
          w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  if (WT) {
    dead_heads<MT>(H, g, f, mx, inv);
    Ring<NST, NST - 1, false> again;
    again.init(irow, 0, topk, 0, 1, kbase, kcap, kv4, kv4_scale, mem, lane);
    weigh_again<MT>(again, qf, f, mx, inv, lane, weights + kbase, status);
  }
}

// ---------------------------------------------------------------------------
// Few rows: the four warps of a CTA, and the C CTAs of a cluster, share a row.

template <int MT>
struct SplitSmem {
  static constexpr int QBYTES = MT * 4096;
  static constexpr int NH = 16 * MT;
  // ring of every warp | query fragments | partial outputs from the cluster's CTAs | their m
  // and l | m, l of every warp and head | m, l of the CTA | merge factors of the cluster
  static constexpr size_t bytes = (size_t)A4_WARPS * a4_ring(MT) + QBYTES + NH * KV4_DIM * 4 +
                                  A4_MAX_CLUSTER * NH * 8 + (size_t)A4_WARPS * NH * 8 +
                                  (size_t)NH * 8 + (size_t)NH * A4_MAX_CLUSTER * 4;
};

template <int MT, bool WT>
__global__ void __launch_bounds__(A4_THREADS, a4_ctas(MT))
attn_kv4_split_kernel(const uint16_t *__restrict__ q, const uint8_t *__restrict__ kv4,
                      const uint8_t *__restrict__ kv4_scale, const int32_t *__restrict__ idx,
                      const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int S,
                      int H, int topk, int per_cta, float scale, uint16_t *__restrict__ out,
                      float *__restrict__ lse, unsigned long long *__restrict__ weights,
                      int *status) {
  extern __shared__ __align__(16) uint8_t a4_smem[];
  constexpr int NST = a4_stages(MT), RING = a4_ring(MT), NH = 16 * MT;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), me = (int)cl.block_rank();
  const int row = blockIdx.x >> (31 - __clz(C));  // C is a power of two
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2;
  const float NEG = -__int_as_float(0x7f800000);
  uint8_t *qs = a4_smem + A4_WARPS * RING;
  float *recv = reinterpret_cast<float *>(qs + SplitSmem<MT>::QBYTES);  // [C][heads][128]
  float2 *recv_ml = reinterpret_cast<float2 *>(recv + NH * KV4_DIM);    // [C][NH]
  float *wm = reinterpret_cast<float *>(recv_ml + A4_MAX_CLUSTER * NH);  // [warps][NH]
  float *wl = wm + A4_WARPS * NH;                                     // [warps][NH]
  float *cm = wl + A4_WARPS * NH, *cs = cm + NH;  // the CTA's maximum and sum per head
  float *xm = cs + NH;                            // factors of the cluster's CTAs [NH][C]
  if (C > 1) cluster_arrive();  // this CTA runs: the others may write to it
  const LanePlaces<true> lp(lane);
  const int e0 = me * per_cta, e1 = min(topk, e0 + per_cta);
  const int32_t *irow = idx + (size_t)row * topk;
  uint8_t *mem = a4_smem + warp * RING;
  // the row's first tokens and the query arrive while the sequence is looked up (14400 cycles
  // of a CTA against 15100)
  Ring<NST, NST - 1, true> ring;
  ring.entries(irow, e0, e1, warp, A4_WARPS, lane);
  QueryRaw<MT> raw;
  raw.load(q, (size_t)row, H, lane);
  const Region rg = region_of(cu_q, cu_k, S, row, lane);
  const int kbase = rg.base, kcap = rg.tokens;
  ring.region(kbase, kcap, kv4, kv4_scale, mem, lane);
  ring.start(lp, lane);
  float f[MT][2];
  convert_query<MT, A4_WARPS>(raw, scale, reinterpret_cast<uint4 *>(qs), lane, warp, f);
  __syncthreads();
  const uint32_t qf = smem_u32(qs + lane * 16);
  Running<MT> st;
  st.clear();
  attend<MT>(ring, lp, qf, f, lane, st);
  if (__any_sync(0xffffffffu, ring.bad) && lane == 0) raise_status(status, HISA_ERR_INVALID_ARG);
  store_share<MT>(st, mem, wm + warp * NH, wl + warp * NH, lane);
  __syncthreads();
  if (tid < NH) join_shares<A4_WARPS>(wm, wl, NH, tid, cm[tid], cs[tid]);
  __syncthreads();
  // With several CTAs every one sums its own warps first and sends the heads r, r + C, ... to
  // CTA r, which finishes them, and its maxima and sums to all.  Sending leaves one exchange
  // to wait for, where reading the others' shares took three and a last barrier before the
  // shared memory may go (16 rows of 2048 tokens and 16 heads: 15100 cycles against 16600).
  if (C > 1) {
    const int lc = 31 - __clz(C);
    const int HL = (H + C - 1) >> lc;  // heads of a CTA; C * HL <= NH
    cluster_wait();
    for (int x = tid; x < C * NH; x += A4_THREADS) {
      const int r = x / NH, h = x % NH;
      cl.map_shared_rank(recv_ml, r)[me * NH + h] = make_float2(cm[h], cs[h]);
    }
#pragma unroll
    for (int i = 0; i < NH * (KV4_DIM / 4) / A4_THREADS; i++) {
      const int x = tid + i * A4_THREADS, h = x >> 5, b = (x >> 3) & 3, u = x & 7;
      if (h < H) {
        const float4 v = sum_shares<A4_WARPS>(a4_smem, RING, wm, NH, h,
                                              h * A4_OSTRIDE + 32 * b + 4 * (u ^ (2 * b)));
        *reinterpret_cast<float4 *>(cl.map_shared_rank(recv, h & (C - 1)) +
                                    (me * HL + (h >> lc)) * KV4_DIM + 32 * b + 4 * u) = v;
      }
    }
    cl.sync();
    if (tid < H) {
      float mr[A4_MAX_CLUSTER], lr[A4_MAX_CLUSTER], mx = NEG, sum = 0.f;
#pragma unroll
      for (int r = 0; r < A4_MAX_CLUSTER; r++) {
        const float2 v = r < C ? recv_ml[r * NH + tid] : make_float2(NEG, 0.f);
        mr[r] = v.x;
        lr[r] = v.y;
        mx = fmaxf(mx, v.x);
      }
#pragma unroll
      for (int r = 0; r < A4_MAX_CLUSTER; r++) {
        mr[r] = share_factor(mr[r], lr[r], mx);
        if (r < C) sum += lr[r] != lr[r] ? lr[r] : mr[r] * lr[r];
      }
      const float inv = inverse_sum(sum);
#pragma unroll
      for (int r = 0; r < A4_MAX_CLUSTER; r++)
        if (r < C) xm[tid * A4_MAX_CLUSTER + r] = mr[r] * inv;
      if (lse && (tid & (C - 1)) == me) lse[(size_t)row * H + tid] = lse_of(mx, sum);
      wm[tid] = mx;  // the warps' factors are not needed any more
      wl[tid] = inv;
    }
    __syncthreads();
    const int nloc = me < H ? (H - me + C - 1) >> lc : 0;
    for (int x = tid; x < nloc * (KV4_DIM / 4); x += A4_THREADS) {
      const int hl = x >> 5, h = me + C * hl, d = 4 * (x & 31);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < A4_MAX_CLUSTER; r++)
        if (r < C)
          add_share(acc, xm[h * A4_MAX_CLUSTER + r],
                    *reinterpret_cast<const float4 *>(recv + (r * HL + hl) * KV4_DIM + d));
      store_out(out + ((size_t)row * H + h) * KV4_DIM + d, acc, 1.f);
    }
  } else {
    for (int x = tid; x < H * (KV4_DIM / 4); x += A4_THREADS) {
      const int h = x >> 5, b = (x >> 3) & 3, u = x & 7;
      const float4 acc = sum_shares<A4_WARPS>(a4_smem, RING, wm, NH, h,
                                              h * A4_OSTRIDE + 32 * b + 4 * (u ^ (2 * b)));
      store_out(out + ((size_t)row * H + h) * KV4_DIM + 32 * b + 4 * u, acc, inverse_sum(cs[h]));
    }
    if (tid < H && lse) lse[(size_t)row * H + tid] = lse_of(cm[tid], cs[tid]);
    if (WT) {
      __syncthreads();
      if (tid < H) {
        wm[tid] = cm[tid];
        wl[tid] = inverse_sum(cs[tid]);
      }
      __syncthreads();
    }
  }
  if (WT) {
    float mx[MT][2], inv[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int r = 0; r < 2; r++) {
        mx[mt][r] = wm[16 * mt + g + 8 * r];
        inv[mt][r] = wl[16 * mt + g + 8 * r];
      }
    dead_heads<MT>(H, g, f, mx, inv);
    __syncthreads();  // the partial outputs in the rings have been read
    Ring<NST, NST - 1, false> again;
    again.init(irow, e0, e1, warp, A4_WARPS, kbase, kcap, kv4, kv4_scale, mem, lane);
    weigh_again<MT>(again, qf, f, mx, inv, lane, weights + kbase, status);
  }
}

struct AttnArgs {
  const uint16_t *q;
  const uint8_t *kv4, *kv4_scale;
  const int32_t *idx, *cu_q, *cu_k;
  int S, total_q, H, topk;
  float scale;
  uint16_t *out;
  float *lse;
  unsigned long long *weights;
  int *status;
};

template <int MT, bool WT>
static cudaError_t launch_rows(const AttnArgs &a, cudaStream_t st) {
  static std::atomic<int> attr[64];
  constexpr size_t smem = (size_t)A4_WARPS * (a4_ring(MT) + MT * 4096);
  static_assert((smem + 1024) * a4_ctas(MT) <= 233472, "the CTAs of an SM");
  const auto fn = attn_kv4_rows_kernel<MT, WT>;
  const cudaError_t e = set_smem_once((const void *)fn, smem, attr);
  if (e != cudaSuccess) return e;
  ProfScope ps(K_ATTENTION_KV4, st);
  fn<<<(a.total_q + A4_WARPS - 1) / A4_WARPS, A4_THREADS, smem, st>>>(
      a.q, a.kv4, a.kv4_scale, a.idx, a.cu_q, a.cu_k, a.S, a.total_q, a.H, a.topk, a.scale, a.out,
      a.lse, a.weights, a.status);
  return cudaGetLastError();
}

template <int MT, bool WT>
static cudaError_t launch_split(const AttnArgs &a, int C, cudaStream_t st) {
  static std::atomic<int> attr[64];
  const int per = ((a.topk + A4_STEP - 1) / A4_STEP + C - 1) / C;
  constexpr size_t smem = SplitSmem<MT>::bytes;
  static_assert((smem + 1024) * a4_ctas(MT) <= 233472, "the CTAs of an SM");
  const auto fn = attn_kv4_split_kernel<MT, WT>;
  const cudaError_t e = set_smem_once((const void *)fn, smem, attr);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.total_q * C);
  cfg.blockDim = dim3(A4_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = C;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  ProfScope ps(K_ATTENTION_KV4, st);
  return cudaLaunchKernelEx(&cfg, fn, a.q, a.kv4, a.kv4_scale, a.idx, a.cu_q, a.cu_k, a.S, a.H,
                            a.topk, per * A4_STEP, a.scale, a.out, a.lse, a.weights, a.status);
}

// CTAs of a row (1, 2, 4 or 8: a cluster) when there are few rows.  In tenths of a step (0.87 us
// for one tile of heads, 1.23 for two): a warp's steps, slower where a second or third CTA
// shares its SM (clusters leave some SMs of the chip's groups out), and the merge.  Measured
// in us with 1, 2, 4 and 8 CTAs, 16 heads: 16 rows of 2048 tokens 17.8, 12.4, 8.7, 8.3; 64
// rows 18.1, 12.4, 11.2, 17.8; 16 rows of 512 tokens 7.4, 6.8, 5.9, 6.5; 16 of 256 5.5, 6.1,
// 5.8, 6.4; 32 heads: 64 rows of 2048 26.9, 18.1, 16.9, 22.7; 100 rows 27.1, 25.1, 30.8, 40.9.
static int cluster_of_row(int MT, int total_q, int steps, int num_sms) {
  int best = 1;
  long long least = 0;
  for (int C = 1; C <= A4_MAX_CLUSTER && total_q <= num_sms; C *= 2) {
    const int room = C <= 2 ? num_sms : C == 4 ? num_sms * 8 / 9 : num_sms * 13 / 16;
    const int share = (total_q * C + room - 1) / room;  // CTAs of an SM
    if (share > a4_ctas(MT)) break;
    const int merge = C == 1 ? 0 : C == 2 ? (MT == 1 ? 20 : 11) : (MT == 1 ? 15 : 6);
    const long long w = (steps + A4_WARPS * C - 1) / (A4_WARPS * C);
    const long long cost = w * (share == 1 ? 10 : share == 2 ? 16 : 25) + merge;
    if (C > 1 && cost >= least) continue;
    best = C;
    least = cost;
  }
  return best;
}

template <int MT, bool WT>
static cudaError_t launch_attn(const AttnArgs &a, int num_sms, cudaStream_t st) {
  const int steps = (a.topk + A4_STEP - 1) / A4_STEP;
  // Few rows: a row is split over a CTA's warps, and over the CTAs of a cluster
  const int C = cluster_of_row(MT, a.total_q, steps, num_sms);
  // With many rows a warp has one to itself.  A row's start and end cost a warp about 2.5
  // steps, four times if four warps share it; one warp alone leaves half a row's steps idle
  // in the last wave instead of half of a quarter.  Measured (us, one warp / four): 16 heads,
  // 2048 tokens 2400 rows 200 / 184, 4800 rows 350 / 350; 512 tokens 1200 rows 38 / 36, 2400
  // rows 58 / 63; 128 tokens 600 rows 12.1 / 13.0; 32 heads, 2048 tokens 2400 rows 329 / 303,
  // 4800 rows 585 / 612; two warps were never the best of the three by 5%.
  const long long slots = (long long)num_sms * a4_ctas(MT) * A4_WARPS;
  const int spared = steps - (steps + A4_WARPS - 1) / A4_WARPS;
  if (C > 1 || 15ll * a.total_q <= slots * spared) return launch_split<MT, WT>(a, C, st);
  return launch_rows<MT, WT>(a, st);
}

cudaError_t launch_attention_kv4(const uint16_t *q, const uint8_t *kv4, const uint8_t *kv4_scale,
                                 const int32_t *idx, const int32_t *cu_q, const int32_t *cu_k,
                                 int S, int total_q, int H, int topk, float scale, uint16_t *out,
                                 float *lse, int64_t *weights, int num_sms, int *status,
                                 cudaStream_t st) {
  const AttnArgs a = {q, kv4, kv4_scale, idx, cu_q, cu_k, S, total_q, H, topk, scale, out, lse,
                      reinterpret_cast<unsigned long long *>(weights), status};
  if (H <= 16)
    return weights ? launch_attn<1, true>(a, num_sms, st) : launch_attn<1, false>(a, num_sms, st);
  return weights ? launch_attn<2, true>(a, num_sms, st) : launch_attn<2, false>(a, num_sms, st);
}

// ---------------------------------------------------------------------------
// Token weights of the bf16 cache: the scores again, against the row's log-sum-exp.  A warp
// takes 32 tokens at a time; sum_h 2^(x - lse) of every token ends in one lane, which adds
// it to the token's accumulator as a whole multiple of 2^-32: integer sums do not depend on
// the order in which the rows arrive.

constexpr int TW_WARPS = 4;

// The heads' log-sum-exps of lane (g, c), negated and in powers of two, as a pair of fp32:
// the rounding of a single one would move every weight of the row.  -inf (no weights) for
// a head with no index and past the last.
struct NegLse {
  float hi, lo;
};
__device__ __forceinline__ NegLse neg_lse(const float *lse, size_t row, int H, int h) {
  const float INF = __int_as_float(0x7f800000);
  const float v = h < H ? __ldg(lse + row * H + h) : -INF;
  NegLse n;
  n.hi = v == -INF ? -INF : -v * LOG2E;
  n.lo = v == -INF ? 0.f : fmaf(-v, LOG2E_LO, fmaf(-v, LOG2E, -n.hi));
  return n;
}

// v[i] = sum over the lane's heads of 2^(x f - lse), x the score fragments of 32 tokens, f2
// what f and the fragments lost
template <int MT>
__device__ __forceinline__ void weigh(const float (&x)[MT][4][4], float f, float f2,
                                      const NegLse (&nl)[MT][2], float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int r = 0; r < 2; r++) {
        const float2 t = make_float2(x[mt][j][2 * r], x[mt][j][2 * r + 1]);
        const float2 e = add2(fma2(t, f, nl[mt][r].hi), fma2(t, f2, nl[mt][r].lo));
        sum = add2(sum, make_float2(ex2(e.x), ex2(e.y)));
      }
    v[2 * j] = sum.x;
    v[2 * j + 1] = sum.y;
  }
}

// The rows (256 bytes) come through a ring as above: lane (g, c) takes the 16-byte chunks
// 4i + c of token g of every 8, chunk i being the fragments 2i and 2i + 1, of the query
// alike; an odd token's chunks change places in pairs of four, so that two tokens' fall
// into different banks.  The matrix unit cuts sums off instead of rounding them, which in a
// chain of eight would lower every score by a few 2^-24 of itself and every weight by that
// times the score; so pairs are summed there and the four sums here.  Each of a pair's two
// sums still loses half a unit in its last place on average, 2^-25 to 2^-24 of it; f2 gives
// 2^-24 of the score back.  Weights of 4096 rows of 32 heads, against 64 bits: 6e-7 of them
// (root mean square) without it, most of that of one sign, 1.2e-7 with it; sums of single
// matrix instructions instead of pairs 4e-7, and 2% slower.  Where the sums are exact (whole
// numbers, few bits) nothing was cut off, and weights come out 2^-24 of their score, relative,
// too large: 9e-7 at scores of up to 29.  That is what a single rounding of the score to fp32
// may cost, and it is always in that direction.
//
// A warp has a row, or a part of one, to itself: its start hides behind the other warps.
constexpr int TWB_ROW = KV4_DIM * 2, TWB_STAGE = A4_STEP * TWB_ROW;
constexpr int tw_ctas(int MT) { return MT == 1 ? 3 : 2; }  // 168 and 255 registers
constexpr int tw_smem() { return TW_WARPS * 2 * TWB_STAGE; }

template <int MT>
__global__ void __launch_bounds__(TW_WARPS * 32, tw_ctas(MT))
token_weights_kernel(const uint16_t *__restrict__ q, const uint16_t *__restrict__ k,
                     const int32_t *__restrict__ idx, const float *__restrict__ lse,
                     const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int S,
                     int total_q, int parts, int H, int topk, float scale,
                     unsigned long long *__restrict__ weights, int *status) {
  extern __shared__ __align__(16) uint8_t a4_smem[];
  const int lane = threadIdx.x & 31, warp = warp_index();
  const long long item = (long long)blockIdx.x * TW_WARPS + warp;
  const int row = (int)(item / parts);
  if (row >= total_q) return;  // the whole warp; the others do not wait for it
  const int g = lane >> 2, c = lane & 3;
  const Region rg = region_of(cu_q, cu_k, S, row, lane);
  const int kbase = rg.base, kcap = rg.tokens;
  const int32_t *irow = idx + (size_t)row * topk;
  const int steps = (topk + A4_STEP - 1) / A4_STEP;
  const int first = (int)(item - (long long)row * parts), stride = parts;
  const uint32_t ring = smem_u32(a4_smem) + warp * 2 * TWB_STAGE;
  // this lane's place in token g: chunks 0 and 2 from `even`, 1 and 3 from `odd`
  const uint32_t even = g * TWB_ROW + ((g & 1) << 6) + (c << 4), odd = even ^ 64u;
  const uint8_t *keys = reinterpret_cast<const uint8_t *>(k) + (size_t)kbase * TWB_ROW + c * 16;
  auto token = [&](int n) {
    const int e = n * A4_STEP + lane;
    return e < topk ? __ldg(irow + e) : -1;
  };
  // j: this lane's token, -1 where it is none; four lanes copy 64 bytes of a token together
  auto copy = [&](int &j, uint32_t stage) {
    if (j >= kcap) {
      raise_status(status, HISA_ERR_INVALID_ARG);
      j = -1;
    }
    const uint32_t valid = __ballot_sync(0xffffffffu, j >= 0);
    if (valid) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int t = __shfl_sync(0xffffffffu, j, 8 * i + g);
        const uint8_t *src = keys + (size_t)(uint32_t)max(t, 0) * TWB_ROW;
        const uint32_t dst = stage + i * 8 * TWB_ROW;
        cp_async_16_or_zero(dst + even, src, t >= 0);
        cp_async_16_or_zero(dst + odd, src + 64, t >= 0);
        cp_async_16_or_zero(dst + even + 128, src + 128, t >= 0);
        cp_async_16_or_zero(dst + odd + 128, src + 192, t >= 0);
      }
    }
    cp_async_commit();
  };
  int now = token(first), next = token(first + stride);
  copy(now, ring);
  float f, f2;
  NegLse nl[MT][2];
  uint4 qw[MT][2][4];
  f = scale * LOG2E;
  f2 = fmaf(scale, LOG2E, -f) + scale * LOG2E_LO + f * 0x1p-24f;
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int r = 0; r < 2; r++) {
      const int h = 16 * mt + g + 8 * r;
#pragma unroll
      for (int i = 0; i < 4; i++)
        qw[mt][r][i] = h < H ? __ldg(reinterpret_cast<const uint4 *>(
                                         q + ((size_t)row * H + h) * KV4_DIM) + 4 * i + c)
                             : make_uint4(0u, 0u, 0u, 0u);
      nl[mt][r] = neg_lse(lse, (size_t)row, H, h);
    }
  __syncwarp();
  uint32_t stage = ring;
  for (int n = first; n < steps; n += stride) {
    __syncwarp();  // every lane has read the stage that is filled now
    const uint32_t other = ring + (stage == ring ? TWB_STAGE : 0);
    int then = next;
    copy(then, other);
    next = token(n + 2 * stride);
    cp_async_wait_group<1>();
    __syncwarp();  // the step has landed for every lane
    if (__any_sync(0xffffffffu, now >= 0)) {
      float x[MT][4][4], v[8];
#pragma unroll
      for (int i = 0; i < 4; i++) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint4 kw = lds<uint4>(stage + j * 8 * TWB_ROW + ((i & 1) ? odd : even) +
                                      (i >> 1) * 128);
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            float d[4];
            const uint4 a = qw[mt][0][i], b = qw[mt][1][i];
            mma_bf16_first(d, a.x, b.x, a.y, b.y, kw.x, kw.y);
            mma_bf16(d, a.z, b.z, a.w, b.w, kw.z, kw.w);
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
              float2 y = make_float2(d[u], d[u + 1]);
              if (i > 0) y = add2(make_float2(x[mt][j][u], x[mt][j][u + 1]), y);
              x[mt][j][u] = y.x;
              x[mt][j][u + 1] = y.y;
            }
          }
        }
      }
      weigh<MT>(x, f, f2, nl, v);
      add_weights(v, now, weights + kbase, lane, status);
    }
    now = then;
    stage = other;
  }
  cp_async_wait_all();
}

cudaError_t launch_token_weights(const uint16_t *q, const uint16_t *k, const int32_t *idx,
                                 const float *lse, const int32_t *cu_q, const int32_t *cu_k, int S,
                                 int total_q, int H, int topk, float scale, int64_t *weights,
                                 int num_sms, int *status, cudaStream_t st) {
  static std::atomic<int> attr[2][64];
  const auto fn = H <= 16 ? token_weights_kernel<1> : token_weights_kernel<2>;
  const cudaError_t e = set_smem_once((const void *)fn, tw_smem(), attr[H > 16]);
  if (e != cudaSuccess) return e;
  // parts of a row: enough for four waves of warps, each with a step at least (8 x 64 rows
  // of 2048 tokens: 44 us with one wave, 39 with four, 45 with eight)
  const int steps = (topk + A4_STEP - 1) / A4_STEP;
  const int slots = num_sms * tw_ctas(H <= 16 ? 1 : 2) * TW_WARPS;
  const int want = (4 * slots + total_q - 1) / total_q, parts = want < steps ? want : steps;
  const long long items = (long long)total_q * parts;
  ProfScope ps(K_TOKEN_WEIGHTS, st);
  fn<<<(unsigned)((items + TW_WARPS - 1) / TW_WARPS), TW_WARPS * 32, tw_smem(), st>>>(
      q, k, idx, lse, cu_q, cu_k, S, total_q, parts, H, topk, scale,
      reinterpret_cast<unsigned long long *>(weights), status);
  return cudaGetLastError();
}

}  // namespace hisa
