// Sparse attention over the 4-bit cache, and the attention weight of every token
// (hisa_sparse_attention_kv4, hisa_token_weights).
//
//   s_j = scale * q[i][h] . k_j,   out[i][h] = sum_j softmax(s)_j v_j,
//   weight[j] += sum_h softmax(s)_j
//
// over the entries j >= 0 of the index row.  One warp takes 32 selected tokens at a time
// and does everything to them: it copies their rows (144 bytes each) into a ring of its
// own, turns the key nibbles into fp16 fragments, multiplies, keeps the running maximum
// and sum of its share, turns the value nibbles into fragments and multiplies again.  No
// warp waits for another until its share is done; then the warps of a CTA, and the CTAs
// of a row's cluster, are merged by their maxima and sums.
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
// sums are fp32; the softmax weights enter the value product as fp16 (relative error at
// most 2^-12, an eighth of the bf16 output's own rounding), taken against a reference that
// the maximum never exceeds by more than 2^8.
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
constexpr float A4_TAU = 8.f;    // tolerated growth of a head's maximum, in powers of two
constexpr int A4_OSTRIDE = KV4_DIM + 4;                       // padded row of partial outputs
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__host__ __device__ constexpr int a4_stages(int MT) { return MT == 1 ? 3 : 4; }
// a warp's ring, which later holds its partial output
__host__ __device__ constexpr int a4_ring(int MT) { return a4_stages(MT) * A4_STAGE; }
static_assert(16 * A4_OSTRIDE * 4 <= a4_ring(1) && 32 * A4_OSTRIDE * 4 <= a4_ring(2),
              "a warp's partial output fits its ring");

// 16-byte chunk of token t's 128-byte row: the key chunks of two neighbouring tokens, and
// the value chunks of every second token, fall into different banks
__device__ __forceinline__ int a4_chunk(int t, int chunk) {
  return chunk ^ (((t >> 1) & 3) << 1) ^ ((t & 1) << 2);
}

// 16 bytes global -> shared; zeros when !ok
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
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

// Query fragments of heads 16 mt + g and + g + 8: fragment ks = 2 w + half holds the
// dimension pairs (d, d + 4) of word w (32c + 8w ..), d = 0 and 1 (half 0) or 2 and 3.
// `down` of the two heads comes back in dn.  Heads >= H are zeros.
__device__ __forceinline__ void load_q_frags(const uint16_t *__restrict__ q, size_t row, int H, int mt,
                                             int lane, uint32_t (&f)[8][4], float (&dn)[2]) {
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int r = 0; r < 2; r++) {
    const int h = 16 * mt + g + 8 * r;
    uint4 w[4];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h < H)
        w[i] = __ldg(reinterpret_cast<const uint4 *>(q + (row * H + h) * KV4_DIM + 32 * c) + i);
      mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu),
                                 __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu)));
    }
    mx = max(mx & 0xFFFFu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    float up;
    q_shift(mx, up, dn[r]);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      // dimensions 0..7 of the word: pairs (0,4) (1,5) (2,6) (3,7)
      const float x[8] = {bf_lo(w[i].x), bf_hi(w[i].x), bf_lo(w[i].y), bf_hi(w[i].y),
                          bf_lo(w[i].z), bf_hi(w[i].z), bf_lo(w[i].w), bf_hi(w[i].w)};
#pragma unroll
      for (int p = 0; p < 4; p++)
        f[2 * i + (p >> 1)][2 * (p & 1) + r] =
            as_u32(__floats2half2_rn(x[p] * up, x[p + 4] * up));
    }
  }
}

// Query fragments of one 16-head tile: in registers for one tile, in shared memory (a
// lane's 16 bytes per fragment) for two, whose outputs leave no room for them.
template <int MT>
struct QFrags;
template <>
struct QFrags<1> {
  uint32_t f[8][4];
  __device__ __forceinline__ uint4 get(int, int ks) const {
    return make_uint4(f[ks][0], f[ks][1], f[ks][2], f[ks][3]);
  }
};
template <>
struct QFrags<2> {
  const uint4 *s;  // [mt][ks][lane]
  int lane;
  __device__ __forceinline__ uint4 get(int mt, int ks) const {
    return s[(mt * 8 + ks) * 32 + lane];
  }
};

// Raw scores of the 32 tokens in a ring stage: s[mt][j][.] is the score fragment of the
// 8 tokens 8j .. 8j + 7.
template <int MT>
__device__ __forceinline__ void kv4_scores(const uint8_t *stage, const QFrags<MT> &qf, int lane,
                                           float (&s)[MT][4][4]) {
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int t = 8 * j + g;
    const uint4 kw =
        *reinterpret_cast<const uint4 *>(stage + t * KV4_ROW + (a4_chunk(t, c) << 4));
    const uint32_t sb =
        *reinterpret_cast<const uint16_t *>(stage + A4_CODES + t * KV4_NS + 2 * c);
    const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int e = 0; e < 4; e++) s[mt][j][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      // both halves of the scale pair: byte 0 (words 0, 1) or byte 1 (words 2, 3)
      const __half2 sc = as_half2(__byte_perm(sb, 0u, i < 2 ? 0x4040 : 0x4141) << 7);
      const __half2 c72 = kv4_c72(sc);
      const uint32_t b0 = kv4_pair(w[i] << 4, sc, c72), b1 = kv4_pair(w[i], sc, c72);
      const uint32_t b2 = kv4_pair(w[i] >> 4, sc, c72), b3 = kv4_pair(w[i] >> 8, sc, c72);
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
        const uint4 qa = qf.get(mt, 2 * i), qb = qf.get(mt, 2 * i + 1);
        mma_f16(s[mt][j], qa.x, qa.y, qa.z, qa.w, b0, b1);
        mma_f16(s[mt][j], qb.x, qb.y, qb.z, qb.w, b2, b3);
      }
    }
  }
}

// A warp's walk over its steps: the token ids are read one step ahead of the copies, the
// copies run NST - 1 steps ahead of the products.
template <int NST>
struct Ring {
  const int32_t *irow;
  int e0, e1, nsteps, stride, first;  // entries [e0, e1); steps first, first + stride, ...
  int kcap;
  size_t kbase;
  const uint8_t *kv4, *kv4_scale;
  uint8_t *ring;
  int lane;
  int next_tok;             // this lane's token of the next step to copy (-1 = none)
  uint32_t mask[NST];       // valid tokens of the steps in flight, oldest first
  bool bad;

  __device__ __forceinline__ int token(int n) const {
    const int e = e0 + (first + n * stride) * A4_STEP + lane;
    return (n < nsteps && e < e1) ? __ldg(irow + e) : -1;
  }
  // start the copy of step n into stage n % NST
  __device__ __forceinline__ uint32_t copy(int n) {
    int j = next_tok;
    next_tok = token(n + 1);
    if (j >= kcap) {
      bad = true;
      j = -1;
    }
    const uint32_t valid = __ballot_sync(0xffffffffu, j >= 0);
    if (n < nsteps && valid) {
      const uint32_t dst = smem_u32(ring + (n % NST) * A4_STAGE);
      const int chunk = lane & 7;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int t = 4 * i + (lane >> 3);
        const int jt = __shfl_sync(0xffffffffu, j, t);
        cp_async_16_or_zero(dst + t * KV4_ROW + (a4_chunk(t, chunk) << 4),
                            kv4 + (kbase + (size_t)max(jt, 0)) * KV4_ROW + chunk * 16, jt >= 0);
      }
      cp_async_16_or_zero(dst + A4_CODES + lane * KV4_NS,
                          kv4_scale + (kbase + (size_t)max(j, 0)) * KV4_NS, j >= 0);
    }
    cp_async_commit();
    return valid;
  }
  __device__ __forceinline__ void start() {
    bad = false;
    next_tok = token(0);
#pragma unroll
    for (int n = 0; n < NST - 1; n++) mask[n] = copy(n);
  }
  // wait for step n; its stage and the mask of its valid tokens
  __device__ __forceinline__ const uint8_t *arrive(int n, uint32_t &valid) {
    cp_async_wait_group<NST - 2>();
    __syncwarp();  // the step has landed for every lane, and stage (n - 1) % NST is read
    valid = mask[0];
#pragma unroll
    for (int i = 0; i + 2 < NST; i++) mask[i] = mask[i + 1];
    mask[NST - 2] = copy(n + NST - 1);
    return ring + (n % NST) * A4_STAGE;
  }
};

template <int MT>
struct A4Smem {
  static constexpr int QBYTES = MT == 1 ? 0 : MT * 8 * 32 * 16;
  // ring of every warp | query fragments | m, l of every warp and head | merge weights
  __host__ __device__ static constexpr size_t bytes(int warps) {
    return (size_t)warps * a4_ring(MT) + QBYTES + (size_t)warps * 16 * MT * 8 +
           (size_t)16 * MT * 8 + (size_t)16 * MT * A4_MAX_CLUSTER * 8;
  }
};

template <int MT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, MT == 1 ? 12 / WARPS : 8 / WARPS)
attn_kv4_kernel(const uint16_t *__restrict__ q, const uint8_t *__restrict__ kv4,
                const uint8_t *__restrict__ kv4_scale, const int32_t *__restrict__ idx,
                const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int S, int H,
                int topk, int per_cta, float scale, uint16_t *__restrict__ out,
                float *__restrict__ lse, int *status) {
  extern __shared__ __align__(16) uint8_t a4_smem[];
  constexpr int NST = a4_stages(MT), RING = a4_ring(MT), NH = 16 * MT;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), me = (int)cl.block_rank();
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const float NEG = -__int_as_float(0x7f800000);
  uint8_t *qs = a4_smem + WARPS * RING;
  float *wm = reinterpret_cast<float *>(qs + A4Smem<MT>::QBYTES);  // [WARPS][NH]
  float *wl = wm + WARPS * NH;                                     // [WARPS][NH]
  float *cm = wl + WARPS * NH, *cs = cm + NH;  // the CTA's maximum and sum per head
  float *xm = cs + NH, *xl = xm + NH * A4_MAX_CLUSTER;  // the cluster's, per own head and CTA

  const int s = find_seq(cu_q, S, row);
  const int kbase = __ldg(cu_k + s);
  Ring<NST> ring;
  ring.e0 = me * per_cta;
  ring.e1 = min(topk, ring.e0 + per_cta);
  const int steps = ring.e1 > ring.e0 ? (ring.e1 - ring.e0 + A4_STEP - 1) / A4_STEP : 0;
  ring.irow = idx + (size_t)row * topk;
  ring.first = warp;
  ring.stride = WARPS;
  ring.nsteps = steps > warp ? (steps - warp + WARPS - 1) / WARPS : 0;
  ring.kcap = __ldg(cu_k + s + 1) - kbase;
  ring.kbase = (size_t)kbase;
  ring.kv4 = kv4;
  ring.kv4_scale = kv4_scale;
  ring.ring = a4_smem + warp * RING;
  ring.lane = lane;
  ring.start();

  QFrags<MT> qf;
  float f[MT][2];  // score -> power-of-two exponent, of heads g and g + 8
  if constexpr (MT == 1) {
    load_q_frags(q, (size_t)row, H, 0, lane, qf.f, f[0]);
  } else {
    uint4 *sq = reinterpret_cast<uint4 *>(qs);
    qf.s = sq;
    qf.lane = lane;
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      uint32_t t[8][4];
      load_q_frags(q, (size_t)row, H, mt, lane, t, f[mt]);
      // every warp computes every fragment (it needs the shifts) and stores its part
#pragma unroll
      for (int ks = 0; ks < 8; ks++)
        if ((mt * 8 + ks) % WARPS == warp)
          sq[(mt * 8 + ks) * 32 + lane] = make_uint4(t[ks][0], t[ks][1], t[ks][2], t[ks][3]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int r = 0; r < 2; r++) f[mt][r] *= scale * LOG2E;

  float o[MT][16][4];
  float m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; mt++) {
#pragma unroll
    for (int t = 0; t < 16; t++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[mt][t][e] = 0.f;
#pragma unroll
    for (int r = 0; r < 2; r++) {
      m[mt][r] = NEG;
      l[mt][r] = 0.f;
    }
  }

  for (int n = 0; n < ring.nsteps; n++) {
    uint32_t valid;
    const uint8_t *stage = ring.arrive(n, valid);
    if (!valid) continue;
    float x[MT][4][4];
    kv4_scores<MT>(stage, qf, lane, x);
    bool over = false;
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const bool live = (valid >> (8 * j + 2 * c + (e & 1))) & 1u;
          x[mt][j][e] = live ? x[mt][j][e] * f[mt][e >> 1] : NEG;
          over |= x[mt][j][e] > m[mt][e >> 1] + A4_TAU;
        }
    // the reference maxima rise (and sums and outputs are rescaled) only where a score
    // exceeds one by 2^TAU; a first score always does
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
          float mx = m[mt][r];
#pragma unroll
          for (int j = 0; j < 4; j++)
            mx = fmaxf(mx, fmaxf(x[mt][j][2 * r], x[mt][j][2 * r + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float a = mx == NEG ? 1.f : ex2(m[mt][r] - mx);
          m[mt][r] = mx;
          l[mt][r] *= a;
#pragma unroll
          for (int t = 0; t < 16; t++) {
            o[mt][t][2 * r] *= a;
            o[mt][t][2 * r + 1] *= a;
          }
        }
    }
    uint32_t p[MT][4][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int r = 0; r < 2; r++) {
        const float mu = m[mt][r] == NEG ? 0.f : m[mt][r];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float p0 = ex2(x[mt][j][2 * r] - mu), p1 = ex2(x[mt][j][2 * r + 1] - mu);
          l[mt][r] += p0 + p1;
          p[mt][j][r] = as_u32(__floats2half2_rn(p0, p1));
        }
      }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      uint2 v[4];       // nibbles of tokens 2c, 2c + 1, 2c + 8, 2c + 9 of this half
      uint32_t sb[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int t = 16 * i + 8 * (u >> 1) + 2 * c + (u & 1);
        v[u] = *reinterpret_cast<const uint2 *>(stage + t * KV4_ROW +
                                                (a4_chunk(t, 4 + (g >> 1)) << 4) + (g & 1) * 8);
        sb[u] = stage[A4_CODES + t * KV4_NS + 8 + g];
      }
      const __half2 s0 = as_half2((sb[0] | (sb[1] << 16)) << 7);
      const __half2 s1 = as_half2((sb[2] | (sb[3] << 16)) << 7);
      const __half2 k0 = kv4_c72(s0), k1 = kv4_c72(s1);
#pragma unroll
      for (int w = 0; w < 4; w++) {  // dimensions 4w .. 4w + 3 of the group
        const uint32_t sel = (w & 1) ? 0x7632 : 0x5410;
        const uint32_t r0 = __byte_perm(w < 2 ? v[0].x : v[0].y, w < 2 ? v[1].x : v[1].y, sel);
        const uint32_t r1 = __byte_perm(w < 2 ? v[2].x : v[2].y, w < 2 ? v[3].x : v[3].y, sel);
#pragma unroll
        for (int d = 0; d < 4; d++) {
          const uint32_t b0 = kv4_pair(d == 0 ? r0 << 4 : r0 >> (4 * d - 4), s0, k0);
          const uint32_t b1 = kv4_pair(d == 0 ? r1 << 4 : r1 >> (4 * d - 4), s1, k1);
#pragma unroll
          for (int mt = 0; mt < MT; mt++)
            mma_f16(o[mt][4 * w + d], p[mt][2 * i][0], p[mt][2 * i][1], p[mt][2 * i + 1][0],
                    p[mt][2 * i + 1][1], b0, b1);
        }
      }
    }
  }
  cp_async_wait_all();
  __syncwarp();  // the ring is free: it takes the warp's partial output
  if (__any_sync(0xffffffffu, ring.bad) && lane == 0) raise_status(status, HISA_ERR_INVALID_ARG);

  // Partial outputs, [head][dimension] with the 4-value pieces of a 32-dimension block
  // turned by the block so that the lanes' stores spread over the banks.
  float *po = reinterpret_cast<float *>(ring.ring);
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int r = 0; r < 2; r++) {
      float sum = l[mt][r];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int h = 16 * mt + g + 8 * r;
      if (c == 0) {
        wm[warp * NH + h] = m[mt][r];
        wl[warp * NH + h] = sum;
      }
#pragma unroll
      for (int u = 0; u < 8; u++) {
        // piece u of dimensions 32c ..: tiles 4 (u & 3) .., column 2c + (u >> 2)
        const int e = 2 * r + (u >> 2), t = 4 * (u & 3);
        *reinterpret_cast<float4 *>(po + h * A4_OSTRIDE + 32 * c + 4 * (u ^ (2 * c))) =
            make_float4(o[mt][t][e], o[mt][t + 1][e], o[mt][t + 2][e], o[mt][t + 3][e]);
      }
    }
  __syncthreads();
  // factors of the CTA's warps: 2^(m_w - m); a share with no score has the factor 0
  if (tid < NH) {
    float mx = NEG, sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; w++) mx = fmaxf(mx, wm[w * NH + tid]);
#pragma unroll
    for (int w = 0; w < WARPS; w++) {
      const float mw = wm[w * NH + tid];
      const float a = mw == NEG ? 0.f : ex2(mw - mx);
      // a share that holds a NaN keeps it whatever its maximum says
      const float lw = wl[w * NH + tid];
      wm[w * NH + tid] = lw != lw ? lw : a;
      sum += lw != lw ? lw : a * lw;
    }
    cm[tid] = mx;
    cs[tid] = sum;
  }
  __syncthreads();
  if (C == 1) {
    for (int x = tid; x < H * (KV4_DIM / 4); x += WARPS * 32) {
      const int h = x >> 5, b = (x >> 3) & 3, u = x & 7;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; w++) {
        const float a = wm[w * NH + h];
        const float4 v = *reinterpret_cast<const float4 *>(
            reinterpret_cast<const float *>(a4_smem + w * RING) + h * A4_OSTRIDE + 32 * b +
            4 * (u ^ (2 * b)));
        acc.x = fmaf(a, v.x, acc.x);
        acc.y = fmaf(a, v.y, acc.y);
        acc.z = fmaf(a, v.z, acc.z);
        acc.w = fmaf(a, v.w, acc.w);
      }
      const float L = cs[h], inv = L == 0.f ? 0.f : 1.f / L;
      const __nv_bfloat162 a2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2 *>(out + ((size_t)row * H + h) * KV4_DIM + 32 * b + 4 * u) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&a2),
                     *reinterpret_cast<const uint32_t *>(&b2));
    }
    if (tid < H && lse)
      lse[(size_t)row * H + tid] = cs[tid] == 0.f ? NEG : (cm[tid] + log2f(cs[tid])) * LN2;
    return;
  }
  // The cluster: every CTA first sums its own warps (into the first warp's share, each
  // value by the thread that read it), then finishes heads me, me + C, ...
  float *own = reinterpret_cast<float *>(a4_smem);
  for (int x = tid; x < H * (KV4_DIM / 4); x += WARPS * 32) {
    const int h = x >> 5, at = h * A4_OSTRIDE + 4 * (x & 31);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; w++) {
      const float a = wm[w * NH + h];
      const float4 v = *reinterpret_cast<const float4 *>(
          reinterpret_cast<const float *>(a4_smem + w * RING) + at);
      acc.x = fmaf(a, v.x, acc.x);
      acc.y = fmaf(a, v.y, acc.y);
      acc.z = fmaf(a, v.z, acc.z);
      acc.w = fmaf(a, v.w, acc.w);
    }
    *reinterpret_cast<float4 *>(own + at) = acc;
  }
  cl.sync();
  const int nloc = me < H ? (H - me + C - 1) / C : 0;
  for (int x = tid; x < nloc * C; x += WARPS * 32) {
    const int i = x / C, r = x - i * C, h = me + C * i;
    xm[i * A4_MAX_CLUSTER + r] = cl.map_shared_rank(cm, r)[h];
    xl[i * A4_MAX_CLUSTER + r] = cl.map_shared_rank(cs, r)[h];
  }
  __syncthreads();
  if (tid < nloc) {
    float mx = NEG, sum = 0.f;
    for (int r = 0; r < C; r++) mx = fmaxf(mx, xm[tid * A4_MAX_CLUSTER + r]);
    for (int r = 0; r < C; r++) {
      const float mr = xm[tid * A4_MAX_CLUSTER + r], lr = xl[tid * A4_MAX_CLUSTER + r];
      const float a = lr != lr ? lr : mr == NEG ? 0.f : ex2(mr - mx);
      xm[tid * A4_MAX_CLUSTER + r] = a;
      sum += lr != lr ? lr : a * lr;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int r = 0; r < C; r++) xm[tid * A4_MAX_CLUSTER + r] *= inv;
    if (lse)
      lse[(size_t)row * H + me + C * tid] = sum == 0.f ? NEG : (mx + log2f(sum)) * LN2;
  }
  __syncthreads();
  for (int x = tid; x < nloc * (KV4_DIM / 4); x += WARPS * 32) {
    const int i = x >> 5, h = me + C * i, b = (x >> 3) & 3, u = x & 7;
    const int at = h * A4_OSTRIDE + 32 * b + 4 * (u ^ (2 * b));
    float4 part[A4_MAX_CLUSTER];
#pragma unroll
    for (int r = 0; r < A4_MAX_CLUSTER; r++)
      if (r < C) part[r] = *reinterpret_cast<const float4 *>(cl.map_shared_rank(own, r) + at);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < A4_MAX_CLUSTER; r++)
      if (r < C) {
        const float a = xm[i * A4_MAX_CLUSTER + r];
        acc.x = fmaf(a, part[r].x, acc.x);
        acc.y = fmaf(a, part[r].y, acc.y);
        acc.z = fmaf(a, part[r].z, acc.z);
        acc.w = fmaf(a, part[r].w, acc.w);
      }
    const __nv_bfloat162 a2 = __floats2bfloat162_rn(acc.x, acc.y);
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc.z, acc.w);
    *reinterpret_cast<uint2 *>(out + ((size_t)row * H + h) * KV4_DIM + 32 * b + 4 * u) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a2),
                   *reinterpret_cast<const uint32_t *>(&b2));
  }
  cl.sync();  // no CTA leaves while another reads its shared memory
}

template <int MT, int WARPS>
static cudaError_t launch_attn_kv4_as(const uint16_t *q, const uint8_t *kv4,
                                      const uint8_t *kv4_scale, const int32_t *idx,
                                      const int32_t *cu_q, const int32_t *cu_k, int S, int total_q,
                                      int H, int topk, float scale, int C, uint16_t *out,
                                      float *lse, int *status, cudaStream_t st) {
  static std::atomic<int> attr[64];
  constexpr size_t smem = A4Smem<MT>::bytes(WARPS);
  static_assert(smem <= 232448, "a CTA's shared memory");
  const void *fn = (const void *)attn_kv4_kernel<MT, WARPS>;
  cudaError_t e = set_smem_once(fn, smem, attr);
  if (e != cudaSuccess) return e;
  const int steps = (topk + A4_STEP - 1) / A4_STEP;
  const int per = (steps + C - 1) / C * A4_STEP;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)total_q * C);
  cfg.blockDim = dim3(WARPS * 32);
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
  return cudaLaunchKernelEx(&cfg, attn_kv4_kernel<MT, WARPS>, q, kv4, kv4_scale, idx, cu_q, cu_k,
                            S, H, topk, per, scale, out, lse, status);
}

cudaError_t launch_attention_kv4(const uint16_t *q, const uint8_t *kv4, const uint8_t *kv4_scale,
                                 const int32_t *idx, const int32_t *cu_q, const int32_t *cu_k,
                                 int S, int total_q, int H, int topk, float scale, uint16_t *out,
                                 float *lse, int num_sms, int *status, cudaStream_t st) {
  // A row is split over the CTAs of a cluster while the rows alone leave SMs idle and
  // every CTA still has a step for each of its warps.
  int C = 1;
  while (C < A4_MAX_CLUSTER && total_q * C * 2 <= num_sms && topk >= C * 2 * 4 * A4_STEP) C *= 2;
  if (H <= 16)
    return launch_attn_kv4_as<1, 4>(q, kv4, kv4_scale, idx, cu_q, cu_k, S, total_q, H, topk, scale,
                                    C, out, lse, status, st);
  return launch_attn_kv4_as<2, 4>(q, kv4, kv4_scale, idx, cu_q, cu_k, S, total_q, H, topk, scale,
                                  C, out, lse, status, st);
}

// ---------------------------------------------------------------------------
// Token weights: the scores again, against the row's log-sum-exp.  A warp takes 32 tokens
// at a time; sum_h 2^(x - lse) of every token ends in one lane, which adds it to the
// token's accumulator as a whole multiple of 2^-32: integer sums do not depend on the
// order in which the rows arrive.

constexpr int TW_WARPS = 4;

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

// Adds the weights of a step's 32 tokens: x = scores in powers of two, fl = the heads'
// log-sum-exps in powers of two (+inf: the head adds nothing).
template <int MT>
__device__ __forceinline__ void add_weights(const float (&x)[MT][4][4], const float (&fl)[MT][2],
                                            int tok, size_t kbase, int lane,
                                            unsigned long long *weights, int *status) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[i] = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int r = 0; r < 2; r++) v[i] += ex2(x[mt][i >> 1][2 * r + (i & 1)] - fl[mt][r]);
  }
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
  if (fx) atomicAdd(weights + kbase + (size_t)j, fx);
}

template <int MT>
__global__ void __launch_bounds__(TW_WARPS * 32)
token_weights_kv4_kernel(const uint16_t *__restrict__ q, const uint8_t *__restrict__ kv4,
                         const uint8_t *__restrict__ kv4_scale, const int32_t *__restrict__ idx,
                         const float *__restrict__ lse, const int32_t *__restrict__ cu_q,
                         const int32_t *__restrict__ cu_k, int S, int H, int topk, float scale,
                         unsigned long long *__restrict__ weights, int *status) {
  extern __shared__ __align__(16) uint8_t a4_smem[];
  constexpr int NST = 3;
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = find_seq(cu_q, S, row);
  const int kbase = __ldg(cu_k + s);
  Ring<NST> ring;
  ring.e0 = 0;
  ring.e1 = topk;
  const int steps = (topk + A4_STEP - 1) / A4_STEP;
  ring.irow = idx + (size_t)row * topk;
  ring.first = blockIdx.y * TW_WARPS + warp;
  ring.stride = gridDim.y * TW_WARPS;
  ring.nsteps = steps > ring.first ? (steps - ring.first + ring.stride - 1) / ring.stride : 0;
  ring.kcap = __ldg(cu_k + s + 1) - kbase;
  ring.kbase = (size_t)kbase;
  ring.kv4 = kv4;
  ring.kv4_scale = kv4_scale;
  ring.ring = a4_smem + warp * NST * A4_STAGE;
  ring.lane = lane;
  ring.start();
  QFrags<MT> qf;
  float f[MT][2], fl[MT][2];
  if constexpr (MT == 1) {
    load_q_frags(q, (size_t)row, H, 0, lane, qf.f, f[0]);
  } else {
    uint4 *sq = reinterpret_cast<uint4 *>(a4_smem + TW_WARPS * NST * A4_STAGE);
    qf.s = sq;
    qf.lane = lane;
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      uint32_t t[8][4];
      load_q_frags(q, (size_t)row, H, mt, lane, t, f[mt]);
#pragma unroll
      for (int ks = 0; ks < 8; ks++)
        if ((mt * 8 + ks) % TW_WARPS == warp)
          sq[(mt * 8 + ks) * 32 + lane] = make_uint4(t[ks][0], t[ks][1], t[ks][2], t[ks][3]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int r = 0; r < 2; r++) {
      f[mt][r] *= scale * LOG2E;
      const int h = 16 * mt + (lane >> 2) + 8 * r;
      const float v = h < H ? __ldg(lse + (size_t)row * H + h) : -__int_as_float(0x7f800000);
      // a head of no index (or past the last) has no weights
      fl[mt][r] = v == -__int_as_float(0x7f800000) ? -v : v * LOG2E;
    }
  for (int n = 0; n < ring.nsteps; n++) {
    uint32_t valid;
    int tok = ring.token(n);
    if (tok >= ring.kcap) tok = -1;
    const uint8_t *stage = ring.arrive(n, valid);
    if (!valid) continue;
    float x[MT][4][4];
    kv4_scores<MT>(stage, qf, lane, x);
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) x[mt][j][e] *= f[mt][e >> 1];
    add_weights<MT>(x, fl, tok, (size_t)kbase, lane, weights, status);
  }
  cp_async_wait_all();
  if (__any_sync(0xffffffffu, ring.bad) && lane == 0) raise_status(status, HISA_ERR_INVALID_ARG);
}

// The same for bf16 keys.  Lane (g, c) takes dimensions 32c .. 32c + 31 of token g of
// every 8 straight from memory (64 bytes): fragment w holds the pairs of its 8-dimension
// word w, as does the query's.
template <int MT>
__global__ void __launch_bounds__(TW_WARPS * 32)
token_weights_kernel(const uint16_t *__restrict__ q, const uint16_t *__restrict__ k,
                     const int32_t *__restrict__ idx, const float *__restrict__ lse,
                     const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int S,
                     int H, int topk, float scale, unsigned long long *__restrict__ weights,
                     int *status) {
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int s = find_seq(cu_q, S, row);
  const int kbase = __ldg(cu_k + s), kcap = __ldg(cu_k + s + 1) - kbase;
  const int32_t *irow = idx + (size_t)row * topk;
  const int steps = (topk + A4_STEP - 1) / A4_STEP;
  uint4 qw[MT][2][4];
  float fl[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int r = 0; r < 2; r++) {
      const int h = 16 * mt + g + 8 * r;
#pragma unroll
      for (int i = 0; i < 4; i++)
        qw[mt][r][i] = h < H ? __ldg(reinterpret_cast<const uint4 *>(
                                         q + ((size_t)row * H + h) * KV4_DIM + 32 * c) + i)
                             : make_uint4(0u, 0u, 0u, 0u);
      const float v = h < H ? __ldg(lse + (size_t)row * H + h) : -__int_as_float(0x7f800000);
      fl[mt][r] = v == -__int_as_float(0x7f800000) ? -v : v * LOG2E;
    }
  const float f = scale * LOG2E;
  for (int n = blockIdx.y * TW_WARPS + warp; n < steps; n += gridDim.y * TW_WARPS) {
    const int e = n * A4_STEP + lane;
    int tok = e < topk ? __ldg(irow + e) : -1;
    if (tok >= kcap) {
      raise_status(status, HISA_ERR_INVALID_ARG);
      tok = -1;
    }
    if (!__any_sync(0xffffffffu, tok >= 0)) continue;
    float x[MT][4][4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int t = __shfl_sync(0xffffffffu, tok, 8 * j + g);
      uint4 kw[4];
#pragma unroll
      for (int i = 0; i < 4; i++)
        kw[i] = t >= 0 ? __ldg(reinterpret_cast<const uint4 *>(
                                   k + ((size_t)kbase + t) * KV4_DIM + 32 * c) + i)
                       : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
#pragma unroll
        for (int u = 0; u < 4; u++) x[mt][j][u] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          mma_bf16(x[mt][j], qw[mt][0][i].x, qw[mt][1][i].x, qw[mt][0][i].y, qw[mt][1][i].y,
                   kw[i].x, kw[i].y);
          mma_bf16(x[mt][j], qw[mt][0][i].z, qw[mt][1][i].z, qw[mt][0][i].w, qw[mt][1][i].w,
                   kw[i].z, kw[i].w);
        }
#pragma unroll
        for (int u = 0; u < 4; u++) x[mt][j][u] *= f;
      }
    }
    add_weights<MT>(x, fl, tok, (size_t)kbase, lane, weights, status);
  }
}

// CTAs per row: enough to fill the GPU, at most one step per warp
static int weight_splits(int total_q, int topk, int num_sms) {
  const int steps = (topk + A4_STEP - 1) / A4_STEP, most = (steps + TW_WARPS - 1) / TW_WARPS;
  const int want = (4 * num_sms + total_q - 1) / total_q;
  return want < most ? want : most;
}

cudaError_t launch_token_weights(const uint16_t *q, const uint16_t *k, const int32_t *idx,
                                 const float *lse, const int32_t *cu_q, const int32_t *cu_k, int S,
                                 int total_q, int H, int topk, float scale, int64_t *weights,
                                 int num_sms, int *status, cudaStream_t st) {
  const dim3 grid(total_q, weight_splits(total_q, topk, num_sms));
  unsigned long long *w = reinterpret_cast<unsigned long long *>(weights);
  ProfScope ps(K_TOKEN_WEIGHTS, st);
  if (H <= 16)
    token_weights_kernel<1><<<grid, TW_WARPS * 32, 0, st>>>(q, k, idx, lse, cu_q, cu_k, S, H, topk,
                                                            scale, w, status);
  else
    token_weights_kernel<2><<<grid, TW_WARPS * 32, 0, st>>>(q, k, idx, lse, cu_q, cu_k, S, H, topk,
                                                            scale, w, status);
  return cudaGetLastError();
}

cudaError_t launch_token_weights_kv4(const uint16_t *q, const uint8_t *kv4,
                                     const uint8_t *kv4_scale, const int32_t *idx,
                                     const float *lse, const int32_t *cu_q, const int32_t *cu_k,
                                     int S, int total_q, int H, int topk, float scale,
                                     int64_t *weights, int num_sms, int *status, cudaStream_t st) {
  const dim3 grid(total_q, weight_splits(total_q, topk, num_sms));
  unsigned long long *w = reinterpret_cast<unsigned long long *>(weights);
  constexpr size_t ring = (size_t)TW_WARPS * 3 * A4_STAGE, qb = 2 * 8 * 32 * 16;
  static std::atomic<int> attr[2][64];
  cudaError_t e = H <= 16 ? set_smem_once((const void *)token_weights_kv4_kernel<1>, ring, attr[0])
                          : set_smem_once((const void *)token_weights_kv4_kernel<2>, ring + qb,
                                          attr[1]);
  if (e != cudaSuccess) return e;
  ProfScope ps(K_TOKEN_WEIGHTS, st);
  if (H <= 16)
    token_weights_kv4_kernel<1><<<grid, TW_WARPS * 32, ring, st>>>(
        q, kv4, kv4_scale, idx, lse, cu_q, cu_k, S, H, topk, scale, w, status);
  else
    token_weights_kv4_kernel<2><<<grid, TW_WARPS * 32, ring + qb, st>>>(
        q, kv4, kv4_scale, idx, lse, cu_q, cu_k, S, H, topk, scale, w, status);
  return cudaGetLastError();
}

}  // namespace hisa
