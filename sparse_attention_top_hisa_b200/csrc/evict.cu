// Eviction from a cache by accumulated attention weight (hisa_evict_select,
// hisa_evict_rows).
//
// Select: of a sequence's len tokens at most keep stay: the first n_sink, the last
// n_recent, and of those between the ones with the largest weight, a tie going to the
// lower position.  The threshold is found by radix over 64-bit keys of the weights, 11 bits
// a pass, with one histogram per CTA of the sequence's cluster; a pass whose bucket is
// taken whole is the last.  Then one pass emits the positions in ascending order.
//
// Rows: the rows that stay move to the front of their destination region, in order.  In
// place, row i comes from a row kept[i] >= i: a step of rows may be written once all of
// its own rows have been read, and later steps read behind everything it writes.
#include <cooperative_groups.h>

#include "common.cuh"
#include "prof.cuh"

namespace cg = cooperative_groups;

namespace hisa {

constexpr int EV_THREADS = 1024;
constexpr int EV_BITS = 11, EV_BINS = 1 << EV_BITS;
constexpr int EV_PER = 4;                            // consecutive tokens of a thread
constexpr int EV_STRIDE = EV_THREADS * EV_PER;       // tokens of a group
constexpr int EV_MAX_GROUPS = 4;                     // groups whose keys stay in registers
constexpr int EV_MAX_CLUSTER = 8;

// Order-preserving keys.  Weights of 0 .. 2^58 - 1 (any sum of attention weights below 2^26)
// become a 6-bit exponent and the 58 bits behind the leading one, so that the first 11
// bits already tell weights 3% apart, wherever in their range the threshold lies; if a
// sequence has any other weight, its keys are the 64 bits with the sign turned.
__device__ __forceinline__ unsigned long long weight_key(long long w, bool plain) {
  if (plain) return (unsigned long long)w ^ 0x8000000000000000ull;
  if (w == 0) return 0ull;
  const int e = 64 - __clzll(w);  // 1 .. 58
  return ((unsigned long long)e << 58) | ((((unsigned long long)w << (64 - e)) << 1) >> 6);
}

constexpr int EV_FINE = 32, EV_COARSE = EV_BINS / EV_FINE;  // bins of a coarse bin; coarse bins
static_assert(EV_COARSE == 64 && EV_THREADS == 1024, "two coarse bins per warp and per lane");

struct EvictShared {
  int hist[2][EV_BINS];
  int coarse[2][EV_COARSE];
  unsigned long long red[2][EV_THREADS / 32];
  int odd;                       // a weight below 0 or of 2^58 and more among this CTA's
  int bin, above, in_bin;        // the bin in which the count passes, the counts above and in it
  int any_odd;                   // of the cluster
  int2 counts;                   // middle and fixed tokens above the threshold, ties
};

// Warp 0: the bin, from the highest, in which the counts of the cluster's C CTAs pass `left`.
// Two steps of one remote look each: 64 coarse bins, then the 32 bins of one of them.
__device__ __forceinline__ void find_bin(cg::cluster_group &cl, EvictShared &sm, int C, int buf,
                                         int left, int lane) {
  int hi = 0, lo = 0;  // coarse bins 63 - 2 lane and 62 - 2 lane
#pragma unroll
  for (int r = 0; r < EV_MAX_CLUSTER; r++)
    if (r < C) {
      const int2 h =
          *reinterpret_cast<const int2 *>(cl.map_shared_rank(sm.coarse[buf], r) + 62 - 2 * lane);
      lo += h.x;
      hi += h.y;
    }
  int x = hi + lo;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  const int before = x - hi - lo;
  const unsigned at = __ballot_sync(0xffffffffu, before < left && x >= left);
  const int src = __ffs(at) - 1;  // one lane: left <= the count of the keys looked at
  const bool upper = before + hi >= left;
  const int cb = __shfl_sync(0xffffffffu, upper ? 63 - 2 * lane : 62 - 2 * lane, src);
  const int above = __shfl_sync(0xffffffffu, upper ? before : before + hi, src);
  int n = 0;  // bin 31 - lane of the coarse bin
#pragma unroll
  for (int r = 0; r < EV_MAX_CLUSTER; r++)
    if (r < C) n += cl.map_shared_rank(sm.hist[buf], r)[cb * EV_FINE + 31 - lane];
  x = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (above + x - n < left && above + x >= left) {
    sm.bin = cb * EV_FINE + 31 - lane;
    sm.above = above + x - n;
    sm.in_bin = n;
  }
}

// Exclusive sums over the block's threads of four 16-bit fields each; *sa, *sb the totals.
__device__ __forceinline__ void scan_fields(unsigned long long &a, unsigned long long &b,
                                            unsigned long long (*red)[EV_THREADS / 32],
                                            unsigned long long *sa, unsigned long long *sb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = a, y = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, x, d);
    const unsigned long long v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    red[0][warp] = x;
    red[1][warp] = y;
  }
  __syncthreads();
  // every warp sums the warps before it: lane w looks at warp w
  unsigned long long p = red[0][lane], q = red[1][lane];
  unsigned long long pa = lane < warp ? p : 0ull, qa = lane < warp ? q : 0ull;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    p += __shfl_xor_sync(0xffffffffu, p, d);
    q += __shfl_xor_sync(0xffffffffu, q, d);
    pa += __shfl_xor_sync(0xffffffffu, pa, d);
    qa += __shfl_xor_sync(0xffffffffu, qa, d);
  }
  a = pa + x - a;
  b = qa + y - b;
  *sa = p;
  *sb = q;
  __syncthreads();
}

// A sequence belongs to a cluster, its tokens in order to the cluster's CTAs; of a CTA's, a
// thread has EV_PER consecutive ones of every group of EV_STRIDE.  G groups: their keys
// stay in registers; G = 0: any number of groups, every pass reads the weights again.
template <int G>
__global__ void __launch_bounds__(EV_THREADS)
evict_select_kernel(const long long *__restrict__ weights, const int32_t *__restrict__ cu_k,
                    const int32_t *__restrict__ seqlens, const int32_t *__restrict__ keep,
                    int max_seqlen_k, int n_sink, int n_recent, int32_t *__restrict__ kept,
                    int32_t *__restrict__ kept_len, int *status) {
  __shared__ EvictShared sm;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), me = (int)cl.block_rank();
  const int s = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int base = __ldg(cu_k + s), cap = __ldg(cu_k + s + 1) - base;
  const int len = seqlens ? __ldg(seqlens + s) : cap, budget = __ldg(keep + s);
  // these leave the whole cluster together
  if (len < 0 || len > cap || len > max_seqlen_k || budget < 0) {
    if (tid == 0 && me == 0) {
      raise_status(status, HISA_ERR_INVALID_ARG);
      kept_len[s] = -1;
    }
    return;
  }
  int32_t *ks = kept + base;
  if (len <= budget) {
    for (int i = me * EV_THREADS + tid; i < len; i += C * EV_THREADS) ks[i] = i;
    if (tid == 0 && me == 0) kept_len[s] = len;
    return;
  }
  const int sink = min(n_sink, budget), recent = min(n_recent, budget - sink);
  const int quota = budget - sink - recent;  // of the tokens [lo, hi), more than quota
  const int lo = sink, hi = len - recent;
  const long long *ws = weights + base;
  // this CTA's tokens: [c0, c1), a whole number of EV_PER but for the last
  const int chunk = ((len + C - 1) / C + EV_PER - 1) / EV_PER * EV_PER;
  const int c0 = min(len, me * chunk), c1 = min(len, c0 + chunk);
  const int m0 = max(c0, lo), m1 = min(c1, hi);  // its middle tokens
  const int first = c0 + tid * EV_PER;           // this thread's first of group 0
  const int groups = G > 0 ? G : (c1 - c0 + EV_STRIDE - 1) / EV_STRIDE;

  unsigned long long kx[G > 0 ? G : 1][EV_PER];
  bool plain = false;
  // fn(key) for every middle token of this thread
  auto each = [&](auto fn) {
#pragma unroll
    for (int gr = 0; gr < groups; gr++)
#pragma unroll
      for (int u = 0; u < EV_PER; u++) {
        const int i = first + gr * EV_STRIDE + u;
        if (i >= m0 && i < m1) fn(G > 0 ? kx[G > 0 ? gr : 0][u] : weight_key(__ldg(ws + i), plain));
      }
  };

  // keys above `thr` stay, of those equal to it the first `ties`
  unsigned long long thr = ~0ull;
  int ties = 0;
  if (quota > 0) {
    unsigned long long o = 0ull;
#pragma unroll
    for (int gr = 0; gr < groups; gr++)
#pragma unroll
      for (int u = 0; u < EV_PER; u++) {
        const int i = first + gr * EV_STRIDE + u;
        const unsigned long long w =
            i >= m0 && i < m1 ? (unsigned long long)__ldg(ws + i) : 0ull;
        if (G > 0) kx[G > 0 ? gr : 0][u] = w;
        o |= w;
      }
    if (tid == 0) sm.odd = 0;
    for (int i = tid; i < EV_BINS; i += EV_THREADS) sm.hist[0][i] = 0;
    __syncthreads();
    if (o >> 58) sm.odd = 1;
    auto to_keys = [&] {
      if (G > 0) {
#pragma unroll
        for (int gr = 0; gr < (G > 0 ? G : 1); gr++)
#pragma unroll
          for (int u = 0; u < EV_PER; u++) kx[gr][u] = weight_key((long long)kx[gr][u], plain);
      }
    };
    to_keys();
    unsigned long long prefix = 0ull;
    int left = quota, top = 64;  // bits of the keys that are not known yet
    for (int pass = 0; top > 0; pass++) {
      const int shift = max(0, top - EV_BITS), nb = top - shift, buf = pass & 1;
      int *hist = sm.hist[buf];
      int zero = 0;  // tokens that nothing attended to: often many, and all in one bin
      each([&](unsigned long long k) {
        const unsigned long long d = k ^ prefix;
        if (k == 0ull)
          zero++;
        else if (top == 64 || (d >> top) == 0)
          atomicAdd(&hist[(int)((d >> shift) & ((1u << nb) - 1))], 1);
      });
      if (prefix == 0ull) {  // else no bucket of this pass holds the key 0
        zero = __reduce_add_sync(0xffffffffu, zero);
        if (lane == 0 && zero) atomicAdd(&hist[0], zero);
      }
      __syncthreads();
      const int n0 = __reduce_add_sync(0xffffffffu, hist[2 * warp * EV_FINE + lane]);
      const int n1 = __reduce_add_sync(0xffffffffu, hist[(2 * warp + 1) * EV_FINE + lane]);
      if (lane < 2) sm.coarse[buf][2 * warp + lane] = lane ? n1 : n0;
      // every CTA's counts are in; the other buffer has been read
      if (C > 1)
        cl.sync();
      else
        __syncthreads();
      if (warp == 0) {
        if (pass == 0) {
          const int odd = lane < C ? *cl.map_shared_rank(&sm.odd, lane) : 0;
          const bool any = __any_sync(0xffffffffu, odd != 0);
          if (lane == 0) sm.any_odd = any;
        }
        find_bin(cl, sm, C, buf, left, lane);
      }
      int *next = sm.hist[buf ^ 1];
      next[tid] = next[tid + EV_THREADS] = 0;
      __syncthreads();
      if (pass == 0 && sm.any_odd && !plain) {  // once more, on the weights as they are
        plain = true;
        if (G > 0) {
#pragma unroll
          for (int gr = 0; gr < (G > 0 ? G : 1); gr++)
#pragma unroll
            for (int u = 0; u < EV_PER; u++) {
              const int i = first + gr * EV_STRIDE + u;
              kx[gr][u] = i >= m0 && i < m1 ? (unsigned long long)__ldg(ws + i) : 0ull;
            }
          to_keys();
        }
        continue;
      }
      left -= sm.above;
      prefix |= (unsigned long long)sm.bin << shift;
      top = shift;
      // the bin stays whole, or (exponent 0) holds zeros only
      const bool whole = sm.in_bin == left, zeros = !plain && (prefix >> 58) == 0;
      __syncthreads();
      if (whole) break;
      if (zeros) top = 0;
    }
    if (top > 0) {  // the whole bucket stays
      thr = prefix - 1;  // prefix > 0: more tokens than the quota, so a lower key exists
    } else {
      thr = prefix;
      ties = left;
    }
  }
  // Counts of this CTA's tokens above the threshold (the fixed ones among them) and equal
  // to it, for the CTAs behind it; then the positions.
  int above = 0, equal = 0;
  if (C > 1) {
    int gt = 0, eq = 0;
    if (quota > 0)
      each([&](unsigned long long k) {
        gt += k > thr;
        eq += k == thr;
      });
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) sm.red[0][warp] = ((unsigned long long)(uint32_t)eq << 32) | (uint32_t)gt;
    __syncthreads();
    if (warp == 0) {
      const unsigned long long v = sm.red[0][lane];
      gt = __reduce_add_sync(0xffffffffu, (int)(uint32_t)v) + (c1 - c0) - max(0, m1 - m0);
      eq = __reduce_add_sync(0xffffffffu, (int)(v >> 32));
      if (lane == 0) sm.counts = make_int2(gt, eq);
    }
    cl.sync();
    int2 v = make_int2(0, 0);
    if (lane < me) v = *cl.map_shared_rank(&sm.counts, lane);
    above = __reduce_add_sync(0xffffffffu, v.x);
    equal = __reduce_add_sync(0xffffffffu, v.y);
  }
  // EV_MAX_GROUPS groups at a time: four bits of a thread's tokens per group, one scan
  for (int g0 = 0; g0 < groups; g0 += EV_MAX_GROUPS) {
    uint32_t fg = 0, fe = 0;
    unsigned long long a = 0, e = 0, sa, se;
#pragma unroll
    for (int gr = 0; gr < (G > 0 ? G : EV_MAX_GROUPS); gr++) {
#pragma unroll
      for (int u = 0; u < EV_PER; u++) {
        const int i = first + (g0 + gr) * EV_STRIDE + u;
        bool isg = false, ise = false;
        if (i < c1) {
          if (i < lo || i >= hi) {
            isg = true;
          } else if (quota > 0) {
            const unsigned long long k =
                G > 0 ? kx[G > 0 ? gr : 0][u] : weight_key(__ldg(ws + i), plain);
            isg = k > thr;
            ise = k == thr;
          }
        }
        fg |= (uint32_t)isg << (4 * gr + u);
        fe |= (uint32_t)ise << (4 * gr + u);
      }
      a |= (unsigned long long)__popc((fg >> (4 * gr)) & 15u) << (16 * gr);
      e |= (unsigned long long)__popc((fe >> (4 * gr)) & 15u) << (16 * gr);
    }
    scan_fields(a, e, sm.red, &sa, &se);
#pragma unroll
    for (int gr = 0; gr < (G > 0 ? G : EV_MAX_GROUPS); gr++) {
      int at = above + (int)((a >> (16 * gr)) & 0xFFFF);
      int et = equal + (int)((e >> (16 * gr)) & 0xFFFF);
#pragma unroll
      for (int u = 0; u < EV_PER; u++) {
        const bool isg = (fg >> (4 * gr + u)) & 1u, ise = (fe >> (4 * gr + u)) & 1u;
        if (isg || (ise && et < ties))
          ks[at + min(et, ties)] = first + (g0 + gr) * EV_STRIDE + u;
        at += isg;
        et += ise;
      }
      above += (int)((sa >> (16 * gr)) & 0xFFFF);
      equal += (int)((se >> (16 * gr)) & 0xFFFF);
    }
  }
  if (tid == 0 && me == 0) kept_len[s] = budget;
  if (C > 1) cl.sync();  // no CTA leaves while another reads its counts
}

cudaError_t launch_evict_select(const int64_t *weights, const int32_t *cu_k,
                                const int32_t *seqlens, const int32_t *keep, int S,
                                int max_seqlen_k, int n_sink, int n_recent, int32_t *kept,
                                int32_t *kept_len, int num_sms, int *status, cudaStream_t st) {
  // a sequence is split over a cluster while that leaves SMs idle and every CTA has two
  // tokens per thread
  int C = 1;
  while (C < EV_MAX_CLUSTER && (long long)S * C * 2 <= num_sms &&
         max_seqlen_k >= C * 2 * 2 * EV_THREADS)
    C *= 2;
  const int chunk = ((max_seqlen_k + C - 1) / C + EV_PER - 1) / EV_PER * EV_PER;
  const int groups = (chunk + EV_STRIDE - 1) / EV_STRIDE;
  const auto fn = groups <= 1   ? evict_select_kernel<1>
                  : groups <= 2 ? evict_select_kernel<2>
                  : groups <= 4 ? evict_select_kernel<4>
                                : evict_select_kernel<0>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S * C);
  cfg.blockDim = dim3(EV_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = C;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  ProfScope ps(K_EVICT_SELECT, st);
  return cudaLaunchKernelEx(&cfg, fn, reinterpret_cast<const long long *>(weights), cu_k, seqlens,
                            keep, max_seqlen_k, n_sink, n_recent, kept, kept_len, status);
}

// ---------------------------------------------------------------------------

struct RowArrays {
  const uint8_t *src[HISA_MAX_ROW_ARRAYS];
  uint8_t *dst[HISA_MAX_ROW_ARRAYS];
  int bytes[HISA_MAX_ROW_ARRAYS];  // of a row
  int vec[HISA_MAX_ROW_ARRAYS];    // of a copied piece: 16, 8 or 4
  int shift[HISA_MAX_ROW_ARRAYS];  // log2 of a row's pieces, -1 where that is no whole number
  int n;
};

constexpr int ER_THREADS = 256;
// rows of a CTA and pieces of a thread in flight (16 sequences of up to 32768 tokens with
// their selection: 43 us with 128 and 4, 51 with 64 and 4, 52 with 256 and 8)
constexpr int ER_ROWS = 128, ER_UNROLL = 4;

struct EvictSeq {
  int sbase, dbase, scap, n;
};

// The bases and the count of sequence s, n = 0 when it cannot be moved.
__device__ __forceinline__ EvictSeq evict_seq(const int32_t *cu_src, const int32_t *cu_dst,
                                              const int32_t *kept_len, int s, int max_keep,
                                              bool report, int *status) {
  EvictSeq r;
  r.sbase = __ldg(cu_src + s);
  r.scap = __ldg(cu_src + s + 1) - r.sbase;
  r.dbase = __ldg(cu_dst + s);
  const int dcap = __ldg(cu_dst + s + 1) - r.dbase;
  r.n = __ldg(kept_len + s);
  if (r.n < 0 || r.n > r.scap || r.n > max_keep) {
    if (report) raise_status(status, HISA_ERR_INVALID_ARG);
    r.n = 0;
  } else if (r.n > dcap) {
    if (report) raise_status(status, HISA_ERR_CAPACITY);
    r.n = 0;
  }
  return r;
}

// Rows rows[0 .. n) of the source to drow, drow + 1, ...: ER_UNROLL pieces of a thread are
// read before any is written.
template <typename T>
__device__ __forceinline__ void move_rows(const uint8_t *src, uint8_t *dst, int per, int shift,
                                          const int *rows, int n, size_t sbase, size_t drow) {
  const T *s = reinterpret_cast<const T *>(src) + sbase * per;
  T *d = reinterpret_cast<T *>(dst) + drow * per;
  const int total = n * per;
  for (int x0 = threadIdx.x; x0 < total; x0 += ER_UNROLL * ER_THREADS) {
    T v[ER_UNROLL];
    bool ok[ER_UNROLL];
#pragma unroll
    for (int u = 0; u < ER_UNROLL; u++) {
      const int x = x0 + u * ER_THREADS;
      ok[u] = false;
      if (x < total) {
        const int r = shift >= 0 ? x >> shift : x / per, from = rows[r];
        ok[u] = from >= 0;
        if (ok[u]) v[u] = __ldg(s + (size_t)from * per + (x - r * per));
      }
    }
#pragma unroll
    for (int u = 0; u < ER_UNROLL; u++)
      if (ok[u]) d[x0 + u * ER_THREADS] = v[u];
  }
}

__global__ void __launch_bounds__(ER_THREADS)
evict_rows_kernel(const __grid_constant__ RowArrays a, const int32_t *__restrict__ cu_src,
                  const int32_t *__restrict__ cu_dst, const int32_t *__restrict__ kept,
                  const int32_t *__restrict__ kept_len, int max_keep, int *status) {
  __shared__ int rows[ER_ROWS];
  const int s = blockIdx.y, r0 = blockIdx.x * ER_ROWS;
  const EvictSeq q = evict_seq(cu_src, cu_dst, kept_len, s, max_keep,
                               blockIdx.x == 0 && threadIdx.x == 0, status);
  const int n = min(ER_ROWS, q.n - r0);
  if (n <= 0) return;
  for (int i = threadIdx.x; i < n; i += ER_THREADS) {
    const int from = __ldg(kept + q.sbase + r0 + i);
    if (from < 0 || from >= q.scap) raise_status(status, HISA_ERR_INVALID_ARG);
    rows[i] = from < 0 || from >= q.scap ? -1 : from;
  }
  __syncthreads();
  for (int k = 0; k < a.n; k++) {
    const size_t sb = (size_t)q.sbase, d = (size_t)q.dbase + r0;
    if (a.vec[k] == 16)
      move_rows<uint4>(a.src[k], a.dst[k], a.bytes[k] / 16, a.shift[k], rows, n, sb, d);
    else if (a.vec[k] == 8)
      move_rows<uint2>(a.src[k], a.dst[k], a.bytes[k] / 8, a.shift[k], rows, n, sb, d);
    else
      move_rows<uint32_t>(a.src[k], a.dst[k], a.bytes[k] / 4, a.shift[k], rows, n, sb, d);
  }
}

// In place: a CTA (or a cluster) owns a column of the rows of one array, so that nobody
// else writes what it reads.  A column is two pieces of 16 bytes (a 32-byte sector) where
// the row has them, else one piece.
constexpr int EI_THREADS = 512, EI_PER = 8, EI_CLUSTER = 8;

template <typename T>
__device__ __forceinline__ void move_column(const uint8_t *buf, int bytes, int col, int pieces,
                                            const int32_t *kept, const EvictSeq &q, int first,
                                            cg::cluster_group &cl, int *status) {
  const int per = bytes / (int)sizeof(T), C = (int)cl.num_blocks();
  T *b = reinterpret_cast<T *>(const_cast<uint8_t *>(buf));
  const int step = EI_THREADS / pieces * EI_PER;  // rows of a CTA's step
  const int piece = threadIdx.x % pieces, r = threadIdx.x / pieces;
  for (int r0 = first; r0 < q.n; r0 += step * C) {
    const int mine = r0 + (int)cl.block_rank() * step + r;
    T v[EI_PER];
    bool ok[EI_PER];
#pragma unroll
    for (int u = 0; u < EI_PER; u++) {
      const int i = mine + u * (EI_THREADS / pieces);
      ok[u] = false;
      if (i < q.n) {
        const int from = __ldg(kept + q.sbase + i);
        // rows that stay where they are need no copy; any other must come from behind
        ok[u] = from > i && from < q.scap;
        if (from < i || from >= q.scap) raise_status(status, HISA_ERR_INVALID_ARG);
        if (ok[u]) v[u] = b[((size_t)q.sbase + from) * per + col + piece];
      }
    }
    // every row of the step has been read by every CTA of the column
    if (C > 1)
      cl.sync();
    else
      __syncthreads();
#pragma unroll
    for (int u = 0; u < EI_PER; u++)
      if (ok[u])
        b[((size_t)q.sbase + mine + u * (EI_THREADS / pieces)) * per + col + piece] = v[u];
  }
}

__global__ void __launch_bounds__(EI_THREADS)
evict_rows_inplace_kernel(const __grid_constant__ RowArrays a, int cluster,
                          const int32_t *__restrict__ cu_src, const int32_t *__restrict__ cu_dst,
                          const int32_t *__restrict__ kept, const int32_t *__restrict__ kept_len,
                          int max_keep, int *status) {
  cg::cluster_group cl = cg::this_cluster();
  const int s = blockIdx.y;
  int col = blockIdx.x / cluster, k = 0, pieces = 1;
  for (;; k++) {  // the array and the column in it
    const int per = a.bytes[k] / a.vec[k];
    pieces = a.vec[k] == 16 && per % 2 == 0 ? 2 : 1;
    if (col < per / pieces) break;
    col -= per / pieces;
  }
  const bool report = blockIdx.x == 0 && threadIdx.x == 0;
  EvictSeq q = evict_seq(cu_src, cu_dst, kept_len, s, max_keep, report, status);
  if (q.sbase != q.dbase) {  // regions that differ cannot be moved in place
    if (report) raise_status(status, HISA_ERR_INVALID_ARG);
    return;
  }
  // kept[i] - i never falls: the first row that moves, by halving
  int lo = 0, hi = q.n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(kept + q.sbase + mid) > mid) hi = mid; else lo = mid + 1;
  }
  if (a.vec[k] == 16)
    move_column<uint4>(a.src[k], a.bytes[k], col * pieces, pieces, kept, q, lo, cl, status);
  else if (a.vec[k] == 8)
    move_column<uint2>(a.src[k], a.bytes[k], col * pieces, pieces, kept, q, lo, cl, status);
  else
    move_column<uint32_t>(a.src[k], a.bytes[k], col * pieces, pieces, kept, q, lo, cl, status);
}

static int piece_bytes(const hisa_rows &r) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(r.src) | reinterpret_cast<uintptr_t>(r.dst) |
                      (uintptr_t)r.row_bytes;
  return x % 16 == 0 ? 16 : x % 8 == 0 ? 8 : 4;
}

cudaError_t launch_evict_rows(const hisa_rows *arrays, int n, const int32_t *cu_src,
                              const int32_t *cu_dst, const int32_t *kept, const int32_t *kept_len,
                              int S, int max_keep, int num_sms, int *status, cudaStream_t st) {
  RowArrays out = {}, in = {};
  int columns = 0;
  for (int i = 0; i < n; i++) {
    RowArrays &a = arrays[i].src == arrays[i].dst ? in : out;
    const int v = piece_bytes(arrays[i]), per = (int)arrays[i].row_bytes / v;
    a.src[a.n] = static_cast<const uint8_t *>(arrays[i].src);
    a.dst[a.n] = static_cast<uint8_t *>(arrays[i].dst);
    a.bytes[a.n] = (int)arrays[i].row_bytes;
    a.vec[a.n] = v;
    a.shift[a.n] = (per & (per - 1)) == 0 ? __builtin_ctz((unsigned)per) : -1;
    a.n++;
    if (&a == &in) columns += v == 16 && per % 2 == 0 ? per / 2 : per;
  }
  if (out.n > 0) {
    ProfScope ps(K_EVICT_ROWS, st);
    evict_rows_kernel<<<dim3(max_keep / ER_ROWS + (max_keep % ER_ROWS != 0), S), ER_THREADS, 0, st>>>(
        out, cu_src, cu_dst, kept, kept_len, max_keep, status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (in.n == 0) return cudaSuccess;
  // a column is split over a cluster while the columns alone leave SMs idle
  int C = 1;
  while (C < EI_CLUSTER && columns * S * C * 2 <= num_sms &&
         max_keep > C * EI_THREADS / 2 * EI_PER)
    C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(columns * C, S);
  cfg.blockDim = dim3(EI_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = C;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  ProfScope ps(K_EVICT_ROWS, st);
  return cudaLaunchKernelEx(&cfg, evict_rows_inplace_kernel, in, C, cu_src, cu_dst, kept, kept_len,
                            max_keep, status);
}

}  // namespace hisa
