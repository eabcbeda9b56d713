// Eviction from a cache by accumulated attention weight (hisa_evict_select,
// hisa_evict_rows).
//
// Select: of a sequence's len tokens at most keep stay: the first n_sink, the last
// n_recent, and of those between the ones with the largest weight, a tie going to the
// lower position.  The threshold weight is found by radix over the 64-bit weights, from
// the highest bit in which any two differ, 11 bits a pass; a pass that leaves a bucket
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
constexpr int EV_PER = 4;  // consecutive tokens of a thread in the emission

__device__ __forceinline__ unsigned long long weight_key(long long w) {
  return (unsigned long long)w ^ 0x8000000000000000ull;
}

__global__ void __launch_bounds__(EV_THREADS)
evict_select_kernel(const long long *__restrict__ weights, const int32_t *__restrict__ cu_k,
                    const int32_t *__restrict__ seqlens, const int32_t *__restrict__ keep,
                    int max_seqlen_k, int n_sink, int n_recent, int32_t *__restrict__ kept,
                    int32_t *__restrict__ kept_len, int *status) {
  __shared__ int hist[EV_BINS];
  __shared__ int scan[EV_THREADS / 32 + 1];
  __shared__ unsigned long long red[2][EV_THREADS / 32];
  __shared__ int s_bin, s_above;
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int base = __ldg(cu_k + s), cap = __ldg(cu_k + s + 1) - base;
  const int len = seqlens ? __ldg(seqlens + s) : cap, budget = __ldg(keep + s);
  if (len < 0 || len > cap || len > max_seqlen_k || budget < 0) {
    if (tid == 0) {
      raise_status(status, HISA_ERR_INVALID_ARG);
      kept_len[s] = -1;
    }
    return;
  }
  int32_t *ks = kept + base;
  if (len <= budget) {
    for (int i = tid; i < len; i += EV_THREADS) ks[i] = i;
    if (tid == 0) kept_len[s] = len;
    return;
  }
  const int sink = min(n_sink, budget), recent = min(n_recent, budget - sink);
  const int quota = budget - sink - recent;  // of the tokens [lo, hi), more than quota
  const int lo = sink, hi = len - recent;
  const long long *ws = weights + base;

  // keys above `thr` stay, of those equal to it the first `ties`
  unsigned long long thr = ~0ull;
  int ties = 0;
  if (quota > 0) {
    unsigned long long a = ~0ull, o = 0ull;
    for (int i = lo + tid; i < hi; i += EV_THREADS) {
      const unsigned long long u = weight_key(__ldg(ws + i));
      a &= u;
      o |= u;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      a &= __shfl_xor_sync(0xffffffffu, a, d);
      o |= __shfl_xor_sync(0xffffffffu, o, d);
    }
    if (lane == 0) {
      red[0][warp] = a;
      red[1][warp] = o;
    }
    __syncthreads();
    a = red[0][lane];
    o = red[1][lane];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      a &= __shfl_xor_sync(0xffffffffu, a, d);
      o |= __shfl_xor_sync(0xffffffffu, o, d);
    }
    int top = a == o ? 0 : 64 - __clzll((long long)(a ^ o));  // bits that differ
    unsigned long long prefix = top == 64 ? 0ull : (a >> top) << top;
    int left = quota;
    while (top > 0) {
      const int shift = max(0, top - EV_BITS), nb = top - shift;
      for (int i = tid; i < EV_BINS; i += EV_THREADS) hist[i] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += EV_THREADS) {
        const unsigned long long d = weight_key(__ldg(ws + i)) ^ prefix;
        if (top == 64 || (d >> top) == 0)
          atomicAdd(&hist[(int)((d >> shift) & ((1u << nb) - 1))], 1);
      }
      __syncthreads();
      // bins from the top, two per thread: the one in which the count passes `left`
      const int b1 = EV_BINS - 1 - 2 * tid, h1 = hist[b1], h0 = hist[b1 - 1];
      int total;
      const int before = block_exclusive_scan<EV_THREADS>(h1 + h0, scan, &total);
      if (before < left && before + h1 >= left) {
        s_bin = b1;
        s_above = before;
      } else if (before + h1 < left && before + h1 + h0 >= left) {
        s_bin = b1 - 1;
        s_above = before + h1;
      }
      __syncthreads();
      left -= s_above;
      prefix |= (unsigned long long)s_bin << shift;
      top = shift;
      const bool whole = hist[s_bin] == left;
      __syncthreads();
      if (whole) break;
    }
    if (top > 0) {  // the whole bucket stays
      thr = prefix - 1;  // prefix > 0: more tokens than the quota, so a lower key exists
    } else {
      thr = prefix;
      ties = left;
    }
  }
  int above = 0, equal = 0;  // middle tokens before this chunk
  for (int c0 = 0; c0 < len; c0 += EV_THREADS * EV_PER) {
    const int i0 = c0 + tid * EV_PER;
    int gt = 0, eq = 0;
    uint32_t fg = 0, fe = 0;
#pragma unroll
    for (int u = 0; u < EV_PER; u++) {
      const int i = i0 + u;
      bool isg = false, ise = false;
      if (i < len) {
        if (i < lo || i >= hi) {
          isg = true;
        } else if (quota > 0) {
          const unsigned long long k = weight_key(__ldg(ws + i));
          isg = k > thr;
          ise = k == thr;
        }
      }
      fg |= (uint32_t)isg << u;
      fe |= (uint32_t)ise << u;
    }
    gt = __popc(fg);
    eq = __popc(fe);
    int total;
    const int before = block_exclusive_scan<EV_THREADS>(gt | (eq << 16), scan, &total);
    int a = above + (before & 0xFFFF), e = equal + (before >> 16);
#pragma unroll
    for (int u = 0; u < EV_PER; u++) {
      const bool isg = (fg >> u) & 1u, ise = (fe >> u) & 1u;
      if (isg || (ise && e < ties)) ks[a + min(e, ties)] = i0 + u;
      a += isg;
      e += ise;
    }
    above += total & 0xFFFF;
    equal += total >> 16;
  }
  if (tid == 0) kept_len[s] = budget;
}

cudaError_t launch_evict_select(const int64_t *weights, const int32_t *cu_k,
                                const int32_t *seqlens, const int32_t *keep, int S,
                                int max_seqlen_k, int n_sink, int n_recent, int32_t *kept,
                                int32_t *kept_len, int *status, cudaStream_t st) {
  ProfScope ps(K_EVICT_SELECT, st);
  evict_select_kernel<<<S, EV_THREADS, 0, st>>>(reinterpret_cast<const long long *>(weights), cu_k,
                                                seqlens, keep, max_seqlen_k, n_sink, n_recent,
                                                kept, kept_len, status);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------

struct RowArrays {
  const uint8_t *src[HISA_MAX_ROW_ARRAYS];
  uint8_t *dst[HISA_MAX_ROW_ARRAYS];
  int bytes[HISA_MAX_ROW_ARRAYS];  // of a row
  int vec[HISA_MAX_ROW_ARRAYS];    // of a copied piece: 16, 8 or 4
  int n;
};

constexpr int ER_THREADS = 256;
constexpr int ER_ROWS = 64;  // rows of a CTA

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

template <typename T>
__device__ __forceinline__ void move_rows(const uint8_t *src, uint8_t *dst, int bytes,
                                          const int *rows, int n, size_t sbase, size_t drow) {
  const int per = bytes / (int)sizeof(T);
  const T *s = reinterpret_cast<const T *>(src);
  T *d = reinterpret_cast<T *>(dst);
  for (int x = threadIdx.x; x < n * per; x += ER_THREADS) {
    const int r = x / per, p = x - r * per;
    const int from = rows[r];
    if (from >= 0) d[(drow + r) * per + p] = __ldg(s + (sbase + from) * per + p);
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
      move_rows<uint4>(a.src[k], a.dst[k], a.bytes[k], rows, n, sb, d);
    else if (a.vec[k] == 8)
      move_rows<uint2>(a.src[k], a.dst[k], a.bytes[k], rows, n, sb, d);
    else
      move_rows<uint32_t>(a.src[k], a.dst[k], a.bytes[k], rows, n, sb, d);
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
    a.n++;
    if (&a == &in) columns += v == 16 && per % 2 == 0 ? per / 2 : per;
  }
  if (out.n > 0) {
    ProfScope ps(K_EVICT_ROWS, st);
    evict_rows_kernel<<<dim3((max_keep + ER_ROWS - 1) / ER_ROWS, S), ER_THREADS, 0, st>>>(
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
