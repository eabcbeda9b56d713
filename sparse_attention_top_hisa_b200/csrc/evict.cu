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
  uint32_t red[EV_THREADS / 32][2];  // counts of the warps
  int odd;                       // a weight below 0 or of 2^58 and more among this CTA's
  int bin, above, in_bin;        // the bin in which the count passes, the counts above and in it
  int2 ahead;                    // of those, the counts of the CTAs before this one
  int any_odd;                   // of the cluster
};

// Warp 0: the bin, from the highest, in which the counts of the cluster's C CTAs pass `left`.
// Two steps of one remote look each: 64 coarse bins, then the 32 bins of one of them.
__device__ __forceinline__ void find_bin(cg::cluster_group &cl, EvictShared &sm, int C, int me,
                                         int buf, int left, int lane) {
  int hi = 0, lo = 0;    // coarse bins 63 - 2 lane and 62 - 2 lane
  int phi = 0, plo = 0;  // the same of the CTAs before this one
  int2 h2[EV_MAX_CLUSTER] = {};  // all in flight before one is used
  if (C == 1)
    h2[0] = *reinterpret_cast<const int2 *>(sm.coarse[buf] + 62 - 2 * lane);
  else
#pragma unroll
    for (int r = 0; r < EV_MAX_CLUSTER; r++)
      if (r < C)
        h2[r] = *reinterpret_cast<const int2 *>(cl.map_shared_rank(sm.coarse[buf], r) + 62 -
                                                2 * lane);
#pragma unroll
  for (int r = 0; r < EV_MAX_CLUSTER; r++) {
    lo += h2[r].x;
    hi += h2[r].y;
    plo += r < me ? h2[r].x : 0;
    phi += r < me ? h2[r].y : 0;
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
  int n = 0, pn = 0;  // bin 31 - lane of the coarse bin
  int h1[EV_MAX_CLUSTER] = {};
  if (C == 1)
    h1[0] = sm.hist[buf][cb * EV_FINE + 31 - lane];
  else
#pragma unroll
    for (int r = 0; r < EV_MAX_CLUSTER; r++)
      if (r < C) h1[r] = cl.map_shared_rank(sm.hist[buf], r)[cb * EV_FINE + 31 - lane];
#pragma unroll
  for (int r = 0; r < EV_MAX_CLUSTER; r++) {
    n += h1[r];
    pn += r < me ? h1[r] : 0;
  }
  int p = lane < src ? phi + plo : lane == src && !upper ? phi : 0;
  x = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  const bool here = above + x - n < left && above + x >= left;
  const int w = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  p = __reduce_add_sync(0xffffffffu, p + (lane < w ? pn : 0));
  if (here) {
    sm.bin = cb * EV_FINE + 31 - lane;
    sm.above = above + x - n;
    sm.in_bin = n;
    sm.ahead = make_int2(p, pn);
  }
}

// Exclusive sums over the block's threads of a thread's counts a and e (at most EV_PER each) of
// NG groups, packed in bytes: at most 128 in a warp.  Of the whole block two 16-bit fields share
// a word.  pa, pe: the sums; sa, se: the totals.
template <int NG>
__device__ __forceinline__ void scan_counts(uint32_t a, uint32_t e, uint32_t (*red)[2],
                                            int (&pa)[NG], int (&pe)[NG], int (&sa)[NG],
                                            int (&se)[NG]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = a, y = e;
  if (NG <= 2) x |= e << 16;  // one word has room for both
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += u;
    if (NG > 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += v;
    }
  }
  if (lane == 31) {
    red[warp][0] = x;
    red[warp][1] = NG <= 2 ? x >> 16 : y;
  }
  __syncthreads();
  if (NG <= 2) y = x >> 16;
  // every warp sums the warps before it: lane w looks at warp w
  const uint2 r = *reinterpret_cast<const uint2 *>(red[lane]);
#pragma unroll
  for (int i = 0; i < NG; i += 2) {  // groups i and i + 1
    const uint32_t ra = __byte_perm(r.x, 0u, i ? 0x4342 : 0x4140);
    const uint32_t re = __byte_perm(r.y, 0u, i ? 0x4342 : 0x4140);
    const uint32_t ta = __reduce_add_sync(0xffffffffu, ra);
    const uint32_t te = __reduce_add_sync(0xffffffffu, re);
    const uint32_t ba = __reduce_add_sync(0xffffffffu, lane < warp ? ra : 0u);
    const uint32_t be = __reduce_add_sync(0xffffffffu, lane < warp ? re : 0u);
#pragma unroll
    for (int j = i; j < NG && j < i + 2; j++) {
      const int h = 16 * (j - i), f = 8 * j;
      sa[j] = (ta >> h) & 0xFFFF;
      se[j] = (te >> h) & 0xFFFF;
      pa[j] = ((ba >> h) & 0xFFFF) + ((x >> f) & 0xFF) - ((a >> f) & 0xFF);
      pe[j] = ((be >> h) & 0xFFFF) + ((y >> f) & 0xFF) - ((e >> f) & 0xFF);
    }
  }
  __syncthreads();
}

template <int N>
struct Const {
  static constexpr int v = N;
};

// 32 bytes from an address that is a multiple of 32
__device__ __forceinline__ void load_four(const long long *p, unsigned long long (&w)[EV_PER]) {
  // volatile: a statement without it may be moved before the check of the alignment
  asm volatile("ld.global.nc.v4.b64 {%0, %1, %2, %3}, [%4];"
               : "=l"(w[0]), "=l"(w[1]), "=l"(w[2]), "=l"(w[3])
               : "l"(p)
               : "memory");
}

// Bits n0 .. n1 - 1 of a group's four, of tokens i .. i + 3: those in [from, to)
__device__ __forceinline__ uint32_t group_bits(int i, int from, int to) {
  const int n0 = min(max(from - i, 0), EV_PER), n1 = min(max(to - i, 0), EV_PER);
  return ((1u << n1) - 1u) & ~((1u << n0) - 1u);
}

// A sequence belongs to a cluster, its tokens in order to the cluster's CTAs; of a CTA's, a
// thread has EV_PER consecutive ones of every group of EV_STRIDE.  G groups: their keys
// stay in registers, 0 for tokens that are not in question; G = 0: any number of groups,
// every pass reads the weights again.
//
// What bounds it: latency, and with several groups the instructions of a token.  Of 31000
// cycles for one sequence of 131072 tokens (eight CTAs, four groups) the loads and the keys
// take 6400, the counts of its two passes 2700 and 1900, each look for the bin 3100, each
// cluster barrier 1000 to 1500, the positions 8000; 1100 tokens of one CTA take 12000 in all.
// So every pass has code of its own, in which the shifts of the 64-bit keys are constants, and
// the counts of the CTAs before this one come with the look for the bin instead of an exchange
// at the end (32.1 us before these two, 24.8 with them, the rows' 6 us among them).
template <int G>
__global__ void __launch_bounds__(EV_THREADS)
evict_select_kernel(const long long *__restrict__ weights, const int32_t *__restrict__ cu_k,
                    const int32_t *__restrict__ seqlens, const int32_t *__restrict__ keep,
                    int max_seqlen_k, int n_sink, int n_recent, int32_t *__restrict__ kept,
                    int32_t *__restrict__ kept_len, int *status) {
  __shared__ EvictShared sm;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), me = (int)cl.block_rank();
  const int lc = 31 - __clz(C);  // C is a power of two
  const int s = blockIdx.x >> lc, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const int chunk = (((len + C - 1) >> lc) + EV_PER - 1) / EV_PER * EV_PER;
  const int c0 = min(len, me * chunk), c1 = min(len, c0 + chunk);
  const int m0 = max(c0, lo), m1 = max(m0, min(c1, hi));  // its middle tokens
  const int first = c0 + tid * EV_PER;                    // this thread's first of group 0
  const int groups = G > 0 ? G : (c1 - c0 + EV_STRIDE - 1) / EV_STRIDE;
  auto middle = [&](int i) { return (uint32_t)(i - m0) < (uint32_t)(m1 - m0); };

  constexpr int KG = G > 0 ? G : 1;
  unsigned long long kx[KG][EV_PER];
  bool plain = false;
  // a thread's four weights of a group are one load where they are all its CTA's and
  // aligned (four groups: 4400 cycles; 6800 by single ones, 32 bytes apart in a warp)
  const bool wide = reinterpret_cast<uintptr_t>(ws) % (EV_PER * sizeof(*ws)) == 0;
  auto read = [&](int i, unsigned long long (&w)[EV_PER]) {
    if (wide && i + EV_PER <= c1) {
      load_four(ws + i, w);
#pragma unroll
      for (int u = 0; u < EV_PER; u++) w[u] = middle(i + u) ? w[u] : 0ull;
    } else {
#pragma unroll
      for (int u = 0; u < EV_PER; u++)
        w[u] = middle(i + u) ? (unsigned long long)__ldg(ws + i + u) : 0ull;
    }
  };
  // the weights, as they are, of this thread's tokens; the bits of all of them
  auto load = [&] {
    unsigned long long o = 0ull;
#pragma unroll
    for (int gr = 0; gr < groups; gr++) {
      unsigned long long w[EV_PER];
      read(first + gr * EV_STRIDE, w);
#pragma unroll
      for (int u = 0; u < EV_PER; u++) {
        if (G > 0) kx[G > 0 ? gr : 0][u] = w[u];
        o |= w[u];
      }
    }
    return o;
  };
  int outside = 0;  // tokens of this thread with a key of 0 that are not in question
  auto to_keys = [&] {
    if (G == 0) return;
    outside = KG * EV_PER;
#pragma unroll
    for (int gr = 0; gr < KG; gr++) {
      const int i = first + gr * EV_STRIDE;
      outside -= __popc(group_bits(i, m0, m1));
#pragma unroll
      for (int u = 0; u < EV_PER; u++)
        kx[gr][u] = plain && !middle(i + u) ? 0ull : weight_key((long long)kx[gr][u], plain);
    }
  };
  // fn(key) for every middle token of this thread (G > 0: for every other one fn(0))
  auto each = [&](auto fn) {
#pragma unroll
    for (int gr = 0; gr < groups; gr++) {
      const int i = first + gr * EV_STRIDE;
      unsigned long long w[EV_PER];
      if (G == 0) read(i, w);
#pragma unroll
      for (int u = 0; u < EV_PER; u++) {
        if (G > 0)
          fn(kx[G > 0 ? gr : 0][u]);
        else if (middle(i + u))
          fn(weight_key((long long)w[u], plain));
      }
    }
  };

  // keys above `thr` stay, of those equal to it the first `ties`
  unsigned long long thr = ~0ull, prefix = 0ull;
  int ties = 0, left = quota, buf = 0;
  // tokens before this CTA's that stay whatever the ties (the fixed ones to begin with), and
  // ties
  int above = min(c0, lo) + max(0, c0 - hi), equal = 0;
  // counts the bits SHIFT .. TOP - 1 of the keys that are `prefix` above them
  auto count = [&](auto top_bit) {
    constexpr int TOP = decltype(top_bit)::v, SHIFT = TOP > EV_BITS ? TOP - EV_BITS : 0;
    int *hist = sm.hist[buf];
    int zero = 0;  // tokens that nothing attended to: often many, and all in one bin
    each([&](unsigned long long k) {
      if (TOP == 64) {
        if (k == 0ull)
          zero++;
        else
          atomicAdd(&hist[(int)(k >> SHIFT)], 1);
      } else {
        const unsigned long long d = k ^ prefix;
        if ((d >> (TOP % 64)) == 0) atomicAdd(&hist[(int)(d >> SHIFT)], 1);
      }
    });
    if (prefix == 0ull) {  // else no key of this pass is 0
      zero = __reduce_add_sync(0xffffffffu, zero - outside);
      if (lane == 0 && zero) atomicAdd(&hist[0], zero);
    }
  };
  if (quota > 0) {
    const unsigned long long o = load();
    if (tid == 0) sm.odd = 0;
    for (int i = tid; i < EV_BINS; i += EV_THREADS) sm.hist[0][i] = 0;
    __syncthreads();
    if (o >> 58) sm.odd = 1;
    to_keys();
    for (int top = 64;;) {  // bits of the keys that are not known yet
      switch (top) {
        case 64: count(Const<64>()); break;
        case 53: count(Const<53>()); break;
        case 42: count(Const<42>()); break;
        case 31: count(Const<31>()); break;
        case 20: count(Const<20>()); break;
        default: count(Const<9>());
      }
      const int shift = max(0, top - EV_BITS);
      __syncthreads();
      const int *hist = sm.hist[buf];
      const int n0 = __reduce_add_sync(0xffffffffu, hist[2 * warp * EV_FINE + lane]);
      const int n1 = __reduce_add_sync(0xffffffffu, hist[(2 * warp + 1) * EV_FINE + lane]);
      if (lane < 2) sm.coarse[buf][2 * warp + lane] = lane ? n1 : n0;
      // every CTA's counts are in; the other buffer has been read
      if (C > 1)
        cl.sync();
      else
        __syncthreads();
      if (warp == 0) {
        if (top == 64) {
          const int odd = lane < C ? *cl.map_shared_rank(&sm.odd, lane) : 0;
          const bool any = __any_sync(0xffffffffu, odd != 0);
          if (lane == 0) sm.any_odd = any;
        }
        find_bin(cl, sm, C, me, buf, left, lane);
      }
      buf ^= 1;
      int *next = sm.hist[buf];
      next[tid] = next[tid + EV_THREADS] = 0;
      __syncthreads();
      if (top == 64 && sm.any_odd && !plain) {  // again, on the weights as they are
        plain = true;
        load();
        to_keys();
        continue;
      }
      left -= sm.above;
      prefix |= (unsigned long long)sm.bin << shift;
      top = shift;
      // the bin stays whole, or (exponent 0) holds zeros only
      const bool whole = sm.in_bin == left, zeros = !plain && (prefix >> 58) == 0;
      const int2 ahead = sm.ahead;
      above += ahead.x;
      __syncthreads();
      if (whole) {
        thr = prefix - 1;  // prefix > 0: more tokens than the quota, so a lower key exists
        above += ahead.y;
        break;
      }
      if (zeros || top == 0) {
        thr = prefix;
        ties = left;
        equal = ahead.y;
        break;
      }
    }
    if (C > 1) cluster_arrive();  // this CTA reads the others' counts no more
  }
  // Bits of this thread's tokens of NG groups from g0 on, four of a group: those above the
  // threshold, the fixed ones among them, and those equal to it.
  constexpr int NG = G > 0 ? G : EV_MAX_GROUPS;
  auto classify = [&](int g0, uint32_t &fg, uint32_t &fe) {
    fg = fe = 0;
#pragma unroll
    for (int gr = 0; gr < NG; gr++) {
      const int i = first + (g0 + gr) * EV_STRIDE;
      const uint32_t mid = group_bits(i, m0, m1) << (4 * gr);
      uint32_t above = 0, equal = 0;
      if (quota > 0) {
        unsigned long long w[EV_PER];
        if (G == 0) read(i, w);
#pragma unroll
        for (int u = 0; u < EV_PER; u++) {
          const unsigned long long k =
              G > 0 ? kx[G > 0 ? gr : 0][u] : weight_key((long long)w[u], plain);
          if (k > thr) above |= 1u << (4 * gr + u);
          if (ties > 0 && k == thr) equal |= 1u << (4 * gr + u);
        }
      }
      fg |= (above & mid) | ((group_bits(i, c0, c1) << (4 * gr)) & ~mid);
      fe |= equal & mid;
    }
  };
  uint32_t fg = 0, fe = 0;
  if (G > 0) classify(0, fg, fe);
  // the positions: NG groups at a time, one scan of their counts
  for (int g0 = 0; g0 < groups; g0 += NG) {
    if (G == 0) classify(g0, fg, fe);
    uint32_t a = 0, e = 0;
#pragma unroll
    for (int gr = 0; gr < NG; gr++) {
      a |= __popc((fg >> (4 * gr)) & 15u) << (8 * gr);
      e |= __popc((fe >> (4 * gr)) & 15u) << (8 * gr);
    }
    int pa[NG], pe[NG], sa[NG], se[NG];
    scan_counts<NG>(a, e, sm.red, pa, pe, sa, se);
#pragma unroll
    for (int gr = 0; gr < NG; gr++) {
      int et = equal + pe[gr], at = above + pa[gr] + min(et, ties);
#pragma unroll
      for (int u = 0; u < EV_PER; u++) {
        const bool tie = (fe >> (4 * gr + u)) & 1u;
        if (((fg >> (4 * gr + u)) & 1u) || (tie && et < ties))
          ks[at++] = first + (g0 + gr) * EV_STRIDE + u;
        et += tie;
      }
      above += sa[gr];
      equal += se[gr];
    }
  }
  if (tid == 0 && me == 0) kept_len[s] = budget;
  if (quota > 0 && C > 1) cluster_wait();  // no CTA leaves while another reads its counts
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
// their selection: 40 us with 128 and 4, 45 with 64 and 4 or 128 and 8, 42 with 256 and 8)
constexpr int ER_ROWS = 128, ER_UNROLL = 4;
// CTAs that an SM holds (48 registers), and how often they may be launched: 47360, 6 million
// rows, which without work are gone in 30 us
constexpr int ER_CTAS = 5, ER_WAVES = 64;

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

// TURNS: a sequence may have more rows than its CTAs have in one turn (code of its own: the loop
// costs the others registers, 32.3 us against 30.4 for 16 sequences of up to 16384 rows).
template <bool TURNS>
__global__ void __launch_bounds__(ER_THREADS)
evict_rows_kernel(const __grid_constant__ RowArrays a, const int32_t *__restrict__ cu_src,
                  const int32_t *__restrict__ cu_dst, const int32_t *__restrict__ kept,
                  const int32_t *__restrict__ kept_len, int max_keep, int *status) {
  __shared__ int rows[ER_ROWS];
  const int s = blockIdx.y;
  const EvictSeq q = evict_seq(cu_src, cu_dst, kept_len, s, max_keep,
                               blockIdx.x == 0 && threadIdx.x == 0, status);
  for (uint32_t r0 = blockIdx.x * ER_ROWS; r0 < (uint32_t)q.n; r0 += gridDim.x * ER_ROWS) {
    const int n = min(ER_ROWS, q.n - (int)r0);
    for (int i = threadIdx.x; i < n; i += ER_THREADS) {
      const int from = __ldg(kept + q.sbase + (size_t)r0 + i);
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
    if (!TURNS) return;
    __syncthreads();  // the positions have been read
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
    // max_keep is only a bound: past ER_WAVES times the CTAs that the card holds, those of a
    // sequence take turns
    const int want = max_keep / ER_ROWS + (max_keep % ER_ROWS != 0);
    const int most = (ER_WAVES * ER_CTAS * num_sms + S - 1) / S;
    const auto fn = want > most ? evict_rows_kernel<true> : evict_rows_kernel<false>;
    fn<<<dim3(want < most ? want : most, S), ER_THREADS, 0, st>>>(
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
