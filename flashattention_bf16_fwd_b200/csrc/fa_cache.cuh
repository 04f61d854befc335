// fa_cache.cuh - writing tokens into a paged key/value cache, and the page
// operators: reserve, fork, free and compact.
//
// Nothing here computes on K and V; they are moved as 16-byte words, and the
// bound is HBM for the copies (append, the tokens of a fork, compact) and
// latency for the rest.  Page numbers are planned by one CTA, which scans the
// reference counts in ascending order, so that the pages chosen are always the
// lowest free ones; the copies then run on the whole GPU in a second kernel
// that reads the plan.
#pragma once

#include "sm100.cuh"

namespace fa {

constexpr int kCacheMaxSeqs = 8192;
constexpr int kPlanThreads = 1024;

struct CacheParams {
  uint4* k_pages;        // [L, P, Hkv, page, d] of 16-bit elements, as 16-byte words
  uint4* v_pages;
  int32_t* refs;         // [P]
  int32_t* table;        // [S, M]
  int32_t* lens;         // [S]
  int* dev_error;
  int S, P, page, M, L, hkv;
  int row_log2;          // a token in one head is 2^row_log2 16-byte words: d / 8
};

__device__ __forceinline__ void cache_error(const CacheParams& p) { atomicExch(p.dev_error, kDevErrPages); }
__device__ __forceinline__ int cache_len(const CacheParams& p, int len) { return min(max(len, 0), p.M * p.page); }
__device__ __forceinline__ bool cache_len_ok(const CacheParams& p, int len) { return len >= 0 && len <= p.M * p.page; }

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
struct AppendParams {
  CacheParams c;
  const uint4* k;        // [T, Hkv, d], k_stride words between tokens
  const uint4* v;
  const int32_t* cu;     // [S + 1] or nullptr
  long long k_stride, v_stride;
  int T;
};

// One warp per token, K and V: the 16-byte words of a token are contiguous in
// the input, and d / 8 of them per head are in a page.  Finding the place takes
// some dependent loads (cu, lens, table), so the token's first 128 words of K and
// V are already on their way: 21600 tokens of 8 x 128 in 28 us (32 us
// with the loads after it and a grid-stride loop).
__global__ void __launch_bounds__(256) fa_cache_append_kernel(const AppendParams a) {
  grid_dep_wait();
  grid_dep_launch();
  const CacheParams& p = a.c;
  const int lane = int(lane_id());
  const int t = int(blockIdx.x) * 8 + int(warp_id());
  if (t >= a.T) return;
  const uint4* k = a.k + t * a.k_stride;
  const uint4* v = a.v + t * a.v_stride;
  const int words = p.hkv << p.row_log2;
  uint4 kw[4], vw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i * 32 + lane < words) {
      kw[i] = k[i * 32 + lane];
      vw[i] = v[i * 32 + lane];
    }
  int s, left;                                   // the sequence, and how many of its tokens follow t - 1
  if (a.cu) {
    if (t < a.cu[0] || t >= a.cu[p.S]) return;
    int lo = 0, hi = p.S;                        // the last s with cu[s] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t) lo = mid; else hi = mid;
    }
    s = lo;
    left = a.cu[s + 1] - t;
  } else {
    s = t;
    left = 1;
    if (p.lens[s] == 0) return;
  }
  const int len = p.lens[s], pos = left > 0 && len >= left ? len - left : -1;
  int id = -1;
  if (pos >= 0 && pos < p.M * p.page) id = p.table[size_t(s) * p.M + pos / p.page];
  if (id < 0 || id >= p.P) {
    if (lane == 0) cache_error(p);
    return;
  }
  const size_t head = size_t(p.page) << p.row_log2;               // words between heads of a page
  const size_t base = size_t(id) * p.hkv * head + (size_t(pos % p.page) << p.row_log2);
  auto place = [&](int w) { return base + (w >> p.row_log2) * head + (w & ((1 << p.row_log2) - 1)); };
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i * 32 + lane < words) {
      p.k_pages[place(i * 32 + lane)] = kw[i];
      p.v_pages[place(i * 32 + lane)] = vw[i];
    }
  for (int w = 128 + lane; w < words; w += 32) {
    const uint4 x = k[w], y = v[w];
    p.k_pages[place(w)] = x;
    p.v_pages[place(w)] = y;
  }
}

// ---------------------------------------------------------------------------
// planning, one CTA of kPlanThreads
// ---------------------------------------------------------------------------
// The sum of x over the CTA's threads before this one; `total` gets the sum of
// all.  `sums`: 32 values of shared memory.
template <typename T>
__device__ __forceinline__ T cta_scan(T x, T* sums, T& total) {
  const int lane = int(lane_id()), warp = int(warp_id());
  T inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  __syncthreads();                                 // the previous scan's sums have been read
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    T y = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T up = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += up;
    }
    sums[lane] = y;
  }
  __syncthreads();
  total = sums[31];
  return (warp ? sums[warp - 1] : T(0)) + inc - x;
}

// Two counts scanned at once, as the halves of a word.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(int hi, int lo) { return Pair(unsigned(hi)) << 32 | unsigned(lo); }
__device__ __forceinline__ int hi_of(Pair x) { return int(x >> 32); }
__device__ __forceinline__ int lo_of(Pair x) { return int(unsigned(x)); }

// The four pages of thread i in the round that begins at page `base`: which are
// free (count 0, or below: a corrupt one) and which in use, as bits.  (16 pages a
// thread make fewer rounds of a large pool, but a thread then hands out up to 16
// pages one after the other: a fork among 1300 pages 9.5 us instead of 7.1.)
constexpr int kPer = 4;
constexpr int kRound = kPer * kPlanThreads;
struct Pages {
  int first;
  unsigned free_bits, used_bits;
  __device__ __forceinline__ Pages(const int32_t* refs, int P, int base)
      : first(base + kPer * int(threadIdx.x)), free_bits(0), used_bits(0) {
    if (first + kPer <= P) {
      const int4 v = *reinterpret_cast<const int4*>(refs + first);
      used_bits = (v.x > 0 ? 1u : 0u) | (v.y > 0 ? 2u : 0u) | (v.z > 0 ? 4u : 0u) | (v.w > 0 ? 8u : 0u);
      free_bits = ~used_bits & 15u;
    } else {
      for (int i = 0; first + i < P; ++i) (refs[first + i] > 0 ? used_bits : free_bits) |= 1u << i;
    }
  }
};

// Calls take(rank, page) for the free pages in ascending order, rank counting
// them from 0, until `most` have been taken.
template <typename F>
__device__ __forceinline__ void take_free(const CacheParams& p, int most, int* sums, F take) {
  int found = 0;
  for (int base = 0; base < p.P && found < most; base += kRound) {
    const Pages q(p.refs, p.P, base);
    int total, rank = found + cta_scan(__popc(q.free_bits), sums, total);
    for (unsigned left = q.free_bits; left && rank < most; left &= left - 1, ++rank) take(rank, q.first + __ffs(left) - 1);
    found += total;
  }
}

__device__ __forceinline__ int count_pages(const CacheParams& p, bool used, int* sums) {
  int n = 0, total;
#pragma unroll 4
  for (int base = 0; base < p.P; base += kRound) {
    const Pages q(p.refs, p.P, base);
    n += __popc(used ? q.used_bits : q.free_bits);
  }
  cta_scan(n, sums, total);
  return total;
}

// Pages that hold len >= 0 tokens.  (The sum may pass 2^31 where a table's row has room for nearly that many.)
__device__ __forceinline__ int pages_of(const CacheParams& p, int len) {
  return int((unsigned(len) + unsigned(p.page - 1)) / unsigned(p.page));
}

// The request that page `rank` belongs to, where need[i] pages are wanted before
// request i: the last i with need[i] <= rank (several may begin at one rank; the
// last of them wants it).
__device__ __forceinline__ int request_of(const int* need, int n, int rank) {
  int a = 0, b = n;
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (need[mid] <= rank) a = mid; else b = mid;
  }
  return a;
}

// need[i] = pages wanted by request i (in shared memory, i < n) -> pages wanted
// before it, and the free pages handed out by take(rank, page) if there are
// enough.  Returns how many are missing.  One scan over both counts where one
// round covers the requests and its pages are enough: a step of a serving loop
// waits for this CTA, and a scan's barriers and a load of the counts are each
// about a tenth of its time.
template <typename F>
__device__ __forceinline__ int hand_out(const CacheParams& p, int* need, int n, F take) {
  __shared__ Pair pair_sums[32];
  __shared__ int sums[32];
  const Pages q(p.refs, p.P, 0);
  const int i = int(threadIdx.x);
  Pair total;
  const Pair before = cta_scan(pair_of(i < n ? need[i] : 0, __popc(q.free_bits)), pair_sums, total);
  if (n <= kPlanThreads && hi_of(total) <= lo_of(total)) {
    if (i < n) need[i] = hi_of(before);
    __syncthreads();
    int rank = lo_of(before);
    for (unsigned left = q.free_bits; left && rank < hi_of(total); left &= left - 1, ++rank)
      take(rank, q.first + __ffs(left) - 1);
    return 0;
  }
  int wanted = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int x = base + i < n ? need[base + i] : 0;
    int round;
    const int at = cta_scan(x, sums, round);
    if (base + i < n) need[base + i] = wanted + at;
    wanted += round;
  }
  const int have = count_pages(p, false, sums);
  if (have < wanted) return wanted - have;
  __syncthreads();                                 // every count and need has been read and written
  take_free(p, wanted, sums, take);
  return 0;
}

// reserve: one CTA.  Dynamic shared memory: S ints.
__global__ void __launch_bounds__(kPlanThreads) fa_cache_reserve_kernel(const CacheParams p, const int32_t* add,
                                                                        int32_t* missing) {
  extern __shared__ int need[];
  grid_dep_wait();
  grid_dep_launch();
  bool bad = false;
  for (int s = threadIdx.x; s < p.S; s += kPlanThreads) {
    const int len = p.lens[s], more = add[s];
    const bool ok = cache_len_ok(p, len) && more >= 0 && more <= p.M * p.page - len;
    bad |= !ok;
    need[s] = ok ? pages_of(p, len + more) - pages_of(p, len) : 0;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      *missing = -1;
      cache_error(p);
    }
    return;
  }
  const int lacking = hand_out(p, need, p.S, [&](int rank, int page) {
    const int s = request_of(need, p.S, rank);
    p.table[size_t(s) * p.M + pages_of(p, p.lens[s]) + rank - need[s]] = page;
    p.refs[page] = 1;
  });
  __syncthreads();                                 // the old lengths have been read
  if (lacking == 0)
    for (int s = threadIdx.x; s < p.S; s += kPlanThreads) p.lens[s] += add[s];
  if (threadIdx.x == 0) *missing = lacking;
}

// One fork: dst takes `whole` shared pages of src and, if rest > 0, page `to`
// with the first `rest` tokens of page `from`.  A `from` that is no page stands in
// dst's row itself, and there is no `to`.
struct ForkPlan {
  int src, dst, whole, rest, from, to;
};

// fork, first kernel: one CTA.  Dynamic shared memory: F ints, F lengths, and
// a bit for each sequence.  The plan holds F entries; plan_n gets F or 0.
__global__ void __launch_bounds__(kPlanThreads) fa_cache_fork_plan_kernel(const CacheParams p, const int32_t* src,
                                                                          const int32_t* dst, int F, ForkPlan* plan,
                                                                          int32_t* plan_n, int32_t* missing) {
  extern __shared__ int need[];
  int* len = need + F;
  unsigned* taken = reinterpret_cast<unsigned*>(len + F);
  grid_dep_wait();
  grid_dep_launch();
  for (int i = threadIdx.x; i < (p.S + 31) / 32; i += kPlanThreads) taken[i] = 0;
  if (threadIdx.x == 0) *plan_n = 0;
  __syncthreads();
  bool bad = false;
  for (int f = threadIdx.x; f < F; f += kPlanThreads) {
    const int a = src[f], b = dst[f];
    bool ok = a >= 0 && a < p.S && b >= 0 && b < p.S;
    const int n = ok ? p.lens[a] : 0;
    if (ok) {
      ok = cache_len_ok(p, n) && p.lens[b] == 0;
      ok &= !(atomicOr(&taken[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u);
    }
    bad |= !ok;
    const int from = ok && n % p.page ? p.table[size_t(a) * p.M + n / p.page] : -1;
    plan[f].from = from;
    len[f] = n;
    need[f] = from >= 0 && from < p.P;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      *missing = -1;
      cache_error(p);
    }
    return;
  }
  const int lacking = hand_out(p, need, F, [&](int rank, int page) {
    const int f = request_of(need, F, rank);
    plan[f].to = page;
    p.table[size_t(dst[f]) * p.M + len[f] / p.page] = page;
    p.refs[page] = 1;
  });
  if (threadIdx.x == 0) *missing = lacking;
  if (lacking) return;
  for (int f = threadIdx.x; f < F; f += kPlanThreads) {
    ForkPlan* e = plan + f;                        // `from` and `to` are written above
    e->src = src[f];
    e->dst = dst[f];
    e->whole = len[f] / p.page;
    e->rest = len[f] % p.page;
    if (e->rest && (e->from < 0 || e->from >= p.P)) p.table[size_t(e->dst) * p.M + e->whole] = e->from;
    p.lens[e->dst] = len[f];
  }
  if (threadIdx.x == 0) *plan_n = F;
}

// fork, second kernel: CTA (f, y) copies the used tokens of fork f's last page
// in the layers y, y + gridDim.y, ...; the CTAs (f, 0) also share the full pages.
__global__ void __launch_bounds__(256) fa_cache_fork_copy_kernel(const CacheParams p, const ForkPlan* plan,
                                                                 const int32_t* plan_n) {
  grid_dep_wait();
  grid_dep_launch();
  if (int(blockIdx.x) >= *plan_n) return;
  const ForkPlan e = plan[blockIdx.x];
  if (blockIdx.y == 0) {
    for (int i = threadIdx.x; i < e.whole; i += 256) {
      const int id = p.table[size_t(e.src) * p.M + i];
      p.table[size_t(e.dst) * p.M + i] = id;
      if (id >= 0 && id < p.P)
        atomicAdd(&p.refs[id], 1);
      else
        cache_error(p);
    }
  }
  if (e.rest == 0) return;
  if (e.from < 0 || e.from >= p.P) {
    if (threadIdx.x == 0) cache_error(p);
    return;
  }
  const int per_head = e.rest << p.row_log2, words = p.hkv * per_head;
  const size_t head = size_t(p.page) << p.row_log2, page = head * p.hkv;
  for (int l = int(blockIdx.y); l < p.L; l += int(gridDim.y)) {
    const size_t from = (size_t(l) * p.P + e.from) * page, to = (size_t(l) * p.P + e.to) * page;
    for (int w = threadIdx.x; w < words; w += 256) {
      const size_t at = (w / per_head) * head + w % per_head;
      const uint4 kw = p.k_pages[from + at], vw = p.v_pages[from + at];
      p.k_pages[to + at] = kw;
      p.v_pages[to + at] = vw;
    }
  }
}

// free: one CTA per entry of seqs.
__global__ void __launch_bounds__(256) fa_cache_free_kernel(const CacheParams p, const int32_t* seqs) {
  grid_dep_wait();
  grid_dep_launch();
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= p.S) {
    if (threadIdx.x == 0) cache_error(p);
    return;
  }
  bool again = false;                              // an earlier entry ends this sequence already
  for (int f = threadIdx.x; f < int(blockIdx.x); f += 256) again |= seqs[f] == s;
  if (__syncthreads_or(again)) return;
  const int len = p.lens[s];
  if (!cache_len_ok(p, len) && threadIdx.x == 0) cache_error(p);
  const int used = pages_of(p, cache_len(p, len));
  for (int i = threadIdx.x; i < used; i += 256) {
    int32_t* entry = p.table + size_t(s) * p.M + i;
    const int id = *entry;
    *entry = -1;
    if (id < 0 || id >= p.P) {
      cache_error(p);
    } else if (atomicSub(&p.refs[id], 1) <= 0) {   // it was free
      atomicAdd(&p.refs[id], 1);
      cache_error(p);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) p.lens[s] = 0;
}

// compact, first kernel: one CTA.  Writes the moves (source pages, and their
// destinations) and which move each of those pages belongs to; counts move with
// the pages.
// With u(x) pages in use before page x, a free page x < live is the destination
// number x - u(x), and a used page x >= live the source number u(x) - u(live).
__global__ void __launch_bounds__(kPlanThreads) fa_cache_compact_plan_kernel(const CacheParams p, int32_t* live_out,
                                                                             int32_t* moves, int32_t* from,
                                                                             int32_t* to, int32_t* went) {
  __shared__ int sums[32];
  __shared__ int u_live;
  grid_dep_wait();
  grid_dep_launch();
  const int live = count_pages(p, true, sums);
  if (threadIdx.x == 0) u_live = live;             // where all pages are in use, and none moves
  int used = 0;
  Pages next(p.refs, p.P, 0);
  for (int base = 0; base < p.P; base += kRound) {
    const Pages q = next;
    next = Pages(p.refs, p.P, base + kRound);      // on its way during this round's scan
    int total;
    int u = used + cta_scan(__popc(q.used_bits), sums, total);
    if (live >= q.first && live < q.first + kPer) u_live = u + __popc(q.used_bits & ((1u << (live - q.first)) - 1u));
    __syncthreads();                               // u(live) is known from its round on
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = q.first + i;
      const bool in_use = q.used_bits >> i & 1u;
      if (x < live && !in_use) {                   // (live <= P)
        to[x - u] = x;
        went[x] = x - u;
      }
      if (x >= live && in_use) {
        from[u - u_live] = x;
        went[x] = u - u_live;
      }
      u += in_use;
    }
    used += total;
  }
  __syncthreads();
  const int n = live - u_live;                     // as many pages in use past live as free ones before it
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int a = from[i], b = to[i];
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  if (threadIdx.x == 0) {
    *moves = n;
    *live_out = live;
  }
}

// compact, second kernel: the moves in all layers, K and V, and the tables.
__global__ void __launch_bounds__(256) fa_cache_compact_copy_kernel(const CacheParams p, const int32_t* live,
                                                                    const int32_t* moves, const int32_t* from,
                                                                    const int32_t* to, const int32_t* went) {
  grid_dep_wait();
  grid_dep_launch();
  const int n = *moves, first = *live;
  const long long entries = (long long)p.S * p.M;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < entries; i += (long long)gridDim.x * 256) {
    const int s = int(i / p.M), at = int(i % p.M), len = p.lens[s];
    if (at == 0 && !cache_len_ok(p, len)) cache_error(p);
    if (at >= pages_of(p, cache_len(p, len))) continue;
    const int id = p.table[i];
    // the move of a page that has one (of others `went` says nothing, and what it
    // holds is checked against the moves)
    const int m = n > 0 && id >= 0 && id < p.P ? went[id] : -1;
    const bool moves_here = m >= 0 && m < n;
    if (id >= 0 && id < first) {
      if (!(moves_here && to[m] == id)) continue;  // a page in use that stays
    } else if (moves_here && from[m] == id) {
      p.table[i] = to[m];
      continue;
    }
    // no page, or a free one: the number may be another page's by now, or soon
    p.table[i] = -1;
    cache_error(p);
  }
  // A group of threads has four words each under way: the CTA where a page is 16 KB
  // or more (8 layers of 32 KB pages: 158 us, warp by warp 161), a warp where it is
  // less, so that as many pages are (4160 moves of 2 KB pages: 33 us, by CTAs 39).
  // All pieces of a pool that fits a GPU are below 2^32.
  const long long page = (long long)p.hkv * p.page << p.row_log2;   // words of a page in one layer
  const int width = page >= 1024 ? 256 : 32, lane = int(threadIdx.x) % width;
  const unsigned pieces = unsigned((page + 4 * width - 1) / (4 * width));
  const unsigned items = 2u * unsigned(p.L) * unsigned(n) * pieces, groups = unsigned(256 / width);
  for (unsigned it = blockIdx.x * groups + threadIdx.x / width; it < items; it += gridDim.x * groups) {
    const unsigned piece = it % pieces, mv = it / pieces, m = mv % unsigned(n), lv = mv / unsigned(n);
    uint4* pool = (lv & 1) ? p.v_pages : p.k_pages;                 // lv: layer, K or V
    const uint4* a = pool + ((long long)(lv >> 1) * p.P + from[m]) * page;
    uint4* b = pool + ((long long)(lv >> 1) * p.P + to[m]) * page;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long w = ((long long)piece * 4 + i) * width + lane;
      if (w < page) x[i] = a[w];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long w = ((long long)piece * 4 + i) * width + lane;
      if (w < page) b[w] = x[i];
    }
  }
}

}  // namespace fa
