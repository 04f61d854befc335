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
// all.  `sums`: 33 ints of shared memory.
__device__ __forceinline__ int cta_scan(int x, int* sums, int& total) {
  const int lane = int(lane_id()), warp = int(warp_id());
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  __syncthreads();                                 // the previous scan's sums have been read
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int y = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += up;
    }
    sums[lane] = y;
  }
  __syncthreads();
  total = sums[31];
  return (warp ? sums[warp - 1] : 0) + inc - x;
}

// Visits the pages [from, to) in ascending order, 4 per thread and round, and
// calls take(rank, page) for those that are free (kFree) or in use (!kFree),
// rank counting them from 0, until `most` have been found.  Returns how many
// were found (at least `most` if there are so many).
template <bool kFree, typename F>
__device__ __forceinline__ int visit_pages(const int32_t* refs, int from, int to, int most, int* sums, F take) {
  int found = 0;
  for (int base = from & ~3; base < to && found < most; base += 4 * kPlanThreads) {
    const int at = base + 4 * int(threadIdx.x);
    int r[4] = {0, 0, 0, 0};
    if (at >= from && at + 4 <= to) {
      const int4 v = *reinterpret_cast<const int4*>(refs + at);
      r[0] = v.x;
      r[1] = v.y;
      r[2] = v.z;
      r[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i >= from && at + i < to) r[i] = refs[at + i];
    }
    bool hit[4];
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hit[i] = at + i >= from && at + i < to && (kFree ? r[i] <= 0 : r[i] > 0);
      n += hit[i];
    }
    int total;
    int rank = found + cta_scan(n, sums, total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (hit[i] && rank < most) {
        take(rank, at + i);
        ++rank;
      }
    found += total;
  }
  return found;
}

__device__ __forceinline__ int pages_of(const CacheParams& p, int len) { return (len + p.page - 1) / p.page; }

// need[i] = pages wanted by request i, i < n (in shared memory) -> need[i] =
// pages wanted before request i; returns the total.
__device__ __forceinline__ int scan_needs(int* need, int n, int* sums) {
  int before = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + int(threadIdx.x);
    const int x = i < n ? need[i] : 0;
    int total;
    const int at = cta_scan(x, sums, total);
    if (i < n) need[i] = before + at;
    before += total;
  }
  __syncthreads();
  return before;
}

// The request that page `rank` belongs to: the last i with need[i] <= rank.
__device__ __forceinline__ int request_of(const int* need, int n, int rank) {
  int a = 0, b = n;
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (need[mid] <= rank) a = mid; else b = mid;
  }
  return a;
}

// reserve: one CTA.  Dynamic shared memory: S ints.
__global__ void __launch_bounds__(kPlanThreads) fa_cache_reserve_kernel(const CacheParams p, const int32_t* add,
                                                                        int32_t* missing) {
  extern __shared__ int need[];
  __shared__ int sums[33];
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
  const int total = scan_needs(need, p.S, sums);
  const int have = visit_pages<true>(p.refs, 0, p.P, total, sums, [](int, int) {});
  if (have < total) {
    if (threadIdx.x == 0) *missing = total - have;
    return;
  }
  __syncthreads();                                 // every count has been read
  visit_pages<true>(p.refs, 0, p.P, total, sums, [&](int rank, int page) {
    const int s = request_of(need, p.S, rank);
    p.table[size_t(s) * p.M + pages_of(p, p.lens[s]) + rank - need[s]] = page;
    p.refs[page] = 1;
  });
  __syncthreads();                                 // the old lengths have been read
  for (int s = threadIdx.x; s < p.S; s += kPlanThreads) p.lens[s] += add[s];
  if (threadIdx.x == 0) *missing = 0;
}

// One fork: dst takes `whole` shared pages of src and, if rest > 0, page `to`
// with the first `rest` tokens of page `from`.
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
  __shared__ int sums[33];
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
    len[f] = n;
    need[f] = ok && n % p.page != 0;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      *missing = -1;
      cache_error(p);
    }
    return;
  }
  const int total = scan_needs(need, F, sums);
  const int have = visit_pages<true>(p.refs, 0, p.P, total, sums, [](int, int) {});
  if (have < total) {
    if (threadIdx.x == 0) *missing = total - have;
    return;
  }
  for (int f = threadIdx.x; f < F; f += kPlanThreads) {
    ForkPlan e;
    e.src = src[f];
    e.dst = dst[f];
    e.whole = len[f] / p.page;
    e.rest = len[f] % p.page;
    e.from = e.rest ? p.table[size_t(e.src) * p.M + e.whole] : -1;
    e.to = -1;
    plan[f] = e;
    p.lens[e.dst] = len[f];
  }
  __syncthreads();
  visit_pages<true>(p.refs, 0, p.P, total, sums, [&](int rank, int page) {
    const int f = request_of(need, F, rank);       // several requests may start at one rank: the last of them needs it
    plan[f].to = page;
    p.table[size_t(plan[f].dst) * p.M + plan[f].whole] = page;
    p.refs[page] = 1;
  });
  if (threadIdx.x == 0) {
    *plan_n = F;
    *missing = 0;
  }
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
// destinations) and which move each source page is; counts move with the pages.
__global__ void __launch_bounds__(kPlanThreads) fa_cache_compact_plan_kernel(const CacheParams p, int32_t* live_out,
                                                                             int32_t* moves, int32_t* from,
                                                                             int32_t* to, int32_t* went) {
  __shared__ int sums[33];
  grid_dep_wait();
  grid_dep_launch();
  const int live = visit_pages<false>(p.refs, 0, p.P, p.P, sums, [](int, int) {});
  const int n = visit_pages<false>(p.refs, live, p.P, p.P, sums, [&](int rank, int page) { from[rank] = page; });
  __syncthreads();
  visit_pages<true>(p.refs, 0, live, n, sums, [&](int rank, int page) { to[rank] = page; });
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int a = from[i], b = to[i];
    went[a] = i;
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  if (threadIdx.x == 0) {
    *moves = n;
    *live_out = live;
  }
}

// compact, second kernel: the moves in all layers, K and V, one piece of a page
// per CTA and round, and the tables.
__global__ void __launch_bounds__(256) fa_cache_compact_copy_kernel(const CacheParams p, const int32_t* live,
                                                                    const int32_t* moves, const int32_t* from,
                                                                    const int32_t* to, const int32_t* went) {
  grid_dep_wait();
  grid_dep_launch();
  const int n = *moves, first = *live;
  const long long entries = (long long)p.S * p.M;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < entries; i += (long long)gridDim.x * 256) {
    const int s = int(i / p.M);
    if (int(i % p.M) >= pages_of(p, cache_len(p, p.lens[s]))) continue;
    const int id = p.table[i];
    if (id < first && id >= 0) continue;
    // a page past the pages in use moved, unless the table names a free page
    const int m = id >= 0 && id < p.P ? went[id] : -1;
    if (m >= 0 && m < n && from[m] == id)
      p.table[i] = to[m];
    else
      cache_error(p);
  }
  const long long page = (long long)p.hkv * p.page << p.row_log2;   // words of a page in one layer
  constexpr int kPiece = 256 * 4;                                   // words that a CTA has in flight
  const long long pieces = (page + kPiece - 1) / kPiece;
  const long long items = 2ll * p.L * n * pieces;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const long long piece = it % pieces;
    const int m = int(it / pieces % n);
    const int lv = int(it / pieces / n);                            // layer, K or V
    uint4* pool = (lv & 1) ? p.v_pages : p.k_pages;
    const uint4* a = pool + ((long long)(lv >> 1) * p.P + from[m]) * page;
    uint4* b = pool + ((long long)(lv >> 1) * p.P + to[m]) * page;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long w = piece * kPiece + i * 256 + threadIdx.x;
      if (w < page) x[i] = a[w];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long w = piece * kPiece + i * 256 + threadIdx.x;
      if (w < page) b[w] = x[i];
    }
  }
}

}  // namespace fa
