// fa_decode.cuh - attention of one new token per sequence over a paged cache.
//
// Per sequence and query head, over the keys j that it sees:
//   x_j = scale q.K_j,  O = sum_j e^(x_j - m) V_j / sum_j e^(x_j - m),
//   LSE = m + log sum_j e^(x_j - m).
// Every K and V element is used by the group of query heads that share it and
// by nothing else, so the bound is the bandwidth at which the visible tokens
// come out of HBM; the arithmetic only has to stay out of the way.
//
// Work.  The keys of a sequence are cut into tiles of 64 (d = 64: 128, so that a
// tile is 32 KB of K and V either way); the tiles of all (sequence, key/value
// head) units, laid end to end, are divided evenly among the CTAs, whatever the
// lengths: each CTA takes one stretch.  A place without a tile follows each
// unit's tiles, for finishing a unit costs about as much as a tile (that, and
// joining the warps' O in a stage at once instead of 32 columns at a time: 256
// sequences of up to 300 tokens, H = 32 over Hkv = 8, d = 128: 60 -> 53 us).  A
// unit that lies in one stretch is finished there; one that is cut leaves
// unnormalised partial results (O, m, l), at most two per CTA, which
// fa_decode_join_kernel puts together.  The cut depends on lens alone, so that
// sums always run in the same order.  Where the table has room for few tiles per
// sequence, units are left whole and the second launch is not made.
//
// A CTA: warp 4 fetches tiles with TMA into a ring, one box per page (or piece of
// one) and 64 elements of d, with the queries in front of a unit's first tile;
// page numbers are read for up to 32 boxes at a time, a batch ahead.  Warps 0-3
// take a quarter of a tile's keys each and keep a running maximum, sum and O of
// their own in registers, so that they meet only at the end of a unit.
// The products run on mma.sync with the keys as rows, S^T = K Q^T and
// O^T = V^T P^T: 8 query heads are one N = 8 tile, where tcgen05 would spend
// 128 rows on them.  P enters as P_hi + P_lo, two values of the element format:
// two products instead of one, on a tensor core that is idle otherwise, and no
// rounding of P in O.
#pragma once

#include "sm100.cuh"

namespace fa {

struct DecodeParams {
  const void* q;         // [S, H, D], q_stride elements between sequences
  const int32_t* table;  // [S, M]
  const int32_t* lens;   // [S]
  void* o;               // [S, H, D]
  float* lse;            // [S, H]
  int32_t* cum;          // workspace: [S + 1] places of a unit of each earlier sequence
  float* part;           // workspace: [2 * CTAs] partial results
  int* dev_error;
  long long q_stride;
  int S, H, group, units;   // query heads per K/V head; units per sequence (K/V heads x head blocks)
  int blocks;               // head blocks per K/V head
  int P, page, M, box;      // box: keys per TMA box (a divisor of the tile and of the page)
  int z_none;               // a third TMA coordinate past the cache: the box reads as zeros
  int window, sinks;
  int ctas;                 // CTAs that the places are divided among
  int whole;                // no unit is cut: a stretch begins and ends with one
  float scale_log2;
};

constexpr int dec_tile(int D) { return D == 64 ? 128 : 64; }   // keys per tile
constexpr int kDecMaxSeqs = 8192;
constexpr int kDecMaxCtas = 320;   // two per SM

template <int D, int NB>
struct DecLayout {
  static constexpr int kTile = dec_tile(D);
  static constexpr int kSub = D / 64;
  static constexpr int kSubBytes = kTile * 128;              // a tile's keys x 64 elements
  static constexpr int kTileBytes = kSub * kSubBytes;        // 16 KB of K, and of V
  static constexpr int kStages = 3;                          // 96 KB in flight per CTA, two CTAs per SM
  // the warps' O are joined in the stage that held the unit's last tile, this
  // many columns of d at a time: [4 warps][8 NB heads][kJoinRow] floats
  static constexpr int kJoinCols = NB == 1 ? D : 64;
  static constexpr int kJoinRow = kJoinCols + 4;             // rows 4 banks apart: the warps' writes do not collide
  static_assert(4 * 8 * NB * kJoinRow * 4 <= 2 * kTileBytes, "the join does not fit a stage");
  static constexpr int kMlOff = kStages * 2 * kTileBytes;    // [2][4 warps][8 NB] m and l
  static constexpr int kMlFloats = 4 * 8 * NB * 2;
  // the queries of a unit, beside the stage of its first tile; 16 heads of 128
  // would cost the second CTA per SM and are read from global memory
  static constexpr bool kQSmem = !(NB == 2 && D == 128);
  static constexpr int kQBytes = kQSmem ? 8 * NB * D * 2 : 0;
  static constexpr int kQOff = kMlOff + 2 * kMlFloats * 4;
  static constexpr int kBarOff = kQOff + kStages * kQBytes;
  static constexpr int kCumOff = kBarOff + 128;              // [S + 1] as DecodeParams::cum, then [S] lengths
  static constexpr int kThreads = 160;
  // lengths are kept beside them while that leaves two CTAs per SM
  // (113 KB each; one CTA alone took 84 us for 256 sequences of up to 300 tokens,
  // two 60 us), and are read from global memory in larger batches
  static constexpr int kLensMost = 512;
  static size_t bytes(int S) { return size_t(kCumOff) + (size_t(S) + 1 + (S <= kLensMost ? S : 0)) * 4 + 1024; }
  static_assert(kCumOff + (2 * kLensMost + 1) * 4 + 1024 <= 113 * 1024, "a second CTA does not fit");
};

// The tiles of a sequence: those with a sink, then those of the window (all
// keys where nothing is hidden).  Keys are counted without a sign: a table's row
// may have room for 2^31 - 8 tokens, and the last tile then ends past 2^31.
struct DecSpan {
  unsigned n, lo, sk;    // visible: key < n and (key >= lo or key < sk)
  int st, skip;     // tiles before the gap; tiles in the gap
  int nt;           // tiles
};

template <int kTile>
__device__ __forceinline__ DecSpan dec_span(const DecodeParams& p, int len) {
  DecSpan s;
  const int n = min(max(len, 0), p.M * p.page);
  s.n = n;
  s.lo = p.window > 0 ? max(0, n - p.window) : 0;
  s.sk = min(p.sinks, n);
  const int all = int((s.n + kTile - 1) / kTile);
  s.st = int((s.sk + kTile - 1) / kTile);
  s.skip = max(0, int(s.lo / kTile) - s.st);
  s.nt = all - s.skip;
  return s;
}

template <int kTile>
__device__ __forceinline__ unsigned dec_key0(const DecSpan& s, int t) {
  return unsigned(t < s.st ? t : t + s.skip) * kTile;
}

// First place of CTA c's stretch when T places are divided among G CTAs.
__device__ __forceinline__ long long dec_cut(long long T, int G, int c) { return T * c / G; }

// A place in the sequence of all units' tiles: tile t of a unit of sequence s,
// or, where t is the unit's number of tiles, the place without one behind it.
struct DecWalk {
  int s, unit, t, nt;
  __device__ __forceinline__ void start(const int32_t* cum, int S, int units, long long x) {
    int a = 0, b = S;               // the last s with cum[s] * units <= x and tiles of its own
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if ((long long)cum[mid] * units <= x) a = mid; else b = mid;
    }
    s = a;
    const int places = cum[s + 1] - cum[s];
    const int r = int(x - (long long)cum[s] * units);
    unit = r / places;
    t = r % places;
    nt = places - 1;
  }
  __device__ __forceinline__ void next(const int32_t* cum, int S, int units) {
    if (++t <= nt) return;
    t = 0;
    if (++unit < units) return;
    unit = 0;
    do ++s; while (s < S && cum[s + 1] == cum[s]);
    nt = s < S ? cum[s + 1] - cum[s] - 1 : 0;
  }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// The transpose of an 8 x 8 matrix of 16-bit elements held across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <typename E>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (E::kMmaFmt == 1)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An untiled copy of `bytes` (a multiple of 16) from global to shared memory,
// both 16-byte aligned, completing on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// NB: blocks of 8 query heads that one CTA takes together.
template <int D, int NB, typename E>
__global__ void __launch_bounds__(160, 2)
    fa_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const DecodeParams p) {
  using L = DecLayout<D, NB>;
  using T = typename E::T;
  constexpr int kTile = L::kTile, kRows = kTile / 64;       // kRows: pieces of 16 keys per warp and tile
  constexpr float kLn2 = 0.69314718055994531f;
  const float kNegInf = -__int_as_float(0x7f800000);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* ml_both = reinterpret_cast<float*>(smem + L::kMlOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + L::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + L::kStages);
  int* warp_sum = reinterpret_cast<int*>(smem + L::kBarOff + 64);
  int32_t* cum = reinterpret_cast<int32_t*>(smem + L::kCumOff);
  int32_t* lens_smem = cum + p.S + 1;
  const int32_t* lens = p.S <= L::kLensMost ? lens_smem : p.lens;
  const int warp = int(warp_id()), lane = int(lane_id());

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  grid_dep_wait();
  grid_dep_launch();

  // cum: each thread sums a run of sequences, the runs are scanned over the CTA.
  const int run = (p.S + L::kThreads - 1) / L::kThreads;
  const int s_begin = min(p.S, int(threadIdx.x) * run), s_end = min(p.S, s_begin + run);
  int mine = 0;
  bool bad = false;
  for (int s = s_begin; s < s_end; ++s) {
    const int len = p.lens[s];
    bad |= len < 0 || len > p.M * p.page;
    if (p.S <= L::kLensMost) lens_smem[s] = len;
    const int nt = dec_span<kTile>(p, len).nt;
    mine += nt ? nt + 1 : 0;
    cum[s + 1] = mine;
  }
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += up;
  }
  if (lane == 31) warp_sum[warp] = before;
  before -= mine;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  for (int s = s_begin; s < s_end; ++s) cum[s + 1] += before;
  if (threadIdx.x == 0) cum[0] = 0;
  if (bad && blockIdx.x == 0) atomicExch(p.dev_error, kDevErrPages);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s <= p.S; s += L::kThreads) p.cum[s] = cum[s];
  // empty sequences: O = 0, LSE = -inf
  for (int s = blockIdx.x; s < p.S; s += gridDim.x) {
    if (cum[s + 1] != cum[s]) continue;
    for (int i = threadIdx.x; i < p.H * D / 8; i += L::kThreads)
      reinterpret_cast<uint4*>(static_cast<T*>(p.o) + size_t(s) * p.H * D)[i] = make_uint4(0, 0, 0, 0);
    for (int h = threadIdx.x; h < p.H; h += L::kThreads) p.lse[size_t(s) * p.H + h] = kNegInf;
  }

  const long long total = (long long)cum[p.S] * p.units;
  long long x0 = dec_cut(total, p.ctas, blockIdx.x), x1 = dec_cut(total, p.ctas, blockIdx.x + 1);
  if (x0 == x1) return;
  DecWalk w;
  if (p.whole) {                      // both on to the next unit's first place
    w.start(cum, p.S, p.units, x0);
    if (w.t) x0 += w.nt + 1 - w.t;
    if (x1 < total) {
      w.start(cum, p.S, p.units, x1);
      if (w.t) x1 += w.nt + 1 - w.t;
    }
  }
  const int n = int(x1 - x0);
  if (n <= 0) return;
  const Watchdog wd{abort_flag, p.dev_error};
  w.start(cum, p.S, p.units, x0);
  // the query heads of a unit: the first one, and how many
  auto heads = [&](const DecWalk& u, int& h0, int& nh) {
    const int kvh = u.unit / p.blocks;
    h0 = kvh * p.group + (u.unit % p.blocks) * 8 * NB;
    nh = min(8 * NB, (kvh + 1) * p.group - h0);
  };

  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    // Lanes take the boxes of 32 / boxes places at a time, K and V: where their
    // box begins, and its page.  A batch's page numbers are read while the batch
    // before it is copied.
    const int boxes = kTile / p.box, batch = 32 / boxes;
    const int my_place = lane / boxes, my_box = lane % boxes;
    const uint64_t pol = l2_policy_evict_first();
    const int hkv = p.units / p.blocks;
    int id = 0, row = 0, head = 0;           // this lane's box: page number, row of the page, K/V head
    bool seen = false, real = false;         // a query sees a key of the box; the place has a tile
    const void* q = nullptr;                 // lane of a tile's first box: the queries to fetch with it
    uint32_t q_bytes = 0;
    auto look = [&](int i0) {
      const int i = i0 + my_place;
      q_bytes = 0;
      seen = real = false;
      if (i >= n) return;
      DecWalk u;
      u.start(cum, p.S, p.units, x0 + i);
      real = u.t < u.nt;
      if (!real) return;
      const DecSpan sp = dec_span<kTile>(p, lens[u.s]);
      const unsigned key = dec_key0<kTile>(sp, u.t) + unsigned(my_box * p.box);
      row = int(key % unsigned(p.page));
      head = u.unit / p.blocks;
      seen = key < sp.n && (key + p.box > sp.lo || key < sp.sk);
      if (seen) id = p.table[size_t(u.s) * p.M + key / unsigned(p.page)];   // not looked at before its batch's turn
      if (L::kQSmem && my_box == 0 && (i == 0 || u.t == 0)) {          // the unit's first tile here
        int h0, nh;
        heads(u, h0, nh);
        q = static_cast<const T*>(p.q) + size_t(u.s) * p.q_stride + size_t(h0) * D;
        q_bytes = uint32_t(nh) * D * 2;
      }
    };
    look(0);
    bool ok = true;
    int i = 0;                               // tiles fetched
    for (int i0 = 0; ok && i0 < n; i0 += batch) {
      if (seen && (id < 0 || id >= p.P)) {
        seen = false;
        atomicExch(p.dev_error, kDevErrPages);
      }
      const int z = seen ? id * hkv + head : p.z_none, r = row;       // unseen and bad pages read as zeros
      const void* src = q;
      const uint32_t src_bytes = q_bytes, tiles = __ballot_sync(0xffffffffu, real && my_box == 0);
      if (i0 + batch < n) look(i0 + batch);
      for (int b = 0; b < batch; ++b) {
        if (!(tiles >> (b * boxes) & 1u)) continue;
        const int st = i % L::kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ((i / L::kStages) & 1) ^ 1, wd));
        if (!ok) break;
        const bool mine = my_place == b;
        if (mine && my_box == 0) {
          mbar_arrive_expect_tx(&full[st], uint32_t(2 * L::kTileBytes) + src_bytes);
          if (src_bytes) bulk_load(smem + L::kQOff + st * L::kQBytes, src, src_bytes, &full[st]);
        }
        __syncwarp();
        if (mine) {
          uint8_t* sk = smem + st * 2 * L::kTileBytes + my_box * p.box * 128;
#pragma unroll
          for (int s = 0; s < L::kSub; ++s) {
            tma_load_3d(sk + s * L::kSubBytes, &tm_k, &full[st], s * 64, r, z, pol);
            tma_load_3d(sk + L::kTileBytes + s * L::kSubBytes, &tm_v, &full[st], s * 64, r, z, pol);
          }
        }
        ++i;
      }
    }
    // given up: the copies in flight still write this CTA's shared memory; wait
    // for them (at most a second each) before the CTA ends
    if (!ok) {
      for (int k = max(0, i - L::kStages); k < i; ++k) {
        const uint64_t end = globaltimer_ns() + 1000000000ull;
        while (!mbar_try_wait(&full[k % L::kStages], (k / L::kStages) & 1) && globaltimer_ns() < end) {
        }
      }
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int g = lane >> 2, tq = lane & 3;
  uint32_t qf[D / 16][NB][2];
  float ms[NB][2], l[NB][2], o[D / 16][NB][4];
  bool ok = true, fresh = true;
  int seg_t0 = 0;                     // the unit's first tile in this stretch
  DecSpan sp{};
  const uint32_t tile0 = smem_u32(smem);
  const int row_k = warp * (16 * kRows) + (lane & 15);                          // K: rows of the four matrices
  const int row_v = warp * (16 * kRows) + (lane & 7) + ((lane >> 4) << 3);      // V: keys of the four matrices

  int i = 0, ends = 0;                // tiles taken; results joined
  for (int x = 0; x < n; ++x, w.next(cum, p.S, p.units)) {
    if (w.t == w.nt) continue;        // the place behind a unit
    int h0, nh;
    heads(w, h0, nh);
    const int st = i % L::kStages;
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (i / L::kStages) & 1, wd));
    if (fresh) {
      sp = dec_span<kTile>(p, lens[w.s]);
      seg_t0 = w.t;
      // heads past the unit's last are computed from whatever is there and not
      // stored; no column of S^T or O^T depends on another
      const T* q = L::kQSmem ? reinterpret_cast<const T*>(smem + L::kQOff + st * L::kQBytes)
                             : static_cast<const T*>(p.q) + size_t(w.s) * p.q_stride + size_t(h0) * D;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const T* qr = q + (L::kQSmem || nb * 8 + g < nh ? nb * 8 + g : 0) * D + tq * 2;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][nb][0] = *reinterpret_cast<const uint32_t*>(qr + k * 16);
          qf[k][nb][1] = *reinterpret_cast<const uint32_t*>(qr + k * 16 + 8);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ms[nb][e] = kNegInf;
          l[nb][e] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][nb][e] = 0.f;
      }
      fresh = false;
    }
    auto seen = [&](unsigned key) { return key < sp.n && (key >= sp.lo || key < sp.sk); };
    const unsigned kw = dec_key0<kTile>(sp, w.t) + unsigned(warp * (16 * kRows));   // this warp's first key
    const bool whole = kw + 16 * kRows <= sp.n && (kw >= sp.lo || kw + 16 * kRows <= sp.sk);
    const bool none = kw >= sp.n || (kw >= sp.sk && kw + 16 * kRows <= sp.lo);
    if (ok && !none) {
      const uint32_t tk = tile0 + st * 2 * L::kTileBytes, tv = tk + L::kTileBytes;
      float c[kRows][NB][4];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[r][nb][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          uint32_t a[4];
          ldsm4(a, tk + (k >> 2) * L::kSubBytes + (row_k + 16 * r) * 128 +
                       ((((k & 3) * 2 + (lane >> 4)) ^ (row_k & 7)) << 4));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816<E>(c[r][nb], a, qf[k][nb][0], qf[k][nb][1]);
        }
      }
      if (!whole) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const bool sa = seen(kw + 16 * r + g), sb = seen(kw + 16 * r + g + 8);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            c[r][nb][0] = sa ? c[r][nb][0] : kNegInf;
            c[r][nb][1] = sa ? c[r][nb][1] : kNegInf;
            c[r][nb][2] = sb ? c[r][nb][2] : kNegInf;
            c[r][nb][3] = sb ? c[r][nb][3] : kNegInf;
          }
        }
      }
      uint32_t ph[kRows][NB][2], pl[kRows][NB][2];
      bool moved = false;
      float alpha[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(c[0][nb][e], c[0][nb][e + 2]);
#pragma unroll
          for (int r = 1; r < kRows; ++r) mx = fmaxf(mx, fmaxf(c[r][nb][e], c[r][nb][e + 2]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float m_new = fmaxf(ms[nb][e], mx * p.scale_log2);
          const float shift = m_new == kNegInf ? 0.f : m_new;
          alpha[nb][e] = ex2(ms[nb][e] - shift);           // 0 where nothing was seen before
          moved |= m_new != ms[nb][e];
          ms[nb][e] = m_new;
          float sum = 0.f;
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            c[r][nb][e] = ex2(fmaf(c[r][nb][e], p.scale_log2, -shift));
            c[r][nb][e + 2] = ex2(fmaf(c[r][nb][e + 2], p.scale_log2, -shift));
            sum += c[r][nb][e] + c[r][nb][e + 2];
          }
          l[nb][e] = fmaf(l[nb][e], alpha[nb][e], sum);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int hv = 0; hv < 2; ++hv) {                  // keys 0-7, 8-15 of the 16
            const float a = c[r][nb][2 * hv], b = c[r][nb][2 * hv + 1];
            const uint32_t hi = E::pack(a, b);
            const float2 q = E::unpack(hi);
            ph[r][nb][hv] = transpose8(hi);
            pl[r][nb][hv] = transpose8(E::pack(a - q.x, b - q.y));
          }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][nb][e] *= alpha[nb][e & 1];
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        // hidden keys: P is 0, and V is cleared because 0 times what lies there
        // need not be 0
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (!whole) {
          const unsigned kk = kw + 16 * r + tq * 2;
          keep0 = (seen(kk) ? 0xffffu : 0u) | (seen(kk + 1) ? 0xffff0000u : 0u);
          keep1 = (seen(kk + 8) ? 0xffffu : 0u) | (seen(kk + 9) ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t a[4];
          ldsm4_t(a, tv + (k >> 2) * L::kSubBytes + (row_v + 16 * r) * 128 +
                         ((((k & 3) * 2 + ((lane >> 3) & 1)) ^ (row_v & 7)) << 4));
          a[0] &= keep0;
          a[1] &= keep0;
          a[2] &= keep1;
          a[3] &= keep1;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma16816<E>(o[k][nb], a, ph[r][nb][0], ph[r][nb][1]);
            mma16816<E>(o[k][nb], a, pl[r][nb][0], pl[r][nb][1]);
          }
        }
      }
    }
    ++i;
    const bool unit_end = w.t + 1 == w.nt;
    if (!unit_end && x + 1 < n) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      continue;
    }

    // The unit's end, or the stretch's: the four warps' results are joined.  m and
    // l of one unit and the next lie apart, for a warp may come here again while
    // another still reads them.
    float* ml = ml_both + (ends++ & 1) * L::kMlFloats;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[nb][e];
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (g == 0) {
          const int hd = nb * 8 + tq * 2 + e;
          ml[(warp * 8 * NB + hd) * 2] = ms[nb][e];
          ml[(warp * 8 * NB + hd) * 2 + 1] = y;
        }
      }
    named_bar_sync(1, 128);           // m and l are written, and all warps are done with the stage
    float* join = reinterpret_cast<float*>(smem + st * 2 * L::kTileBytes);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hd = nb * 8 + tq * 2 + e;
        float m = kNegInf;
#pragma unroll
        for (int v = 0; v < 4; ++v) m = fmaxf(m, ml[(v * 8 * NB + hd) * 2]);
        const float f = ms[nb][e] == kNegInf ? 0.f : ex2(ms[nb][e] - m);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          o[k][nb][e] *= f;
          o[k][nb][e + 2] *= f;
        }
      }
    const bool done = unit_end && seg_t0 == 0;       // the unit lies in this stretch
    // the first slot belongs to a unit that began in an earlier stretch, or with this one
    float* part = p.part + (size_t(blockIdx.x) * 2 + (x - w.t <= 0 ? 0 : 1)) * (8 * NB * (D + 2));
#pragma unroll
    for (int ch = 0; ch < D / L::kJoinCols; ++ch) {
      constexpr int kPer = L::kJoinCols / 16;        // 16-wide pieces of d at a time
#pragma unroll
      for (int k = 0; k < kPer; ++k)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            join[(warp * 8 * NB + nb * 8 + tq * 2 + (e & 1)) * L::kJoinRow + k * 16 + g + (e >> 1) * 8] =
                o[ch * kPer + k][nb][e];
      named_bar_sync(1, 128);
      constexpr int kItems = 8 * NB * L::kJoinCols / 4;   // four columns of a head
#pragma unroll
      for (int it = int(threadIdx.x); it < kItems; it += 128) {
        const int hd = it / (L::kJoinCols / 4), col = it % (L::kJoinCols / 4) * 4;
        float m = kNegInf, lsum = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) m = fmaxf(m, ml[(v * 8 * NB + hd) * 2]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float mv = ml[(v * 8 * NB + hd) * 2];
          lsum += mv == kNegInf ? 0.f : ml[(v * 8 * NB + hd) * 2 + 1] * ex2(mv - m);
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float4 b = *reinterpret_cast<const float4*>(join + (v * 8 * NB + hd) * L::kJoinRow + col);
          a.x += b.x;
          a.y += b.y;
          a.z += b.z;
          a.w += b.w;
        }
        const int dd = ch * L::kJoinCols + col;
        if (!done) {
          *reinterpret_cast<float4*>(part + 16 * NB + hd * D + dd) = a;
          if (dd == 0) {
            part[hd] = m;
            part[8 * NB + hd] = lsum;
          }
        } else if (hd < nh) {
          const float inv = 1.f / lsum;
          uint2 r;
          r.x = E::pack(a.x * inv, a.y * inv);
          r.y = E::pack(a.z * inv, a.w * inv);
          *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + (size_t(w.s) * p.H + h0 + hd) * D + dd) = r;
          if (dd == 0) p.lse[size_t(w.s) * p.H + h0 + hd] = (m + lg2(lsum)) * kLn2;
        }
      }
      if (ch + 1 < D / L::kJoinCols) named_bar_sync(1, 128);
    }
    // the next copy into this stage follows the join's reads and writes there
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    fresh = true;
  }
}

// Puts a cut unit's partial results together: one CTA per (sequence, query
// head); units that one CTA finished, and empty sequences, are left alone.
// A thread holds four elements of d and every fourth (d = 64: eighth) of the
// unit's pieces, with a running maximum of its own, so that all loads of a unit
// of up to 16 pieces are in flight together: this kernel is the tail of every
// call, and a second round trip to the L2 is a quarter of its time.
template <int D, int NB, typename E>
__global__ void __launch_bounds__(128) fa_decode_join_kernel(const DecodeParams p) {
  using T = typename E::T;
  constexpr float kLn2 = 0.69314718055994531f;
  const float kNegInf = -__int_as_float(0x7f800000);
  constexpr int kCols = D / 4, kRuns = 128 / kCols;
  __shared__ float4 acc[128];
  __shared__ float run_m[kRuns], run_l[kRuns];
  grid_dep_wait();
  grid_dep_launch();
  const int s = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int kvh = h / p.group, hg = h % p.group;
  const int unit = kvh * p.blocks + hg / (8 * NB), hd = hg % (8 * NB);
  const int c0 = p.cum[s], places = p.cum[s + 1] - c0, all = p.cum[p.S];
  if (places == 0) return;
  const long long total = (long long)all * p.units;
  const long long xa = (long long)c0 * p.units + (long long)unit * places, xb = xa + places - 1;
  const int ca = int(((xa + 1) * p.ctas - 1) / total), cb = int((xb * p.ctas - 1) / total);
  if (ca == cb) return;                     // a whole unit in one stretch
  const size_t slot = 8 * NB * (D + 2);
  const int run = threadIdx.x / kCols, dd = (threadIdx.x % kCols) * 4;
  // CTAs ca .. cb hold one piece each (those whose stretch is empty, none); only
  // the first may have begun before xa, and then holds it in its second slot
  float m = kNegInf, l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = ca + run; c <= cb; c += kRuns) {
    const long long x0 = dec_cut(total, p.ctas, c), x1 = dec_cut(total, p.ctas, c + 1);
    const float* x = p.part + (size_t(c) * 2 + (x0 >= xa ? 0 : 1)) * slot;
    if (x0 == x1) continue;
    const float pm = x[hd], pl = x[8 * NB + hd];
    const float4 b = *reinterpret_cast<const float4*>(x + 16 * NB + hd * D + dd);
    const float m_new = fmaxf(m, pm), shift = m_new == kNegInf ? 0.f : m_new;
    const float f = ex2(m - shift), g = ex2(pm - shift);
    m = m_new;
    l = fmaf(l, f, pl * g);
    a.x = fmaf(a.x, f, b.x * g);
    a.y = fmaf(a.y, f, b.y * g);
    a.z = fmaf(a.z, f, b.z * g);
    a.w = fmaf(a.w, f, b.w * g);
  }
  acc[threadIdx.x] = a;
  if (dd == 0) {
    run_m[run] = m;
    run_l[run] = l;
  }
  __syncthreads();
  if (run != 0) return;
  float top = run_m[0];
#pragma unroll
  for (int r = 1; r < kRuns; ++r) top = fmaxf(top, run_m[r]);
  const float shift = top == kNegInf ? 0.f : top;
  float sum = 0.f;
  a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const float f = ex2(run_m[r] - shift);
    const float4 b = acc[threadIdx.x + r * kCols];
    sum = fmaf(run_l[r], f, sum);
    a.x = fmaf(b.x, f, a.x);
    a.y = fmaf(b.y, f, a.y);
    a.z = fmaf(b.z, f, a.z);
    a.w = fmaf(b.w, f, a.w);
  }
  const float inv = 1.f / sum;
  uint2 r;
  r.x = E::pack(a.x * inv, a.y * inv);
  r.y = E::pack(a.z * inv, a.w * inv);
  *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + (size_t(s) * p.H + h) * D + dd) = r;
  if (threadIdx.x == 0) p.lse[size_t(s) * p.H + h] = (top + lg2(sum)) * kLn2;
}

}  // namespace fa
