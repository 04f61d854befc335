// fa_cache.cu - the C ABI declared in include/fa_b200_cache.h: argument
// checks, tensor maps and launches of the paged-cache kernels.
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/fa_b200_cache.h"
#include "fa_cache.cuh"
#include "fa_decode.cuh"
#include "fa_host.h"

namespace fa {
namespace {

constexpr int kMaxDevices = 64;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_cache(int S, int Hkv, int d, int P, int page, int M) {
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (Hkv < 1) return FA_ERR_SHAPE;
  if (S < 1 || S > kCacheMaxSeqs || P < 1 || M < 1 || page < 8 || page > 32768 || page % 8) return FA_ERR_CACHE_SHAPE;
  constexpr long long kLimit = 1ll << 31;
  // each product is checked before the next factor can overflow it
  if ((long long)M * page >= kLimit || (long long)M * page * S >= kLimit) return FA_ERR_CACHE_SHAPE;
  if ((long long)P * Hkv >= kLimit || (long long)P * Hkv * page >= kLimit) return FA_ERR_CACHE_SHAPE;
  return FA_OK;
}

CacheParams cache_params(void* k_pages, void* v_pages, int32_t* refs, int32_t* table, int32_t* lens, int* dev_error,
                         int S, int P, int page, int M, int L, int Hkv, int d) {
  CacheParams p{};
  p.k_pages = static_cast<uint4*>(k_pages);
  p.v_pages = static_cast<uint4*>(v_pages);
  p.refs = refs;
  p.table = table;
  p.lens = lens;
  p.dev_error = dev_error;
  p.S = S;
  p.P = P;
  p.page = page;
  p.M = M;
  p.L = L;
  p.hkv = Hkv;
  p.row_log2 = d == 64 ? 3 : 4;
  return p;
}

// Large shared memory for the kernels that may need it, once per device.
struct Setup {
  std::once_flag once;
  bool ok = false;
};
Setup g_setup[kMaxDevices];

template <int D, int NB>
size_t decode_smem_most() {
  return DecLayout<D, NB>::bytes(kCacheMaxSeqs);
}
constexpr int kForkSmemMost = kCacheMaxSeqs * 8 + kCacheMaxSeqs / 8;

bool setup_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  Setup* st = &g_setup[dev];
  std::call_once(st->once, [st] {
    auto large = [](auto kernel, size_t smem) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) == cudaSuccess;
    };
    st->ok = large(fa_decode_kernel<64, 1, ElemBF16>, decode_smem_most<64, 1>()) &&
             large(fa_decode_kernel<64, 2, ElemBF16>, decode_smem_most<64, 2>()) &&
             large(fa_decode_kernel<128, 1, ElemBF16>, decode_smem_most<128, 1>()) &&
             large(fa_decode_kernel<128, 2, ElemBF16>, decode_smem_most<128, 2>()) &&
             large(fa_decode_kernel<64, 1, ElemF16>, decode_smem_most<64, 1>()) &&
             large(fa_decode_kernel<64, 2, ElemF16>, decode_smem_most<64, 2>()) &&
             large(fa_decode_kernel<128, 1, ElemF16>, decode_smem_most<128, 1>()) &&
             large(fa_decode_kernel<128, 2, ElemF16>, decode_smem_most<128, 2>()) &&
             large(fa_cache_fork_plan_kernel, kForkSmemMost);
  });
  return st->ok;
}

// Blocks of 8 query heads that a CTA takes together: 2 where a key/value head
// serves more than 8 query heads (more would not fit the registers).
int decode_nb(int group) { return group > 8 ? 2 : 1; }

template <int D, int NB, typename E>
int launch_decode(const void* k_pages, const void* v_pages, DecodeParams prm, int Hkv, cudaStream_t stream) {
  CUtensorMap mk, mv;
  // one layer of the cache: (d, token of the page, page and head), boxes of 64 x box
  constexpr CUtensorMapDataType dt = map_type<E>();
  if (!make_map(&mk, k_pages, prm.P * Hkv, prm.page, D, dt, prm.box) ||
      !make_map(&mv, v_pages, prm.P * Hkv, prm.page, D, dt, prm.box))
    return FA_ERR_DEVICE;
  if (launch(fa_decode_kernel<D, NB, E>, dim3(prm.ctas), dim3(DecLayout<D, NB>::kThreads),
             DecLayout<D, NB>::bytes(prm.S), stream, mk, mv, prm) != cudaSuccess)
    return FA_ERR_LAUNCH;
  if (!prm.whole &&
      launch(fa_decode_join_kernel<D, NB, E>, dim3(prm.S * prm.H), dim3(128), 0, stream, prm) != cudaSuccess)
    return FA_ERR_LAUNCH;
  return FA_OK;
}

size_t page_workspace(int S, int P) { return align256(size_t(P) * 12) + align256(size_t(S) * sizeof(ForkPlan)) + 256; }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_decode_workspace_size(int S, int H, int Hkv, int d) {
  if ((d != 64 && d != 128) || S < 1 || S > kCacheMaxSeqs || Hkv < 1 || H < Hkv || H % Hkv) return 0;
  const int nb = decode_nb(H / Hkv);
  return align256((size_t(S) + 1) * 4) + size_t(2 * kDecMaxCtas) * 8 * nb * (d + 2) * sizeof(float);
}

int fa_decode(const void* q, const void* k_pages, const void* v_pages, const int32_t* table, const int32_t* lens,
              void* o, float* lse, void* workspace, size_t workspace_bytes, int S, int H, int Hkv, int d, int P,
              int page, int M, long long q_stride, int window, int sinks, float scale, int elem, void* stream) {
  if (!q || !k_pages || !v_pages || !table || !lens || !o || !lse) return FA_ERR_NULL;
  int rc = check_cache(S, Hkv, d, P, page, M);
  if (rc != FA_OK) return rc;
  if (H < Hkv || H % Hkv || (long long)S * H * d >= (1ll << 31)) return FA_ERR_SHAPE;
  if (q_stride < (long long)H * d || q_stride % 8 || q_stride >= (1ll << 31) || window < 0 || sinks < 0 ||
      (window == 0 && sinks != 0))
    return FA_ERR_CACHE_SHAPE;
  // the kernel counts the tiles of one sequence, over all its heads, and of one CTA in 32 bits
  const long long tiles = ((long long)M * page / 64 + 2) * H;
  if (tiles >= (1ll << 31) || tiles * S >= (1ll << 38)) return FA_ERR_CACHE_SHAPE;
  if (!std::isfinite(scale) || !(scale > 0.f) || (elem != FA_ELEM_BF16 && elem != FA_ELEM_F16)) return FA_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) || !aligned4(table) ||
      !aligned4(lens) || !aligned4(lse))
    return FA_ERR_ALIGN;
  if (!workspace || !aligned16(workspace) || workspace_bytes < fa_decode_workspace_size(S, H, Hkv, d))
    return FA_ERR_WORKSPACE;
  DecodeParams prm{};
  int num_sms = 0;
  if ((rc = host_device(&num_sms, &prm.dev_error)) != FA_OK) return rc;
  if (!setup_device()) return FA_ERR_DEVICE;
  const int nb = decode_nb(H / Hkv);
  prm.q = q;
  prm.table = table;
  prm.lens = lens;
  prm.o = o;
  prm.lse = lse;
  prm.cum = static_cast<int32_t*>(workspace);
  prm.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256((size_t(S) + 1) * 4));
  prm.q_stride = q_stride;
  prm.S = S;
  prm.H = H;
  prm.group = H / Hkv;
  prm.blocks = (prm.group + 8 * nb - 1) / (8 * nb);
  prm.units = Hkv * prm.blocks;
  prm.P = P;
  prm.page = page;
  prm.M = M;
  const int tile = dec_tile(d);
  prm.box = tile;
  while (page % prm.box) prm.box /= 2;                    // 8 at least
  prm.z_none = P * Hkv;
  prm.window = window;
  prm.sinks = sinks;
  // two CTAs per SM, or one per place where there are fewer
  const long long places = ((long long)M * page + tile - 1) / tile + 1;      // of a unit, at most
  const long long most = (long long)S * prm.units * places;
  const int two = 2 * num_sms < kDecMaxCtas ? 2 * num_sms : kDecMaxCtas;
  prm.ctas = int(most < two ? most : two);
  // The second launch costs 2 to 3 us, a tile more on a CTA's way 0.7 us: units are
  // left whole where a table has room for up to 2 tiles (16 sequences of 2, H = 32
  // over Hkv = 8, d = 128: 8.3 us, cut 10.5), or 4 where there are as many units as
  // SMs (64 sequences: 16.8 us, cut 20.0; but 1 sequence of 4: 8.1, cut 7.6).
  prm.whole = places - 1 <= 2 || (places - 1 <= 4 && (long long)S * prm.units >= num_sms);
  prm.scale_log2 = float(double(scale) * 1.4426950408889634);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
#define FA_DECODE(D, NB) \
  (elem == FA_ELEM_BF16 ? launch_decode<D, NB, ElemBF16>(k_pages, v_pages, prm, Hkv, s) \
                        : launch_decode<D, NB, ElemF16>(k_pages, v_pages, prm, Hkv, s))
  if (d == 64) return nb == 1 ? FA_DECODE(64, 1) : FA_DECODE(64, 2);
  return nb == 1 ? FA_DECODE(128, 1) : FA_DECODE(128, 2);
#undef FA_DECODE
}

int fa_cache_append(const void* k, const void* v, void* k_pages, void* v_pages, const int32_t* table,
                    const int32_t* lens, const int32_t* cu, int T, int S, int Hkv, int d, int P, int page, int M,
                    long long k_stride, long long v_stride, void* stream) {
  if (!k || !v || !k_pages || !v_pages || !table || !lens) return FA_ERR_NULL;
  int rc = check_cache(S, Hkv, d, P, page, M);
  if (rc != FA_OK) return rc;
  const long long row = (long long)Hkv * d;
  if (T < 0 || (!cu && T != S) || k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8 ||
      k_stride >= (1ll << 31) || v_stride >= (1ll << 31))
    return FA_ERR_CACHE_SHAPE;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned4(table) ||
      !aligned4(lens) || !aligned4(cu))
    return FA_ERR_ALIGN;
  AppendParams a{};
  int num_sms = 0, *dev_error = nullptr;
  if ((rc = host_device(&num_sms, &dev_error)) != FA_OK) return rc;
  if (T == 0) return FA_OK;
  a.c = cache_params(k_pages, v_pages, nullptr, const_cast<int32_t*>(table), const_cast<int32_t*>(lens), dev_error, S,
                     P, page, M, 1, Hkv, d);
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.cu = cu;
  a.k_stride = k_stride / 8;
  a.v_stride = v_stride / 8;
  a.T = T;
  return launch(fa_cache_append_kernel, dim3(T / 8 + (T % 8 != 0)), dim3(256), 0,
                static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

size_t fa_cache_workspace_size(int S, int P) {
  if (S < 1 || S > kCacheMaxSeqs || P < 1) return 0;
  return page_workspace(S, P);
}

int fa_cache_reserve(int32_t* refs, int32_t* table, int32_t* lens, const int32_t* add, int32_t* missing, int S, int P,
                     int page, int M, void* stream) {
  if (!refs || !table || !lens || !add || !missing) return FA_ERR_NULL;
  int rc = check_cache(S, 1, 64, P, page, M);
  if (rc != FA_OK) return rc;
  if (!aligned16(refs) || !aligned4(table) || !aligned4(lens) || !aligned4(add) || !aligned4(missing))
    return FA_ERR_ALIGN;
  int num_sms = 0, *dev_error = nullptr;
  if ((rc = host_device(&num_sms, &dev_error)) != FA_OK) return rc;
  const CacheParams p = cache_params(nullptr, nullptr, refs, table, lens, dev_error, S, P, page, M, 1, 1, 64);
  return launch(fa_cache_reserve_kernel, dim3(1), dim3(kPlanThreads), size_t(S) * 4,
                static_cast<cudaStream_t>(stream), p, add, missing) == cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

int fa_cache_fork(void* k_pages, void* v_pages, int32_t* refs, int32_t* table, int32_t* lens, const int32_t* src,
                  const int32_t* dst, int32_t* missing, void* workspace, size_t workspace_bytes, int F, int L, int S,
                  int Hkv, int d, int P, int page, int M, void* stream) {
  if (!k_pages || !v_pages || !refs || !table || !lens || !src || !dst || !missing) return FA_ERR_NULL;
  int rc = check_cache(S, Hkv, d, P, page, M);
  if (rc != FA_OK) return rc;
  if (F < 1 || F > S || L < 1) return FA_ERR_CACHE_SHAPE;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(refs) || !aligned4(table) || !aligned4(lens) ||
      !aligned4(src) || !aligned4(dst) || !aligned4(missing))
    return FA_ERR_ALIGN;
  if (!workspace || !aligned16(workspace) || workspace_bytes < page_workspace(S, P)) return FA_ERR_WORKSPACE;
  int num_sms = 0, *dev_error = nullptr;
  if ((rc = host_device(&num_sms, &dev_error)) != FA_OK) return rc;
  if (!setup_device()) return FA_ERR_DEVICE;
  const CacheParams p = cache_params(k_pages, v_pages, refs, table, lens, dev_error, S, P, page, M, L, Hkv, d);
  int32_t* plan_n = static_cast<int32_t*>(workspace);
  ForkPlan* plan = reinterpret_cast<ForkPlan*>(static_cast<uint8_t*>(workspace) + 256);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = size_t(F) * 8 + (size_t(S) + 31) / 32 * 4;
  if (launch(fa_cache_fork_plan_kernel, dim3(1), dim3(kPlanThreads), smem, s, p, src, dst, F, plan, plan_n,
             missing) != cudaSuccess)
    return FA_ERR_LAUNCH;
  if (launch(fa_cache_fork_copy_kernel, dim3(F, L < 64 ? L : 64), dim3(256), 0, s, p,
             static_cast<const ForkPlan*>(plan), static_cast<const int32_t*>(plan_n)) != cudaSuccess)
    return FA_ERR_LAUNCH;
  return FA_OK;
}

int fa_cache_free(int32_t* refs, int32_t* table, int32_t* lens, const int32_t* seqs, int F, int S, int P, int page,
                  int M, void* stream) {
  if (!refs || !table || !lens || !seqs) return FA_ERR_NULL;
  int rc = check_cache(S, 1, 64, P, page, M);
  if (rc != FA_OK) return rc;
  if (F < 1 || F > S) return FA_ERR_CACHE_SHAPE;
  if (!aligned16(refs) || !aligned4(table) || !aligned4(lens) || !aligned4(seqs)) return FA_ERR_ALIGN;
  int num_sms = 0, *dev_error = nullptr;
  if ((rc = host_device(&num_sms, &dev_error)) != FA_OK) return rc;
  const CacheParams p = cache_params(nullptr, nullptr, refs, table, lens, dev_error, S, P, page, M, 1, 1, 64);
  return launch(fa_cache_free_kernel, dim3(F), dim3(256), 0, static_cast<cudaStream_t>(stream), p, seqs) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

int fa_cache_compact(void* k_pages, void* v_pages, int32_t* refs, int32_t* table, const int32_t* lens, int32_t* live,
                     void* workspace, size_t workspace_bytes, int L, int S, int Hkv, int d, int P, int page, int M,
                     void* stream) {
  if (!k_pages || !v_pages || !refs || !table || !lens || !live) return FA_ERR_NULL;
  int rc = check_cache(S, Hkv, d, P, page, M);
  if (rc != FA_OK) return rc;
  if (L < 1) return FA_ERR_CACHE_SHAPE;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(refs) || !aligned4(table) || !aligned4(lens) ||
      !aligned4(live))
    return FA_ERR_ALIGN;
  if (!workspace || !aligned16(workspace) || workspace_bytes < page_workspace(S, P)) return FA_ERR_WORKSPACE;
  int num_sms = 0, *dev_error = nullptr;
  if ((rc = host_device(&num_sms, &dev_error)) != FA_OK) return rc;
  const CacheParams p = cache_params(k_pages, v_pages, refs, table, const_cast<int32_t*>(lens), dev_error, S, P, page,
                                     M, L, Hkv, d);
  int32_t* moves = static_cast<int32_t*>(workspace);
  int32_t* from = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + 256);
  int32_t *to = from + P, *went = to + P;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch(fa_cache_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, live, moves, from, to, went) !=
      cudaSuccess)
    return FA_ERR_LAUNCH;
  if (launch(fa_cache_compact_copy_kernel, dim3(8 * num_sms), dim3(256), 0, s, p, static_cast<const int32_t*>(live),
             static_cast<const int32_t*>(moves), static_cast<const int32_t*>(from), static_cast<const int32_t*>(to),
             static_cast<const int32_t*>(went)) != cudaSuccess)
    return FA_ERR_LAUNCH;
  return FA_OK;
}

}  // extern "C"
