// fa_window.cu - the C ABI declared in include/fa_b200_window.h: argument
// checks, tensor maps and launches of the windowed forward and backward.
#include <cstdint>
#include <mutex>

#include "../../include/fa_b200_window.h"
#include "fa_bwd.cuh"
#include "fa_fwd.cuh"
#include "fa_host.h"
#include "fa_window_pre.cuh"

namespace fa {
namespace {

constexpr int kMaxDevices = 64;

struct Setup {
  std::once_flag once;
  int status = FA_ERR_DEVICE;
};
Setup g_setup[kMaxDevices];

// Large shared memory and the register count at launch that the kernels'
// register split assumes, once per device.
int setup_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_DEVICE;
  Setup* st = &g_setup[dev];
  std::call_once(st->once, [st] {
    bool ok = true, regs_ok = true;
    auto setup = [&](auto kernel, int smem, int regs) {
      cudaFuncAttributes a{};
      ok &= cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
      ok &= cudaFuncGetAttributes(&a, kernel) == cudaSuccess;
      regs_ok &= a.numRegs == regs;
    };
    auto both = [&](auto elem) {
      using E = decltype(elem);
      setup(fa_fwd_kernel<64, false, E, 1>, FwdLayout<64>::kAlloc, FwdLayout<64>::kLaunchRegs);
      setup(fa_fwd_kernel<64, true, E, 1>, FwdLayout<64>::kAlloc, FwdLayout<64>::kLaunchRegs);
      setup(fa_fwd_kernel<64, false, E, 2>, FwdLayout<64>::kAlloc, FwdLayout<64>::kLaunchRegs);
      setup(fa_fwd_kernel<128, false, E, 1>, FwdLayout<128>::kAlloc, FwdLayout<128>::kLaunchRegs);
      setup(fa_fwd_kernel<128, true, E, 1>, FwdLayout<128>::kAlloc, FwdLayout<128>::kLaunchRegs);
      setup(fa_fwd_kernel<128, false, E, 2>, FwdLayout<128>::kAlloc, FwdLayout<128>::kLaunchRegs);
      setup(fa_bwd_kernel<64, E, false, 1>, BwdLayout<64>::kAlloc, BwdLayout<64>::kLaunchRegs);
      setup(fa_bwd_kernel<128, E, false, 1>, BwdLayout<128>::kAlloc, BwdLayout<128>::kLaunchRegs);
      setup(fa_bwd_kernel<64, E, false, 2>, BwdLayout<64>::kAlloc, BwdLayout<64>::kLaunchRegs);
      setup(fa_bwd_kernel<128, E, false, 2>, BwdLayout<128>::kAlloc, BwdLayout<128>::kLaunchRegs);
    };
    both(ElemBF16{});
    both(ElemF16{});
    st->status = !ok ? FA_ERR_DEVICE : !regs_ok ? FA_ERR_BUILD : FA_OK;
  });
  return st->status;
}

int check_window(int B, int H, int Hkv, int N, int d, int window, int sinks, float scale) {
  int rc = check_common(B, H, N, d, 1, scale);
  if (rc != FA_OK) return rc;
  if ((rc = check_heads(H, Hkv)) != FA_OK) return rc;
  return window >= 1 && sinks >= 0 ? FA_OK : FA_ERR_WINDOW;
}

// How the backward cuts its work (BwdPieces), and where its workspace keeps what.
// It goes by the sizes alone, so that the sums do not depend on the device.
struct BwdPlan {
  int window, sinks;
  BwdPieces pc;
  long long n_items;
  size_t dsum, near, far, bytes;   // offsets; the dQ accumulator is at 0
};

BwdPlan bwd_plan(int B, int H, int Hkv, int N, int d, int window, int sinks) {
  BwdPlan w{};
  w.window = window < N ? window : N;
  w.sinks = sinks < N ? sinks : N;
  BwdPieces& pc = w.pc;
  pc.n_q = (N + 127) / 128;
  pc.near = (126 + w.window) / 128 + 1;
  if (pc.near > pc.n_q) pc.near = pc.n_q;
  pc.far_from = pc.near;
  pc.group = H / Hkv;
  const int far = pc.n_q - pc.near, sink_tiles = (w.sinks + 127) / 128;
  pc.split = sink_tiles < far ? sink_tiles : far;
  pc.far_rows = w.sinks < 128 * pc.split ? w.sinks : 128 * pc.split;
  // steps of all items; a third of a CTA's share of them, but four at least (an item
  // loads K and V and writes its sums, about two steps' time), or where a CTA's
  // share is smaller that, but two (8 heads over 2, N = 1024, d = 128, window 256:
  // backward 27.9 us with four, 24.3 with two; 2 heads, N = 4096, d = 64, window 300:
  // 20.0 and 19.4, with two in any case 25.2)
  const long long BHkv = (long long)B * Hkv;
  const long long near_steps = (long long)pc.n_q * pc.near - (long long)pc.near * (pc.near - 1) / 2;
  const long long far_steps = (long long)pc.split * far - (long long)pc.split * (pc.split - 1) / 2;
  const long long steps = (near_steps + far_steps) * BHkv * pc.group;
  const long long share = (steps + 3 * 148 - 1) / (3 * 148), whole = (steps + 147) / 148;
  const int least = whole < 2 ? 2 : whole < 4 ? int(whole) : 4;
  const long long item = share > least ? share : least;
  pc.near_parts = int(((long long)pc.near * pc.group + item - 1) / item);
  // far parts about as long as the others: every CTA takes as many items
  const int part = pc.near * pc.group / pc.near_parts, far_item = part > least ? part : least;
  const long long far_len = (long long)far * pc.group;
  pc.far_parts = !pc.split ? 0 : far_len < far_item ? 1 : int((far_len + far_item / 2) / far_item);
  // A window and a far part that are one part each are one item where that is at
  // most two thirds of a CTA's share: no sums, K and V loaded once (8 x 12 heads of
  // 1024 tokens, d = 64, window 256: backward 84.8 us apart, 79.6 as one item; 4 x
  // 12 heads 47.6, as one item 49.2.  Far parts of any length as one item: 4 x 12
  // heads of 8192 tokens, window 1024, 508 us apart, 564).
  if (pc.near_parts == 1 && pc.far_parts == 1 && 3ll * (pc.near + far) * pc.group <= 2 * whole) {
    pc.near_first = pc.split;
    pc.split = pc.far_rows = pc.far_from = 0;
  }
  pc.gaps = pc.near_parts > pc.group || (pc.split && pc.far_parts > (far - pc.split + 1) * pc.group);
  pc.by_heads = FastDiv(int(BHkv));
  pc.by_tiles = FastDiv(pc.n_q - pc.near_first > 0 ? pc.n_q - pc.near_first : 1);
  pc.by_near = FastDiv(pc.near_parts);
  pc.by_far = FastDiv(pc.far_parts ? pc.far_parts : 1);
  w.n_items = BHkv * ((long long)(pc.n_q - pc.near_first) * pc.near_parts +
                      (long long)(pc.split + pc.near_first) * pc.far_parts);
  const size_t rows = size_t(B) * H * N, row = size_t(2) * d * sizeof(float);
  w.dsum = align256(rows * d * sizeof(float));
  w.near = w.dsum + align256(rows * sizeof(float));
  w.far = w.near + (pc.near_parts > 1 ? align256(size_t(BHkv) * pc.near_parts * N * row) : 0);
  w.bytes = w.far + (pc.split ? align256(size_t(BHkv) * (1 + pc.far_parts) * pc.far_rows * row) : 0);
  return w;
}

template <int D, typename E>
int window_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Hkv, int N,
               int window, int sinks, float scale, int fix_mode, int num_sms, int* dev_error, cudaStream_t stream) {
  using L = FwdLayout<D>;
  constexpr CUtensorMapDataType dt = map_type<E>();
  CUtensorMap mq, mk, mv, mo;
  if (!make_map(&mq, q, B * H, N, D, dt) || !make_map(&mk, k, B * Hkv, N, D, dt) ||
      !make_map(&mv, v, B * Hkv, N, D, dt) || !make_map(&mo, o, B * H, N, D, dt, 32))
    return FA_ERR_DEVICE;
  FwdParams p{};
  p.o = o;
  p.lse = lse;
  p.dev_error = dev_error;
  p.BH = B * H;
  p.N = N;
  // Two query tiles per CTA keep it busy, but a step of both takes longer than one
  // of one: where there are CTAs for all tiles each has its own (8 heads over 2,
  // N = 1024, d = 128, window 256: 15.7 us in pairs, 12.5 one by one; 1 head,
  // N = 16384, window 4096: 72 and 63).  The results are the same bits.
  p.item_log2 = (long long)((N + 127) / 128) * B * H <= num_sms ? 7 : 8;
  p.n_pairs = (N + (1 << p.item_log2) - 1) >> p.item_log2;
  p.causal = 1;
  p.H = H;
  p.group = H / Hkv;
  p.scale_log2 = float(double(scale) * 1.4426950408889634);
  set_fix(p, fix_mode, E::kMmaFmt == 0);
  p.window = window < N ? window : N;
  p.sinks = sinks < N ? sinks : N;
  const int n_items = p.n_pairs * p.BH;
  auto kern = fix_mode == 1  ? fa_fwd_kernel<D, false, E, 2>
              : fix_mode == 0 ? fa_fwd_kernel<D, false, E, 1>
                              : fa_fwd_kernel<D, true, E, 1>;
  return launch(kern, dim3(n_items < num_sms ? n_items : num_sms), dim3(L::kThreads), L::kAlloc, stream, mq, mk, mv,
                mo, p) == cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

template <int D, typename E>
int window_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
               void* dq, void* dk, void* dv, uint8_t* workspace, const BwdPlan& w, int B, int H, int Hkv, int N,
               float scale, int num_sms, int* dev_error, cudaStream_t stream) {
  using L = BwdLayout<D>;
  using T = typename E::T;
  constexpr CUtensorMapDataType dt = map_type<E>();
  const int BH = B * H, BHkv = B * Hkv;
  CUtensorMap mq, mk, mv, mdo, mdq, mdk, mdv;
  if (!make_map(&mq, q, BH, N, D, dt) || !make_map(&mk, k, BHkv, N, D, dt) || !make_map(&mv, v, BHkv, N, D, dt) ||
      !make_map(&mdo, dout, BH, N, D, dt) || !make_map_dq(&mdq, workspace, BH, N, D) ||
      !make_map(&mdk, dk, BHkv, N, D, dt, 32) || !make_map(&mdv, dv, BHkv, N, D, dt, 32))
    return FA_ERR_DEVICE;
  float* dq_acc = reinterpret_cast<float*>(workspace);
  float* dsum = reinterpret_cast<float*>(workspace + w.dsum);
  float* near_part = reinterpret_cast<float*>(workspace + w.near);
  float* far_part = reinterpret_cast<float*>(workspace + w.far);
  const long long rows = (long long)BH * N;
  const float scale_log2 = float(double(scale) * 1.4426950408889634);
  const int few = w.window + (long long)w.sinks <= kFewKeys || N < kFewKeys ? N : kFewKeys;
  const unsigned few_blocks = unsigned(((long long)BH * few + 7) / 8);
  // One query tile per head (N <= 128) has one step, and no sum: the main kernel
  // writes dQ itself, and where dK and dV are whole too there is no last launch
  // (2 x 16 heads over 8 of 100 tokens, d = 64: backward 10.7 -> 9.4 us; 4 x 8 over 1
  // of 60: 14.7 -> 12.3).
  const bool whole_dq = w.pc.n_q == 1;
  const BwdPreParams pre{lse,      dsum,    whole_dq ? nullptr : dq_acc, rows, N, H, H / Hkv,
                         w.window, w.sinks, few, few_blocks, scale_log2};
  if (launch(fa_bwd_window_pre_kernel<D, E>, dim3(few_blocks + unsigned((rows * 8 + 255) / 256)), dim3(256), 0, stream,
             static_cast<const T*>(o), static_cast<const T*>(dout), static_cast<const T*>(q),
             static_cast<const T*>(k), static_cast<const T*>(v), pre) != cudaSuccess)
    return FA_ERR_LAUNCH;
  BwdWindowParams p{};
  p.lse = lse;
  p.dsum = dsum;
  p.dq_acc = dq_acc;
  p.dk = dk;
  p.dv = dv;
  p.dev_error = dev_error;
  p.BH = BHkv;
  p.H = H;
  p.group = H / Hkv;
  p.N = N;
  p.n_kv = (N + 127) / 128;
  p.causal = 1;
  p.scale = scale;
  p.scale_log2 = scale_log2;
  p.after_pre = 1;
  p.window = w.window;
  p.sinks = w.sinks;
  p.pc = w.pc;
  p.near_part = near_part;
  p.far_part = far_part;
  p.dq = dq;
  if (launch(whole_dq ? fa_bwd_kernel<D, E, false, 2> : fa_bwd_kernel<D, E, false, 1>,
             dim3(unsigned(w.n_items < num_sms ? w.n_items : num_sms)), dim3(L::kThreads), L::kAlloc, stream, mq, mk,
             mv, mdo, mdq, mdk, mdv, p) != cudaSuccess)
    return FA_ERR_LAUNCH;
  const long long n8 = whole_dq ? 0 : rows * D / 8;
  const unsigned dq_blocks = unsigned((n8 + 255) / 256);
  const int part_rows = w.pc.near_parts > 1 ? N : w.pc.far_rows;
  const long long part_items = (long long)BHkv * part_rows * (D / 2);
  const unsigned blocks = dq_blocks + unsigned((part_items + 255) / 256);
  if (blocks == 0) return FA_OK;
  if (launch(fa_bwd_window_finish_kernel<E>, dim3(blocks), dim3(256), 0,
             stream, static_cast<const float*>(dq_acc), static_cast<T*>(dq), scale, n8, dq_blocks,
             static_cast<const float*>(near_part), static_cast<const float*>(far_part), static_cast<T*>(dk),
             static_cast<T*>(dv), w.pc, part_rows, N, D, part_items) != cudaSuccess)
    return FA_ERR_LAUNCH;
  return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_window_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Hkv, int N,
                  int d, int window, int sinks, float scale, int fix_mode, int elem, void* stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
  int rc = check_window(B, H, Hkv, N, d, window, sinks, scale);
  if (rc != FA_OK) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_ALIGN;
  if (fix_mode < 0 || fix_mode > 5) return FA_ERR_FIXMODE;
  if (elem != FA_ELEM_BF16 && elem != FA_ELEM_F16) return FA_ERR_ARG;
  int num_sms = 0, *dev_error = nullptr;
  if ((rc = host_device(&num_sms, &dev_error)) != FA_OK || (rc = setup_device()) != FA_OK) return rc;
  auto run = [&](auto fn) {
    return fn(q, k, v, o, lse, B, H, Hkv, N, window, sinks, scale, fix_mode, num_sms, dev_error,
              static_cast<cudaStream_t>(stream));
  };
  if (elem == FA_ELEM_BF16) return run(d == 64 ? window_fwd<64, ElemBF16> : window_fwd<128, ElemBF16>);
  return run(d == 64 ? window_fwd<64, ElemF16> : window_fwd<128, ElemF16>);
}

size_t fa_window_bwd_workspace_size(int B, int H, int Hkv, int N, int d, int window, int sinks) {
  if (check_window(B, H, Hkv, N, d, window, sinks, 1.f) != FA_OK) return 0;
  return bwd_plan(B, H, Hkv, N, d, window, sinks).bytes;
}

int fa_window_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                  void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int N,
                  int d, int window, int sinks, float scale, int elem, void* stream) {
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv) return FA_ERR_NULL;
  int rc = check_window(B, H, Hkv, N, d, window, sinks, scale);
  if (rc != FA_OK) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv))
    return FA_ERR_ALIGN;
  if (elem != FA_ELEM_BF16 && elem != FA_ELEM_F16) return FA_ERR_ARG;
  const BwdPlan w = bwd_plan(B, H, Hkv, N, d, window, sinks);
  if (!workspace || !aligned16(workspace) || workspace_bytes < w.bytes) return FA_ERR_WORKSPACE;
  int num_sms = 0, *dev_error = nullptr;
  if ((rc = host_device(&num_sms, &dev_error)) != FA_OK || (rc = setup_device()) != FA_OK) return rc;
  auto run = [&](auto fn) {
    return fn(q, k, v, o, lse, dout, dq, dk, dv, static_cast<uint8_t*>(workspace), w, B, H, Hkv, N, scale, num_sms,
              dev_error, static_cast<cudaStream_t>(stream));
  };
  if (elem == FA_ELEM_BF16) return run(d == 64 ? window_bwd<64, ElemBF16> : window_bwd<128, ElemBF16>);
  return run(d == 64 ? window_bwd<64, ElemF16> : window_bwd<128, ElemF16>);
}

}  // extern "C"
