/*
 * fa_b200_window.h - C ABI of attention behind a sliding window with sinks.
 * Part of libfa_b200.so; layouts, status codes, streams, ownership, fix_mode
 * and element formats are those of fa_b200.h.
 *
 * Query i sees key j where j <= i and (i - j < window or j < sinks): itself and
 * the window - 1 tokens before it, and the first `sinks` tokens of the sequence,
 * which trained models keep weight on ("attention sinks").  window >= 1,
 * sinks >= 0; both may be larger than N.  With window >= N this is causal
 * attention.  Work and memory traffic grow with N * (window + sinks), not N^2.
 * Inputs are finite: an infinity or NaN in one token of K or V reaches every
 * query whose 128-row tile sees that token's 128-key tile, as in fa_fwd.
 */
#ifndef FA_B200_WINDOW_H
#define FA_B200_WINDOW_H

#include "fa_b200.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further fa_status value. */
#define FA_ERR_WINDOW (-15)   /* window < 1 or sinks < 0 */

/*
 * fa_window_fwd - forward pass: fa_fwd_ex with the mask above.
 *   q, o : [B,H,N,d];  k, v : [B,Hkv,N,d], Hkv dividing H;  lse : float32 [B,H,N].
 *   fix_mode : 0, 2, 3, 4, 5 as in fa_fwd.  1, the fast one, applies the fix to
 *       every row: the shift stays above the running maximum, by 2^8 at most (in
 *       fp16 2^4), so that every exponential, the maxima included, is below 1
 *       whether or not the maximum is repeated; a maximum maps to 1 - 2^-8 (fp16
 *       1 - 2^-11) times a power of two where it set the shift.
 */
FA_API int fa_window_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Hkv,
                         int N, int d, int window, int sinks, float scale, int fix_mode, int elem, void* stream);

/*
 * fa_window_bwd - backward pass: fa_bwd_ex with the mask above (o and lse from
 * fa_window_fwd with the same window and sinks).  dK and dV of a shared head
 * are the sums over its query heads.
 *   workspace : device scratch, >= fa_window_bwd_workspace_size() bytes,
 *       16-byte aligned, contents on entry ignored; calls that may run at the
 *       same time need one each.  It holds the FP32 dQ accumulator and D of
 *       fa_bwd, and FP32 pieces of dK and dV that several CTAs sum.
 * D, the row sums of dO * O, is taken from the rounded o; in rows that see up to
 * 8 keys (the first 8 tokens, and every one where window + sinks <= 8) it is
 * recomputed from q, k, v and lse, where the rounding of o would be the largest
 * error, and a token that sees itself alone then has no gradient but dV.
 * dK and dV are the same bits from run to run; dQ is summed in an order that
 * varies, as in fa_bwd.
 */
FA_API size_t fa_window_bwd_workspace_size(int B, int H, int Hkv, int N, int d, int window, int sinks);
FA_API int fa_window_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                         const void* dout, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                         int B, int H, int Hkv, int N, int d, int window, int sinks, float scale, int elem,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_B200_WINDOW_H */
