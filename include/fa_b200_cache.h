/*
 * fa_b200_cache.h - C ABI of the paged key/value cache: attention of one new
 * token per sequence, writing tokens, and the page operators.
 * Part of libfa_b200.so; status codes, streams, ownership and element formats
 * are those of fa_b200.h.
 *
 * The cache
 *   k_pages, v_pages : bf16 or fp16 [P, Hkv, page, d], contiguous, device, one
 *       layer.  The page operators take all layers at once, [L, P, Hkv, page, d].
 *   table : int32 [S, M], contiguous, device.  Entry i of row s is the page
 *       that holds tokens i*page .. i*page + page - 1 of sequence s.
 *   lens  : int32 [S], device.  Tokens of each sequence; 0 = an empty slot.
 *       The first ceil(lens[s] / page) entries of a row are in use.
 *   refs  : int32 [P], device.  How many table entries name each page; 0 = free.
 * Tables, lengths and reference counts live on the device and every call is
 * asynchronous, so that a step can be captured into a CUDA graph and replayed
 * while they change.  Values found there are checked by the kernels: a page
 * number outside [0, P), a length outside [0, M*page] or a sequence index
 * outside [0, S) never leads to an access out of range; it is left out as
 * each call says, and fa_check_device_error() then reports FA_ERR_PAGES.
 * Pages are handed out lowest free number first, in the order of the request,
 * so that results do not depend on timing.
 *
 * Limits: d is 64 or 128; page is a multiple of 8, 8 .. 32768; 1 <= S <= 8192;
 * M, P >= 1; S*M*page and P*Hkv*page below 2^31 (FA_ERR_CACHE_SHAPE).  Base
 * addresses of element tensors, refs and workspaces are 16-byte aligned,
 * the other int32 and float arrays 4-byte aligned (FA_ERR_ALIGN).
 */
#ifndef FA_B200_CACHE_H
#define FA_B200_CACHE_H

#include "fa_b200.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further fa_status values. */
#define FA_ERR_PAGES (-13)       /* a kernel found a page number, length or index
                                    of the cache out of range (device flag)      */
#define FA_ERR_CACHE_SHAPE (-14) /* page size, P, M, S, L, token count, stride,
                                    window or sinks out of range                 */

/*
 * fa_decode - attention of one new token per sequence over the paged cache.
 *   q    in : [S, H, d], rows of H*d elements, q_stride elements from one
 *             sequence to the next (a multiple of 8, >= H*d).
 *   o   out : [S, H, d], contiguous.
 *   lse out : float32 [S, H], natural log.
 * The new token is the last one of its sequence: query s sits at position
 * lens[s] - 1, and its key and value are already in the cache (fa_cache_append).
 * It sees key j where j < lens[s] and, if window > 0,
 * lens[s] - 1 - j < window or j < sinks; window = 0 shows every key (sinks must
 * then be 0).  Query head h reads key/value head h / (H / Hkv).
 *   O = sum_j P_j V_j / sum_j P_j,  P_j = exp(scale q.K_j - m).
 * P enters the product as the sum of two values of the element format (its
 * rounding and the rest), so that no rounding of P reaches O; there is no
 * fix_mode because no P_bar is rounded to 1.
 * A sequence of length 0 gets O = 0 and LSE = -inf.  What lies in a page behind
 * the last token or outside the window is not used, whatever it is (infinities
 * and NaN included); pages with no visible token are not read and their table
 * entries not looked at.  A page number out of range among the visible tokens
 * counts as a page of zeros, a length out of range as the nearest in range;
 * both are reported.
 * Equal lens, shapes and inputs give equal bits; the split of the work, and so
 * the order of the sums, depends on the lengths of the whole batch.
 * H*M*page/64 below 2^31, S*H*M*page/64 below 2^38 (FA_ERR_CACHE_SHAPE).
 *   workspace : device scratch of fa_decode_workspace_size() bytes, used from
 *       the call until its kernels have run: calls that may run at the same
 *       time need one each.
 */
FA_API size_t fa_decode_workspace_size(int S, int H, int Hkv, int d);
FA_API int fa_decode(const void* q, const void* k_pages, const void* v_pages, const int32_t* table,
                     const int32_t* lens, void* o, float* lse, void* workspace, size_t workspace_bytes,
                     int S, int H, int Hkv, int d, int P, int page, int M, long long q_stride,
                     int window, int sinks, float scale, int elem, void* stream);

/*
 * fa_cache_append - writes the newest tokens of each sequence into their pages.
 *   k, v in : [T, Hkv, d], rows of Hkv*d elements of 16 bits, k_stride and
 *             v_stride elements from one token to the next (multiples of 8,
 *             >= Hkv*d: a slice of a fused projection is taken as it is).
 *   cu   in : int32 [S+1], non-decreasing: tokens cu[s] .. cu[s+1]-1 are the
 *             last ones of sequence s, so that its token t goes to position
 *             lens[s] - (cu[s+1] - t).  NULL: T == S, one token per sequence;
 *             a sequence of length 0 has none and its row is not used.
 * lens already counts the new tokens (fa_cache_reserve).  Tokens outside
 * [cu[0], cu[S]) are not used.  A token whose position or page is out of range
 * is not written, and is reported.  T >= 0.
 */
FA_API int fa_cache_append(const void* k, const void* v, void* k_pages, void* v_pages, const int32_t* table,
                           const int32_t* lens, const int32_t* cu, int T, int S, int Hkv, int d, int P,
                           int page, int M, long long k_stride, long long v_stride, void* stream);

/*
 * fa_cache_reserve - makes room: lens[s] += add[s], and each sequence gets the
 * pages that its new length needs, with reference count 1.
 *   add     in : int32 [S], >= 0.
 *   missing out: int32 [1], device.  0: done.  > 0: that many pages are
 *       missing; nothing was changed.  -1: a length or an entry of add is out
 *       of range (the new length too); nothing was changed, and it is reported.
 */
FA_API int fa_cache_reserve(int32_t* refs, int32_t* table, int32_t* lens, const int32_t* add, int32_t* missing,
                            int S, int P, int page, int M, void* stream);

/*
 * fa_cache_fork - sequence dst[f] becomes a copy of sequence src[f], f < F.
 * Full pages are shared (their counts rise by 1); the last page, if it is not
 * full, is copied to a free one, its used tokens in all layers, so that
 * appending to a sequence never writes into a page that another one reads.
 * (Lengths may be lowered by the caller only where no full page is shared.)
 *   src, dst in : int32 [F], 1 <= F <= S.  A source may appear several times.
 *       Every dst is an empty slot (lens 0), and appears once.
 *   missing out : as in fa_cache_reserve; -1 also for a src or dst out of
 *       range, a dst that is not empty or appears twice.
 * All lengths are read before any is changed.  A page number out of range in a
 * source's row is copied as it is, no page counted or read for it, and reported.
 *   workspace : fa_cache_workspace_size(S, P) bytes, as in fa_decode.
 */
FA_API size_t fa_cache_workspace_size(int S, int P);
FA_API int fa_cache_fork(void* k_pages, void* v_pages, int32_t* refs, int32_t* table, int32_t* lens,
                         const int32_t* src, const int32_t* dst, int32_t* missing, void* workspace,
                         size_t workspace_bytes, int F, int L, int S, int Hkv, int d, int P, int page, int M,
                         void* stream);

/*
 * fa_cache_free - ends the sequences seqs[f], f < F: the counts of their pages
 * fall by 1, the entries in use become -1 and the lengths 0.
 *   seqs in : int32 [F], 1 <= F <= S.  An index out of range is left out and
 *       reported; one that appears again, or whose slot is empty, has no effect.
 */
FA_API int fa_cache_free(int32_t* refs, int32_t* table, int32_t* lens, const int32_t* seqs, int F, int S, int P,
                         int page, int M, void* stream);

/*
 * fa_cache_compact - moves the pages in use to the numbers 0 .. live-1.
 * Pages already there stay; the k-th used page from live on (ascending) moves
 * to the k-th free page below live, in all layers, and tables and counts
 * follow.  The pages from live on are then free, and their contents unchanged.
 * An entry in use that names a free page, or a number out of range, becomes -1
 * (a page that moves could take its place) and is reported.  A length out of
 * range counts as the nearest in range, here and in fa_cache_free, and is
 * reported.
 *   live out  : int32 [1], device: the number of pages in use.
 *   workspace : fa_cache_workspace_size(S, P) bytes, as in fa_decode.
 */
FA_API int fa_cache_compact(void* k_pages, void* v_pages, int32_t* refs, int32_t* table, const int32_t* lens,
                            int32_t* live, void* workspace, size_t workspace_bytes, int L, int S, int Hkv, int d,
                            int P, int page, int M, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_B200_CACHE_H */
