"""The paged cache on the GPU against plain 64-bit statements (oracle/paged64.py).

Tolerances of decoding, from the arithmetic.  A score is a sum of d products in
FP32, off by at most 2^-23 (d + 8) times the size of its terms (`reach`, which
includes the scale); the exponent, its rounding and ex2 add 2^-22 (1 + reach),
so each P is off by the relative amount
    e = 2^-23 (d + 8) reach + 2^-22 (4 + 2 reach),
once in the numerator and once in the sum.  P enters the product as two values
of the element format: 2^-16 of it is lost at most (bf16, 2 * 8 bits; fp16 less,
but for P below 2^-14, whose second value is a subnormal: 2^-24 absolute, under
2^-16 of the largest term), and the FP32 sums over n keys add 2^-23 sqrt(n) or
less in either.  The output is rounded by half a step of its type:
    |O - O_ref| <= eps / 2 |O_ref| + (2 e + 2^-15) weight,
weight = sum_j P_j |V_j|.  LSE is off by e, and by its own rounding 2^-23 |LSE|.
"""
import numpy as np
import pytest
import torch

from oracle import paged64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
FA_ERR_PAGES = -13


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from flashattention_bf16_fwd_b200 import cache, fa as binding
    binding.cache = cache
    assert binding.fa_check_device_error() == 0
    return binding


def make(lens, Hkv, d, page, dt, seed, window=0, sinks=0, spare=3):
    """A cache in which everything that no query may use is NaN, and every table
    entry that no query may look at is -1."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lens]
    P, M = sum(held) + spare, max(held + [1]) + 1
    ids = torch.randperm(P, generator=g).tolist()
    table = torch.full((len(lens), M), -1, dtype=torch.int32)
    kp, vp = (torch.full((P, Hkv, page, d), float("nan"), dtype=dt) for _ in range(2))
    at = 0
    for s, n in enumerate(lens):
        seen = [j for j in range(n) if not window or n - 1 - j < window or j < sinks]
        for i in range(held[s]):
            if any(j // page == i for j in seen):
                table[s, i] = ids[at]
            at += 1
        for j in seen:
            for pool in (kp, vp):
                pool[table[s, j // page], :, j % page] = torch.randn(Hkv, d, generator=g).to(dt)
    return kp, vp, table, torch.tensor(lens, dtype=torch.int32)


def check_decode(o, lse, q, kp, vp, table, lens, window, sinks, scale=None):
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    ref, ref_lse, weight, reach = paged64.decode(q, kp, vp, table.tolist(), lens.tolist(), scale, window, sinks)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    e = 2.0 ** -23 * (d + 8) * reach + 2.0 ** -22 * (4 + 2 * reach)
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(ref) + (2 * e[..., None] + 2.0 ** -15) * weight
    assert np.isfinite(o).all()
    assert (np.abs(o - ref) <= tol).all(), np.max(np.abs(o - ref) / np.maximum(tol, 1e-30))
    empty = np.isinf(ref_lse)
    assert (lse[empty] == -np.inf).all() and (o[empty] == 0).all()
    assert (np.abs(lse[~empty] - ref_lse[~empty]) <= (e + 2.0 ** -23 * np.abs(ref_lse))[~empty]).all()


DECODE = [  # lens, H, Hkv, d, page, window, sinks, type
    ([1], 1, 1, 64, 8, 0, 0, "bf16"),
    ([0], 2, 1, 128, 16, 0, 0, "fp16"),
    ([63, 64, 65, 0, 1, 130], 4, 4, 64, 16, 0, 0, "bf16"),
    ([200, 17, 128, 5], 8, 2, 128, 16, 0, 0, "fp16"),
    ([300, 31, 33, 64], 6, 2, 64, 48, 0, 0, "bf16"),
    ([129, 500], 12, 1, 128, 64, 0, 0, "bf16"),
    ([77, 256, 255], 16, 1, 64, 128, 0, 0, "fp16"),
    ([90, 300], 24, 1, 128, 32, 0, 0, "bf16"),
    ([70, 33], 34, 2, 64, 8, 0, 0, "fp16"),
    ([1700], 8, 8, 128, 16, 0, 0, "bf16"),
    ([400, 64, 65, 1, 0, 130], 4, 2, 64, 16, 64, 4, "bf16"),
    ([400, 64, 65, 1, 0, 130], 4, 2, 128, 16, 1, 0, "fp16"),
    ([500, 222, 70], 8, 1, 128, 64, 100, 70, "bf16"),
    ([500, 129, 3], 4, 4, 64, 8, 37, 1, "fp16"),
    ([300, 200], 2, 2, 64, 32, 1000, 9, "bf16"),
    ([333], 2, 1, 128, 256, 130, 65, "bf16"),
]


@pytest.mark.parametrize("lens,H,Hkv,d,page,window,sinks,dt", DECODE)
def test_decode(fa, lens, H, Hkv, d, page, window, sinks, dt):
    kp, vp, table, n = make(lens, Hkv, d, page, DT[dt], len(lens) + H, window, sinks)
    q = torch.randn(len(lens), H, d, generator=torch.Generator().manual_seed(7)).to(DT[dt])
    dev = [x.cuda() for x in (q, kp, vp, table, n)]
    o, lse = fa.cache.attention_decode(*dev, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == 0
    check_decode(o, lse, q, kp, vp, table, n, window, sinks)
    o2, lse2 = fa.cache.attention_decode(*dev, window=window, sinks=sinks)     # the same bits again
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_many_short_sequences(fa):
    lens = [(7 * i) % 150 for i in range(700)]
    kp, vp, table, n = make(lens, 2, 64, 16, torch.bfloat16, 3)
    q = torch.randn(len(lens), 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    o, lse = fa.cache.attention_decode(*(x.cuda() for x in (q, kp, vp, table, n)))
    assert fa.fa_check_device_error() == 0
    check_decode(o, lse, q, kp, vp, table, n, 0, 0)


def test_decode_large_scores(fa):
    """Scores of some hundreds, where only a maximum subtracted first avoids overflow; ties of the maximum too."""
    kp, vp, table, n = make([300, 90], 1, 64, 16, torch.bfloat16, 3)
    kp *= 8
    kp[table[0, 3], :, 5] = kp[table[0, 9], :, 2]
    q = 8 * torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    o, lse = fa.cache.attention_decode(*(x.cuda() for x in (q, kp, vp, table, n)), scale=1.0)
    check_decode(o, lse, q, kp, vp, table, n, 0, 0, scale=1.0)


def test_decode_strided_queries_another_stream_and_own_workspace(fa):
    lens = [100, 300, 40]
    kp, vp, table, n = make(lens, 2, 64, 16, torch.float16, 5)
    fused = torch.randn(3, 8 + 4, 64, generator=torch.Generator().manual_seed(2)).half().cuda()
    q = fused[:, :8]
    dev = [x.cuda() for x in (kp, vp, table, n)]
    ws = torch.empty(fa.cache.fa_decode_workspace_size(3, 8, 2, 64), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    o, lse = fa.cache.attention_decode(q, *dev, stream=stream, workspace=ws)
    o2, lse2 = fa.cache.attention_decode(q, *dev, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    check_decode(o, lse, q.cpu(), kp, vp, table, n, 0, 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_reports_pages_and_lengths_out_of_range(fa):
    kp, vp, table, n = make([100, 50, 30], 1, 64, 16, torch.bfloat16, 5)
    q = torch.randn(3, 2, 64).to(torch.bfloat16)
    good, good_lse = fa.cache.attention_decode(*(x.cuda() for x in (q, kp, vp, table, n)))
    for bad in (-1, kp.shape[0], 2**31 - 1, -2**31):
        t = table.clone()
        t[0, 2] = bad
        o, lse = fa.cache.attention_decode(*(x.cuda() for x in (q, kp, vp, t, n)))
        assert fa.fa_check_device_error() == FA_ERR_PAGES
        assert torch.isfinite(o).all()
        assert torch.equal(o[1:], good[1:]) and torch.equal(lse[1:], good_lse[1:])
        k2, v2 = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (kp, vp))
        t[0, 2] = kp.shape[0]                         # the same with a page of zeros
        want, _ = fa.cache.attention_decode(*(x.cuda() for x in (q, k2, v2, t, n)))
        assert torch.equal(o, want)
    for length in (-5, 10**6, -2**31):
        m = n.clone()
        m[2] = length
        o, lse = fa.cache.attention_decode(*(x.cuda() for x in (q, kp, vp, table, m)))
        assert fa.fa_check_device_error() == FA_ERR_PAGES
        assert torch.equal(o[0], good[0]) and torch.isinf(lse[2]).all() == (length < 0)
    assert fa.fa_check_device_error() == 0


APPEND = [  # new tokens of each sequence, old ones, Hkv, d, page, type
    ([1], [0], 1, 64, 8, "bf16"),
    ([3, 0, 40, 1], [5, 9, 0, 15], 2, 128, 16, "fp16"),
    ([130, 1, 17], [31, 32, 100], 3, 64, 48, "bf16"),
]


@pytest.mark.parametrize("new,old,Hkv,d,page,dt", APPEND)
def test_append(fa, new, old, Hkv, d, page, dt):
    lens = [a + b for a, b in zip(new, old)]
    kp, vp, table, n = make(lens, Hkv, d, page, DT[dt], 11)
    kp, vp = kp.nan_to_num(0.5), vp.nan_to_num(0.25)
    T = sum(new)
    x = torch.randn(T + 2, 3 * Hkv, d, generator=torch.Generator().manual_seed(5)).to(DT[dt])   # a fused projection; two rows of padding
    cu = [sum(new[:s]) for s in range(len(new) + 1)]
    want_k, want_v = kp.float().numpy().copy(), vp.float().numpy().copy()
    k, v = x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
    paged64.append(k.float().numpy(), v.float().numpy(), want_k, want_v, table.tolist(), lens, cu)
    xd, kd, vd = x.cuda(), kp.cuda(), vp.cuda()
    fa.cache.cache_append(xd[:, Hkv:2 * Hkv], xd[:, 2 * Hkv:], kd, vd, table.cuda(), n.cuda(),
                          torch.tensor(cu, dtype=torch.int32).cuda())
    assert fa.fa_check_device_error() == 0
    assert np.array_equal(kd.float().cpu().numpy(), want_k) and np.array_equal(vd.float().cpu().numpy(), want_v)


def test_append_one_each_skips_empty_slots(fa):
    lens = [17, 0, 16, 1]
    kp, vp, table, n = make(lens, 2, 64, 16, torch.bfloat16, 11)
    kp, vp = kp.nan_to_num(0.5), vp.nan_to_num(0.25)
    k, v = (torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in (1, 2))
    want_k, want_v = kp.float().numpy().copy(), vp.float().numpy().copy()
    paged64.append(k.float().numpy(), v.float().numpy(), want_k, want_v, table.tolist(), lens)
    kd, vd = kp.cuda(), vp.cuda()
    fa.cache.cache_append(k.cuda(), v.cuda(), kd, vd, table.cuda(), n.cuda())
    assert fa.fa_check_device_error() == 0
    assert np.array_equal(kd.float().cpu().numpy(), want_k) and np.array_equal(vd.float().cpu().numpy(), want_v)
    # nothing is written where the place is out of range, and it is reported
    before = kd.clone()
    for t, m in ((torch.full_like(table, -1), n), (torch.full_like(table, kp.shape[0]), n), (table, torch.full_like(n, 10**6)),
                 (table, torch.full_like(n, -3))):
        fa.cache.cache_append(k.cuda(), v.cuda(), kd, vd, t.cuda(), m.cuda())
        assert fa.fa_check_device_error() == FA_ERR_PAGES
        assert torch.equal(kd, before)
    fa.cache.cache_append(k.cuda()[:0], v.cuda()[:0], kd, vd, table.cuda(), n.cuda(), torch.zeros(5, dtype=torch.int32).cuda())
    assert torch.equal(kd, before) and fa.fa_check_device_error() == 0


class Both:
    """A cache on the GPU and the same one in plain lists, driven together."""

    def __init__(self, fa, L, P, Hkv, page, d, S, M, seed):
        self.fa, self.page = fa, page
        g = torch.Generator().manual_seed(seed)
        self.dev = [torch.randn(L, P, Hkv, page, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
        self.refs, self.lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (P, S))
        self.table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
        self.pools = [x.float().cpu().numpy() for x in self.dev]
        self.r, self.t, self.n = [0] * P, [[-1] * M for _ in range(S)], [0] * S

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def reserve(self, add):
        got = self.fa.cache.cache_reserve(self.refs, self.table, self.lens, self.i32(add), self.page)
        assert got.item() == paged64.reserve(self.r, self.t, self.n, add, self.page)
        return got.item()

    def fork(self, src, dst):
        got = self.fa.cache.cache_fork(*self.dev, self.refs, self.table, self.lens, self.i32(src), self.i32(dst))
        assert got.item() == paged64.fork(self.pools, self.r, self.t, self.n, src, dst, self.page)
        return got.item()

    def free(self, seqs):
        self.fa.cache.cache_free(self.refs, self.table, self.lens, self.i32(seqs), self.page)
        paged64.free(self.r, self.t, self.n, seqs, self.page)

    def compact(self):
        got = self.fa.cache.cache_compact(*self.dev, self.refs, self.table, self.lens)
        assert got.item() == paged64.compact(self.pools, self.r, self.t, self.n, self.page)

    def check(self, error=0):
        assert self.fa.fa_check_device_error() == error
        assert self.refs.tolist() == self.r
        assert self.lens.tolist() == self.n
        assert self.table.tolist() == self.t
        for x, y in zip(self.dev, self.pools):
            assert np.array_equal(x.float().cpu().numpy(), y)


@pytest.mark.parametrize("L,P,Hkv,page,d,S,M", [(1, 40, 1, 8, 64, 5, 20), (3, 90, 2, 16, 64, 9, 12), (2, 33, 3, 24, 128, 6, 7)])
def test_page_operators_together(fa, L, P, Hkv, page, d, S, M):
    """Random sequences of calls leave the same tables, counts and pages as the plain statements."""
    import random
    rng = random.Random(P)
    b = Both(fa, L, P, Hkv, page, d, S, M, 1)
    outcomes = set()
    for step in range(60):
        what = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        if what == "reserve":
            outcomes.add(("reserve", min(1, b.reserve([rng.choice([0, 1, rng.randint(0, M * page // 3)]) if n + M * page // 3 <= M * page
                                                       else 0 for n in b.n]))))
        elif what == "fork":
            empty = [s for s in range(S) if b.n[s] == 0]
            if empty:
                dst = rng.sample(empty, rng.randint(1, len(empty)))
                outcomes.add(("fork", min(1, b.fork([rng.randrange(S) for _ in dst], dst))))
        elif what == "free":
            b.free(rng.sample(range(S), rng.randint(1, max(1, S // 2))))
        else:
            b.compact()
        b.check()
    assert {("reserve", 0), ("fork", 0)} <= outcomes


def test_page_operators_refuse_without_changing(fa):
    b = Both(fa, 1, 10, 1, 8, 64, 4, 6, 2)
    assert b.reserve([20, 8, 0, 0]) == 0              # 3 + 1 pages
    b.check()
    assert b.reserve([28, 40, 0, 20]) == 5            # 3 + 5 + 3 wanted, 6 free
    b.check()
    assert b.reserve([0, 0, 0, 49]) == -1             # longer than the table's row
    b.check(FA_ERR_PAGES)
    assert b.reserve([0, -1, 0, 0]) == -1
    b.check(FA_ERR_PAGES)
    assert b.reserve([2**31 - 1, 0, 0, 0]) == -1
    b.check(FA_ERR_PAGES)
    for src, dst in (([0, 0], [2, 2]), ([0], [1]), ([4], [2]), ([0], [-1]), ([-7], [2]), ([0, 1], [3, 4])):
        assert b.fork(src, dst) == -1
        b.check(FA_ERR_PAGES)
    assert b.fork([2], [2]) == 0                      # an empty slot onto itself
    b.check()
    assert b.fork([0, 0], [2, 3]) == 0
    b.check()
    b.free([0, 2, 0, 2])                              # twice in one call counts once
    b.check()
    b.fa.cache.cache_free(b.refs, b.table, b.lens, b.i32([9, -1]), b.page)
    b.check(FA_ERR_PAGES)
    b.compact()
    b.check()
    # no page left for a branch's last page
    assert b.reserve([0, 8 * 4, 0, 0]) == 0
    while b.r.count(0):
        s = b.n.index(min(b.n))
        assert b.reserve([8 * (i == s) for i in range(4)]) == 0
    b.check()


def test_large_pool_scan(fa):
    """More pages than one round of the planning kernel covers, free ones scattered."""
    P, S, M, page = 9001, 40, 300, 8
    b = Both(fa, 1, P, 1, page, 64, S, M, 3)
    assert b.reserve([8 * 220] * S) == 0
    b.free(list(range(0, S, 3)))
    assert b.reserve([(17 * s) % 90 for s in range(S)]) == 0
    b.check()
    b.free(list(range(1, S, 3)))
    b.compact()
    b.check()


def test_more_sequences_than_planning_threads(fa):
    """Requests beyond one round of the planning kernel, with and without enough pages."""
    P, S, M, page = 5000, 2500, 4, 8
    b = Both(fa, 1, P, 1, page, 64, S, M, 4)
    assert b.reserve([(5 * s) % 24 if s < 1250 else 0 for s in range(S)]) == 0
    assert b.fork([(3 * f) % 1250 for f in range(1150)], list(range(1300, 2450))) == 0
    b.check()
    assert b.reserve([8 if n <= 24 else 0 for n in b.n]) > 0          # too many
    b.check()
    b.free(list(range(0, 1250, 2)))
    assert b.reserve([s % 2 for s in range(S)]) == 0
    b.compact()
    b.check()


def test_serving_run(fa):
    """Prompts, decoding, branches, ended sequences and compaction, as a server does them: every step's
    attention equals the plain one over each sequence's own tokens."""
    L, P, H, Hkv, page, d, S, M = 2, 60, 4, 2, 16, 64, 6, 12
    g = torch.Generator().manual_seed(9)
    kp, vp = (torch.full((L, P, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    refs, lens = torch.zeros(P, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    held = [[[torch.zeros(0, Hkv, d, dtype=torch.bfloat16) for _ in range(2)] for _ in range(S)] for _ in range(L)]

    def write(counts):
        add = i32(counts)
        assert fa.cache.cache_reserve(refs, table, lens, add, page).item() == 0
        cu = i32([sum(counts[:s]) for s in range(S + 1)])
        for l in range(L):
            k, v = rand(sum(counts), Hkv, d), rand(sum(counts), Hkv, d)
            fa.cache.cache_append(k.cuda(), v.cuda(), kp[l], vp[l], table, lens, cu)
            at = 0
            for s, c in enumerate(counts):
                for j, x in enumerate((k, v)):
                    held[l][s][j] = torch.cat([held[l][s][j], x[at:at + c]])
                at += c

    def check(window=0, sinks=0):
        n = [held[0][s][0].shape[0] for s in range(S)]
        assert lens.tolist() == n
        for l in range(L):
            q = rand(S, H, d)
            o, lse = fa.cache.attention_decode(q.cuda(), kp[l], vp[l], table, lens, window=window, sinks=sinks)
            most = max(n + [1])
            flat = [torch.zeros(S, Hkv, most, d, dtype=torch.bfloat16) for _ in range(2)]
            for s in range(S):
                for j in range(2):
                    flat[j][s, :, :n[s]] = held[l][s][j].transpose(0, 1)
            check_decode(o, lse, q, flat[0], flat[1], torch.arange(S).view(S, 1), torch.tensor(n), window, sinks)

    write([50, 16, 33, 0, 0, 0])
    check()
    for _ in range(3):
        write([1, 1, 1, 0, 0, 0])
        check()
    assert fa.cache.cache_fork(kp, vp, refs, table, lens, i32([0, 2]), i32([3, 5])).item() == 0
    for l in range(L):
        held[l][3], held[l][5] = list(held[l][0]), list(held[l][2])
    check(window=20, sinks=3)
    write([1, 0, 2, 1, 0, 1])                          # the branches go their own ways
    check()
    fa.cache.cache_free(refs, table, lens, i32([0, 2]), page)
    for l in range(L):
        for s in (0, 2):
            held[l][s] = [x[:0] for x in held[l][s]]
    check()
    live = fa.cache.cache_compact(kp, vp, refs, table, lens).item()
    assert (refs > 0).sum().item() == live and (refs[:live] > 0).all()
    check(window=9, sinks=1)
    write([5, 1, 100, 1, 20, 0])
    check()
    assert fa.fa_check_device_error() == 0


def test_decoding_step_in_a_graph(fa):
    """A captured step (reserve, append, decode) replayed while the cache grows past pages, beside a second
    graph with its own workspace on another stream."""
    S, H, Hkv, page, d, P, M = 3, 4, 2, 8, 64, 40, 10
    g = torch.Generator().manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    caches = []
    for _ in range(2):
        c = dict(kp=torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda"),
                 vp=torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda"),
                 refs=torch.zeros(P, dtype=torch.int32, device="cuda"), lens=torch.zeros(S, dtype=torch.int32, device="cuda"),
                 table=torch.full((S, M), -1, dtype=torch.int32, device="cuda"), q=rand(S, H, d), k=rand(S, Hkv, d),
                 v=rand(S, Hkv, d), one=torch.ones(S, dtype=torch.int32, device="cuda"))
        caches.append(c)

    def step(c):
        fa.cache.cache_reserve(c["refs"], c["table"], c["lens"], c["one"], page)
        fa.cache.cache_append(c["k"], c["v"], c["kp"], c["vp"], c["table"], c["lens"])
        return fa.cache.attention_decode(c["q"], c["kp"], c["vp"], c["table"], c["lens"])

    for c in caches:
        step(c)                                        # loads the kernels; one token each
        c["seen"] = [(c["k"].cpu(), c["v"].cpu())]
    torch.cuda.synchronize()
    for c in caches:
        c["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c["graph"]):
            c["out"] = step(c)
    streams = [torch.cuda.Stream() for _ in caches]
    for i in range(20):
        for c in caches:
            for n in "qkv":
                c[n].copy_(rand(*c[n].shape))
            c["seen"].append((c["k"].cpu(), c["v"].cpu()))
        torch.cuda.synchronize()
        for c, stream in zip(caches, streams):
            with torch.cuda.stream(stream):
                c["graph"].replay()
        torch.cuda.synchronize()
        for c in caches:
            assert c["lens"].tolist() == [i + 2] * S
            flat = [torch.stack([x[j] for x in c["seen"]], 2) for j in range(2)]
            check_decode(*c["out"], c["q"].cpu(), *flat, torch.arange(S).view(S, 1), torch.full((S,), i + 2), 0, 0)
    assert fa.fa_check_device_error() == 0


def test_cache_of_more_than_2_to_the_32_elements(fa):
    """Pages whose offsets pass 32 bits: appended to, read, forked, moved.  (Nothing else of the pool is touched.)"""
    P, Hkv, page, d, S, M = 270_000, 8, 16, 128, 3, 8
    kp, vp = (torch.empty(1, P, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kp.numel() > 2**32
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    refs = torch.ones(P, dtype=torch.int32, device="cuda")         # all in use but the last ones and one early page
    refs[-9:] = 0
    refs[2] = 0
    lens, table = i32([0] * S), torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    assert fa.cache.cache_reserve(refs, table, lens, i32([40, 0, 0]), page).item() == 0
    assert table[0, :3].tolist() == [2, P - 9, P - 8]
    g = torch.Generator().manual_seed(3)
    k, v, q = (torch.randn(*s, generator=g).to(torch.bfloat16) for s in ((40, Hkv, d), (40, Hkv, d), (S, 16, d)))
    fa.cache.cache_append(k.cuda(), v.cuda(), kp[0], vp[0], table, lens, i32([0, 40, 40, 40]))
    assert torch.equal(kp[0, P - 8, :, 7].cpu(), k[39])
    assert fa.cache.cache_fork(kp, vp, refs, table, lens, i32([0]), i32([2])).item() == 0
    assert table[2, :3].tolist() == [2, P - 9, P - 7]
    refs[10:16] = 0                                                # compaction brings the high pages down
    live = fa.cache.cache_compact(kp, vp, refs, table, lens).item()
    assert live == P - 6 - 6 and table[:, :3].max().item() < live
    flat = [x.transpose(0, 1)[None].expand(S, -1, -1, -1) for x in (k, v)]
    o, lse = fa.cache.attention_decode(q.cuda(), kp[0], vp[0], table, lens)
    check_decode(o, lse, q, *flat, torch.arange(S).view(S, 1), torch.tensor([40, 0, 40]), 0, 0)
    assert fa.fa_check_device_error() == 0


def test_both_ways_through_the_binding(fa, monkeypatch):
    """The compiled way and the ctypes one give the same results, and the same errors."""
    from flashattention_bf16_fwd_b200 import window
    from flashattention_bf16_fwd_b200.fa import FAError
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").half()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q, k, v, do = rand(2, 4, 300, 64), rand(2, 2, 300, 64), rand(2, 2, 300, 64), rand(2, 4, 300, 64)
    new_k, new_v, new_q = rand(90, 6, 64)[:, 2:4], rand(90, 2, 64), rand(4, 4, 64)

    def everything():
        kp, vp = (torch.zeros(2, 40, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2))
        refs, lens, table = i32([0] * 40), i32([0] * 4), torch.full((4, 9), -1, dtype=torch.int32, device="cuda")
        out = list(window.attention_window_fwd(q, k, v, 50, 3))
        out += window.attention_window_bwd(q, k, v, *out, do, 50, 3, 0.2)[1:]
        out.append(fa.cache.cache_reserve(refs, table, lens, i32([40, 33, 17, 0]), 16))
        fa.cache.cache_append(new_k, new_v, kp[0], vp[0], table, lens, i32([0, 40, 73, 90, 90]))
        out.append(fa.cache.cache_fork(kp, vp, refs, table, lens, i32([1]), i32([3])))
        fa.cache.cache_append(new_k[:4], new_v[:4], kp[1], vp[1], table, lens)
        out += fa.cache.attention_decode(new_q, kp[0], vp[0], table, lens, scale=0.3)
        out += fa.cache.attention_decode(new_q, kp[0], vp[0], table, lens, window=9, sinks=2)
        fa.cache.cache_free(refs, table, lens, i32([0]), 16)
        out.append(fa.cache.cache_compact(kp, vp, refs, table, lens))
        return out + [kp, vp, refs, table, lens]

    def errors():
        kp = torch.zeros(9, 2, 16, 64, dtype=torch.float16, device="cuda")
        lens, table = i32([1]), i32([[0]])
        said = []
        for call in (lambda: window.attention_window_fwd(q, k, v, 0), lambda: window.attention_window_fwd(q, k, v, 5, -1),
                     lambda: window.attention_window_fwd(q, k, v, 5, fix_mode=6),
                     lambda: window.attention_window_fwd(q, k, v, 5, scale=-1.0), lambda: window.attention_window_fwd(q, k[:1], v, 5),
                     lambda: window.attention_window_fwd(q, k.float(), v.float(), 5), lambda: window.attention_window_fwd(q, k.cpu(), v, 5),
                     lambda: window.attention_window_bwd(q, k, v, q, do[..., 0], do, 5),
                     lambda: fa.cache.attention_decode(new_q[:1], kp, kp, table, lens, sinks=3),
                     lambda: fa.cache.attention_decode(new_q[:1], kp, kp, table, lens, window=-2),
                     lambda: fa.cache.attention_decode(new_q[:2], kp, kp, table, lens),
                     lambda: fa.cache.cache_append(new_k, new_v, kp, kp, table, lens),
                     lambda: fa.cache.cache_reserve(i32([0] * 9), table, lens, lens, 12),
                     lambda: fa.cache.cache_reserve(i32([0] * 9), table, lens, lens, 2**32 + 16),
                     lambda: fa.cache.cache_free(i32([0] * 9), table, lens, i32([0, 0]), 16),
                     lambda: fa.cache.cache_fork(kp, kp, i32([0] * 8), table, lens, lens, lens)):
            with pytest.raises((ValueError, FAError)) as e:
                call()
            said.append((type(e.value), str(e.value)))
        return said

    fast, fast_errors = everything(), errors()
    class Never:
        def __getattr__(self, name):
            return lambda *a: None
    monkeypatch.setattr(fa.cache, "_fast", Never())
    monkeypatch.setattr(window, "_fast", Never())
    for a, b in zip(fast, everything()):
        assert torch.equal(a, b)
    assert errors() == fast_errors
    assert fa.fa_check_device_error() == 0
