"""The page operators on tables and lengths that are wrong: what the header says of each is left out, everything
else is done, and it is reported."""
import pytest
import torch

pytestmark = pytest.mark.gpu
FA_ERR_PAGES = -13


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from flashattention_bf16_fwd_b200 import cache, fa as binding
    binding.cache = cache
    assert binding.fa_check_device_error() == 0
    return binding


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pools(L, P, page=8):
    """Two pools in which every element of a page says which page and layer it is."""
    at = torch.arange(L * P).view(L, P, 1, 1, 1).expand(L, P, 1, page, 64).float()
    return at.half().cuda(), (-at).half().cuda()


def counts(P, held):
    refs = [0] * P
    for p in held:
        refs[p] += 1
    return i32(refs)


@pytest.mark.parametrize("stray", [3, 11, 12, -1, 2**31 - 1, -2**31])
def test_compact_takes_out_entries_of_free_pages(fa, stray):
    """Page 3 is free, and page 10 moves into it: an entry that named it would read another sequence's tokens."""
    kp, vp = pools(2, 12)
    refs = counts(12, [9, 2, 10, 0])
    table, lens = i32([[9, 2, 10, -1], [0, stray, -1, -1]]), i32([24, 9])
    live = fa.cache.cache_compact(kp, vp, refs, table, lens)
    assert live.item() == 4 and fa.fa_check_device_error() == FA_ERR_PAGES
    assert table.tolist() == [[1, 2, 3, -1], [0, -1, -1, -1]]
    assert refs.tolist() == [1, 1, 1, 1] + [0] * 8 and lens.tolist() == [24, 9]
    for layer in range(2):
        assert kp[layer, :4, 0, 0, 0].tolist() == [12 * layer + p for p in (0, 9, 2, 10)]
        assert vp[layer, :4, 0, 0, 0].tolist() == [-12 * layer - p for p in (0, 9, 2, 10)]


def test_compact_with_nothing_to_move(fa):
    kp, vp = pools(1, 8)
    refs, table, lens = counts(8, [0, 1]), i32([[1, 0, 5]]), i32([24])
    assert fa.cache.cache_compact(kp, vp, refs, table, lens).item() == 2
    assert fa.fa_check_device_error() == FA_ERR_PAGES
    assert table.tolist() == [[1, 0, -1]] and refs.tolist() == [1, 1] + [0] * 6
    table = i32([[1, 0, 5]])                            # not in use: not looked at
    assert fa.cache.cache_compact(kp, vp, refs, table, i32([16])).item() == 2
    assert fa.fa_check_device_error() == 0 and table.tolist() == [[1, 0, 5]]


@pytest.mark.parametrize("length,row", [(-1, [6, 5]), (-2**31, [6, 5]), (17, [0, 1]), (2**31 - 1, [0, 1])])
def test_compact_reports_lengths_out_of_range(fa, length, row):
    """They count as the nearest in range."""
    kp, vp = pools(1, 8)
    refs, table, lens = counts(8, [6, 5]), i32([[6, 5], [7, 7]]), i32([length, 0])
    assert fa.cache.cache_compact(kp, vp, refs, table, lens).item() == 2
    assert fa.fa_check_device_error() == FA_ERR_PAGES
    want = {6: 1, 5: 0}
    assert table.tolist() == [[want[6], want[5]] if length > 0 else row, [7, 7]] and lens.tolist() == [length, 0]


@pytest.mark.parametrize("bad", [10, -1, 2**31 - 1, -2**31])
def test_fork_of_a_last_page_out_of_range(fa, bad):
    """The number is copied as it is: no page is taken for it, and none is missing."""
    kp, vp = pools(2, 10)
    refs = counts(10, [4, 2, 7])
    table, lens = i32([[4, bad, -1], [2, 7, -1], [-1] * 3, [-1] * 3, [-1] * 3]), i32([12, 11, 0, 0, 0])
    refs[torch.tensor([0, 1, 3, 5, 6])] = 1             # two pages are free, for the two forks of sequence 1
    missing = fa.cache.cache_fork(kp, vp, refs, table, lens, i32([1, 0, 1]), i32([2, 3, 4]))
    assert missing.item() == 0 and fa.fa_check_device_error() == FA_ERR_PAGES
    assert table.tolist() == [[4, bad, -1], [2, 7, -1], [2, 8, -1], [4, bad, -1], [2, 9, -1]]
    assert refs.tolist() == [1, 1, 3, 1, 2, 1, 1, 1, 1, 1] and lens.tolist() == [12, 11, 11, 12, 11]
    for layer in range(2):
        for new in (8, 9):
            assert kp[layer, new, 0, :, 0].tolist() == [10 * layer + 7] * 3 + [10 * layer + new] * 5
            assert vp[layer, new, 0, :, 0].tolist() == [-10 * layer - 7] * 3 + [-10 * layer - new] * 5


def test_fork_of_a_full_page_out_of_range(fa):
    kp, vp = pools(1, 6)
    refs, table, lens = counts(6, [1, 3]), i32([[1, 6, 3], [-1] * 3]), i32([20, 0])
    assert fa.cache.cache_fork(kp, vp, refs, table, lens, i32([0]), i32([1])).item() == 0
    assert fa.fa_check_device_error() == FA_ERR_PAGES
    assert table.tolist() == [[1, 6, 3], [1, 6, 0]] and refs.tolist() == [1, 2, 0, 1, 0, 0] and lens.tolist() == [20, 20]
    assert kp[0, 0, 0, :, 0].tolist() == [3] * 4 + [0] * 4


@pytest.mark.parametrize("bad", [6, -1, 2**31 - 1, 2])
def test_free_of_entries_that_name_no_page_in_use(fa, bad):
    refs, table, lens = counts(6, [1, 3, 5]), i32([[1, bad, 3], [5, -1, -1]]), i32([20, 8])
    fa.cache.cache_free(refs, table, lens, i32([0]), 8)
    assert fa.fa_check_device_error() == FA_ERR_PAGES
    assert refs.tolist() == [0, 0, 0, 0, 0, 1] and table.tolist() == [[-1] * 3, [5, -1, -1]] and lens.tolist() == [0, 8]


@pytest.mark.parametrize("length", [-3, 25, 2**31 - 1])
def test_free_of_lengths_out_of_range(fa, length):
    refs, table, lens = counts(6, [1, 2, 3]), i32([[1, 2, 3]]), i32([length])
    fa.cache.cache_free(refs, table, lens, i32([0]), 8)
    assert fa.fa_check_device_error() == FA_ERR_PAGES and lens.tolist() == [0]
    assert refs.tolist() == ([0, 1, 1, 1, 0, 0] if length < 0 else [0] * 6)
