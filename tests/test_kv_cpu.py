"""Page bookkeeping of the paged cache (sparse_moe_expert_gemv_b200/kv.py)
without a GPU."""
import random

import pytest

from sparse_moe_expert_gemv_b200.kv import PagedKV


def make(n_pages=20, max_seqs=3, max_len=100, window=0, n_sink=0):
    return PagedKV(None, None, n_layers=1, n_q=2, n_kv=1, head_dim=64, page_size=16, n_pages=n_pages,
                   max_seqs=max_seqs, max_len=max_len, window=window, n_sink=n_sink, device="cpu")


def check(kv, n_pages):
    used = [p for s in kv.pages for p in s if p >= 0]
    assert len(used) == len(set(used)) and len(used) + kv.free_pages() == n_pages
    assert not set(used) & set(kv._free)
    for s, pages in enumerate(kv.pages):
        assert kv.table[s, :len(pages)].tolist() == pages
        assert (kv.table[s, len(pages):] == -1).all()
        assert len(pages) * kv.page >= kv.length[s]


def test_steps_give_pages_and_offsets():
    kv = make()
    assert kv.step([5, 0, 17]) == 22
    assert kv.row_off.tolist() == [0, 5, 5, 22] and kv.kv_len.tolist() == [5, 0, 17]
    assert [len(p) for p in kv.pages] == [1, 0, 2]
    assert kv.step([12, 1, 0]) == 13
    assert kv.kv_len.tolist() == [17, 1, 17] and [len(p) for p in kv.pages] == [2, 1, 2]
    check(kv, 20)
    kv.trim(0, 3)
    kv.step([2, 0, 0])
    assert kv.kv_len.tolist() == [16, 1, 17] and len(kv.pages[0]) == 2
    kv.release(2)
    kv.step([0, 0, 0])
    check(kv, 20)


def test_refusals_change_nothing():
    kv = make(n_pages=3)
    kv.step([30, 0, 0])
    for bad, err in (([0, 33, 0], MemoryError), ([80, 0, 0], ValueError), ([1, 1], ValueError), ([-1, 0, 0], ValueError)):
        before = (kv.free_pages(), list(kv.length), [list(p) for p in kv.pages])
        with pytest.raises(err):
            kv.step(bad)
        assert before == (kv.free_pages(), list(kv.length), [list(p) for p in kv.pages])
    with pytest.raises(ValueError):
        kv.trim(0, 31)


def test_window_gives_back_only_what_no_later_token_sees():
    window, sink, page = 20, 3, 16
    kv = make(n_pages=12, max_seqs=1, max_len=100, window=window, n_sink=sink)
    rng = random.Random(3)
    while kv.length[0] < 90:
        old = kv.length[0]
        r = rng.randint(1, 6)
        kv.step([r])
        for i in range(old, old + r):        # every key that the step's tokens see is there
            for j in range(i + 1):
                if i - j < window or j < sink:
                    assert kv.pages[0][j // page] >= 0
        check(kv, 12)
        kv.trim(0, rng.randint(0, r - 1))    # rejected draft tokens
    assert kv.pages[0].count(-1) >= 3
