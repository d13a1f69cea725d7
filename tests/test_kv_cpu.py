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


def visible(kv, s, rows):
    """Every key that the last `rows` tokens of slot s see has a page."""
    return all(kv.pages[s][j // kv.page] >= 0 for i in range(kv.length[s] - rows, kv.length[s])
               for j in range(i + 1) if i - j < kv.window or j < kv.n_sink)


@pytest.mark.parametrize("first,second,refused,back", [
    ([38, 0], [14, 0], [1, 97], 13),   # other slots' tokens do not fit
    ([26, 16], [10, 0], [1, 60], 9),
    ([26, 16], [10, 0], [64, 20], 9),
])
def test_refused_step_gives_no_page_back(first, second, refused, back):
    """A step that finds too few pages changes nothing, so the step before it
    can still be trimmed: its tokens' windows reach back to pages that the
    refused one would have given back."""
    kv = make(n_pages=6, max_seqs=2, max_len=100, window=20)
    kv.step(first)
    kv.step(second)
    before = (sorted(kv._free), list(kv.length), list(kv.rows), [list(p) for p in kv.pages], kv._table.tolist())
    with pytest.raises(MemoryError):
        kv.step(refused)
    assert before == (sorted(kv._free), list(kv.length), list(kv.rows), [list(p) for p in kv.pages],
                      kv._table.tolist())
    kv.trim(0, back)
    kv.step([1, 0])
    assert visible(kv, 0, 1)
    check(kv, 6)


def test_steps_trims_and_refusals_at_random():
    rng = random.Random(7)
    refused = 0
    for trial in range(40):
        window, sink = rng.choice([1, 5, 20, 40]), rng.choice([0, 3, 16, 17])
        kv = make(n_pages=7, max_seqs=2, max_len=200, window=window, n_sink=sink)
        for _ in range(30):
            rows = [rng.choice([0, 1, 3, 30]) for _ in range(2)]
            try:
                kv.step(rows)
            except (MemoryError, ValueError):
                refused += 1
            else:
                assert all(visible(kv, s, r) for s, r in enumerate(rows))
            check_given(kv, 7)
            s = rng.randrange(2)
            kv.trim(s, rng.randint(0, max(0, kv.rows[s] - 1)))
            if rng.random() < 0.1:
                kv.release(s)
    assert refused > 20


def check_given(kv, n_pages):
    used = [p for s in kv.pages for p in s if p >= 0]
    assert sorted(used + kv._free) == list(range(n_pages))


def test_batches_of_many_row_counts_are_not_all_kept():
    class B:
        MOE_KV_BF16 = MOE_KV_E4M3 = 1
        moe_attn_configure = staticmethod(lambda *a: None)
        KvBatch = staticmethod(lambda *a, **kw: a)

    kv = PagedKV(B, None, n_layers=3, n_q=2, n_kv=1, head_dim=64, page_size=16, n_pages=4, max_seqs=1, max_len=64,
                 device="cpu")
    for n in range(1, 500):
        for layer in range(3):
            batch = kv.batch(layer, n)
            assert batch[0] is kv.k[layer] and batch[-1] == n and kv.batch(layer, n) is batch
        assert len(kv._batches) <= 48
