"""Pages that requests share and give back, on the CPU."""
import pytest

from serving_router_top_gb300.decoder import Pages


@pytest.fixture
def pages(monkeypatch):
    import torch
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self, *a, **k: self)
    return Pages(3, 8, 4, 32)


def held(p, r):
    return p.table[r, :p.held[r]].tolist()


def test_a_fork_shares_whole_pages_and_copies_the_last(pages):
    pages.reserve(0, 11)
    assert pages.fork(0, 1, 11) == [(held(pages, 0)[2], held(pages, 1)[2], 3)]
    assert held(pages, 1)[:2] == held(pages, 0)[:2] and held(pages, 1)[2] not in held(pages, 0)
    assert len(pages.free) == 4 and pages.users == [sum(i in held(pages, r) for r in range(3)) for i in range(8)]
    assert pages.fork(1, 2, 8) == [] and held(pages, 2) == held(pages, 0)[:2]
    pages.reserve(2, 9)
    assert held(pages, 2)[2] not in held(pages, 0) + held(pages, 1)


def test_pages_are_free_once_nobody_holds_them(pages):
    pages.reserve(0, 8)
    pages.fork(0, 1, 6)
    pages.release(0)
    assert pages.held[0] == 0 and (pages.table[0] == -1).all() and len(pages.free) == 6
    pages.release(1)
    assert sorted(pages.free) == list(range(8)) and not any(pages.users)
    pages.release(1)
    assert len(pages.free) == 8


def test_forks_that_cannot_be_change_nothing(pages):
    pages.reserve(0, 30)
    before = pages.table.clone(), list(pages.free), list(pages.users), list(pages.held)
    for call in (lambda: pages.fork(0, 0, 4), lambda: pages.fork(1, 2, 4), lambda: pages.fork(0, 1, 33),
                 lambda: pages.fork(0, 1, 30)):
        with pytest.raises((ValueError, RuntimeError)):
            call()
        assert (pages.table == before[0]).all() and (pages.free, pages.users, pages.held) == before[1:]
    assert pages.fork(0, 1, 28) == []
