"""Lengths and pages of a decoder's requests, on the CPU."""
import pytest
import torch

from serving_router_top_gb300.decoder import Decoder, Pages


@pytest.fixture
def decoder(monkeypatch):
    """A decoder's host state alone: 2 requests of 32 places in pages of 4, 16 tokens a call."""
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self, *a, **k: self)
    d = Decoder.__new__(Decoder)
    d.pages, d.lens, d.maxT = Pages(2, 16, 4, 32), [0, 0], 16
    return d


def state(d):
    return list(d.lens), list(d.pages.held), list(d.pages.free), d.pages.table.tolist()


def test_lengths_and_pages_follow_the_batches(decoder):
    for new, lens, held in [([5, 0], [5, 0], [2, 0]), ([3, 9], [8, 9], [2, 3]), ([0, 1], [8, 10], [2, 3])]:
        b = decoder.batch(new)
        assert decoder.lens == lens and decoder.pages.held == held and b.kv_len.tolist() == lens
        assert b.q_start.tolist() == [0, new[0], sum(new)] and b.c.T == sum(new) and b.c.max_n == max(new)
    pages = [x for row in decoder.pages.table.tolist() for x in row if x >= 0]
    assert len(set(pages)) == 5 and not set(pages) & set(decoder.pages.free)


@pytest.mark.parametrize("new", [[4, 4],       # request 1 has two places left
                                 [16, 1],      # more than a call's tokens
                                 [1], [1, 1, 1], [3, -1]])
def test_a_refused_batch_changes_nothing(decoder, new):
    decoder.batch([8, 8])
    decoder.batch([0, 14])
    decoder.batch([0, 8])
    before = state(decoder)
    with pytest.raises((RuntimeError, ValueError)):
        decoder.batch(new)
    assert state(decoder) == before
    decoder.batch([1, 2])
    assert decoder.lens == [9, 32]


def test_pages_run_out_for_all_or_none(decoder):
    decoder.pages.free = decoder.pages.free[:3]
    before = state(decoder)
    with pytest.raises(RuntimeError):
        decoder.batch([8, 8])
    assert state(decoder) == before
    decoder.batch([8, 4])
    assert decoder.pages.held == [2, 1] and decoder.pages.free == []
