"""What other requests do between a tree and its verification, on the CPU: the kernels are stood in for."""
import pytest
import torch

from serving_router_top_gb300 import moe
from serving_router_top_gb300.decoder import Decoder, Pages

PAGE = 4


class Kernels:
    """Verification keeps a given number of nodes; a compaction writes the lengths that moe_kv_compact does."""

    def __init__(self):
        self.keep, self.moved, self.copied, self.fails = {}, [], [], False

    def verify(self, batch, desc, path, count, token, err=None, stream=None):
        if self.fails:
            raise moe.MoeError(moe.MOE_EINVAL, "moe_verify_drafts")
        path.fill_(-1)
        for b, n in enumerate((batch.q_start[1:] - batch.q_start[:-1]).tolist()):
            count[b] = min(self.keep.get(b, n), n, path.shape[1])
            token[b] = 7 if n else -1
            path[b, :count[b]] = torch.arange(int(count[b]), dtype=torch.int32)

    def compact(self, layers, batch, path, count, lens=None, err=None, stream=None):
        self.moved.append(count.tolist())
        if lens is not None:
            lens.copy_(batch.kv_len - (batch.q_start[1:] - batch.q_start[:-1]) + count)

    def copy(self, layers, src, dst, tokens=None, err=None, stream=None):
        self.copied.append((src.tolist(), dst.tolist(), tokens.tolist()))


@pytest.fixture
def kernels(monkeypatch):
    k, empty = Kernels(), torch.empty
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self, *a, **kw: self)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw))
    monkeypatch.setattr(moe, "moe_tree_prepare", lambda *a, **kw: None)
    monkeypatch.setattr(moe, "moe_verify_drafts", k.verify)
    monkeypatch.setattr(moe, "moe_kv_compact", k.compact)
    monkeypatch.setattr(moe, "moe_kv_copy_pages", k.copy)
    return k


@pytest.fixture
def decoder(kernels):
    """A decoder's host state alone: 4 requests of 64 places in pages of 4; 0 has 18 tokens, 1 three, 2 has 40."""
    class Word:
        error_ptr = 0
    d = Decoder.__new__(Decoder)
    d.pages, d.lens, d.maxT, d.ws, d.kv_layers = Pages(4, 64, PAGE, 64), [0] * 4, 64, Word, None
    d.batch([18, 3, 40, 0])
    return d


def sound(d):
    """Every request holds pages for its tokens, and a page that two hold is whole in both."""
    for r, n in enumerate(d.lens):
        assert d.pages.held[r] * PAGE >= n
        for j in range(d.pages.held[r]):
            id = int(d.pages.table[r, j])
            users = [(q, i) for q in range(4) for i in range(d.pages.held[q]) if int(d.pages.table[q, i]) == id]
            assert len(users) == d.pages.users[id] and id not in d.pages.free
            assert len(users) == 1 or all(i == j and d.lens[q] >= (j + 1) * PAGE for q, i in users)


def test_a_fork_of_another_request_keeps_its_tokens(decoder, kernels):
    bt, _ = decoder.tree_batch([[-1, 0, 0, 1, 1], [], [], []])
    decoder.fork(2, 3)
    kernels.keep = {0: 3}
    assert decoder.accept(bt, None) == ([[0, 1, 2], [], [], []], [7, -1, -1, -1])
    assert decoder.lens == [21, 3, 40, 40]
    sound(decoder)
    decoder.batch([0, 0, 0, 2])
    assert decoder.lens[3] == 42
    sound(decoder)


def test_a_batch_of_another_request_keeps_its_tokens(decoder, kernels):
    bt, _ = decoder.tree_batch([[-1, 0, 0, 1, 1], [], [], []])
    decoder.batch([0, 5, 0, 9])
    kernels.keep = {0: 1}
    decoder.accept(bt, None)
    assert decoder.lens == [19, 8, 40, 9]
    sound(decoder)


def test_a_release_of_another_request_stays(decoder, kernels):
    bt, _ = decoder.tree_batch([[-1, 0, 0, 1, 1], [], [], []])
    decoder.release(2)
    kernels.keep = {0: 2}
    decoder.accept(bt, None)
    assert decoder.lens == [20, 3, 0, 0]
    sound(decoder)


def test_a_request_released_with_its_tree_keeps_nothing(decoder, kernels):
    """Its pages may be another's by then: nothing of it is moved."""
    bt, _ = decoder.tree_batch([[-1, 0, 0, 1, 1], [-1, 0], [], []])
    decoder.release(0)
    decoder.batch([0, 0, 0, 50])
    kernels.keep = {0: 3, 1: 1}
    assert decoder.accept(bt, None) == ([[], [0], [], []], [-1, 7, -1, -1])
    assert decoder.lens == [0, 4, 40, 50] and kernels.moved == [[0, 1, 0, 0]]
    sound(decoder)


def test_a_released_request_may_begin_again(decoder, kernels):
    bt, _ = decoder.tree_batch([[-1, 0], [-1, 0, 1], [], []])
    decoder.release(1)
    decoder.fork(2, 1)
    second, _ = decoder.tree_batch([[], [-1, 0, 0], [], []])
    kernels.keep = {0: 1, 1: 2}
    decoder.accept(bt, None)
    assert decoder.lens == [19, 43, 40, 0]
    assert decoder.accept(second, None)[0][1] == [0, 1]
    assert decoder.lens == [19, 42, 40, 0]
    sound(decoder)


@pytest.mark.parametrize("first", [0, 1])
def test_trees_of_two_calls_are_verified_in_any_order(decoder, kernels, first):
    a, _ = decoder.tree_batch([[-1, 0, 0, 1, 1], [], [], []])
    b, _ = decoder.tree_batch([[], [-1, 0, 1], [-1, 0], []])
    kernels.keep = {0: 4, 1: 1, 2: 2}
    for bt in ((a, b), (b, a))[first]:
        decoder.accept(bt, None)
    assert decoder.lens == [22, 4, 42, 0]
    sound(decoder)


def test_a_request_waits_for_its_verification(decoder, kernels):
    bt, _ = decoder.tree_batch([[-1, 0, 0, 1, 1], [], [], []])
    before = list(decoder.lens), list(decoder.pages.held), list(decoder.pages.free), decoder.pages.table.tolist()
    for call in (lambda: decoder.fork(0, 3), lambda: decoder.fork(2, 0), lambda: decoder.batch([1, 0, 0, 0]),
                 lambda: decoder.tree_batch([[-1], [-1], [], []])):
        with pytest.raises(ValueError):
            call()
        assert (decoder.lens, decoder.pages.held, decoder.pages.free, decoder.pages.table.tolist()) == before
    assert kernels.copied == []
    kernels.keep = {0: 4}
    decoder.accept(bt, None)
    decoder.fork(0, 3)
    decoder.batch([1, 1, 0, 1])
    assert decoder.lens == [23, 4, 40, 23]
    sound(decoder)


def test_a_tree_is_verified_once(decoder, kernels):
    bt, _ = decoder.tree_batch([[-1, 0], [], [], []])
    kernels.fails = True
    with pytest.raises(moe.MoeError):
        decoder.accept(bt, None)
    assert decoder.lens == [20, 3, 40, 0]  # a call that raises leaves it to be verified
    kernels.fails, kernels.keep = False, {0: 1}
    for most in (0, -1):
        with pytest.raises(ValueError):
            decoder.accept(bt, None, most=most)
    decoder.accept(bt, None)
    for other in (bt, decoder.batch([0, 1, 0, 0])):
        with pytest.raises(ValueError):
            decoder.accept(other, None)
    assert decoder.lens == [19, 4, 40, 0] and len(kernels.moved) == 1


def test_trees_without_nodes(decoder, kernels):
    bt, _ = decoder.tree_batch([[], [], [], []])
    assert decoder.accept(bt, None) == ([[]] * 4, [-1] * 4) and decoder.lens == [18, 3, 40, 0]


def test_a_step_whose_requests_are_all_released_ends(decoder, kernels):
    bt, _ = decoder.tree_batch([[-1, 0], [], [], []])
    decoder.release(0)
    assert decoder.accept(bt, None) == ([[]] * 4, [-1] * 4) and decoder.lens == [0, 3, 40, 0]
    for _ in range(3):  # dropped without a verification: nothing of them is kept
        decoder.tree_batch([[-1, 0], [], [], []])
        decoder.release(0)
    decoder.tree_batch([[], [-1], [], []])
    assert len(decoder.trees) == 1
    with pytest.raises(ValueError):
        decoder.batch([0, 1, 0, 0])
