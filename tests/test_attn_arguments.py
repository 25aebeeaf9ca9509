"""What the attention half's binding refuses before the library is called, on the CPU."""
import pytest
import torch

from serving_router_top_gb300 import moe

BF = torch.bfloat16


@pytest.fixture
def no_call(monkeypatch):
    """Any call of the library fails the test: the arguments have to be refused before it."""
    def load():
        raise AssertionError("the library was called")
    monkeypatch.setattr(moe, "load", load)
    monkeypatch.setattr(moe, "_stream", lambda stream: None)


def apart(t):
    """The same shape and type with columns two elements apart."""
    return torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]


def test_norm_columns_are_contiguous(no_call):
    x, y = torch.zeros(3, 64), torch.zeros(3, 64, dtype=BF)
    d = moe.block_norm_desc(y=y)
    for rows in [(apart(x), x, y), (x, apart(x), y), (x, x, apart(y)), (torch.zeros(64, 3).t(), x, y)]:
        with pytest.raises(ValueError):
            moe.moe_block_norm(d, *rows, 3, 64)
