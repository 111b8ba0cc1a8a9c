"""examples/decode_4bit.py: the decode operators together, as a program uses them."""
import os
import sys

import pytest
import torch

from conftest import ROOT
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(gpu):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_4bit
    return decode_4bit


def near(got, want):
    """Logits of the same tokens by calls of other shapes.  Their sums round
    differently, a bf16 activation (2^-8) may land on the other side and a
    cached value on the next E2M1 level (up to a quarter of its size); over two
    layers that stays well under a tenth of the logits' norm, while a token or
    a page read wrongly changes them by their whole size."""
    off = ((got - want).norm() / want.norm()).item()
    assert off < 0.1, off


def test_chunks_steps_and_forks_agree(example):
    announce("decode example")
    ids = torch.randint(0, 2048, (1, 75), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    model = example.Decoder(example.Config())
    whole = model.forward(["whole"], ids)
    parts = torch.cat([model.forward(["parts"], part) for part in ids.split((40, 1, 5, 1, 28), 1)], 1)
    near(parts, whole)
    model.pool.fork("parts", "fork")
    model.pool.truncate("fork", 50)
    again = model.forward(["fork"], ids[:, 50:])  # writes into pages of its own
    near(again, whole[:, 50:])
    both = model.forward(["parts", "fork"], ids[:, :3].expand(2, 3))
    near(both[1], both[0])
    model.pool.free("whole")
    before = model.pool.pages("fork")
    assert model.compact() > 0 and model.pool.pages("fork") != before
    alone = model.forward(["fork"], ids[:, 3:9])
    near(alone, model.forward(["parts"], ids[:, 3:9]))
    assert torch.isfinite(alone).all()


def test_the_program_runs(example, capsys):
    announce("decode example program")
    out = example.main(["--prompt", "70", "--tokens", "5", "--chunk", "33"])
    assert out.shape == (2, 6) and "ms a step" in capsys.readouterr().out
