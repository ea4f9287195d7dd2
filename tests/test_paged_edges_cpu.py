"""Sizes at the ends of what the paged and verification calls take (no GPU:
nothing is launched)."""
import pytest
import torch

import block_discrete_diffusion_dd_b200 as dd
from block_discrete_diffusion_dd_b200 import build as libbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return dd.load()


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("batch,total,vocab,fits", [
    (BIG, BIG, 1000, False),        # rows past 2^31
    (BIG, 1, 1, False),
    (1 << 30, 0, 1 << 20, False),   # rows times chunks past 2^31
    (1 << 21, 1 << 20, 1 << 20, True),
    (0, 0, 1, True),
])
def test_verify_workspace_of_the_largest_calls(batch, total, vocab, fits):
    n = dd.verify_draft_workspace_bytes(batch, total, vocab)
    rows, chunks = batch + total, -(-vocab // 4096)
    assert (n >= 8 * rows * chunks) if fits else n == 0


def test_workspaces_whose_elements_overlap_are_refused():
    cpu = torch.device("cpu")
    ws = torch.zeros(512, dtype=torch.uint8)
    dd._own(ws, cpu)
    dd._own(ws[256:], cpu)
    for bad in (ws[:1].expand(4096), ws[::2], ws.int()):
        with pytest.raises(ValueError):
            dd._own(bad, cpu)
