"""Page operations over a table that does not agree with its counts."""

import pytest
import torch

from oracle import pages
from rotated_bit_kv_iq_b200 import binding as B
from tests.test_gpu_pages import Both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_bit_kv_iq_b200 import build

    build.build()
    B.lib()


@pytest.mark.parametrize("moves", [True, False])
def test_compaction_leaves_and_flags_entries_of_pages_that_nobody_holds(moves):
    """Entries that name a free page at or above the number of held ones, one below it, or none of the pool stay as they
    are; everything else moves as ever."""
    t = Both(8, 5, 64, 24)
    t.extend([0, 1, 2, 3, 4], [320, 320, 320, 320, 100])  # pages 0..21; the free list stays in the workspace
    t.free([1, 3] if moves else [3, 4])
    t.extend([1] if moves else [], [64] if moves else [])
    t.check()
    held = sum(r > 0 for r in t.o.ref)
    free = [p for p, r in enumerate(t.o.ref) if r <= 0]
    below, above = [p for p in free if p < held], [p for p in free if p >= held]
    assert above and (below or not moves)
    for row, col, p in ((5, 0, above[0]), (5, 4, above[-1]), (6, 1, below[0] if below else above[0]), (6, 3, 24), (7, 2, 10 ** 9)):
        t.pt.block_table[row, col] = p
        t.o.table[row][col] = p
    t.compact()
    assert t.o.status == pages.PAGE
    t.check()
    t.pt.status.zero_()
    t.o.status = 0
    t.compact()  # the entries are still there
    t.check()
    torch.cuda.synchronize()
