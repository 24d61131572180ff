"""The 8-bit cache on the GPU at the ends of its types: infinities beside the largest numbers, records in which nothing was
written, queries near float32's largest number, values of very different size, and batches most of whose blocks are empty.
Tolerances of attention as in tests/test_gpu_cache8.py unless a test says otherwise."""

import numpy as np
import pytest
import torch

from oracle import cache8
from rotated_bit_kv_iq_b200 import binding as B
from tests.test_gpu_cache8 import BF16, DEV, F16, F32, Held, _check_prefill, _check_rows, _decode, _filled, _i32, _prefill, _tokens  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_bit_kv_iq_b200 import build

    build.build()
    B.lib()


def _codes(h, side, b, head, n, layer=1):
    """The first n tokens' codes as the numbers that they stand for, from the records' bytes."""
    kind = torch.float8_e4m3fn if h.code == "e4m3" else torch.int8
    tiles, out = h.c.tiles()[layer].cpu(), []
    for t in range(n):
        page = b if h.table is None else int(h.table[b, t // h.ps])
        rec, s = tiles[page, head, t % h.ps // 32], t % 32
        row = rec[4096 * side + 128 * s: 4096 * side + 128 * s + 128].view(8, 16)
        out.append(torch.cat([row[c ^ (s & 7)] for c in range(8)]).view(kind).double())
    return torch.stack(out).numpy()


@pytest.mark.parametrize("code", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_append_infinities_beside_the_largest_numbers(code, dtype):
    """An infinity is the largest code of its sign whatever its block's scale: in one block with the type's largest numbers,
    and appended behind them."""
    big = torch.finfo(dtype).max
    h = Held(1, 1, 96, 1, code, contiguous=True)
    x = torch.zeros((1, 70, 1, 128))
    x[0, :, 0, :6] = torch.tensor([big, -big, float("inf"), float("-inf"), float("nan"), 1.0])
    x[0, 1::3, 0, 8:] = torch.tensor([float("inf"), -big, float("-inf"), big / 2, float("inf")]).repeat(24)
    x[0, 40, 0, :] = float("-inf")
    x[0, 69, 0, :] = float("inf")
    x = x.to(dtype)
    h.append(x[:, :50], -x[:, :50], [0])
    h.append(x[:, 50:], -x[:, 50:], [50])
    for side in (0, 1):
        np.testing.assert_array_equal(_codes(h, side, 0, 0, 70), h.o.codes[side, 0, 0, :70])
    assert h.c.status.item() == 0
    h.pool.check("pool")
