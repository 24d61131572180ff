"""Rotary positions of many heads: more items than a CTA takes in one round.  Tolerance as in tests/test_gpu_rope.py."""

import pytest
import torch

from rotated_bit_kv_iq_b200 import binding as B
from tests.test_gpu_rope import BF16, DEV, F16, F32, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("layout,rd", [("interleaved", 128), ("interleaved", 38), ("half", 128), ("half", 64), ("half", 74)])
@pytest.mark.parametrize("hq,hk", [(64, 8), (57, 8), (128, 16), (9, 200)])
def test_rope_of_many_heads(dtype, layout, rd, hq, hk):
    """Heads whose items take several rounds, the last one part-filled; as slices of a fused projection, and in place."""
    freq, ms = B.iq_rope_frequencies(rd, 10000.0, "yarn", 4.0, 4096.0)
    f = torch.from_numpy(freq).to(DEV)
    n, pos = 3, [0, 77, 65535]
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)
    qkv = torch.randn((n, hq + 2 * hk, 128), generator=torch.Generator().manual_seed(hq)).to(dtype).to(DEV)
    keep = qkv.clone()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    qo, ko = torch.full_like(q, 9.0).contiguous(), torch.full_like(k, 9.0).contiguous()
    B.iq_rope(q, k, p, f, qo, ko, layout, ms)
    assert torch.equal(qkv, keep)
    _check(qo, q, pos, freq, layout, ms, False, dtype)
    _check(ko, k, pos, freq, layout, ms, False, dtype)
    B.iq_rope(q, k, p, f, layout=layout, mscale=ms)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, hq + hk:], keep[:, hq + hk:])
