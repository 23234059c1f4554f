"""The appends with nothing, or nothing that has a place, to append."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests import heads_ref as R

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_steps_without_tokens(qkvp):
    """A step of no tokens with its queries: every tensor of it is empty. Nothing is written."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")          # noqa: E731
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    cs = torch.from_numpy(R.table(100, 64)).cuda()
    pool = torch.full((2, 64, 576), 0x5A, dtype=torch.uint8, device="cuda")
    q.mla_append_rope(bf(0, 512), bf(0, 64), none, none, cs, q.ROPE_PAIRS, pool, None, q.KV_FP8_E4M3, q_pe=bf(0, 16, 64), q=bf(0, 16, 576))
    codes, scale = torch.full((2, 2, 1, 64, 64), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((2, 2, 1), 3.0, device="cuda")
    q.gqa_append_rope(bf(0, 1, 64), bf(0, 1, 64), _i32(0, 0), _i32(5), _i32(0, 2), _i32(0, 1), cs, q.ROPE_HALVES, codes, scale, q.CACHE_E4M3,
                      q=bf(0, 4, 64), q_out=bf(0, 4, 64))
    torch.cuda.synchronize()
    assert (pool == 0x5A).all() and (codes == 0x5A).all() and (scale == 3).all()
