"""Edges of the head-pool plan and of the appends' host checks, without a GPU."""
import numpy as np
import pytest

import quantized_kv_paged_gb300 as q


@pytest.fixture(scope="module")
def lib():
    from quantized_kv_paged_gb300 import build
    build.build()
    return q.load()


LONGEST = 2 ** 31 - 1


@pytest.mark.parametrize("window,sinks,status,pages,tokens", [
    (0, 0, q.QKVP_E_UNSUPPORTED, 0, 0),                       # every page of it is visible: more than the plan addresses
    (1, LONGEST, q.QKVP_E_UNSUPPORTED, 0, 0), (62, LONGEST - 62, q.QKVP_E_UNSUPPORTED, 0, 0),
    (63, LONGEST, q.QKVP_E_UNSUPPORTED, 0, 0), (LONGEST, 0, q.QKVP_E_UNSUPPORTED, 0, 0),
    (1, 0, q.QKVP_OK, 1, 1), (62, 65, q.QKVP_OK, 3, 127), (64, 0, q.QKVP_OK, 2, 64)])
def test_longest_request(lib, window, sinks, status, pages, tokens):
    p = q.gqa_decode_plan(np.array([0, 1 << 25], np.int32), np.array([LONGEST], np.int32), 4, 1, 64, q.CACHE_E4M3, window=window, sinks=sinks,
                          num_sms=4, raise_on_error=False)
    assert p.status == status
    if status == q.QKVP_OK:
        assert (p.total_pages, p.total_tokens) == (pages, tokens)


def test_a_step_without_tokens_may_have_queries(lib):
    """An empty tensor has no address: no tokens, a head count and NULL queries are nothing to do, not a misfit."""
    assert lib.mla_append_rope(None, 512, None, 64, 0, None, None, 16, 9, 1, None, 1024, 64, 16, None, 16, None, 1, 1.0, 64, 4, None) == q.QKVP_OK
    assert lib.gqa_append_rope(None, 256, None, 256, 0, 4, 4, 1, 4, 4, 9, None, 16, 100, 64, 0, 2, 128, 16, 4, 1, 64, 9, None, 512, 4, None,
                               None) == q.QKVP_OK


@pytest.mark.parametrize("name", ["gqa_decode.cu", "append_rope.cu"])
def test_overlapped_kernels_read_by_ordinary_loads(name):
    """Kernels that are resident while the one before them still writes their inputs may not read these through the
    read-only path, whose loads nothing orders behind the wait. No run shows a wrong order reliably; the source does."""
    import os
    from tests.conftest import ROOT
    with open(os.path.join(ROOT, "quantized_kv_paged_gb300", "csrc", name)) as f:
        text = f.read()
    assert "launch_overlapped(" in text and "wait_for_previous()" in text
    assert not [w for w in ("__ldg(", "ldg_nc", "ld.global.nc", "__restrict__") if w in text]


def test_binding_refuses_workspaces_that_are_strided_or_elsewhere(lib):
    """The plan's table is copied on the current device's stream, and the whole byte range from the workspace's start is
    written: a workspace on another device would not be ordered before the run, a strided one would lose its gaps."""
    import torch
    ptr, lens = np.array([0, 2], np.int32), np.array([100], np.int32)
    args = (ptr, lens, 4, 2, 128, q.CACHE_E4M3)
    need = q.gqa_decode_plan(*args, num_sms=4).workspace_bytes
    with pytest.raises(ValueError, match="current CUDA device"):
        q.gqa_decode_plan(*args, num_sms=4, workspace=torch.zeros(need, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        q.gqa_decode_plan(*args, num_sms=4, workspace=torch.zeros(2 * need, dtype=torch.uint8)[::2])
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)          # noqa: E731
    run = dict(plan=q.gqa_decode_plan(*args, num_sms=4), q=bf(1, 4, 128), kv_data=torch.zeros((4, 2, 2, 64, 128), dtype=torch.uint8),
               kv_scale=torch.zeros((4, 2, 2)), kv_indices=torch.zeros(2, dtype=torch.int32), sm_scale=0.1, out=bf(1, 4, 128), lse=None)
    with pytest.raises(ValueError, match="contiguous"):
        q.gqa_decode_run(workspace=torch.zeros(2 * need, dtype=torch.uint8)[::2], **run)
    with pytest.raises(ValueError, match="current CUDA device"):
        q.gqa_decode_run(workspace=torch.zeros(need, dtype=torch.uint8), **run)
