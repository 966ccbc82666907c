"""Calls of the paged cache's operators as programs make them: function transforms, other streams, tables with
holes, bounds far from the lengths.  Against the plain 64-bit forms of paged_reference.py, with its bounds."""
from __future__ import annotations

import pytest
import torch

import paged_reference as ref
from test_gpu_paged import put, say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import geometric_map_reduce_amd as gm


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def test_batched_tensors_are_refused():
    """A tensor that torch.vmap batches has no memory of its own: an error in Python, and the calls go on working."""
    say("torch.vmap over q, and over k and v")
    b = ref.Batch(1, [20], [2], 4, 2, 64, 16, junk=0.0)
    q, k, v, table, lens, starts = (put(t) for t in (b.q, b.k, b.v, b.table, b.lens_t(), b.starts))
    want = gm.keops_paged_attention(q, k, v, table, lens, starts, 2, 20)
    rows = q[:, :2].contiguous()
    with pytest.raises((RuntimeError, ValueError)):
        torch.vmap(lambda t: gm.keops_paged_attention(t, k, v, table, lens, starts, 2, 20)[0])(torch.stack([q, q]))
    with pytest.raises((RuntimeError, ValueError)):
        torch.vmap(lambda t: (gm.keops_cache_append(t, t, k, v, table, lens, starts), t)[1])(torch.stack([rows, rows]))
    got = gm.keops_paged_attention(q, k, v, table, lens, starts, 2, 20)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
