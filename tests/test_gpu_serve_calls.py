"""A step of new tokens over the paged cache on a GPU: calls that are allowed but
seldom made, and what is refused."""

import numpy as np
import pytest

from tests.gpu_util import ensure_built
from tests.test_gpu_serve import Chunk, ints, paged_dims, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    ensure_built()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_without_new_tokens(dtype):
    """Tensors of no rows, with the pages and the statistics: nothing is done, by any of the calls."""
    import torch
    from kv_cache_token_tip_gb300 import FasaRope, fasa_paged_assign, fasa_paged_chunk_attention, fasa_paged_rope_append
    k = Chunk(dtype, 2, 2, 3, 64, 16, [20, 5], [3, 4], seed=61)
    token_pos = torch.full(k.weight.shape, 7, dtype=torch.int32, device="cuda")
    before = [x.clone() for x in (k.kp, k.vp, k.weight, token_pos)]
    none, cu, m = k.q[:0], ints([0, 0, 0]), torch.empty((0, 4), dtype=torch.int32, device="cuda")
    assert none.data_ptr() == 0
    fasa_paged_assign(k.lens, k.lens, k.table, ints([0] * k.kp.shape[0]), ints([0]), ints([0, 0]), cu, m, dims=k.dims)
    rope = FasaRope(1, 64)
    fasa_paged_rope_append(none, none[:, :2], none[:, :2], m, torch.empty_like(none), k.kp, k.vp, weight=k.weight,
                           token_pos=token_pos, rope=rope, dims=k.dims)
    fasa_paged_rope_append(None, none[:, :2], none[:, 2:4], m, None, k.kp, k.vp, rope=rope, dims=k.dims)
    fasa_paged_rope_append(none, None, None, m, none, None, None, rope=rope, dims=k.dims)
    fasa_paged_chunk_attention(none, k.kp, k.vp, k.table, k.lens, torch.empty_like(none), cu_new=cu, weight=k.weight,
                               dims=k.dims)
    assert status() == 0
    assert all(torch.equal(x, y) for x, y in zip((k.kp, k.vp, k.weight, token_pos), before))
