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


@pytest.mark.parametrize("dtype,G,tokens", [("bf16", 4, (4,)), ("bf16", 4, (3,)), ("f32", 8, (2, 0, 1)), ("bf16", 2, (8, 1, 9, 0, 300)),
                                            ("f32", 1, (16, 17))])
def test_weights_where_the_logits_of_some_sequences_are_kept(dtype, G, tokens):
    """Under a table of many entries there is room for the logits of the first sequences alone; the others' are worked
    out again.  Sequences and slots as under a narrow table."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_chunk_attention, fasa_paged_chunk_workspace_size
    B, Hkv, d, page, wide = 64, 8, 64, 16, 4000
    rng = np.random.default_rng(G)
    k = Chunk(dtype, B, Hkv, G, d, page, [int(x) for x in rng.integers(0, 400, B)], [tokens[b % len(tokens)] for b in range(B)],
              seed=62)
    start = k.weight.clone()
    out = k.run().clone()
    rows = min(k.n * G, 16 * B)
    assert rows * Hkv * wide * page * 4 > 480 << 20 > rows * Hkv * (k.cap + 128) * 4
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    table[:, :k.table.shape[1]] = k.table
    weight = torch.zeros((B, Hkv, wide * page), device="cuda")
    weight[:, :, :k.cap] = start
    dims = paged_dims(dtype, B, Hkv, G, d, page, k.kp.shape[0], wide)
    size = fasa_paged_chunk_workspace_size(dims, k.n, True)
    room = torch.full((size + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    fasa_paged_chunk_attention(k.q, k.kp, k.vp, table, k.lens, k.out, cu_new=k.cu, weight=weight, workspace=room[:size],
                               dims=dims)
    assert status() == 0 and torch.equal(k.out, out)
    assert (room[size:] == 0x5a).all()
    # the same logits, summed in another order: 16 u of each exp2, a sum of up to 300 G terms, and u of the weight
    u, got = 2.0 ** -24, (k.weight - start).abs()
    assert ((weight[:, :, :k.cap] - k.weight).abs() <= (32 + max(tokens) * G) * u * got + 8 * u * k.weight + 1e-30).all()
    assert not weight[:, :, k.cap:].any()
