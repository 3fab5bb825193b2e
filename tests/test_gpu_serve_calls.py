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


BAD_ROWS = [
    # cu_new, the ranges that it gives, and of those the sequences that share no row with another
    ([0, 40, 45, 65, 99], {0: (0, 40), 1: (40, 45), 2: (45, 65)}, (0, 1, 2)),
    ([5, 40, 45, 65, 68], {0: (5, 40), 1: (40, 45), 2: (45, 65), 3: (65, 68)}, (0, 1, 2, 3)),
    ([-1, 40, 45, 65, 68], {1: (40, 45), 2: (45, 65), 3: (65, 68)}, (1, 2, 3)),
    ([0, 40, 30, 65, 68], {0: (0, 40), 2: (30, 65), 3: (65, 68)}, (3,)),
    ([0, 40, 45, 40, 68], {0: (0, 40), 1: (40, 45), 3: (40, 68)}, (0,)),
    ([0, 2 ** 31 - 1, -2 ** 31, 65, 68], {3: (65, 68)}, (3,)),
    ([69, 69, 69, 69, 69], {}, ()),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cu,ranges,alone", BAD_ROWS, ids=["past_the_end", "late", "negative", "back", "back_again", "extreme", "behind"])
def test_rows_that_do_not_ascend(dtype, cu, ranges, alone):
    """What is wrong with some rows is reported; ranges within the call's rows are worked on, as by themselves, the
    others and the rows of none are left as they were.  Rows (and weights) that two ranges claim may hold either's."""
    from oracle import serve_oracle as SO
    from tests.test_gpu_serve import E, U
    k = Chunk(dtype, 4, 2, 2, 64, 16, [100, 60, 30, 30], [40, 5, 20, 3], seed=63)
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run(cu_new=ints(cu))
    assert status() == 1
    out, after, q, kp, vp = k.host(k.out), k.weight.cpu().numpy().astype(np.float64), k.host(k.q), k.host(k.kp), k.host(k.vp)
    claims = np.zeros(k.n, dtype=int)
    for x0, x1 in ranges.values():
        claims[x0:x1] += 1
    assert np.isnan(out[claims == 0]).all() and np.isfinite(out[claims > 0]).all()
    for b in range(4):
        if b not in ranges:
            assert np.array_equal(after[b], before[b])
            continue
        x0, x1 = ranges[b]
        n = int(k.lens[b])
        ref, got, A, pv = SO.chunk_attention(q[x0:x1], [0, x1 - x0], kp, vp, k.table[b:b + 1].cpu().numpy(), [n])
        rel = 2 * (2 * k.d + 16) * U * A + (16 + n + 64) * U
        bound = (rel + (2.0 ** -8 if dtype == "bf16" else 0.0) + 2 * (n + 64) * U)[..., None] * pv + E[dtype] * np.abs(ref)
        mine = claims[x0:x1] == 1
        assert np.all(np.abs(out[x0:x1] - ref)[mine] <= bound[mine] + 1e-30), b
        if b in alone:
            lim = (rel.max() + ((x1 - x0) * k.G + 64) * U) * got[0] + 2 * U * (before[b] + got[0])
            assert np.all(np.abs(after[b] - before[b] - got[0]) <= lim), b


def test_statistics_of_no_keys_are_refused():
    """With the queries or without: the statistics begin as keys are stored."""
    import torch
    from kv_cache_token_tip_gb300 import FasaError, FasaRope, fasa_paged_rope_append
    k = Chunk("bf16", 2, 2, 2, 64, 16, [20, 30], [4, 5], seed=64)
    m, rope = torch.full((9, 4), -1, dtype=torch.int32, device="cuda"), FasaRope(1, 64)
    token_pos = torch.zeros(k.weight.shape, dtype=torch.int32, device="cuda")
    for q, out in ((None, None), (k.q, torch.empty_like(k.q))):
        for kw in (dict(weight=k.weight), dict(token_pos=token_pos), dict(weight=k.weight, token_pos=token_pos)):
            with pytest.raises(FasaError):
                fasa_paged_rope_append(q, None, None, m, out, None, None, rope=rope, dims=k.dims, **kw)
        fasa_paged_rope_append(q, None, None, m, out, None, None, rope=rope, dims=k.dims)
    assert status() == 0


def test_chunk_queries_that_are_no_tensor_are_refused():
    from kv_cache_token_tip_gb300 import fasa_paged_chunk_attention
    k = Chunk("bf16", 2, 2, 2, 64, 16, [20, 30], [4, 5], seed=65)
    for bad in (None, 3, [1.0]):
        with pytest.raises(ValueError):
            fasa_paged_chunk_attention(bad, k.kp, k.vp, k.table, k.lens, k.out, cu_new=k.cu, dims=k.dims)
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_alone_and_in_a_batch(dtype):
    """The batch around a sequence moves the cuts of its work: by itself it gives the same within the rounding, though
    not the same bits, and each of the two the same bits again."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_chunk_attention
    from tests.test_gpu_serve import E, U
    k = Chunk(dtype, 4, 2, 4, 128, 32, [700, 20, 3000, 0], [90, 300, 40, 2], seed=66)
    start = k.weight.clone()
    before = start.cpu().numpy().astype(np.float64)
    out = k.run().clone()
    k.check(before)
    weight = k.weight.clone()
    k.weight.copy_(start)
    assert torch.equal(k.run(), out) and torch.equal(k.weight, weight)
    dims = paged_dims(dtype, 1, 2, 4, 128, 32, k.kp.shape[0], k.table.shape[1])
    for b in range(4):
        x0, x1, n = k.cu_host[b], k.cu_host[b + 1], int(k.lens[b])
        alone, again, w = torch.empty_like(k.q[x0:x1]), torch.empty_like(k.q[x0:x1]), start[b:b + 1].clone()
        for to in (alone, again):
            w.copy_(start[b:b + 1])
            fasa_paged_chunk_attention(k.q[x0:x1], k.kp, k.vp, k.table[b:b + 1], k.lens[b:b + 1], to,
                                       cu_new=ints([0, x1 - x0]), weight=w, dims=dims)
        assert torch.equal(alone, again)
        # sums of n terms in another order (2 u a term at most), maxima that lag elsewhere (bf16: other roundings of P),
        # and the result's rounding, of results below 8 (values and weights' sums of 1)
        err = (alone.double() - out[x0:x1].double()).abs().max()
        assert float(err) <= 8 * (2 * n * U + 64 * U + 2 * E[dtype] + (2.0 ** -7 if dtype == "bf16" else 0))
        got = (weight[b] - start[b]).double()
        lim = (2 * n + 64 + (x1 - x0) * 4) * U * got.abs() + 4 * U * weight[b].double() + 1e-30
        assert ((w[0] - weight[b]).double().abs() <= lim).all()
    assert status() == 0
