"""The attention of chunks where keys, logits and values are not finite, against the
fp64 oracle on the same stored values.

Bounds as in test_gpu_serve.py; the logits' scale A is that of the finite elements: a
logit of -inf or NaN is exact.
"""

import numpy as np
import pytest

from oracle import serve_oracle as SO
from tests.gpu_util import ensure_built
from tests.test_gpu_serve import E, U, Chunk, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    ensure_built()


def key(k, b, h, slot):
    """A slot's key, to be written."""
    return k.kp[k.table[b, slot // k.page].long(), h, slot % k.page]


def check(k, before):
    """out and the weights, NaN where the definition gives NaN and nowhere else."""
    lens, table = k.lens.cpu().numpy(), k.table.cpu().numpy()
    q, kp, vp = k.host(k.q), k.host(k.kp), k.host(k.vp)
    with np.errstate(invalid="ignore"):
        ref, got, _, pv = SO.chunk_attention(q, k.cu_host, kp, vp, table, lens)
    _, _, A, _ = SO.chunk_attention(q, k.cu_host, np.where(np.isfinite(kp), kp, 0.0), vp, table, lens)
    T = np.zeros((k.n, 1))
    for b in range(k.B):
        T[k.cu_host[b]:k.cu_host[b + 1]] = lens[b]
    rel = 2 * (2 * k.d + 16) * U * A + (16 + T + 64) * U
    bound = (rel + (2.0 ** -8 if k.dtype == "bf16" else 0.0) + 2 * (T + 64) * U)[..., None] * pv + E[k.dtype] * np.abs(ref)
    out = k.host(k.out)
    assert np.array_equal(np.isnan(out), np.isnan(ref))
    fine = ~np.isnan(ref)
    assert np.all(np.abs(out - ref)[fine] <= bound[fine] + 1e-30)
    after, want = k.weight.cpu().numpy().astype(np.float64), before + got
    assert np.array_equal(np.isnan(after), np.isnan(want))
    for b in range(k.B):
        x0, x1 = k.cu_host[b], k.cu_host[b + 1]
        relw = (rel[x0:x1].max() if x1 > x0 else 0.0) + ((x1 - x0) * k.G + 64) * U
        fine = ~np.isnan(want[b])
        lim = relw * got[b][fine] + 2 * U * np.abs(want[b][fine])
        assert np.all(np.abs(after[b] - want[b])[fine] <= lim)
        none = got[b] == 0
        assert np.array_equal(after[b][none], before[b][none])
    return ref, got


# dtype, B, Hkv, G, d, page, tokens before, new tokens: few rows (their logits are kept), rows that are no
# multiple of a warp's, more rows than a tile's, caches that are cut into parts
CASES = [("f32", 2, 2, 1, 64, 16, [40, 90], [17, 31]), ("f32", 1, 1, 4, 128, 32, [200], [5]), ("f32", 1, 2, 3, 64, 64, [7], [9]),
         ("f32", 2, 1, 1, 128, 16, [64, 700], [130, 19]), ("f32", 1, 2, 4, 64, 16, [300], [3]), ("f32", 1, 1, 8, 64, 16, [3000], [20]),
         ("bf16", 2, 2, 1, 64, 16, [40, 90], [17, 31]), ("bf16", 1, 1, 4, 128, 32, [200], [5]), ("bf16", 1, 2, 3, 64, 64, [7], [9]),
         ("bf16", 2, 1, 1, 128, 16, [64, 700], [300, 19]), ("bf16", 1, 2, 4, 64, 16, [300], [3]), ("bf16", 1, 1, 8, 128, 16, [3000], [40])]
NAMES = [f"{c[0]}-B{c[1]}h{c[2]}g{c[3]}d{c[4]}-{max(c[6])}+{max(c[7])}" for c in CASES]


@pytest.mark.parametrize("c", CASES, ids=NAMES)
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_keys_of_no_weight(c, sign):
    """An infinite element of a key that all rows see, their queries of the other sign there: the logit is -inf, its
    weight 0, and everything else as if the slot were not there."""
    k = Chunk(*c, seed=51)
    dim, inf = k.d // 2 + 1, float("inf")
    k.q[:, :, dim] = -sign * (k.q[:, :, dim].abs() + 0.25)
    for b in range(k.B):
        for h in range(k.Hkv):
            key(k, b, h, 3 + h)[dim] = sign * inf
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run()
    ref, got = check(k, before)
    assert np.all(np.isfinite(ref)) and np.all(np.isfinite(got)) and np.all(got[:, 0, 3] == 0)
    assert status() == 0


@pytest.mark.parametrize("c", CASES, ids=NAMES)
def test_an_infinite_logit(c):
    """One token's head has a logit of +inf (the others -inf there): its row is NaN, and so are the weights of all slots
    that it sees, of its KV head; those behind them are not."""
    k = Chunk(*c, seed=52)
    dim, b, h, inf = k.d // 2 + 1, k.B - 1, k.Hkv - 1, float("inf")
    n = k.cu_host[b + 1] - k.cu_host[b]
    j = n // 3
    k.q[:, :, dim] = -(k.q[:, :, dim].abs() + 0.25)
    k.q[k.cu_host[b] + j, h * k.G + k.G // 2, dim] = 0.5
    key(k, b, h, 2)[dim] = inf
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run()
    ref, got = check(k, before)
    rows = np.isnan(ref).all(axis=2)
    assert rows.sum() == 1 and rows[k.cu_host[b] + j, h * k.G + k.G // 2]
    see = int(k.lens[b]) - n + j + 1
    assert np.isnan(got[b, h, :see]).all() and not np.isnan(got[b, h, see:]).any() and np.isnan(got).sum() == see
    assert status() == 0


@pytest.mark.parametrize("c", CASES, ids=NAMES)
def test_weights_of_a_key_that_is_nan(c):
    """A new token's key is NaN in one head: the rows that see it give NaN, out and weights, in that head alone."""
    k = Chunk(*c, seed=53)
    b, h = k.B - 1, 0
    n = k.cu_host[b + 1] - k.cu_host[b]
    start = k.weight.clone()
    k.run()
    first = k.weight.clone()
    k.weight.copy_(start)
    key(k, b, h, int(k.lens[b]) - n + n // 2)[:] = float("nan")
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run()
    ref, got = check(k, before)
    assert np.isnan(got[b, h, :int(k.lens[b])]).all() and np.isnan(got).sum() == int(k.lens[b])
    for i in range(k.B):
        for g in range(k.Hkv):
            if (i, g) != (b, h):
                assert bool((k.weight[i, g] == first[i, g]).all())
    assert status() == 0


@pytest.mark.parametrize("dtype,G,d", [("bf16", 4, 128), ("bf16", 1, 64), ("f32", 4, 64), ("f32", 2, 128)])
def test_infinite_values_in_a_cache_that_is_cut(dtype, G, d):
    """An early slot's logits lie hundreds of powers of two above all others', so that the weight of a new token's value,
    in another part of the cache, is below the smallest number: an infinite or NaN value reaches the rows that see it
    all the same, whatever lies in between, and no others."""
    import torch
    have, new, page, inf = 8000, 12, 32, float("inf")
    k = Chunk(dtype, 1, 2, G, d, page, [have], [new], seed=54)
    h, dim = 1, d // 2 + 5
    k.q[..., 0] = 40.0
    for slot in (10, 11):  # 40 * 100 / sqrt(d) >= 350 against a few times ten
        key(k, 0, 0, slot)[0] = 100.0
        key(k, 0, h, slot)[0] = 100.0
    clean = k.run(False).clone()
    assert torch.isfinite(clean).all()
    pool = k.vp.clone()
    rows = torch.arange(new, device="cuda")
    for j in (1, new // 2, new - 1):
        for bad in (inf, -inf, float("nan")):
            k.vp = pool.clone()
            k.vp[k.table[0, (have + j) // page].long(), h, (have + j) % page, dim] = bad
            out = k.run(False).clone()
            want = clean.clone()
            want[rows >= j, h * G:(h + 1) * G, dim] = bad
            same = (out == want) | (torch.isnan(out) & torch.isnan(want))
            assert same.all(), (j, bad, int((~same).sum()))
    assert status() == 0


@pytest.mark.parametrize("c", CASES, ids=NAMES)
def test_logits_that_are_all_minus_infinity(c):
    """Rows of which no slot counts give zeros, and nothing to the weights."""
    k = Chunk(*c, seed=55)
    dim = k.d // 2 + 1
    k.q[:, :, dim] = -(k.q[:, :, dim].abs() + 0.25)
    k.kp[..., dim] = float("inf")
    before = k.weight.clone()
    k.run()
    assert not k.out.any() and bool((k.weight == before).all())
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,d,new", [(1, 64, 300), (3, 128, 100), (4, 64, 70), (5, 64, 60), (7, 128, 41), (8, 64, 33), (3, 64, 5)])
def test_infinite_keys_of_new_tokens(dtype, G, d, new):
    """A new token's key is infinite in an element where the queries before it have its sign (a logit of +inf, did they
    see it) and those from it on the other: no row and no slot gives anything but numbers."""
    import torch
    TU = 128 // G
    for j in sorted({1, new // 2, new - 1} | {x for t in (TU, 2 * TU) for x in (t - 1, t, t + 1) if 0 < x < new}):
        k = Chunk(dtype, 2, 2, G, d, 16, [50, 9], [new, 20], seed=56, pad=3)
        dim = d // 2 + 1
        q = k.q[:new, :, dim].abs() + 0.25
        k.q[:new, :, dim] = torch.where(torch.arange(new, device="cuda").view(-1, 1) < j, q, -q)
        key(k, 0, 1, 50 + j)[dim] = float("inf")
        k.q[-3:] = float("nan")
        before = k.weight.cpu().numpy().astype(np.float64)
        k.run()
        live = k.cu_host[-1]
        k.q[live:] = 0  # (rows of no sequence: zeros in the reference, too)
        k.out[live:] = 0
        ref, got = check(k, before)
        assert np.isfinite(ref).all() and np.isfinite(got).all() and np.all(got[0, 1, 50 + j] == 0)
    assert status() == 0
