"""A step of new tokens over the paged cache on a GPU: pages assigned, queries and
keys turned and stored, attention of chunks, against the fp64 oracle on the same
stored values.

Tolerances (u = 2^-24, the half step of fp32, e the stored type's: bf16 2^-8, fp32
2^-24; derived, not fitted):
  * assignments are whole numbers: exact;
  * a turned element: 2e-6 of its pair's norm (the angle in turns rounds to 2^-25 of
    a half turn, cos and sin to 2 ulp, their product with the magnitude, two products
    and a sum) plus e of its value;
  * a logit z (natural units): an fp32 sum of d products, which the tensor cores round
    towards zero (2 u each), and its scaling to powers of two: |dz| <= (2 d + 16) u A
    with A = sum |q| |k| / sqrt(d);
  * a softmax weight: relative 2 max |dz|, 16 u of exp2 and the divisions, and
    (T + 64) u for a sum of T terms in any order;
  * out: that relative error and, for bf16, the 2^-8 of the weight that multiplies V,
    times sum p |V|; a sum of T terms at 2 u each; e of its value;
  * a weight: that relative error of what it receives, (n G + 64) u for the sum over
    the queries, and 2 u of its new value.
"""

import numpy as np
import pytest

from oracle import serve_oracle as SO
from tests.gpu_util import ensure_built
from tests.parity import host_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    ensure_built()


def status():
    from kv_cache_token_tip_gb300 import fasa_device_status
    return fasa_device_status()


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def paged_dims(dtype, B, Hkv, G, d, page, n_pages, max_pages, theta=1e4):
    from kv_cache_token_tip_gb300 import FASA_BF16, FASA_F32, FasaPagedDims
    return FasaPagedDims(B, Hkv * G, Hkv, d, page, n_pages, max_pages, FASA_F32 if dtype == "f32" else FASA_BF16, theta)


# ------------------------------------------------------------------- assign
class Pool:
    """A table, a list of free pages and lengths, seeded."""

    def __init__(self, have, page, max_pages, free, seed=0, spare=4):
        rng = np.random.default_rng(seed)
        self.page, self.B = page, len(have)
        held = [-(-h // page) for h in have]
        self.n_pages = sum(held) + free + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((self.B, max_pages), -7, dtype=np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.free = np.full(self.n_pages, -9, dtype=np.int32)
        self.free[:free] = order[at:at + free]
        self.count, self.have, self.max_pages = free, have, max_pages

    def run(self, want, max_tokens, pos=None, in_place=False, stream=None):
        """The call's outputs, checked against the oracle's."""
        import torch
        from kv_cache_token_tip_gb300 import fasa_paged_assign
        dims = paged_dims("bf16", self.B, 2, 2, 64, self.page, self.n_pages, self.max_pages)
        have, wanted, table, free, count = ints(self.have), ints(want), ints(self.table), ints(self.free), ints([self.count])
        lens = have if in_place else ints([-5] * self.B)
        left = None if in_place else ints([-5])
        cu, m = ints([-5] * (self.B + 1)), torch.full((max_tokens, 4), -5, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        fasa_paged_assign(have, wanted, table, free, count, lens, cu, m, pos=None if pos is None else ints(pos),
                          free_count_out=left, dims=dims, stream=stream)
        torch.cuda.synchronize()
        ref_t, ref_f = self.table.copy(), self.free.copy()
        ref = SO.assign(self.have, want, pos, ref_t, ref_f, self.count, max_tokens, self.page)
        assert lens.tolist() == ref[0]
        assert cu.tolist() == ref[1]
        assert np.array_equal(m.cpu().numpy().reshape(-1, 4), np.array(ref[2], dtype=np.int64).reshape(-1, 4))
        assert (count if in_place else left).item() == ref[3]
        assert np.array_equal(table.cpu().numpy(), ref_t)
        assert np.array_equal(free.cpu().numpy(), ref_f)
        self.table, self.free, self.count, self.have = ref_t, ref_f, ref[3], ref[0]
        return ref


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("B,page,hi,new,tokens", [
    (1, 16, 0, 1, 1), (1, 256, 300, 0, 5), (3, 16, 40, 20, 64), (64, 16, 500, 1, 64), (33, 32, 100, 90, 4096),
    (33, 64, 100, 300, 10000), (700, 16, 60, 30, 20000), (1500, 16, 40, 3, 1500), (2048, 16, 20, 12, 4097),
    (2048, 128, 200, 40, 60000)])
def test_assign(B, page, hi, new, tokens, in_place):
    """Sequences that grow, shrink, end and stay, with and without enough pages and rows."""
    rng = np.random.default_rng(B + new)
    have = [int(x) for x in rng.integers(0, hi + 1, B)]
    max_pages = -(-(hi + 4 * new + 1) // page)
    for free in (0, B // 3, 4 * B * (new // page + 2)):
        p = Pool(have, page, max_pages, free, seed=free)
        for _ in range(3):
            grow = rng.integers(0, new + 1, B)
            want = np.where(rng.random(B) < 0.2, rng.integers(0, np.array(p.have) + 1), np.array(p.have) + grow)
            want = [int(min(x, max_pages * page)) for x in want]
            pos = [int(x) for x in rng.integers(0, 1 << 20, B)]
            p.run(want, tokens, pos=pos if free else None, in_place=in_place)
    assert status() == 0


def test_assign_takes_back_what_the_same_call_gives():
    p = Pool([64, 0, 48, 0], 16, 8, 1)
    lens, cu, rows, left = p.run([0, 70, 16, 30], 200)
    assert lens == [0, 70, 16, 30] and left == 0
    assert status() == 0


def test_assign_serves_in_order_until_one_does_not_fit():
    p = Pool([16, 16, 16, 16], 16, 8, 3)
    lens, cu, _, left = p.run([17, 80, 17, 16], 500)   # one page, four, one: the second does not fit
    assert lens == [17, 16, 16, 16] and cu == [0, 1, 1, 1, 1] and left == 2
    p = Pool([5, 5, 5, 5], 16, 8, 3)
    lens, cu, _, left = p.run([8, 12, 6, 2], 9)        # ten tokens for nine rows; no page needed
    assert lens == [8, 5, 5, 2] and left == 3
    assert status() == 0


def test_assign_no_tokens_and_no_rows():
    p = Pool([20, 0, 33], 16, 8, 3)
    assert p.run([20, 0, 33], 7)[0] == [20, 0, 33]
    assert p.run([21, 0, 3], 0)[0] == [20, 0, 3]
    assert status() == 0


def test_assign_bad_values_are_reported():
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_assign

    def call(have, want, table, free, count, n_pages, page=16):
        B, mp = len(have), len(table[0])
        dims = paged_dims("bf16", B, 2, 2, 64, page, n_pages, mp)
        t, f, lens, cu, m, left = ints(table), ints(free), ints([0] * B), ints([0] * (B + 1)), ints([[0] * 4] * 40), ints([0])
        fasa_paged_assign(ints(have), ints(want), t, f, ints([count]), lens, cu, m, free_count_out=left, dims=dims)
        torch.cuda.synchronize()
        return lens.tolist(), left.item(), t.tolist(), f.tolist()

    assert call([-3], [5], [[9, 9]], [0, 1, 2], 3, 3) == ([5], 2, [[2, 9]], [0, 1, 2]) and status() == 1
    assert call([3], [5000], [[2, 9]], [0, 1, 2], 3, 3)[0] == [32] and status() == 1
    assert call([0], [5], [[9, 9]], [0, 1, 2], 99, 3)[1] == 2 and status() == 1
    assert call([0], [5], [[9, 9]], [0, 1, 2], -1, 3) == ([0], 0, [[9, 9]], [0, 1, 2]) and status() == 1
    # a page outside the pool comes back, or goes out: as it is
    assert call([20], [0], [[1, 77]], [5, 5, 5], 0, 3) == ([0], 2, [[1, 77]], [1, 77, 5]) and status() == 1
    assert call([0], [5], [[9, 9]], [0, 1, -4], 3, 3)[2] == [[-4, 9]] and status() == 1
    # more pages than the list can hold
    assert call([20], [0], [[1, 2]], [0, 1, 2], 2, 3) == ([0], 3, [[1, 2]], [0, 1, 1]) and status() == 1


# -------------------------------------------------------------- rope_append
def ropes(d):
    from kv_cache_token_tip_gb300 import FasaRope
    return [FasaRope(0, d, 0, 1e4), FasaRope(1, d, 0, 5e5), FasaRope(1, d // 2, 1, 1e6, factor=4.0),
            FasaRope(0, 16, 1, 1e4, factor=2.0), FasaRope(1, d, 2, 5e5, factor=8.0, low=1.0, high=4.0, original=8192.0),
            FasaRope(0, d, 2, 1e4, factor=3.0, low=0.5, high=6.0, original=1024.0, magnitude=0.7),
            FasaRope(1, 48, 3, 1e6, factor=4.0, low=1.0, high=32.0, original=4096.0, magnitude=1.1386294361119891),
            FasaRope(0, d, 3, 1e4, factor=16.0, low=1.0, high=1.0001, original=2048.0)]


def _check_rope(dtype, B, Hkv, G, d, page, n_tok, rope, seed, fused=True, pad=3, q_only=False, kv_only=False):
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_rope_append
    rng = np.random.default_rng(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    max_pages = max(1, -(-(n_tok // B + 2) // page) + 1)
    n_pages, cap = B * max_pages + 2, max_pages * page
    table = rng.permutation(n_pages)[:B * max_pages].reshape(B, max_pages)
    slots = {(b, t) for b in range(B) for t in range(cap)}
    chosen = [sorted(slots)[i] for i in rng.choice(len(slots), n_tok, replace=False)]
    m = [(b, t, int(table[b, t // page]), int(rng.integers(0, 1 << int(rng.integers(1, 31))))) for b, t in chosen]
    m = [(-1,) * 4] + m + [(-1,) * 4] * (pad - 1) if pad else m
    n = len(m)
    Hq = Hkv * G
    big = torch.randn((n, Hq + 2 * Hkv, d), generator=g, device="cuda").to(dt)
    q, k, v = big[:, :Hq], big[:, Hq:Hq + Hkv], big[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    kp, vp = (torch.randn((n_pages, Hkv, page, d), generator=g, device="cuda").to(dt) for _ in range(2))
    w, tp = torch.rand((B, Hkv, cap), generator=g, device="cuda"), torch.full((B, Hkv, cap), -3, dtype=torch.int32, device="cuda")
    q_out = torch.randn((n, Hq, d), generator=g, device="cuda").to(dt)
    dims = paged_dims(dtype, B, Hkv, G, d, page, n_pages, max_pages)
    host = lambda x: host_f64(x.contiguous(), dtype)
    rq, rk, rv, rqo = host(q), host(k), host(v), host(q_out)
    rkp, rvp, rw, rtp = host(kp), host(vp), w.cpu().numpy().astype(np.float64), tp.cpu().numpy()
    SO.rope_append(None if kv_only else rq, None if q_only else rk, rv, m, rqo, rkp, rvp, rw, rtp, rope)
    args = [None if kv_only else q, None if q_only else k, None if q_only else v, ints(m), None if kv_only else q_out,
            None if q_only else kp, None if q_only else vp]
    fasa_paged_rope_append(*args, weight=None if q_only else w, token_pos=None if q_only else tp, rope=rope, dims=dims)
    assert status() == 0

    def close(got, ref, live, pairs_of):
        """live: rows that were turned, with their pairs' norms."""
        err = np.abs(host(got) - ref)
        bound = E[dtype] * np.abs(ref) + 2e-6 * pairs_of
        assert np.all(err[live] <= bound[live] + 1e-30), np.max(err[live] / (bound[live] + 1e-30))
        assert np.array_equal(host(got)[~live], ref[~live])

    def norms(x):  # every element's pair's
        r = rope.rotary_dim
        y = np.zeros(x.shape)
        i = np.arange(r // 2) if rope.layout == 1 else 2 * np.arange(r // 2)
        j = i + r // 2 if rope.layout == 1 else i + 1
        y[..., i] = y[..., j] = np.hypot(x[..., i], x[..., j])
        return y

    live = np.array([x[0] >= 0 for x in m])
    close(q_out, rqo, live & (not kv_only), norms(rqo))
    at = np.zeros((n_pages, page), dtype=bool)
    for b, t, pg, _ in (m if not q_only else []):
        if b >= 0:
            at[pg, t % page] = True
    rows = np.broadcast_to(at[:, None], (n_pages, Hkv, page))
    close(kp, rkp, rows, norms(rkp))
    assert np.array_equal(host(vp), rvp)
    assert np.array_equal(w.cpu().numpy().astype(np.float64), rw) and np.array_equal(tp.cpu().numpy(), rtp)
    # elements behind the turned part are copied
    r = rope.rotary_dim
    assert np.array_equal(host(q_out)[..., r:][live], (rqo if kv_only else rq)[..., r:][live])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", range(8))
def test_rope_append(dtype, d, kind):
    _check_rope(dtype, 3, 2, 3, d, 16, 40, ropes(d)[kind], seed=kind)


@pytest.mark.parametrize("dtype,B,Hkv,G,d,page,n,kw", [
    ("bf16", 1, 1, 1, 64, 16, 1, dict(pad=0)), ("f32", 1, 1, 1, 128, 256, 1, dict(pad=0, fused=False)),
    ("bf16", 2, 8, 4, 128, 64, 33, {}), ("bf16", 2, 4, 7, 128, 32, 17, dict(fused=False)),
    ("f32", 5, 3, 5, 64, 16, 29, {}), ("bf16", 2, 5, 3, 64, 16, 13, {}), ("f32", 2, 8, 8, 128, 16, 9, {}),
    ("bf16", 2, 2, 2, 128, 16, 20, dict(q_only=True)), ("bf16", 2, 2, 2, 128, 16, 20, dict(kv_only=True)),
    ("f32", 2, 1, 2, 64, 128, 20, dict(kv_only=True, fused=False)),
    ("bf16", 7, 1, 2, 64, 64, 4200, {}), ("f32", 3, 1, 1, 64, 16, 4100, dict(fused=False))])
def test_rope_append_shapes(dtype, B, Hkv, G, d, page, n, kw):
    _check_rope(dtype, B, Hkv, G, d, page, n, ropes(d)[1 + n % 6], seed=n, **kw)


def test_rope_append_in_place_and_attention_of_turned_queries():
    """q_out may be q; positions of 0 turn nothing, so that the attention of single tokens takes turned queries."""
    import torch
    from kv_cache_token_tip_gb300 import FasaRope, fasa_paged_attention, fasa_paged_rope_append
    dims = paged_dims("bf16", 2, 2, 4, 128, 16, 4, 2)
    q = torch.randn((2, 8, 128), device="cuda").bfloat16()
    m = ints([(0, 3, 1, 1234567), (1, 0, 2, 77)])
    rope = FasaRope(1, 128, 2, 5e5, factor=8.0)
    apart = torch.zeros_like(q)
    fasa_paged_rope_append(q, None, None, m, apart, None, None, rope=rope, dims=dims)
    fasa_paged_rope_append(q, None, None, m, q, None, None, rope=rope, dims=dims)
    assert torch.equal(q, apart)
    kp, vp = torch.randn((2, 4, 2, 16, 128), device="cuda").bfloat16()
    table, lens, zero = ints([[1, 3], [2, 0]]), ints([30, 7]), ints([0, 0])
    out = torch.zeros((2, 8, 128), device="cuda")
    fasa_paged_attention(q, zero, kp, vp, table, lens, out, dims=dims)
    ref, _, A, pv = SO.chunk_attention(host_f64(q, "bf16"), [0, 1, 2], host_f64(kp, "bf16"), host_f64(vp, "bf16"),
                                       table.cpu().numpy(), [30, 7])
    rel = 2 * (2 * 128 + 16) * U * A[..., None] + 2.0 ** -16 + (30 + 80) * U
    assert np.all(np.abs(out.cpu().numpy() - ref) <= (rel + 100 * U) * pv)
    assert status() == 0


def test_rope_append_bad_entries_are_left_out():
    import torch
    from kv_cache_token_tip_gb300 import FasaRope, fasa_paged_rope_append
    dims = paged_dims("bf16", 2, 2, 1, 64, 16, 4, 2)
    for bad in [(2, 0, 0, 0), (0, 32, 0, 0), (0, -1, 0, 0), (0, 0, 4, 0), (0, 0, -1, 0), (1 << 30, 0, 0, 0)]:
        x = torch.ones((2, 2, 64), device="cuda").bfloat16()
        kp, vp, qo = (torch.zeros(s, device="cuda").bfloat16() for s in ((4, 2, 16, 64), (4, 2, 16, 64), (2, 2, 64)))
        w, tp = torch.ones((2, 2, 32), device="cuda"), torch.ones((2, 2, 32), dtype=torch.int32, device="cuda")
        fasa_paged_rope_append(x, x, x, ints([bad, (1, 5, 2, 0)]), qo, kp, vp, weight=w, token_pos=tp,
                               rope=FasaRope(1, 64), dims=dims)
        assert status() == 1
        assert qo[0].abs().sum() == 0 and torch.equal(qo[1], x[1])
        assert kp.sum() == 128 and vp.sum() == 128 and torch.equal(kp[2, :, 5], x[1])
        assert w.sum() == 126 and tp.sum() == 126


# ---------------------------------------------------------- chunk attention
class Chunk:
    def __init__(self, dtype, B, Hkv, G, d, page, have, new, seed=0, sigma=1.0, max_pages=None, pad=0, spare=3):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.dtype, self.B, self.Hkv, self.G, self.d, self.page = dtype, B, Hkv, G, d, page
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        lens = [h + n for h, n in zip(have, new)]
        max_pages = max_pages or max(1, -(-max(lens) // page))
        self.cap = max_pages * page
        n_pages = B * max_pages + spare
        self.cu_host = [sum(new[:b]) for b in range(B + 1)]
        self.n = self.cu_host[-1] + pad

        def normal(*s):
            return torch.randn(s, generator=g, device="cuda")

        self.table = torch.randperm(n_pages, generator=g, device="cuda")[:B * max_pages].to(torch.int32).view(
            B, max_pages).contiguous()
        self.lens, self.cu = ints(lens), ints(self.cu_host)
        self.kp, self.vp = normal(n_pages, Hkv, page, d).to(dt), normal(n_pages, Hkv, page, d).to(dt)
        self.q = (sigma * normal(self.n, Hkv * G, d)).to(dt)
        self.weight = torch.exp(normal(B, Hkv, self.cap))
        self.out = torch.full((self.n, Hkv * G, d), float("nan"), device="cuda").to(dt)
        self.dims = paged_dims(dtype, B, Hkv, G, d, page, n_pages, max_pages)

    def host(self, x):
        return host_f64(x, self.dtype)

    def run(self, weights=True, **kw):
        from kv_cache_token_tip_gb300 import fasa_paged_chunk_attention
        kw.setdefault("cu_new", self.cu)
        fasa_paged_chunk_attention(self.q, self.kp, self.vp, self.table, self.lens, self.out,
                                   weight=self.weight if weights else None, dims=self.dims, **kw)
        return self.out

    def check(self, before=None, lens=None, table=None):
        """out, and the weights where `before` (numpy) is what they were."""
        lens = self.lens.cpu().numpy() if lens is None else lens
        table = self.table.cpu().numpy() if table is None else table
        ref, got, A, pv = SO.chunk_attention(self.host(self.q), self.cu_host, self.host(self.kp), self.host(self.vp),
                                             table, lens)
        T = np.zeros((self.n, 1))
        for b in range(self.B):
            T[self.cu_host[b]:self.cu_host[b + 1]] = min(max(int(lens[b]), 0), self.cap)
        out = self.host(self.out)
        live = np.arange(self.n) < self.cu_host[-1]
        rel = 2 * (2 * self.d + 16) * U * A + (16 + T + 64) * U  # [n, Hq]
        round_p = 2.0 ** -8 if self.dtype == "bf16" else 0.0
        bound = (rel + round_p + 2 * (T + 64) * U)[..., None] * pv + E[self.dtype] * np.abs(ref)
        assert np.all(np.isfinite(out[live]))
        assert np.all(np.isnan(out[~live]))  # padding is left as it was
        err = np.abs(out - ref)[live]
        assert np.all(err <= bound[live] + 1e-30), f"out: {np.max(err / (bound[live] + 1e-30)):.3g}x the bound"
        if before is not None:
            after, want = self.weight.cpu().numpy().astype(np.float64), before + got
            for b in range(self.B):
                x0, x1 = self.cu_host[b], self.cu_host[b + 1]
                relw = (rel[x0:x1].max() if x1 > x0 else 0.0) + ((x1 - x0) * self.G + 64) * U
                err = np.abs(after[b] - want[b])
                lim = relw * got[b] + 2 * U * np.abs(want[b])
                assert np.all(err <= lim), f"weight {b}: {np.max(err / lim):.3g}x the bound"
                assert np.array_equal(after[b][got[b] == 0], before[b][got[b] == 0])
        return ref


CHUNKS = [
    # dtype, B, Hkv, G, d, page, tokens before, new tokens
    ("bf16", 1, 1, 1, 128, 16, [0], [1]), ("bf16", 1, 2, 4, 128, 64, [100], [1]),
    ("bf16", 1, 1, 1, 64, 16, [0], [130]), ("bf16", 1, 2, 1, 128, 256, [3], [300]),
    ("bf16", 2, 2, 2, 128, 32, [0, 77], [129, 64]), ("bf16", 2, 1, 3, 64, 16, [5, 250], [100, 43]),
    ("bf16", 1, 2, 4, 128, 64, [1000], [200]), ("bf16", 3, 1, 5, 128, 128, [0, 1, 400], [51, 25, 1]),
    ("bf16", 2, 1, 6, 64, 64, [30, 0], [22, 85]), ("bf16", 2, 2, 7, 128, 16, [0, 513], [73, 37]),
    ("bf16", 4, 1, 8, 128, 32, [127, 128, 129, 0], [33, 16, 17, 1]), ("bf16", 5, 2, 4, 64, 16, [9, 0, 64, 200, 0], [0, 3, 0, 90, 1]),
    ("f32", 1, 1, 1, 64, 16, [0], [1]), ("f32", 1, 2, 2, 64, 64, [60], [65]), ("f32", 2, 1, 4, 128, 32, [0, 130], [70, 33]),
    ("f32", 2, 2, 3, 64, 16, [7, 0], [0, 45]), ("f32", 1, 1, 7, 128, 256, [300], [20]), ("f32", 3, 1, 8, 64, 128, [0, 63, 64], [9, 8, 17]),
    ("f32", 1, 1, 5, 128, 16, [200], [27]), ("f32", 1, 3, 1, 128, 64, [1], [200]),
    ("f32", 2, 1, 6, 64, 32, [64, 500], [11, 12]),
]


@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("c", CHUNKS, ids=lambda c: f"{c[0]}-B{c[1]}h{c[2]}g{c[3]}d{c[4]}p{c[5]}-{max(c[6])}+{max(c[7])}")
def test_chunk(c, weights):
    k = Chunk(*c, seed=sum(c[7]), pad=3)
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run(weights)
    k.check(before if weights else None)
    if not weights:
        assert np.array_equal(k.weight.cpu().numpy(), before.astype(np.float32))
    assert status() == 0


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257])
@pytest.mark.parametrize("dtype,G,d", [("bf16", 1, 128), ("bf16", 4, 64), ("bf16", 8, 128), ("f32", 2, 64)])
def test_chunk_lengths(n, dtype, G, d):
    """Prompts of every length about the tiles' sizes, and the same behind a few cached tokens."""
    k = Chunk(dtype, 2, 1, G, d, 16, [0, 128 - n % 7], [n, n], seed=n, sigma=2.0)
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run()
    k.check(before)
    assert status() == 0


def test_chunk_one_token_each():
    """Without a table of rows, a token a sequence: a decode step."""
    for dtype, d in (("bf16", 128), ("f32", 64)):
        k = Chunk(dtype, 6, 2, 4, d, 16, [0, 15, 16, 300, 1, 999], [1] * 6, seed=5)
        before = k.weight.cpu().numpy().astype(np.float64)
        k.run(cu_new=None)
        k.check(before)
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_rows_that_see_nothing(dtype):
    """More new tokens than the cache holds: the first see no slot, and give zeros."""
    k = Chunk(dtype, 3, 2, 3, 64, 16, [0, 0, 40], [100, 70, 5], seed=2)
    k.lens.copy_(ints([37, 0, 45]))
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run()
    ref = k.check(before)
    assert not ref[:63].any() and ref[63:100].all() and not ref[100:170].any()
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_rows_behind_the_end_may_hold_anything(dtype):
    import torch
    for G, d, page, have, new in ((4, 128, 16, [120, 3], [13, 70]), (1, 64, 256, [0, 300], [130, 1]), (3, 128, 64, [1, 64], [64, 63])):
        k = Chunk(dtype, 2, 2, G, d, page, have, new, seed=3, max_pages=-(-max(h + n for h, n in zip(have, new)) // page) + 1)
        start = k.weight.clone()
        clean = k.run().clone()
        first = k.weight.clone()
        pool_k, pool_v = k.kp.clone(), k.vp.clone()
        held = torch.zeros(k.kp.shape[0], page, dtype=torch.bool, device="cuda")
        for b in range(2):
            t = torch.arange(int(k.lens[b]), device="cuda")
            held[k.table[b, t // page].long(), t % page] = True
        for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(k.kp.dtype).min):
            k.kp, k.vp = pool_k.clone(), pool_v.clone()
            k.kp.masked_fill_(~held[:, None, :, None], bad)
            k.vp.masked_fill_(~held[:, None, :, None], bad)
            k.weight.copy_(start)
            assert torch.equal(k.run(), clean) and torch.equal(k.weight, first)
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_bad_pages_and_lengths(dtype):
    import torch
    k = Chunk(dtype, 4, 2, 2, 64, 16, [100, 60, 0, 30], [40, 5, 20, 3], seed=4)
    k.table[0, 2] = -1
    k.table[0, 8] = k.kp.shape[0]
    k.table[1, :] = 1 << 30
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run()
    ref = k.check(before)
    assert status() == 1
    assert not ref[40:45].any()  # no page of its own: nothing cached
    k.lens.copy_(ints([140, -4, 1 << 20, 33]))
    k.table[1, :] = 0
    k.table[2, :] = k.table[3, :]
    before = k.weight.cpu().numpy().astype(np.float64)
    k.run()
    k.check(before)
    assert status() == 1
    # rows that do not ascend, or run out of the call: reported, their sequences left out
    for cu, live in (([0, 40, 30, 65, 68], (0, 2, 3)), ([0, 40, 45, 65, 99], (0, 1, 2)), ([5, 40, 45, 65, 68], (0, 1, 2, 3)),
                     ([-1, 40, 45, 65, 68], (1, 2, 3))):
        k = Chunk(dtype, 4, 2, 2, 64, 16, [100, 60, 0, 30], [40, 5, 20, 3], seed=4)
        torch.cuda.synchronize()
        k.run(cu_new=ints(cu))
        torch.cuda.synchronize()
        assert status() == 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_sharp_and_flat_softmax(dtype):
    """Logits that climb by far more than a running maximum's slack, tie, or are all the same."""
    import torch
    for kind in ("climb", "fall", "spike", "same", "large"):
        k = Chunk(dtype, 1, 1, 4, 64, 16, [500], [60], seed=6)
        if kind in ("climb", "fall"):
            t = torch.arange(560, device="cuda").float()
            k.kp.zero_()
            at = k.table[0, (t // 16).long()].long(), 0, (t % 16).long()
            k.kp[at[0], 0, at[2], 0] = (t / 8 if kind == "climb" else 70 - t / 8).to(k.kp.dtype)
            k.q.zero_()
            k.q[..., 0] = 20.0
        elif kind == "spike":
            k.kp[k.table[0, 20].long(), 0, 5] = 30 * torch.sign(k.q[-1, 0]).to(k.kp.dtype)
        elif kind == "same":
            k.kp.zero_()
        else:
            k.kp.mul_(30)
        before = k.weight.cpu().numpy().astype(np.float64)
        k.run()
        k.check(before)
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_equal_calls_give_equal_bits(dtype):
    """Alone, on another stream, in a graph, and with a batch around it that changes the cuts of the others' work."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_chunk_workspace_size
    k = Chunk(dtype, 3, 2, 4, 128, 32, [700, 20, 0], [90, 300, 2], seed=7, pad=5)
    w0 = k.weight.clone()
    a = k.run().clone()
    wa = k.weight.clone()
    k.weight.copy_(w0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k.run(stream=s)
    s.synchronize()
    assert torch.equal(k.out.view(torch.uint8), a.view(torch.uint8)) and torch.equal(k.weight, wa)
    ws = torch.empty(fasa_paged_chunk_workspace_size(k.dims, k.n, True), dtype=torch.uint8, device="cuda").fill_(255)
    k.weight.copy_(w0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k.run(workspace=ws)
    for _ in range(3):
        k.weight.copy_(w0)
        ws.fill_(127)
        k.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(k.out[:392], a[:392]) and torch.equal(k.weight, wa)
    assert status() == 0


# -------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,d,page,G", [("bf16", 128, 16, 4), ("bf16", 64, 64, 3), ("f32", 64, 32, 2)])
def test_a_server_s_steps(dtype, d, page, G):
    """Prompts arrive in chunks, sequences decode, are cut and end: assign, rope_append and chunk attention step by
    step, then an eviction, against a plain cache kept by the oracle."""
    import torch
    from kv_cache_token_tip_gb300 import (FasaRope, fasa_paged_assign, fasa_paged_chunk_attention, fasa_paged_evict,
                                          fasa_paged_rope_append)
    from oracle import paged_oracle as PO
    rng = np.random.default_rng(d + G)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    B, Hkv, max_pages, n_tok, keep = 4, 2, 512 // page, 160, 64
    n_pages, Hq = 2 * 512 // page, Hkv * G
    dims = paged_dims(dtype, B, Hkv, G, d, page, n_pages, max_pages)
    rope = FasaRope(1, d // 2, 2, 5e5, factor=8.0, low=1.0, high=4.0, original=256.0)
    table, free, count = ints([[-1] * max_pages] * B), ints(rng.permutation(n_pages)), ints([n_pages])
    lens, cu, m = ints([0] * B), ints([0] * (B + 1)), torch.zeros((n_tok, 4), dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros((n_pages, Hkv, page, d), device="cuda").to(dt) for _ in range(2))
    w = torch.zeros((B, Hkv, max_pages * page), device="cuda")
    tp = torch.zeros((B, Hkv, max_pages * page), dtype=torch.int32, device="cuda")
    pos, news = [0] * B, None
    host = lambda x: host_f64(x.contiguous(), dtype)
    for step, news in enumerate([(100, 0, 50, 0), (60, 90, 1, 0), (1, 40, 1, 77), (1, 1, 1, -300), (1, 1, 1, 20), (1, 1, 0, 1)]):
        have = lens.tolist()
        want = [max(0, h + x) for h, x in zip(have, news)]
        posd = ints(pos)
        fasa_paged_assign(lens, ints(want), table, free, count, lens, cu, m, pos=posd, dims=dims)
        assert lens.tolist() == want
        n = int(cu[-1])
        assert n == sum(max(x, 0) for x in news)
        qkv = torch.from_numpy(rng.standard_normal((n_tok, Hq + 2 * Hkv, d))).cuda().to(dt)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        q_rot, out = torch.zeros((n_tok, Hq, d), device="cuda").to(dt), torch.zeros((n_tok, Hq, d), device="cuda").to(dt)
        rkp, rvp, rw, rtp = host(kp), host(vp), w.cpu().numpy().astype(np.float64), tp.cpu().numpy()
        fasa_paged_rope_append(q, k, v, m, q_rot, kp, vp, weight=w, token_pos=tp, rope=rope, dims=dims)
        rq = np.zeros((n_tok, Hq, d))
        SO.rope_append(host(q), host(k), host(v), m.cpu().numpy(), rq, rkp, rvp, rw, rtp, rope)
        tol = E[dtype] + 4e-6
        assert np.all(np.abs(host(q_rot) - rq) <= tol * 8) and np.all(np.abs(host(kp) - rkp) <= tol * 8)
        assert np.array_equal(host(vp), rvp) and np.array_equal(tp.cpu().numpy(), rtp)
        assert np.array_equal(w.cpu().numpy(), rw.astype(np.float32))
        fasa_paged_chunk_attention(q_rot, kp, vp, table, lens, out, cu_new=cu, weight=w, dims=dims)
        ref, got, A, pv = SO.chunk_attention(host(q_rot), cu.tolist(), host(kp), host(vp), table.cpu().numpy(), want)
        rel = 2 * (2 * d + 16) * U * A + (16 + 512 + 64) * U
        bound = (rel + (2.0 ** -8 if dtype == "bf16" else 0.0) + 2 * (512 + 64) * U)[..., None] * pv + E[dtype] * np.abs(ref)
        assert np.all(np.abs(host(out) - ref)[:n] <= bound[:n])
        assert np.all(np.abs(w.cpu().numpy() - rw - got) <= (rel.max() + (n_tok * G + 64) * U) * got + 2 * U * (rw + got))
        pos = [0 if x < 0 else p + max(x, 0) for p, x in zip(pos, news)]
        if step == 4:  # cut to `keep`, and give the pages back
            new = ints([0] * B)
            stay = lens.tolist()
            rkp, rvp, rw, rtp = host(kp), host(vp), w.cpu().numpy().astype(np.float64), tp.cpu().numpy().copy()
            at = ints([p - 1 for p in pos])
            rnew = PO.paged_evict(rw, rtp, at.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy(), keep, 2, 8, rkp, rvp, rw, rtp)
            fasa_paged_evict(w, tp, at, kp, vp, table, lens, keep, new, sinks=2, recent=8, dims=dims)
            assert np.array_equal(host(kp), rkp) and new.tolist() == rnew.tolist()
            free_before = count.item()
            fasa_paged_assign(lens, new, table, free, count, lens, cu, m, dims=dims)
            assert lens.tolist() == new.tolist()
            assert count.item() - free_before == sum(-(-a // page) - -(-b // page) for a, b in zip(stay, rnew))
    used = [table[b, e].item() for b in range(B) for e in range(-(-lens.tolist()[b] // page))]
    rest = free[:count.item()].tolist()
    assert sorted(used + rest) == list(range(n_pages))  # every page is somewhere, once
    assert status() == 0


# ------------------------------------------------------------- hard conditions
def reference(k, sequences=None):
    """out [n, Hq, d] of a Chunk in 64 bits by torch on the GPU (long caches), and sum p |V| beside it."""
    import torch
    out = torch.zeros(k.q.shape, dtype=torch.float64, device="cuda")
    pv = torch.zeros_like(out)
    for b in range(k.B) if sequences is None else sequences:
        x0, x1, n = k.cu_host[b], k.cu_host[b + 1], int(k.lens[b])
        t = torch.arange(n, device="cuda")
        pg, at = k.table[b, t // k.page].long(), t % k.page
        for h in range(k.Hkv):
            K, V = k.kp[pg, h, at].double(), k.vp[pg, h, at].double()
            q = k.q[x0:x1, h * k.G:(h + 1) * k.G].double()
            z = torch.einsum("jgd,td->jgt", q, K) / k.d ** 0.5
            z.masked_fill_((t.view(1, 1, -1) > (n - (x1 - x0) + torch.arange(x1 - x0, device="cuda")).view(-1, 1, 1)), -float("inf"))
            p = torch.softmax(z, dim=-1)
            out[x0:x1, h * k.G:(h + 1) * k.G] = torch.einsum("jgt,td->jgd", p, V)
            pv[x0:x1, h * k.G:(h + 1) * k.G] = torch.einsum("jgt,td->jgd", p, V.abs())
    return out, pv


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 3, 4, 7])
def test_chunk_queries_of_others_may_hold_anything(dtype, G):
    """NaN and infinities in padding and in one sequence's queries stay in that sequence's rows and weights."""
    import torch
    k = Chunk(dtype, 3, 2, G, 128, 16, [40, 3, 100], [30, 45, 37], seed=8, pad=40)
    start = k.weight.clone()
    clean, first = k.run().clone(), k.weight.clone()
    for bad in (float("nan"), float("inf")):
        k.weight.copy_(start)
        k.q[30:75] = bad
        k.q[112:] = bad
        k.run()
        assert torch.equal(k.out[:30], clean[:30]) and torch.equal(k.out[75:112], clean[75:112])
        assert torch.equal(k.weight[0], first[0]) and torch.equal(k.weight[2], first[2])
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,d,page,have,new", [
    (4, 128, 16, 40, 200), (4, 128, 64, 3000, 300), (1, 64, 256, 3, 300), (7, 128, 32, 100, 80), (3, 64, 16, 2000, 90), (8, 128, 16, 126, 5)])
def test_chunk_tokens_behind_a_row_may_hold_anything(dtype, G, d, page, have, new):
    """What is not finite in a new token's values reaches the rows that see it, in its dims, and no other bit; the same
    of keys, whose rows are NaN."""
    import torch
    k = Chunk(dtype, 1, 2, G, d, page, [have], [new], seed=21)
    start = k.weight.clone()
    clean, first = k.run().clone(), k.weight.clone()
    pool_k, pool_v = k.kp.clone(), k.vp.clone()

    def place(j):
        return k.table[0, (have + j) // page].item(), (have + j) % page

    h, dim, inf = 1, d // 2 + 5, float("inf")
    rows = torch.arange(new, device="cuda")
    for j in sorted({1, 2, new // 2, new - 2, new - 1}):
        for bad in (float("nan"), inf, -inf):
            k.vp = pool_v.clone()
            pg, at = place(j)
            k.vp[pg, h, at, dim] = bad
            k.weight.copy_(start)
            out = k.run().clone()
            want = clean.clone()
            want[rows >= j, h * G:(h + 1) * G, dim] = bad
            same = (out == want) | (torch.isnan(out) & torch.isnan(want))
            assert same.all(), (j, bad, int((~same).sum()))
            assert torch.equal(k.weight, first)
    a, b = 1, new - 2  # of both signs: infinite between them, NaN behind
    k.vp = pool_v.clone()
    for j, bad in ((a, inf), (b, -inf)):
        pg, at = place(j)
        k.vp[pg, h, at, dim] = bad
    k.weight.copy_(start)
    out = k.run().clone()
    hit = out[:, h * G:(h + 1) * G, dim].float()
    assert torch.equal(out[:a], clean[:a]) and (hit[a:b] == inf).all() and torch.isnan(hit[b:]).all()
    k.vp, k.kp = pool_v, pool_k.clone()
    pg, at = place(new // 2)
    k.kp[pg, h, at] = float("nan")
    k.run(False)
    assert torch.equal(k.out[:new // 2], clean[:new // 2])
    assert torch.isnan(k.out[new // 2:, h * G:(h + 1) * G].float()).all()
    assert torch.equal(k.out[:, :h * G], clean[:, :h * G])
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_no_tokens_at_all(dtype):
    import torch
    k = Chunk(dtype, 3, 2, 2, 64, 16, [40, 0, 20], [0, 0, 0], seed=8, pad=9)
    w = k.weight.clone()
    k.run()
    assert torch.isnan(k.out).all() and torch.equal(k.weight, w)
    k = Chunk(dtype, 3, 2, 2, 64, 16, [40, 0, 20], [0, 0, 0], seed=8)
    k.run()   # a call without rows
    assert status() == 0


@pytest.mark.parametrize("dtype,B,Hkv,G,d", [("bf16", 2048, 4, 8, 64), ("f32", 2048, 2, 1, 64), ("bf16", 300, 16, 1, 128),
                                             ("bf16", 1, 64, 1, 64)])
def test_chunk_many_sequences_and_heads(dtype, B, Hkv, G, d):
    import torch
    rng = np.random.default_rng(B)
    k = Chunk(dtype, B, Hkv, G, d, 16, [int(x) for x in rng.integers(0, 60, B)], [int(x) for x in rng.integers(0, 4, B)],
              seed=9, pad=1)
    w0 = k.weight.clone()
    k.run()
    ref, pv = reference(k)
    live = slice(0, k.cu_host[-1])
    err = (k.out.double() - ref).abs()[live]
    # (the logits' rounding: 2 (2 d + 16) u A, A below 4 d^0.5 here)
    e = E[dtype]
    assert (err <= (2 * e + 8 * d ** 0.5 * (2 * d + 16) * U + 400 * U) * pv[live] + 1e-30).all()
    # every row's weights sum to 1
    for b in range(0, B, 97):
        m = k.cu_host[b + 1] - k.cu_host[b]
        got = (k.weight[b].double() - w0[b].double()).sum(dim=1)
        assert ((got - m * G).abs() <= 1e-5 * (m * G + w0[b].double().sum(dim=1))).all()
    assert status() == 0


@pytest.mark.parametrize("dtype,d,G,page", [("bf16", 64, 4, 256), ("bf16", 128, 8, 16), ("f32", 64, 2, 128),
                                            ("bf16", 128, 1, 64), ("f32", 128, 1, 16)])
def test_chunk_long_cache(dtype, d, G, page):
    """One sequence over the whole range of slots, and a short one beside it."""
    k = Chunk(dtype, 2, 1, G, d, page, [262144 - 5, 7], [5, 30], seed=10, max_pages=262144 // page)
    before = k.weight.clone()
    k.run()
    ref, pv = reference(k)
    err = (k.out.double() - ref).abs()
    # sums of 262144 terms in parts: of tiles, and over a part's 1725 tiles or fewer
    rel = 8 * d ** 0.5 * (2 * d + 16) * U + (2 * 2 ** 12 + 400) * U + (2.0 ** -8 if dtype == "bf16" else 0)
    assert (err <= rel * pv + E[dtype] * ref.abs() + 1e-30).all()
    got = (k.weight.double() - before.double()).clamp(min=0)
    assert abs(float(got[0].sum()) - 5 * G) <= 1e-3 * 5 * G + float(before[0].double().sum()) * U
    assert status() == 0


@pytest.mark.parametrize("dtype,G", [("bf16", 4), ("bf16", 1), ("f32", 8)])
def test_chunk_weights_of_few_rows_either_way(dtype, G):
    """Sequences of few rows have their logits kept for the weights, where a batch's logits are not too many: a
    table of many more entries, and the second pass works them out again."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_chunk_attention, fasa_paged_chunk_workspace_size
    B, Hkv, d, page = 64, 8, 64, 16
    rng = np.random.default_rng(G)
    k = Chunk(dtype, B, Hkv, G, d, page, [int(x) for x in rng.integers(0, 400, B)], [int(x) for x in rng.integers(0, 3, B)],
              seed=17)
    k.table[3, 1] = -1   # (reported where that sequence has a new token, and slots there)
    looked = int(k.cu_host[4] > k.cu_host[3] and int(k.lens[3]) > page)
    start = k.weight.clone()
    out = k.run().clone()
    assert status() == looked
    wide = 2200
    assert B * Hkv * 8 * wide * page * 4 > 1 << 29 > B * Hkv * 8 * (k.cap + 128) * 4
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    table[:, :k.table.shape[1]] = k.table
    weight = torch.zeros((B, Hkv, wide * page), device="cuda")
    weight[:, :, :k.cap] = start
    dims = paged_dims(dtype, B, Hkv, G, d, page, k.kp.shape[0], wide)
    assert fasa_paged_chunk_workspace_size(dims, k.n, True) < 1 << 29
    fasa_paged_chunk_attention(k.q, k.kp, k.vp, table, k.lens, k.out, cu_new=k.cu, weight=weight, dims=dims)
    assert status() == looked and torch.equal(k.out, out)
    # the same logits, summed in another order: 16 u of each exp2 and 9 sums, and u of the weight
    got = k.weight - start
    assert ((weight[:, :, :k.cap] - k.weight).abs() <= 64 * U * got.abs() + 8 * U * k.weight + 1e-30).all()
    assert not weight[:, :, k.cap:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,new", [(1, [15, 16, 17, 1]), (4, [3, 4, 5, 1]), (8, [1, 2, 3, 0]), (3, [5, 6, 2, 1]), (5, [3, 4, 1, 2])])
def test_chunk_weights_around_few_rows(dtype, G, new):
    """Weights of sequences on both sides of the number of rows up to which logits are kept, some cut into parts."""
    for d, page, have in ((128, 16, [500, 130, 0, 64]), (64, 256, [1, 2000, 700, 255])):
        k = Chunk(dtype, 4, 2, G, d, page, have, new, seed=31)
        before = k.weight.cpu().numpy().astype(np.float64)
        k.run()
        assert status() == 0
        k.check(before)


def test_chunk_long_sums_in_fp32():
    """Sums of P V over long caches: 64 slots at a time, then those.

    A sum of n random terms is off by u / sqrt(3) sqrt(n / 2) of its size: sqrt(32) of that for a tile's 64 slots and
    sqrt(128) for the 256 tiles of a cache, 5.8e-7 with u = 2^-24; flat weights (2^x and their sum) bring 1e-7 more, the
    rounding of the result 3e-8.  One after another, 16384 slots would be off by 3.1e-6, cut in half 2.2e-6."""
    import torch
    k = Chunk("f32", 20, 8, 4, 128, 256, [16376] * 20, [8] * 20, seed=41, sigma=0.05)
    k.run(False)
    for b in (0, 9, 19):
        ref, _ = reference(k, [b])
        x0, x1 = k.cu_host[b], k.cu_host[b + 1]
        err = (k.out[x0:x1].double() - ref[x0:x1]).norm() / ref[x0:x1].norm()
        assert err <= 1e-6, f"{err:.3g}"
    assert status() == 0


def test_offsets_past_32_bits():
    """Pools of more than 2^32 elements, used at their far end by all the calls."""
    import torch
    from kv_cache_token_tip_gb300 import FasaRope, fasa_paged_assign, fasa_paged_chunk_attention, fasa_paged_rope_append
    B, Hkv, G, d, page, mp, n_tok = 2, 8, 4, 128, 16, 14, 90
    dt, rope = torch.bfloat16, FasaRope(1, 128, 1, 5e5, factor=2.0)
    got = []
    for n_pages in (40, 270_000):
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        kp, vp = (torch.zeros((n_pages, Hkv, page, d), dtype=dt, device="cuda") for _ in range(2))
        dims = paged_dims("bf16", B, Hkv, G, d, page, n_pages, mp)
        free = torch.arange(n_pages, dtype=torch.int32, device="cuda")   # (the last pages are taken first)
        count, table, lens = ints([n_pages]), ints([[-1] * mp] * B), ints([0, 0])
        cu, m = ints([0] * 3), torch.zeros((n_tok, 4), dtype=torch.int32, device="cuda")
        w, tp = torch.zeros((B, Hkv, mp * page), device="cuda"), torch.zeros((B, Hkv, mp * page), dtype=torch.int32, device="cuda")
        outs = []
        for want in ([60, 30], [61, 100], [140, 101]):
            fasa_paged_assign(lens, ints(want), table, free, count, lens, cu, m, dims=dims)
            qkv = torch.randn((n_tok, Hkv * (G + 2), d), generator=g, device="cuda").to(dt)
            q, o = torch.zeros((n_tok, Hkv * G, d), dtype=dt, device="cuda"), torch.zeros((n_tok, Hkv * G, d), dtype=dt, device="cuda")
            fasa_paged_rope_append(qkv[:, :Hkv * G], qkv[:, Hkv * G:-Hkv], qkv[:, -Hkv:], m, q, kp, vp, weight=w,
                                   token_pos=tp, rope=rope, dims=dims)
            fasa_paged_chunk_attention(q, kp, vp, table, lens, o, cu_new=cu, weight=w, dims=dims)
            outs += [q, o]
        got.append(outs + [w, tp, kp[-30:].clone(), vp[-30:].clone()])
        del kp, vp
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][1].abs().sum() > 0
    assert status() == 0


def test_chunk_shared_pages():
    """Two sequences with the same prompt's pages: as with pages of their own."""
    import torch
    k = Chunk("bf16", 2, 2, 4, 128, 32, [256, 256], [9, 40], seed=11)
    shared = k.table.clone()
    shared[1, :8] = shared[0, :8]
    own = k.table
    k.kp[own[1, :8].long()], k.vp[own[1, :8].long()] = k.kp[own[0, :8].long()], k.vp[own[0, :8].long()]
    w = k.weight.clone()
    a, wa = k.run().clone(), k.weight.clone()
    k.weight.copy_(w)
    k.table = shared
    assert torch.equal(k.run(), a) and torch.equal(k.weight, wa) and status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_graphs_that_share_a_workspace(dtype):
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_chunk_workspace_size
    ks = [Chunk(dtype, 3, 2, 4, 128, 32, [700, 20, 0], [90, 30, 2], seed=12), Chunk(dtype, 1, 4, 2, 64, 16, [5], [300], seed=13)]
    ref = []
    for k in ks:
        k.start = k.weight.clone()
        ref.append((k.run().clone(), k.weight.clone()))
    ws = torch.empty(max(fasa_paged_chunk_workspace_size(k.dims, k.n, True) for k in ks), dtype=torch.uint8, device="cuda")
    graphs = []
    torch.cuda.synchronize()
    for k in ks:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            k.run(workspace=ws)
    for _ in range(4):
        for k in ks:
            k.weight.copy_(k.start)
        for g in graphs + graphs[::-1]:
            g.replay()
        for k, (out, w) in zip(ks, ref):
            assert torch.equal(k.out, out)
            assert (k.weight - k.start - 2 * (w - k.start)).abs().max() <= 1e-4 * float(k.weight.max())
    assert status() == 0


def test_chunks_of_two_streams_at_once():
    """Two calls with their own workspaces, on two streams: blocks of both wait for an SM, and no result changes."""
    import torch
    ks = [Chunk("bf16", 4, 4, 4, 128, 16, [900, 30, 5, 0], [200, 300, 1, 77], seed=14 + i) for i in range(2)]
    ref = []
    for k in ks:
        k.start = k.weight.clone()
        ref.append((k.run().clone(), k.weight.clone()))
    streams = [torch.cuda.Stream() for _ in ks]
    torch.cuda.synchronize()
    for _ in range(10):
        for k, s in zip(ks, streams):
            with torch.cuda.stream(s):
                k.weight.copy_(k.start)
                k.out.fill_(float("nan"))
                k.run()
    torch.cuda.synchronize()
    for k, (out, w) in zip(ks, ref):
        assert torch.equal(k.out, out) and torch.equal(k.weight, w)
    assert status() == 0


def test_calls_of_two_threads():
    """Other types, rotations and shapes in two threads: what the library keeps between calls is not mixed up."""
    import threading
    import torch
    from kv_cache_token_tip_gb300 import FasaRope, fasa_paged_rope_append

    def steps(i):
        k = Chunk(*(("bf16", 2, 2, 4, 128, 16, [100, 40], [60, 7]), ("f32", 3, 1, 2, 64, 32, [10, 0, 70], [5, 50, 1]))[i], seed=20 + i)
        m = [(b, int(k.lens[b]) - (k.cu_host[b + 1] - k.cu_host[b]) + j) for b in range(k.B) for j in range(k.cu_host[b + 1] - k.cu_host[b])]
        m = ints([(b, t, int(k.table[b, t // k.page]), 31 * t) for b, t in m])
        outs = []
        for r in range(20):
            rope = FasaRope(i, 64, r % 4, 1e4 * (1 + i), factor=2.0 + r, low=1.0, high=8.0, original=512.0)
            q = torch.zeros_like(k.q)
            fasa_paged_rope_append(k.q, k.q[:, :k.Hkv], k.q[:, -k.Hkv:], m, q, k.kp, k.vp, rope=rope, dims=k.dims)
            outs += [q, k.run().clone()]
        return torch.stack(outs), k.weight

    alone = [steps(i) for i in range(2)]
    got = [None, None]
    torch.cuda.synchronize()

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got[i] = steps(i)
        s.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(x, y) for g, a in zip(got, alone) for x, y in zip(g, a)) and status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_bounded_waits(dtype):
    """A copy that is never issued: the waits on it run out within the bound, the call says so, drains what it has
    under way and gives tensor memory back, and the next call gives the bits of the first.  (The wait is on a barrier
    in shared memory that no copy targets.)"""
    import torch
    from kv_cache_token_tip_gb300 import FASA_DEV_TIMEOUT, FASA_DEV_UNDRAINED, fasa_test_fault_injection
    k = Chunk(dtype, 2, 4, 4, 128, 32, [3000, 50], [200, 10], seed=15)
    ref = k.run(False).clone()
    assert status() == 0
    try:
        fasa_test_fault_injection(wait_limit_ns=2_000_000)
        assert torch.equal(k.run(False), ref) and status() == 0   # a short bound alone changes nothing
        fasa_test_fault_injection(wait_limit_ns=2_000_000, drop_tip_tile=1)
        k.run(False)
        assert status() == FASA_DEV_TIMEOUT | FASA_DEV_UNDRAINED
    finally:
        fasa_test_fault_injection()
    assert torch.equal(k.run(False), ref) and status() == 0


def test_binding_refuses_what_does_not_fit():
    import torch
    from kv_cache_token_tip_gb300 import (FasaError, FasaRope, fasa_paged_assign, fasa_paged_chunk_attention,
                                          fasa_paged_rope_append)
    k = Chunk("bf16", 2, 2, 2, 64, 16, [20, 30], [4, 5], seed=16)
    m, rope = torch.zeros((9, 4), dtype=torch.int32, device="cuda"), FasaRope(1, 64)

    def chunk(**kw):
        t = dict(q=k.q, kp=k.kp, vp=k.vp, table=k.table, lens=k.lens, out=k.out, cu=k.cu, weight=k.weight, ws=None)
        t.update(kw)
        fasa_paged_chunk_attention(t["q"], t["kp"], t["vp"], t["table"], t["lens"], t["out"], cu_new=t["cu"],
                                   weight=t["weight"], workspace=t["ws"], dims=k.dims)

    for bad in (dict(q=k.q.float()), dict(q=k.q.cpu()), dict(q=k.q[:, 1:]), dict(q=k.q.transpose(0, 1)), dict(kp=k.kp[:-1]),
                dict(vp=k.vp.float()), dict(table=k.table[:, :-1]), dict(lens=k.lens[:1]), dict(lens=k.lens.long()),
                dict(out=k.out.float()), dict(out=k.out[1:]), dict(cu=k.cu[1:]), dict(weight=k.weight[:1]),
                dict(weight=k.weight.double()), dict(ws=torch.empty(9))):
        with pytest.raises(ValueError):
            chunk(**bad)
    for bad in (dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(out=k.q), dict(cu=None)):
        with pytest.raises(FasaError):
            chunk(**bad)

    def append(q=k.q, kk=k.q[:, :2], v=k.q[:, 2:], m=m, qo=k.out, kp=k.kp, vp=k.vp, rope=rope, **kw):
        fasa_paged_rope_append(q, kk, v, m, qo, kp, vp, rope=rope, dims=k.dims, **kw)

    for bad in (dict(q=k.q.float()), dict(q=k.q[:, :, ::2]), dict(q=k.q.transpose(1, 2)), dict(q=k.q[0]), dict(kk=k.q),
                dict(kk=k.q[:8, :2]), dict(v=None), dict(m=m[1:]), dict(m=m.long()), dict(qo=k.out[1:]), dict(qo=None),
                dict(kp=None), dict(vp=k.vp[1:]), dict(weight=k.weight[:, :1]), dict(token_pos=k.weight)):
        with pytest.raises(ValueError):
            append(**bad)
    odd = torch.empty(9 * 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(9, 4, 64)
    for bad in (dict(q=odd), dict(qo=odd), dict(qo=k.q[:9], q=k.q, kk=k.q[:, :2]), dict(rope=FasaRope(1, 72)),
                dict(rope=FasaRope(5, 64)), dict(kk=None, v=None, kp=None, vp=None, weight=k.weight)):
        with pytest.raises(FasaError):
            append(**bad)
    n = k.kp.shape[0]
    free, one, cu = torch.zeros(n, dtype=torch.int32, device="cuda"), ints([0]), ints([0, 0, 0])
    lens = k.lens.clone()

    def assign(have=k.lens, want=k.lens, table=k.table, free=free, count=one, out=lens, cu=cu, m=m, **kw):
        fasa_paged_assign(have, want, table, free, count, out, cu, m, dims=k.dims, **kw)

    for bad in (dict(have=k.lens[:1]), dict(want=k.lens.long()), dict(table=k.table.t()), dict(free=free[1:]),
                dict(count=ints([0, 0])), dict(out=lens.cpu()), dict(cu=cu[1:]), dict(m=m.view(-1)[:-1]), dict(pos=one)):
        with pytest.raises(ValueError):
            assign(**bad)
    for bad in (dict(pos=lens), dict(out=cu[1:]), dict(free_count_out=lens[:1])):
        with pytest.raises(FasaError):
            assign(**bad)
    assert status() == 0


FIRST_CALLS = """
import torch
from kv_cache_token_tip_gb300 import (FasaPagedDims, FasaRope, fasa_device_status, fasa_paged_assign,
                                      fasa_paged_chunk_attention, fasa_paged_rope_append)
for dtype, code, d in ((torch.bfloat16, 1, 128), (torch.float32, 0, 64)):
    B, H, G, page, n, T = 2, 2, 4, 16, 6, 40
    dims, rope = FasaPagedDims(B, H * G, H, d, page, B * n, n, code, 1e4), FasaRope(1, d)
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")
    i = lambda *s: z(*s, t=torch.int32)
    kp, vp, w, tp = z(B * n, H, page, d, t=dtype), z(B * n, H, page, d, t=dtype), z(B, H, n * page), i(B, H, n * page)
    table, free, count = i(B, n), torch.arange(B * n, dtype=torch.int32, device="cuda"), i(1) + B * n
    lens, want, cu, m = i(B), i(B), i(B + 1), i(T, 4)
    qkv = torch.ones(T, H * (G + 2), d, device="cuda").to(dtype)
    q, out = z(T, H * G, d, t=dtype), z(T, H * G, d, t=dtype)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        want.copy_(lens)
        want.add_(7)
        fasa_paged_assign(lens, want, table, free, count, lens, cu, m, dims=dims)
        fasa_paged_rope_append(qkv[:, :H * G], qkv[:, H * G:-H], qkv[:, -H:], m, q, kp, vp, weight=w, token_pos=tp,
                               rope=rope, dims=dims)
        fasa_paged_chunk_attention(q, kp, vp, table, lens, out, cu_new=cu, weight=w, dims=dims)
    for _ in range(9):
        g.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [63, 63] and count.item() == B * n - 8 and cu.tolist() == [0, 7, 14]
    # out = o / l with V being 1: at most 2^-8 of the weights' rounding to bf16, and sums of 63 terms
    assert (out[:14].float() - 1).abs().max() <= (2.0 ** -7 if code else 200 * 2.0 ** -24), out
    assert (w[:, :, :63].sum(-1) - 9 * 7 * G).abs().max() <= 1e-3 and fasa_device_status() == 0
print("fine")
"""


def test_first_calls_of_a_process_in_a_capture():
    """Nothing of the library has run before: what it sets up on first use does
    not end the capture, and the graph's steps go on from replay to replay."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
