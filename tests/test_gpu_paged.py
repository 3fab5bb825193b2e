"""The paged cache on a GPU: append, attention with accumulated weights and
eviction against the fp64 oracle on the same stored values.

Tolerances (u = 2^-24, the half step of fp32; derived, not fitted):
  * a rotated element: 2e-6 of its pair's norm (the angle in turns rounds to
    2^-25 of a half turn, cos and sin to 2 ulp, two products and a sum), plus
    half a step of the stored type;
  * a logit z (natural units): the query's 2e-6 and an fp32 sum of d products,
    |dz| <= eps_z * A with A = sum |q||k| / sqrt(d), eps_z = 2e-6 + (d + 8) u,
    plus 4 u |z|, |z| <= A, of the scaling to powers of two;
  * a softmax weight p: relative 2 max |dz| (the weight and the sum it is divided
    by), 2^-16 of the two-term split of P, 16 u of exp2 and the divisions, and
    (T + 64) u for a sum of T terms in any order;
  * out: that relative error times sum p |V|, plus an fp32 sum's (T + 64) u of it;
  * a weight: that relative error of what it receives, plus u of its new value
    for each of the G + 1 sums.
Eviction moves and compares stored values: exact.
"""

import numpy as np
import pytest

from oracle import paged_oracle as PO
from tests.gpu_util import ensure_built
from tests.parity import host_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    ensure_built()


class Cache:
    """A paged cache on the GPU with what its calls need, seeded."""

    def __init__(self, dtype, B, Hkv, G, d, page, lens, max_pages=None, theta=5e5, seed=0, sigma=1.0, spare=3):
        import torch
        from kv_cache_token_tip_gb300 import FASA_BF16, FASA_F32, FasaPagedDims
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.dtype, self.B, self.Hkv, self.G, self.d, self.page, self.theta = dtype, B, Hkv, G, d, page, theta
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        max_pages = max_pages or max(1, -(-max(max(lens), 1) // page))
        self.cap = max_pages * page
        n_pages = B * max_pages + spare

        def normal(*s):
            return torch.randn(s, generator=g, device="cuda")

        self.table = torch.randperm(n_pages, generator=g, device="cuda")[:B * max_pages].to(torch.int32).view(
            B, max_pages).contiguous()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.kp, self.vp = normal(n_pages, Hkv, page, d).to(dt), normal(n_pages, Hkv, page, d).to(dt)
        self.q = (sigma * normal(B, Hkv * G, d)).to(dt)
        self.pos = torch.tensor([n + 3 for n in lens], dtype=torch.int32, device="cuda")
        self.weight = torch.exp(normal(B, Hkv, self.cap))
        self.token_pos = torch.arange(self.cap, dtype=torch.int32, device="cuda").expand(B, Hkv, self.cap).contiguous()
        self.out = torch.full((B, Hkv * G, d), float("nan"), device="cuda")
        self.dims = FasaPagedDims(B, Hkv * G, Hkv, d, page, n_pages, max_pages,
                                  FASA_F32 if dtype == "f32" else FASA_BF16, theta)
        self.gen = g

    def host(self, x):
        return host_f64(x, self.dtype)

    def attend(self, weight=True, **kw):
        from kv_cache_token_tip_gb300 import fasa_paged_attention
        fasa_paged_attention(self.q, self.pos, self.kp, self.vp, self.table, self.lens, self.out,
                             weight=self.weight if weight else None, dims=self.dims, **kw)
        return self.out


def status():
    from kv_cache_token_tip_gb300 import fasa_device_status
    return fasa_device_status()


def check_attention(c, before, out, after, lens=None, table=None):
    """out and the statistics after a call against the oracle; before, after:
    the weights (numpy), or None."""
    lens = c.lens.cpu().numpy() if lens is None else lens
    table = c.table.cpu().numpy() if table is None else table
    ref, got, A, pv = PO.paged_attention(c.host(c.q), c.pos.cpu().numpy(), c.host(c.kp), c.host(c.vp), table, lens,
                                         c.theta)
    out = out.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(out))
    T = np.array([min(max(int(n), 0), c.cap) for n in lens], dtype=np.float64)
    eps_z = 2e-6 + (c.d + 8) * U + 4 * U
    rel = 2 * eps_z * A.max(-1) + 2.0 ** -16 + (16 + T[:, None] + 64) * U   # [B, Hq]
    bound = (rel + (T[:, None] + 64) * U)[..., None] * pv
    err = np.abs(out - ref)
    assert np.all(err <= bound + 1e-30), f"out: {np.max(err / (bound + 1e-30)):.3g}x the bound"
    assert np.all(out[T == 0] == 0)
    if before is not None:
        want = before + got
        relw = rel.reshape(c.B, c.Hkv, c.G).max(-1)[..., None]
        bound = relw * got + (c.G + 1) * U * np.abs(want)
        err = np.abs(after - want)
        assert np.all(err <= bound), f"weight: {np.nanmax(err / np.maximum(bound, 1e-30)):.3g}x the bound"
        untouched = got == 0
        assert np.array_equal(after[untouched], before[untouched])


SHAPES = [
    # dtype, B, Hkv, G, d, page, lengths
    ("bf16", 1, 1, 1, 64, 16, [1]),
    ("f32", 1, 1, 1, 64, 16, [1]),
    ("bf16", 1, 2, 2, 128, 16, [15]),
    ("bf16", 2, 1, 8, 128, 32, [16, 17]),
    ("f32", 2, 2, 8, 128, 16, [33, 0]),
    ("bf16", 4, 2, 7, 128, 64, [0, 1, 130, 127]),
    ("f32", 3, 2, 3, 64, 256, [255, 257, 700]),
    ("bf16", 3, 4, 5, 64, 128, [513, 2, 128]),
    ("bf16", 1, 8, 4, 128, 64, [3001]),
    ("f32", 1, 4, 4, 128, 64, [1999]),
    ("bf16", 9, 2, 4, 64, 16, [0, 0, 5, 200, 0, 31, 32, 1000, 0]),
    ("bf16", 40, 4, 2, 128, 16, [(i * 37) % 300 for i in range(40)]),
    ("f32", 33, 8, 1, 64, 32, [(i * 53) % 200 for i in range(33)]),
    # more units than parts: a unit is found by the part it begins in
    ("bf16", 300, 8, 1, 64, 16, [(i * 37) % 90 for i in range(300)]),
    ("f32", 260, 8, 2, 64, 16, [(i * 41) % 70 for i in range(260)]),
    ("bf16", 200, 8, 5, 128, 16, [(i * 29) % 60 for i in range(200)]),
    # cut units joined by warps, beside those that add weights, and by blocks
    ("bf16", 8, 8, 4, 128, 64, [700 + 31 * i for i in range(8)]), ("bf16", 16, 8, 4, 64, 32, [250 + 17 * i for i in range(16)]),
    ("bf16", 12, 4, 7, 128, 16, [900 - 61 * i for i in range(12)]), ("f32", 4, 4, 8, 128, 64, [1500, 0, 1100, 1501]),
    ("f32", 24, 4, 6, 64, 16, [300 + 13 * i for i in range(24)]),
    # the largest batch
    ("bf16", 2048, 1, 2, 64, 16, [(i * 31) % 40 for i in range(2048)]),
]


@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-B{s[1]}h{s[2]}g{s[3]}d{s[4]}p{s[5]}n{max(s[6])}")
def test_attention(shape, weights):
    c = Cache(*shape, sigma=1.5, seed=len(shape[6]) + shape[4])
    before = c.weight.cpu().numpy().astype(np.float64) if weights else None
    out = c.attend(weights)
    assert status() == 0
    check_attention(c, before, out, c.weight.cpu().numpy().astype(np.float64) if weights else None)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1100])
@pytest.mark.parametrize("dtype,page,d", [("bf16", 16, 128), ("f32", 64, 64), ("bf16", 256, 64), ("f32", 32, 128)])
def test_attention_lengths(n, dtype, page, d):
    c = Cache(dtype, 2, 2, 3, d, page, [n, max(n - 1, 0)], seed=n, sigma=2.0)
    before = c.weight.cpu().numpy().astype(np.float64)
    out = c.attend()
    assert status() == 0
    check_attention(c, before, out, c.weight.cpu().numpy().astype(np.float64))


def test_attention_long_and_short_together():
    """One long sequence among short and empty ones: units cut over many parts
    beside parts that hold many units."""
    for dtype in ("bf16", "f32"):
        c = Cache(dtype, 6, 2, 4, 128, 32, [3, 20011, 0, 64, 1, 500], seed=5, sigma=2.0)
        before = c.weight.cpu().numpy().astype(np.float64)
        out = c.attend()
        assert status() == 0
        check_attention(c, before, out, c.weight.cpu().numpy().astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_rows_behind_the_end_may_hold_anything(dtype):
    import torch
    c = Cache(dtype, 3, 2, 4, 128, 64, [70, 1, 0], seed=6)
    for x, bad in ((c.kp, float("nan")), (c.vp, float("inf"))):
        keep = torch.zeros(x.shape[0], 64, dtype=torch.bool, device="cuda")
        for b, n in enumerate([70, 1, 0]):
            for t in range(n):
                keep[c.table[b, t // 64].item(), t % 64] = True
        x.masked_fill_(~keep[:, None, :, None], bad)
        x[~keep[:, None, :, None].expand_as(x)] = float("nan") if x is c.vp else bad
    before = c.weight.cpu().numpy().astype(np.float64)
    out = c.attend()
    assert status() == 0
    kp, vp = c.kp, c.vp
    c.kp, c.vp = torch.nan_to_num(kp, 0.0), torch.nan_to_num(vp, 0.0)
    check_attention(c, before, out, c.weight.cpu().numpy().astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_bad_pages_and_lengths(dtype):
    """Entries of the page table outside the pool hold nothing; lengths are clamped."""
    c = Cache(dtype, 4, 2, 3, 64, 16, [100, 48, 40, 33], max_pages=7, seed=7)
    c.table[0, 2], c.table[0, 6], c.table[1, :] = -1, c.dims.n_pages, 2 ** 31 - 1
    c.lens[2], c.lens[3] = -5, 10 ** 6
    before = c.weight.cpu().numpy().astype(np.float64)
    out = c.attend()
    assert status() == 1 and status() == 0
    assert np.all(out[1].cpu().numpy() == 0)   # a sequence whose every page is bad
    check_attention(c, before, out, c.weight.cpu().numpy().astype(np.float64))


def test_attention_sharp_and_flat_softmax():
    import torch
    for sigma in (0.0, 30.0):
        c = Cache("bf16", 1, 2, 4, 128, 16, [777], sigma=sigma, seed=8)
        before = c.weight.cpu().numpy().astype(np.float64)
        out = c.attend()
        check_attention(c, before, out, c.weight.cpu().numpy().astype(np.float64))
    # one token far above all others takes everything: out is its value
    c = Cache("bf16", 1, 1, 2, 128, 16, [300], seed=9)
    c.pos.zero_()
    c.kp.zero_()
    c.kp[c.table[0, 200 // 16], 0, 200 % 16] = c.q[0, 0]
    c.q[0, 1] = c.q[0, 0]
    c.kp *= 100
    out = c.attend(False)
    v = c.vp[c.table[0, 200 // 16], 0, 200 % 16].float()
    assert torch.equal(out[0, 0], v) and torch.equal(out[0, 1], v)


def test_attention_shared_pages_and_far_positions():
    """Two sequences read the same pages; a position near 2^31 turns exactly."""
    import torch
    c = Cache("bf16", 2, 2, 2, 128, 16, [40, 35], max_pages=4, seed=10)
    c.table[1] = c.table[0]
    c.pos = torch.tensor([2 ** 31 - 1, 1], dtype=torch.int32, device="cuda")
    before = c.weight.cpu().numpy().astype(np.float64)
    out = c.attend()
    check_attention(c, before, out, c.weight.cpu().numpy().astype(np.float64))


def test_attention_equal_calls_give_equal_bits_and_streams():
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_attention, fasa_paged_workspace_size
    c = Cache("bf16", 5, 4, 4, 128, 32, [5000, 1, 0, 333, 4097], seed=11, sigma=2.0)
    w0 = c.weight.clone()
    out = c.attend().clone()
    w1 = c.weight.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # garbage in the workspace, another stream, two calls at once with a workspace each
    runs = []
    for s in (torch.cuda.current_stream(), side):
        ws = torch.full((fasa_paged_workspace_size(c.dims, True),), 0xFF, dtype=torch.uint8, device="cuda")
        w, o = w0.clone(), torch.empty_like(out)
        runs.append((s, ws, w, o))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, ws, w, o in runs:
            w.copy_(w0) if s is not side else None
            with torch.cuda.stream(s):
                if s is side:
                    w.copy_(w0)
                fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, c.lens, o, weight=w, workspace=ws, dims=c.dims)
    torch.cuda.synchronize()
    for _, _, w, o in runs:
        assert torch.equal(o, out) and torch.equal(w, w1)


def test_calls_of_two_threads():
    """Caches of another type, head size and rotation base each, a stream each:
    what the library keeps between calls is not mixed up."""
    import threading
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_append, fasa_paged_evict

    def steps(c, k, v):
        outs = []
        for i in range(25):
            fasa_paged_append(k, v, c.pos, c.kp, c.vp, c.table, c.lens, weight=c.weight, token_pos=c.token_pos,
                              dims=c.dims)
            c.lens.add_(1)
            outs.append(c.attend().clone())
            fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, c.lens, 300, new := c.lens.clone(),
                             sinks=2, recent=9, dims=c.dims)
            c.lens.copy_(new)
            c.pos.add_(1)
        return torch.stack(outs)

    def make(i):
        c = Cache(*(("bf16", 3, 4, 4, 128, 16, [299, 300, 7]) if i else ("f32", 2, 2, 8, 64, 32, [298, 40])),
                  max_pages=24 if i else 12, theta=1e4 if i else 1e6, seed=60 + i)
        k, v = (torch.randn(c.B, c.Hkv, c.d, generator=c.gen, device="cuda").to(c.q.dtype) for _ in range(2))
        return c, k, v

    alone = [steps(*make(i)) for i in range(2)]
    made, got = [make(i) for i in range(2)], [None, None]
    torch.cuda.synchronize()

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got[i] = steps(*made[i])
        s.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(g, a) for g, a in zip(got, alone)) and status() == 0


def test_attention_in_graphs_that_share_a_workspace():
    """Two captured graphs over one workspace, replayed in turn with new lengths and queries."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_attention, fasa_paged_workspace_size
    a = Cache("bf16", 2, 2, 4, 128, 16, [900, 37], max_pages=60, seed=12)
    b = Cache("bf16", 3, 2, 4, 128, 32, [5, 64, 2000], max_pages=64, seed=13)
    ws = torch.empty(max(fasa_paged_workspace_size(x.dims, True) for x in (a, b)), dtype=torch.uint8, device="cuda")
    graphs = []
    for c in (a, b):
        c.attend(workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, c.lens, c.out, weight=c.weight, workspace=ws,
                                 dims=c.dims)
        graphs.append(g)
    for step in range(3):
        before = [c.weight.cpu().numpy().astype(np.float64) for c in (a, b)]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, w in zip((a, b), before):
            check_attention(c, w, c.out, c.weight.cpu().numpy().astype(np.float64))
        a.lens[0], b.lens[1] = 100 * (step + 1), 0
        a.q.copy_(torch.randn(a.q.shape, generator=a.gen, device="cuda"))
    assert status() == 0


def test_attention_bounded_waits():
    """A copy that is never issued: its wait runs out within the bound, the call says
    so and drains what it has under way, and the next call gives the bits of the
    first.  (The wait is on a barrier in shared memory that no copy targets.)"""
    import torch
    from kv_cache_token_tip_gb300 import FASA_DEV_TIMEOUT, FASA_DEV_UNDRAINED, fasa_test_fault_injection
    for dtype in ("bf16", "f32"):
        c = Cache(dtype, 2, 4, 4, 128, 32, [9000, 5000], seed=14)
        ref = c.attend(False).clone()
        assert status() == 0
        try:
            fasa_test_fault_injection(wait_limit_ns=2_000_000)
            assert torch.equal(c.attend(False), ref) and status() == 0   # a short bound alone changes nothing
            fasa_test_fault_injection(wait_limit_ns=2_000_000, drop_tip_tile=1)
            c.attend(False)
            assert status() == FASA_DEV_TIMEOUT | FASA_DEV_UNDRAINED
        finally:
            fasa_test_fault_injection()
        assert torch.equal(c.attend(False), ref) and status() == 0


def test_attention_reads_no_entry_behind_the_end():
    """Entries of the page table behind a sequence's last page may be anything."""
    c = Cache("bf16", 3, 2, 2, 128, 16, [33, 16, 0], max_pages=9, seed=15)
    for b, n in enumerate([33, 16, 0]):
        c.table[b, -(-n // 16):] = -7
    out = c.attend()
    assert status() == 0
    before = c.weight.cpu().numpy().astype(np.float64)
    check_attention(c, before, c.attend(), c.weight.cpu().numpy().astype(np.float64))
    assert out is c.out and status() == 0
    new = _run_evict(c, 9, 1, 2)   # (an eviction reads none either)
    assert new.tolist() == [9, 9, 0] and status() == 0


def test_offsets_past_32_bits():
    """Pools of more than 2^32 elements, used at their far end by all three calls."""
    import torch
    from kv_cache_token_tip_gb300 import (FasaPagedDims, fasa_paged_append, fasa_paged_attention, fasa_paged_evict)
    small = Cache("bf16", 2, 8, 4, 128, 16, [200, 77], max_pages=14, seed=16, spare=0)
    used, n_pages = small.kp.shape[0], 270_000
    shape = (n_pages, 8, 16, 128)
    assert n_pages * 8 * 16 * 128 > 2 ** 32
    kp, vp = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp[-used:], vp[-used:] = small.kp, small.vp
    d = small.dims
    dims = FasaPagedDims(d.batch, d.n_q_heads, d.n_kv_heads, d.head_dim, d.page_size, n_pages, d.max_pages, d.dtype,
                         d.rope_theta)
    far = small.table + (n_pages - used)
    out, w, tp = torch.empty_like(small.out), small.weight.clone(), small.token_pos.clone()
    k_new = torch.randn((2, 8, 128), generator=small.gen, device="cuda").bfloat16()
    new = [torch.zeros_like(small.lens) for _ in range(2)]
    for kk, vv, table, dd, o, ww, tt, nn in ((kp, vp, far, dims, out, w, tp, new[0]),
                                             (small.kp, small.vp, small.table, d, small.out, small.weight,
                                              small.token_pos, new[1])):
        fasa_paged_append(k_new, k_new, small.pos, kk, vv, table, small.lens, weight=ww, token_pos=tt, dims=dd)
        fasa_paged_attention(small.q, small.pos, kk, vv, table, small.lens + 1, o, weight=ww, dims=dd)
        fasa_paged_evict(ww, tt, small.pos, kk, vv, table, small.lens + 1, 60, nn, 2, 9, dims=dd)
    assert status() == 0
    assert torch.equal(out, small.out) and torch.equal(w, small.weight) and torch.equal(tp, small.token_pos)
    assert torch.equal(kp[-used:], small.kp) and torch.equal(vp[-used:], small.vp) and torch.equal(*new)


def test_calls_wait_for_copies_and_events_between_them():
    """What comes between two of the calls in a stream, a copy or an event of
    another stream, is waited for although the second call begins early."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_append, fasa_paged_attention
    c = Cache("bf16", 4, 8, 4, 128, 16, [700, 600, 500, 400], max_pages=80, seed=17)
    n = 200
    k_new = torch.randn((4 * n, 8, 128), generator=c.gen, device="cuda").bfloat16()
    cu = torch.arange(0, 4 * n + 1, n, dtype=torch.int32, device="cuda")
    after = c.lens + n
    host = after.cpu().pin_memory()

    def append():
        fasa_paged_append(k_new, k_new, c.pos, c.kp, c.vp, c.table, c.lens, cu_new=cu, dims=c.dims)

    def attend(lens):
        fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, lens, c.out, dims=c.dims)

    append()
    torch.cuda.synchronize()
    attend(after)
    ref = c.out.clone()
    lens, side = torch.zeros_like(after), torch.cuda.Stream()
    for i in range(10):
        lens.zero_()
        torch.cuda.synchronize()
        append()
        lens.copy_(host, non_blocking=True)
        attend(lens)
        assert torch.equal(c.out, ref)
        lens.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000 * (i % 3))
            lens.copy_(after)
        append()
        torch.cuda.current_stream().wait_stream(side)
        attend(lens)
        assert torch.equal(c.out, ref)
    g, lens2 = torch.cuda.CUDAGraph(), torch.zeros_like(after)
    with torch.cuda.graph(g):   # the same in a graph, with a copy and a kernel between
        append()
        lens2.copy_(after)
        attend(lens2)
        lens2.zero_()
    for _ in range(5):
        c.out.zero_()
        g.replay()
        assert torch.equal(c.out, ref)
    assert status() == 0


def test_own_workspace_of_a_call_on_another_stream():
    """Without a workspace the call's own one outlives it on the stream it runs on."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_attention, fasa_paged_evict
    c = Cache("bf16", 2, 8, 4, 128, 32, [9000, 4000], seed=18, sigma=2.0)
    w0 = c.weight.clone()
    ref = c.attend().clone()
    w1, new = c.weight.clone(), torch.zeros_like(c.lens)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        c.weight.copy_(w0)
        c.out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(3_000_000)
        fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, c.lens, c.out, weight=c.weight, dims=c.dims,
                             stream=stream)
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(40)]
        torch.cuda.synchronize()
        assert torch.equal(c.out, ref) and torch.equal(c.weight, w1) and len(junk) == 40
    fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, c.lens, 100, new, dims=c.dims, stream=side)
    torch.cuda.synchronize()
    assert new.tolist() == [100, 100] and status() == 0


def test_own_workspaces_of_calls_on_two_streams_at_once():
    """A call without a workspace on the current stream, held up there, then one on
    another stream, with nothing between them: neither uses what the other does."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_attention, fasa_paged_evict

    def make(seed):
        return Cache("bf16", 2, 8, 4, 128, 32, [9000 - seed, 4000 + seed], max_pages=300, seed=seed, sigma=2.0)

    def run(c, new, stream):
        fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, c.lens, c.out, weight=c.weight, dims=c.dims,
                             stream=stream)
        fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, c.lens, 2500, new, sinks=4, recent=100,
                         dims=c.dims, stream=stream)

    def state(c, new):
        return [x.clone() for x in (c.out, c.weight, c.token_pos, c.kp, c.vp, new)]

    alone, side = [], torch.cuda.Stream()
    for seed in (30, 31):
        c, new = make(seed), torch.zeros(2, dtype=torch.int32, device="cuda")
        run(c, new, None)
        alone.append(state(c, new))
    torch.cuda.synchronize()
    for first, second in ((None, side), (side.cuda_stream, None), (None, side.cuda_stream), (side, None)):
        both = [(make(seed), torch.zeros(2, dtype=torch.int32, device="cuda")) for seed in (30, 31)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side if first is not None else torch.cuda.current_stream()):
            torch.cuda._sleep(3_000_000)
        run(*both[0], first)
        run(*both[1], second)
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            assert all(torch.equal(x, y) for x, y in zip(state(*got), want))
    assert status() == 0


# ---------------------------------------------------------------------- append
def _append_ref(c, k_new, v_new, cu, kp, vp, w, tp):
    PO.paged_append(c.host(k_new), c.host(v_new), cu, c.pos.cpu().numpy(), c.table.cpu().numpy(),
                    c.lens.cpu().numpy(), kp, vp, w, tp, c.theta)


def _check_append(c, k_new, v_new, cu, got, ref, k_before):
    kp, vp, w, tp = got
    rk, rv, rw, rt = ref
    # the rows written are those of the oracle, the others keep their bits
    written = np.any(rk != k_before, axis=-1) | np.any(rv != c.v_before, axis=-1)
    gk = c.host(kp)
    assert np.array_equal(gk[~written], k_before[~written])
    norm = np.sqrt(rk[..., 0::2] ** 2 + rk[..., 1::2] ** 2).repeat(2, -1)
    bound = 2e-6 * norm + EPS[c.dtype] * (np.abs(rk) + 2e-6 * norm)
    err = np.abs(gk - rk)[written]
    assert np.all(err <= bound[written] + 1e-38), f"{np.max(err / (bound[written] + 1e-38)):.3g}x the bound"
    assert np.array_equal(c.host(vp), rv)
    if w is not None:
        assert np.array_equal(w.cpu().numpy().astype(np.float64), rw)
    if tp is not None:
        assert np.array_equal(tp.cpu().numpy(), rt)
    return int(written.sum())


def _run_append(c, news, stats=True, cu=None, pad=0):
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_append
    n = sum(news) + pad
    dt = c.kp.dtype
    k_new = torch.randn((n, c.Hkv, c.d), generator=c.gen, device="cuda").to(dt)
    v_new = torch.randn((n, c.Hkv, c.d), generator=c.gen, device="cuda").to(dt)
    cu_host = [sum(news[:i]) for i in range(len(news) + 1)]
    cu_dev = None if cu is None else torch.tensor(cu_host, dtype=torch.int32, device="cuda")
    ref = [c.host(c.kp).copy(), c.host(c.vp).copy(), c.weight.cpu().numpy().astype(np.float64),
           c.token_pos.cpu().numpy().copy()]
    k_before, c.v_before = ref[0].copy(), ref[1].copy()
    if not stats:
        ref[2:] = [None, None]
    _append_ref(c, k_new, v_new, cu_host, *ref)
    fasa_paged_append(k_new, v_new, c.pos, c.kp, c.vp, c.table, c.lens, cu_new=cu_dev,
                      weight=c.weight if stats else None, token_pos=c.token_pos if stats else None, dims=c.dims)
    return _check_append(c, k_new, v_new, cu_host, (c.kp, c.vp, c.weight if stats else None,
                                                    c.token_pos if stats else None), ref, k_before)


@pytest.mark.parametrize("dtype,B,Hkv,d,page,lens,news", [
    ("bf16", 1, 1, 64, 16, [0], [1]), ("bf16", 3, 8, 128, 16, [15, 16, 40], [1, 1, 1]),
    ("f32", 2, 3, 64, 32, [31, 0], [1, 70]), ("bf16", 4, 2, 128, 64, [1, 64, 0, 7], [0, 130, 1, 33]),
    ("f32", 3, 5, 128, 128, [3, 500, 127], [257, 1, 2]), ("bf16", 7, 7, 64, 256, [i * 9 for i in range(7)], [5] * 7),
    ("bf16", 2, 8, 128, 16, [100, 3], [600, 1500])])
def test_append(dtype, B, Hkv, d, page, lens, news):
    cap = max(n + m for n, m in zip(lens, news))
    c = Cache(dtype, B, Hkv, 1, d, page, lens, max_pages=-(-cap // page) + 1, seed=20, theta=1e4)
    assert _run_append(c, news, cu=True) == sum(news) * Hkv
    if all(m == 1 for m in news):
        assert _run_append(c, news) == B * Hkv
        assert _run_append(c, news, stats=False) == B * Hkv
    assert status() == 0


def test_append_padding_is_left_out():
    c = Cache("bf16", 2, 2, 1, 128, 16, [3, 20], max_pages=3, seed=21)
    assert _run_append(c, [2, 5], cu=True, pad=9) == 14 and status() == 0


def test_append_bad_slots_pages_and_tables():
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_append
    c = Cache("f32", 4, 2, 1, 64, 16, [30, 2, 5, 5], max_pages=2, seed=22)
    c.table[1, 0] = -1
    c.table[2, 0] = c.dims.n_pages
    c.lens[3] = -2
    # sequence 0 runs out of slots after two tokens, the others have no page or length
    assert _run_append(c, [4, 1, 1, 1], cu=True) == 4
    assert status() == 1
    k = torch.randn((4, 2, 64), device="cuda")
    before = c.kp.clone()
    for cu in ([1, 2, 3, 4, 4], [0, 5, 3, 2, 4], [0, 0, 0, 0, 9]):
        c.lens.fill_(0)
        c.lens[1:3] = -1
        cu_new = torch.tensor(cu, dtype=torch.int32, device="cuda")
        fasa_paged_append(k, k, c.pos, c.kp, c.vp, c.table, c.lens, cu_new=cu_new, dims=c.dims)
        assert status() == 1
    assert c.kp.shape == before.shape


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("cu,taken", [
    # cu_new, and how many of its own rows each sequence gets
    ([0, 4, 9], [4, 0]),            # the second range runs past the rows, none of which it has
    ([0, 5, 3], [0, 0]), ([0, 2, 1], [1, 0]), ([0, 4, -1], [0, 0]),    # descends at the end
    ([0, 0, 5], [0, 0]),            # past the rows
    ([1, 2, 4], [1, 2]), ([-1, 2, 4], [0, 2]), ([1, 1, 1], [0, 0]),    # does not begin at 0
    ([0, 9, 4], [0, 0]), ([0, 9, 0], [0, 0]),
    ([0, 1, 4, 2, 4], None), ([0] * 150 + [9, 4], [0] * 151), ([0, 4] + [9] * 150, [4] + [0] * 150),
    ([0, 4, 3] + [4] * 150, None),
    # and tables that are right
    ([0, 4, 4], [4, 0]), ([0, 0, 0], [0, 0]), ([0] * 300 + [3], [0] * 299 + [3])],
    ids=lambda x: f"{x[:5]}{len(x)}".replace(" ", "") if isinstance(x, list) else None)
def test_append_tables_of_rows(cu, taken, dtype, d):
    """A table of rows that does not ascend from 0 within the rows is reported,
    wherever it is wrong; rows without a sequence and all other pages keep out."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_append
    rows, B = 4, len(cu) - 1
    right = cu[0] == 0 and all(a <= b for a, b in zip(cu, cu[1:])) and cu[-1] <= rows
    c = Cache(dtype, B, 2, 1, d, 16, [(3 * i) % 29 for i in range(B)], max_pages=3, seed=24)
    k_new, v_new = (torch.randn((rows, 2, d), generator=c.gen, device="cuda").to(c.kp.dtype) for _ in range(2))
    ref = [c.host(c.kp).copy(), c.host(c.vp).copy(), c.weight.cpu().numpy().astype(np.float64),
           c.token_pos.cpu().numpy().copy()]
    k_before, c.v_before = ref[0].copy(), ref[1].copy()
    if taken is not None:
        for b, n in enumerate(taken):   # one sequence at a time, from its first row
            if n:
                only = [0] * (b + 1) + [n] * (B - b)
                at = slice(cu[b], cu[b] + n)
                _append_ref(c, k_new[at], v_new[at], only, *ref)
    fasa_paged_append(k_new, v_new, c.pos, c.kp, c.vp, c.table, c.lens,
                      cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"), weight=c.weight,
                      token_pos=c.token_pos, dims=c.dims)
    assert status() == (0 if right else 1) and status() == 0
    if taken is not None:
        assert _check_append(c, k_new, v_new, cu, (c.kp, c.vp, c.weight, c.token_pos), ref, k_before) == 2 * sum(taken)


# ---------------------------------------------------------------------- evict
def _run_evict(c, keep, sinks=0, recent=0, apart=False):
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_evict
    kp, vp = c.host(c.kp).copy(), c.host(c.vp).copy()
    w, tp = c.weight.cpu().numpy().copy(), c.token_pos.cpu().numpy().copy()
    wo = torch.full_like(c.weight, -7.0) if apart else c.weight
    to = torch.full_like(c.token_pos, -7) if apart else c.token_pos
    rwo, rto = (wo.cpu().numpy().copy(), to.cpu().numpy().copy()) if apart else (w, tp)
    new = torch.full((c.B,), -1, dtype=torch.int32, device="cuda")
    w0, tp0 = c.weight.clone(), c.token_pos.clone()
    ref_new = PO.paged_evict(w, tp, c.pos.cpu().numpy(), c.table.cpu().numpy(), c.lens.cpu().numpy(), keep, sinks,
                             recent, kp, vp, rwo, rto)
    fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, c.lens, keep, new, sinks=sinks,
                     recent=recent, weight_out=wo if apart else None, token_pos_out=to if apart else None,
                     dims=c.dims)
    assert np.array_equal(new.cpu().numpy(), ref_new)
    assert np.array_equal(to.cpu().numpy(), rto)
    assert np.array_equal(wo.cpu().numpy(), rwo, equal_nan=True)
    assert np.array_equal(c.host(c.kp), kp) and np.array_equal(c.host(c.vp), vp)
    if apart:
        assert torch.equal(c.token_pos, tp0) and torch.equal(torch.nan_to_num(c.weight), torch.nan_to_num(w0))
    return new


EVICTS = [
    # dtype, B, Hkv, d, page, lengths, keep, sinks, recent
    ("bf16", 1, 1, 64, 16, [2], 1, 0, 0), ("f32", 1, 1, 64, 16, [1], 1, 0, 1),
    ("bf16", 3, 2, 128, 16, [0, 33, 32], 32, 4, 8), ("f32", 2, 3, 128, 32, [100, 99], 98, 0, 0),
    ("bf16", 2, 8, 128, 64, [1000, 513], 512, 4, 100), ("bf16", 1, 2, 64, 256, [3000], 7, 2, 5),
    ("f32", 5, 2, 64, 16, [17, 40, 16, 300, 0], 16, 16, 0), ("bf16", 1, 1, 128, 128, [5000], 4999, 0, 0),
    ("bf16", 2, 4, 128, 16, [9000, 8200], 1025, 0, 1025), ("bf16", 1, 2, 128, 64, [20000], 4096, 4, 256),
    # clusters of 1 with long shares, of 2, and of 16 with a share near the most
    ("bf16", 40, 4, 64, 64, [5000 - 61 * (i % 9) for i in range(40)], 4700, 4, 32),
    ("f32", 30, 4, 64, 16, [2500 + i for i in range(30)], 2510, 1, 0), ("bf16", 1, 1, 64, 256, [230001], 1200, 3, 99),
    # more moves than a CTA lists at once, on a cluster of 16 and on one CTA
    ("bf16", 1, 1, 64, 256, [200003], 100001, 4, 64), ("bf16", 40, 4, 64, 64, [6850 - i for i in range(40)], 3400, 4, 32),
    # more units than SMs can hold of the wide CTAs, a few and many tokens over
    ("bf16", 85, 4, 128, 16, [300 + i % 21 for i in range(85)], 305, 4, 32),
    ("f32", 90, 4, 128, 16, [280 - i for i in range(90)], 270, 0, 3), ("bf16", 170, 2, 64, 64, [900 - i for i in range(170)], 333, 4, 32),
]


@pytest.mark.parametrize("apart", [False, True], ids=["in_place", "apart"])
@pytest.mark.parametrize("case", EVICTS, ids=lambda c: f"{c[0]}-B{c[1]}h{c[2]}d{c[3]}p{c[4]}n{max(c[5])}k{c[6]}")
def test_evict(case, apart):
    dtype, B, Hkv, d, page, lens, keep, sinks, recent = case
    c = Cache(dtype, B, Hkv, 1, d, page, lens, seed=30 + keep)
    c.pos = (c.lens - 1).clamp_min(0)
    new = _run_evict(c, keep, sinks, recent, apart)
    assert status() == 0
    if not apart:   # again: nothing is over the bound
        c.lens = new
        _run_evict(c, keep, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "nan", "extreme", "rising", "falling", "near"])
@pytest.mark.parametrize("n,keep", [(40, 13), (3000, 1234), (20001, 20000), (20001, 3)])
def test_evict_hard_weights(kind, n, keep):
    """Ties, signed zeros, NaN and infinities, sorted weights, weights one step apart."""
    import torch
    c = Cache("bf16", 1, 2, 1, 64, 16, [n], seed=n + keep)
    shape, cap = c.weight.shape, c.cap
    t = torch.arange(cap, device="cuda").expand(shape)
    if kind == "equal":
        c.weight.fill_(2.5)
    elif kind == "few":
        c.weight.copy_(torch.randint(0, 3, shape, generator=c.gen, device="cuda"))
    elif kind == "zeros":
        c.weight.copy_(torch.where(torch.rand(shape, generator=c.gen, device="cuda") < 0.5, 0.0, -0.0))
    elif kind == "nan":
        c.weight.masked_fill_(torch.rand(shape, generator=c.gen, device="cuda") < 0.7, float("nan"))
        c.weight[:, :, ::3] *= -1
    elif kind == "extreme":
        vals = torch.tensor([float("inf"), -float("inf"), 3.4e38, -3.4e38, 1e-45, -1e-45, 0.0, 1.0], device="cuda")
        c.weight.copy_(vals[torch.randint(0, 8, shape, generator=c.gen, device="cuda")])
    elif kind == "rising":
        c.weight.copy_(t.float())
    elif kind == "falling":
        c.weight.copy_(-t.float())
    else:
        c.weight.copy_((torch.randint(0, 4 * n, shape, generator=c.gen, device="cuda") + 0x3F800000).to(
            torch.int32).view(torch.float32))
    c.pos = c.lens - 1
    for sinks, recent in ((0, 0), (1, 2)):
        if sinks + recent <= keep:
            _run_evict(c, keep, sinks, recent, apart=True)
    assert status() == 0


def test_evict_shuffled_positions_and_held_overflow():
    """Positions in any order, and more held tokens than `keep` (the lower slots stay)."""
    import torch
    c = Cache("f32", 2, 2, 1, 64, 16, [700, 650], seed=40)
    perm = torch.stack([torch.randperm(c.cap, generator=c.gen, device="cuda") for _ in range(4)])
    c.token_pos.copy_(perm.view(2, 2, -1))
    c.pos = torch.tensor([690, 640], dtype=torch.int32, device="cuda")
    _run_evict(c, 100, 10, 50, apart=True)
    c.token_pos.fill_(3)
    _run_evict(c, 100, 10, 50, apart=True)   # every token is a sink
    c.token_pos.fill_(-2 ** 31)
    c.pos.fill_(-2 ** 31)
    _run_evict(c, 64, 0, 64)
    assert status() == 0


@pytest.mark.parametrize("over", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n", [20, 3000, 9000, 33000])
def test_evict_a_few(n, over):
    """A few tokens over the bound, on one CTA and on clusters: the order's last
    ones go, among weights, ties, NaN and held tokens."""
    import torch
    for kind in ("plain", "ties", "nan", "held", "struck"):
        c = Cache("bf16", 3, 2, 1, 64, 16, [n, n - 1, max(n - over, 1)], seed=n + over)
        c.pos = c.lens - 1
        if kind == "ties":
            c.weight.fill_(0.5)
        elif kind == "nan":   # NaN goes first, the higher slots of it
            c.weight[:, :, ::max(n // 7, 1)] = float("nan")
        elif kind == "held":
            c.token_pos.fill_(0)
        elif kind == "struck":   # weights whose order ends in the last CTA's share
            c.weight.copy_(torch.arange(c.cap, 0, -1, device="cuda").float().expand(c.weight.shape))
        _run_evict(c, n - over, 3, 5 if kind != "held" else 0, apart=True)
        _run_evict(c, n - over, 3, 5 if kind != "held" else 0)
    assert status() == 0


@pytest.mark.parametrize("dtype,d,page", [("bf16", 64, 16), ("bf16", 128, 64), ("f32", 64, 16), ("f32", 128, 32)])
@pytest.mark.parametrize("over", [1, 3, 8, 9])
def test_evict_a_few_rows(dtype, d, page, over):
    """The few rows that move, of every type and size: the tokens that go lie before
    the bound in any order, behind it, or both; then with pages that are not there."""
    import torch
    for kind in ("before", "descending", "behind", "both", "bad"):
        c = Cache(dtype, 2, 3, 1, d, page, [300, 300 - over], max_pages=-(-304 // page), seed=over)
        c.pos = c.lens - 1
        keep = 300 - over
        c.weight.copy_(1 + torch.rand(c.weight.shape, generator=c.gen, device="cuda"))
        for i in range(over):
            slot = {"before": 3 + 17 * i, "descending": 290 - over - 17 * i, "behind": 299 - i,
                    "both": 299 - i if i % 2 else 40 + i, "bad": 20 * i}[kind]
            c.weight[:, :, slot] = 0.1 + 0.01 * i
        if kind == "bad":
            c.table[0, 0], c.table[0, (300 - over) // page] = -1, c.dims.n_pages
        _run_evict(c, keep, 0, 0)
        assert status() == (1 if kind == "bad" else 0)


@pytest.mark.parametrize("B,cap", [(80, 16400), (20, 70016), (10, 140000)])
def test_evict_many_clusters(B, cap):
    """Clusters of 2, 8 and 16, more CTAs than two to an SM, of caches with room for
    far more than they hold (table entries behind the end are not pages)."""
    import torch
    for over in (1, 7, 150):
        c = Cache("bf16", B, 2, 1, 64, 16, [600 - i for i in range(B)], seed=over)
        table = torch.full((B, cap // 16), -1, dtype=torch.int32, device="cuda")
        table[:, :c.table.shape[1]] = c.table
        c.table, c.dims.max_pages, c.cap = table, cap // 16, cap
        c.weight = torch.exp(torch.randn(B, 2, cap, generator=c.gen, device="cuda"))
        c.token_pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, 2, cap).contiguous()
        c.pos = c.lens - 1
        _run_evict(c, 600 - over, 4, 32, apart=over == 7)
        assert status() == 0


def test_evict_bound_of_the_whole_cache():
    """A bound that no length can pass needs no workspace and moves nothing."""
    c = Cache("bf16", 2, 2, 1, 64, 16, [64, 10], seed=42)
    for keep in (64, 1000):
        assert _run_evict(c, keep, 3, 5).tolist() == [64, 10]
        assert _run_evict(c, keep, 3, 5, apart=True).tolist() == [64, 10]
    assert status() == 0


def test_evict_bad_pages_and_lengths():
    c = Cache("bf16", 3, 2, 1, 64, 16, [100, 80, 60], max_pages=7, seed=41)
    c.table[0, 0], c.table[0, 5], c.table[1, 3] = -1, 10 ** 6, c.dims.n_pages
    c.lens[2] = 10 ** 6
    c.pos = c.lens.clamp(max=112) - 1
    _run_evict(c, 40, 2, 8)
    assert status() == 1 and status() == 0


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,d,page,G", [("bf16", 128, 16, 4), ("f32", 64, 32, 2)])
def test_decode_loop_of_a_bounded_cache(dtype, d, page, G):
    """A prompt, cut after it was read, then steps of append, attention with
    weights and eviction, every call against the oracle on the library's own
    state before it."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_append, fasa_paged_evict
    B, Hkv, keep = 3, 2, 64
    c = Cache(dtype, B, Hkv, G, d, page, [0, 0, 0], max_pages=-(-200 // page), seed=50, sigma=2.0)
    c.lens.zero_()
    c.pos.zero_()
    news = [150, 64, 3]
    assert _run_append(c, news, cu=True) == sum(news) * Hkv
    c.lens += torch.tensor(news, dtype=torch.int32, device="cuda")
    c.pos = c.lens - 1
    before = c.weight.cpu().numpy().astype(np.float64)
    check_attention(c, before, c.attend(), c.weight.cpu().numpy().astype(np.float64))
    c.lens = _run_evict(c, keep, 2, 10)
    for step in range(12):
        c.pos = c.pos + 1
        _run_append(c, [1] * B)
        c.lens = c.lens + 1
        before = c.weight.cpu().numpy().astype(np.float64)
        c.q = torch.randn(c.q.shape, generator=c.gen, device="cuda").to(c.q.dtype)
        check_attention(c, before, c.attend(), c.weight.cpu().numpy().astype(np.float64))
        c.lens = _run_evict(c, keep, 2, 10)
    assert c.lens.tolist() == [64, 64, 15] and status() == 0
    newest = c.token_pos[:2, :, :64].amax(-1).cpu().tolist()
    assert newest == [[161, 161], [75, 75]]


def test_each_call_sees_what_the_one_before_it_wrote():
    """Calls one behind the other in a stream, each reading what the last one
    writes: lengths from the eviction, rows from the append, weights from the
    attention; nothing in between that waits."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_append, fasa_paged_attention, fasa_paged_evict
    keep = 200
    c = Cache("bf16", 6, 4, 4, 128, 16, [3000, 201, 10, 0, 900, 200], max_pages=200, seed=61, sigma=2.0)
    c.pos = (c.lens - 1).clamp_min(0)
    first = [x.clone() for x in (c.kp, c.vp, c.weight, c.token_pos)]
    new, q0 = torch.zeros_like(c.lens), c.q.clone()
    k_new, v_new = c.kp[:6, :, 3].contiguous(), c.vp[:6, :, 5].contiguous()
    out = [torch.empty_like(c.out) for _ in range(3)]

    def calls(wait):
        fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, c.lens, out[0], weight=c.weight, dims=c.dims)
        wait()
        fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, c.lens, keep, new, 2, 16, dims=c.dims)
        wait()
        fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, new, out[1], weight=c.weight, dims=c.dims)
        wait()
        fasa_paged_append(k_new, v_new, c.pos, c.kp, c.vp, c.table, new, weight=c.weight, token_pos=c.token_pos,
                          dims=c.dims)
        wait()
        fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, new, out[2], dims=c.dims)
        wait()
        return [x.clone() for x in (c.kp, c.vp, c.weight, c.token_pos, new, *out)]

    ref = calls(torch.cuda.synchronize)
    assert new.tolist() == [200, 200, 10, 0, 200, 200]
    for _ in range(20):
        for x, y in zip((c.kp, c.vp, c.weight, c.token_pos), first):
            x.copy_(y)
        new.fill_(77)
        torch.cuda.synchronize()
        for x, y in zip(calls(lambda: None), ref):
            assert torch.equal(x, y)
    assert torch.equal(c.q, q0) and status() == 0


def test_lengths_written_and_read_in_turn():
    """Two length buffers that evictions with ever smaller bounds write in turn, each
    read by the attention and the eviction right behind: no call may see what a
    buffer held two evictions ago."""
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_attention, fasa_paged_evict
    keeps = [900, 700, 512, 333, 200, 100, 31, 5]

    def run(wait):
        c = Cache("bf16", 5, 4, 4, 64, 16, [1000, 950, 400, 30, 0], seed=62, sigma=2.0)
        c.pos = (c.lens - 1).clamp_min(0)
        bufs, lens, outs = [torch.zeros_like(c.lens) for _ in range(2)], c.lens, []
        torch.cuda.synchronize()
        for i, keep in enumerate(keeps):
            out = torch.empty_like(c.out)
            fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, lens, keep, bufs[i % 2], dims=c.dims)
            wait()
            lens = bufs[i % 2]
            fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, lens, out, weight=c.weight, dims=c.dims)
            wait()
            outs.append(out)
        torch.cuda.synchronize()
        return outs + [c.weight, c.token_pos, c.kp, c.vp, *bufs]

    ref = run(torch.cuda.synchronize)
    for _ in range(5):
        for x, y in zip(run(lambda: None), ref):
            assert torch.equal(x, y)
    assert status() == 0


def test_decode_steps_in_one_graph():
    """append, attention and eviction captured together and replayed give the
    bits of the same calls made one by one."""
    import torch
    from kv_cache_token_tip_gb300 import (fasa_paged_append, fasa_paged_attention, fasa_paged_evict,
                                          fasa_paged_evict_workspace_size, fasa_paged_workspace_size)
    keep, runs = 100, []
    for _ in range(2):
        c = Cache("bf16", 2, 2, 4, 128, 16, [100, 100], max_pages=7, seed=60)
        c.k_new, c.v_new = c.kp[0, :, :2].transpose(0, 1).contiguous(), c.vp[1, :, :2].transpose(0, 1).contiguous()
        c.ws = torch.empty(fasa_paged_workspace_size(c.dims, True), dtype=torch.uint8, device="cuda")
        c.ws2 = torch.empty(fasa_paged_evict_workspace_size(c.dims, keep), dtype=torch.uint8, device="cuda")
        c.after, c.new = c.lens + 1, torch.zeros(2, dtype=torch.int32, device="cuda")
        runs.append(c)

    def step(c):
        c.pos.add_(1)
        fasa_paged_append(c.k_new, c.v_new, c.pos, c.kp, c.vp, c.table, c.lens, weight=c.weight,
                          token_pos=c.token_pos, dims=c.dims)
        fasa_paged_attention(c.q, c.pos, c.kp, c.vp, c.table, c.after, c.out, weight=c.weight, workspace=c.ws,
                             dims=c.dims)
        fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, c.after, keep, c.new, sinks=2, recent=9,
                         workspace=c.ws2, dims=c.dims)

    a, b = runs
    step(a)
    step(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    for _ in range(5):
        step(a)
        g.replay()
    torch.cuda.synchronize()
    for x in ("kp", "vp", "weight", "token_pos", "out", "new"):
        assert torch.equal(getattr(a, x), getattr(b, x)), x
    assert status() == 0


def test_binding_refuses_what_does_not_fit():
    import torch
    from kv_cache_token_tip_gb300 import FasaError, fasa_paged_append, fasa_paged_attention, fasa_paged_evict
    c = Cache("bf16", 2, 2, 2, 64, 16, [20, 30], seed=70)
    a = dict(dims=c.dims)

    def attend(**kw):
        t = dict(q=c.q, pos=c.pos, kp=c.kp, vp=c.vp, table=c.table, lens=c.lens, out=c.out, weight=c.weight)
        t.update(kw)
        fasa_paged_attention(t["q"], t["pos"], t["kp"], t["vp"], t["table"], t["lens"], t["out"],
                             weight=t["weight"], dims=t.get("dims", c.dims), workspace=t.get("ws"))

    for bad in (dict(q=c.q.float()), dict(q=c.q.cpu()), dict(pos=c.pos.long()), dict(kp=c.kp[:-1]),
                dict(vp=c.vp.transpose(1, 2)), dict(table=c.table[:, :-1]), dict(lens=c.lens[:1]),
                dict(out=c.out.bfloat16()), dict(weight=c.weight[:, :1]), dict(out=c.out[:1])):
        with pytest.raises(ValueError):
            attend(**bad)
    with pytest.raises(FasaError):
        attend(ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    for keep, kw in ((0, {}), (8, dict(recent=9)), (8, dict(sinks=-1)), (8, dict(weight_out=torch.zeros_like(c.weight)))):
        with pytest.raises(FasaError):
            fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, c.lens, keep, new, dims=c.dims, **kw)
    with pytest.raises(FasaError):
        fasa_paged_evict(c.weight, c.token_pos, c.pos, c.kp, c.vp, c.table, c.lens, 8, c.lens, dims=c.dims)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(FasaError):   # three rows for two sequences, and no table of rows
        fasa_paged_append(k, k, c.pos, c.kp, c.vp, c.table, c.lens, **a)
    with pytest.raises(ValueError):
        fasa_paged_append(k, k[:2], c.pos, c.kp, c.vp, c.table, c.lens, cu_new=new[:1], **a)
    assert status() == 0


FIRST_CALLS = """
import torch
from kv_cache_token_tip_gb300 import fasa_paged_append, fasa_paged_attention, fasa_paged_evict
from kv_cache_token_tip_gb300.fasa import FasaPagedDims
B, H, G, d, page, n = 2, 2, 4, 128, 16, 6
dims = FasaPagedDims(B, H * G, H, d, page, B * n, n, 1, 1e4)
z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")
kp, vp = z(B * n, H, page, d, t=torch.bfloat16), z(B * n, H, page, d, t=torch.bfloat16)
table = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n)
lens, pos, new = z(B, t=torch.int32), z(B, t=torch.int32), z(B, t=torch.int32)
w, tp = z(B, H, n * page), z(B, H, n * page, t=torch.int32)
k, v = torch.ones(B, H, d, device="cuda").bfloat16(), torch.ones(B, H, d, device="cuda").bfloat16()
q, out = torch.ones(B, H * G, d, device="cuda").bfloat16(), z(B, H * G, d)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fasa_paged_append(k, v, pos, kp, vp, table, lens, weight=w, token_pos=tp, dims=dims)
    lens.add_(1)
    fasa_paged_attention(q, pos, kp, vp, table, lens, out, weight=w, dims=dims)
    fasa_paged_evict(w, tp, pos, kp, vp, table, lens, 4, new, dims=dims)
    lens.copy_(new)
    pos.add_(1)
for _ in range(9):
    g.replay()
torch.cuda.synchronize()
assert lens.tolist() == [4, 4] and pos.tolist() == [9, 9]
# out = o / l with o = l = the sum of at most 5 softmax weights, V being 1.  o: three products and a sum of four of
# the tensor cores, which round towards zero (4 * 2^-23), then at most 5 parts (5 * 2^-24); l: at most 7 sums of a
# part's lanes and 5 parts (12 * 2^-24); the division and the product 3 * 2^-24.  28 * 2^-24 in all.
assert (out - 1).abs().max() <= 28 * 2.0 ** -24, out
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
