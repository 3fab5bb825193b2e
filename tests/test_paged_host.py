"""The paged cache without a GPU: argument checks of the entry points, the
index arithmetic of the kernels compiled as plain C++, and pins of the oracle."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import paged_oracle as PO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    from kv_cache_token_tip_gb300 import build, lib
    build.build()
    return lib()


def _dims(**kw):
    from kv_cache_token_tip_gb300 import FasaPagedDims
    d = dict(batch=2, n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=16, n_pages=64, max_pages=32, dtype=1,
             rope_theta=5e5)
    d.update(kw)
    return FasaPagedDims(*[d[k] for k, _ in FasaPagedDims._fields_])


def _append(L, d, n=2, cu=None, k=P, v=P, pos=P, table=P, lens=P, kp=P, vp=P, w=P, tp=P):
    return L.fasa_paged_append(k, v, n, cu, pos, table, lens, kp, vp, w, tp, d and ctypes.byref(d), None)


def _attend(L, d, q=P, pos=P, kp=P, vp=P, table=P, lens=P, out=P, w=None, ws=P, n=1 << 40):
    return L.fasa_paged_attention(q, pos, kp, vp, table, lens, out, w, ws, n, d and ctypes.byref(d), None)


def _evict(L, d, w=P, tp=P, pos=P, table=P, lens=P, keep=100, sinks=4, recent=16, kp=P, vp=P, wo=P, tpo=P,
           new=2 * P, ws=P, n=1 << 40):
    return L.fasa_paged_evict(w, tp, pos, table, lens, keep, sinks, recent, kp, vp, wo, tpo, new, ws, n,
                              d and ctypes.byref(d), None)


BAD_DIMS = [
    (dict(batch=0), 1), (dict(n_kv_heads=0), 1), (dict(n_q_heads=30), 1), (dict(head_dim=7), 1),
    (dict(page_size=0), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(rope_theta=0.0), 1),
    (dict(rope_theta=float("nan")), 1), (dict(dtype=7), 2), (dict(head_dim=96), 2),
    (dict(n_q_heads=72, n_kv_heads=8), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
    (dict(page_size=512), 2), (dict(batch=2049), 2), (dict(batch=2048, n_kv_heads=32, n_q_heads=32), 2),
    (dict(max_pages=16385), 2), (dict(n_pages=1 << 24), 2),
]


@pytest.mark.parametrize("kw,code", BAD_DIMS)
def test_bad_dims_rejected(L, kw, code):
    d = _dims(**kw)
    n = ctypes.c_size_t(7)
    assert _append(L, d) == code and _attend(L, d) == code and _evict(L, d) == code
    assert L.fasa_paged_workspace_size(ctypes.byref(d), 1, ctypes.byref(n)) == code and n.value == 0
    assert L.fasa_paged_evict_workspace_size(ctypes.byref(d), 8, ctypes.byref(n)) == code and n.value == 0


def test_arguments_rejected_before_launch(L):
    d = _dims()
    assert _append(L, None) == 1 and _attend(L, None) == 1 and _evict(L, None) == 1
    for name in ("k", "v", "pos", "table", "lens", "kp", "vp"):
        assert _append(L, d, **{name: None}) == 1
    for name in ("k", "v", "kp", "vp", "w", "tp"):
        assert _append(L, d, **{name: P + 8}) == 1
    assert _append(L, d, n=3) == 1 and _append(L, d, n=-1, cu=P) == 1   # one per sequence, or a table of rows
    assert _append(L, d, n=0, cu=P) == 0   # nothing to write, nothing launched
    for name in ("q", "pos", "kp", "vp", "table", "lens", "out"):
        assert _attend(L, d, **{name: None}) == 1
    for name in ("q", "kp", "vp", "out", "w"):
        assert _attend(L, d, **{name: P + 4}) == 1
    for name in ("w", "tp", "pos", "table", "lens", "kp", "vp", "wo", "tpo", "new"):
        assert _evict(L, d, **{name: None}) == 1
    for name in ("w", "tp", "kp", "vp", "wo", "tpo"):
        assert _evict(L, d, **{name: P + 4}) == 1
    assert _evict(L, d, keep=0) == 1 and _evict(L, d, sinks=-1) == 1 and _evict(L, d, recent=-1) == 1
    assert _evict(L, d, keep=19) == 1    # sinks + recent > keep
    assert _evict(L, d, sinks=2 ** 31 - 1, recent=2 ** 31 - 1) == 1
    assert _evict(L, d, new=P) == 1 and _evict(L, d, new=P + 4) == 1      # new_lens is seq_lens, or overlaps it
    stat = 2 * 8 * 512 * 4
    A, B, C, D = (P + i * stat for i in range(4))
    assert _evict(L, d, w=A, tp=B, wo=A, tpo=C) == 1           # one in place, the other not
    assert _evict(L, d, w=A, tp=B, wo=A + 16, tpo=D) == 1      # overlapping
    assert _evict(L, d, w=A, tp=B, wo=B, tpo=A) == 1
    assert _evict(L, d, w=A, tp=B, wo=C, tpo=C) == 1
    assert _evict(L, d, w=A, tp=B, wo=A, tpo=B, ws=None) == 3 and _evict(L, d, w=A, tp=B, wo=C, tpo=D, n=0) == 3
    assert _evict(L, d, w=A, tp=B, wo=C, tpo=D, ws=P + 8) == 3


def test_workspace_sizes(L):
    d, n = _dims(), ctypes.c_size_t(0)
    size = L.fasa_paged_workspace_size
    assert size(ctypes.byref(d), 0, None) == 1
    assert size(ctypes.byref(d), 0, ctypes.byref(n)) == 0
    plain = n.value
    assert plain > 0 and _attend(L, d, n=plain - 1) == 3 and _attend(L, d, ws=None) == 3
    assert _attend(L, d, ws=P + 8) == 3
    assert size(ctypes.byref(d), 1, ctypes.byref(n)) == 0
    # with weights: every query head's logit of every slot
    assert n.value >= plain + 2 * 32 * 512 * 4 and _attend(L, d, w=P, n=n.value - 1) == 3
    ev = L.fasa_paged_evict_workspace_size
    assert ev(ctypes.byref(d), 0, ctypes.byref(n)) == 1 and ev(ctypes.byref(d), 8, None) == 1
    assert ev(ctypes.byref(d), 100, ctypes.byref(n)) == 0 and n.value >= 2 * 8 * 100 * 16
    assert ev(ctypes.byref(d), 500, ctypes.byref(n)) == 0 and n.value >= 2 * 8 * 12 * 16
    assert ev(ctypes.byref(d), 512, ctypes.byref(n)) == 0 and n.value == 0   # nothing can be over the bound


INDEX_PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "fasa_paged_index.h"
using namespace fasa;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

static std::vector<unsigned> words(const std::vector<int>& lens) {
  std::vector<unsigned> w;
  int before = 0;
  for (int n : lens) {
    w.push_back(paged_word(before, n));
    before += paged_groups(n);
  }
  w.push_back(paged_word(before, 0));
  return w;
}

// The parts cover the line once, in order; part_of is their inverse; the walk
// meets every unit's groups once, and the records of a cut unit are those of
// its first to its last part, none of them empty.
static int check(const std::vector<int>& lens, int Hkv, int grid) {
  const std::vector<unsigned> w = words(lens);
  const int B = (int)lens.size();
  const PagedLine line{w.data(), B, Hkv};
  int groups = 0;
  for (int b = 0; b < B; ++b) {
    CHECK(line.tokens(b) == lens[b] && line.groups(b) == paged_groups(lens[b]));
    groups += paged_groups(lens[b]);
  }
  CHECK(line.total() == groups * Hkv);
  const PagedCuts cuts = line.cuts(grid);
  const int n = cuts.n;
  CHECK(n >= 1 && n <= grid);
  CHECK(line.part_begin(cuts, 0) == 0 && line.part_begin(cuts, n) == line.total());
  std::vector<int> seen(B * Hkv, 0), last(B * Hkv, -1);
  long long most = 0;
  for (int c = 0; c < n; ++c) {
    const int r0 = line.part_begin(cuts, c), r1 = line.part_begin(cuts, c + 1);
    CHECK(r0 <= r1);
    PagedSegments s;
    s.start(line, r0, r1);
    long long cost = 0;
    for (; s.at(); s.next()) {
      CHECK(s.b < B && s.h < Hkv && s.x >= s.unit_begin && s.x < s.seg_end());
      CHECK(s.unit_end - s.unit_begin == line.groups(s.b));
      const int u = s.unit();
      CHECK(s.x - s.unit_begin == seen[u]);
      for (int x = s.x; x < s.seg_end(); ++x) CHECK(line.part_of(cuts, s.b, s.h, x - s.unit_begin) == c);
      if (seen[u]) CHECK(last[u] == c - 1);
      else CHECK(s.first_part(cuts) == c);
      seen[u] += s.seg_end() - s.x;
      last[u] = c;
      if (seen[u] == line.groups(s.b)) CHECK(s.last_part(cuts) == c);
      else CHECK(s.last_part(cuts) > c);
      cost += s.seg_end() - s.x + (s.x == s.unit_begin ? PAGED_UNIT_COST : 0);
    }
    most = cost > most ? cost : most;
  }
  for (int u = 0; u < B * Hkv; ++u) CHECK(seen[u] == line.groups(u / Hkv));
  CHECK(most <= line.cost() / n + 1 + PAGED_UNIT_COST);   // even in cost
  return 0;
}

int main() {
  const int grids[] = {1, 3, 152, 608, PAGED_MAX_PARTS};
  srand(7);
  for (int grid : grids)
    for (int Hkv : {1, 2, 7, 8}) {
      for (int len = 1; len < 40000; len = len * 7 / 4 + 1)
        if (check({len}, Hkv, grid) || check({0, len, 0, 0, 1, len / 3}, Hkv, grid)) return 1;
      if (check({0}, Hkv, grid) || check({0, 0, 0}, Hkv, grid)) return 1;
      for (int i = 0; i < 30; ++i) {
        std::vector<int> lens(1 + rand() % 300);
        for (int& n : lens) n = rand() % 4 ? rand() % (1 + rand() % 900) : 0;
        if (check(lens, Hkv, grid)) return 1;
      }
    }
  // the longest lines: 65535 units of PAGED_MAX_SLOTS slots; the largest batch
  for (int B : {1, PAGED_MAX_BATCH}) {
    const int Hkv = 65535 / B, g = PAGED_MAX_SLOTS / PAGED_GROUP;
    const std::vector<unsigned> w = words(std::vector<int>(B, PAGED_MAX_SLOTS - 1));
    const PagedLine line{w.data(), B, Hkv};
    CHECK(line.total() == B * Hkv * g && line.total() > 0 && line.tokens(B - 1) == PAGED_MAX_SLOTS - 1);
    const PagedCuts cuts = line.cuts(PAGED_MAX_PARTS);
    const int n = cuts.n;
    CHECK(n == PAGED_MAX_PARTS && line.part_begin(cuts, n) == line.total());
    for (int c = 0; c < n; ++c) {
      PagedSegments s;
      s.start(line, line.part_begin(cuts, c), line.part_begin(cuts, c + 1));
      CHECK(s.at() && line.part_of(cuts, s.b, s.h, s.x - s.unit_begin) == c);
    }
  }
  CHECK(paged_groups(0) == 0 && paged_groups(1) == 1 && paged_groups(16) == 1 && paged_groups(17) == 2);
  // rows: inside the pool for every page in it, -1 for every other entry
  for (int lp = 4; lp <= 8; ++lp)
    for (int page = -2; page < 9; ++page)
      for (int h = 0; h < 3; ++h)
        for (int slot = 0; slot < 1024; ++slot) {
          const long long r = paged_row(page, 7, 3, h, lp, slot);
          if (page < 0 || page >= 7) CHECK(r == -1);
          else CHECK(r == ((long long)page * 3 + h) * (1 << lp) + slot % (1 << lp) && r < (7ll * 3 << lp));
        }
  CHECK(paged_row((1 << 30), 1 << 20, 8, 0, 8, 0) == -1);
  CHECK(paged_row((1 << 20) - 1, 1 << 20, 7, 6, 8, 255) == (7ll << 28) - 1);
  puts("ok");
  return 0;
}
"""


def test_index_arithmetic(tmp_path):
    src = tmp_path / "index.cpp"
    src.write_text(INDEX_PROGRAM)
    exe = str(tmp_path / "index")
    inc = os.path.join(ROOT, "kv_cache_token_tip_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", inc, str(src), "-o", exe],
                   check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


# ------------------------------------------------------------------ oracle pins
def _pool(rng, B, Hkv, d, page, max_pages):
    n_pages = B * max_pages + 2
    table = rng.permutation(n_pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    return rng.standard_normal((n_pages, Hkv, page, d)), rng.standard_normal((n_pages, Hkv, page, d)), table


def test_oracle_attention_is_softmax_attention():
    import torch
    rng = np.random.default_rng(1)
    B, Hkv, G, d, page = 3, 2, 3, 64, 16
    kp, vp, table = _pool(rng, B, Hkv, d, page, 4)
    lens = [64, 17, 0]
    q, pos = rng.standard_normal((B, Hkv * G, d)), np.array([70, 5, 9])
    out, got, _, _ = PO.paged_attention(q, pos, kp, vp, table, lens, 1e4)
    for b, n in enumerate(lens):
        if n == 0:
            assert np.all(out[b] == 0) and np.all(got[b] == 0)
            continue
        z = (q[b].reshape(-1, d // 2, 2) @ [1, 1j]) * np.exp(1j * pos[b] * np.exp(-np.arange(0, d, 2) / d * np.log(1e4)))
        qr = np.stack([z.real, z.imag], -1).reshape(Hkv * G, d)
        K = kp[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n]
        V = vp[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n]
        t = [torch.from_numpy(np.ascontiguousarray(x)) for x in (qr[:, None], K.repeat(G, 0), V.repeat(G, 0))]
        ref = torch.nn.functional.scaled_dot_product_attention(*t)[:, 0].numpy()
        assert np.allclose(out[b], ref, rtol=1e-12, atol=1e-12)
        assert np.allclose(got[b].sum(-1), G, rtol=1e-12) and np.all(got[b, :, n:] == 0)


def test_oracle_append_then_attention_equals_a_cache_that_holds_the_token():
    rng = np.random.default_rng(2)
    kp, vp, table = _pool(rng, 2, 2, 64, 16, 3)
    lens, pos = np.array([16, 30]), np.array([16, 99])
    k_new, v_new = rng.standard_normal((3, 2, 64)), rng.standard_normal((3, 2, 64))
    w, tp = np.ones((2, 2, 48)), np.full((2, 2, 48), -1)
    PO.paged_append(k_new, v_new, [0, 2, 3], pos, table, lens, kp, vp, w, tp, 1e4)
    assert np.array_equal(vp[table[0, 1], :, 0], v_new[0]) and np.array_equal(vp[table[0, 1], :, 1], v_new[1])
    assert np.array_equal(vp[table[1, 1], :, 14], v_new[2])
    # a rotated key meets a query at its own position as if neither were rotated
    q = rng.standard_normal((2, 64))
    assert np.allclose((PO.rotate(q, 17, 1e4) * kp[table[0, 1], :, 1]).sum(-1), (q * k_new[1]).sum(-1))
    assert list(tp[0, 0, 15:19]) == [-1, 16, 17, -1] and list(w[1, 1, 29:32]) == [1, 0, 1] and tp[1, 0, 30] == 99


def test_oracle_eviction_by_hand_and_by_brute_force():
    import itertools
    stay = PO.evict_choice(np.array([5.0, 1, 4, 4, 0, 9]), np.arange(6), 5, 4, 1, 1)
    assert list(stay) == [0, 2, 5, 3] or list(stay) == [0, 2, 3, 5]
    # ties keep the lower slot, held tokens come before any weight, NaN last
    assert list(PO.evict_choice(np.array([1.0, 1, 1, 1]), np.arange(4), 3, 2, 0, 0)) == [0, 1]
    assert list(PO.evict_choice(np.array([0.0, np.inf, 2, 3]), np.array([9, 0, 2, 5]), 9, 2, 0, 1)) == [0, 1]
    assert list(PO.evict_choice(np.array([np.nan, -np.inf, 2]), np.arange(3), 2, 2, 0, 0)) == [1, 2]
    assert list(PO.evict_choice(np.array([-0.0, 0.0, -1]), np.arange(3), 2, 1, 0, 0)) == [0]
    rng = np.random.default_rng(3)
    for _ in range(20):
        w = rng.integers(0, 6, 8).astype(float)
        k = int(rng.integers(1, 8))
        best = max(itertools.combinations(range(8), k), key=lambda s: (sum(w[list(s)]), [-i for i in s]))
        assert list(PO.evict_choice(w, np.zeros(8, dtype=int) + 3, 7, k, 0, 0)) == list(best)


def test_oracle_eviction_keeps_every_kept_row_once():
    rng = np.random.default_rng(4)
    kp, vp, table = _pool(rng, 2, 2, 64, 16, 4)
    w, tp = rng.random((2, 2, 64)), np.tile(np.arange(64), (2, 2, 1))
    k0, w0 = kp.copy(), w.copy()
    lens = [64, 20]
    new = PO.paged_evict(w, tp, [63, 19], table, lens, 24, 2, 5, kp, vp, w, tp)
    assert list(new) == [24, 20]
    for h in range(2):
        assert len(set(tp[0, h, :24])) == 24 and set(tp[0, h, :24]) >= {0, 1, 59, 60, 61, 62, 63}
        for t in range(24):
            m = tp[0, h, t]
            assert w[0, h, t] == w0[0, h, m]
            assert np.array_equal(kp[table[0, t // 16], h, t % 16], k0[table[0, m // 16], h, m % 16])
        assert np.array_equal(w[1, h], w0[1, h])


def test_binding_without_a_gpu_raises():
    """The compiled marshalling turns every failure into an exception."""
    import torch
    from kv_cache_token_tip_gb300 import build, fasa_paged_append, fasa_paged_attention, fasa_paged_evict
    build.build()
    x = torch.zeros(8)
    with pytest.raises(TypeError):
        fasa_paged_append(x, x, x, x, x, x, x, dims=None)
    with pytest.raises(TypeError):
        fasa_paged_attention(x, x, x, x, x, x, x, workspace=x, dims=7)
    if torch.cuda.is_available():
        return
    d = _dims()
    with pytest.raises((RuntimeError, ValueError)):
        fasa_paged_append(x, x, x, x, x, x, x, dims=d)
    with pytest.raises((RuntimeError, ValueError)):
        fasa_paged_attention(x, x, x, x, x, x, x, workspace=x, dims=d)
    with pytest.raises((RuntimeError, ValueError)):
        fasa_paged_evict(x, x, x, x, x, x, x, 4, x, workspace=x, dims=d)


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("call", ["attention", "evict", "agreement", "compound"])
def test_own_workspace_belongs_to_the_stream_of_the_call(monkeypatch, call, handle):
    """A call's own workspace is allocated with the call's stream as the current
    one: memory that another stream freed may still be in use there."""
    import contextlib
    import types

    import torch
    from kv_cache_token_tip_gb300 import FasaDims, fasa
    now, asked = ["its own"], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s.cuda_stream if s is not None else now[-1])
        yield
        now.pop()

    def empty(size, dtype=None, device=None):
        asked.append((now[-1], dtype))
        return types.SimpleNamespace(numel=lambda: size, element_size=lambda: 1, size=size)

    calls = []

    class Anything:
        """The library and the compiled calls: each answers 0."""

        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *a: types.SimpleNamespace(cuda_stream=h))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream="its own"))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(fasa, "lib", Anything)
    monkeypatch.setattr(fasa, "_native", Anything())
    monkeypatch.setattr(fasa, "_ptr", lambda *a: 0)
    x = types.SimpleNamespace(device="cuda")
    d, dp = FasaDims(), _dims()

    def run(**kw):
        if call == "attention":
            fasa.fasa_paged_attention(x, x, x, x, x, x, x, dims=dp, **kw)
        elif call == "evict":
            fasa.fasa_paged_evict(x, x, x, x, x, x, x, 4, x, dims=dp, **kw)
        elif call == "agreement":
            fasa.fasa_fc_agreement(x, x, x, 4, x, d, **kw)
        else:
            fasa.fasa_compound_agreement(x, x, x, x, 4, x, d, **kw)

    run(stream=77 if handle else types.SimpleNamespace(cuda_stream=77))
    run()
    run(stream=0 if handle else types.SimpleNamespace(cuda_stream=0))
    assert asked == [(77, torch.uint8), ("its own", torch.uint8), (0, torch.uint8)]
    assert len(calls) == 6   # a size and a call, three times


CUTS_PROGRAM = r"""
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "fasa_paged_index.h"
using namespace fasa;

static float steps(float x, int n) {
  for (; n > 0; --n) x = std::nextafter(x, 2e9f);
  for (; n < 0; ++n) x = std::nextafter(x, 0.f);
  return x;
}

// begin(c) is floor(cost * c / n) for every count of parts and part, with an inverse that
// is `off` steps from the nearest fp32.
static int exact(int off) {
  for (int n = 1; n <= PAGED_MAX_PARTS; ++n) {
    PagedCuts cuts(n, n);
    cuts.inv = steps(cuts.inv, off);
    for (int r = n - 1; r >= 0; r -= n < 200 ? 1 : 1 + rand() % 13)  // the largest products first
      for (int c = 0; c <= n; ++c) {
        cuts.r = r;
        if (cuts.begin(c) != c + (int)((long long)r * c / n)) return printf("begin: %d parts, %d, %d\n", n, r, c), 1;
      }
  }
  return 0;
}

// part_of finds every group's part with the quotients as far off.
static int inverse(int off) {
  for (int i = 0; i < 60; ++i) {
    const int B = 1 + rand() % 200, Hkv = 1 + rand() % 8, long_one = rand() % B;
    std::vector<unsigned> w;
    int before = 0;
    for (int b = 0; b <= B; ++b) {
      const int len = b == B ? 0 : b == long_one ? rand() % PAGED_MAX_SLOTS : rand() % 500;
      w.push_back(paged_word(before, len));
      before += paged_groups(len);
    }
    const PagedLine line{w.data(), B, Hkv};
    PagedCuts cuts = line.cuts(i % 2 ? PAGED_MAX_PARTS : 1 + rand() % PAGED_MAX_PARTS);
    cuts.inv = steps(cuts.inv, off);
    cuts.part = steps(cuts.part, i % 3 ? off : -off);
    for (int c = 0; c < cuts.n; ++c) {
      const int r0 = line.part_begin(cuts, c), r1 = line.part_begin(cuts, c + 1);
      PagedSegments s;
      s.start(line, r0, r1);
      for (; s.at(); s.next())
        for (int x : std::vector<int>{s.x, s.x + (s.seg_end() - s.x) / 2, s.seg_end() - 1})
          if (line.part_of(cuts, s.b, s.h, x - s.unit_begin) != c) return printf("part of %d\n", x), 1;
    }
  }
  return 0;
}

int main() {
  srand(5);
  for (int off = -2; off <= 2; ++off)
    if (exact(off) || inverse(off)) return printf("%d steps off\n", off), 1;
  puts("ok");
  return 0;
}
"""


def test_cuts_are_exact_with_the_devices_quotients(tmp_path):
    """The device's quotients may be two steps from a / b: the cuts in fp32 are the integer
    ones all the same, and a group's part is found."""
    src = tmp_path / "cuts.cpp"
    src.write_text(CUTS_PROGRAM)
    exe = str(tmp_path / "cuts")
    inc = os.path.join(ROOT, "kv_cache_token_tip_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-I", inc, str(src), "-o", exe], check=True,
                   capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_c_library_builds_without_torch(monkeypatch):
    """The C library needs nvcc alone: without torch only the binding's module is left out."""
    import importlib.util
    from kv_cache_token_tip_gb300 import build
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    for force in (False, True):
        assert build._build_torch(force=force) is None
    assert build.build()[0] == build.LIBFASA


def test_binding_module_is_rebuilt_for_another_torch(monkeypatch, tmp_path):
    """Its file carries the Python ABI's tag, and it is built anew for another torch, whatever the dates."""
    import importlib.util
    import sysconfig
    import types
    from kv_cache_token_tip_gb300 import build
    assert build.LIBTORCH.endswith("_fasa_torch" + sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIBTORCH", str(tmp_path / "module.so"))
    torch = {"at": "a", "version": "__version__ = '1'"}
    runs = []

    def find(name, *a):
        d = tmp_path / torch["at"]
        d.mkdir(exist_ok=True)
        (d / "version.py").write_text(torch["version"])
        os.utime(d / "version.py", (1, 1))   # older than every build
        return types.SimpleNamespace(origin=str(d / "__init__.py"))

    def run(cmd, verbose):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")

    monkeypatch.setattr(importlib.util, "find_spec", find)
    monkeypatch.setattr(build, "_run", run)
    built = []
    for change in ({}, {}, {"version": "__version__ = '2'"}, {}, {"at": "b"}, {}):
        torch.update(change)
        assert build._build_torch() == build.LIBTORCH
        built.append(len(runs))
    assert built == [1, 1, 2, 2, 3, 3]


def test_binding_refuses_a_module_of_another_torch(monkeypatch):
    import sys
    import types
    import kv_cache_token_tip_gb300 as pkg
    from kv_cache_token_tip_gb300 import build, fasa
    build.build()
    bound = []
    for version, fits in (("0.1.2", False), (None, False)):
        m = types.SimpleNamespace(bind=lambda *a: bound.append(a))
        if version:
            m.torch_version = version
        monkeypatch.setitem(sys.modules, pkg.__name__ + "._fasa_torch", m)
        monkeypatch.setattr(pkg, "_fasa_torch", m, raising=False)
        monkeypatch.setattr(fasa, "_native", None)
        with pytest.raises(RuntimeError, match="build it"):
            fasa._marshal()
    assert not bound


def test_new_lens_apart_from_what_other_heads_still_read(L):
    """new_lens is written while heads of other blocks read the positions and the pages."""
    d, far = _dims(), 16 * P

    def evict(new, **kw):   # right but for new_lens, until the workspace that is missing (3)
        t = dict(pos=far, table=far, lens=far, w=far, tp=far + 8 * P, wo=far, tpo=far + 8 * P, ws=None, new=new)
        t.update(kw)
        return _evict(L, d, **t)

    for at in (P, P + 4, P - 4):   # pos [2]: itself, overlapping from either side
        assert evict(at, pos=P) == 1
    table = 2 * 32 * 4             # page_table [2, 32]
    for at in (P, P + 64, P + table - 4, P - 4):
        assert evict(at, table=P) == 1
    assert evict(P + 8, pos=P) == 3 and evict(P - 8, pos=P) == 3
    assert evict(P + table, table=P) == 3 and evict(P - 8, table=P) == 3
