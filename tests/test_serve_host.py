"""A step of new tokens over the paged cache without a GPU: what the entry points
refuse, the split of the chunks' work, and the oracle."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that is never read


@pytest.fixture(scope="module")
def L():
    from kv_cache_token_tip_gb300 import build, lib
    build.build()
    return lib()


def _dims(**kw):
    from kv_cache_token_tip_gb300 import FasaPagedDims
    d = dict(batch=2, n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=16, n_pages=100, max_pages=32, dtype=1,
             rope_theta=1e4)
    d.update(kw)
    return FasaPagedDims(*d.values())


# addresses far enough apart for every tensor of these dims
A = [P + (i << 28) for i in range(16)]


def _assign(L, d, have=A[0], want=A[1], pos=A[2], table=A[3], free=A[4], count=A[5], lens=A[6], left=A[7], cu=A[8], m=A[9],
            n=50):
    return L.fasa_paged_assign(have, want, pos, table, free, count, lens, left, cu, m, n, d and ctypes.byref(d), None)


def _rope(L, d, r, q=A[0], qs=32 * 128, k=A[1], ks=8 * 128, v=A[2], vs=8 * 128, m=A[3], n=5, qo=A[4], kp=A[5], vp=A[6],
          w=A[7], tp=A[8]):
    return L.fasa_paged_rope_append(q, qs, k, ks, v, vs, m, n, qo, kp, vp, w, tp, r and ctypes.byref(r),
                                    d and ctypes.byref(d), None)


def _chunk(L, d, q=A[0], n=5, cu=A[1], kp=A[2], vp=A[3], table=A[4], lens=A[5], out=A[6], w=A[7], ws=A[8], size=1 << 40):
    return L.fasa_paged_chunk_attention(q, n, cu, kp, vp, table, lens, out, w, ws, size, d and ctypes.byref(d), None)


BAD_DIMS = [
    (dict(batch=0), 1), (dict(n_q_heads=30), 1), (dict(max_pages=0), 1), (dict(rope_theta=0.0), 1), (dict(dtype=7), 2),
    (dict(head_dim=96), 2), (dict(n_q_heads=72), 2), (dict(page_size=8), 2), (dict(page_size=512), 2),
    (dict(batch=2049), 2), (dict(max_pages=16385), 2), (dict(n_pages=1 << 24), 2),
]


@pytest.mark.parametrize("kw,code", BAD_DIMS)
def test_bad_dims_rejected(L, kw, code):
    from kv_cache_token_tip_gb300 import FasaRope
    d, n = _dims(**kw), ctypes.c_size_t(7)
    assert _assign(L, d) == code and _rope(L, d, FasaRope()) == code and _chunk(L, d) == code
    assert L.fasa_paged_chunk_workspace_size(ctypes.byref(d), 5, 1, ctypes.byref(n)) == code and n.value == 0


def test_assign_arguments_rejected(L):
    d = _dims()
    assert _assign(L, None) == 1
    for name in ("have", "want", "table", "free", "count", "lens", "left", "cu", "m"):
        assert _assign(L, d, **{name: None}) == 1
        assert _assign(L, d, **{name: P + 3 * (1 << 29) + 2}) == 1
    assert _assign(L, d, m=A[9] + 8) == 1 and _assign(L, d, n=-1) == 1 and _assign(L, d, n=(1 << 24) + 1) == 2
    # what is written lies apart from everything, but for the lengths and the count in place
    for name in ("table", "free", "cu", "m"):
        for other in (0, 1, 2, 5, 6, 7):
            assert _assign(L, d, **{name: A[other]}) == 1, (name, other)
    assert _assign(L, d, table=A[4]) == 1 and _assign(L, d, cu=A[9] + 16) == 1 and _assign(L, d, free=A[3] + 128) == 1
    assert _assign(L, d, lens=A[0] + 4) == 1 and _assign(L, d, lens=A[1] - 4) == 1
    assert _assign(L, d, lens=A[2]) == 1 and _assign(L, d, lens=A[5]) == 1 and _assign(L, d, left=A[0]) == 1
    assert _assign(L, d, left=A[6]) == 1


def test_rope_arguments_rejected(L):
    from kv_cache_token_tip_gb300 import FasaRope
    d = _dims()
    nan, inf = float("nan"), float("inf")
    assert _rope(L, None, FasaRope()) == 1 and _rope(L, d, None) == 1
    for kw, code in ((dict(layout=2), 2), (dict(layout=-1), 2), (dict(scaling=4), 2), (dict(scaling=-1), 2),
                     (dict(rotary_dim=0), 1), (dict(rotary_dim=24), 1), (dict(rotary_dim=144), 1),
                     (dict(rope_theta=0.0), 1), (dict(rope_theta=inf), 1), (dict(magnitude=0.0), 1),
                     (dict(magnitude=nan), 1), (dict(magnitude=1e300), 1), (dict(magnitude=1e-300), 1),
                     (dict(scaling=1, factor=0.0), 1),
                     (dict(scaling=1, factor=nan), 1), (dict(scaling=2, low=0.0), 1), (dict(scaling=2, low=4.0), 1),
                     (dict(scaling=2, high=inf), 1), (dict(scaling=2, original=0.0), 1),
                     (dict(scaling=3, rope_theta=1.0), 1), (dict(scaling=3, low=nan), 1)):
        assert _rope(L, d, FasaRope(**kw)) == code, kw
    bad = FasaRope()
    bad.reserved = 1
    assert _rope(L, d, bad) == 1
    r = FasaRope()
    for name in ("q", "k", "v", "m", "qo", "kp", "vp"):
        assert _rope(L, d, r, **{name: None}) == 1
    for name in ("q", "k", "v", "m", "qo", "kp", "vp", "w", "tp"):
        assert _rope(L, d, r, **{name: A[12] + 8}) == 1
    for name in ("qs", "ks", "vs"):  # tokens that overlap, or begin off a 16-byte word
        assert _rope(L, d, r, **{name: 8 * 128 - 8}) == 1 and _rope(L, d, r, **{name: 48 * 128 + 4}) == 1
        assert _rope(L, d, r, **{name: -32 * 128}) == 1 and _rope(L, d, r, **{name: (1 << 32) + 8}) == 1
    assert _rope(L, d, r, n=-1) == 1 and _rope(L, d, r, n=(1 << 24) + 1) == 2
    assert _rope(L, d, r, k=None, v=None, kp=None, vp=None) == 1    # statistics of no keys
    assert _rope(L, d, r, qo=A[0] + 16) == 1 and _rope(L, d, r, qo=A[0], qs=48 * 128) == 1
    assert _rope(L, d, r, qo=A[1]) == 1 and _rope(L, d, r, qo=A[2] - 256) == 1 and _rope(L, d, r, qo=A[3]) == 1
    assert _rope(L, d, r, n=0) == 0 and _rope(L, d, r, None, 0, None, 0, None, 0, A[3], 5, None, None, None, None, None) == 0


def test_chunk_arguments_rejected(L):
    d = _dims()
    assert _chunk(L, None) == 1
    for name in ("q", "kp", "vp", "table", "lens", "out"):
        assert _chunk(L, d, **{name: None}) == 1
    for name in ("q", "kp", "vp", "out", "w"):
        assert _chunk(L, d, **{name: A[12] + 8}) == 1
    assert _chunk(L, d, cu=None) == 1 and _chunk(L, d, n=-1) == 1 and _chunk(L, d, n=(1 << 20) + 1) == 2
    assert _chunk(L, d, out=A[0]) == 1 and _chunk(L, d, out=A[0] + 32 * 128 * 2) == 1
    assert _chunk(L, d, ws=None) == 3 and _chunk(L, d, ws=A[8] + 8) == 3 and _chunk(L, d, size=0) == 3
    assert _chunk(L, d, n=0) == 0
    n, size = ctypes.c_size_t(0), L.fasa_paged_chunk_workspace_size
    assert size(ctypes.byref(d), 5, 0, None) == 1 and size(ctypes.byref(d), -1, 0, ctypes.byref(n)) == 1
    assert size(ctypes.byref(d), (1 << 20) + 1, 0, ctypes.byref(n)) == 2
    assert size(ctypes.byref(d), 0, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert size(ctypes.byref(d), 500, 0, ctypes.byref(n)) == 0 and n.value > 0
    plain = n.value
    assert _chunk(L, d, n=500, w=None, size=plain - 1) == 3
    assert size(ctypes.byref(d), 500, 1, ctypes.byref(n)) == 0
    assert n.value >= plain + 500 * 32 * 4 and _chunk(L, d, n=500, size=n.value - 1) == 3


def test_workspace_is_no_larger_for_fewer_tokens(L):
    n, size = ctypes.c_size_t(0), L.fasa_paged_chunk_workspace_size
    for kw in (dict(), dict(dtype=0, head_dim=64), dict(n_q_heads=56), dict(n_q_heads=8)):
        d, last = _dims(**kw), 0
        for t in (1, 2, 3, 7, 20, 100, 101, 1000, 5000, 1 << 20):
            assert size(ctypes.byref(d), t, 1, ctypes.byref(n)) == 0
            assert n.value >= last and n.value % 16 == 0
            last = n.value


INDEX_PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>
#include "fasa_chunk_index.h"
using namespace fasa;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

// The parts hold every tile of every unit once and in order, a unit without tiles has one
// part that it begins in, and the place of a cut is found again from the cut alone.
static int check(const std::vector<int>& n, const std::vector<int>& len, int Hkv, int T, int KT, int unit, int most) {
  const int B = (int)n.size();
  std::vector<long long> costs(B + 1);
  std::vector<int> cu(B + 1);
  for (int b = 0; b < B; ++b) cu[b + 1] = cu[b] + n[b];
  const ChunkLine line{costs.data(), cu.data(), len.data(), cu[B], 1 << 18, B, Hkv, T, KT, unit};
  long long before = 0;
  for (int b = 0; b < B; ++b) {
    costs[b] = before;
    before += line.cost_of(n[b], len[b]);
  }
  costs[B] = before;
  const int parts = line.parts(most);
  if (before == 0) { CHECK(parts == 0); return 0; }
  CHECK(parts >= 1 && parts <= most && line.part_begin(parts, 0) == 0 && line.part_begin(parts, parts) == line.total());
  std::map<std::tuple<int, int, int>, int> done, begun;
  for (int c = 0; c < parts; ++c) {
    const long long y0 = line.part_begin(parts, c), y1 = line.part_begin(parts, c + 1);
    CHECK(y0 < y1);
    ChunkUnit u;
    for (u.find(line, y0);;) {
      CHECK(u.b >= 0 && u.b < B && u.h >= 0 && u.h < Hkv && u.i >= 0 && u.i < ChunkLine::tiles_of(n[u.b], T));
      CHECK(u.begin < y1 && u.begin + u.cost > y0 && u.q.n == n[u.b] && u.q.len == len[u.b] && u.q.first == cu[u.b]);
      const int last = (u.i + 1) * T < n[u.b] ? (u.i + 1) * T : n[u.b], see = len[u.b] - n[u.b] + last;
      CHECK(u.tiles == (see > 0 ? (see + KT - 1) / KT : 0));
      const int f0 = u.before(line, y0), f1 = u.before(line, y1);
      CHECK(0 <= f0 && f0 <= f1 && f1 <= u.tiles);
      auto key = std::make_tuple(u.b, u.h, u.i);
      CHECK(done[key] == f0);
      done[key] = f1;
      if (u.begin >= y0) ++begun[key];
      if (u.begin >= y0) CHECK(f0 == 0);
      else CHECK(f0 > 0 || u.tiles == 0);
      ChunkUnit v;  // the same unit from any place of it
      v.find(line, u.begin);
      CHECK(v.b == u.b && v.h == u.h && v.i == u.i && v.begin == u.begin && v.cost == u.cost);
      v.find(line, u.begin + u.cost - 1);
      CHECK(v.b == u.b && v.h == u.h && v.i == u.i && v.begin == u.begin);
      if (u.begin + u.cost >= y1) break;
      u.next(line);
    }
  }
  long long units = 0;
  for (int b = 0; b < B; ++b)
    for (int h = 0; h < Hkv; ++h)
      for (int i = 0; i < ChunkLine::tiles_of(n[b], T); ++i) {
        const int last = (i + 1) * T < n[b] ? (i + 1) * T : n[b], see = len[b] - n[b] + last;
        CHECK(done[std::make_tuple(b, h, i)] == (see > 0 ? (see + KT - 1) / KT : 0));
        CHECK(begun[std::make_tuple(b, h, i)] == 1);
        ++units;
      }
  CHECK((long long)begun.size() == units);
  return 0;
}

int main() {
  srand(1);
  for (int k = 0; k < 1500; ++k) {
    const int B = 1 + rand() % (k % 10 ? 6 : 60), G = 1 + rand() % 8;
    const int rows = rand() % 2 ? 256 : 64, T = rows / G, KT = rand() % 2 ? 128 : 64;
    std::vector<int> n, len;
    const int long_n = 1 + rand() % (k % 7 ? 300 : 3000), long_a = rand() % (k % 5 ? 400 : 20000);
    for (int b = 0; b < B; ++b) {
      n.push_back(rand() % 4 ? rand() % (long_n + 1) : rand() % 2);
      len.push_back(n[b] + rand() % (long_a + 1));
      if (rand() % 9 == 0) len[b] = rand() % (n[b] + 1);  // more new tokens than cached ones
    }
    if (check(n, len, 1 + rand() % 8, T, KT, rand() % 4 * 64, 1 + rand() % 320)) return printf("case %d\n", k), 1;
  }
  // the largest: positions past 32 bits
  if (check({1 << 20}, {262144}, 2, 32, 128, 128, 152) || check({1 << 18, 1 << 18}, {262144, 262144}, 3, 256, 128, 16, 152)) return 1;
  printf("ok\n");
}
"""


def test_index_arithmetic(tmp_path):
    src = tmp_path / "index.cpp"
    src.write_text(INDEX_PROGRAM)
    exe = str(tmp_path / "index")
    inc = os.path.join(ROOT, "kv_cache_token_tip_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", inc, str(src), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


# ------------------------------------------------------------------ the oracle
def test_oracle_assign_by_hand():
    from oracle import serve_oracle as SO
    table = np.array([[3, 4], [5, -1], [-1, -1]], dtype=np.int32)
    free = np.array([7, 8, 0, 0, 0, 0, 0, 0, 0], dtype=np.int32)
    # the first gives page 4 back, the second takes it, the third takes 8
    lens, cu, rows, count = SO.assign([20, 15, 0], [16, 18, 2], [0, 40, 9], table, free, 2, 6, 16)
    assert (lens, cu, count) == ([16, 18, 2], [0, 0, 3, 5], 1)
    assert table.tolist() == [[3, 4], [5, 4], [8, -1]] and free[:3].tolist() == [7, 8, 4]
    assert rows == [(1, 15, 5, 40), (1, 16, 4, 41), (1, 17, 4, 42), (2, 0, 8, 9), (2, 1, 8, 10), (-1, -1, -1, -1)]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
def test_oracle_turns_depend_on_distance_alone(layout, scaling):
    """<R(m) q, R(n) k> goes by m - n, and a turn keeps a pair's norm but for the magnitude."""
    from kv_cache_token_tip_gb300 import FasaRope
    from oracle import serve_oracle as SO
    rope = FasaRope(layout, 48, scaling, 1e4, factor=4.0, low=1.0, high=16.0, original=512.0, magnitude=1.25)
    rng = np.random.default_rng(scaling)
    q, k = rng.standard_normal((2, 3, 64))
    dots = [np.sum(SO.turn(q, m + 7, rope) * SO.turn(k, m, rope), axis=1) for m in (0, 5, 1000)]
    assert np.allclose(dots[0], dots[1]) and np.allclose(dots[0], dots[2])
    y = SO.turn(q, 33, rope)
    assert np.array_equal(y[:, 48:], q[:, 48:])
    assert np.allclose(np.linalg.norm(y[:, :48]), 1.25 * np.linalg.norm(q[:, :48]))
    f = SO.frequencies(rope)
    t = 1e4 ** (-2.0 * np.arange(24) / 48)
    if scaling >= 2:  # the fastest stay, the slowest are stretched by the whole factor
        assert np.isclose(f[0], t[0]) and np.isclose(f[-1], t[-1] / 4.0) and np.all(np.diff(f) < 0)


def test_oracle_plain_turn_is_the_one_of_the_decode_step():
    from kv_cache_token_tip_gb300 import FasaRope
    from oracle import paged_oracle as PO, serve_oracle as SO
    x = np.random.default_rng(3).standard_normal((4, 128))
    assert np.allclose(SO.turn(x, 777, FasaRope(0, 128, 0, 5e5)), PO.rotate(x, 777, 5e5))


def test_oracle_chunk_is_single_tokens_one_after_the_other():
    from oracle import paged_oracle as PO, serve_oracle as SO
    rng = np.random.default_rng(4)
    B, Hkv, G, d, page = 2, 2, 3, 8, 4
    kp, vp = rng.standard_normal((2, 9, Hkv, page, d))
    table = rng.permutation(9)[:8].reshape(B, 4)
    lens, n = [13, 6], [5, 2]
    q = rng.standard_normal((7, Hkv * G, d))
    out, got, _, _ = SO.chunk_attention(q, [0, 5, 7], kp, vp, table, lens)
    want_w = np.zeros_like(got)
    for b in range(B):
        for j in range(n[b]):
            at = [0, 0]
            at[b] = lens[b] - n[b] + j + 1
            one = np.zeros((B, Hkv * G, d))
            one[b] = q[5 * b + j]
            o, w, _, _ = PO.paged_attention(one, [0, 0], kp, vp, table, at, 1e4)
            assert np.allclose(o[b], out[5 * b + j])
            want_w[b] += w[b]
    assert np.allclose(want_w, got)


def test_binding_without_a_gpu_raises():
    import torch
    from kv_cache_token_tip_gb300 import (FasaRope, build, fasa_paged_assign, fasa_paged_chunk_attention,
                                          fasa_paged_rope_append)
    build.build()
    x, d = torch.zeros(8), _dims()
    with pytest.raises(TypeError):
        fasa_paged_assign(x, x, x, x, x, x, x, x, dims=None)
    with pytest.raises(TypeError):
        fasa_paged_rope_append(x, x, x, x, x, x, x, rope=None, dims=d)
    with pytest.raises(TypeError):
        fasa_paged_rope_append(x, x, x, x, x, x, x, rope=FasaRope(), dims=3)
    with pytest.raises(TypeError):
        fasa_paged_chunk_attention(x, x, x, x, x, x, workspace=x, dims=3)
    if torch.cuda.is_available():
        return
    with pytest.raises((RuntimeError, ValueError)):
        fasa_paged_assign(x, x, x, x, x, x, x, x, dims=d)
    with pytest.raises((RuntimeError, ValueError)):
        fasa_paged_rope_append(x, x, x, x, x, x, x, rope=FasaRope(), dims=d)
    with pytest.raises((RuntimeError, ValueError)):
        fasa_paged_chunk_attention(x, x, x, x, x, x, workspace=x, dims=d)


def test_summary_of_the_captures_names_its_sources():
    import re
    import warnings

    import bench
    text = open(os.path.join(ROOT, "profiles", "fasa_serve.md")).read()
    names = re.search(r"kernel_sources: `([^`]*)`", text).group(1).split()
    told = re.search(r"kernel_source_hash: `([0-9a-f]{16})`", text).group(1)
    csrc = "kv_cache_token_tip_gb300/csrc"
    assert {"fasa_chunk.cuh", "fasa_chunk_bf16.cu", "fasa_chunk_f32.cu", "fasa_serve_tokens.cu"} <= set(names)
    assert all(os.path.exists(os.path.join(ROOT, csrc, f)) for f in names)
    if bench.kernel_source_hash([os.path.join(csrc, f) for f in names]) != told:
        warnings.warn("profiles/fasa_serve.md was taken on other sources")
