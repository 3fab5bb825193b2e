"""A step of new tokens over the paged cache without a GPU: calls without rows, what
may not overlap, how the workspace grows, and the split of the chunks' work as the
kernels make it."""

import ctypes
import os
import subprocess

import pytest

from tests.test_serve_host import A, L, _chunk, _dims, _rope  # noqa: F401 (L: the fixture)


def test_calls_without_rows(L):
    """Tensors without rows have no addresses: such calls do nothing."""
    from kv_cache_token_tip_gb300 import FasaRope
    d, r = _dims(), FasaRope()
    assert _rope(L, d, r, n=0, q=None, k=None, v=None, qo=None, m=None) == 0
    assert _rope(L, d, r, n=0, q=None, k=None, v=None, qo=None, m=None, w=None, tp=None) == 0
    assert _rope(L, d, r, n=0, q=None, qo=None, k=None, v=None, kp=None, vp=None, m=None) == 0
    assert _rope(L, d, r, n=0, k=None, v=None) == 0 and _rope(L, d, r, n=0, q=None) == 0
    assert _chunk(L, d, q=None, out=None, n=0, ws=None, size=0) == 0
    # the dims and the rotation are looked at all the same
    assert _rope(L, _dims(batch=0), r, n=0) == 1 and _rope(L, d, FasaRope(rotary_dim=24), n=0) == 1
    assert _rope(L, d, r, n=5, q=None) == 1 and _rope(L, d, r, n=5, k=None, v=None) == 1


def _size(L, d, n_tokens, weights):
    n = ctypes.c_size_t(0)
    assert L.fasa_paged_chunk_workspace_size(ctypes.byref(d), n_tokens, weights, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("weights", [0, 1])
@pytest.mark.parametrize("kw", [dict(), dict(dtype=0, head_dim=64), dict(n_q_heads=56), dict(n_q_heads=8),
                                dict(n_q_heads=128, n_kv_heads=64, head_dim=64)])
def test_a_workspace_serves_every_smaller_call(L, kw, weights):
    """The size does not fall as the batch, the table or the tokens grow."""
    batches, tables, tokens = (1, 2, 50, 100, 200, 700, 1000), (1, 31, 100, 512, 2000, 16384), (1, 4, 50, 200, 1024, 100000)
    size = {(b, t, n): _size(L, _dims(batch=b, max_pages=t, **kw), n, weights) for b in batches for t in tables for n in tokens}
    for axis, values in enumerate((batches, tables, tokens)):
        for at, s in size.items():
            i = values.index(at[axis])
            if i + 1 < len(values):
                more = list(at)
                more[axis] = values[i + 1]
                assert s <= size[tuple(more)], (at, more)


def test_workspace_has_room_for_the_rows_that_there_are(L):
    """Kept logits: by the new tokens' rows where they are few (a decode step), by 16 rows a sequence where not, half a
    GB at most."""
    for batch, n, rows in ((32, 32, 32 * 4), (32, 64, 64 * 4), (32, 100, 400), (32, 5000, 32 * 16), (1, 1, 4)):
        d = _dims(batch=batch, max_pages=512)  # 8192 slots
        log_sums = -(-n * 32 * 4 // 256) * 256
        assert _size(L, d, n, 1) - _size(L, d, n, 0) == rows * 8 * 8192 * 4 + log_sums
    d = _dims(batch=2000, max_pages=16384)
    assert _size(L, d, 2000, 1) - _size(L, d, 2000, 0) == (480 << 20) + 2000 * 32 * 4


def test_chunk_overlaps_rejected(L):
    """What the call writes lies apart from what it reads and from itself: the smallest overlap, at either end."""
    from tests.test_serve_host import P
    d = _dims()  # of 2 sequences, 32 pages each of a pool of 100, 8 of 32 heads of 128 dims, bf16
    io, pool, stat = 5 * 32 * 128 * 2, 100 * 8 * 16 * 128 * 2, 2 * 8 * 512 * 4
    at = [x + (1 << 30) for x in A]
    read = dict(q=(at[0], io), cu=(at[1], 12), kp=(at[2], pool), vp=(at[3], pool), table=(at[4], 2 * 32 * 4), lens=(at[5], 8))
    written = dict(out=(at[6], io), w=(at[7], stat), ws=(at[8], _size(L, d, 5, 1)))
    every = {name: x for name, (x, _) in (read | written).items()}
    for name, (_, size) in written.items():
        for other, (x, n) in list(read.items()) + [y for y in written.items() if y[0] != name]:
            for to in (x, x + (n - 1) // 16 * 16, x - (size - 1) // 16 * 16):
                assert _chunk(L, d, **{**every, name: to}) == 1, (name, other, to - x)
    for name in ("cu", "table", "lens"):
        assert _chunk(L, d, **{name: P + (3 << 29) + 2}) == 1


def test_rope_overlaps_rejected(L):
    from kv_cache_token_tip_gb300 import FasaRope
    d, r = _dims(), FasaRope()
    q, kv, pool, stat = 5 * 32 * 128 * 2, 5 * 8 * 128 * 2, 100 * 8 * 16 * 128 * 2, 2 * 8 * 512 * 4
    at = [x + (1 << 30) for x in A]
    read = dict(q=(at[0], q), k=(at[1], kv), v=(at[2], kv), m=(at[3], 5 * 16))
    written = dict(qo=(at[4], q), kp=(at[5], pool), vp=(at[6], pool), w=(at[7], stat), tp=(at[8], stat))
    every = {name: x for name, (x, _) in (read | written).items()}
    for name, (_, size) in written.items():
        for other, (x, n) in list(read.items()) + [y for y in written.items() if y[0] != name]:
            for to in (x, x + (n - 1) // 16 * 16, x - (size - 1) // 16 * 16):
                if (name, other, to) != ("qo", "q", x):  # (in place)
                    assert _rope(L, d, r, **{**every, name: to}) == 1, (name, other, to - x)
    # rows of one projection's output: what lies between them counts as theirs
    parts = dict(q=at[0], qs=48 * 128, k=at[0] + 32 * 256, ks=48 * 128, v=at[0] + 40 * 256, vs=48 * 128)
    for name in ("qo", "kp", "w", "tp"):
        assert _rope(L, d, r, **{**every, **parts, name: at[0] + 3 * 48 * 256}) == 1


KERNELS_LINE = r"""
// The kernels' own units, tiles and costs: those of either type, with every number of heads to a group.
int main() {
  srand(2);
  for (int k = 0; k < 1600; ++k) {
    const bool bf16 = k & 1;
    const int G = 1 + k / 2 % 8, Hkv = 1 + rand() % 8, B = 1 + rand() % (k % 10 ? 6 : 60);
    const ChunkShape s = chunk_shape(bf16, G);
    CHECK(s.tokens == (bf16 ? 2 * (128 / G) : 128 / G) && s.tile == (bf16 ? 128 : 64) && s.unit == (bf16 ? 512 : 48));
    std::vector<int> n, len;
    const int long_n = 1 + rand() % (k % 7 ? 300 : 3000), long_a = rand() % (k % 5 ? 400 : 20000);
    for (int b = 0; b < B; ++b) {
      n.push_back(rand() % 4 ? rand() % (long_n + 1) : rand() % 2);
      len.push_back(n[b] + rand() % (long_a + 1));
      if (rand() % 9 == 0) len[b] = rand() % (n[b] + 1);
    }
    if (check(n, len, Hkv, s.tokens, s.tile, s.unit, k % 3 ? 152 : 1 + rand() % 160)) return printf("case %d\n", k), 1;
  }
  for (int G = 1; G <= 8; ++G)
    for (int bf16 = 0; bf16 < 2; ++bf16) {
      const ChunkShape s = chunk_shape(bf16, G);
      const int T = s.tokens;
      // a token a sequence; lengths about the tiles'; more new tokens than cached ones; nothing cached
      if (check(std::vector<int>(2048, 1), std::vector<int>(2048, 1 + 77 * G), 2, T, s.tile, s.unit, 152)) return 1;
      for (int d = -1; d <= 1; ++d)
        if (check({T + d, 2 * T + d, 1}, {s.tile + d, 3 * s.tile + T + d, 5 * s.tile + d}, 3, T, s.tile, s.unit, 152)) return 1;
      if (check({100, 1, 7}, {0, 0, 3}, 2, T, s.tile, s.unit, 152)) return 1;
      // the largest: positions past 32 bits
      if (check({1 << 20}, {262144}, 2, T, s.tile, s.unit, 152) || check({1 << 18, 1 << 18}, {262144, 262144}, 3, T, s.tile, s.unit, 152)) return 1;
    }
  printf("ok\n");
}
"""


def test_index_arithmetic_of_the_kernels(tmp_path):
    from tests.test_serve_host import INDEX_PROGRAM, ROOT
    src = tmp_path / "line.cpp"
    src.write_text(INDEX_PROGRAM[:INDEX_PROGRAM.index("int main()")] + KERNELS_LINE)
    exe = str(tmp_path / "line")
    inc = os.path.join(ROOT, "kv_cache_token_tip_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", inc, str(src), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_chunk_binding_without_a_workspace_names_what_is_wrong(L):
    import torch
    from kv_cache_token_tip_gb300 import fasa_paged_chunk_attention
    x = torch.zeros(8)
    for dims in (None, 3):
        with pytest.raises(TypeError):
            fasa_paged_chunk_attention(x, x, x, x, x, x, dims=dims)
