"""What the paged attention's three bf16 terms are for: inputs whose softmax
weights, or whose rotated queries, need the third one.

Every sequence has two tokens, and every head one nonzero pair at position 0, so
that nothing but the roundings below is left: the logits (in powers of two) are 0
and z = y k, y = q log2(e) / sqrt(d); the values 0 and plus or minus a power of two
V; out = V w / (1 + w), w = 2^z.  Tolerances (u = 2^-24, the half step of fp32;
derived, not fitted):
  * z: the constant log2(e) / sqrt(d) and the product y round once each, y's three
    bf16 terms leave 2^-27 (three roundings to nearest of 2^-9), a term's product
    with k is exact in 32 bits, and two sums follow: 4.2 u |z|, in w ln 2 times that,
    2.92 |z| u;
  * w: exp2f 2 ulp, 4 u;
  * o: three terms (0.2 u), joined by at most two sums of the tensor cores, which may
    round towards zero (2 u each), 4.2 u;
  * l = 1 + w, its inverse and the product, 3 u.
  Together less than (3 |z| + 12) u of out (fp32 caches have fewer roundings still).
  * a received weight, 1 / l or w / l of each head: it is 2^(z - m - log2 l), with l's
    own error (w's and a sum: (2.92 |z| + 5) u, half of it at most where l <= 2), log2f
    to 1 ulp (2 u in powers of two), the two differences (u each of at most |z| + 1)
    and exp2f: less than (6 |z| + 15) u, and G u of a sum of G.
With two terms instead of three, w is 2^-18 off at worst (3.8e-6, 64 u) and y as much,
which z makes |z| ln 2 times larger in w; the inputs are chosen near that.
"""

import numpy as np
import pytest

from oracle import paged_oracle as PO
from tests.test_gpu_paged import U, Cache, status
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    ensure_built()


def _bf16(x):
    import torch
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).bfloat16().double().numpy()


def _two_terms(x):
    """x (fp32) in two bf16 terms, each rounded to nearest."""
    hi = _bf16(x)
    return hi + _bf16(x - hi)


def _inputs(kind, units, G, d, seed):
    """k [units] and q [units, G], bf16 values, whose w ("weights") or y ("query") two
    terms miss by much; and w with two terms there [units, G]."""
    rng = np.random.default_rng(seed)
    scale = np.float32(1.4426950408889634 / np.sqrt(float(d)))
    qs = _bf16((1 + np.arange(128) / 128.0)[None] * 2.0 ** np.arange(-2, 2)[:, None]).ravel()
    y = (qs.astype(np.float32) * scale).astype(np.float64)
    lo, hi, least = (0.3, 1.5, 2.9e-6) if kind == "weights" else (9.0, 11.0, 2.5e-6)
    ks, q, planted = [], [], []
    while len(ks) < units:
        k = -_bf16(rng.uniform(lo, hi) / rng.choice(y))
        z = y * k
        if kind == "weights":
            w2 = _two_terms(np.exp2(z).astype(np.float32))
            off = np.abs(w2 / np.exp2(z) - 1)
        else:
            w2 = np.exp2(_two_terms(y) * k)
            off = np.abs(_two_terms(y) / y - 1)
        fit = np.flatnonzero((off >= least) & (-z >= lo) & (-z <= hi))
        if len(fit) < G:
            continue
        pick = rng.choice(fit, G, replace=False)
        ks.append(k)
        q.append(qs[pick])
        planted.append(w2[pick])
    return np.array(ks), np.array(q), np.array(planted)


@pytest.mark.parametrize("kind", ["weights", "query"])
@pytest.mark.parametrize("dtype,G,d", [("bf16", 1, 128), ("bf16", 3, 64), ("bf16", 4, 128), ("bf16", 5, 128),
                                       ("bf16", 8, 64), ("f32", 4, 64), ("f32", 8, 128)])
def test_attention_needs_the_third_term(dtype, G, d, kind):
    import torch
    B, Hkv = 24, 2
    c = Cache(dtype, B, Hkv, G, d, 16, [2] * B, seed=80 + G)
    k, q, planted = _inputs(kind, B * Hkv, G, d, seed=G + d)
    rng = np.random.default_rng(81)
    dim = 2 * rng.integers(0, d // 2, B * Hkv)   # a pair's first element, another one in every unit
    v = torch.tensor([(-1.0) ** (i // 3) * 2.0 ** (i % 5 - 2) for i in range(d)], device="cuda").to(c.kp.dtype)
    c.pos.zero_()
    c.q.zero_()
    c.weight.zero_()
    for u in range(B * Hkv):
        b, h = divmod(u, Hkv)
        page = c.table[b, 0].item()
        c.kp[page, h, :2] = 0
        c.kp[page, h, 1, dim[u]] = float(k[u])
        c.vp[page, h, 0] = 0
        c.vp[page, h, 1] = v
        c.q[b, h * G:(h + 1) * G, dim[u]] = torch.tensor(q[u], device="cuda").to(c.q.dtype)
    assert np.array_equal(c.host(c.q).reshape(B * Hkv, G, d)[np.arange(B * Hkv), :, dim], q)   # exact in bf16
    ref, got, _, _ = PO.paged_attention(c.host(c.q), c.pos.cpu().numpy(), c.host(c.kp), c.host(c.vp),
                                        c.table.cpu().numpy(), c.lens.cpu().numpy(), c.theta)
    z = np.abs(np.log2(np.e) / np.sqrt(d) * q * k[:, None]).reshape(B, Hkv * G, 1)
    bound = (3 * z + 12) * U * np.abs(ref)
    # two terms would be seen: the same formula with them is out of bounds by twice the tolerance
    two = (planted / (1 + planted)).reshape(B, Hkv * G, 1) * c.host(v)
    assert np.all(np.abs(two - ref) > 2 * bound)
    out = c.attend(True).cpu().numpy().astype(np.float64)
    assert status() == 0
    err = np.abs(out - ref)
    assert np.all(err <= bound), f"out: {np.max(err / bound):.3g}x the bound"
    bound = ((6 * z + 15).reshape(B, Hkv, G).max(-1) + G)[..., None] * U * got
    err = np.abs(c.weight.cpu().numpy() - got)
    assert np.all(err <= bound), f"weight: {np.nanmax(err / np.maximum(bound, 1e-30)):.3g}x the bound"
