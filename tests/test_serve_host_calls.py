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
