"""Binding of libfasa.so (ctypes; the paged cache's calls are marshalled by the
extension module _fasa_torch).

Each function has the name of its C entry point and takes torch CUDA tensors
(or, but for the paged cache, raw device addresses as ints).  It checks dtypes
and contiguity, passes ``data_ptr()`` and the current CUDA stream, and raises
``FasaError`` on a non-zero status.  Nothing here computes on the data.
"""

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(PKG, "libfasa.so")

FASA_F32, FASA_BF16 = 0, 1
FASA_DEV_BAD_INPUT, FASA_DEV_TIMEOUT, FASA_DEV_UNDRAINED = 1, 2, 4

EXPORTS = [
    "fasa_version", "fasa_status_string", "fasa_last_cuda_error", "fasa_max_budget",
    "fasa_workspace_size", "fasa_apply_rope_q", "fasa_build_kdom", "fasa_append_kdom",
    "fasa_tip_score", "fasa_topk_select", "fasa_focused_attention", "fasa_dense_attention",
    "fasa_decode_step", "fasa_device_status", "fasa_cluster_size", "fasa_decode_step_noalloc",
    "fasa_decode_step_append", "fasa_fc_agreement_workspace_size", "fasa_fc_agreement",
    "fasa_select_dominant_fcs", "fasa_compound_agreement", "fasa_test_fault_injection", "fasa_step_kernel",
    "fasa_build_knondom", "fasa_decode_step_split", "fasa_decode_step_append_split",
    "fasa_paged_append", "fasa_paged_attention", "fasa_paged_evict", "fasa_paged_workspace_size",
    "fasa_paged_evict_workspace_size", "fasa_paged_assign", "fasa_paged_rope_append", "fasa_paged_chunk_attention",
    "fasa_paged_chunk_workspace_size",
]


class FasaError(RuntimeError):
    def __init__(self, fn, status, lib):
        msg = lib.fasa_status_string(status).decode()
        if status == 4:
            msg += f" (cudaError {lib.fasa_last_cuda_error()})"
        super().__init__(f"{fn}: {msg}")
        self.status = status


class FasaDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("t_max", ctypes.c_int32), ("n_tip", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("rope_theta", ctypes.c_double),
    ]


def dims_for(cfg, cluster_ctas: int = 0, **override) -> FasaDims:
    """FasaDims from a workload config (anything with the same field names)."""
    d = dict(batch=cfg.batch, n_q_heads=cfg.n_q_heads, n_kv_heads=cfg.n_kv_heads,
             head_dim=cfg.head_dim, t_max=cfg.context, n_tip=cfg.n_tip,
             dtype=FASA_F32 if cfg.dtype == "f32" else FASA_BF16, rope_theta=cfg.rope_theta)
    d.update(override)
    return FasaDims(d["batch"], d["n_q_heads"], d["n_kv_heads"], d["head_dim"], d["t_max"],
                    d["n_tip"], d["dtype"], cluster_ctas, float(d["rope_theta"]))


class FasaPagedDims(ctypes.Structure):
    """Shapes of a paged cache and of the queries that read it (include/fasa.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("dtype", ctypes.c_int32), ("rope_theta", ctypes.c_double),
    ]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libfasa.so once.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m kv_cache_token_tip_gb300.build` (there is no fallback)")
        L = ctypes.CDLL(_LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        dp = ctypes.POINTER(FasaDims)
        sig = {
            "fasa_version": ([], ctypes.c_int),
            "fasa_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "fasa_last_cuda_error": ([], ctypes.c_int),
            "fasa_max_budget": ([dp, ctypes.POINTER(i32)], ctypes.c_int),
            "fasa_workspace_size": ([dp, i32, ctypes.POINTER(sz)], ctypes.c_int),
            "fasa_cluster_size": ([dp, ctypes.POINTER(i32)], ctypes.c_int),
            "fasa_step_kernel": ([dp, ctypes.POINTER(i32)], ctypes.c_int),
            "fasa_apply_rope_q": ([vp, vp, vp, dp, vp], ctypes.c_int),
            "fasa_build_kdom": ([vp, vp, vp, vp, dp, vp], ctypes.c_int),
            "fasa_build_knondom": ([vp, vp, vp, vp, dp, vp], ctypes.c_int),
            "fasa_decode_step_split": ([vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, dp, vp],
                                       ctypes.c_int),
            "fasa_append_kdom": ([vp, vp, vp, vp, dp, vp], ctypes.c_int),
            "fasa_tip_score": ([vp, vp, vp, vp, vp, dp, vp], ctypes.c_int),
            "fasa_topk_select": ([vp, vp, i32, vp, vp, dp, vp], ctypes.c_int),
            "fasa_focused_attention": ([vp, vp, vp, vp, vp, vp, i32, vp, dp, vp], ctypes.c_int),
            "fasa_dense_attention": ([vp, vp, vp, vp, vp, dp, vp], ctypes.c_int),
            "fasa_decode_step": ([vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, dp, vp],
                                 ctypes.c_int),
            "fasa_device_status": ([vp, ctypes.POINTER(i32)], ctypes.c_int),
            "fasa_decode_step_noalloc": ([vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, dp, vp], ctypes.c_int),
            "fasa_decode_step_append": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, dp, vp],
                                        ctypes.c_int),
            "fasa_decode_step_append_split": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, dp, vp],
                                              ctypes.c_int),
            "fasa_fc_agreement_workspace_size": ([dp, ctypes.POINTER(sz)], ctypes.c_int),
            "fasa_fc_agreement": ([vp, vp, vp, i32, vp, vp, sz, dp, vp], ctypes.c_int),
            "fasa_compound_agreement": ([vp, vp, vp, vp, i32, vp, vp, sz, dp, vp], ctypes.c_int),
            "fasa_select_dominant_fcs": ([vp, i32, vp, dp, vp], ctypes.c_int),
            "fasa_test_fault_injection": ([ctypes.c_uint64, i32, i32], ctypes.c_int),
        }
        pp = ctypes.POINTER(FasaPagedDims)
        sig.update({
            "fasa_paged_append": ([vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, pp, vp], ctypes.c_int),
            "fasa_paged_workspace_size": ([pp, i32, ctypes.POINTER(sz)], ctypes.c_int),
            "fasa_paged_attention": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, pp, vp], ctypes.c_int),
            "fasa_paged_evict_workspace_size": ([pp, i32, ctypes.POINTER(sz)], ctypes.c_int),
            "fasa_paged_evict": ([vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, pp, vp],
                                 ctypes.c_int),
            "fasa_paged_assign": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, pp, vp], ctypes.c_int),
            "fasa_paged_rope_append": ([vp, i64, vp, i64, vp, i64, vp, i32, vp, vp, vp, vp, vp,
                                        ctypes.POINTER(FasaRope), pp, vp], ctypes.c_int),
            "fasa_paged_chunk_workspace_size": ([pp, i32, i32, ctypes.POINTER(sz)], ctypes.c_int),
            "fasa_paged_chunk_attention": ([vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, pp, vp], ctypes.c_int),
        })
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


# ---------------------------------------------------------------- marshalling
def _ptr(x, dtype=None, name="tensor", host_ok=False):
    """Device pointer of a contiguous tensor.  With host_ok, a tensor in pinned
    host memory is accepted too (the GPU reads or writes it in place over the
    host link: the FASA-M placement of the K/V caches, zero-copy step I/O)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    import torch
    if not x.is_cuda and not (host_ok and x.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor" + (" or pinned host memory" if host_ok else ""))
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and x.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {x.dtype}, expected {dtype}")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _scratch(size, stream, device="cuda"):
    """A workspace for one call, allocated as memory of the call's stream: what
    was freed on another stream may still be in use there, and what this call
    leaves is handed out again behind it."""
    import torch
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _store_dtypes():
    import torch
    return (torch.float32, torch.bfloat16)


def _check(fn, st):
    if st != 0:
        raise FasaError(fn, st, lib())


def _i32():
    import torch
    return torch.int32


def _f32():
    import torch
    return torch.float32


# ---------------------------------------------------------------- entry points
def fasa_max_budget(dims: FasaDims) -> int:
    out = ctypes.c_int32(0)
    _check("fasa_max_budget", lib().fasa_max_budget(ctypes.byref(dims), ctypes.byref(out)))
    return out.value


def fasa_workspace_size(dims: FasaDims, budget: int) -> int:
    out = ctypes.c_size_t(0)
    _check("fasa_workspace_size", lib().fasa_workspace_size(ctypes.byref(dims), budget, ctypes.byref(out)))
    return out.value


def fasa_cluster_size(dims: FasaDims) -> int:
    out = ctypes.c_int32(0)
    _check("fasa_cluster_size", lib().fasa_cluster_size(ctypes.byref(dims), ctypes.byref(out)))
    return out.value


FASA_KERNEL_CLUSTER, FASA_KERNEL_SINGLE_EXCHANGE = 0, 1


def fasa_step_kernel(dims: FasaDims) -> int:
    """Which fused kernel serves fasa_decode_step for these dims on this
    device (FASA_KERNEL_CLUSTER or FASA_KERNEL_SINGLE_EXCHANGE)."""
    out = ctypes.c_int32(0)
    _check("fasa_step_kernel", lib().fasa_step_kernel(ctypes.byref(dims), ctypes.byref(out)))
    return out.value


def fasa_apply_rope_q(q, pos, q_rot, dims: FasaDims, stream=None):
    _check("fasa_apply_rope_q", lib().fasa_apply_rope_q(
        _ptr(q, _store_dtypes(), "q"), _ptr(pos, _i32(), "pos"), _ptr(q_rot, _f32(), "q_rot"),
        ctypes.byref(dims), _stream(stream)))


def fasa_build_kdom(k_cache, dom_fc, seq_lens, k_dom, dims: FasaDims, stream=None):
    _check("fasa_build_kdom", lib().fasa_build_kdom(
        _ptr(k_cache, _store_dtypes(), "k_cache"), _ptr(dom_fc, _i32(), "dom_fc"),
        _ptr(seq_lens, _i32(), "seq_lens"), _ptr(k_dom, _store_dtypes(), "k_dom"),
        ctypes.byref(dims), _stream(stream)))


def fasa_build_knondom(k_cache, dom_fc, seq_lens, k_nondom, dims: FasaDims, stream=None):
    """The non-dominant key pairs of every token, in FC order (FASA-M split
    keys); k_cache and k_nondom may live in page-locked host memory."""
    _check("fasa_build_knondom", lib().fasa_build_knondom(
        _ptr(k_cache, _store_dtypes(), "k_cache", True), _ptr(dom_fc, _i32(), "dom_fc"),
        _ptr(seq_lens, _i32(), "seq_lens"), _ptr(k_nondom, _store_dtypes(), "k_nondom", True),
        ctypes.byref(dims), _stream(stream)))


def fasa_decode_step_split(q, pos, k_nondom, v_cache, k_dom, dom_fc, seq_lens, budget: int, out,
                           idx_out=None, count_out=None, workspace=None, dims: FasaDims = None, stream=None):
    """fasa_decode_step with the keys split: non-dominant pairs in k_nondom,
    dominant ones in k_dom (FASA-M)."""
    ws_bytes = 0
    if workspace is not None and not isinstance(workspace, int):
        ws_bytes = workspace.numel() * workspace.element_size()
    _check("fasa_decode_step_split", lib().fasa_decode_step_split(
        _ptr(q, _store_dtypes(), "q", True), _ptr(pos, _i32(), "pos", True),
        _ptr(k_nondom, _store_dtypes(), "k_nondom", True), _ptr(v_cache, _store_dtypes(), "v_cache", True),
        _ptr(k_dom, _store_dtypes(), "k_dom"), _ptr(dom_fc, _i32(), "dom_fc"),
        _ptr(seq_lens, _i32(), "seq_lens", True), int(budget), _ptr(out, _f32(), "out", True),
        _ptr(idx_out, _i32(), "idx_out", True), _ptr(count_out, _i32(), "count_out", True),
        _ptr(workspace, None, "workspace"), ws_bytes, ctypes.byref(dims), _stream(stream)))


def fasa_append_kdom(k_new, dom_fc, tok_pos, k_dom, dims: FasaDims, stream=None):
    _check("fasa_append_kdom", lib().fasa_append_kdom(
        _ptr(k_new, _store_dtypes(), "k_new"), _ptr(dom_fc, _i32(), "dom_fc"),
        _ptr(tok_pos, _i32(), "tok_pos"), _ptr(k_dom, _store_dtypes(), "k_dom"),
        ctypes.byref(dims), _stream(stream)))


def fasa_tip_score(q_rot, k_dom, dom_fc, seq_lens, scores, dims: FasaDims, stream=None):
    _check("fasa_tip_score", lib().fasa_tip_score(
        _ptr(q_rot, _f32(), "q_rot"), _ptr(k_dom, _store_dtypes(), "k_dom"),
        _ptr(dom_fc, _i32(), "dom_fc"), _ptr(seq_lens, _i32(), "seq_lens"),
        _ptr(scores, _f32(), "scores"), ctypes.byref(dims), _stream(stream)))


def fasa_topk_select(scores, seq_lens, budget: int, idx, count, dims: FasaDims, stream=None):
    _check("fasa_topk_select", lib().fasa_topk_select(
        _ptr(scores, _f32(), "scores"), _ptr(seq_lens, _i32(), "seq_lens"), int(budget),
        _ptr(idx, _i32(), "idx"), _ptr(count, _i32(), "count"), ctypes.byref(dims), _stream(stream)))


def fasa_focused_attention(q_rot, k_cache, v_cache, seq_lens, idx, count, budget: int, out,
                           dims: FasaDims, stream=None):
    _check("fasa_focused_attention", lib().fasa_focused_attention(
        _ptr(q_rot, _f32(), "q_rot"), _ptr(k_cache, _store_dtypes(), "k_cache", True),
        _ptr(v_cache, _store_dtypes(), "v_cache", True), _ptr(seq_lens, _i32(), "seq_lens"),
        _ptr(idx, _i32(), "idx"), _ptr(count, _i32(), "count"), int(budget),
        _ptr(out, _f32(), "out"), ctypes.byref(dims), _stream(stream)))


def fasa_dense_attention(q_rot, k_cache, v_cache, seq_lens, out, dims: FasaDims, stream=None):
    _check("fasa_dense_attention", lib().fasa_dense_attention(
        _ptr(q_rot, _f32(), "q_rot"), _ptr(k_cache, _store_dtypes(), "k_cache", True),
        _ptr(v_cache, _store_dtypes(), "v_cache", True), _ptr(seq_lens, _i32(), "seq_lens"),
        _ptr(out, _f32(), "out"), ctypes.byref(dims), _stream(stream)))


def fasa_decode_step(q, pos, k_cache, v_cache, k_dom, dom_fc, seq_lens, budget: int, out,
                     idx_out=None, count_out=None, workspace=None, dims: FasaDims = None, stream=None):
    ws_bytes = 0
    if workspace is not None and not isinstance(workspace, int):
        ws_bytes = workspace.numel() * workspace.element_size()
    _check("fasa_decode_step", lib().fasa_decode_step(
        _ptr(q, _store_dtypes(), "q", True), _ptr(pos, _i32(), "pos", True),
        _ptr(k_cache, _store_dtypes(), "k_cache", True), _ptr(v_cache, _store_dtypes(), "v_cache", True),
        _ptr(k_dom, _store_dtypes(), "k_dom"), _ptr(dom_fc, _i32(), "dom_fc"),
        _ptr(seq_lens, _i32(), "seq_lens", True), int(budget), _ptr(out, _f32(), "out", True),
        _ptr(idx_out, _i32(), "idx_out", True), _ptr(count_out, _i32(), "count_out", True),
        _ptr(workspace, None, "workspace"), ws_bytes, ctypes.byref(dims), _stream(stream)))


def fasa_decode_step_append(q, k_new, v_new, seq_lens, k_cache, v_cache, k_dom, dom_fc, budget: int, out,
                            idx_out=None, count_out=None, workspace=None, dims: FasaDims = None, stream=None):
    """The decode step with the new token appended first: k_new (pre-RoPE)
    and v_new [B,Hkv,d] go to index seq_lens[b] of the caches (and K_dom),
    and the step attends over seq_lens[b] + 1 tokens with the query at
    position seq_lens[b].  seq_lens is not advanced."""
    ws_bytes = 0
    if workspace is not None and not isinstance(workspace, int):
        ws_bytes = workspace.numel() * workspace.element_size()
    _check("fasa_decode_step_append", lib().fasa_decode_step_append(
        _ptr(q, _store_dtypes(), "q"), _ptr(k_new, _store_dtypes(), "k_new"),
        _ptr(v_new, _store_dtypes(), "v_new"), _ptr(seq_lens, _i32(), "seq_lens"),
        _ptr(k_cache, _store_dtypes(), "k_cache", True), _ptr(v_cache, _store_dtypes(), "v_cache", True),
        _ptr(k_dom, _store_dtypes(), "k_dom"), _ptr(dom_fc, _i32(), "dom_fc"), int(budget),
        _ptr(out, _f32(), "out"), _ptr(idx_out, _i32(), "idx_out"), _ptr(count_out, _i32(), "count_out"),
        _ptr(workspace, None, "workspace"), ws_bytes, ctypes.byref(dims), _stream(stream)))


def fasa_decode_step_append_split(q, k_new, v_new, seq_lens, k_nondom, v_cache, k_dom, dom_fc, budget: int, out,
                                  idx_out=None, count_out=None, workspace=None, dims: FasaDims = None, stream=None):
    """fasa_decode_step_append over split keys: the new token's non-dominant
    pairs go to its k_nondom row, its dominant pairs to K_dom, v_new to
    v_cache; then the split step attends over seq_lens[b] + 1 tokens."""
    ws_bytes = 0
    if workspace is not None and not isinstance(workspace, int):
        ws_bytes = workspace.numel() * workspace.element_size()
    _check("fasa_decode_step_append_split", lib().fasa_decode_step_append_split(
        _ptr(q, _store_dtypes(), "q"), _ptr(k_new, _store_dtypes(), "k_new"),
        _ptr(v_new, _store_dtypes(), "v_new"), _ptr(seq_lens, _i32(), "seq_lens"),
        _ptr(k_nondom, _store_dtypes(), "k_nondom", True), _ptr(v_cache, _store_dtypes(), "v_cache", True),
        _ptr(k_dom, _store_dtypes(), "k_dom"), _ptr(dom_fc, _i32(), "dom_fc"), int(budget),
        _ptr(out, _f32(), "out"), _ptr(idx_out, _i32(), "idx_out"), _ptr(count_out, _i32(), "count_out"),
        _ptr(workspace, None, "workspace"), ws_bytes, ctypes.byref(dims), _stream(stream)))


def fasa_fc_agreement_workspace_size(dims: FasaDims) -> int:
    out = ctypes.c_size_t(0)
    _check("fasa_fc_agreement_workspace_size",
           lib().fasa_fc_agreement_workspace_size(ctypes.byref(dims), ctypes.byref(out)))
    return out.value


def fasa_fc_agreement(q_rot, k_cache, seq_lens, topk: int, ca, dims: FasaDims, workspace=None, stream=None):
    """Contextual Agreement of every FC for every (batch, KV head):
    ca [B, Hkv, d/2] fp32.  Without a workspace one is allocated here."""
    if workspace is None:
        workspace = _scratch(fasa_fc_agreement_workspace_size(dims), stream, ca.device)
    _check("fasa_fc_agreement", lib().fasa_fc_agreement(
        _ptr(q_rot, _f32(), "q_rot"), _ptr(k_cache, _store_dtypes(), "k_cache"),
        _ptr(seq_lens, _i32(), "seq_lens"), int(topk), _ptr(ca, _f32(), "ca"),
        _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(), ctypes.byref(dims),
        _stream(stream)))


def fasa_compound_agreement(q_rot, k_cache, dom_fc, seq_lens, topk: int, cca, dims: FasaDims, workspace=None,
                            stream=None):
    """Compound CA of the chosen FCs dom_fc [Hkv, n_tip] per (batch, KV head):
    cca [B, Hkv] fp32.  Without a workspace one is allocated here."""
    if workspace is None:
        workspace = _scratch(fasa_fc_agreement_workspace_size(dims), stream, cca.device)
    _check("fasa_compound_agreement", lib().fasa_compound_agreement(
        _ptr(q_rot, _f32(), "q_rot"), _ptr(k_cache, _store_dtypes(), "k_cache"), _ptr(dom_fc, _i32(), "dom_fc"),
        _ptr(seq_lens, _i32(), "seq_lens"), int(topk), _ptr(cca, _f32(), "cca"),
        _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(), ctypes.byref(dims),
        _stream(stream)))


def fasa_select_dominant_fcs(ca_mean, n_tip: int, dom_fc, dims: FasaDims, stream=None):
    """dom_fc [Hkv, n_tip] int32 <- the n_tip FCs of highest mean CA per head."""
    _check("fasa_select_dominant_fcs", lib().fasa_select_dominant_fcs(
        _ptr(ca_mean, _f32(), "ca_mean"), int(n_tip), _ptr(dom_fc, _i32(), "dom_fc"), ctypes.byref(dims),
        _stream(stream)))


def fasa_decode_step_noalloc(q, pos, k_cache, v_cache, k_dom, dom_fc, seq_lens, budget: int, out,
                             idx_out=None, count_out=None, dims: FasaDims = None, stream=None):
    """fasa_decode_step without a workspace argument: for callers that cannot
    allocate device memory, the step uses the library's fixed scratch array."""
    _check("fasa_decode_step_noalloc", lib().fasa_decode_step_noalloc(
        _ptr(q, _store_dtypes(), "q"), _ptr(pos, _i32(), "pos"),
        _ptr(k_cache, _store_dtypes(), "k_cache", True), _ptr(v_cache, _store_dtypes(), "v_cache", True),
        _ptr(k_dom, _store_dtypes(), "k_dom"), _ptr(dom_fc, _i32(), "dom_fc"),
        _ptr(seq_lens, _i32(), "seq_lens"), int(budget), _ptr(out, _f32(), "out"),
        _ptr(idx_out, _i32(), "idx_out"), _ptr(count_out, _i32(), "count_out"),
        ctypes.byref(dims), _stream(stream)))


# ---------------------------------------------------------------- paged cache
# (the tensors are checked and their addresses passed in csrc/fasa_torch.cpp: a
# small call's time is the host's)
_native = None


def _marshal():
    """The extension module, its calls bound to libfasa.so's entry points."""
    global _native
    if _native is None:
        import torch  # (whose libraries it needs)
        how = "build it with `python -m kv_cache_token_tip_gb300.build` (there is no fallback)"
        try:
            from . import _fasa_torch as m
        except ImportError as e:
            raise RuntimeError(f"the module _fasa_torch is missing or does not load: {how}") from e
        if getattr(m, "torch_version", None) != str(torch.__version__):
            raise RuntimeError(f"the module _fasa_torch was built for another torch: {how}")
        m.bind(*(ctypes.cast(getattr(lib(), f"fasa_paged_{n}"), ctypes.c_void_p).value
                 for n in ("append", "attention", "evict", "assign", "rope_append", "chunk_attention")))
        _native = m
    return _native


def _where(dims):
    if not isinstance(dims, FasaPagedDims):
        raise TypeError("dims must be FasaPagedDims")
    return ctypes.addressof(dims)


def fasa_paged_append(k_new, v_new, pos, k_pages, v_pages, page_table, seq_lens, cu_new=None, weight=None,
                      token_pos=None, dims: FasaPagedDims = None, stream=None):
    """Writes new tokens behind each sequence's cached ones: k_new (pre-RoPE)
    and v_new [n_tokens, Hkv, d], those of sequence b at cu_new[b] ..
    cu_new[b+1], or one per sequence without cu_new; the first of b gets the
    position pos[b].  seq_lens is not advanced."""
    st = (_native or _marshal()).append(k_new, v_new, pos, k_pages, v_pages, page_table, seq_lens, cu_new, weight,
                                        token_pos, _where(dims), None if stream is None else _stream(stream))
    if st:
        _check("fasa_paged_append", st)


def fasa_paged_workspace_size(dims: FasaPagedDims, weights: bool = False) -> int:
    out = ctypes.c_size_t(0)
    _check("fasa_paged_workspace_size",
           lib().fasa_paged_workspace_size(ctypes.byref(dims), int(bool(weights)), ctypes.byref(out)))
    return out.value


def fasa_paged_attention(q, pos, k_pages, v_pages, page_table, seq_lens, out, weight=None, workspace=None,
                         dims: FasaPagedDims = None, stream=None):
    """Attention of one new token per sequence over its cached tokens; with
    weight, each cached token's softmax weights are added to it.  Without a
    workspace one is allocated here."""
    if workspace is None:
        workspace = _scratch(fasa_paged_workspace_size(dims, weight is not None), stream)
    st = (_native or _marshal()).attention(q, pos, k_pages, v_pages, page_table, seq_lens, out, weight, workspace,
                                           _where(dims), None if stream is None else _stream(stream))
    if st:
        _check("fasa_paged_attention", st)


def fasa_paged_evict_workspace_size(dims: FasaPagedDims, keep: int) -> int:
    out = ctypes.c_size_t(0)
    _check("fasa_paged_evict_workspace_size",
           lib().fasa_paged_evict_workspace_size(ctypes.byref(dims), int(keep), ctypes.byref(out)))
    return out.value


def fasa_paged_evict(weight, token_pos, pos, k_pages, v_pages, page_table, seq_lens, keep: int, new_lens,
                     sinks: int = 0, recent: int = 0, weight_out=None, token_pos_out=None, workspace=None,
                     dims: FasaPagedDims = None, stream=None):
    """Cuts every (sequence, KV head) down to the `keep` heaviest tokens (the
    first `sinks` positions and the last `recent` up to pos always stay); the
    kept ones behind slot `keep` move into the slots the others leave.
    new_lens [B] <- min(seq_lens, keep).  The statistics change in place, or
    go to weight_out and token_pos_out.  Without a workspace one is allocated
    here."""
    if workspace is None:
        workspace = _scratch(fasa_paged_evict_workspace_size(dims, keep), stream)
    st = (_native or _marshal()).evict(weight, token_pos, pos, k_pages, v_pages, page_table, seq_lens, keep, new_lens,
                                       sinks, recent, weight_out, token_pos_out, workspace, _where(dims),
                                       None if stream is None else _stream(stream))
    if st:
        _check("fasa_paged_evict", st)


# ------------------------------------------------ a step of new tokens, paged
FASA_ROPE_INTERLEAVED, FASA_ROPE_HALF = 0, 1
FASA_ROPE_PLAIN, FASA_ROPE_LINEAR, FASA_ROPE_WAVELENGTH, FASA_ROPE_RAMP = 0, 1, 2, 3


class FasaRope(ctypes.Structure):
    """Rotary positions (include/fasa.h): which elements of a head make a pair,
    how many of them turn, and how their frequencies are scaled."""
    _fields_ = [
        ("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32),
        ("reserved", ctypes.c_int32), ("rope_theta", ctypes.c_double), ("factor", ctypes.c_double),
        ("low", ctypes.c_double), ("high", ctypes.c_double), ("original", ctypes.c_double),
        ("magnitude", ctypes.c_double),
    ]

    def __init__(self, layout: int = FASA_ROPE_INTERLEAVED, rotary_dim: int = 128, scaling: int = FASA_ROPE_PLAIN,
                 rope_theta: float = 1e4, factor: float = 1.0, low: float = 1.0, high: float = 4.0,
                 original: float = 8192.0, magnitude: float = 1.0):
        super().__init__(layout, rotary_dim, scaling, 0, float(rope_theta), float(factor), float(low), float(high),
                         float(original), float(magnitude))


def fasa_paged_assign(have_lens, want_lens, page_table, free_pages, free_count, lens_out, cu_new, token_map, pos=None,
                      free_count_out=None, dims: FasaPagedDims = None, stream=None):
    """Pages for the sequences that grow from have_lens to want_lens, from the
    end of the list of free ones, and back to it from those that shrink:
    page_table, free_pages and free_count change in place (the count goes to
    free_count_out where that is given).  lens_out [B], cu_new [B+1] and
    token_map [max_tokens, 4] (sequence, slot, page, position of each new token,
    -1 behind the last) are written; growing sequences are served in order while
    the pages and the map's rows last.  The first new token of b has the position
    pos[b], or its slot."""
    st = (_native or _marshal()).assign(have_lens, want_lens, page_table, free_pages, free_count, lens_out, cu_new,
                                        token_map, pos, free_count_out, _where(dims),
                                        None if stream is None else _stream(stream))
    if st:
        _check("fasa_paged_assign", st)


def fasa_paged_rope_append(q, k, v, token_map, q_out, k_pages, v_pages, weight=None, token_pos=None,
                           rope: FasaRope = None, dims: FasaPagedDims = None, stream=None):
    """Turns the new tokens' queries (to q_out [n_tokens, Hq, d]) and keys (to their
    pages, with the values) by the positions of token_map, and begins their
    statistics.  q [n_tokens, Hq, d], k and v [n_tokens, Hkv, d] may be parts of
    wider rows.  q with q_out, or k and v with the pages, may be None."""
    if not isinstance(rope, FasaRope):
        raise TypeError("rope must be FasaRope")
    st = (_native or _marshal()).rope_append(q, k, v, token_map, q_out, k_pages, v_pages, weight, token_pos,
                                             ctypes.addressof(rope), _where(dims),
                                             None if stream is None else _stream(stream))
    if st:
        _check("fasa_paged_rope_append", st)


def fasa_paged_chunk_workspace_size(dims: FasaPagedDims, n_tokens: int, weights: bool = False) -> int:
    out = ctypes.c_size_t(0)
    _check("fasa_paged_chunk_workspace_size",
           lib().fasa_paged_chunk_workspace_size(ctypes.byref(dims), int(n_tokens), int(bool(weights)),
                                                 ctypes.byref(out)))
    return out.value


def fasa_paged_chunk_attention(q, k_pages, v_pages, page_table, seq_lens, out, cu_new=None, weight=None,
                               workspace=None, dims: FasaPagedDims = None, stream=None):
    """Attention of each sequence's new tokens, the last of its seq_lens cached ones,
    every one over the slots up to its own.  q and out [n_tokens, Hq, d] in the
    storage dtype, q already turned; those of sequence b are cu_new[b] ..
    cu_new[b+1], or one per sequence without cu_new.  With weight, each slot's
    softmax weights are added to it.  Without a workspace one is allocated here."""
    where, native = _where(dims), _native or _marshal()
    if workspace is None:  # (of what is no tensor: none; the call says so)
        n = q.numel() // max(dims.n_q_heads * dims.head_dim, 1) if hasattr(q, "numel") else 0
        workspace = _scratch(fasa_paged_chunk_workspace_size(dims, n, weight is not None), stream)
    st = native.chunk(q, k_pages, v_pages, page_table, seq_lens, out, cu_new, weight, workspace, where,
                      None if stream is None else _stream(stream))
    if st:
        _check("fasa_paged_chunk_attention", st)


def fasa_device_status(stream=None) -> int:
    out = ctypes.c_int32(0)
    _check("fasa_device_status", lib().fasa_device_status(_stream(stream), ctypes.byref(out)))
    return out.value


def fasa_test_fault_injection(wait_limit_ns: int = 1_000_000_000, drop_tip_tile: int = -1,
                              drop_fac_refill: int = -1) -> None:
    """Test hook: bound of every device wait, one TIP tile whose copy the
    fused step never issues, and one refill of the single-exchange kernel's
    FAC whose completion is never reported (-1: none).  The defaults restore
    normal runs."""
    _check("fasa_test_fault_injection", lib().fasa_test_fault_injection(int(wait_limit_ns), int(drop_tip_tile),
                                                                         int(drop_fac_refill)))
