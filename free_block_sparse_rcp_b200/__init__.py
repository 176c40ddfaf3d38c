"""SparsePR per-call sparse attention on B200 (sm_100a): Python binding.

A thin ctypes layer over ``libsparsepr.so`` (the C ABI declared in
``include/sparsepr.h``).  Every function here only marshals torch tensors into
device pointers and the current CUDA stream and raises ``SparsePRError`` on a
non-zero status; all arithmetic runs in the library's CUDA kernels.  There is no
fallback: importing this package without the built library raises ImportError.
"""
from __future__ import annotations

import ctypes
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsparsepr.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python free_block_sparse_rcp_b200/build.py`")
_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_ip = ctypes.POINTER(ctypes.c_int)


class Params(ctypes.Structure):
    """Mirror of ``sparsepr_params``."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int), ("d", ctypes.c_int),
                ("block", ctypes.c_int), ("density", ctypes.c_float), ("n_kgroups", ctypes.c_int),
                ("n_qgroups", ctypes.c_int), ("n_samples", ctypes.c_int), ("n_probes", ctypes.c_int),
                ("eig_rank", ctypes.c_int), ("sub_rank", ctypes.c_int), ("kmeans_iters", ctypes.c_int),
                ("ridge_lambda", ctypes.c_float), ("scale", ctypes.c_float), ("seed", ctypes.c_ulonglong),
                ("frame_id", _vp), ("n_frames", ctypes.c_int), ("partition_mode", ctypes.c_int),
                ("fit_weighted", ctypes.c_int), ("fit_input", ctypes.c_int), ("head_offset", ctypes.c_int),
                ("heads_total", ctypes.c_int)]

    @property
    def BH(self) -> int:
        return self.B * self.H

    @property
    def tiles(self) -> int:
        return (self.N + self.block - 1) // self.block

    def eff_scale(self) -> float:
        return self.scale if self.scale > 0 else 1.0 / math.sqrt(self.d)

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_ if k not in ("frame_id", "n_frames")}

    @classmethod
    def make(cls, B, H, N, d, *, block, density, n_kgroups, n_qgroups, n_samples, n_probes, eig_rank,
             sub_rank, kmeans_iters, ridge_lambda=1e-2, scale=0.0, seed=0, frame_id=None, n_frames=0,
             partition_mode=0, fit_weighted=0, fit_input=0, head_offset=0, heads_total=0):
        """frame_id: optional int32 device tensor [N] (frame-causal masking, kept alive by the
        caller for as long as the params are used).  fit_input: 0 = the affine map takes the
        whole sparse output row, 1 = its projection on the residual subspace.  head_offset /
        heads_total: this call's heads within the layer (random streams only)."""
        fid = None if frame_id is None else frame_id.data_ptr()
        return cls(B=B, H=H, N=N, d=d, block=block, density=density, n_kgroups=n_kgroups,
                   n_qgroups=n_qgroups, n_samples=n_samples, n_probes=n_probes, eig_rank=eig_rank,
                   sub_rank=sub_rank, kmeans_iters=kmeans_iters, ridge_lambda=ridge_lambda, scale=scale,
                   seed=seed, frame_id=fid, n_frames=n_frames, partition_mode=partition_mode,
                   fit_weighted=fit_weighted, fit_input=fit_input, head_offset=head_offset,
                   heads_total=heads_total)


class PartitionTrace(ctypes.Structure):
    """Mirror of ``sparsepr_partition_trace`` (NULL fields are skipped)."""
    _fields_ = [(n, _vp) for n in ("sample_idx", "metric", "eigval", "eigvec", "key_coords", "key_init",
                                   "key_label_iters", "key_centroids", "query_coords", "query_init",
                                   "query_label_iters", "cell_mass", "alpha")]


class ProbeTrace(ctypes.Structure):
    """Mirror of ``sparsepr_probe_trace``."""
    _fields_ = [(n, _vp) for n in ("probe_o_sparse", "probe_lse_dense", "probe_lse_sparse", "sigma", "b_sub")]


BF16, FP16, FP32 = 0, 1, 2
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


def _dtype_code(dt) -> int:
    """SPARSEPR_BF16 / FP16 / FP32 of a torch dtype (integers pass through)."""
    if isinstance(dt, int):
        return dt
    import torch
    codes = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
    if dt not in codes:
        raise ValueError(f"unsupported dtype {dt}")
    return codes[dt]


_ll3 = ctypes.c_longlong * 3
_ll2 = ctypes.c_longlong * 2


class RopeParams(ctypes.Structure):
    """Mirror of ``sparsepr_rope_params``."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "N", "d", "H2", "dtype", "rot_dim", "layout", "n_axes")] + \
               [("axis_dim", ctypes.c_int * 3)] + \
               [(n, ctypes.c_int) for n in ("pos_batched", "scaling", "orig_len")] + \
               [(n, ctypes.c_double) for n in ("theta", "factor", "beta_fast", "beta_slow", "magnitude")] + \
               [(n, _ll3) for n in ("x_stride", "y_stride", "x2_stride", "y2_stride")]

    @classmethod
    def make(cls, B, H, N, d, *, H2=0, dtype=BF16, rot_dim=None, layout="half", axis_dim=None, pos_batched=0,
             scaling="none", orig_len=0, theta=10000.0, factor=1.0, beta_fast=32.0, beta_slow=1.0, magnitude=0.0):
        """layout: "half" or "interleaved"; axis_dim: rotated elements per position axis
        (default one axis of rot_dim); scaling: "none", "linear", "base" or "parts"."""
        rot = d if rot_dim is None else rot_dim
        axes = [rot] if axis_dim is None else list(axis_dim)
        if not 1 <= len(axes) <= 3:
            raise ValueError("axis_dim must name 1 to 3 axes")
        p = cls(B=B, H=H, N=N, d=d, H2=H2, dtype=_dtype_code(dtype), rot_dim=rot,
                layout=ROPE_LAYOUTS.get(layout, layout), n_axes=len(axes), pos_batched=pos_batched,
                scaling=ROPE_SCALINGS.get(scaling, scaling), orig_len=orig_len, theta=theta, factor=factor,
                beta_fast=beta_fast, beta_slow=beta_slow, magnitude=magnitude)
        for i, a in enumerate(axes):
            p.axis_dim[i] = a
        return p


class CacheParams(ctypes.Structure):
    """Mirror of ``sparsepr_cache_params``."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "Hq", "Hkv", "d", "dtype", "page", "n_pages", "max_pages", "T",
                                            "max_chunk", "frame")] + [("scale", ctypes.c_float)] + \
               [(n, ctypes.c_int) for n in ("q_block", "n_select", "n_sink", "n_recent")] + \
               [(n, _ll2) for n in ("q_stride", "o_stride", "k_stride", "v_stride")]

    @classmethod
    def make(cls, B, Hq, Hkv, d, *, page, n_pages, max_pages, T, max_chunk, frame=1, dtype=BF16, scale=0.0, q_block=0,
             n_select=0, n_sink=0, n_recent=0):
        return cls(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=_dtype_code(dtype), page=page, n_pages=n_pages,
                   max_pages=max_pages, T=T, max_chunk=max_chunk, frame=frame, scale=scale, q_block=q_block,
                   n_select=n_select, n_sink=n_sink, n_recent=n_recent)


_P = ctypes.POINTER(Params)
_R = ctypes.POINTER(RopeParams)
_C = ctypes.POINTER(CacheParams)
_sz = ctypes.c_size_t
_sig = {
    "sparsepr_workspace_bytes": (ctypes.c_size_t, [_P]),
    "sparsepr_forward_workspace_bytes": (ctypes.c_size_t, [_P]),
    "sparsepr_validate": (ctypes.c_int, [_P]),
    "sparsepr_partition": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                          ctypes.POINTER(PartitionTrace), _vp, ctypes.c_size_t, _vp]),
    "sparsepr_attend": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                       ctypes.c_size_t, _vp]),
    "sparsepr_probe_fit": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                          _vp, ctypes.POINTER(ProbeTrace), _vp, ctypes.c_size_t, _vp]),
    "sparsepr_probe_fit_noalloc": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                  _vp, _vp, _vp]),
    "sparsepr_reconstruct": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "sparsepr_forward": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "sparsepr_forward_host": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "sparsepr_forward_host_chunked": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp,
                                                     ctypes.c_size_t, _vp, _vp, _vp]),
    "sparsepr_dense_attention": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "sparsepr_workspace_error": (ctypes.c_int, [_P, _vp, _vp]),
    "sparsepr_workspace_clear_error": (ctypes.c_int, [_P, _vp, _vp]),
    "sparsepr_rope_validate": (ctypes.c_int, [_R]),
    "sparsepr_rope_frequencies": (ctypes.c_int, [_R, ctypes.POINTER(ctypes.c_double)]),
    "sparsepr_rope": (ctypes.c_int, [_R] + [_vp] * 7),
    "sparsepr_rope_backward": (ctypes.c_int, [_R] + [_vp] * 7),
    "sparsepr_cache_validate": (ctypes.c_int, [_C]),
    "sparsepr_paged_workspace_bytes": (_sz, [_C]),
    "sparsepr_cache_append": (ctypes.c_int, [_C] + [_vp] * 8 + [_R, _vp, _vp, _vp, _sz, _vp]),
    "sparsepr_select_units": (ctypes.c_int, [_C]),
    "sparsepr_page_select": (ctypes.c_int, [_C] + [_vp] * 8 + [_sz, _vp]),
    "sparsepr_paged_attention": (ctypes.c_int, [_C] + [_vp] * 11 + [_sz, _vp]),
    "sparsepr_paged_error": (ctypes.c_int, [_vp, _vp]),
    "sparsepr_paged_clear_error": (ctypes.c_int, [_vp, _vp]),
    "sparsepr_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sparsepr_last_error": (ctypes.c_char_p, []),
    "sparsepr_last_launch_count": (ctypes.c_int, []),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sig)


class SparsePRError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.sparsepr_status_string(status).decode()
        detail = _lib.sparsepr_last_error().decode()
        super().__init__(f"{where}: {msg} ({detail})")


def _check(status: int, where: str):
    if status != 0:
        raise SparsePRError(status, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(t):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _trace(cls, d):
    if d is None:
        return None
    tr = cls()
    for k, v in d.items():
        setattr(tr, k, v.data_ptr() if v is not None else None)
    return ctypes.byref(tr)


def last_launch_count() -> int:
    return _lib.sparsepr_last_launch_count()


def sparsepr_validate(p: Params) -> int:
    return _lib.sparsepr_validate(ctypes.byref(p))


def sparsepr_workspace_bytes(p: Params) -> int:
    return _lib.sparsepr_workspace_bytes(ctypes.byref(p))


def sparsepr_forward_workspace_bytes(p: Params) -> int:
    return _lib.sparsepr_forward_workspace_bytes(ctypes.byref(p))


def workspace(p: Params, device, forward: bool = False):
    """A caller-owned workspace tensor of the size the library asks for."""
    import torch
    n = sparsepr_forward_workspace_bytes(p) if forward else sparsepr_workspace_bytes(p)
    if n == 0:
        _check(sparsepr_validate(p), "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def sparsepr_partition(p, Q, K, perm_q, perm_k, label_q, label_k, qoff, koff, route, block_mask, rho_exec,
                       ws, trace=None):
    _check(_lib.sparsepr_partition(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(perm_q), _ptr(perm_k),
                                   _ptr(label_q), _ptr(label_k), _ptr(qoff), _ptr(koff), _ptr(route),
                                   _ptr(block_mask), _ptr(rho_exec), _trace(PartitionTrace, trace),
                                   _ptr(ws), ws.numel(), _stream(Q)), "sparsepr_partition")


def sparsepr_attend(p, Q, K, V, perm_q, perm_k, qoff, koff, route, O_sparse, lse, ws):
    _check(_lib.sparsepr_attend(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(perm_q), _ptr(perm_k),
                                _ptr(qoff), _ptr(koff), _ptr(route), _ptr(O_sparse), _ptr(lse), _ptr(ws),
                                ws.numel(), _stream(Q)), "sparsepr_attend")


def sparsepr_probe_fit(p, Q, K, V, label_k, perm_q, qoff, route, probe_idx, probe_o_dense, b_full, Vr, W,
                       Bmat, ws, trace=None):
    _check(_lib.sparsepr_probe_fit(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(label_k), _ptr(perm_q),
                                   _ptr(qoff), _ptr(route), _ptr(probe_idx), _ptr(probe_o_dense),
                                   _ptr(b_full), _ptr(Vr), _ptr(W), _ptr(Bmat), _trace(ProbeTrace, trace),
                                   _ptr(ws), ws.numel(), _stream(Q)), "sparsepr_probe_fit")


def sparsepr_probe_fit_noalloc(p, Q, K, V, label_k, perm_q, qoff, route, probe_idx, probe_o_dense, b_full,
                               Vr, W, Bmat):
    _check(_lib.sparsepr_probe_fit_noalloc(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(label_k),
                                           _ptr(perm_q), _ptr(qoff), _ptr(route), _ptr(probe_idx),
                                           _ptr(probe_o_dense), _ptr(b_full), _ptr(Vr), _ptr(W), _ptr(Bmat),
                                           _stream(Q)), "sparsepr_probe_fit_noalloc")


def sparsepr_reconstruct(p, O_sparse, probe_idx, probe_o_dense, b_full, Vr, W, O):
    _check(_lib.sparsepr_reconstruct(ctypes.byref(p), _ptr(O_sparse), _ptr(probe_idx), _ptr(probe_o_dense),
                                     _ptr(b_full), _ptr(Vr), _ptr(W), _ptr(O), _stream(O)),
           "sparsepr_reconstruct")


def sparsepr_forward(p, Q, K, V, O, rho_exec, ws):
    _check(_lib.sparsepr_forward(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(rho_exec),
                                 _ptr(ws), ws.numel(), _stream(Q)), "sparsepr_forward")


def sparsepr_forward_host(p, Q_host, K_host, V_host, O_host, qkv_dev, o_dev, ws):
    _check(_lib.sparsepr_forward_host(ctypes.byref(p), _ptr(Q_host), _ptr(K_host), _ptr(V_host),
                                      _ptr(O_host), _ptr(qkv_dev), _ptr(o_dev), _ptr(ws), ws.numel(),
                                      _stream(qkv_dev)), "sparsepr_forward_host")


def sparsepr_forward_host_chunked(p, Q_host, K_host, V_host, O_host, qkv_dev, o_dev, n_chunks, ws,
                                  copy_in_stream=None, copy_out_stream=None):
    """The chunked host pipeline on the current stream of qkv_dev's device; the copy streams
    are torch.cuda.Stream objects (None: the current stream)."""
    def sp(s):
        return None if s is None else ctypes.c_void_p(s.cuda_stream)
    _check(_lib.sparsepr_forward_host_chunked(ctypes.byref(p), _ptr(Q_host), _ptr(K_host), _ptr(V_host),
                                              _ptr(O_host), _ptr(qkv_dev), _ptr(o_dev), int(n_chunks), _ptr(ws),
                                              ws.numel(), _stream(qkv_dev), sp(copy_in_stream),
                                              sp(copy_out_stream)), "sparsepr_forward_host_chunked")


def chunk_params(p: Params, n_chunks: int) -> Params:
    """Params of the largest chunk of sparsepr_forward_host_chunked (for its workspace size)."""
    q = Params.from_buffer_copy(p)
    q.B, q.H = 1, -(-p.BH // n_chunks)
    q.head_offset, q.heads_total = 0, 0
    return q


def sparsepr_dense_attention(p, Q, K, V, O, lse, ws=None):
    _check(_lib.sparsepr_dense_attention(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse),
                                         _ptr(ws), 0 if ws is None else ws.numel(), _stream(Q)),
           "sparsepr_dense_attention")


def sparsepr_workspace_error(p, ws) -> int:
    return _lib.sparsepr_workspace_error(ctypes.byref(p), _ptr(ws), _stream(ws))


def sparsepr_workspace_clear_error(p, ws):
    _check(_lib.sparsepr_workspace_clear_error(ctypes.byref(p), _ptr(ws), _stream(ws)),
           "sparsepr_workspace_clear_error")


# ---------------------------------------------------------------------------
# Output allocation helpers (torch.empty only; no arithmetic)
# ---------------------------------------------------------------------------
def alloc_partition(p: Params, device):
    import torch
    BH, N = p.BH, p.N
    i32 = dict(dtype=torch.int32, device=device)
    return dict(perm_q=torch.empty(BH, N, **i32), perm_k=torch.empty(BH, N, **i32),
                label_q=torch.empty(BH, N, **i32), label_k=torch.empty(BH, N, **i32),
                qoff=torch.empty(BH, p.n_qgroups + 1, **i32), koff=torch.empty(BH, p.n_kgroups + 1, **i32),
                route=torch.empty(BH, p.n_qgroups, p.n_kgroups, dtype=torch.uint8, device=device),
                block_mask=torch.empty(BH, p.tiles, p.tiles, dtype=torch.uint8, device=device),
                rho_exec=torch.empty(BH, dtype=torch.float32, device=device))


def alloc_partition_trace(p: Params, device):
    import torch
    BH, N, d, T = p.BH, p.N, p.d, p.kmeans_iters
    f32 = dict(dtype=torch.float32, device=device)
    i32 = dict(dtype=torch.int32, device=device)
    return dict(sample_idx=torch.empty(BH, p.n_samples, **i32), metric=torch.empty(BH, d, d, **f32),
                eigval=torch.empty(BH, p.eig_rank, **f32), eigvec=torch.empty(BH, d, p.eig_rank, **f32),
                key_coords=torch.empty(BH, N, p.eig_rank, **f32), key_init=torch.empty(BH, p.n_kgroups, **i32),
                key_label_iters=torch.empty(T, BH, N, **i32), key_centroids=torch.empty(BH, p.n_kgroups, d, **f32),
                query_coords=torch.empty(BH, N, p.n_kgroups, **f32), query_init=torch.empty(BH, p.n_qgroups, **i32),
                query_label_iters=torch.empty(T, BH, N, **i32),
                cell_mass=torch.empty(BH, p.n_qgroups, p.n_kgroups, **f32),
                alpha=torch.empty(BH, dtype=torch.float64, device=device))


def alloc_probe(p: Params, device, with_bmat: bool = False):
    import torch
    BH, d, P, r = p.BH, p.d, p.n_probes, p.sub_rank
    f32 = dict(dtype=torch.float32, device=device)
    return dict(probe_idx=torch.empty(BH, P, dtype=torch.int32, device=device),
                probe_o_dense=torch.empty(BH, P, d, **f32), b_full=torch.empty(BH, d, **f32),
                Vr=torch.empty(BH, d, r, **f32), W=torch.empty(BH, d, r, **f32),
                Bmat=torch.empty(BH, d, d, **f32) if with_bmat else None)


def alloc_probe_trace(p: Params, device):
    import torch
    BH, d, P, r = p.BH, p.d, p.n_probes, p.sub_rank
    f32 = dict(dtype=torch.float32, device=device)
    return dict(probe_o_sparse=torch.empty(BH, P, d, **f32), probe_lse_dense=torch.empty(BH, P, **f32),
                probe_lse_sparse=torch.empty(BH, P, **f32), sigma=torch.empty(BH, r, **f32),
                b_sub=torch.empty(BH, r, **f32))


def run_call(p: Params, Q, K, V, ws=None, trace=False):
    """The four calls in order on the current stream; returns every output."""
    import torch
    dev = Q.device
    ws = workspace(p, dev) if ws is None else ws
    part = alloc_partition(p, dev)
    ptr = alloc_partition_trace(p, dev) if trace else None
    sparsepr_partition(p, Q, K, part["perm_q"], part["perm_k"], part["label_q"], part["label_k"], part["qoff"],
                       part["koff"], part["route"], part["block_mask"], part["rho_exec"], ws, ptr)
    o_sparse = torch.empty_like(Q)
    lse = torch.empty(p.BH, p.N, dtype=torch.float32, device=dev)
    sparsepr_attend(p, Q, K, V, part["perm_q"], part["perm_k"], part["qoff"], part["koff"], part["route"],
                    o_sparse, lse, ws)
    pr = alloc_probe(p, dev, with_bmat=trace)
    prt = alloc_probe_trace(p, dev) if trace else None
    sparsepr_probe_fit(p, Q, K, V, part["label_k"], part["perm_q"], part["qoff"], part["route"],
                       pr["probe_idx"], pr["probe_o_dense"], pr["b_full"], pr["Vr"], pr["W"], pr["Bmat"], ws, prt)
    o = torch.empty_like(Q)
    sparsepr_reconstruct(p, o_sparse, pr["probe_idx"], pr["probe_o_dense"], pr["b_full"], pr["Vr"], pr["W"], o)
    out = dict(part, o_sparse=o_sparse, lse=lse, o=o, ws=ws, **pr)
    if trace:
        out["trace"] = ptr
        out["probe_trace"] = prt
    return out


# ---------------------------------------------------------------------------
# Rotary positions and the paged K/V cache
# ---------------------------------------------------------------------------
# Tensors may be strided views (the last dimension contiguous): their strides go into a copy
# of the params, so one params object serves calls with different layouts.  Shapes, types and
# devices are checked here, because the library sees pointers only.  A step of a rollout makes
# several of these calls, each shorter on the GPU than a few microseconds of Python, so the
# checks compare first and build their messages only when something is wrong.
_tc = None          # torch, and its types by code, from the first call on


class _Torch:
    def __init__(self):
        import torch
        self.mod = torch
        self.elem = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32}
        self.i32, self.u8, self.f64, self.f32 = torch.int32, torch.uint8, torch.float64, torch.float32


def _torch():
    global _tc
    if _tc is None:
        _tc = _Torch()
    return _tc


def _refuse(check, name, t, shape, dtype, dev):
    """Raises for a tensor that differs from what the params say (invalid params first)."""
    _check(*check)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected device {dev}")
    raise ValueError(f"{name} must be contiguous")


def _pointers(validate, p, dev, specs):
    """Addresses of contiguous tensors (name, tensor, shape, dtype) on device dev."""
    out = []
    for name, t, shape, dt in specs:
        if t.shape != shape or t.dtype is not dt or t.get_device() != dev or not t.is_contiguous():
            _refuse((validate(p), name), name, t, shape, dt, dev)
        out.append(t.data_ptr())
    return out


def _views(validate, p, dev, first, specs):
    """Addresses of tensors (name, tensor, shape, dtype, stride field) that may be strided views, and
    the params with their strides: p itself when all are contiguous (the stride fields begin at
    byte `first` and are 0 in params from make())."""
    out, plain = [], ctypes.string_at(ctypes.addressof(p) + first, ctypes.sizeof(p) - first) == _ZEROS[first]
    for name, t, shape, dt, _ in specs:
        if t.shape != shape or t.dtype is not dt or t.get_device() != dev:
            _refuse((validate(p), name), name, t, shape, dt, dev)
        if plain and not t.is_contiguous():
            plain = False
        out.append(t.data_ptr())
    if plain:
        return p, out
    q = type(p).from_buffer_copy(p)
    for name, t, _, _, field in specs:
        st = getattr(q, field)
        for i in range(len(st)):
            st[i] = 0
        if t.is_contiguous():
            continue
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        for i in range(len(st)):
            # a dimension of one element has no stride of its own: take a contiguous one
            st[i] = t.stride(i) if t.shape[i] > 1 else _packed(t, i)
        if t.numel() and not any(st):     # all zero would mean contiguous to the library
            raise ValueError(f"{name}: one row expanded over every dimension is not supported")
    return q, out


_ZEROS = {RopeParams.x_stride.offset: bytes(ctypes.sizeof(RopeParams) - RopeParams.x_stride.offset),
          CacheParams.q_stride.offset: bytes(ctypes.sizeof(CacheParams) - CacheParams.q_stride.offset)}


def _packed(t, d):
    n = 1
    for i in range(d + 1, t.dim()):
        n *= max(1, t.shape[i])
    return n


def _elem(p):
    dt = _torch().elem.get(p.dtype)
    if dt is None:
        raise ValueError(f"unknown dtype code {p.dtype}")
    return dt


def _launch(fn, validate, p, name, dev, *args):
    """fn(p, *args, stream) on device dev and its current stream."""
    if dev < 0:
        _check(validate(p), name)
        raise ValueError("tensors must be on a CUDA device")
    torch = _tc.mod
    stream = torch._C._cuda_getCurrentRawStream(dev)     # current_stream(dev).cuda_stream, without the object
    if torch.cuda.current_device() == dev:
        status = fn(p, *args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(p, *args, stream)
    if status != 0:
        raise SparsePRError(status, name)


def sparsepr_rope_validate(p: RopeParams) -> int:
    return _lib.sparsepr_rope_validate(ctypes.byref(p))


def sparsepr_cache_validate(p: CacheParams) -> int:
    return _lib.sparsepr_cache_validate(ctypes.byref(p))


def sparsepr_rope_frequencies(p: RopeParams):
    """Turns per position of every pair (float64 CPU tensor [rot_dim / 2])."""
    import torch
    n = max(0, p.rot_dim // 2)
    buf = (ctypes.c_double * max(1, n))()
    _check(_lib.sparsepr_rope_frequencies(ctypes.byref(p), buf), "sparsepr_rope_frequencies")
    return torch.tensor(list(buf)[:n], dtype=torch.float64)


def rope_frequencies(p: RopeParams, device):
    """sparsepr_rope_frequencies on a device, as the calls take them; keep it with the params."""
    return sparsepr_rope_frequencies(p).to(device)


def _rope(fn, name, p, x, pos, freq, y, x2, y2):
    H2 = p.H2
    if (H2 > 0) != (x2 is not None) or (x2 is None) != (y2 is None):
        raise ValueError("the second tensor goes with H2 > 0")
    check = _lib.sparsepr_rope_validate
    dev, el, B, N, d = x.get_device(), _elem(p), p.B, p.N, p.d
    shape = (B, p.H, N, d)
    specs = [("x", x, shape, el, "x_stride"), ("y", y, shape, el, "y_stride")]
    if x2 is not None:
        shape = (B, H2, N, d)
        specs += [("x2", x2, shape, el, "x2_stride"), ("y2", y2, shape, el, "y2_stride")]
    q, v = _views(check, p, dev, RopeParams.x_stride.offset, specs)
    ps, fr = _pointers(check, p, dev, (("pos", pos, (p.n_axes, B, N) if p.pos_batched else (p.n_axes, N), _tc.i32),
                                       ("freq", freq, (p.rot_dim // 2,), _tc.f64)))
    _launch(fn, check, q, name, dev, v[0], ps, fr, v[1], *(v[2:] or (None, None)))


def sparsepr_rope(p: RopeParams, x, pos, freq, y, x2=None, y2=None):
    """Rotates x [B, H, N, d] into y (and x2 [B, H2, N, d] into y2); strided views are allowed,
    and y may be x.  pos int32 [n_axes, N] or, with pos_batched, [n_axes, B, N]."""
    _rope(_lib.sparsepr_rope, "sparsepr_rope", p, x, pos, freq, y, x2, y2)


def sparsepr_rope_backward(p: RopeParams, dy, pos, freq, dx, dy2=None, dx2=None):
    """Gradient of sparsepr_rope: dx from dy (and dx2 from dy2)."""
    _rope(_lib.sparsepr_rope_backward, "sparsepr_rope_backward", p, dy, pos, freq, dx, dy2, dx2)


def sparsepr_paged_workspace_bytes(p: CacheParams) -> int:
    return _lib.sparsepr_paged_workspace_bytes(ctypes.byref(p))


def paged_workspace(p: CacheParams, device):
    """A workspace for the paged calls, its error word cleared.  Concurrent calls need one each."""
    import torch
    n = sparsepr_paged_workspace_bytes(p)
    if n == 0:
        _check(sparsepr_cache_validate(p), "workspace size")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def sparsepr_paged_error(ws) -> int:
    torch = _torch().mod
    with torch.cuda.device(ws.device):
        return _lib.sparsepr_paged_error(_ptr(ws), _stream(ws))


def sparsepr_paged_clear_error(ws):
    with _torch().mod.cuda.device(ws.device):
        _check(_lib.sparsepr_paged_clear_error(_ptr(ws), _stream(ws)), "sparsepr_paged_clear_error")


def sparsepr_select_units(p: CacheParams) -> int:
    """Most selection units of a call with these params (rows of sel and sel_count)."""
    n = _lib.sparsepr_select_units(ctypes.byref(p))
    if n < 0:
        _check(sparsepr_cache_validate(p), "sparsepr_select_units")
        raise ValueError("sparsepr_select_units needs n_select >= 1")
    return n


def alloc_selection(p: CacheParams, device):
    """sel [units, Hkv, n_select] and sel_count [units, Hkv] for sparsepr_page_select."""
    import torch
    u = sparsepr_select_units(p)
    return (torch.empty(u, p.Hkv, p.n_select, dtype=torch.int32, device=device),
            torch.empty(u, p.Hkv, dtype=torch.int32, device=device))


def alloc_cache(p: CacheParams, device):
    """k_pages, v_pages [n_pages, Hkv, page, d] and k_mean [n_pages, Hkv, d]."""
    import torch
    dt = torch.float16 if p.dtype == FP16 else torch.bfloat16
    shape = (p.n_pages, p.Hkv, p.page, p.d)
    return dict(k_pages=torch.empty(shape, dtype=dt, device=device),
                v_pages=torch.empty(shape, dtype=dt, device=device),
                k_mean=torch.empty(p.n_pages, p.Hkv, p.d, dtype=dt, device=device))


def _sequences(p, q_start, kv_len, page_table):
    i32, B = _tc.i32, p.B
    return [("q_start", q_start, (B + 1,), i32), ("kv_len", kv_len, (B,), i32),
            ("page_table", page_table, (B, p.max_pages), i32)]


def _lists(p, sel, sel_count):
    n = _lib.sparsepr_select_units(p)
    if n < 0:
        sparsepr_select_units(p)     # raises
    return [("sel", sel, (n, p.Hkv, p.n_select), _tc.i32), ("sel_count", sel_count, (n, p.Hkv), _tc.i32)]


def sparsepr_cache_append(p: CacheParams, K, V, q_start, kv_len, page_table, k_pages, v_pages, k_mean, ws, rope=None,
                          pos=None, freq=None):
    """Writes the new rows K, V [T, Hkv, d] into their page slots and the touched pages' mean
    keys; with rope (RopeParams) the keys are rotated by pos int32 [n_axes, T] on the way."""
    check = _lib.sparsepr_cache_validate
    dev, el, T, Hkv, d = K.get_device(), _elem(p), p.T, p.Hkv, p.d
    rows, pages = (T, Hkv, d), (p.n_pages, Hkv, p.page, d)
    q, (kp, vp) = _views(check, p, dev, CacheParams.q_stride.offset, (("K", K, rows, el, "k_stride"),
                                                                     ("V", V, rows, el, "v_stride")))
    specs = _sequences(p, q_start, kv_len, page_table)
    specs += [("k_pages", k_pages, pages, el), ("v_pages", v_pages, pages, el),
              ("k_mean", k_mean, (p.n_pages, Hkv, d), el), ("ws", ws, (ws.numel(),), _tc.u8)]
    if rope is not None:
        if pos is None or freq is None:
            raise ValueError("rope needs pos and freq")
        specs += [("pos", pos, (rope.n_axes, T), _tc.i32), ("freq", freq, (rope.rot_dim // 2,), _tc.f64)]
    t = _pointers(check, p, dev, specs)
    ps, fr = t[7:] or (None, None)
    _launch(_lib.sparsepr_cache_append, check, q, "sparsepr_cache_append", dev, kp, vp, *t[:6], rope, ps, fr, t[6],
            ws.numel())


def sparsepr_page_select(p: CacheParams, Q, q_start, kv_len, page_table, k_mean, sel, sel_count, ws):
    """Page lists of every unit of q_block tokens and key/value head, by mean query . mean key."""
    check = _lib.sparsepr_cache_validate
    dev, el = Q.get_device(), _elem(p)
    q, (qp,) = _views(check, p, dev, CacheParams.q_stride.offset, (("Q", Q, (p.T, p.Hq, p.d), el, "q_stride"),))
    t = _pointers(check, p, dev, _sequences(p, q_start, kv_len, page_table) +
                  [("k_mean", k_mean, (p.n_pages, p.Hkv, p.d), el)] + _lists(p, sel, sel_count) +
                  [("ws", ws, (ws.numel(),), _tc.u8)])
    _launch(_lib.sparsepr_page_select, check, q, "sparsepr_page_select", dev, qp, *t, ws.numel())


def sparsepr_paged_attention(p: CacheParams, Q, q_start, kv_len, page_table, k_pages, v_pages, O, lse, ws, sel=None,
                             sel_count=None):
    """Attention of the new tokens Q [T, Hq, d] over the cache into O (and lse float32 [T, Hq] or
    None); with sel and sel_count over the pages of their lists."""
    if (sel is None) != (sel_count is None):
        raise ValueError("sel and sel_count come together")
    check = _lib.sparsepr_cache_validate
    dev, el, T, Hq, d = Q.get_device(), _elem(p), p.T, p.Hq, p.d
    rows, pages = (T, Hq, d), (p.n_pages, p.Hkv, p.page, d)
    q, (qp, op) = _views(check, p, dev, CacheParams.q_stride.offset, (("Q", Q, rows, el, "q_stride"),
                                                                     ("O", O, rows, el, "o_stride")))
    specs = _sequences(p, q_start, kv_len, page_table)
    specs += [("k_pages", k_pages, pages, el), ("v_pages", v_pages, pages, el), ("ws", ws, (ws.numel(),), _tc.u8)]
    if lse is not None:
        specs.append(("lse", lse, (T, Hq), _tc.f32))
    if sel is not None:
        specs += _lists(p, sel, sel_count)
    t = _pointers(check, p, dev, specs)
    z = t.pop(6) if lse is not None else None
    sp, cp = t[6:] or (None, None)
    _launch(_lib.sparsepr_paged_attention, check, q, "sparsepr_paged_attention", dev, qp, *t[:5], sp, cp, op, z, t[5],
            ws.numel())


def rollout_step(p: CacheParams, cache, Q, K, V, q_start, kv_len, page_table, O, ws, rope=None, pos=None, freq=None,
                 selection=None, lse=None):
    """One step of a rollout on the current stream: K and V (rotated with rope) are appended to
    cache (alloc_cache), then Q attends to it, through the page lists of selection
    (alloc_selection) when given.  Q is rotated by the caller (sparsepr_rope)."""
    sparsepr_cache_append(p, K, V, q_start, kv_len, page_table, cache["k_pages"], cache["v_pages"], cache["k_mean"],
                          ws, rope=rope, pos=pos, freq=freq)
    sel = cnt = None
    if selection is not None:
        sel, cnt = selection
        sparsepr_page_select(p, Q, q_start, kv_len, page_table, cache["k_mean"], sel, cnt, ws)
    sparsepr_paged_attention(p, Q, q_start, kv_len, page_table, cache["k_pages"], cache["v_pages"], O, lse, ws, sel=sel,
                             sel_count=cnt)
    return O
