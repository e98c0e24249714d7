"""Thin ctypes binding of include/ddtree.h: argument marshalling only.

Every step of the computation runs in the CUDA library (lib/libddtree.so).
PyTorch only provides device memory and the current stream.  If the library is
missing this module raises at import-time use; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libddtree.so")

D_QK = 576
D_V = 512
KV8_ROW = 640

DDT_OK = 0
ERRORS = {-1: "DDT_ERR_NULL", -2: "DDT_ERR_DIMS", -3: "DDT_ERR_WORKSPACE", -4: "DDT_ERR_ALIGN",
          -5: "DDT_ERR_LAUNCH", -6: "DDT_ERR_DEVICE", -7: "DDT_ERR_ALIAS"}
STATUS_BAD_SLOT = 1
STATUS_BAD_PARENT = 2
STATUS_BAD_PREFIX = 4
STATUS_TIMEOUT = 8
STATUS_BAD_TREE_LEN = 16
STATUS_BAD_NODE = 32
STATUS_BAD_BLOCK = 64
STATUS_BAD_POSITION = 128
STATUS_BAD_TOKEN = 256
STATUS_BAD_LOGITS = 512

EXPORTS = ("ddtree_verify_workspace_bytes", "ddtree_verify_attn", "ddtree_verify_attn_fused",
           "ddtree_verify_attn_ragged",
           "ddtree_verify_prefix_phase",
           "ddtree_verify_merge_phase", "ddtree_verify_attn_static_scratch", "ddtree_kv_compact",
           "ddtree_kv_compact_check", "ddtree_verify_sparse_workspace_bytes", "ddtree_verify_attn_sparse",
           "ddtree_kv_weight_workspace_bytes", "ddtree_kv_weight", "ddtree_kv_evict", "ddtree_block_summary",
           "ddtree_block_select_workspace_bytes", "ddtree_block_select",
           "ddtree_verify_blocks_workspace_bytes", "ddtree_verify_attn_blocks",
           "ddtree_kv8_write", "ddtree_kv8_read", "ddtree_verify_kv8_workspace_bytes", "ddtree_verify_attn_kv8",
           "ddtree_accept_workspace_bytes", "ddtree_accept",
           "ddtree_read_device_status", "ddtree_status_string")


class DDTError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({status_string(code)})")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_nodes", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("slot_stride", ctypes.c_int32), ("pool_slots", ctypes.c_int64),
                ("max_prefix_len", ctypes.c_int32), ("prefix_len_sum", ctypes.c_int32)]


_lib = None


def load(path: str):
    """Load a build of the library from `path` and declare its C signatures.

    lib() loads the product build; tests also load the test-hooks build this way.
    """
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing (run __graft_entry__.build())")
    L = ctypes.CDLL(path)
    vp, i32p = ctypes.c_void_p, ctypes.c_void_p
    L.ddtree_verify_workspace_bytes.restype = ctypes.c_size_t
    L.ddtree_verify_workspace_bytes.argtypes = [ctypes.POINTER(Dims)]
    for fn in ("ddtree_verify_attn", "ddtree_verify_attn_fused", "ddtree_verify_prefix_phase",
               "ddtree_verify_merge_phase"):
        if not hasattr(L, fn):   # builds that predate an entry point
            continue
        f = getattr(L, fn)
        f.restype = ctypes.c_int
        f.argtypes = [vp, vp, i32p, i32p, i32p, i32p, ctypes.c_float, vp, vp, ctypes.POINTER(Dims), vp,
                      ctypes.c_size_t, vp]
    L.ddtree_verify_attn_ragged.restype = ctypes.c_int
    L.ddtree_verify_attn_ragged.argtypes = [vp, vp, i32p, i32p, i32p, i32p, i32p, ctypes.c_float, vp, vp,
                                            ctypes.POINTER(Dims), vp, ctypes.c_size_t, vp]
    L.ddtree_verify_attn_static_scratch.restype = ctypes.c_int
    L.ddtree_verify_attn_static_scratch.argtypes = [vp, vp, i32p, i32p, i32p, i32p, ctypes.c_float, vp, vp,
                                                    ctypes.POINTER(Dims), vp]
    L.ddtree_kv_compact.restype = ctypes.c_int
    L.ddtree_kv_compact.argtypes = [vp, vp, i32p, i32p, vp, i32p, ctypes.POINTER(Dims), vp, vp]
    if hasattr(L, "ddtree_kv_compact_check"):   # absent from builds that predate the validator
        L.ddtree_kv_compact_check.restype = ctypes.c_int
        L.ddtree_kv_compact_check.argtypes = [vp, vp, vp, vp, ctypes.POINTER(Dims), ctypes.c_int32,
                                              ctypes.POINTER(ctypes.c_int64)]
    if hasattr(L, "ddtree_verify_attn_sparse"):
        L.ddtree_verify_sparse_workspace_bytes.restype = ctypes.c_size_t
        L.ddtree_verify_sparse_workspace_bytes.argtypes = [ctypes.POINTER(Dims)]
        L.ddtree_verify_attn_sparse.restype = ctypes.c_int
        L.ddtree_verify_attn_sparse.argtypes = [vp, vp, i32p, ctypes.c_float, vp, vp, ctypes.POINTER(Dims), vp,
                                                ctypes.c_size_t, vp]
    if hasattr(L, "ddtree_kv_weight"):
        i32, f32, size, dims = ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(Dims)
        L.ddtree_kv_weight_workspace_bytes.restype = size
        L.ddtree_kv_weight_workspace_bytes.argtypes = [dims, i32]
        L.ddtree_kv_weight.restype = ctypes.c_int
        L.ddtree_kv_weight.argtypes = [vp, vp, i32p, i32p, vp, i32p, i32, f32, f32, vp, vp, dims, vp, size, vp]
        L.ddtree_kv_evict.restype = ctypes.c_int
        L.ddtree_kv_evict.argtypes = [vp, i32p, i32p, i32p, i32, i32, i32p, vp, i32p, i32p, dims, vp, vp]
        L.ddtree_block_summary.restype = ctypes.c_int
        L.ddtree_block_summary.argtypes = [vp, i32p, i32p, i32p, i32, vp, vp, dims, vp, vp]
        L.ddtree_block_select_workspace_bytes.restype = size
        L.ddtree_block_select_workspace_bytes.argtypes = [dims, i32]
        L.ddtree_block_select.restype = ctypes.c_int
        L.ddtree_block_select.argtypes = [vp, vp, vp, i32p, i32, i32, i32, i32, i32p, dims, vp, size, vp]
        L.ddtree_verify_blocks_workspace_bytes.restype = size
        L.ddtree_verify_blocks_workspace_bytes.argtypes = [dims, i32, i32]
        L.ddtree_verify_attn_blocks.restype = ctypes.c_int
        L.ddtree_verify_attn_blocks.argtypes = [vp, vp, i32p, i32p, i32p, i32p, i32p, i32, i32, f32, vp, vp, dims, vp,
                                                size, vp]
    if hasattr(L, "ddtree_kv8_write"):
        i32, i64, f32, size, dims = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(Dims)
        L.ddtree_kv8_write.restype = ctypes.c_int
        L.ddtree_kv8_write.argtypes = [vp, i64, i32p, i64, vp, f32, vp, i32p, i32, i32, vp, vp, i64, vp, vp]
        L.ddtree_kv8_read.restype = ctypes.c_int
        L.ddtree_kv8_read.argtypes = [vp, vp, i32p, i64, vp, i64, i64, vp, vp]
        L.ddtree_verify_kv8_workspace_bytes.restype = size
        L.ddtree_verify_kv8_workspace_bytes.argtypes = [dims]
        L.ddtree_verify_attn_kv8.restype = ctypes.c_int
        L.ddtree_verify_attn_kv8.argtypes = [vp, vp, vp, i32p, i32p, i32p, i32p, i32p, f32, vp, vp, dims, vp, size, vp]
        L.ddtree_accept_workspace_bytes.restype = size
        L.ddtree_accept_workspace_bytes.argtypes = [dims, i32]
        L.ddtree_accept.restype = ctypes.c_int
        L.ddtree_accept.argtypes = [vp, i32, i64, i32, vp, i64, i32p, i32p, i32p, vp, vp, i32p, i32p, i32p, dims, vp, size,
                                    vp]
    if hasattr(L, "ddtree_internal_plan"):
        L.ddtree_internal_plan.restype = ctypes.c_int
        L.ddtree_internal_plan.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, ctypes.POINTER(ctypes.c_int32)]
    L.ddtree_read_device_status.restype = ctypes.c_int
    L.ddtree_read_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), vp]
    L.ddtree_status_string.restype = ctypes.c_char_p
    L.ddtree_status_string.argtypes = [ctypes.c_int]
    return L


def lib():
    """Load lib/libddtree.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def status_string(code: int) -> str:
    return lib().ddtree_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_dims(batch, nodes, heads, pool_slots, slot_stride, max_prefix_len, prefix_len_sum=0) -> Dims:
    """prefix_len_sum: optional host-side sum of the prefix lengths (0: unknown); it only steers the split."""
    return Dims(int(batch), int(nodes), int(heads), int(slot_stride), int(pool_slots), int(max_prefix_len),
                int(prefix_len_sum))


def workspace_bytes(dims: Dims) -> int:
    return int(lib().ddtree_verify_workspace_bytes(ctypes.byref(dims)))


def plan(dims: Dims, sm_count: int | None = None, library=None) -> dict:
    """The schedule the library picks for these sizes: row tiles, key splits (keys of split 0 and of
    each later split), or key-range groups (groups > 0).  sm_count: the device's SM count (default: the current device's)."""
    if sm_count is None:
        import torch
        sm_count = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    out = (ctypes.c_int32 * 5)()
    _check((library or lib()).ddtree_internal_plan(ctypes.byref(dims), int(sm_count), out), "ddtree_internal_plan")
    return dict(row_tiles=out[0], splits=out[1], chunk0=out[4], chunk=out[2], groups=out[3])


def _check(rc, what):
    if rc != DDT_OK:
        raise DDTError(rc, what)


def _keep(stream, *tensors):
    """Tell the allocator that `stream` uses tensors which may have been allocated for the current one."""
    if stream is not None:
        for t in tensors:
            t.record_stream(stream)


def _make(stream, fn, *args, **kw):
    """A tensor that a call makes for itself: allocated, and filled, on the stream that the call runs on.

    On the current stream its fill could run after the kernels on `stream`, and its memory could still be in use there.
    """
    import torch
    if stream is None:
        return fn(*args, **kw)
    with torch.cuda.stream(stream):
        t = fn(*args, **kw)
    t.record_stream(torch.cuda.current_stream(t.device))   # where the caller is likely to use it
    return t


class Verifier:
    """Holds a workspace sized for one set of dims and runs verify calls with it.

    q [B,T,H,576] bf16, kv_pool [N,576] bf16, slot_idx [B,stride] int32, prefix_len [B] int32,
    tree_parent [B,T] int32, tree_slot_idx [B,T] int32 -- all CUDA tensors.
    """

    def __init__(self, batch, nodes, heads, pool_slots, slot_stride, max_prefix_len=None, device=None,
                 prefix_len_sum=0, library=None):
        import torch
        self.lib = lib() if library is None else library
        self.dims = make_dims(batch, nodes, heads, pool_slots, slot_stride,
                              slot_stride if max_prefix_len is None else max_prefix_len, prefix_len_sum)
        self.device = torch.device("cuda") if device is None else torch.device(device)
        with torch.cuda.device(self.device):
            n = int(self.lib.ddtree_verify_workspace_bytes(ctypes.byref(self.dims)))
            if n == 0:
                raise DDTError(-2, "ddtree_verify_workspace_bytes")
            self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, q, kv_pool, slot_idx, prefix_len, tree_parent, tree_slot_idx, sm_scale, out=None,
                 lse=None, stream=None, phase="all", tree_len=None):
        """phase: "all" (ddtree_verify_attn), "fused" (ddtree_verify_attn_fused: always one launch),
        "prefix" or "merge" (the two-launch path's halves).

        tree_len: optional int32 [B] CUDA tensor of active nodes per request
        (ddtree_verify_attn_ragged; phase must be "all").
        """
        import torch
        B, T, H, D = q.shape
        if out is None:
            out = _make(stream, torch.empty, (B, T, H, D_V), dtype=torch.float32, device=q.device)
        if lse is None:
            lse = _make(stream, torch.empty, (B, T, H), dtype=torch.float32, device=q.device)
        if tree_len is not None:
            if phase != "all":
                raise ValueError("ragged trees run as one call (phase='all')")
            rc = self.lib.ddtree_verify_attn_ragged(_ptr(q), _ptr(kv_pool), _ptr(slot_idx), _ptr(prefix_len),
                                                 _ptr(tree_parent), _ptr(tree_slot_idx), _ptr(tree_len),
                                                 float(sm_scale), _ptr(out), _ptr(lse), ctypes.byref(self.dims),
                                                 _ptr(self.workspace), self.workspace.numel(), _stream(stream))
            _check(rc, "ddtree_verify_attn_ragged")
            _keep(stream, out, lse, self.workspace)
            return out, lse
        fn = {"all": "ddtree_verify_attn", "fused": "ddtree_verify_attn_fused", "prefix": "ddtree_verify_prefix_phase",
              "merge": "ddtree_verify_merge_phase"}[phase]
        rc = getattr(self.lib, fn)(_ptr(q), _ptr(kv_pool), _ptr(slot_idx), _ptr(prefix_len), _ptr(tree_parent),
                                _ptr(tree_slot_idx), float(sm_scale), _ptr(out), _ptr(lse),
                                ctypes.byref(self.dims), _ptr(self.workspace), self.workspace.numel(),
                                _stream(stream))
        _check(rc, fn)
        _keep(stream, out, lse, self.workspace)
        return out, lse

    def status(self, stream=None) -> int:
        return read_device_status(self.workspace, stream, library=self.lib)


def verify_attn(q, kv_pool, slot_idx, prefix_len, tree_parent, tree_slot_idx, sm_scale, max_prefix_len=None,
                out=None, lse=None, stream=None):
    """One-off verify call (allocates its own workspace); returns (out, lse)."""
    import torch
    B, T, H, _ = q.shape
    with torch.cuda.stream(stream):   # (None: the current one) the workspace is that stream's too
        v = Verifier(B, T, H, kv_pool.shape[0], slot_idx.shape[1], max_prefix_len, device=q.device)
    return v(q, kv_pool, slot_idx, prefix_len, tree_parent, tree_slot_idx, sm_scale, out, lse, stream)


class SparseVerifier:
    """Sparse-index verify attention: node (b, t) attends to the pool rows its index list names.

    indices [B, T, topk] int32 CUDA tensor (-1 = no key); q [B, T, H, 576] bf16; a workspace is
    held for one set of sizes.
    """

    def __init__(self, batch, nodes, heads, pool_slots, topk, device=None, library=None):
        import torch
        self.lib = lib() if library is None else library
        self.dims = make_dims(batch, nodes, heads, pool_slots, topk, topk)
        self.device = torch.device("cuda") if device is None else torch.device(device)
        with torch.cuda.device(self.device):
            n = int(self.lib.ddtree_verify_sparse_workspace_bytes(ctypes.byref(self.dims)))
            if n == 0:
                raise DDTError(-2, "ddtree_verify_sparse_workspace_bytes")
            self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, q, kv_pool, indices, sm_scale, out=None, lse=None, stream=None):
        import torch
        B, T, H, _ = q.shape
        if out is None:
            out = _make(stream, torch.empty, (B, T, H, D_V), dtype=torch.float32, device=q.device)
        if lse is None:
            lse = _make(stream, torch.empty, (B, T, H), dtype=torch.float32, device=q.device)
        rc = self.lib.ddtree_verify_attn_sparse(_ptr(q), _ptr(kv_pool), _ptr(indices), float(sm_scale), _ptr(out),
                                                _ptr(lse), ctypes.byref(self.dims), _ptr(self.workspace),
                                                self.workspace.numel(), _stream(stream))
        _check(rc, "ddtree_verify_attn_sparse")
        _keep(stream, out, lse, self.workspace)
        return out, lse

    def status(self, stream=None) -> int:
        return read_device_status(self.workspace, stream, library=self.lib)


def _need(device, *checks):
    """Check tensors given as (name, tensor, dtype, shape): type, shape, contiguity and device."""
    index = device.index
    for name, t, dtype, shape in checks:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}"
                             + ("" if t.is_contiguous() else " (not contiguous)"))


def _result(stream, device, name, t, dtype, shape):
    """A caller's tensor for a result, checked, or one made for it."""
    import torch
    if t is None:
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=device)
        return _make(stream, torch.empty, shape, dtype=dtype, device=device)
    _need(device, (name, t, dtype, shape))
    return t


def _run_on(device, fn, name, *args):
    """Call the library with `device` current (it works on the current device); raises DDTError."""
    import torch
    if torch.cuda.current_device() == device.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc != DDT_OK:
        raise DDTError(rc, name)


def _run_at(device, fn, name, *args):
    """_run_on for tensors that are on `device`, so CUDA is set up: short calls feel a look at the current device."""
    import torch
    if torch._C._cuda_getDevice() != device.index:
        return _run_on(device, fn, name, *args)
    rc = fn(*args)
    if rc != DDT_OK:
        raise DDTError(rc, name)


def _addr(t):
    """A tensor's address as ctypes takes it (None: NULL); cheaper than a c_void_p a tensor."""
    return None if t is None else t.data_ptr()


def _cuda_device(device):
    import torch
    d = torch.device("cuda") if device is None else torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"a CUDA device is needed, got {d}")
    return d if d.index is not None else torch.device("cuda", torch.cuda.current_device())


def _on_cuda(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    return t.device


def _stream_of(device, stream):
    import torch
    # the raw handle: building a Stream object costs as much as a launch
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


class KeyWeights:
    """Accumulated attention weight of every prefix key (ddtree_kv_weight), with a workspace for one set of sizes.

    Call after a verify call with its q and lse: out[b, j] = decay * weight[b, j] + the softmax weights that the
    chosen nodes' heads gave prefix position j.  node_idx [B, S] int32 (-1 = none) chooses nodes, for example the
    accepted path; without it every node counts.  weight and out are fp32 [B, slot_stride]; out=weight updates in
    place; entries from prefix_len[b] on are not written.  max_sel bounds S (default: the tree's nodes).
    """

    def __init__(self, batch, nodes, heads, pool_slots, slot_stride, max_prefix_len=None, max_sel=None, device=None,
                 library=None):
        import torch
        self.lib = lib() if library is None else library
        self.dims = make_dims(batch, nodes, heads, pool_slots, slot_stride,
                              slot_stride if max_prefix_len is None else max_prefix_len)
        self.max_sel = int(nodes if max_sel is None else max_sel)
        self.device = _cuda_device(device)
        self.dims_ref = ctypes.byref(self.dims)
        with torch.cuda.device(self.device):
            n = max(int(self.lib.ddtree_kv_weight_workspace_bytes(self.dims_ref, k))
                    for k in range(self.max_sel + 1))
        if n == 0:
            raise DDTError(-2, "ddtree_kv_weight_workspace_bytes")
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, q, kv_pool, slot_idx, prefix_len, lse, sm_scale, weight=None, decay=1.0, node_idx=None,
                 out=None, stream=None):
        import torch
        d = self.dims
        table = (d.batch, d.slot_stride)
        if weight is None:
            decay = 0.0
        if out is None:
            out = _make(stream, torch.zeros, table, dtype=torch.float32, device=self.device)
        B, T, H = d.batch, d.num_nodes, d.num_heads
        _need(self.device, ("q", q, torch.bfloat16, (B, T, H, D_QK)),
              ("kv_pool", kv_pool, torch.bfloat16, (d.pool_slots, D_QK)), ("slot_idx", slot_idx, torch.int32, table),
              ("prefix_len", prefix_len, torch.int32, (B,)), ("lse", lse, torch.float32, (B, T, H)),
              ("out", out, torch.float32, table))
        if weight is not None:
            _need(self.device, ("weight", weight, torch.float32, table))
        sel = 0
        if node_idx is not None:
            if node_idx.dim() != 2 or not 1 <= node_idx.shape[1] <= self.max_sel:
                raise ValueError(f"node_idx must be [batch, 1..{self.max_sel}], got {tuple(node_idx.shape)}")
            sel = node_idx.shape[1]
            _need(self.device, ("node_idx", node_idx, torch.int32, (B, sel)))
        _run_on(self.device, self.lib.ddtree_kv_weight, "ddtree_kv_weight", q.data_ptr(), kv_pool.data_ptr(),
                slot_idx.data_ptr(), prefix_len.data_ptr(), lse.data_ptr(), _addr(node_idx), sel, sm_scale, decay,
                _addr(weight), out.data_ptr(), self.dims_ref, self.workspace.data_ptr(), self.workspace.numel(),
                _stream_of(self.device, stream))
        _keep(stream, out, self.workspace)
        return out

    def status(self, stream=None) -> int:
        return read_device_status(self.workspace, stream, library=self.lib)


def kv_evict(weight, slot_idx, prefix_len, keep_len, sink=0, recent=0, slot_idx_out=None, weight_out=None,
             prefix_len_out=None, freed=None, max_prefix_len=None, workspace=None, stream=None):
    """Keep each request's heaviest keep_len[b] positions (ddtree_kv_evict).

    The first `sink` and last `recent` positions stay first, then the larger weight, ties to the lower position.
    Returns (slot_idx_out, weight_out, prefix_len_out, freed): the kept entries in order, and the slots that are
    free now (prefix_len[b] - prefix_len_out[b] of them).  Outputs must be other buffers than the inputs.
    """
    import torch
    device = _on_cuda(weight, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must be [batch, slot_stride]")
    B, stride = weight.shape
    slot_idx_out = _make(stream, torch.zeros_like, slot_idx) if slot_idx_out is None else slot_idx_out
    weight_out = _make(stream, torch.zeros_like, weight) if weight_out is None else weight_out
    prefix_len_out = _make(stream, torch.empty_like, prefix_len) if prefix_len_out is None else prefix_len_out
    freed = _make(stream, torch.zeros_like, slot_idx) if freed is None else freed
    if workspace is None:
        workspace = _make(stream, torch.empty, 256, dtype=torch.uint8, device=device)
    table, lens = (B, stride), (B,)
    _need(device, ("weight", weight, torch.float32, table), ("slot_idx", slot_idx, torch.int32, table),
          ("prefix_len", prefix_len, torch.int32, lens), ("keep_len", keep_len, torch.int32, lens),
          ("slot_idx_out", slot_idx_out, torch.int32, table), ("weight_out", weight_out, torch.float32, table),
          ("prefix_len_out", prefix_len_out, torch.int32, lens), ("freed", freed, torch.int32, table),
          ("workspace", workspace, torch.uint8, workspace.shape))
    if workspace.numel() < 256:
        raise ValueError("workspace must hold 256 bytes")
    dims = make_dims(B, 1, 1, 1, stride, stride if max_prefix_len is None else max_prefix_len)
    _run_on(device, lib().ddtree_kv_evict, "ddtree_kv_evict", weight.data_ptr(), slot_idx.data_ptr(),
            prefix_len.data_ptr(), keep_len.data_ptr(), int(sink), int(recent), slot_idx_out.data_ptr(),
            weight_out.data_ptr(), prefix_len_out.data_ptr(), freed.data_ptr(), ctypes.byref(dims),
            workspace.data_ptr(), _stream_of(device, stream))
    _keep(stream, workspace, slot_idx_out, weight_out, prefix_len_out, freed)
    return slot_idx_out, weight_out, prefix_len_out, freed


def block_summary(kv_pool, slot_idx, prefix_len, block, from_len=None, summary=None, scale=None, max_prefix_len=None,
                  workspace=None, stream=None):
    """8-bit means of each request's blocks of `block` positions (ddtree_block_summary).

    Returns (summary bf16 [B, N, 576] of integers in [-127, 127], scale fp32 [B, N]), N = ceil(max_prefix_len /
    block).  With from_len (int32 [B]) only blocks that hold a position at or after it are computed; pass the
    summary and scale of the step before.
    """
    import torch
    device = _on_cuda(kv_pool, "kv_pool")
    if slot_idx.dim() != 2 or kv_pool.dim() != 2:
        raise ValueError("slot_idx must be [batch, slot_stride] and kv_pool [slots, 576]")
    B, stride = slot_idx.shape
    dims = make_dims(B, 1, 1, kv_pool.shape[0], stride, stride if max_prefix_len is None else max_prefix_len)
    n = -(-dims.max_prefix_len // int(block)) if block > 0 else 0
    if from_len is not None and (summary is None or scale is None):
        raise ValueError("from_len updates the summary and scale of an earlier call: pass both")
    if summary is None:
        summary = _make(stream, torch.zeros, (B, n, D_QK), dtype=torch.bfloat16, device=device)
    if scale is None:
        scale = _make(stream, torch.zeros, (B, n), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = _make(stream, torch.empty, 256, dtype=torch.uint8, device=device)
    _need(device, ("kv_pool", kv_pool, torch.bfloat16, (dims.pool_slots, D_QK)),
          ("slot_idx", slot_idx, torch.int32, (B, stride)), ("prefix_len", prefix_len, torch.int32, (B,)),
          ("summary", summary, torch.bfloat16, (B, n, D_QK)), ("scale", scale, torch.float32, (B, n)),
          ("workspace", workspace, torch.uint8, workspace.shape))
    if from_len is not None:
        _need(device, ("from_len", from_len, torch.int32, (B,)))
    if workspace.numel() < 256:
        raise ValueError("workspace must hold 256 bytes")
    _run_on(device, lib().ddtree_block_summary, "ddtree_block_summary", kv_pool.data_ptr(), slot_idx.data_ptr(),
            prefix_len.data_ptr(), _addr(from_len), int(block), summary.data_ptr(), scale.data_ptr(),
            ctypes.byref(dims), workspace.data_ptr(), _stream_of(device, stream))
    _keep(stream, workspace, summary, scale)
    return summary, scale


class BlockSelector:
    """The best blocks of each tree node by a cheap score (ddtree_block_select), with a workspace for one set of sizes.

    Call with q [B, T, H, 576] bf16 and block_summary's results; returns int32 [B, T, topk], the chosen blocks in
    ascending order, then -1.  The first `first` and last `last` blocks of a prefix are always chosen.
    """

    def __init__(self, batch, nodes, heads, max_prefix_len, block, topk, first=0, last=1, device=None, library=None):
        import torch
        self.lib = lib() if library is None else library
        self.dims = make_dims(batch, nodes, heads, 1, max_prefix_len, max_prefix_len)
        self.block, self.topk, self.first, self.last = int(block), int(topk), int(first), int(last)
        self.device = _cuda_device(device)
        self.dims_ref = ctypes.byref(self.dims)
        n = int(self.lib.ddtree_block_select_workspace_bytes(self.dims_ref, self.block))
        if n == 0:
            raise DDTError(-2, "ddtree_block_select_workspace_bytes")
        self.blocks = -(-int(max_prefix_len) // self.block)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, q, summary, scale, prefix_len, out=None, stream=None):
        import torch
        d = self.dims
        if out is None:
            out = _make(stream, torch.empty, (d.batch, d.num_nodes, self.topk), dtype=torch.int32, device=self.device)
        _need(self.device, ("q", q, torch.bfloat16, (d.batch, d.num_nodes, d.num_heads, D_QK)),
              ("summary", summary, torch.bfloat16, (d.batch, self.blocks, D_QK)),
              ("scale", scale, torch.float32, (d.batch, self.blocks)),
              ("prefix_len", prefix_len, torch.int32, (d.batch,)),
              ("out", out, torch.int32, (d.batch, d.num_nodes, self.topk)))
        _run_on(self.device, self.lib.ddtree_block_select, "ddtree_block_select", q.data_ptr(), summary.data_ptr(),
                scale.data_ptr(), prefix_len.data_ptr(), self.block, self.topk, self.first, self.last, out.data_ptr(),
                self.dims_ref, self.workspace.data_ptr(), self.workspace.numel(), _stream_of(self.device, stream))
        _keep(stream, out, self.workspace)
        return out

    def status(self, stream=None) -> int:
        return read_device_status(self.workspace, stream, library=self.lib)


class BlockVerifier:
    """Verify attention over each node's own blocks (ddtree_verify_attn_blocks), with a workspace for one set of sizes.

    Call with a verify call's tensors and block_idx [B, T, topk] int32 (BlockSelector's, or any list; -1 = none).
    Returns (out bf16 [B, T, H, 512], lse fp32 [B, T, H]).
    """

    def __init__(self, batch, nodes, heads, pool_slots, slot_stride, block, topk, max_prefix_len=None, device=None,
                 library=None):
        import torch
        self.lib = lib() if library is None else library
        self.dims = make_dims(batch, nodes, heads, pool_slots, slot_stride,
                              slot_stride if max_prefix_len is None else max_prefix_len)
        self.block, self.topk = int(block), int(topk)
        self.device = _cuda_device(device)
        self.dims_ref = ctypes.byref(self.dims)
        with torch.cuda.device(self.device):
            n = int(self.lib.ddtree_verify_blocks_workspace_bytes(self.dims_ref, self.block, self.topk))
        if n == 0:
            raise DDTError(-2, "ddtree_verify_blocks_workspace_bytes")
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, q, kv_pool, slot_idx, prefix_len, tree_parent, tree_slot_idx, block_idx, sm_scale, out=None,
                 lse=None, stream=None):
        import torch
        d = self.dims
        B, T, H = d.batch, d.num_nodes, d.num_heads
        if out is None:
            out = _make(stream, torch.empty, (B, T, H, D_V), dtype=torch.bfloat16, device=self.device)
        if lse is None:
            lse = _make(stream, torch.empty, (B, T, H), dtype=torch.float32, device=self.device)
        _need(self.device, ("q", q, torch.bfloat16, (B, T, H, D_QK)),
              ("kv_pool", kv_pool, torch.bfloat16, (d.pool_slots, D_QK)),
              ("slot_idx", slot_idx, torch.int32, (B, d.slot_stride)), ("prefix_len", prefix_len, torch.int32, (B,)),
              ("tree_parent", tree_parent, torch.int32, (B, T)), ("tree_slot_idx", tree_slot_idx, torch.int32, (B, T)),
              ("block_idx", block_idx, torch.int32, (B, T, self.topk)), ("out", out, torch.bfloat16, (B, T, H, D_V)),
              ("lse", lse, torch.float32, (B, T, H)))
        _run_on(self.device, self.lib.ddtree_verify_attn_blocks, "ddtree_verify_attn_blocks", q.data_ptr(),
                kv_pool.data_ptr(), slot_idx.data_ptr(), prefix_len.data_ptr(), tree_parent.data_ptr(),
                tree_slot_idx.data_ptr(), block_idx.data_ptr(), self.block, self.topk, sm_scale, out.data_ptr(),
                lse.data_ptr(), self.dims_ref, self.workspace.data_ptr(), self.workspace.numel(),
                _stream_of(self.device, stream))
        _keep(stream, out, lse, self.workspace)
        return out, lse

    def status(self, stream=None) -> int:
        return read_device_status(self.workspace, stream, library=self.lib)


def kv8_pool(slots, device=None):
    """An empty 8-bit latent cache: (pool uint8 [slots, 640], scale fp32 [slots]), every slot standing for zeros."""
    import torch
    d = _cuda_device(device)
    return torch.zeros(slots, KV8_ROW, dtype=torch.uint8, device=d), torch.ones(slots, dtype=torch.float32, device=d)


def _rows_of(rows, name, device, n):
    """A row stride, in elements, of bf16 rows that may lie in a wider tensor."""
    import torch
    stride = rows.stride()
    if (rows.dtype is not torch.bfloat16 or rows.shape != (n, D_QK) or rows.get_device() != device.index
            or stride[1] != 1 or (n > 1 and stride[0] < D_QK)):
        raise ValueError(f"{name} must be bfloat16 [{n}, {D_QK}] on {device} with consecutive values in a row, got "
                         f"{rows.dtype} {tuple(rows.shape)} on {rows.device}, strides {tuple(stride)}")
    return stride[0] if n > 1 else D_QK


def _kv8_checks(pool, scale, slots, workspace):
    """The device, the cache's slots and the listed ones."""
    import torch
    at, N, n = pool.get_device(), scale.numel(), slots.numel()
    # One condition for what _need checks of three tensors: a short call is bound by these lines.
    if not (at >= 0 and pool.dtype is torch.uint8 and pool.shape == (N, KV8_ROW) and pool.is_contiguous()
            and scale.dtype is torch.float32 and scale.dim() == 1 and scale.get_device() == at and scale.is_contiguous()
            and slots.dtype is torch.int32 and slots.dim() == 1 and slots.get_device() == at and slots.is_contiguous()):
        device = _on_cuda(pool, "pool")
        if pool.dim() != 2 or slots.dim() != 1:
            raise ValueError("pool must be [slots, 640] and slots a list")
        _need(device, ("pool", pool, torch.uint8, (pool.shape[0], KV8_ROW)),
              ("scale", scale, torch.float32, (pool.shape[0],)), ("slots", slots, torch.int32, (n,)))
    device = pool.device
    if workspace is not None:
        _need(device, ("workspace", workspace, torch.uint8, workspace.shape))
        if workspace.numel() < 256:
            raise ValueError("workspace must hold 256 bytes")
    return device, N, n


def kv8_write(rows, slots, pool, scale, norm_weight=None, eps=1e-6, rotation=None, position=None, interleaved=False,
              workspace=None, stream=None):
    """Put bf16 rows [n, 576] into their slots of an 8-bit cache (ddtree_kv8_write); returns (pool, scale).

    slots int32 [n], each slot at most once, -1 = skip the row.  With norm_weight (bf16 [512]) the latent values are
    normalised first, with rotation (fp32 [positions, 64]: cosines, sines) and position (int32 [n]) the rope values
    are rotated: pairs (2 i, 2 i + 1) if interleaved, else (i, i + 32).  rows may be a slice of a wider tensor.
    workspace: 256 bytes for read_device_status; without it bad slots and positions are left out unreported.
    """
    import torch
    device, N, n = _kv8_checks(pool, scale, slots, workspace)
    stride = _rows_of(rows, "rows", device, n)
    if norm_weight is not None:
        _need(device, ("norm_weight", norm_weight, torch.bfloat16, (D_V,)))
    positions = 0
    if (rotation is None) != (position is None):
        raise ValueError("rotation and position go together")
    if rotation is not None:
        if rotation.dim() != 2:
            raise ValueError("rotation must be [positions, 64]")
        positions = rotation.shape[0]
        _need(device, ("rotation", rotation, torch.float32, (positions, 64)), ("position", position, torch.int32, (n,)))
    _run_at(device, lib().ddtree_kv8_write, "ddtree_kv8_write", rows.data_ptr(), stride, slots.data_ptr(), n,
            _addr(norm_weight), eps, _addr(rotation), _addr(position), positions, interleaved, pool.data_ptr(),
            scale.data_ptr(), N, _addr(workspace), _stream_of(device, stream))
    if stream is not None:
        _keep(stream, pool, scale)
    return pool, scale


def kv8_read(pool, scale, slots, out=None, workspace=None, stream=None):
    """The bf16 rows [n, 576] that listed slots of an 8-bit cache stand for (ddtree_kv8_read); -1 gives zeros.

    out may be a slice of a wider tensor; workspace as in kv8_write.
    """
    import torch
    device, N, n = _kv8_checks(pool, scale, slots, workspace)
    if out is None:
        out = _make(stream, torch.empty, (n, D_QK), dtype=torch.bfloat16, device=device)
    stride = _rows_of(out, "out", device, n)
    _run_at(device, lib().ddtree_kv8_read, "ddtree_kv8_read", pool.data_ptr(), scale.data_ptr(), slots.data_ptr(), n,
            out.data_ptr(), stride, N, _addr(workspace), _stream_of(device, stream))
    _keep(stream, out)
    return out


class Kv8Verifier:
    """Verify attention over the 8-bit cache (ddtree_verify_attn_kv8), with a workspace for one set of sizes.

    Call with a verify call's tensors, the cache as (pool, scale) in place of kv_pool; tree_len int32 [B] for trees of
    different sizes.  Returns (out bf16 [B, T, H, 512], lse fp32 [B, T, H]).
    """

    def __init__(self, batch, nodes, heads, pool_slots, slot_stride, max_prefix_len=None, device=None, prefix_len_sum=0,
                 library=None):
        import torch
        self.lib = lib() if library is None else library
        self.dims = make_dims(batch, nodes, heads, pool_slots, slot_stride,
                              slot_stride if max_prefix_len is None else max_prefix_len, prefix_len_sum)
        self.device = _cuda_device(device)
        self.dims_ref = ctypes.byref(self.dims)
        with torch.cuda.device(self.device):
            n = int(self.lib.ddtree_verify_kv8_workspace_bytes(self.dims_ref))
        if n == 0:
            raise DDTError(-2, "ddtree_verify_kv8_workspace_bytes")
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, q, pool, scale, slot_idx, prefix_len, tree_parent, tree_slot_idx, sm_scale, tree_len=None,
                 out=None, lse=None, stream=None):
        import torch
        d = self.dims
        B, T, H = d.batch, d.num_nodes, d.num_heads
        _need(self.device, ("q", q, torch.bfloat16, (B, T, H, D_QK)),
              ("pool", pool, torch.uint8, (d.pool_slots, KV8_ROW)), ("scale", scale, torch.float32, (d.pool_slots,)),
              ("slot_idx", slot_idx, torch.int32, (B, d.slot_stride)), ("prefix_len", prefix_len, torch.int32, (B,)),
              ("tree_parent", tree_parent, torch.int32, (B, T)), ("tree_slot_idx", tree_slot_idx, torch.int32, (B, T)))
        if tree_len is not None:
            _need(self.device, ("tree_len", tree_len, torch.int32, (B,)))
        out = _result(stream, self.device, "out", out, torch.bfloat16, (B, T, H, D_V))
        lse = _result(stream, self.device, "lse", lse, torch.float32, (B, T, H))
        _run_at(self.device, self.lib.ddtree_verify_attn_kv8, "ddtree_verify_attn_kv8", q.data_ptr(), pool.data_ptr(),
                scale.data_ptr(), slot_idx.data_ptr(), prefix_len.data_ptr(), tree_parent.data_ptr(),
                tree_slot_idx.data_ptr(), _addr(tree_len), sm_scale, out.data_ptr(), lse.data_ptr(), self.dims_ref,
                self.workspace.data_ptr(), self.workspace.numel(), _stream_of(self.device, stream))
        _keep(stream, out, lse, self.workspace)
        return out, lse

    def status(self, stream=None) -> int:
        return read_device_status(self.workspace, stream, library=self.lib)


class TreeAcceptor:
    """Which drafted tokens of a tree stand (ddtree_accept), with a workspace for one set of sizes.

    Call with logits [B, T, vocab] (bf16 or fp32; rows may lie in a wider tensor, one stride for all), tokens and
    tree_parent int32 [B, T], uniform fp32 [B, T] in [0, 1) and temperature fp32 [B] (0 = greedy); draft_prob fp32
    [B, T, vocab] where the tokens were drawn from the drafter's distribution, tree_len int32 [B] for trees of
    different sizes.  Returns (path int32 [B, T]: the root and the accepted nodes, then -1; path_len int32 [B];
    next_token int32 [B]).
    """

    def __init__(self, batch, nodes, vocab, device=None, library=None):
        import torch
        self.lib = lib() if library is None else library
        self.dims = make_dims(batch, nodes, 1, 1, 0, 0)
        self.vocab = int(vocab)
        self.device = _cuda_device(device)
        self.dims_ref = ctypes.byref(self.dims)
        n = int(self.lib.ddtree_accept_workspace_bytes(self.dims_ref, self.vocab))
        if n == 0:
            raise DDTError(-2, "ddtree_accept_workspace_bytes")
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def _stride(self, t, name, dtypes):
        """The distance of consecutive nodes' rows, the same over requests."""
        B, T = self.dims.batch, self.dims.num_nodes
        if t.dtype not in dtypes or t.shape != (B, T, self.vocab) or t.get_device() != self.device.index:
            raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))} [{B}, {T}, {self.vocab}] on {self.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        row = t.stride(1) if T > 1 else t.stride(0) if B > 1 else self.vocab
        if ((self.vocab > 1 and t.stride(2) != 1) or (B > 1 and t.stride(0) != T * row)
                or (B * T > 1 and row < self.vocab)):
            raise ValueError(f"{name}'s rows must be consecutive values, at one distance over all nodes: strides "
                             f"{tuple(t.stride())}")
        return row

    def __call__(self, logits, tokens, tree_parent, uniform, temperature, draft_prob=None, tree_len=None, path=None,
                 path_len=None, next_token=None, stream=None):
        import torch
        d = self.dims
        B, T = d.batch, d.num_nodes
        stride = self._stride(logits, "logits", (torch.bfloat16, torch.float32))
        draft_stride = 0 if draft_prob is None else self._stride(draft_prob, "draft_prob", (torch.float32,))
        _need(self.device, ("tokens", tokens, torch.int32, (B, T)), ("tree_parent", tree_parent, torch.int32, (B, T)),
              ("uniform", uniform, torch.float32, (B, T)), ("temperature", temperature, torch.float32, (B,)))
        if tree_len is not None:
            _need(self.device, ("tree_len", tree_len, torch.int32, (B,)))
        path = _result(stream, self.device, "path", path, torch.int32, (B, T))
        path_len = _result(stream, self.device, "path_len", path_len, torch.int32, (B,))
        next_token = _result(stream, self.device, "next_token", next_token, torch.int32, (B,))
        _run_at(self.device, self.lib.ddtree_accept, "ddtree_accept", logits.data_ptr(),
                int(logits.dtype is torch.float32), stride, self.vocab, _addr(draft_prob), draft_stride, tokens.data_ptr(),
                tree_parent.data_ptr(), _addr(tree_len), uniform.data_ptr(), temperature.data_ptr(), path.data_ptr(),
                path_len.data_ptr(), next_token.data_ptr(), self.dims_ref, self.workspace.data_ptr(),
                self.workspace.numel(), _stream_of(self.device, stream))
        _keep(stream, path, path_len, next_token, self.workspace)
        return path, path_len, next_token

    def status(self, stream=None) -> int:
        return read_device_status(self.workspace, stream, library=self.lib)


def verify_attn_static_scratch(q, kv_pool, slot_idx, prefix_len, tree_parent, tree_slot_idx, sm_scale, out,
                               lse, max_prefix_len=None, stream=None):
    """Verify attention with the library's fixed scratch array (no allocation in the call).

    For callers that cannot allocate device memory at call time; out and lse
    are caller-provided.  Calls must not overlap on the GPU (they share the array).
    """
    B, T, H, _ = q.shape
    stride = slot_idx.shape[1]
    dims = make_dims(B, T, H, kv_pool.shape[0], stride, stride if max_prefix_len is None else max_prefix_len)
    rc = lib().ddtree_verify_attn_static_scratch(_ptr(q), _ptr(kv_pool), _ptr(slot_idx), _ptr(prefix_len),
                                                 _ptr(tree_parent), _ptr(tree_slot_idx), float(sm_scale), _ptr(out),
                                                 _ptr(lse), ctypes.byref(dims), _stream(stream))
    _check(rc, "ddtree_verify_attn_static_scratch")
    return out, lse


def kv_compact_check(slot_idx, prefix_len, dst_start, pool_slots, same_pool=True, tree_slot_idx=None,
                     max_prefix_len=None):
    """Host-side check of kv_compact's aliasing contract (numpy arrays or CPU tensors).

    Returns (code, first offending slot or -1); code is DDT_OK or DDT_ERR_ALIAS (-7).
    """
    import numpy as np
    si = np.ascontiguousarray(np.asarray(slot_idx), dtype=np.int32)
    pl = np.ascontiguousarray(np.asarray(prefix_len), dtype=np.int32)
    ds = np.ascontiguousarray(np.asarray(dst_start), dtype=np.int64)
    B, stride = si.shape
    T = 1
    ts = None
    if tree_slot_idx is not None:
        ts = np.ascontiguousarray(np.asarray(tree_slot_idx), dtype=np.int32)
        T = ts.shape[1]
    dims = make_dims(B, T, 1, pool_slots, stride, stride if max_prefix_len is None else max_prefix_len)
    bad = ctypes.c_int64(-1)
    p = lambda a: None if a is None else a.ctypes.data_as(ctypes.c_void_p)
    rc = lib().ddtree_kv_compact_check(p(si), p(pl), p(ds), p(ts), ctypes.byref(dims), int(bool(same_pool)),
                                       ctypes.byref(bad))
    return int(rc), int(bad.value)


def kv_compact(kv_src, kv_dst, slot_idx, prefix_len, dst_start, slot_idx_out=None, max_prefix_len=None,
               workspace=None, stream=None, validate=False, tree_slot_idx=None):
    """Copy each request's prefix rows to dst_start[b] + j; returns slot_idx_out.

    validate=True first runs kv_compact_check on host copies of the tables (a
    debug option: it synchronises with the device) and raises DDTError if the
    aliasing contract is broken.
    """
    import torch
    B, stride = slot_idx.shape
    if validate:
        rc, bad = kv_compact_check(slot_idx.cpu().numpy(), prefix_len.cpu().numpy(), dst_start.cpu().numpy(),
                                   kv_src.shape[0], same_pool=kv_src.data_ptr() == kv_dst.data_ptr(),
                                   tree_slot_idx=None if tree_slot_idx is None else tree_slot_idx.cpu().numpy(),
                                   max_prefix_len=max_prefix_len)
        if rc != DDT_OK:
            raise DDTError(rc, f"kv_compact_check (slot {bad})")
    if slot_idx_out is None:
        slot_idx_out = _make(stream, slot_idx.clone)
    if workspace is None:
        workspace = _make(stream, torch.empty, 256, dtype=torch.uint8, device=slot_idx.device)
    dims = make_dims(B, 1, 1, kv_src.shape[0], stride, stride if max_prefix_len is None else max_prefix_len)
    rc = lib().ddtree_kv_compact(_ptr(kv_src), _ptr(kv_dst), _ptr(slot_idx), _ptr(prefix_len), _ptr(dst_start),
                                 _ptr(slot_idx_out), ctypes.byref(dims), _ptr(workspace), _stream(stream))
    _check(rc, "ddtree_kv_compact")
    _keep(stream, slot_idx_out, workspace)
    return slot_idx_out


def read_device_status(workspace, stream=None, library=None) -> int:
    """The status word of the last call that used `workspace`, after waiting for `stream`.

    Without a stream it waits for the current one of the workspace's device, where the call ran.
    """
    st = ctypes.c_int32(0)
    L = lib() if library is None else library
    device = workspace.device
    _run_on(device, L.ddtree_read_device_status, "ddtree_read_device_status", _ptr(workspace), ctypes.byref(st),
            ctypes.c_void_p(_stream_of(device, stream)))
    return int(st.value)
