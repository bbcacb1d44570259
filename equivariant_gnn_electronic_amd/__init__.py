"""MI355X-native SO(2) equivariant message-passing layer: Python binding of libegnn.so.

The functions here carry the names of the C ABI (include/egnn.h) and only
marshal arguments: torch supplies device memory and the current HIP stream,
and every step of the computation runs in the library's HIP kernels.  There
is no fallback path: if libegnn.so is missing, or the tensors are not on a
GPU, the calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes as ct
import functools
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import EGNN_BF16, EGNN_F32, EgnnError

__all__ = ["Graph", "layer_desc", "egnn_build_graph", "egnn_build_graph_noalloc", "egnn_edge_geom", "egnn_geom_stride",
           "egnn_layer_weight_count", "egnn_layer_sizes", "egnn_layer_fwd", "egnn_layer_bwd",
           "egnn_hblocks", "egnn_hblocks_label_rows", "egnn_timing_enable", "egnn_timing_collect",
           "egnn_timing_reset", "GraphBuilder", "LayerBuffers", "EgnnError", "EGNN_F32", "EGNN_BF16",
           "Basis", "Orbitals", "egnn_label_width", "egnn_orbital_layout", "egnn_matrix_to_label",
           "egnn_label_to_matrix", "egnn_edge_update_fwd", "egnn_edge_update_bwd", "egnn_assemble_bsr",
           "attn_desc", "AttnBuffers", "egnn_diff_attention_sizes", "egnn_diff_attention_fwd",
           "egnn_diff_attention_bwd", "egnn_distance_borders", "egnn_distance_bias_fwd", "egnn_distance_bias_bwd",
           "dropout_desc", "egnn_dropout_fwd", "egnn_dropout_bwd"]

_STORAGE = {EGNN_F32: torch.float32, EGNN_BF16: torch.bfloat16}


def _stream():
    return ct.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ct.c_void_p(t.data_ptr())


def _d3(v):
    return (ct.c_double * 3)(*[float(a) for a in v])


def _expect(t, name, dtype, shape, min_rows=None):
    """Reject a tensor whose dtype or shape differs from what the kernels read.

    The C ABI sees plain pointers, so this is the only place a wrong buffer can be
    caught before a kernel reads or writes past it.  `shape` lists the expected
    sizes (None = any); `min_rows`, when given, replaces an exact first size by a
    lower bound.  Runs before the device check, so it needs no GPU.
    """
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape):
        raise ValueError(f"{name} must have {len(shape)} dimensions, got shape {tuple(t.shape)}")
    for i, (got, want) in enumerate(zip(t.shape, shape)):
        if i == 0 and min_rows is not None:
            if got < min_rows:
                raise ValueError(f"{name} needs at least {min_rows} rows, got {got}")
        elif want is not None and got != want:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _expect_bytes(t, name, n):
    if n > 0 and (t is None or t.numel() * t.element_size() < n):
        have = 0 if t is None else t.numel() * t.element_size()
        raise ValueError(f"{name} holds {have} bytes, needs {n}")


@dataclass
class Graph:
    """Destination-sorted CSR (incoming-edge layout) held in torch tensors."""
    n_dst: int
    n_src: int
    n_edges: int
    row_ptr: torch.Tensor
    src: torch.Tensor
    shift: torch.Tensor
    vec: torch.Tensor
    dist: torch.Tensor
    src_ptr: torch.Tensor
    src_perm: torch.Tensor

    def c_struct(self):
        g = _lib.EgnnGraph()
        g.n_dst, g.n_src = self.n_dst, self.n_src
        g.capacity = self.src.numel()
        g.n_edges = self.n_edges
        for f in ("row_ptr", "src", "shift", "vec", "dist", "src_ptr", "src_perm"):
            t = self.__dict__[f]
            setattr(g, f, None if t is None else t.data_ptr())
        return g

    @classmethod
    def from_csr(cls, row_ptr, src, n_src=None, shift=None, group=False):
        """A graph given by its CSR (row_ptr, src, optional shift).  With
        group=True its source grouping (src_ptr, src_perm) is made by
        egnn_group_sources, so Matrix <-> Label takes the source-grouped order."""
        n_dst = row_ptr.numel() - 1
        _expect(row_ptr, "row_ptr", torch.int32, (n_dst + 1,))
        _expect(src, "src", torch.int32, (None,))
        if shift is not None:
            _expect(shift, "shift", torch.int8, (src.numel(), 3))
        g = cls(n_dst, n_dst if n_src is None else n_src, src.numel(), row_ptr, src, shift,
                None, None, None, None)
        if group:
            egnn_group_sources(g)
        return g


def egnn_group_sources(graph: Graph):
    """Write graph.src_ptr [n_src + 1] and graph.src_perm [n_edges]: the edge ids
    of each source in ascending order (sources outside [0, n_src) in no group)."""
    lib = _lib.load()
    _expect(graph.src, "src", torch.int32, (graph.n_edges,))
    dev = graph.src.device
    graph.src_ptr = torch.empty(graph.n_src + 1, dtype=torch.int32, device=dev)
    graph.src_perm = torch.empty(max(graph.n_edges, 1), dtype=torch.int32, device=dev)
    nbytes = ct.c_size_t(0)
    _lib.check("egnn_group_sources_workspace",
               lib.egnn_group_sources_workspace(graph.n_src, graph.n_edges, ct.byref(nbytes)))
    ws = torch.empty(max(nbytes.value, 1), dtype=torch.uint8, device=dev)
    g = graph.c_struct()
    _lib.check("egnn_group_sources", lib.egnn_group_sources(ct.byref(g), _ptr(ws), nbytes.value, _stream()))
    return graph


def layer_desc(lmax, mmax, C, n_rbf, r_cut, storage=EGNN_F32):
    return _lib.EgnnLayerDesc(lmax, mmax, C, n_rbf, float(r_cut), storage)


def egnn_build_graph(pos, n_dst, lo, box, periodic_mask, r_cut, capacity=None):
    """Build the graph of positions pos [n_src][3] (float64, on the GPU).

    Runs the two-phase protocol of the C call: an edge count (capacity 0
    unless given), then the fill into arrays of exactly that size.
    """
    lib = _lib.load()
    _expect(pos, "pos", torch.float64, (None, 3))
    dev = pos.device
    n_src = pos.shape[0]
    if not 0 <= n_dst <= n_src:
        raise ValueError(f"n_dst ({n_dst}) must lie in [0, n_src = {n_src}]")
    row_ptr = torch.empty(n_dst + 1, dtype=torch.int32, device=dev)
    cap = 0 if capacity is None else int(capacity)

    def arrays(c):
        return dict(src=torch.empty(max(c, 1), dtype=torch.int32, device=dev),
                    shift=torch.empty((max(c, 1), 3), dtype=torch.int8, device=dev),
                    vec=torch.empty((max(c, 1), 3), dtype=torch.float32, device=dev),
                    dist=torch.empty(max(c, 1), dtype=torch.float32, device=dev),
                    src_ptr=torch.empty(n_src + 1, dtype=torch.int32, device=dev),
                    src_perm=torch.empty(max(c, 1), dtype=torch.int32, device=dev))

    lo3, box3 = _d3(lo), _d3(box)
    for _ in range(2):
        a = arrays(cap)
        g = _lib.EgnnGraph()
        g.n_dst, g.n_src, g.capacity = n_dst, n_src, cap
        g.row_ptr = row_ptr.data_ptr()
        g.src_ptr = a["src_ptr"].data_ptr()
        for f in ("src", "shift", "vec", "dist", "src_perm"):
            setattr(g, f, a[f].data_ptr() if cap > 0 else None)
        ws_bytes = ct.c_size_t()
        _lib.check("egnn_build_graph_workspace", lib.egnn_build_graph_workspace(
            n_dst, n_src, lo3, box3, periodic_mask, float(r_cut), cap, ct.byref(ws_bytes)))
        ws = torch.empty(max(ws_bytes.value, 1), dtype=torch.uint8, device=dev)
        st = lib.egnn_build_graph(_ptr(pos), lo3, box3, periodic_mask, float(r_cut), ct.byref(g),
                                  _ptr(ws), ws_bytes.value, _stream())
        if st == _lib.EGNN_E_CAPACITY:
            cap = int(g.n_edges)
            continue
        _lib.check("egnn_build_graph", st)
        E = int(g.n_edges)
        return Graph(n_dst, n_src, E, row_ptr, a["src"][:E], a["shift"][:E], a["vec"][:E], a["dist"][:E],
                     a["src_ptr"], a["src_perm"][:E])
    raise RuntimeError("egnn_build_graph: edge count changed between the two passes")


def egnn_build_graph_noalloc(pos, n_dst, lo, box, periodic_mask, r_cut, capacity=None):
    """egnn_build_graph through the allocation-free entry point (the library's
    static workspace instead of one from torch).  The output arrays are still
    the caller's: they are allocated here, as in egnn_build_graph."""
    lib = _lib.load()
    _expect(pos, "pos", torch.float64, (None, 3))
    dev = pos.device
    n_src = pos.shape[0]
    if not 0 <= n_dst <= n_src:
        raise ValueError(f"n_dst ({n_dst}) must lie in [0, n_src = {n_src}]")
    row_ptr = torch.empty(n_dst + 1, dtype=torch.int32, device=dev)
    src_ptr = torch.empty(n_src + 1, dtype=torch.int32, device=dev)
    cap = 0 if capacity is None else int(capacity)
    lo3, box3 = _d3(lo), _d3(box)
    for _ in range(2):
        a = {f: torch.empty(sh, dtype=dt, device=dev) for f, sh, dt in (
            ("src", (max(cap, 1),), torch.int32), ("shift", (max(cap, 1), 3), torch.int8),
            ("vec", (max(cap, 1), 3), torch.float32), ("dist", (max(cap, 1),), torch.float32),
            ("src_perm", (max(cap, 1),), torch.int32))}
        g = _lib.EgnnGraph()
        g.n_dst, g.n_src, g.capacity = n_dst, n_src, cap
        g.row_ptr, g.src_ptr = row_ptr.data_ptr(), src_ptr.data_ptr()
        for f in a:
            setattr(g, f, a[f].data_ptr() if cap > 0 else None)
        st = lib.egnn_build_graph_noalloc(_ptr(pos), lo3, box3, periodic_mask, float(r_cut), ct.byref(g), _stream())
        if st == _lib.EGNN_E_CAPACITY:
            cap = int(g.n_edges)
            continue
        _lib.check("egnn_build_graph_noalloc", st)
        E = int(g.n_edges)
        return Graph(n_dst, n_src, E, row_ptr, a["src"][:E], a["shift"][:E], a["vec"][:E], a["dist"][:E],
                     src_ptr, a["src_perm"][:E])
    raise RuntimeError("egnn_build_graph_noalloc: edge count changed between the two passes")


class GraphBuilder:
    """Repeated egnn_build_graph calls on one structure size with preallocated arrays.

    The arrays and workspace are sized for `capacity` edges once; each
    build() is a single C call (one edge count + fill).
    """

    def __init__(self, n_dst, n_src, lo, box, periodic_mask, r_cut, capacity, device):
        self.n_dst, self.n_src, self.mask, self.r_cut = n_dst, n_src, periodic_mask, float(r_cut)
        self.lo3, self.box3 = _d3(lo), _d3(box)
        c = max(int(capacity), 1)
        self.cap = int(capacity)
        self.row_ptr = torch.empty(n_dst + 1, dtype=torch.int32, device=device)
        self.src = torch.empty(c, dtype=torch.int32, device=device)
        self.shift = torch.empty((c, 3), dtype=torch.int8, device=device)
        self.vec = torch.empty((c, 3), dtype=torch.float32, device=device)
        self.dist = torch.empty(c, dtype=torch.float32, device=device)
        self.src_ptr = torch.empty(n_src + 1, dtype=torch.int32, device=device)
        self.src_perm = torch.empty(c, dtype=torch.int32, device=device)
        ws_bytes = ct.c_size_t()
        _lib.check("egnn_build_graph_workspace", _lib.load().egnn_build_graph_workspace(
            n_dst, n_src, self.lo3, self.box3, periodic_mask, self.r_cut, self.cap, ct.byref(ws_bytes)))
        self.ws = torch.empty(max(ws_bytes.value, 1), dtype=torch.uint8, device=device)
        self.g = _lib.EgnnGraph()
        g = self.g
        g.n_dst, g.n_src, g.capacity = n_dst, n_src, self.cap
        for f in ("row_ptr", "src", "shift", "vec", "dist", "src_ptr", "src_perm"):
            setattr(g, f, getattr(self, f).data_ptr())

    def build(self, pos):
        _expect(pos, "pos", torch.float64, (self.n_src, 3))
        _lib.check("egnn_build_graph", _lib.load().egnn_build_graph(
            _ptr(pos), self.lo3, self.box3, self.mask, self.r_cut, ct.byref(self.g), _ptr(self.ws),
            self.ws.numel(), _stream()))
        E = int(self.g.n_edges)
        return Graph(self.n_dst, self.n_src, E, self.row_ptr, self.src[:E], self.shift[:E], self.vec[:E],
                     self.dist[:E], self.src_ptr, self.src_perm[:E])


def egnn_timing_enable(on=True):
    _lib.check("egnn_timing_enable", _lib.load().egnn_timing_enable(1 if on else 0))


def egnn_timing_reset():
    _lib.load().egnn_timing_reset()


def egnn_timing_collect():
    """{kernel family: {launches, total_ms, flops, bytes}} accumulated so far (waits for the GPU)."""
    out = (_lib.EgnnTimingEntry * 64)()
    dropped = ct.c_int64()
    n = _lib.load().egnn_timing_collect(out, 64, ct.byref(dropped))
    res = {}
    for i in range(n):
        e = out[i]
        res[e.name.decode()] = dict(launches=int(e.launches), total_ms=float(e.total_ms), flops=float(e.flops),
                                    bytes=float(e.bytes))
    return res, int(dropped.value)


def egnn_geom_stride(desc):
    return int(_lib.load().egnn_geom_stride(ct.byref(desc)))


def egnn_layer_weight_count(desc):
    return int(_lib.load().egnn_layer_weight_count(ct.byref(desc)))


def egnn_edge_geom(desc, graph: Graph, out=None):
    """Per-edge Wigner rows, radial basis and destination row: [E][stride] float32."""
    lib = _lib.load()
    stride = egnn_geom_stride(desc)
    if stride <= 0:
        raise ValueError("invalid layer description")
    if out is None:
        out = torch.empty((max(graph.n_edges, 1), stride), dtype=torch.float32, device=graph.row_ptr.device)
    _expect(out, "out", torch.float32, (None, stride), min_rows=graph.n_edges)
    g = graph.c_struct()
    _lib.check("egnn_edge_geom", lib.egnn_edge_geom(ct.byref(desc), ct.byref(g), _ptr(out), _stream()))
    return out


def egnn_layer_sizes(desc, graph: Graph):
    lib = _lib.load()
    s, f, b = ct.c_size_t(), ct.c_size_t(), ct.c_size_t()
    g = graph.c_struct()
    _lib.check("egnn_layer_sizes", lib.egnn_layer_sizes(ct.byref(desc), ct.byref(g), ct.byref(s), ct.byref(f),
                                                         ct.byref(b)))
    return s.value, f.value, b.value


class LayerBuffers:
    """Saved activations and workspaces for one layer on one graph (allocated by torch)."""

    def __init__(self, desc, graph: Graph, train=True):
        saved, wsf, wsb = egnn_layer_sizes(desc, graph)
        dev = graph.row_ptr.device
        self.saved = torch.empty(max(saved, 1), dtype=torch.uint8, device=dev) if train else None
        self.ws = torch.empty(max(wsf, wsb if train else 0, 1), dtype=torch.uint8, device=dev)


def _check_layer_args(desc, graph: Graph, geom, weights, x):
    """dtype and shape of the inputs every layer call reads; returns (K, storage dtype)."""
    if desc.storage not in _STORAGE:
        raise ValueError(f"unknown storage type {desc.storage}")
    K = (desc.lmax + 1) ** 2
    dt = _STORAGE[desc.storage]
    n_w = egnn_layer_weight_count(desc)
    if n_w == 0:
        raise ValueError("invalid layer description")
    _expect(weights, "weights", torch.float32, (n_w,))
    _expect(geom, "geom", torch.float32, (None, egnn_geom_stride(desc)), min_rows=graph.n_edges)
    _expect(x, "x", dt, (None, K, desc.C), min_rows=graph.n_src)
    return K, dt


def _check_buffers(desc, graph: Graph, buffers, train, bwd):
    saved, wsf, wsb = egnn_layer_sizes(desc, graph)
    if train or bwd:
        if buffers.saved is None:
            raise ValueError("the backward needs buffers made with train=True")
        _expect_bytes(buffers.saved, "buffers.saved", saved)
    _expect_bytes(buffers.ws, "buffers.ws", wsb if bwd else wsf)


def egnn_layer_fwd(desc, graph: Graph, geom, weights, x, x_out=None, edge_out=False, buffers=None):
    """x_out [n_dst][K][C] (and edge_out [E][K][C] if requested) of one layer."""
    lib = _lib.load()
    K, dt = _check_layer_args(desc, graph, geom, weights, x)
    if buffers is None:
        buffers = LayerBuffers(desc, graph, train=False)
    _check_buffers(desc, graph, buffers, train=buffers.saved is not None, bwd=False)
    if x_out is None:
        x_out = torch.empty((graph.n_dst, K, desc.C), dtype=dt, device=x.device)
    _expect(x_out, "x_out", dt, (graph.n_dst, K, desc.C))
    eo = torch.empty((max(graph.n_edges, 1), K, desc.C), dtype=dt, device=x.device) if edge_out else None
    g = graph.c_struct()
    _lib.check("egnn_layer_fwd", lib.egnn_layer_fwd(
        ct.byref(desc), ct.byref(g), _ptr(geom), _ptr(weights), _ptr(x), _ptr(x_out), _ptr(eo),
        _ptr(buffers.saved), _ptr(buffers.ws), buffers.ws.numel(), _stream()))
    return (x_out, eo[:graph.n_edges] if eo is not None else None), buffers


def egnn_layer_bwd(desc, graph: Graph, geom, weights, x, buffers, grad_out, grad_x=None, grad_w=None):
    """(dL/dx [n_src][K][C], dL/dweights) for the loss <grad_out, x_out>."""
    lib = _lib.load()
    K, _ = _check_layer_args(desc, graph, geom, weights, x)
    _check_buffers(desc, graph, buffers, train=True, bwd=True)
    _expect(grad_out, "grad_out", torch.float32, (graph.n_dst, K, desc.C))
    if grad_x is None:
        grad_x = torch.empty((graph.n_src, K, desc.C), dtype=torch.float32, device=x.device)
    if grad_w is None:
        grad_w = torch.empty(egnn_layer_weight_count(desc), dtype=torch.float32, device=x.device)
    _expect(grad_x, "grad_x", torch.float32, (graph.n_src, K, desc.C))
    _expect(grad_w, "grad_w", torch.float32, (egnn_layer_weight_count(desc),))
    g = graph.c_struct()
    _lib.check("egnn_layer_bwd", lib.egnn_layer_bwd(
        ct.byref(desc), ct.byref(g), _ptr(geom), _ptr(weights), _ptr(x), _ptr(buffers.saved), _ptr(grad_out),
        _ptr(grad_x), _ptr(grad_w), _ptr(buffers.ws), buffers.ws.numel(), _stream()))
    return grad_x, grad_w


def egnn_edge_update_fwd(desc, graph: Graph, geom, weights, x, e_in, e_out=None, buffers=None):
    """Edge-update block: e_out = e_in + the per-edge message (in place when e_out is e_in).
    Returns (e_out, buffers); buffers keep the activations the backward reads."""
    lib = _lib.load()
    K, dt = _check_layer_args(desc, graph, geom, weights, x)
    _expect(e_in, "e_in", dt, (graph.n_edges, K, desc.C))
    if buffers is None:
        buffers = LayerBuffers(desc, graph, train=True)
    _check_buffers(desc, graph, buffers, train=buffers.saved is not None, bwd=False)
    if e_out is None:
        e_out = torch.empty_like(e_in)
    _expect(e_out, "e_out", dt, (graph.n_edges, K, desc.C))
    g = graph.c_struct()
    _lib.check("egnn_edge_update_fwd", lib.egnn_edge_update_fwd(
        ct.byref(desc), ct.byref(g), _ptr(geom), _ptr(weights), _ptr(x), _ptr(e_in), _ptr(e_out),
        _ptr(buffers.saved) if buffers.saved is not None else None, _ptr(buffers.ws), buffers.ws.numel(), _stream()))
    return e_out, buffers


def egnn_edge_update_bwd(desc, graph: Graph, geom, weights, x, buffers, grad_e_out, grad_x=None, grad_w=None):
    """Gradients of <grad_e_out, e_out> w.r.t. x and the packed weights (that w.r.t. e_in is grad_e_out)."""
    lib = _lib.load()
    K, _ = _check_layer_args(desc, graph, geom, weights, x)
    _check_buffers(desc, graph, buffers, train=True, bwd=True)
    _expect(grad_e_out, "grad_e_out", torch.float32, (graph.n_edges, K, desc.C))
    if grad_x is None:
        grad_x = torch.empty((graph.n_src, K, desc.C), dtype=torch.float32, device=x.device)
    if grad_w is None:
        grad_w = torch.empty(egnn_layer_weight_count(desc), dtype=torch.float32, device=x.device)
    _expect(grad_x, "grad_x", torch.float32, (graph.n_src, K, desc.C))
    _expect(grad_w, "grad_w", torch.float32, (egnn_layer_weight_count(desc),))
    g = graph.c_struct()
    _lib.check("egnn_edge_update_bwd", lib.egnn_edge_update_bwd(
        ct.byref(desc), ct.byref(g), _ptr(geom), _ptr(weights), _ptr(x), _ptr(buffers.saved), _ptr(grad_e_out),
        _ptr(grad_x), _ptr(grad_w), _ptr(buffers.ws), buffers.ws.numel(), _stream()))
    return grad_x, grad_w


def _as(t, dtype, shape):
    """Whether t is just what a call reads: the quick form of _expect, which says what is wrong otherwise."""
    return isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.is_contiguous()


def _on_one_device(**tensors):
    """The GPU that every given tensor lives on (None entries are skipped)."""
    given = [t for t in tensors.values() if t is not None]
    index = given[0].get_device()
    if index >= 0 and all(t.get_device() == index for t in given):
        return given[0].device
    named, dev = tensors.items(), None
    for name, t in named:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must live on the GPU")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    return dev


def _data(t):
    return None if t is None else t.data_ptr()


_HERE = contextlib.nullcontext()
# the current stream's handle without building a torch.cuda.Stream (about 2 us a call)
_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(dev):
    """Makes dev the current device for a call; nothing to do where it is (torch.cuda.device costs about 2 us)."""
    return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream_of(dev):
    return _handle(dev.index) if _handle is not None else torch.cuda.current_stream(dev).cuda_stream


def _graph_struct(graph, grouped=False, dist=False):
    """The fields that the attention and the bias read."""
    g = _lib.EgnnGraph()
    g.n_dst, g.n_src, g.n_edges = graph.n_dst, graph.n_src, graph.n_edges
    if dist:
        g.dist = graph.dist.data_ptr()
        return g
    g.row_ptr, g.src = graph.row_ptr.data_ptr(), graph.src.data_ptr()
    if grouped:
        g.src_ptr, g.src_perm = graph.src_ptr.data_ptr(), graph.src_perm.data_ptr()
    return g


def _expect_rng(rng, p):
    if rng is not None:
        if not _as(rng, torch.int64, (2,)):
            _expect(rng, "rng", torch.int64, (2,))
    elif not float(p) * 65536 < 0.5:
        raise ValueError("rng ({seed, step}, int64 on the GPU) is required when the dropout probability is not zero")


def attn_desc(lmax, C, n_heads, head_dim, scale=None, drop_p=0.0, site=0, storage=EGNN_F32):
    """Differential attention over value rows [(lmax+1)^2][C]; scale defaults to 1/sqrt(head_dim)."""
    if scale is None:
        scale = float(head_dim) ** -0.5 if head_dim > 0 else 1.0
    return _lib.EgnnAttnDesc(lmax, C, n_heads, head_dim, storage, site, 0, 0, 0, float(scale), float(drop_p))


def egnn_diff_attention_sizes(desc, graph: Graph):
    """(saved, inference workspace, training workspace) bytes."""
    s, i, t = ct.c_size_t(), ct.c_size_t(), ct.c_size_t()
    g = _lib.EgnnGraph()
    g.n_dst, g.n_src, g.n_edges = graph.n_dst, graph.n_src, graph.n_edges
    _lib.check("egnn_diff_attention_sizes", _lib.load().egnn_diff_attention_sizes(
        ct.byref(desc), ct.byref(g), ct.byref(s), ct.byref(i), ct.byref(t)))
    return s.value, i.value, t.value


def _attn_key(desc, graph):
    """What the buffers' sizes depend on."""
    return (desc.lmax, desc.C, desc.n_heads, desc.head_dim, graph.n_dst, graph.n_src, graph.n_edges)


class AttnBuffers:
    """What the attention's backward reads and the workspaces, for one graph (allocated by torch)."""

    def __init__(self, desc, graph: Graph, train=True):
        saved, infer, tr = egnn_diff_attention_sizes(desc, graph)
        dev = graph.row_ptr.device
        self._fits = _attn_key(desc, graph)
        self.saved = torch.empty(max(saved, 1), dtype=torch.uint8, device=dev) if train else None
        self.ws = torch.empty(max(tr if train else infer, 1), dtype=torch.uint8, device=dev)


def _check_attn_buffers(desc, graph, buffers):
    if buffers._fits == _attn_key(desc, graph):
        return
    saved, infer, train = egnn_diff_attention_sizes(desc, graph)
    if buffers.saved is not None:
        _expect_bytes(buffers.saved, "buffers.saved", saved)
    _expect_bytes(buffers.ws, "buffers.ws", infer if buffers.saved is None else train)


def _expect_rows(t, name, dtype, shape, rows):
    """Rows whose elements are packed, any distance apart; returns that distance in elements (0: packed rows)."""
    if _as(t, dtype, (rows, *shape)):
        return 0
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape[1:]) != shape or t.dim() != len(shape) + 1:
        raise ValueError(f"{name} must have shape (rows, {', '.join(map(str, shape))}), got {tuple(t.shape)}")
    if t.shape[0] < rows:
        raise ValueError(f"{name} needs at least {rows} rows, got {t.shape[0]}")
    width = 1
    for size, stride in zip(reversed(shape), reversed(t.stride()[1:])):
        if size > 1 and stride != width:
            raise ValueError(f"the elements of a row of {name} must be packed, strides are {t.stride()}")
        width *= size
    if rows <= 1:
        return 0
    if t.stride(0) < width:
        raise ValueError(f"the rows of {name} overlap: stride {t.stride(0)}, width {width}")
    return t.stride(0)


def _expect_graph(graph: Graph, grouped=False):
    if not _as(graph.row_ptr, torch.int32, (graph.n_dst + 1,)):
        _expect(graph.row_ptr, "graph.row_ptr", torch.int32, (graph.n_dst + 1,))
    if not _as(graph.src, torch.int32, (graph.n_edges,)):
        _expect(graph.src, "graph.src", torch.int32, (None,), min_rows=graph.n_edges)
    if grouped:
        if graph.src_ptr is None or graph.src_perm is None:
            raise ValueError("the backward needs the graph grouped by source (egnn_group_sources)")
        if not _as(graph.src_ptr, torch.int32, (graph.n_src + 1,)):
            _expect(graph.src_ptr, "graph.src_ptr", torch.int32, (graph.n_src + 1,))
        if not _as(graph.src_perm, torch.int32, (graph.n_edges,)):
            _expect(graph.src_perm, "graph.src_perm", torch.int32, (None,), min_rows=graph.n_edges)


def _check_attn(desc, graph: Graph, q, k, v, lam, rng, grouped=False):
    """Checks what both directions read; returns the description with the tensors' strides and (K, storage dtype)."""
    if desc.storage not in _STORAGE:
        raise ValueError(f"unknown storage type {desc.storage}")
    dt, H, D, C, K = _STORAGE[desc.storage], desc.n_heads, desc.head_dim, desc.C, (desc.lmax + 1) ** 2
    _expect_graph(graph, grouped)
    strides = (_expect_rows(q, "q", dt, (H, 2, D), graph.n_dst), _expect_rows(k, "k", dt, (H, 2, D), graph.n_src),
               _expect_rows(v, "v", dt, (K, C), graph.n_src))
    if not _as(lam, torch.float32, (H,)):
        _expect(lam, "lam", torch.float32, (H,))
    _expect_rng(rng, desc.drop_p)
    if strides != (desc.q_stride, desc.k_stride, desc.v_stride):
        desc = _lib.EgnnAttnDesc.from_buffer_copy(desc)
        desc.q_stride, desc.k_stride, desc.v_stride = strides
    return desc, K, dt


def egnn_diff_attention_fwd(desc, graph: Graph, q, k, v, lam, bias=None, mask=None, rng=None, out=None, buffers=None):
    """Differential attention of every row over its incoming edges: (out [n_dst][K][C], buffers).

    q [n_dst][H][2][D], k [n_src][H][2][D], v [n_src][K][C] in the storage
    type (rows may be slices of a wider array), lam [H]; bias [E][2H] or
    [E][H][2]; mask [E] uint8 or bool, 0 = the edge takes no part; rng int64
    [2] = {seed, step} on the GPU, needed for dropout.  buffers made with
    train=True keep what the backward reads; without buffers the call makes
    its own for inference.
    """
    lib = _lib.load()
    d, K, dt = _check_attn(desc, graph, q, k, v, lam, rng)
    E, H = graph.n_edges, desc.n_heads
    if bias is not None and not _as(bias, torch.float32, (E, 2 * H)):
        _expect(bias.reshape(-1) if isinstance(bias, torch.Tensor) and bias.is_contiguous() else bias, "bias",
                torch.float32, (E * 2 * H,))
    if mask is not None and not _as(mask, torch.uint8, (E,)):
        if isinstance(mask, torch.Tensor) and mask.dtype == torch.bool:
            mask = mask.view(torch.uint8)
        _expect(mask, "mask", torch.uint8, (E,))
    dev = _on_one_device(row_ptr=graph.row_ptr, src=graph.src, q=q, k=k, v=v, lam=lam, bias=bias, mask=mask, rng=rng,
                         out=out, saved=buffers.saved if buffers else None, ws=buffers.ws if buffers else None)
    with _on(dev):
        if buffers is None:
            buffers = AttnBuffers(desc, graph, train=False)
        _check_attn_buffers(d, graph, buffers)
        if out is None:
            out = torch.empty((graph.n_dst, K, desc.C), dtype=dt, device=dev)
        else:
            _expect(out, "out", dt, (graph.n_dst, K, desc.C))
        g = _graph_struct(graph)
        _lib.check("egnn_diff_attention_fwd", lib.egnn_diff_attention_fwd(
            ct.byref(d), ct.byref(g), _data(q), _data(k), _data(v), _data(lam), _data(bias), _data(mask), _data(rng),
            _data(out), _data(buffers.saved), _data(buffers.ws), buffers.ws.numel(), _stream_of(dev)))
    return out, buffers


def egnn_diff_attention_bwd(desc, graph: Graph, q, k, v, lam, buffers, grad_out, rng=None):
    """(grad_q, grad_k, grad_v, grad_lam, grad_bias [E][2H]) of <grad_out, out>, fp32.

    buffers are those of the forward on the same inputs (train=True); the
    graph needs its source grouping; grad_bias is the gradient of the logits.
    """
    lib = _lib.load()
    d, K, _ = _check_attn(desc, graph, q, k, v, lam, rng, grouped=True)
    E, H, D, C = graph.n_edges, desc.n_heads, desc.head_dim, desc.C
    if not _as(grad_out, torch.float32, (graph.n_dst, K, C)):
        _expect(grad_out, "grad_out", torch.float32, (graph.n_dst, K, C))
    if buffers is None or buffers.saved is None:
        raise ValueError("the backward needs buffers made with train=True")
    dev = _on_one_device(row_ptr=graph.row_ptr, src=graph.src, src_ptr=graph.src_ptr, src_perm=graph.src_perm, q=q,
                         k=k, v=v, lam=lam, rng=rng, grad_out=grad_out, saved=buffers.saved, ws=buffers.ws)
    with _on(dev):
        _check_attn_buffers(d, graph, buffers)
        f32 = dict(dtype=torch.float32, device=dev)
        gq = torch.empty((graph.n_dst, H, 2, D), **f32)
        gk = torch.empty((graph.n_src, H, 2, D), **f32)
        gv = torch.empty((graph.n_src, K, C), **f32)
        gl = torch.empty(H, **f32)
        gb = torch.empty((E, 2 * H), **f32)
        g = _graph_struct(graph, grouped=True)
        _lib.check("egnn_diff_attention_bwd", lib.egnn_diff_attention_bwd(
            ct.byref(d), ct.byref(g), _data(q), _data(k), _data(v), _data(lam), _data(rng), _data(buffers.saved),
            _data(grad_out), _data(gq), _data(gk), _data(gv), _data(gl), _data(gb), _data(buffers.ws),
            buffers.ws.numel(), _stream_of(dev)))
    return gq, gk, gv, gl, gb


def egnn_distance_borders(n_buckets, n_linear, r_linear, r_max):
    """Bucket borders (CPU float32 [n_buckets - 1]): n_linear of equal width up to r_linear, then equal ratios."""
    out = torch.empty(max(int(n_buckets) - 1, 0), dtype=torch.float32)
    _lib.check("egnn_distance_borders", _lib.load().egnn_distance_borders(
        int(n_buckets), int(n_linear), float(r_linear), float(r_max),
        ct.cast(out.data_ptr(), ct.POINTER(ct.c_float))))
    return out


def _check_bias(graph: Graph, borders, n_buckets, n_columns):
    if not _as(borders, torch.float32, (n_buckets - 1,)):
        _expect(borders, "borders", torch.float32, (n_buckets - 1,))
    if not _as(graph.dist, torch.float32, (graph.n_edges,)):
        _expect(graph.dist, "graph.dist", torch.float32, (None,), min_rows=graph.n_edges)
    return _lib.EgnnBiasDesc(n_buckets, n_columns)


def egnn_distance_bias_fwd(graph: Graph, borders, table, out=None):
    """bias [E][n_columns] = table[bucket of each edge's length]; borders [n_buckets - 1] ascending."""
    _expect(table, "table", torch.float32, (None, None))
    B, M = table.shape
    d = _check_bias(graph, borders, B, M)
    if out is not None:
        _expect(out, "out", torch.float32, (graph.n_edges, M))
    dev = _on_one_device(dist=graph.dist, borders=borders, table=table, out=out)
    with _on(dev):
        if out is None:
            out = torch.empty((graph.n_edges, M), dtype=torch.float32, device=dev)
        g = _graph_struct(graph, dist=True)
        _lib.check("egnn_distance_bias_fwd", _lib.load().egnn_distance_bias_fwd(
            ct.byref(d), ct.byref(g), _data(borders), _data(table), _data(out), _stream_of(dev)))
    return out


@functools.lru_cache(maxsize=64)
def _bias_workspace(n_buckets, n_columns, n_edges):
    """Workspace bytes of the table's gradient: they depend on the sizes alone."""
    d, g, nbytes = _lib.EgnnBiasDesc(n_buckets, n_columns), _lib.EgnnGraph(), ct.c_size_t()
    g.n_edges, g.dist = n_edges, 16   # any address: the query reads nothing
    _lib.check("egnn_distance_bias_workspace",
               _lib.load().egnn_distance_bias_workspace(ct.byref(d), ct.byref(g), ct.byref(nbytes)))
    return nbytes.value


def egnn_distance_bias_bwd(graph: Graph, borders, grad_bias):
    """grad_table [n_buckets][n_columns]: grad_bias [E][n_columns] summed over each bucket's edges."""
    _expect(grad_bias, "grad_bias", torch.float32, (graph.n_edges, None))
    if not isinstance(borders, torch.Tensor):
        raise ValueError("borders must be a torch tensor")
    B, M = borders.numel() + 1, grad_bias.shape[1]
    d = _check_bias(graph, borders, B, M)
    dev = _on_one_device(dist=graph.dist, borders=borders, grad_bias=grad_bias)
    nbytes = _bias_workspace(B, M, graph.n_edges)
    with _on(dev):
        g = _graph_struct(graph, dist=True)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        out = torch.empty((B, M), dtype=torch.float32, device=dev)
        _lib.check("egnn_distance_bias_bwd", _lib.load().egnn_distance_bias_bwd(
            ct.byref(d), ct.byref(g), _data(borders), _data(grad_bias), _data(out), _data(ws), nbytes,
            _stream_of(dev)))
    return out


_SHARE = {"channel": _lib.EGNN_DROP_CHANNEL, "degree": _lib.EGNN_DROP_DEGREE, "row": _lib.EGNN_DROP_ROW}


def dropout_desc(lmax, C, p, share="channel", site=0, storage=EGNN_F32):
    """Dropout of rows [(lmax+1)^2][C]; share: one decision per "channel", per "degree" and channel, or per "row"."""
    if share not in _SHARE:
        raise ValueError(f"unknown sharing {share!r}, one of {sorted(_SHARE)}")
    return _lib.EgnnDropoutDesc(lmax, C, _SHARE[share], storage, site, float(p))


def egnn_dropout_fwd(desc, x, rng, residual=None, out=None):
    """residual + keep/(1-p) x for x [rows][K][C]; rng int64 [2] = {seed, step} on the GPU (None when p is 0)."""
    if desc.storage not in _STORAGE:
        raise ValueError(f"unknown storage type {desc.storage}")
    dt, shape = _STORAGE[desc.storage], (None, (desc.lmax + 1) ** 2, desc.C)
    _expect(x, "x", dt, shape)
    if residual is not None and not _as(residual, dt, x.shape):
        _expect(residual, "residual", dt, tuple(x.shape))
    if out is not None:
        _expect(out, "out", dt, tuple(x.shape))
    _expect_rng(rng, desc.p)
    dev = _on_one_device(x=x, residual=residual, rng=rng, out=out)
    with _on(dev):
        if out is None:
            out = torch.empty_like(x)
        _lib.check("egnn_dropout_fwd", _lib.load().egnn_dropout_fwd(
            ct.byref(desc), x.shape[0], _data(x), _data(residual), _data(rng), _data(out), _stream_of(dev)))
    return out


def egnn_dropout_bwd(desc, grad_y, rng, out=None):
    """Gradient with respect to x for the forward's decisions (that of residual is grad_y itself), fp32."""
    _expect(grad_y, "grad_y", torch.float32, (None, (desc.lmax + 1) ** 2, desc.C))
    if out is not None:
        _expect(out, "out", torch.float32, tuple(grad_y.shape))
    _expect_rng(rng, desc.p)
    dev = _on_one_device(grad_y=grad_y, rng=rng, out=out)
    with _on(dev):
        if out is None:
            out = torch.empty_like(grad_y)
        _lib.check("egnn_dropout_bwd", _lib.load().egnn_dropout_bwd(
            ct.byref(desc), grad_y.shape[0], _data(grad_y), _data(rng), _data(out), _stream_of(dev)))
    return out


def _hdesc(lmax, C, shell_l, storage):
    arr = (ct.c_int32 * len(shell_l))(*shell_l)
    h = _lib.EgnnHDesc(lmax, C, len(shell_l), arr, storage)
    h._keep = arr
    return h


def egnn_hblocks_label_rows(lmax, C, shell_l=(0, 0, 1, 1, 2), storage=EGNN_F32):
    return int(_lib.load().egnn_hblocks_label_rows(ct.byref(_hdesc(lmax, C, shell_l, storage))))


def egnn_hblocks(lmax, C, w_edge, w_node, edge_irreps, node_irreps, shell_l=(0, 0, 1, 1, 2), storage=EGNN_F32):
    """Orbital blocks [E][n_orb][n_orb] and [N][n_orb][n_orb] from irreps."""
    lib = _lib.load()
    h = _hdesc(lmax, C, shell_l, storage)
    n_orb = sum(2 * l + 1 for l in shell_l)
    if storage not in _STORAGE:
        raise ValueError(f"unknown storage type {storage}")
    rows = egnn_hblocks_label_rows(lmax, C, shell_l, storage)
    if rows <= 0:
        raise ValueError("invalid decode description")
    K = (lmax + 1) ** 2
    if edge_irreps is None and node_irreps is None:
        raise ValueError("edge_irreps or node_irreps is required")
    E = 0 if edge_irreps is None else edge_irreps.shape[0]
    N = 0 if node_irreps is None else node_irreps.shape[0]
    if E:
        _expect(edge_irreps, "edge_irreps", _STORAGE[storage], (E, K, C))
        _expect(w_edge.reshape(-1) if isinstance(w_edge, torch.Tensor) else w_edge, "w_edge", torch.float32,
                (rows * C,))
    if N:
        _expect(node_irreps, "node_irreps", _STORAGE[storage], (N, K, C))
        _expect(w_node.reshape(-1) if isinstance(w_node, torch.Tensor) else w_node, "w_node", torch.float32,
                (rows * C,))
    dev = (edge_irreps if edge_irreps is not None else node_irreps).device
    he = torch.empty((max(E, 1), n_orb, n_orb), dtype=torch.float32, device=dev)
    hn = torch.empty((max(N, 1), n_orb, n_orb), dtype=torch.float32, device=dev)
    _lib.check("egnn_hblocks", lib.egnn_hblocks(
        ct.byref(h), E, N, _ptr(w_edge) if E else None, _ptr(w_node) if N else None,
        _ptr(edge_irreps) if E else None, _ptr(node_irreps) if N else None, _ptr(he) if E else None,
        _ptr(hn) if N else None, _stream()))
    return he[:E], hn[:N]


def egnn_assemble_bsr(graph: Graph, h_edge, h_onsite=None):
    """One block-sparse-row matrix over all image shifts from the decode's blocks:
    (row_ptr [n_src+1], col [nnzb], shift [nnzb][3] int8, val [nnzb][n_orb][n_orb])."""
    lib = _lib.load()
    _expect(h_edge, "h_edge", torch.float32, (graph.n_edges, None, None))
    n_orb = h_edge.shape[1]
    if h_edge.shape[2] != n_orb:
        raise ValueError("h_edge blocks must be square")
    if h_onsite is not None:
        _expect(h_onsite, "h_onsite", torch.float32, (graph.n_dst, n_orb, n_orb))
    dev = graph.row_ptr.device
    nnzb = graph.n_edges + (graph.n_dst if h_onsite is not None else 0)
    rp = torch.empty(graph.n_src + 1, dtype=torch.int32, device=dev)
    col = torch.empty(max(nnzb, 1), dtype=torch.int32, device=dev)
    sh = torch.empty((max(nnzb, 1), 3), dtype=torch.int8, device=dev)
    val = torch.empty((max(nnzb, 1), n_orb, n_orb), dtype=torch.float32, device=dev)
    g = graph.c_struct()
    _lib.check("egnn_assemble_bsr", lib.egnn_assemble_bsr(
        ct.byref(g), n_orb, _ptr(h_edge) if graph.n_edges else None,
        _ptr(h_onsite) if h_onsite is not None else None, _ptr(rp), _ptr(col), _ptr(sh), _ptr(val), _stream()))
    return rp, col[:nnzb], sh[:nnzb], val[:nnzb]


class Basis:
    """Full shell list and per-element shell masks (orbital templates)."""

    def __init__(self, shell_l, species_shells):
        self.shell_l = tuple(int(l) for l in shell_l)
        self.species_shells = tuple(int(m) for m in species_shells)
        self._l = (ct.c_int32 * len(self.shell_l))(*self.shell_l)
        self._m = (ct.c_uint32 * len(self.species_shells))(*self.species_shells)
        self.c = _lib.EgnnBasis(len(self.shell_l), self._l, len(self.species_shells), self._m)


@dataclass
class Orbitals:
    """Atom and structure layout of a batch of matrices (egnn_orbital_layout's outputs)."""
    mol_ptr: torch.Tensor
    species: torch.Tensor
    atom_orb: torch.Tensor
    atom_mol: torch.Tensor
    mol_norb: torch.Tensor
    mat_off: torch.Tensor

    @property
    def n_atoms(self):
        return self.species.numel()

    @property
    def n_mols(self):
        return self.mol_ptr.numel() - 1

    def c_struct(self):
        o = _lib.EgnnOrbitals()
        o.n_mols, o.n_atoms = self.n_mols, self.n_atoms
        for f in ("mol_ptr", "species", "atom_orb", "atom_mol", "mol_norb", "mat_off"):
            setattr(o, f, self.__dict__[f].data_ptr())
        return o


def egnn_label_width(basis: Basis):
    return int(_lib.load().egnn_label_width(ct.byref(basis.c)))


def egnn_orbital_layout(basis: Basis, mol_ptr, species):
    """Orbitals of a batch (mol_ptr [n_mols+1], species [n_atoms], int32 on the GPU) and
    the count of invalid structures and element indices (int64 [1] on the GPU)."""
    lib = _lib.load()
    _expect(mol_ptr, "mol_ptr", torch.int32, (None,), min_rows=1)
    _expect(species, "species", torch.int32, (None,))
    dev = species.device
    n_mols, n_atoms = mol_ptr.numel() - 1, species.numel()
    o = Orbitals(mol_ptr, species,
                 torch.empty(max(n_atoms, 1), dtype=torch.int32, device=dev)[:n_atoms],
                 torch.empty(max(n_atoms, 1), dtype=torch.int32, device=dev)[:n_atoms],
                 torch.empty(max(n_mols, 1), dtype=torch.int32, device=dev)[:n_mols],
                 torch.empty(n_mols + 1, dtype=torch.int64, device=dev))
    bad = torch.empty(1, dtype=torch.int64, device=dev)
    for t in (mol_ptr, species):
        _ptr(t)                      # on the GPU and contiguous
    c = o.c_struct()
    _lib.check("egnn_orbital_layout", lib.egnn_orbital_layout(ct.byref(basis.c), ct.byref(c), _ptr(bad), _stream()))
    return o, bad


def egnn_matrix_to_label(basis: Basis, orbitals: Orbitals, graph, H, edges=True, nodes=True):
    """Labels (h_edge [E][n_lab], h_node [n_atoms][n_lab]) of the batch's matrices H
    (fp32, flat, mat_off[-1] entries) and the count of skipped blocks."""
    lib = _lib.load()
    n_lab = egnn_label_width(basis)
    if n_lab <= 0:
        raise ValueError("invalid basis")
    _expect(H, "H", torch.float32, (None,))
    dev = H.device
    E = graph.n_edges if (graph is not None and edges) else 0
    he = torch.empty((max(E, 1), n_lab), dtype=torch.float32, device=dev)
    hn = torch.empty((max(orbitals.n_atoms, 1), n_lab), dtype=torch.float32, device=dev)
    skipped = torch.empty(1, dtype=torch.int64, device=dev)
    g = graph.c_struct() if (graph is not None and edges) else None
    o = orbitals.c_struct()
    _lib.check("egnn_matrix_to_label", lib.egnn_matrix_to_label(
        ct.byref(basis.c), ct.byref(o), ct.byref(g) if g is not None else None, _ptr(H), H.numel(),
        _ptr(he) if g is not None else None, _ptr(hn) if nodes else None, _ptr(skipped), _stream()))
    return he[:E], (hn[:orbitals.n_atoms] if nodes else None), skipped


def egnn_label_to_matrix(basis: Basis, orbitals: Orbitals, graph, h_edge, h_node, H=None, h_elems=None):
    """Writes the blocks of h_edge / h_node (either may be None) into H (zeros of
    h_elems = mat_off[-1] entries when not given); returns (H, skipped count)."""
    lib = _lib.load()
    n_lab = egnn_label_width(basis)
    if n_lab <= 0:
        raise ValueError("invalid basis")
    if h_edge is not None and graph is not None:
        _expect(h_edge, "h_edge", torch.float32, (graph.n_edges, n_lab))
    if h_node is not None:
        _expect(h_node, "h_node", torch.float32, (orbitals.n_atoms, n_lab))
    dev = orbitals.species.device
    if H is None:
        n = int(orbitals.mat_off[-1].item()) if h_elems is None else int(h_elems)
        H = torch.zeros(max(n, 1), dtype=torch.float32, device=dev)[:n]
    _expect(H, "H", torch.float32, (None,))
    skipped = torch.empty(1, dtype=torch.int64, device=dev)
    g = graph.c_struct() if (graph is not None and h_edge is not None) else None
    o = orbitals.c_struct()
    _lib.check("egnn_label_to_matrix", lib.egnn_label_to_matrix(
        ct.byref(basis.c), ct.byref(o), ct.byref(g) if g is not None else None,
        _ptr(h_edge) if g is not None else None, _ptr(h_node) if h_node is not None else None, _ptr(H),
        H.numel(), _ptr(skipped), _stream()))
    return H, skipped
