"""Python face of the MoVA value path: the C ABI of libmova.so, called with
torch CUDA tensors (torch only provides device memory and the stream).

    v = value_routed(x, Wr, br, Wv)            # (T, 1024) -> view (T, 8, 128)
    idx, w = route(x, Wr, br)
    v = value(x, idx, w, Wv)                    # routing given (compact cache)

and, for the paged key-value cache that v goes into,

    lens, starts, slots, positions, taken = page_map(cached, added, table, free_pages, taken, 64, num_pages, T)
    page_write(k, v, slots, k_cache, v_cache)
    o = page_attend(q, k_cache, v_cache, table, lens)

Every function enqueues on torch's current CUDA stream (the host-buffer forms:
on `stream` if given) and returns without synchronising.  Device-side checks
are read with get_status().  A call given no `ws` uses the workspace this
module keeps for its device and stream, so calls on different streams may
overlap on the GPU.  Calls that share a `ws` must run on one stream.  A value
call that a graph captures without a `ws` has the capturing stream's, so that
such graphs are replayed on that stream.  A paged call that a graph captures
without a `ws` has one in the graph's own memory, whose status get_status() does
not read: give it a `ws` to read one.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional

import torch

from . import _lib

_DT = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16,
       torch.int32: _lib.I32, torch.int8: _lib.I8}
_PATH = {"auto": _lib.PATH_AUTO, "stream": _lib.PATH_STREAM, "tensor": _lib.PATH_TENSOR,
         "tensor_1cta": _lib.PATH_TENSOR_1CTA}


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


try:
    _raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object
except AttributeError:  # pragma: no cover - older torch
    _raw_stream = None


try:
    _current_device = torch._C._cuda_getDevice  # torch.cuda.current_device without its lazy initialisation
except AttributeError:  # pragma: no cover - a torch built without CUDA
    _current_device = torch.cuda.current_device


try:
    _capturing = torch._C._cuda_isCurrentStreamCapturing
except AttributeError:  # pragma: no cover - a torch built without CUDA
    def _capturing() -> bool:
        return False


def _current_stream_handle() -> int:
    """The handle of the current stream of the current device."""
    if _raw_stream is not None:
        return int(_raw_stream(torch.cuda.current_device()))
    return int(torch.cuda.current_stream().cuda_stream)


def _stream(stream: Optional["torch.cuda.Stream"] = None):
    """The handle of `stream`, else of the current stream of the current device."""
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(_current_stream_handle())


def _need(t: torch.Tensor, name: str, dtypes=None, ndim=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _shape(t: torch.Tensor, name: str, want) -> None:
    """The library sees only pointers and the sizes passed with them, so a
    tensor of the wrong shape would be read or written out of bounds: refuse
    it here."""
    if t.shape != want:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(want)}")


def _under_capture(dev: torch.device) -> bool:
    return dev.type == "cuda" and _capturing()


class Workspace:
    """A device workspace that grows on demand.  A buffer that a call under
    stream capture was given is in that call's graph: it is kept when a larger
    one takes its place."""

    def __init__(self):
        self.buf: Optional[torch.Tensor] = None
        self.in_graph = False
        self.kept = []

    def get(self, nbytes: int, device) -> torch.Tensor:
        dev = torch.device(device)
        if self.buf is None or self.buf.numel() < nbytes or self.buf.device != dev:
            if self.in_graph:
                self.kept.append(self.buf)
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
            self.in_graph = False
        self.in_graph = self.in_graph or _under_capture(dev)
        return self.buf


# The workspaces of calls made without `ws`: one per (device, stream).  A call
# leaves its routing, grouping and expert rows in its workspace until its last
# kernel has run, so calls that may overlap on the GPU -- calls on different
# streams -- must not share one.  Calls on one stream run in order and share
# that stream's workspace.
_WS = {}


def _devkey(device) -> torch.device:
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    return dev


def _workspace(nbytes: int, device, stream: Optional["torch.cuda.Stream"] = None) -> torch.Tensor:
    """The default workspace of `stream` (else of the current stream) on
    `device`, grown to at least `nbytes`.  It is allocated while that stream is
    current: torch's caching allocator then keeps the memory of a buffer that
    a later, larger call replaces from every other stream's allocations until
    this stream has passed its last use."""
    dev = _devkey(device)
    handle = int(stream.cuda_stream) if stream is not None else _current_stream_handle()
    key = (dev, handle)
    if key not in _WS:
        _WS[key] = Workspace()
    if stream is None:
        return _WS[key].get(nbytes, dev)
    with torch.cuda.stream(stream):
        return _WS[key].get(nbytes, dev)


def release_workspaces() -> None:
    """Drop the default workspaces (each stream that ran a call without `ws`
    keeps one, sized for its largest call, until this is called).  Safe with
    calls still in flight: torch's caching allocator reuses a freed buffer
    only for later work on the stream that used it.  Not while a graph that
    holds a value call made without `ws` is to be replayed."""
    _WS.clear()


@functools.lru_cache(maxsize=256)
def workspace_size(T: int, d: int, E: int, k: int, n: int) -> int:
    return int(_lib.load().mova_workspace_size(T, d, E, k, n))


@functools.lru_cache(maxsize=256)
def workspace_size_host(T: int, d: int, E: int, k: int, n: int) -> int:
    """Device workspace of the host-buffer value calls (value_routed_host, value_host)."""
    return int(_lib.load().mova_workspace_size_host(T, d, E, k, n))


@functools.lru_cache(maxsize=256)
def attend_workspace_size_host(L: int, d: int, E: int, k: int, n: int, H: int) -> int:
    """Device workspace of value_attend_host."""
    return int(_lib.load().mova_attend_workspace_size_host(L, d, E, k, n, H))


def auto_path(T: int, dtype: torch.dtype) -> str:
    code = _lib.load().mova_auto_path(T, _DT[dtype])
    return {v: k for k, v in _PATH.items()}[code]


def launch_count() -> int:
    """Kernel launches the library has enqueued in this process so far."""
    return int(_lib.load().mova_launch_count())


def _opts(path="auto", events=None, wv_stride=0, partitions=0, decode_launches=0, planes=None):
    """A mova_options value (kept alive by the caller for the call)."""
    ev = _events(events)
    o = _lib.Options(_PATH[path], ctypes.cast(ev, ctypes.c_void_p) if ev is not None else None,
                     int(wv_stride), int(partitions), int(decode_launches),
                     None if planes is None else ctypes.c_void_p(planes.data_ptr()))
    return o, ev


def router_planes(Wr: torch.Tensor) -> torch.Tensor:
    """The router weight split exactly into three bf16 planes (mova_router_planes),
    to hand to value_routed(planes=...) so that calls skip the split."""
    _need(Wr, "Wr", (torch.float32,), 2)
    E, d = Wr.shape
    lib = _lib.load()
    nbytes = int(lib.mova_router_planes_bytes(d))
    planes = torch.empty(nbytes // 2, dtype=torch.bfloat16, device=Wr.device)
    _lib.check(lib.mova_router_planes(_ptr(Wr), E, d, _ptr(planes), _stream()), "mova_router_planes")
    return planes


def route(x: torch.Tensor, Wr: torch.Tensor, br: torch.Tensor, k: int = 4, scale: float = 2.5,
          partitions: int = 0):
    """(idx (T, k) int32, w (T, k) fp32).  partitions=2 sums the router's two
    halves of d separately in fp32 and then adds them (mova_options)."""
    _need(x, "x", (torch.float32, torch.bfloat16), 2)
    _need(Wr, "Wr", (torch.float32,), 2)
    _need(br, "br", (torch.float32,), 1)
    T, d = x.shape
    E = Wr.shape[0]
    _shape(Wr, "Wr", (E, d))
    _shape(br, "br", (E,))
    idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    lib = _lib.load()
    o, _ = _opts(partitions=partitions)
    _lib.check(lib.mova_route_opts(_ptr(x), _DT[x.dtype], _ptr(Wr), _ptr(br), T, d, E, k, float(scale),
                                   _ptr(idx), _ptr(w), ctypes.byref(o), _stream()), "mova_route")
    return idx, w


def permute(idx: torch.Tensor, E: int):
    """Stable grouping of the (token, slot) pairs by expert:
    dict(counts (E), offsets (E+1), perm (T*k), pos (T*k)), all int32."""
    _need(idx, "idx", (torch.int32,), 2)
    T, k = idx.shape
    dev = idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    pos = torch.empty(T * k, dtype=torch.int32, device=dev)
    nbytes = workspace_size(T, 64, E, k, 128)
    ws = _workspace(nbytes, dev)
    lib = _lib.load()
    _lib.check(lib.mova_permute(_ptr(idx), T, E, k, _ptr(counts), _ptr(offsets), _ptr(perm),
                                _ptr(pos), _ptr(ws), ws.numel(), _stream()), "mova_permute")
    return dict(counts=counts, offsets=offsets, perm=perm, pos=pos, ws=ws)


def _events(events):
    """Array of raw cudaEvent_t handles (or None) for the _ex entry points."""
    if events is None:
        return None
    assert len(events) == _lib.STAGE_EVENTS
    return (ctypes.c_void_p * _lib.STAGE_EVENTS)(*[ctypes.c_void_p(e.cuda_event) for e in events])


def _expert_view(Wv: torch.Tensor, rows: Optional[tuple]):
    """(E, n, stride in rows, base tensor) of the experts' rows a call reads:
    all of Wv, or rows = (row0, count) of every expert (head-parallel slice)."""
    E, n_total, _ = Wv.shape
    if rows is None:
        return E, n_total, 0, Wv
    row0, count = rows
    if not (0 <= row0 and count > 0 and row0 + count <= n_total):
        raise ValueError(f"rows {rows} outside the {n_total} rows of each expert")
    return E, count, n_total, Wv[:, row0:, :]


def head_slice(n_total: int, world: int, rank: int, head_dim: int = 128) -> tuple:
    """(row0, count) of the expert rows -- whole value heads -- that rank
    `rank` of `world` head-parallel ranks computes: the heads are dealt in
    contiguous blocks, the first n_heads % world ranks taking one extra."""
    if n_total % head_dim != 0:
        raise ValueError("n_total must be whole heads")
    heads = n_total // head_dim
    if not 0 <= rank < world or world > heads:
        raise ValueError(f"rank {rank} of {world} over {heads} heads")
    base, extra = divmod(heads, world)
    h0 = rank * base + min(rank, extra)
    nh = base + (1 if rank < extra else 0)
    return h0 * head_dim, nh * head_dim


def value(x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, Wv: torch.Tensor,
          path: str = "auto", ws: Optional[torch.Tensor] = None,
          events=None, rows: Optional[tuple] = None) -> torch.Tensor:
    """Routing-given mixture: v (T, n) in x's dtype.  rows=(row0, count)
    computes only rows [row0, row0+count) of every expert (v is (T, count)),
    reading them in place from the full Wv."""
    _need(x, "x", (torch.float32, torch.bfloat16), 2)
    _need(idx, "idx", (torch.int32, torch.int8), 2)
    _need(w, "w", (torch.float32, torch.float16), 2)
    _need(Wv, "Wv", (x.dtype,), 3)
    T, d = x.shape
    E, n, stride, Wb = _expert_view(Wv, rows)
    k = idx.shape[1]
    _shape(idx, "idx", (T, k))
    _shape(w, "w", (T, k))
    _shape(Wv, "Wv", (E, Wv.shape[1], d))
    v = torch.empty((T, n), dtype=x.dtype, device=x.device)
    nbytes = workspace_size(T, d, E, k, n)
    if ws is None:
        ws = _workspace(nbytes, x.device)
    lib = _lib.load()
    o, _ev = _opts(path, events, stride)
    _lib.check(lib.mova_value_opts(_ptr(x), _DT[x.dtype], _ptr(idx), _DT[idx.dtype], _ptr(w),
                                   _DT[w.dtype], _ptr(Wb), _DT[Wv.dtype], T, d, E, k, n, _ptr(v),
                                   _ptr(ws), ws.numel(), ctypes.byref(o), _stream()),
               "mova_value")
    return v


def attend_workspace_size(L: int, d: int, E: int, k: int, n: int, H: int) -> int:
    return int(_lib.load().mova_attend_workspace_size(L, d, E, k, n, H))


def value_attend(x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, Wv: torch.Tensor,
                 probs: torch.Tensor, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One query token's attention output over L cached positions whose
    values are recomputed from the compact cache (x, idx, w) and never
    stored: o (H, 128) fp32 = sum_l probs[h, l] * V[l, h // G]."""
    _need(x, "x", (torch.bfloat16,), 2)
    _need(idx, "idx", (torch.int32, torch.int8), 2)
    _need(w, "w", (torch.float32, torch.float16), 2)
    _need(Wv, "Wv", (torch.bfloat16,), 3)
    _need(probs, "probs", (torch.float32,), 2)
    L, d = x.shape
    E, n = Wv.shape[0], Wv.shape[1]
    k = idx.shape[1]
    H = probs.shape[0]
    if probs.shape[1] != L:
        raise ValueError("probs: (H, L) for the L cached positions of x")
    _shape(idx, "idx", (L, k))
    _shape(w, "w", (L, k))
    _shape(Wv, "Wv", (E, n, d))
    o = torch.empty((H, 128), dtype=torch.float32, device=x.device)
    lib = _lib.load()
    nbytes = int(lib.mova_attend_workspace_size(L, d, E, k, n, H))
    if ws is None:
        ws = _workspace(nbytes, x.device)
    _lib.check(lib.mova_value_attend(_ptr(x), _ptr(idx), _DT[idx.dtype], _ptr(w), _DT[w.dtype], _ptr(Wv),
                                     L, d, E, k, n, _ptr(probs), H, _ptr(o), _ptr(ws), ws.numel(),
                                     _stream()), "mova_value_attend")
    return o


def value_routed(x: torch.Tensor, Wr: torch.Tensor, br: torch.Tensor, Wv: torch.Tensor,
                 k: int = 4, scale: float = 2.5, return_routing: bool = False,
                 path: str = "auto", ws: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, events=None, rows: Optional[tuple] = None,
                 partitions: int = 0, decode_launches: int = 0,
                 planes: Optional[torch.Tensor] = None):
    """Full value path: v (T, n) in x's dtype [, idx (T, k) int32, w (T, k) fp32].
    rows=(row0, count): only those rows of every expert (a head-parallel
    slice, v is (T, count)); partitions=2: the router's two-partition sum;
    decode_launches=1: decode batches as one persistent kernel (default two);
    planes: the router's bf16 planes from router_planes(Wr), made once."""
    _need(x, "x", (torch.float32, torch.bfloat16), 2)
    _need(Wr, "Wr", (torch.float32,), 2)
    _need(br, "br", (torch.float32,), 1)
    _need(Wv, "Wv", (x.dtype,), 3)
    T, d = x.shape
    E, n, stride, Wb = _expert_view(Wv, rows)
    _shape(Wr, "Wr", (E, d))
    _shape(br, "br", (E,))
    _shape(Wv, "Wv", (E, Wv.shape[1], d))
    dev = x.device
    if out is not None:
        _need(out, "out", (x.dtype,), 2)
        _shape(out, "out", (T, n))
    v = out if out is not None else torch.empty((T, n), dtype=x.dtype, device=dev)
    idx = w = None
    if return_routing:
        idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
    nbytes = workspace_size(T, d, E, k, n)
    if ws is None:
        ws = _workspace(nbytes, dev)
    lib = _lib.load()
    if planes is not None:
        _need(planes, "planes", (torch.bfloat16,), 1)
        if planes.numel() * 2 < int(lib.mova_router_planes_bytes(d)):
            raise ValueError("planes: too small for this d; make them with router_planes(Wr)")
    o, _ev = _opts(path, events, stride, partitions, decode_launches, planes)
    _lib.check(lib.mova_value_routed_opts(_ptr(x), _DT[x.dtype], _ptr(Wr), _ptr(br), _ptr(Wb),
                                          _DT[Wv.dtype], T, d, E, k, n, float(scale), _ptr(v),
                                          _ptr(idx), _ptr(w), _ptr(ws), ws.numel(), ctypes.byref(o),
                                          _stream()), "mova_value_routed")
    if return_routing:
        return v, idx, w
    return v


def _need_host(t: torch.Tensor, name: str, dtypes=None, ndim=None):
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor; pinned memory makes the copy asynchronous")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _host_out(out, shape, dtype, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, pin_memory=True)
    _need_host(out, name, (dtype,), len(shape))
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(out.shape)}, expected {tuple(shape)}")
    return out


def value_routed_host(x: torch.Tensor, Wr: torch.Tensor, br: torch.Tensor, Wv: torch.Tensor,
                      k: int = 4, scale: float = 2.5, out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None, return_routing: bool = False):
    """value_routed for a batch in host memory (mova_value_routed_host): x is a
    CPU tensor (pinned for an asynchronous copy), the weights are on the
    device, and v (and the routing) come back in host tensors, valid once the
    stream has passed the call."""
    _need_host(x, "x", (torch.float32, torch.bfloat16), 2)
    _need(Wr, "Wr", (torch.float32,), 2)
    _need(br, "br", (torch.float32,), 1)
    _need(Wv, "Wv", (x.dtype,), 3)
    T, d = x.shape
    E, n = Wv.shape[0], Wv.shape[1]
    _shape(Wr, "Wr", (E, d))
    _shape(br, "br", (E,))
    _shape(Wv, "Wv", (E, n, d))
    v = _host_out(out, (T, n), x.dtype)
    idx = w = None
    if return_routing:
        idx = torch.empty((T, k), dtype=torch.int32, pin_memory=True)
        w = torch.empty((T, k), dtype=torch.float32, pin_memory=True)
    if ws is None:
        ws = _workspace(workspace_size_host(T, d, E, k, n), Wv.device, stream)
    _lib.check(_lib.load().mova_value_routed_host(
        _ptr(x), _DT[x.dtype], _ptr(Wr), _ptr(br), _ptr(Wv), _DT[Wv.dtype], T, d, E, k, n, float(scale),
        _ptr(v), _ptr(idx), _ptr(w), _ptr(ws), ws.numel(), _stream(stream)), "mova_value_routed_host")
    return (v, idx, w) if return_routing else v


def value_host(x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, Wv: torch.Tensor,
               out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """value for a batch and stored routing in host memory (mova_value_host);
    v comes back in a host tensor, valid once the stream has passed the call."""
    _need_host(x, "x", (torch.float32, torch.bfloat16), 2)
    _need_host(idx, "idx", (torch.int32, torch.int8), 2)
    _need_host(w, "w", (torch.float32, torch.float16), 2)
    _need(Wv, "Wv", (x.dtype,), 3)
    T, d = x.shape
    E, n = Wv.shape[0], Wv.shape[1]
    k = idx.shape[1]
    _shape(idx, "idx", (T, k))
    _shape(w, "w", (T, k))
    _shape(Wv, "Wv", (E, n, d))
    v = _host_out(out, (T, n), x.dtype)
    if ws is None:
        ws = _workspace(workspace_size_host(T, d, E, k, n), Wv.device, stream)
    _lib.check(_lib.load().mova_value_host(
        _ptr(x), _DT[x.dtype], _ptr(idx), _DT[idx.dtype], _ptr(w), _DT[w.dtype], _ptr(Wv), _DT[Wv.dtype],
        T, d, E, k, n, _ptr(v), _ptr(ws), ws.numel(), _stream(stream)), "mova_value_host")
    return v


def value_attend_host(x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, Wv: torch.Tensor,
                      probs: torch.Tensor, out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """value_attend for a compact cache and probabilities in host memory
    (mova_value_attend_host); o (H, 128) fp32 comes back in a host tensor,
    valid once the stream has passed the call."""
    _need_host(x, "x", (torch.bfloat16,), 2)
    _need_host(idx, "idx", (torch.int32, torch.int8), 2)
    _need_host(w, "w", (torch.float32, torch.float16), 2)
    _need_host(probs, "probs", (torch.float32,), 2)
    _need(Wv, "Wv", (torch.bfloat16,), 3)
    L, d = x.shape
    E, n = Wv.shape[0], Wv.shape[1]
    k = idx.shape[1]
    H = probs.shape[0]
    if probs.shape[1] != L:
        raise ValueError("probs: (H, L) for the L cached positions of x")
    _shape(idx, "idx", (L, k))
    _shape(w, "w", (L, k))
    _shape(Wv, "Wv", (E, n, d))
    o = _host_out(out, (H, 128), torch.float32)
    if ws is None:
        ws = _workspace(attend_workspace_size_host(L, d, E, k, n, H), Wv.device, stream)
    _lib.check(_lib.load().mova_value_attend_host(
        _ptr(x), _ptr(idx), _DT[idx.dtype], _ptr(w), _DT[w.dtype], _ptr(Wv), L, d, E, k, n, _ptr(probs), H,
        _ptr(o), _ptr(ws), ws.numel(), _stream(stream)), "mova_value_attend_host")
    return o


# ---- Paged key-value cache ------------------------------------------------------
# Caches are (num_pages, KV heads, page_size, 128) tensors whose pages may lie
# further apart than dense (a part of a larger tensor); tables (requests,
# max_pages) int32, rows possibly a part of longer ones; q, k and v rows of a
# fused projection's output.  Types: fp32 with fp32 caches; bf16 with bf16 or
# float8_e4m3fn caches, the latter with one fp32 scale per KV head.

_CACHE_DT = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float8_e4m3fn: _lib.E4M3}
_CACHE_IO = {torch.float32: torch.float32, torch.bfloat16: torch.bfloat16, torch.float8_e4m3fn: torch.bfloat16}
_STATUS_BYTES = 256
_I32 = torch.int32
_RSQRT_128 = 0.08838834764831845


# mova_pages, packed: the fields of _lib.Pages.
_PAGES = struct.Struct("@QQiiiiqqQQ")


# The checks below are written for the common case to cost little: one test of
# everything, and only if it fails a second look that says what is wrong.

def _on(index: int, **tensors) -> None:
    """Every tensor on CUDA device `index`: the library sees addresses only."""
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _elsewhere(t: torch.Tensor) -> bool:
    """Whether t's device is not the current one (whose stream a call uses)."""
    index = t.get_device()
    if index < 0:
        raise ValueError("the paged calls take CUDA tensors")
    return index != _current_device()


def _vector(t: torch.Tensor, name: str, n: int, index: int, dtype=_I32) -> int:
    """The address of a contiguous vector of n elements on device `index`."""
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} vector of {n}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index:
        _on(index, **{name: t})
    return t.data_ptr()


def _row_stride(t: torch.Tensor, name: str, width: int) -> int:
    """Elements from one row to the next of a tensor whose rows (all dims but
    the first) hold `width` elements in order."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 3 and strides[1:] == (shape[2], 1) and shape[1] * shape[2] == width <= strides[0] and shape[0] > 1:
        return strides[0]
    want = 1
    for size, stride in zip(shape[:0:-1], strides[:0:-1]):
        if stride != want and size != 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        want *= size
    if want != width:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected rows of {width} elements")
    if shape[0] <= 1:
        return width
    if strides[0] < width:
        raise ValueError(f"{name}: rows overlap")
    return strides[0]


def _heads(t: torch.Tensor, name: str, dtype):
    """(rows, heads) of a (rows, heads, 128) tensor."""
    shape = t.shape
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if len(shape) != 3 or shape[2] != 128:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected (rows, heads, 128)")
    return shape[0], shape[1]


def _pages(index: int, k_cache, v_cache=None, k_scale=None, v_scale=None):
    """The packed mova_pages of a cache, and its (num_pages, KV heads)."""
    dtype, shape = k_cache.dtype, k_cache.shape
    if dtype not in _CACHE_IO:
        raise ValueError(f"k_cache: dtype {dtype} not in {tuple(_CACHE_IO)}")
    if len(shape) != 4 or shape[3] != 128:
        raise ValueError(f"k_cache: shape {tuple(shape)}, expected (num_pages, KV heads, page_size, 128)")
    num, kv, page, _ = shape
    k_stride = 0 if k_cache.is_contiguous() else _row_stride(k_cache, "k_cache", kv * page * 128)
    v = v_stride = ks = vs = 0
    if v_cache is not None:
        if v_cache.dtype is not dtype or v_cache.shape != shape:
            raise ValueError(f"v_cache: expected {dtype} of shape {tuple(shape)}")
        v_stride = 0 if v_cache.is_contiguous() else _row_stride(v_cache, "v_cache", kv * page * 128)
        v = v_cache.data_ptr()
        if v_cache.get_device() != index:
            _on(index, v_cache=v_cache)
    if k_scale is not None or v_scale is not None:
        if dtype is not torch.float8_e4m3fn:
            raise ValueError("k_scale, v_scale: only float8_e4m3fn caches have scales")
        ks = 0 if k_scale is None else _vector(k_scale, "k_scale", kv, index, torch.float32)
        vs = 0 if v_scale is None else _vector(v_scale, "v_scale", kv, index, torch.float32)
    if k_cache.get_device() != index:
        _on(index, k_cache=k_cache)
    return _PAGES.pack(k_cache.data_ptr(), v, _CACHE_DT[dtype], num, kv, page, k_stride, v_stride, ks, vs), num, kv


def _table(index: int, table, B: int):
    """(address, row stride, max_pages) of a page table for B requests."""
    shape = table.shape
    if table.dtype is not _I32 or len(shape) != 2 or shape[0] != B:
        raise ValueError(f"table: expected int32 of shape ({B}, max_pages), got {table.dtype} {tuple(shape)}")
    if table.get_device() != index:
        _on(index, table=table)
    width = shape[1]
    return table.data_ptr(), (width if table.is_contiguous() else _row_stride(table, "table", width)), width


def _page_ws(ws, nbytes: int, dev):
    """(address, bytes, stream handle): `ws`, or the current stream's workspace
    on `dev`, the current device.  A call that a graph captures gets one of the
    graph's own memory instead: graphs captured on one stream may be replayed on
    several, and the stream's workspace may grow and move."""
    handle = _raw_stream(dev.index) if _raw_stream is not None else _current_stream_handle()
    if ws is None:
        if _capturing():
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            return ws.data_ptr(), nbytes, handle
        own = _WS.get((dev, handle))
        ws = own.buf if own is not None else None
        if ws is None or ws.numel() < nbytes:
            ws = _workspace(nbytes, dev)
        return ws.data_ptr(), ws.numel(), handle
    _on(dev.index, ws=ws)
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size(), handle


@functools.lru_cache(maxsize=256)
def page_workspace_size(B: int, max_pages: int, kv_heads: int, H: int) -> int:
    """Device workspace of every paged call of these sizes (0: refused)."""
    return int(_lib.load().mova_page_workspace_size(B, max_pages, kv_heads, H))


def page_map(cached: torch.Tensor, added: torch.Tensor, table: torch.Tensor, free_pages: torch.Tensor,
             taken: torch.Tensor, page_size: int, num_pages: int, tokens: int,
             taken_out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """One step's pages and slots from request lengths (mova_page_map):
    (lens (B), starts (B+1), slots (tokens), positions (tokens), taken (1)),
    all int32.  Writes the new pages into `table`; `taken` counts the entries
    of free_pages handed out so far, and the new count goes to taken_out
    (which may be `taken` itself) or to a new tensor.  `tokens` is the size of
    the step's token batch, at least the sum of `added`; slots and positions past
    the last token are -1."""
    if _elsewhere(cached):
        with torch.cuda.device(cached.device):
            return page_map(cached, added, table, free_pages, taken, page_size, num_pages, tokens, taken_out, ws)
    dev, index, B, n_free = cached.device, cached.get_device(), cached.shape[0], free_pages.shape[0]
    p_cached, p_added = _vector(cached, "cached", B, index), _vector(added, "added", B, index)
    p_table, stride, max_pages = _table(index, table, B)
    p_free, p_taken = _vector(free_pages, "free_pages", n_free, index), _vector(taken, "taken", 1, index)
    # The outputs, in one allocation.
    buf = torch.empty(2 * (B + tokens + 1), dtype=_I32, device=dev)
    lens, starts, slots, positions, out = buf.split_with_sizes([B, B + 1, tokens, tokens, 1])
    p_lens = buf.data_ptr()
    p_starts = p_lens + 4 * B
    p_slots = p_starts + 4 * (B + 1)
    p_positions = p_slots + 4 * tokens
    p_out = p_positions + 4 * tokens
    if taken_out is not None:
        out, p_out = taken_out, _vector(taken_out, "taken_out", 1, index)
    p_ws, n_ws, stream = _page_ws(ws, _STATUS_BYTES, dev)
    code = _lib.load().mova_page_map(p_cached, p_added, B, p_table, stride, max_pages, p_free, n_free, p_taken, page_size,
                                     num_pages, tokens, p_lens, p_starts, p_slots, p_positions, p_out, p_ws, n_ws, stream)
    if code:
        _lib.check(code, "mova_page_map")
    return lens, starts, slots, positions, out


def page_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
               ws: Optional[torch.Tensor] = None) -> None:
    """Writes the keys and values of T tokens into the cache at `slots`
    (mova_page_write): k and v (T, KV heads, 128) or (T, KV heads * 128), v as
    value_routed returns it.  Slots of -1 are skipped."""
    if _elsewhere(k):
        with torch.cuda.device(k.device):
            return page_write(k, v, slots, k_cache, v_cache, k_scale, v_scale, ws)
    dev, index, T = k.device, k.get_device(), k.shape[0]
    p, _, kv = _pages(index, k_cache, v_cache, k_scale, v_scale)
    io = _CACHE_IO[k_cache.dtype]
    if k.dtype is not io or v.dtype is not io:
        raise ValueError(f"k, v: {k.dtype}, {v.dtype}; a {k_cache.dtype} cache takes {io}")
    k_stride, v_stride = _row_stride(k, "k", kv * 128), _row_stride(v, "v", kv * 128)
    if v.shape[0] != T:
        raise ValueError(f"v: {v.shape[0]} tokens, expected {T}")
    p_slots = _vector(slots, "slots", T, index)
    if v.get_device() != index:
        _on(index, v=v)
    p_ws, n_ws, stream = _page_ws(ws, _STATUS_BYTES, dev)
    code = _lib.load().mova_page_write(k.data_ptr(), v.data_ptr(), _DT[io], k_stride, v_stride, p_slots, T, p, p_ws, n_ws,
                                       stream)
    if code:
        _lib.check(code, "mova_page_write")


def _bounds(index: int, k_lo, k_hi, want, dtype) -> None:
    for t in (k_lo, k_hi):
        if t.dtype is not dtype or t.shape != want or not t.is_contiguous():
            raise ValueError(f"k_lo, k_hi: expected contiguous {dtype} of shape {tuple(want)}, got {t.dtype} "
                             f"{tuple(t.shape)}")
        if t.get_device() != index:
            _on(index, k_lo=k_lo, k_hi=k_hi)


def page_bounds(k_cache: torch.Tensor, table: torch.Tensor, cached: torch.Tensor, lens: torch.Tensor,
                k_lo: torch.Tensor, k_hi: torch.Tensor, ws: Optional[torch.Tensor] = None) -> None:
    """Updates the per-page key bounds k_lo, k_hi (num_pages, KV heads, 128)
    of the pages that the step from `cached` to `lens` tokens has filled
    (mova_page_bounds)."""
    if _elsewhere(k_cache):
        with torch.cuda.device(k_cache.device):
            return page_bounds(k_cache, table, cached, lens, k_lo, k_hi, ws)
    dev, index, B = k_cache.device, k_cache.get_device(), lens.shape[0]
    p, num, kv = _pages(index, k_cache)
    p_table, stride, max_pages = _table(index, table, B)
    p_cached, p_lens = _vector(cached, "cached", B, index), _vector(lens, "lens", B, index)
    _bounds(index, k_lo, k_hi, (num, kv, 128), k_cache.dtype)
    p_ws, n_ws, stream = _page_ws(ws, _STATUS_BYTES, dev)
    code = _lib.load().mova_page_bounds(p, p_table, stride, max_pages, p_cached, p_lens, B, k_lo.data_ptr(),
                                        k_hi.data_ptr(), p_ws, n_ws, stream)
    if code:
        _lib.check(code, "mova_page_bounds")


def page_select(q: torch.Tensor, k_lo: torch.Tensor, k_hi: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                page_size: int, top: int, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The `top` pages of each request that a bound on the scores ranks first,
    the last page always among them (mova_page_select): (B, KV heads, top)
    int32 page numbers within the request, ascending, then -1.  q (B, H, 128)."""
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return page_select(q, k_lo, k_hi, table, lens, page_size, top, ws)
    dev, index, dtype, shape = q.device, q.get_device(), k_lo.dtype, k_lo.shape
    if dtype not in _CACHE_IO or len(shape) != 3 or shape[2] != 128:
        raise ValueError(f"k_lo: expected (num_pages, KV heads, 128) of a cache's dtype, got {dtype} {tuple(shape)}")
    num, kv, _ = shape
    _bounds(index, k_lo, k_hi, shape, dtype)
    B, H = _heads(q, "q", _CACHE_IO[dtype])
    q_stride = _row_stride(q, "q", H * 128)
    p_table, stride, max_pages = _table(index, table, B)
    p_lens = _vector(lens, "lens", B, index)
    picked = torch.empty(B, kv, top, dtype=_I32, device=dev)
    p = _PAGES.pack(0, 0, _CACHE_DT[dtype], num, kv, page_size, 0, 0, 0, 0)
    p_ws, n_ws, stream = _page_ws(ws, page_workspace_size(B, max_pages, kv, H), dev)
    code = _lib.load().mova_page_select(q.data_ptr(), _DT[q.dtype], q_stride, H, p, k_lo.data_ptr(), k_hi.data_ptr(),
                                        p_table, stride, max_pages, p_lens, B, top, picked.data_ptr(), p_ws, n_ws, stream)
    if code:
        _lib.check(code, "mova_page_select")
    return picked


def page_attend(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                lens: torch.Tensor, scale: Optional[float] = None, picked: Optional[torch.Tensor] = None,
                k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                return_lse: bool = False, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Attention of one new token per request over its cached tokens
    (mova_page_attend): o (B, H, 128) in q's dtype [, lse (B, H) fp32], zeros
    (and -inf) for requests of length 0.  scale defaults to 1 / sqrt(128).
    picked (B, KV heads, top): only these pages, from page_select.  The width
    of `table` bounds the lengths that the call is laid out for: a table no
    wider than the longest request needs is fastest."""
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return page_attend(q, k_cache, v_cache, table, lens, scale, picked, k_scale, v_scale, return_lse, out, ws)
    dev, index = q.device, q.get_device()
    p, _, kv = _pages(index, k_cache, v_cache, k_scale, v_scale)
    B, H = _heads(q, "q", _CACHE_IO[k_cache.dtype])
    q_stride = _row_stride(q, "q", H * 128)
    p_table, stride, max_pages = _table(index, table, B)
    p_lens = _vector(lens, "lens", B, index)
    p_picked = top = p_lse = 0
    if picked is not None:
        if picked.dtype is not _I32 or picked.dim() != 3 or picked.shape[:2] != (B, kv) or not picked.is_contiguous():
            raise ValueError(f"picked: expected contiguous int32 of shape ({B}, {kv}, top), got {picked.dtype} "
                             f"{tuple(picked.shape)}")
        if picked.get_device() != index:
            _on(index, picked=picked)
        p_picked, top = picked.data_ptr(), picked.shape[2]
    if out is None:
        out = torch.empty(B, H, 128, dtype=q.dtype, device=dev)
    elif out.dtype is not q.dtype or out.shape != q.shape or not out.is_contiguous():
        raise ValueError(f"out: expected contiguous {q.dtype} of shape {tuple(q.shape)}")
    else:
        _on(index, out=out)
    if return_lse:
        lse = torch.empty(B, H, dtype=torch.float32, device=dev)
        p_lse = lse.data_ptr()
    p_ws, n_ws, stream = _page_ws(ws, page_workspace_size(B, max_pages, kv, H), dev)
    code = _lib.load().mova_page_attend(q.data_ptr(), _DT[q.dtype], q_stride, H, p, p_table, stride, max_pages, p_lens, B,
                                        _RSQRT_128 if scale is None else scale, p_picked, top, out.data_ptr(), p_lse,
                                        p_ws, n_ws, stream)
    if code:
        _lib.check(code, "mova_page_attend")
    return (out, lse) if return_lse else out


def workspace_parts(T: int, d: int, E: int, k: int, n: int) -> dict:
    """Byte offsets of the routing and grouping a value call leaves in its
    workspace: dict(idx, w, counts, offsets, perm, pos) -> offset."""
    offs = (ctypes.c_size_t * len(_lib.WS_PARTS))()
    _lib.check(_lib.load().mova_workspace_parts(T, d, E, k, n, offs), "mova_workspace_parts")
    return dict(zip(_lib.WS_PARTS, (int(o) for o in offs)))


def grouping(ws: torch.Tensor, T: int, d: int, E: int, k: int, n: int) -> dict:
    """The grouping by expert (counts, offsets, perm, pos; int32 copies) that
    the last value call with these sizes ran on, read from its workspace
    (call after the stream has passed that call)."""
    offs = workspace_parts(T, d, E, k, n)
    size = {"counts": E, "offsets": E + 1, "perm": T * k, "pos": T * k}
    out = {}
    for name, count in size.items():
        o = offs[name]
        out[name] = ws[o:o + 4 * count].view(torch.int32).clone()
    return out


def arm_stream_stall(stall_stage: int, limit_cycles: int) -> None:
    """Test hook: the next weight-streaming launch stops issuing weight copies
    in its first CTA at `stall_stage` and gives up waiting after
    `limit_cycles`, reporting MOVA_ERR_TIMEOUT (mova_selftest_arm_stream_stall)."""
    _lib.check(_lib.load().mova_selftest_arm_stream_stall(int(stall_stage), int(limit_cycles)),
               "mova_selftest_arm_stream_stall")


def get_status(ws: Optional[torch.Tensor] = None, device=None, stream=None):
    """(status name, detail) of the last call on this workspace; without
    `ws`, on the default workspace of `stream` (else of the current stream),
    i.e. of the last call made there without `ws`.  Waits for that stream."""
    if ws is None:
        dev = _devkey(device if device is not None else "cuda")
        handle = int(stream.cuda_stream) if stream is not None else _current_stream_handle()
        entry = _WS.get((dev, handle))
        if entry is None or entry.buf is None:
            raise ValueError(f"no call on {dev} has used the default workspace of this stream")
        ws = entry.buf
    detail = ctypes.c_int32(0)
    code = _lib.load().mova_get_status(_ptr(ws), ctypes.byref(detail), _stream(stream))
    return _lib.STATUS_NAMES.get(code, str(code)), int(detail.value)
