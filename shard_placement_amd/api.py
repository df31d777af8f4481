"""Python binding of libtide: argument marshalling only.

Functions carry the C ABI's names (include/tide.h) and pass torch tensors'
device addresses and the current HIP stream straight through; every step of
the data path runs in the library's HIP kernels (or, for
``tide_ag_place_sdma``, on the DMA engines).  ``Plan`` bundles one layer's
descriptor table (host blob + its device copy) with the tensors it points
at, so that they outlive it.

Operations (Abstract of "The Endgame of FSDP Communication",
weekinpapers.com): the reduce-scatter reads R ranks' per-parameter bf16
gradients in place and writes each rank's fp32 dim-0 shards; the placement
writes a rank-major bf16 gathered buffer into per-parameter tensors.
"""
from __future__ import annotations

import ctypes
from typing import Sequence, Tuple

import numpy as np
import torch

from . import _lib
from ._lib import (TideError, TideGatedBackwardArgs, TideGatedForwardArgs,
                   TideLinearBackwardArgs, TideLinearForwardArgs, TideNormBackwardArgs,
                   TideNormForwardArgs, TideOpts, TidePlanInfo, TideShape, check)

ORDERS = {"fixed": 0, "tree": 1}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
NORMS = {"rms": 0, "layer": 1}


def _shapes(shapes: Sequence[Sequence[int]]):
    arr = (TideShape * max(1, len(shapes)))()
    for i, shp in enumerate(shapes):
        shp = tuple(int(x) for x in shp)
        if len(shp) == 0:
            arr[i].dim0, arr[i].row_numel = 1, 1
        else:
            c = 1
            for d in shp[1:]:
                c *= d
            arr[i].dim0, arr[i].row_numel = shp[0], c
    return arr


def _opts(align: int = 1, rs_tile: int = 0, ag_tile: int = 0, flags: int = -1,
          launch_mib: int = 0) -> TideOpts:
    return TideOpts(int(align), int(rs_tile), int(ag_tile), int(flags), int(launch_mib))


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream))


def tide_desc_geometry(shapes, R: int, align: int = 1) -> Tuple[np.ndarray, np.ndarray, np.ndarray, int]:
    """(chunk rows, shard numel, offsets, slot numel S) from the library."""
    L = _lib.lib()
    P = len(shapes)
    s = np.zeros(max(1, P), np.int64)
    m = np.zeros(max(1, P), np.int64)
    off = np.zeros(max(1, P), np.int64)
    S = ctypes.c_int64(0)
    i64p = ctypes.POINTER(ctypes.c_int64)
    o = _opts(align)
    check(L.tide_desc_geometry(_shapes(shapes), P, int(R), ctypes.byref(o),
                               s.ctypes.data_as(i64p), m.ctypes.data_as(i64p),
                               off.ctypes.data_as(i64p), ctypes.byref(S)), "tide_desc_geometry")
    return s[:P], m[:P], off[:P], int(S.value)


def tide_desc_size(shapes, R: int, align: int = 1, rs_tile: int = 0, ag_tile: int = 0,
                   flags: int = -1, launch_mib: int = 0) -> int:
    n = ctypes.c_size_t(0)
    o = _opts(align, rs_tile, ag_tile, flags, launch_mib)
    check(_lib.lib().tide_desc_size(_shapes(shapes), len(shapes), int(R), ctypes.byref(o),
                                    ctypes.byref(n)), "tide_desc_size")
    return int(n.value)


def tide_desc_build(shapes, R: int, grad_ptrs=None, out_ptrs=None, gathered_ptr=None,
                    full_ptrs=None, align: int = 1, rs_tile: int = 0, ag_tile: int = 0,
                    flags: int = -1, launch_mib: int = 0) -> Tuple[np.ndarray, TidePlanInfo]:
    """Build a host plan blob from raw device addresses (ints).  grad_ptrs is
    rank-major [R*P]; out_ptrs [R]; full_ptrs [P].  Returns (blob, info)."""
    L = _lib.lib()
    P = len(shapes)
    size = tide_desc_size(shapes, R, align, rs_tile, ag_tile, flags, launch_mib)
    blob = np.zeros(size, np.uint8)
    vp = ctypes.c_void_p

    def arr(ptrs, n):
        if ptrs is None:
            return None
        a = (vp * max(1, n))()
        for i, x in enumerate(ptrs):
            a[i] = int(x) if x else None
        return a

    info = TidePlanInfo()
    o = _opts(align, rs_tile, ag_tile, flags, launch_mib)
    st = L.tide_desc_build(_shapes(shapes), P, int(R), ctypes.byref(o), arr(grad_ptrs, R * P),
                           arr(out_ptrs, R), vp(int(gathered_ptr)) if gathered_ptr else None,
                           arr(full_ptrs, P), blob.ctypes.data, blob.nbytes, ctypes.byref(info))
    check(st, "tide_desc_build")
    return blob, info


def tide_plan_rank_tiles(h_plan: np.ndarray, r: int) -> Tuple[int, int]:
    """(tile_begin, tile_count) of output rank r's reduce-scatter tiles."""
    b, c = ctypes.c_int64(0), ctypes.c_int64(0)
    check(_lib.lib().tide_plan_rank_tiles(h_plan.ctypes.data, int(r), ctypes.byref(b), ctypes.byref(c)),
          "tide_plan_rank_tiles")
    return int(b.value), int(c.value)


def tide_rs_bf16_to_fp32(h_plan: np.ndarray, d_plan: torch.Tensor, order: int = 0,
                         max_workgroups: int = 0, stream=None) -> None:
    check(_lib.lib().tide_rs_bf16_to_fp32(h_plan.ctypes.data, d_plan.data_ptr(), int(order),
                                          int(max_workgroups), _stream(stream)),
          "tide_rs_bf16_to_fp32")


def tide_rs_bf16_to_fp32_tiles(h_plan: np.ndarray, d_plan: torch.Tensor, order: int,
                               tile_begin: int, tile_count: int, max_workgroups: int = 0,
                               stream=None) -> None:
    check(_lib.lib().tide_rs_bf16_to_fp32_tiles(h_plan.ctypes.data, d_plan.data_ptr(), int(order),
                                                int(tile_begin), int(tile_count),
                                                int(max_workgroups), _stream(stream)),
          "tide_rs_bf16_to_fp32_tiles")


def tide_rs_bf16_to_fp32_streams(h_plan: np.ndarray, d_plan: torch.Tensor, streams,
                                 order: int = 0, max_workgroups: int = 0) -> None:
    """The reduce-scatter's launches dealt over ``streams`` in turn (the
    caller orders the streams against its other work)."""
    arr = (ctypes.c_void_p * len(streams))(*[int(s.cuda_stream) for s in streams])
    check(_lib.lib().tide_rs_bf16_to_fp32_streams(h_plan.ctypes.data, d_plan.data_ptr(), int(order),
                                                  int(max_workgroups), arr, len(streams)),
          "tide_rs_bf16_to_fp32_streams")


def tide_rs_bf16_to_fp32_census(h_plan: np.ndarray, d_plan: torch.Tensor, census: torch.Tensor,
                                order: int = 0, max_workgroups: int = 0, stream=None) -> None:
    if census.dtype != torch.int32 or census.device.type != "cuda" or not census.is_contiguous():
        raise TideError(-6, "census must be a contiguous int32 GPU tensor")
    check(_lib.lib().tide_rs_bf16_to_fp32_census(h_plan.ctypes.data, d_plan.data_ptr(), int(order),
                                                 int(max_workgroups), census.data_ptr(),
                                                 census.numel(), _stream(stream)),
          "tide_rs_bf16_to_fp32_census")


def tide_rs_bf16_to_fp32_trace(h_plan: np.ndarray, d_plan: torch.Tensor, census: torch.Tensor,
                               stamps: torch.Tensor, order: int = 0, max_workgroups: int = 0,
                               stream=None) -> None:
    """The census call that also records each tile's start and end on the
    GPU's real-time counter (stamps: int64, two per tile)."""
    if census.dtype != torch.int32 or census.device.type != "cuda" or not census.is_contiguous():
        raise TideError(-6, "census must be a contiguous int32 GPU tensor")
    if stamps.dtype != torch.int64 or stamps.device.type != "cuda" or not stamps.is_contiguous():
        raise TideError(-6, "stamps must be a contiguous int64 GPU tensor")
    n = min(census.numel(), stamps.numel() // 2)
    check(_lib.lib().tide_rs_bf16_to_fp32_trace(h_plan.ctypes.data, d_plan.data_ptr(), int(order),
                                                int(max_workgroups), census.data_ptr(),
                                                stamps.data_ptr(), n, _stream(stream)),
          "tide_rs_bf16_to_fp32_trace")


def tide_ag_place(h_plan: np.ndarray, d_plan: torch.Tensor, max_workgroups: int = 0,
                  stream=None) -> None:
    check(_lib.lib().tide_ag_place(h_plan.ctypes.data, d_plan.data_ptr(), int(max_workgroups),
                                   _stream(stream)), "tide_ag_place")


def tide_ag_place_sdma(h_plan: np.ndarray, engine_only: bool = True, stream=None) -> None:
    check(_lib.lib().tide_ag_place_sdma(h_plan.ctypes.data, 1 if engine_only else 0,
                                        _stream(stream)), "tide_ag_place_sdma")


def tide_ag_place_sdma_streams(h_plan: np.ndarray, streams) -> None:
    arr = (ctypes.c_void_p * len(streams))(*[int(s.cuda_stream) for s in streams])
    check(_lib.lib().tide_ag_place_sdma_streams(h_plan.ctypes.data, arr, len(streams)),
          "tide_ag_place_sdma_streams")


def tide_ag_place_dma(h_plan: np.ndarray, stream=None) -> None:
    """Placement on the DMA engines (ROCr engine-pinned copies); returns
    when the copies are done."""
    check(_lib.lib().tide_ag_place_dma(h_plan.ctypes.data, _stream(stream)), "tide_ag_place_dma")


def tide_dma_engine_count() -> int:
    n = ctypes.c_int32(0)
    check(_lib.lib().tide_dma_engine_count(ctypes.byref(n)), "tide_dma_engine_count")
    return int(n.value)


def tide_rs_stage_dma(h_plan: np.ndarray, h_stage: np.ndarray, slot_stride: int,
                      stream=None) -> None:
    """Phase 1 of the copy-engine-staged reduce-scatter; h_stage: uint64
    array of R device addresses.  Returns when the copies are done."""
    check(_lib.lib().tide_rs_stage_dma(h_plan.ctypes.data, h_stage.ctypes.data, int(slot_stride),
                                       _stream(stream)), "tide_rs_stage_dma")


def tide_rs_fold_staged(h_plan: np.ndarray, d_plan: torch.Tensor, order: int,
                        h_stage: np.ndarray, d_stage: torch.Tensor, slot_stride: int,
                        max_workgroups: int = 0, stream=None) -> None:
    """Phase 2: fold the staged slots into the fp32 arenas (asynchronous)."""
    check(_lib.lib().tide_rs_fold_staged(h_plan.ctypes.data, d_plan.data_ptr(), int(order),
                                         h_stage.ctypes.data, d_stage.data_ptr(),
                                         int(slot_stride), int(max_workgroups), _stream(stream)),
          "tide_rs_fold_staged")


def tide_rs_tiles_to_stage(h_plan: np.ndarray, d_plan: torch.Tensor, tile_begin: int,
                           tile_count: int, stage: torch.Tensor, max_workgroups: int = 0,
                           stream=None) -> None:
    """Pipeline phase 1: reduce tiles [tile_begin, +tile_count) into the
    dense fp32 staging chunk ``stage``."""
    _require(stage, torch.float32, "stage")
    check(_lib.lib().tide_rs_tiles_to_stage(h_plan.ctypes.data, d_plan.data_ptr(), int(tile_begin),
                                            int(tile_count), stage.data_ptr(), stage.numel(),
                                            int(max_workgroups), _stream(stream)),
          "tide_rs_tiles_to_stage")


def tide_rs_stage_to_shards(h_plan: np.ndarray, d_plan: torch.Tensor, tile_begin: int,
                            tile_count: int, stage: torch.Tensor, max_workgroups: int = 0,
                            stream=None) -> None:
    """Pipeline phase 2: move a staging chunk's results into the arenas."""
    _require(stage, torch.float32, "stage")
    check(_lib.lib().tide_rs_stage_to_shards(h_plan.ctypes.data, d_plan.data_ptr(), int(tile_begin),
                                             int(tile_count), stage.data_ptr(), stage.numel(),
                                             int(max_workgroups), _stream(stream)),
          "tide_rs_stage_to_shards")


def tide_rs_stage_to_shards_sdma(h_plan: np.ndarray, tile_begin: int, tile_count: int,
                                 stage: torch.Tensor, stream=None) -> None:
    """Pipeline phase 2 on the copy engines (stream-ordered copies)."""
    _require(stage, torch.float32, "stage")
    check(_lib.lib().tide_rs_stage_to_shards_sdma(h_plan.ctypes.data, int(tile_begin),
                                                  int(tile_count), stage.data_ptr(), stage.numel(),
                                                  _stream(stream)),
          "tide_rs_stage_to_shards_sdma")


def tide_rs_two_phase_noalloc(h_plan: np.ndarray, d_plan: torch.Tensor, tile_begin: int,
                              tile_count: int, max_workgroups: int = 0, stream=None) -> None:
    """Both pipeline phases over tiles [tile_begin, +tile_count) through the
    library's own staging array (no allocation by anyone; at most
    TIDE_SCRATCH_BYTES of staging per call)."""
    check(_lib.lib().tide_rs_two_phase_noalloc(h_plan.ctypes.data, d_plan.data_ptr(),
                                               int(tile_begin), int(tile_count),
                                               int(max_workgroups), _stream(stream)),
          "tide_rs_two_phase_noalloc")


def tide_stream_create_cu_limited(n_cu: int) -> torch.cuda.ExternalStream:
    """A torch stream wrapping a HIP stream confined to the first n_cu CUs.
    Release it with tide_stream_destroy."""
    h = ctypes.c_void_p(0)
    check(_lib.lib().tide_stream_create_cu_limited(int(n_cu), ctypes.byref(h)),
          "tide_stream_create_cu_limited")
    return torch.cuda.ExternalStream(int(h.value))


def tide_stream_create_cu_range(first_cu: int, n_cu: int) -> torch.cuda.ExternalStream:
    """A torch stream wrapping a HIP stream confined to CU mask bits
    [first_cu, first_cu + n_cu).  Release it with tide_stream_destroy."""
    h = ctypes.c_void_p(0)
    check(_lib.lib().tide_stream_create_cu_range(int(first_cu), int(n_cu), ctypes.byref(h)),
          "tide_stream_create_cu_range")
    return torch.cuda.ExternalStream(int(h.value))


def tide_pipeline_create(depth: int, phase2_cus: int = 0) -> int:
    """Handle of a two-phase pipeline object (two streams, per-slot events)
    on the current device; release it with tide_pipeline_destroy."""
    h = ctypes.c_void_p(0)
    check(_lib.lib().tide_pipeline_create(int(depth), int(phase2_cus), ctypes.byref(h)),
          "tide_pipeline_create")
    return int(h.value)


def tide_pipeline_run(handle: int, h_plan: np.ndarray, d_plan: torch.Tensor, chunk_tiles: int,
                      ring: torch.Tensor, phase2: int = 0, stream=None) -> None:
    """The whole reduce-scatter through the pipeline, ordered on ``stream``
    (default: the current stream)."""
    _require(ring, torch.float32, "ring")
    check(_lib.lib().tide_pipeline_run(ctypes.c_void_p(handle), h_plan.ctypes.data,
                                       d_plan.data_ptr(), int(chunk_tiles), ring.data_ptr(),
                                       ring.numel(), int(phase2), _stream(stream)),
          "tide_pipeline_run")


def tide_pipeline_destroy(handle: int) -> None:
    check(_lib.lib().tide_pipeline_destroy(ctypes.c_void_p(handle)), "tide_pipeline_destroy")


def tide_stream_destroy(stream) -> None:
    check(_lib.lib().tide_stream_destroy(ctypes.c_void_p(int(stream.cuda_stream))),
          "tide_stream_destroy")


def _require(t: torch.Tensor, dtype, what: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if t.dtype != dtype:
        raise TideError(-6, "%s has dtype %s, expected %s" % (what, t.dtype, dtype))
    if t.device.type != "cuda":
        raise TideError(-6, "%s is on %s, expected a GPU tensor" % (what, t.device))
    if not t.is_contiguous():
        raise TideError(-6, "%s is not contiguous" % what)


# What torch.cuda.current_stream / current_device wrap, without the objects.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _on_device(index: int, stream, call, *args):
    """call(stream handle, *args) with device ``index`` current and ``stream``
    (default: the device's current stream) the one that allocations belong to."""
    if stream is None and index == _current_device():
        return call(_raw_stream(index), *args)
    if stream is not None and stream.device_index != index:
        # entering it would make its device current, and the kernels run there
        raise TideError(-1, "stream belongs to cuda:%d, the tensors to cuda:%d"
                        % (stream.device_index, index))
    with torch.cuda.device(index):
        if stream is None:
            return call(_raw_stream(index), *args)
        with torch.cuda.stream(stream):
            return call(int(stream.cuda_stream), *args)


def _index(t: torch.Tensor, what: str) -> int:
    """Index of the GPU that the bf16 matrix ``t`` is on."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if t.dtype != torch.bfloat16:
        raise TideError(-6, "%s has dtype %s, expected %s" % (what, t.dtype, torch.bfloat16))
    if t.dim() != 2:
        raise TideError(-1, "%s has %d dimensions, expected 2" % (what, t.dim()))
    if not t.is_cuda:
        raise TideError(-6, "%s is on %s, expected a GPU" % (what, t.device))
    return t.get_device()


def _rows(t: torch.Tensor, what: str):
    """(address, row distance) of a matrix whose rows may lie apart but are
    contiguous themselves."""
    rows, cols = t.shape
    ld, one = t.stride()
    if rows <= 1:
        ld = cols
    if one != 1 and cols > 1:
        raise TideError(-6, "%s has rows that are not contiguous" % what)
    if ld < cols:
        raise TideError(-6, "%s has rows that share memory" % what)
    return t.data_ptr(), ld


def _no_graph(t: torch.Tensor, what: str) -> None:
    """The layer calls are not recorded by autograd: a tensor whose gradient it
    would follow through them is refused, not detached without a word."""
    if t.requires_grad and torch.is_grad_enabled():
        raise TideError(-6, "%s requires a gradient that autograd would not see: detach it, or call "
                        "under torch.no_grad()" % what)


def _matrix(t: torch.Tensor, rows: int, cols: int, what: str, index: int):
    """The same of a bf16 [rows, cols] matrix on GPU ``index``."""
    if _index(t, what) != index:
        raise TideError(-6, "%s is on %s, expected cuda:%d" % (what, t.device, index))
    if t.shape != (rows, cols):
        raise TideError(-1, "%s is %s, expected [%d, %d]" % (what, list(t.shape), rows, cols))
    _no_graph(t, what)
    return _rows(t, what)


def _whole(t: torch.Tensor, shape, what: str, index: int) -> int:
    """Address of a contiguous bf16 tensor of this shape on GPU ``index``."""
    _require(t, torch.bfloat16, what)
    if t.shape != shape:
        raise TideError(-1, "%s is %s, expected %s" % (what, list(t.shape), list(shape)))
    if t.get_device() != index:
        raise TideError(-6, "%s is on %s, expected cuda:%d" % (what, t.device, index))
    return t.data_ptr()


def _kept(t: torch.Tensor, rows: int, cols: int, what: str, index: int) -> int:
    """Address of a checkpoint of a [rows, cols] matrix (a flat uint8 tensor)."""
    _require(t, torch.uint8, what)
    if t.get_device() != index:
        raise TideError(-6, "%s is on %s, expected cuda:%d" % (what, t.device, index))
    need = rows * (-(-cols // 32)) * 33
    if t.numel() < need:
        raise TideError(-1, "%s holds %d bytes, need %d" % (what, t.numel(), need))
    return t.data_ptr()


def _act(act: str) -> int:
    if act not in ACTS:
        raise TideError(-1, "act is %r, expected one of %s" % (act, ", ".join(ACTS)))
    return ACTS[act]


def _workspace(query, args, index):
    """(tensor, address, bytes) of the call's workspace.  It is taken from
    torch's allocator for each call: calls on different streams, or captured
    into different graphs, never share one."""
    n = ctypes.c_size_t(0)
    status = query(ctypes.byref(args), ctypes.byref(n))
    if status:
        check(status, query.__name__)
    if not n.value:
        return None, None, 0
    t = torch.empty(n.value, dtype=torch.uint8, device=index)
    return t, t.data_ptr(), n.value


def tide_act8_bytes(rows: int, cols: int) -> int:
    """Bytes of an 8-bit checkpoint of a [rows, cols] matrix."""
    n = ctypes.c_size_t(0)
    check(_lib.lib().tide_act8_bytes(int(rows), int(cols), ctypes.byref(n)), "tide_act8_bytes")
    return int(n.value)


def _pack_on(s, px, ldx, rows, cols, pk):
    check(_lib.lib().tide_act8_pack(px, ldx, rows, cols, pk, s), "tide_act8_pack")


def _unpack_on(s, pk, rows, cols, px, ldx):
    check(_lib.lib().tide_act8_unpack(pk, rows, cols, px, ldx, s), "tide_act8_unpack")


def tide_act8_pack(x: torch.Tensor, kept: torch.Tensor, stream=None) -> None:
    """Write the checkpoint of the bf16 matrix ``x`` into ``kept`` (uint8)."""
    index = _index(x, "x")
    rows, cols = x.shape
    px, ldx = _rows(x, "x")
    _on_device(index, stream, _pack_on, px, ldx, rows, cols,
               _kept(kept, rows, cols, "kept", index))


def tide_act8_unpack(kept: torch.Tensor, x: torch.Tensor, stream=None) -> None:
    """Write the values of the checkpoint ``kept`` into the bf16 matrix ``x``."""
    index = _index(x, "x")
    rows, cols = x.shape
    px, ldx = _rows(x, "x")
    _on_device(index, stream, _unpack_on, _kept(kept, rows, cols, "kept", index), rows, cols, px,
               ldx)


def _forward_on(s, a, y, index):
    if y is None:
        y = torch.empty(a.tokens, a.out_features, dtype=torch.bfloat16, device=index)
        a.y, a.ldy = y.data_ptr(), a.out_features
    L = _lib.lib()
    ws, ptr, n = _workspace(L.tide_linear_forward_workspace, a, index)
    check(L.tide_linear_forward(ctypes.byref(a), ptr, n, s), "tide_linear_forward")
    return y


def tide_linear_forward(x: torch.Tensor, weight: torch.Tensor, y: torch.Tensor = None, bias=None,
                        residual=None, act: str = "none", z_kept=None, stream=None) -> torch.Tensor:
    """y = act(x weight^T + bias) + residual; z_kept (uint8), where given,
    receives the checkpoint of act's argument.  Returns y (allocated when not
    given).  Nothing is recorded by autograd (tide_linear_backward is the
    gradient): x, residual and y may not require one in grad mode."""
    index = _index(x, "x")
    _no_graph(x, "x")
    T, K = x.shape
    if weight.dim() != 2:
        raise TideError(-1, "weight has %d dimensions, expected 2" % weight.dim())
    N = weight.shape[0]
    px, ldx = _rows(x, "x")
    a = TideLinearForwardArgs(T, N, K, _act(act), 0, px, ldx,
                              _whole(weight, (N, K), "weight", index))
    if bias is not None:
        a.bias = _whole(bias, (N,), "bias", index)
    if residual is not None:
        a.residual, a.ldr = _matrix(residual, T, N, "residual", index)
    if y is not None:
        a.y, a.ldy = _matrix(y, T, N, "y", index)
    if z_kept is not None:
        a.z_kept = _kept(z_kept, T, N, "z_kept", index)
    return _on_device(index, stream, _forward_on, a, y, index)


def _backward_on(s, a, dx, index):
    if dx is True:
        dx = torch.empty(a.tokens, a.in_features, dtype=torch.bfloat16, device=index)
        a.dx, a.lddx = dx.data_ptr(), a.in_features
    L = _lib.lib()
    ws, ptr, n = _workspace(L.tide_linear_backward_workspace, a, index)
    check(L.tide_linear_backward(ctypes.byref(a), ptr, n, s), "tide_linear_backward")
    return dx


def tide_linear_backward(dy: torch.Tensor, in_features: int, weight=None, x_kept=None,
                         z_kept=None, act: str = "none", dx=None, dweight=None, dbias=None,
                         stream=None):
    """The gradients that are given: dx = dz weight, dweight = dz^T x, dbias =
    the sum of dz over the tokens, dz = dy act'(z).  dx=True allocates it.
    Returns dx."""
    index = _index(dy, "dy")
    _no_graph(dy, "dy")
    T, N = dy.shape
    K = int(in_features)
    pdy, lddy = _rows(dy, "dy")
    a = TideLinearBackwardArgs(T, N, K, _act(act), 0, pdy, lddy)
    if a.act:
        if z_kept is None:
            raise TideError(-1, "act %r needs the checkpoint of its argument" % act)
        a.z_kept = _kept(z_kept, T, N, "z_kept", index)
    if dx is not None:
        if weight is None:
            raise TideError(-1, "dx needs the weight")
        a.weight = _whole(weight, (N, K), "weight", index)
        if dx is not True:
            a.dx, a.lddx = _matrix(dx, T, K, "dx", index)
    if dweight is not None:
        if x_kept is None:
            raise TideError(-1, "dweight needs the checkpoint of x")
        a.x_kept = _kept(x_kept, T, K, "x_kept", index)
        a.dweight = _whole(dweight, (N, K), "dweight", index)
    if dbias is not None:
        a.dbias = _whole(dbias, (N,), "dbias", index)
    return _on_device(index, stream, _backward_on, a, dx, index)


def _norm_kind(kind: str) -> int:
    if kind not in NORMS:
        raise TideError(-1, "kind is %r, expected one of %s" % (kind, ", ".join(NORMS)))
    return NORMS[kind]


def _norm_forward_on(s, a, y, index):
    if y is None:
        y = torch.empty(a.rows, a.cols, dtype=torch.bfloat16, device=index)
        a.y, a.ldy = y.data_ptr(), a.cols
    check(_lib.lib().tide_norm_forward(ctypes.byref(a), s), "tide_norm_forward")
    return y


def tide_norm_forward(x: torch.Tensor, weight: torch.Tensor, y: torch.Tensor = None, bias=None,
                      kind: str = "rms", eps: float = 1e-6, x_kept=None, y_kept=None,
                      stream=None) -> torch.Tensor:
    """y = (x - mean) / sqrt(var + eps) weight + bias for each row ("layer"), or
    with mean 0 and the mean square ("rms"); x_kept and y_kept (uint8), where
    given, receive the checkpoints of x and y.  Returns y (allocated when not
    given).  Nothing is recorded by autograd (tide_norm_backward is the
    gradient): x and y may not require one in grad mode."""
    index = _index(x, "x")
    _no_graph(x, "x")
    T, C = x.shape
    px, ldx = _rows(x, "x")
    a = TideNormForwardArgs(T, C, _norm_kind(kind), eps, px, ldx, _whole(weight, (C,), "weight", index))
    if bias is not None:
        a.bias = _whole(bias, (C,), "bias", index)
    if y is not None:
        a.y, a.ldy = _matrix(y, T, C, "y", index)
    if x_kept is not None:
        a.x_kept = _kept(x_kept, T, C, "x_kept", index)
    if y_kept is not None:
        a.y_kept = _kept(y_kept, T, C, "y_kept", index)
    return _on_device(index, stream, _norm_forward_on, a, y, index)


def _norm_backward_on(s, a, dx, index):
    if dx is True:
        dx = torch.empty(a.rows, a.cols, dtype=torch.bfloat16, device=index)
        a.dx, a.lddx = dx.data_ptr(), a.cols
    L = _lib.lib()
    ws, ptr, n = _workspace(L.tide_norm_backward_workspace, a, index)
    check(L.tide_norm_backward(ctypes.byref(a), ptr, n, s), "tide_norm_backward")
    return dx


def tide_norm_backward(dy: torch.Tensor, x=None, x_kept=None, weight=None, kind: str = "rms",
                       eps: float = 1e-6, add=None, dx=None, dweight=None, dbias=None,
                       stream=None):
    """The gradients that are given, from x in bf16 or its checkpoint x_kept: dx
    (plus ``add``), dweight = the sum of dy n over the rows, n the normalised x,
    dbias = the sum of dy.  dx=True allocates it; dx may be add itself.  Returns
    dx."""
    index = _index(dy, "dy")
    _no_graph(dy, "dy")
    T, C = dy.shape
    pdy, lddy = _rows(dy, "dy")
    a = TideNormBackwardArgs(T, C, _norm_kind(kind), eps, pdy, lddy)
    if x is not None:
        a.x, a.ldx = _matrix(x, T, C, "x", index)
    if x_kept is not None:
        if x is not None:
            raise TideError(-1, "x and x_kept are given: one of them is what forward read")
        a.x_kept = _kept(x_kept, T, C, "x_kept", index)
    if x is None and x_kept is None and not (dx is None and dweight is None):
        raise TideError(-1, "dx and dweight need x or its checkpoint")
    if dx is not None:
        if weight is None:
            raise TideError(-1, "dx needs the weight")
        a.weight = _whole(weight, (C,), "weight", index)
        if add is not None:
            a.add, a.ldadd = _matrix(add, T, C, "add", index)
        if dx is not True:
            a.dx, a.lddx = _matrix(dx, T, C, "dx", index)
    elif add is not None:
        raise TideError(-1, "add is added to dx, which is not asked for")
    if dweight is not None:
        a.dweight = _whole(dweight, (C,), "dweight", index)
    if dbias is not None:
        a.dbias = _whole(dbias, (C,), "dbias", index)
    return _on_device(index, stream, _norm_backward_on, a, dx, index)


def _gated_forward_on(s, a, h, index):
    if h is None:
        h = torch.empty(a.tokens, a.out_features, dtype=torch.bfloat16, device=index)
        a.h, a.ldh = h.data_ptr(), a.out_features
    L = _lib.lib()
    ws, ptr, n = _workspace(L.tide_gated_forward_workspace, a, index)
    check(L.tide_gated_forward(ctypes.byref(a), ptr, n, s), "tide_gated_forward")
    return h


def tide_gated_forward(x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                       h: torch.Tensor = None, gate_bias=None, up_bias=None, act: str = "silu",
                       g_kept=None, u_kept=None, h_kept=None, stream=None) -> torch.Tensor:
    """h = act(g) u, g = x gate^T + gate_bias, u = x up^T + up_bias; g_kept,
    u_kept and h_kept (uint8), where given, receive their checkpoints.  Returns
    h (allocated when not given).  Nothing is recorded by autograd
    (tide_gated_backward is the gradient): x and h may not require one in grad
    mode."""
    index = _index(x, "x")
    _no_graph(x, "x")
    T, K = x.shape
    if gate.dim() != 2:
        raise TideError(-1, "gate has %d dimensions, expected 2" % gate.dim())
    N = gate.shape[0]
    px, ldx = _rows(x, "x")
    a = TideGatedForwardArgs(T, N, K, _act(act), 0, px, ldx, _whole(gate, (N, K), "gate", index),
                             _whole(up, (N, K), "up", index))
    if gate_bias is not None:
        a.gate_bias = _whole(gate_bias, (N,), "gate_bias", index)
    if up_bias is not None:
        a.up_bias = _whole(up_bias, (N,), "up_bias", index)
    if h is not None:
        a.h, a.ldh = _matrix(h, T, N, "h", index)
    for name, kept in (("g_kept", g_kept), ("u_kept", u_kept), ("h_kept", h_kept)):
        if kept is not None:
            setattr(a, name, _kept(kept, T, N, name, index))
    return _on_device(index, stream, _gated_forward_on, a, h, index)


def _gated_backward_on(s, a, dx, index):
    if dx is True:
        dx = torch.empty(a.tokens, a.in_features, dtype=torch.bfloat16, device=index)
        a.dx, a.lddx = dx.data_ptr(), a.in_features
    L = _lib.lib()
    ws, ptr, n = _workspace(L.tide_gated_backward_workspace, a, index)
    check(L.tide_gated_backward(ctypes.byref(a), ptr, n, s), "tide_gated_backward")
    return dx


def tide_gated_backward(dh: torch.Tensor, in_features: int, g_kept: torch.Tensor,
                        u_kept: torch.Tensor, gate=None, up=None, x_kept=None, act: str = "silu",
                        dx=None, dgate=None, dup=None, dgate_bias=None, dup_bias=None, stream=None):
    """The gradients that are given, with dg = dh u act'(g) and du = dh act(g):
    dx = dg gate + du up, dgate = dg^T x and dup = du^T x (both or neither),
    dgate_bias and dup_bias = the sums of dg and du over the tokens.  dx=True
    allocates it.  Returns dx."""
    index = _index(dh, "dh")
    _no_graph(dh, "dh")
    T, N = dh.shape
    K = int(in_features)
    pdh, lddh = _rows(dh, "dh")
    a = TideGatedBackwardArgs(T, N, K, _act(act), 0, pdh, lddh)
    a.g_kept = _kept(g_kept, T, N, "g_kept", index)
    a.u_kept = _kept(u_kept, T, N, "u_kept", index)
    if dx is not None:
        if gate is None or up is None:
            raise TideError(-1, "dx needs gate and up")
        a.gate, a.up = _whole(gate, (N, K), "gate", index), _whole(up, (N, K), "up", index)
        if dx is not True:
            a.dx, a.lddx = _matrix(dx, T, K, "dx", index)
    if (dgate is None) != (dup is None):
        raise TideError(-1, "dgate and dup are computed together")
    if dgate is not None:
        if x_kept is None:
            raise TideError(-1, "dgate and dup need the checkpoint of x")
        a.x_kept = _kept(x_kept, T, K, "x_kept", index)
        a.dgate, a.dup = _whole(dgate, (N, K), "dgate", index), _whole(dup, (N, K), "dup", index)
    if dgate_bias is not None:
        a.dgate_bias = _whole(dgate_bias, (N,), "dgate_bias", index)
    if dup_bias is not None:
        a.dup_bias = _whole(dup_bias, (N,), "dup_bias", index)
    return _on_device(index, stream, _gated_backward_on, a, dx, index)


class Plan:
    """One layer's descriptor table.

    grads:    R lists of P bf16 tensors (rank q's per-parameter gradients);
    out:      R fp32 tensors of >= S elements (each rank's shard arena);
    gathered: one bf16 tensor of >= R*S elements (rank-major slots);
    full:     P bf16 tensors (the per-parameter full tensors).
    Either pair may be omitted.  Shapes come from ``shapes`` (torch-style).
    """

    def __init__(self, shapes, R: int, grads=None, out=None, gathered=None, full=None,
                 align: int = 1, rs_tile: int = 0, ag_tile: int = 0, flags: int = -1,
                 launch_mib: int = 0):
        self.shapes = [tuple(int(d) for d in s) for s in shapes]
        self.R = int(R)
        self.P = len(self.shapes)
        _, self.m, self.off, self.S = tide_desc_geometry(self.shapes, self.R, align)
        numels = [int(np.prod(s)) if len(s) else 1 for s in self.shapes]
        device = None
        grad_ptrs = out_ptrs = full_ptrs = None
        gptr = None
        if grads is not None:
            if out is None or len(grads) != self.R or len(out) != self.R:
                raise TideError(-1, "need R gradient lists and R output arenas")
            grad_ptrs = []
            for q, gl in enumerate(grads):
                if len(gl) != self.P:
                    raise TideError(-1, "rank %d has %d gradients, expected %d" % (q, len(gl), self.P))
                for p, g in enumerate(gl):
                    _require(g, torch.bfloat16, "grads[%d][%d]" % (q, p))
                    if g.numel() != numels[p]:
                        raise TideError(-1, "grads[%d][%d] has %d elements, expected %d"
                                        % (q, p, g.numel(), numels[p]))
                    grad_ptrs.append(g.data_ptr() if g.numel() else 0)
                    device = g.device
            out_ptrs = []
            for r, o in enumerate(out):
                _require(o, torch.float32, "out[%d]" % r)
                if o.numel() < self.S:
                    raise TideError(-1, "out[%d] holds %d floats, need S=%d" % (r, o.numel(), self.S))
                out_ptrs.append(o.data_ptr())
                device = o.device
        if gathered is not None:
            if full is None or len(full) != self.P:
                raise TideError(-1, "need P full tensors with the gathered buffer")
            _require(gathered, torch.bfloat16, "gathered")
            if gathered.numel() < self.R * self.S:
                raise TideError(-1, "gathered holds %d elements, need R*S=%d"
                                % (gathered.numel(), self.R * self.S))
            gptr = gathered.data_ptr()
            full_ptrs = []
            for p, f in enumerate(full):
                _require(f, torch.bfloat16, "full[%d]" % p)
                if f.numel() != numels[p]:
                    raise TideError(-1, "full[%d] has %d elements, expected %d" % (p, f.numel(), numels[p]))
                full_ptrs.append(f.data_ptr() if f.numel() else 0)
            device = gathered.device
        if device is None:
            raise TideError(-1, "a plan needs gradients or a gathered buffer")
        self.blob, self.info = tide_desc_build(self.shapes, self.R, grad_ptrs, out_ptrs, gptr,
                                               full_ptrs, align, rs_tile, ag_tile, flags,
                                               launch_mib)
        used = int(self.info.blob_bytes)
        self.blob = self.blob[:used].copy()
        self.d_blob = torch.from_numpy(self.blob).to(device)
        self._keep = (grads, out, gathered, full)

    def rs(self, order: str = "fixed", max_workgroups: int = 0, stream=None) -> None:
        tide_rs_bf16_to_fp32(self.blob, self.d_blob, ORDERS[order], max_workgroups, stream)

    def rs_streams(self, streams, order: str = "fixed", max_workgroups: int = 0,
                   stream=None) -> None:
        """The reduce-scatter with its launches dealt over ``stream`` (default:
        the current stream) and the extra ``streams`` in turn, ordered after
        ``stream``'s earlier work and before its later work (events)."""
        main = stream if stream is not None else torch.cuda.current_stream()
        start = torch.cuda.Event()
        start.record(main)
        for s in streams:
            s.wait_event(start)
        tide_rs_bf16_to_fp32_streams(self.blob, self.d_blob, [main] + list(streams),
                                     ORDERS[order], max_workgroups)
        for s in streams:
            done = torch.cuda.Event()
            done.record(s)
            main.wait_event(done)

    def rs_chunked(self, chunk_tiles: int, order: str = "fixed", max_workgroups: int = 0,
                   stream=None) -> int:
        """The reduce-scatter as ceil(rs_tiles / chunk_tiles) launches of at
        most chunk_tiles tiles each; returns the number of launches."""
        n = int(self.info.rs_tiles)
        launches = 0
        for b in range(0, n, chunk_tiles):
            tide_rs_bf16_to_fp32_tiles(self.blob, self.d_blob, ORDERS[order], b,
                                       min(chunk_tiles, n - b), max_workgroups, stream)
            launches += 1
        return launches

    def rs_rank(self, r: int, order: str = "fixed", max_workgroups: int = 0, stream=None) -> None:
        """Only output rank r's shards (one contiguous tile range)."""
        b, c = tide_plan_rank_tiles(self.blob, r)
        if c:
            tide_rs_bf16_to_fp32_tiles(self.blob, self.d_blob, ORDERS[order], b, c, max_workgroups,
                                       stream)

    def rs_census(self, order: str = "fixed", max_workgroups: int = 0, stream=None) -> torch.Tensor:
        """The reduce-scatter, returning for every tile the packed id of the
        compute unit that processed it (int32 GPU tensor)."""
        census = torch.full((max(1, int(self.info.rs_tiles)),), -1, dtype=torch.int32,
                            device=self.d_blob.device)
        tide_rs_bf16_to_fp32_census(self.blob, self.d_blob, census, ORDERS[order],
                                    max_workgroups, stream)
        return census

    def rs_trace(self, order: str = "fixed", max_workgroups: int = 0, stream=None):
        """The reduce-scatter, returning (census, stamps): per tile the packed
        compute-unit id (int32) and its start and end ticks on the GPU's
        real-time counter (int64 [tiles, 2]); GPU tensors."""
        n = max(1, int(self.info.rs_tiles))
        census = torch.full((n,), -1, dtype=torch.int32, device=self.d_blob.device)
        stamps = torch.zeros((n, 2), dtype=torch.int64, device=self.d_blob.device)
        tide_rs_bf16_to_fp32_trace(self.blob, self.d_blob, census, stamps, ORDERS[order],
                                   max_workgroups, stream)
        return census, stamps

    def ag(self, max_workgroups: int = 0, stream=None) -> None:
        tide_ag_place(self.blob, self.d_blob, max_workgroups, stream)

    def ag_sdma(self, engine_only: bool = True, stream=None) -> None:
        tide_ag_place_sdma(self.blob, engine_only, stream)

    def ag_sdma_streams(self, streams) -> None:
        """Engine-only placement spread over several streams.  The caller
        orders them against other work (e.g. with events)."""
        tide_ag_place_sdma_streams(self.blob, streams)

    def ag_dma(self, stream=None) -> None:
        """Placement on the DMA engines through ROCr (host-synchronous)."""
        tide_ag_place_dma(self.blob, stream)

    def shard(self, out_arena: torch.Tensor, p: int) -> torch.Tensor:
        """View of param p's shard in one rank's fp32 arena, shaped [s, rest...]."""
        shp = self.shapes[p]
        s = int(self.m[p]) // (int(np.prod(shp[1:])) if len(shp) > 1 else 1) if int(self.m[p]) else 0
        v = out_arena[int(self.off[p]):int(self.off[p]) + int(self.m[p])]
        return v.view((s,) + tuple(shp[1:])) if len(shp) else v


class StagedRS:
    """Copy-engine-staged reduce-scatter over a plan: ``stage`` holds R bf16
    tensors (rank r's staging buffer of R slots of ``slot_stride`` elements,
    e.g. the rank's vacated gathered buffer with slot_stride = S).
    ``stage_dma()`` moves every rank's slices into the slots on the DMA
    engines (host-synchronous); ``fold()`` reduces the slots into the plan's
    fp32 arenas on the compute units (asynchronous)."""

    def __init__(self, plan: Plan, stage, slot_stride: int = 0):
        if len(stage) != plan.R:
            raise TideError(-1, "need R staging buffers")
        self.plan = plan
        self.slot_stride = int(slot_stride) if slot_stride else int(plan.S)
        for r, t in enumerate(stage):
            _require(t, torch.bfloat16, "stage[%d]" % r)
            if t.numel() < plan.R * self.slot_stride:
                raise TideError(-1, "stage[%d] holds %d elements, need R*slot_stride=%d"
                                % (r, t.numel(), plan.R * self.slot_stride))
        self.stage = list(stage)
        self.h_stage = np.array([t.data_ptr() for t in stage], dtype=np.uint64)
        self.d_stage = torch.from_numpy(self.h_stage.view(np.int64).copy()).to(stage[0].device)

    def stage_dma(self, stream=None) -> None:
        tide_rs_stage_dma(self.plan.blob, self.h_stage, self.slot_stride, stream)

    def fold(self, order: str = "fixed", max_workgroups: int = 0, stream=None) -> None:
        tide_rs_fold_staged(self.plan.blob, self.plan.d_blob, ORDERS[order], self.h_stage,
                            self.d_stage, self.slot_stride, max_workgroups, stream)
