"""Python binding of librtp (resharding and 1D tensor parallelism on a virtual
mesh inside one GB300).

Argument marshalling and buffer checks only: every step of the path runs in the library's CUDA
kernels. PyTorch supplies device memory and streams. Loading fails loudly if
the compiled library is missing; there is no fallback.

Names mirror the C ABI in ``include/rtp.h``:
  spec_from_dims_mapping, spec_from_onnx, spec_nd_sbp (the ND-SBP form filled
  directly), shard_shape, shard_box, shard, reshard, reshard_cost,
  infer_spmd, infer_reshape, tp_mlp, last_error; tp_linear, tp_glu and their
  backward calls, grad_norm, clip_grad_norm (GradGroup keeps their tables).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import List, Optional, Sequence, Tuple, Union

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librtp.so")

MAX_NDIM = 8
MAX_MESH_NDIM = 4
MAX_RANKS = 64
F32, BF16 = 0, 1
SPLIT, BROADCAST, PARTIAL, PARTIAL_MIN, PARTIAL_MAX = 0, 1, 2, 3, 4
STATUS = {0: "RTP_OK", -1: "RTP_EINVAL", -2: "RTP_ESHAPE", -3: "RTP_EUNSUPPORTED", -4: "RTP_ECONFLICT",
          -5: "RTP_ECUDA", -6: "RTP_ENOMEM"}


class RtpError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), message))
        self.status = status


class Spec(ctypes.Structure):
    """rtp_spec: the canonical (ND-SBP) layout of a tensor on a virtual mesh."""

    _fields_ = [
        ("mesh_ndim", ctypes.c_int32),
        ("mesh_shape", ctypes.c_int64 * MAX_MESH_NDIM),
        ("rank_ids", ctypes.c_int32 * MAX_RANKS),
        ("sbp_kind", ctypes.c_int32 * MAX_MESH_NDIM),
        ("sbp_axis", ctypes.c_int32 * MAX_MESH_NDIM),
    ]

    @property
    def num_ranks(self) -> int:
        n = 1
        for d in range(self.mesh_ndim):
            n *= self.mesh_shape[d]
        return n

    def describe(self):
        ents = []
        for d in range(self.mesh_ndim):
            k = self.sbp_kind[d]
            ents.append(("S", self.sbp_axis[d]) if k == SPLIT else
                        {BROADCAST: "B", PARTIAL: "P", PARTIAL_MIN: "Pmin", PARTIAL_MAX: "Pmax"}[k])
        mesh = tuple(self.mesh_shape[d] for d in range(self.mesh_ndim))
        return mesh, tuple(ents), tuple(self.rank_ids[p] for p in range(self.num_ranks))

    def __repr__(self):
        mesh, ents, ranks = self.describe()
        return "Spec(mesh=%s, sbp=%s, ranks=%s)" % (mesh, ents, ranks)


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("librtp.so is not built (%s); run `python -c \"import __graft_entry__ as g; g.build()\"`"
                          % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    i64p, i32p, u32p, vp = P(ctypes.c_int64), P(ctypes.c_int32), P(ctypes.c_uint32), ctypes.c_void_p
    vpp = P(ctypes.c_void_p)
    c_int, i64 = ctypes.c_int, ctypes.c_int64
    sig = {
        "rtp_spec_from_dims_mapping": [c_int, i32p, c_int, i64p, i32p, ctypes.c_uint32, P(Spec)],
        "rtp_spec_from_onnx": [c_int, c_int, i64p, c_int, i64p, i32p, i64p, c_int, i64p, i64p, P(Spec)],
        "rtp_spec_check": [c_int, P(Spec)],
        "rtp_shard_shape": [c_int, i64p, P(Spec), c_int, i64p],
        "rtp_shard_box": [c_int, i64p, P(Spec), c_int, i64p, i64p, i32p],
        "rtp_shard": [c_int, c_int, i64p, vp, P(Spec), vpp, vp],
        "rtp_reshard": [c_int, c_int, i64p, vpp, P(Spec), vpp, P(Spec), vp],
        "rtp_reshard_cost": [c_int, c_int, i64p, P(Spec), P(Spec), i64p, i64p, i32p, i32p],
        "rtp_reshard_forms": [c_int, c_int, i64p, P(Spec), P(Spec), i32p],
        "rtp_infer_spmd": [ctypes.c_char_p, c_int, P(i32p), c_int, i32p, u32p, u32p, P(i32p)],
        "rtp_infer_reshape": [c_int, i64p, i32p, c_int, i64p, c_int, i64p, i32p, i32p],
        "rtp_infer_sbp_signature": [c_int, c_int, i64p, c_int, c_int, i32p, i32p, i32p, i32p, i32p, i32p,
                                    P(ctypes.c_double), i32p],
        "rtp_infer_broadcast": [c_int, i32p, P(i64p), P(Spec), P(c_int), i64p, P(Spec)],
        # tables of pointers are passed as void*: ctypes arrays or bytes
        "rtp_tp_linear": [c_int, c_int, i64, i64, i64, vp, vp, vp, vp, c_int, c_int, vp, vp, vp],
        "rtp_tp_linear_backward": [c_int, c_int, i64, i64, i64, vp, vp, vp, vp, c_int, vp, c_int, vp, c_int, vp, vp, vp],
        "rtp_tp_glu": [c_int, i64, i64, i64, i64, vp, vp, vp, vp, vp, c_int, vp, c_int, vp, vp],
        "rtp_tp_glu_train_forward": [c_int, i64, i64, i64, i64, vp, vp, vp, vp, vp, c_int, vp, vp, vp, c_int, vp, vp],
        "rtp_tp_glu_backward": [c_int, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, c_int, vp, vp, c_int, vp,
                                c_int, vp, vp, vp, vp],
        "rtp_grad_norm": [c_int, i32p, i64p, vp, vp, vp, vp, vp],
        "rtp_clip_grad_norm": [c_int, i32p, i64p, vp, vp, ctypes.c_float, vp, vp, vp, vp],
        "rtp_device_error": [vp, u32p],
        "rtp_wait_selftest": [c_int, ctypes.c_ulonglong, vp, vp],
        "rtp_test_hook": [c_int, ctypes.c_int64],
        "rtp_product_launches": [i32p],
        "rtp_tp_mlp_overlap": [c_int, P(c_int)],
        "rtp_tp_mlp_sp": [c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vpp, vpp, vpp, vpp,
                          vpp, vp],
        "rtp_tp_mlp_noalloc": [c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp, vpp, vpp,
                               vp, vp],
        "rtp_tp_mlp": [c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp, vpp, vpp, vpp,
                       vpp, vp, c_int, c_int, c_int, vp, vp],
        "rtp_tp_mlp_train_forward": [c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp, vpp,
                                     vpp, vpp, vpp, vp, vp],
        "rtp_tp_mlp_backward": [c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp, vpp, vpp,
                                vpp, vpp, vp, vpp, vpp, vp, vpp, vpp, c_int, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = c_int
    lib.rtp_last_error.restype = ctypes.c_char_p
    lib.rtp_last_error.argtypes = []
    lib.rtp_version.restype = ctypes.c_char_p
    lib.rtp_version.argtypes = []
    lib.rtp_grad_workspace_bytes.restype = ctypes.c_int64
    lib.rtp_grad_workspace_bytes.argtypes = [c_int]
    _lib = lib
    return lib


def lib():
    """The loaded ctypes library (loads it on first use)."""
    return _load()


def last_error() -> str:
    return _load().rtp_last_error().decode()


def _check(rc: int) -> None:
    if rc != 0:
        raise RtpError(rc, last_error())


def _i64(xs) -> ctypes.Array:
    xs = [int(x) for x in xs]
    return (ctypes.c_int64 * max(1, len(xs)))(*xs)


def _i32(xs) -> ctypes.Array:
    xs = [int(x) for x in xs]
    return (ctypes.c_int32 * max(1, len(xs)))(*xs)


def _ptrs(ptrs) -> ctypes.Array:
    return (ctypes.c_void_p * max(1, len(ptrs)))(*[p if p else None for p in ptrs])


# ---- specs ------------------------------------------------------------------------

Entry = Union[str, Tuple[str, int]]


def spec_nd_sbp(mesh: Sequence[int], entries: Sequence[Entry], rank_ids: Sequence[int] = ()) -> Spec:
    """ND-SBP form: one entry per mesh dim, ("S", axis), "B", "P" (partial sum),
    "Pmin" or "Pmax" (partial min / max) (OneFlow page)."""
    s = Spec()
    s.mesh_ndim = len(mesh)
    n = 1
    for d, m in enumerate(mesh):
        s.mesh_shape[d] = int(m)
        n *= int(m)
    ranks = list(rank_ids) if rank_ids else list(range(n))
    if len(ranks) > MAX_RANKS:
        raise RtpError(-3, "more than %d ranks" % MAX_RANKS)
    for p, r in enumerate(ranks):
        s.rank_ids[p] = int(r)
    for d, e in enumerate(entries):
        if e == "B":
            s.sbp_kind[d], s.sbp_axis[d] = BROADCAST, -1
        elif e in ("P", "Pmin", "Pmax"):
            s.sbp_kind[d], s.sbp_axis[d] = {"P": PARTIAL, "Pmin": PARTIAL_MIN, "Pmax": PARTIAL_MAX}[e], -1
        else:
            s.sbp_kind[d], s.sbp_axis[d] = SPLIT, int(e[1])
    return s


def spec_from_dims_mapping(dims_mapping: Sequence[int], mesh: Sequence[int], rank_ids: Sequence[int] = (),
                           partial: Sequence[int] = ()) -> Spec:
    mask = 0
    for d in partial:
        mask |= 1 << int(d)
    out = Spec()
    _check(_load().rtp_spec_from_dims_mapping(len(dims_mapping), _i32(dims_mapping), len(mesh), _i64(mesh),
                                              _i32(rank_ids) if rank_ids else None, mask, ctypes.byref(out)))
    return out


def spec_from_onnx(ndim: int, device: Sequence[int], device_map: dict, sharded_dim: Sequence[Tuple[int, int]]
                   ) -> Spec:
    """device: ids or negative keys; device_map: {key: [ids]}; sharded_dim: [(axis, num_shards)]."""
    keys = list(device_map.keys())
    sizes = [len(device_map[k]) for k in keys]
    flat = [d for k in keys for d in device_map[k]]
    out = Spec()
    _check(_load().rtp_spec_from_onnx(ndim, len(device), _i64(device), len(keys), _i64(keys), _i32(sizes),
                                      _i64(flat), len(sharded_dim), _i64([a for a, _ in sharded_dim]),
                                      _i64([s for _, s in sharded_dim]), ctypes.byref(out)))
    return out


def spec_check(ndim: int, spec: Spec) -> None:
    _check(_load().rtp_spec_check(ndim, ctypes.byref(spec)))


def shard_shape(shape: Sequence[int], spec: Spec, rank: int) -> Tuple[int, ...]:
    out = _i64([0] * len(shape))
    _check(_load().rtp_shard_shape(len(shape), _i64(shape), ctypes.byref(spec), rank, out))
    return tuple(out[a] for a in range(len(shape)))


def shard_box(shape: Sequence[int], spec: Spec, rank: int):
    nd = len(shape)
    lo, hi, hv = _i64([0] * nd), _i64([0] * nd), ctypes.c_int32()
    _check(_load().rtp_shard_box(nd, _i64(shape), ctypes.byref(spec), rank, lo, hi, ctypes.byref(hv)))
    return tuple(lo[a] for a in range(nd)), tuple(hi[a] for a in range(nd)), bool(hv.value)


# ---- data movement ----------------------------------------------------------------

_T = None


def _torch():
    """The torch module, imported on first use (an import statement costs 0.3 us a call)."""
    global _T
    if _T is None:
        import torch
        _T = torch
    return _T


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("rtp tensors are float32 or bfloat16, got %s" % t.dtype)


def _stream_ptr(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:  # the current stream's handle, without building a Stream object (3 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


_PIECE_SHAPES: dict = {}


def piece_shapes(shape: Sequence[int], spec: Spec) -> List[Tuple[int, ...]]:
    """shard_shape of every rank, cached per (shape, spec)."""
    key = (tuple(shape), bytes(spec))
    got = _PIECE_SHAPES.get(key)
    if got is None:
        got = [shard_shape(shape, spec, r) for r in range(spec.num_ranks)]
        if len(_PIECE_SHAPES) > 4096:
            _PIECE_SHAPES.clear()
        _PIECE_SHAPES[key] = got
    return got


def _alloc_pieces(shapes, like, out):
    torch = _torch()
    if out is not None:
        return list(out)
    return [torch.empty(s, dtype=like.dtype, device=like.device) for s in shapes]


def _check_cuda(ts, what):
    for t in ts:
        if t is not None and t.numel() > 0:
            if not t.is_cuda:
                raise RtpError(-1, "%s: tensors must live on the GPU" % what)
            if not t.is_contiguous():
                raise RtpError(-1, "%s: tensors must be contiguous (row-major)" % what)


def _check_buffers(what, device: int, groups):
    """The library gets raw pointers and cannot see buffer sizes, so every
    buffer is checked here against the shape and dtype the call will read or
    write: a wrong buffer raises instead of reaching the GPU. device: the CUDA
    device index the call runs on. groups: (name, tensors, shape, dtype), shape
    one tuple for all the tensors or a list of one tuple per tensor (which also
    fixes their count)."""
    for name, ts, shape, dtype in groups:
        per = isinstance(shape, list)
        if per and len(ts) != len(shape):
            raise RtpError(-1, "%s: %d %s buffers given, %d expected" % (what, len(ts), name, len(shape)))
        for i, t in enumerate(ts):
            s = shape[i] if per else shape
            if t.dtype is not dtype or t.shape != s or not t.is_contiguous() or t.get_device() != device:
                _buffer_error(what, name, i, t, s, dtype, device)


def _buffer_error(what, name, i, t, shape, dtype, device):
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape):
        raise RtpError(-2, "%s: %s[%d] is %s %s, expected %s %s" % (
            what, name, i, t.dtype, tuple(t.shape), dtype, tuple(shape)))
    if t.numel() == 0:
        return  # an empty piece is never touched, wherever it lives
    if not t.is_contiguous():
        raise RtpError(-1, "%s: %s[%d] must be contiguous (row-major)" % (what, name, i))
    raise RtpError(-1, "%s: %s[%d] is on %s, the call runs on device %d" % (what, name, i, t.device, device))


def _device_of(t) -> int:
    """Index of the current CUDA device, which must hold `t`."""
    torch = _torch()
    if not t.is_cuda:
        raise RtpError(-1, "tensors must live on the GPU")
    device = t.get_device()
    if device != torch._C._cuda_getDevice():
        raise RtpError(-1, "tensors are on %s but the current CUDA device is %d" % (t.device,
                                                                                  torch.cuda.current_device()))
    return device


def shard(full, spec: Spec, out=None, stream=None):
    """Rank pieces of the logical tensor `full` (a CUDA tensor) under `spec`."""
    shape = tuple(full.shape)
    shapes = piece_shapes(shape, spec)
    code = _dtype_code(full)
    pieces = _alloc_pieces(shapes, full, out)
    _check_buffers("shard", _device_of(full), [("full", [full], shape, full.dtype),
                                               ("out", pieces, shapes, full.dtype)])
    _check(_load().rtp_shard(code, len(shape), _i64(shape), full.data_ptr(), ctypes.byref(spec),
                             _ptrs([p.data_ptr() for p in pieces]), _stream_ptr(stream)))
    return pieces


def reshard(pieces, shape: Sequence[int], src: Spec, dst: Spec, out=None, stream=None):
    """Pieces laid out by `dst`, from `pieces` laid out by `src`."""
    shape = tuple(int(s) for s in shape)
    like = pieces[0]
    dshapes = piece_shapes(shape, dst)
    code = _dtype_code(like)
    outs = _alloc_pieces(dshapes, like, out)
    _check_buffers("reshard", _device_of(like), [("pieces", pieces, piece_shapes(shape, src), like.dtype),
                                                 ("out", outs, dshapes, like.dtype)])
    _check(_load().rtp_reshard(code, len(shape), _i64(shape), _ptrs([p.data_ptr() for p in pieces]),
                               ctypes.byref(src), _ptrs([o.data_ptr() for o in outs]), ctypes.byref(dst),
                               _stream_ptr(stream)))
    return outs


def reshard_forms(dtype_code: int, shape: Sequence[int], src: Spec, dst: Spec):
    """Tasks per kernel form a reshard would use: (registers, bulk staging,
    TMA tiles 3D, TMA tiles 4D), for 256-byte aligned buffers."""
    c = (ctypes.c_int32 * 4)()
    _check(_load().rtp_reshard_forms(dtype_code, len(shape), _i64(shape), ctypes.byref(src), ctypes.byref(dst), c))
    return tuple(c)


def reshard_cost(dtype_code: int, shape: Sequence[int], src: Spec, dst: Spec):
    """(bytes_read, bytes_written, n_tasks, n_launches) planned for a reshard."""
    rd, wr, nt, nl = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
    _check(_load().rtp_reshard_cost(dtype_code, len(shape), _i64(shape), ctypes.byref(src), ctypes.byref(dst),
                                    ctypes.byref(rd), ctypes.byref(wr), ctypes.byref(nt), ctypes.byref(nl)))
    return rd.value, wr.value, nt.value, nl.value


# ---- inference --------------------------------------------------------------------

def infer_spmd(einsum: str, dims_mappings: Sequence[Sequence[int]], mesh_ndim: int):
    """(out_dims_mapping, partial_mesh_dims, inputs_needing_reshard, inferred_input_mappings)."""
    lhs, rhs = einsum.split("->") if "->" in einsum else (einsum, "")
    ins = lhs.split(",")
    P = ctypes.POINTER(ctypes.c_int32)
    arrs = [_i32(dm) for dm in dims_mappings]
    merged = [_i32([0] * max(1, len(t))) for t in ins]
    inp = (P * max(1, len(arrs)))(*[ctypes.cast(a, P) for a in arrs])
    mp = (P * max(1, len(merged)))(*[ctypes.cast(a, P) for a in merged])
    out = _i32([0] * max(1, len(rhs)))
    pm, rm = ctypes.c_uint32(), ctypes.c_uint32()
    _check(_load().rtp_infer_spmd(einsum.encode(), len(dims_mappings), inp, mesh_ndim, out, ctypes.byref(pm),
                                  ctypes.byref(rm), mp))
    return ([out[i] for i in range(len(rhs))], [d for d in range(32) if (pm.value >> d) & 1],
            [j for j in range(len(ins)) if (rm.value >> j) & 1],
            [[merged[j][i] for i in range(len(ins[j]))] for j in range(len(ins))])


def infer_reshape(in_shape, in_dims_mapping, out_shape, mesh):
    """(in_dims_after, out_dims_mapping) for a reshape."""
    ni, no = len(in_shape), len(out_shape)
    after, outm = _i32([0] * ni), _i32([0] * no)
    _check(_load().rtp_infer_reshape(ni, _i64(in_shape), _i32(in_dims_mapping), no, _i64(out_shape), len(mesh),
                                     _i64(mesh), after, outm))
    return [after[i] for i in range(ni)], [outm[o] for o in range(no)]


def _sbp_entry(e):
    if e == "B":
        return BROADCAST, -1
    if e in ("P", "Pmin", "Pmax"):
        return {"P": PARTIAL, "Pmin": PARTIAL_MIN, "Pmax": PARTIAL_MAX}[e], -1
    return SPLIT, int(e[1])


def infer_sbp_signature(shape, elem_bytes, inputs, constraint=None):
    """OneFlow-style SBP signature of an element-wise op. inputs: per input its
    ND-SBP (entries ("S", axis) / "B" / "P" per mesh dim). Returns
    (signature entries, CopyCost, OrderValue)."""
    md = len(inputs[0])
    kinds, axes = [], []
    for sbp in inputs:
        for e in sbp:
            k, a = _sbp_entry(e)
            kinds.append(k)
            axes.append(a)
    ck = ca = None
    if constraint is not None:
        c = [_sbp_entry(e) for e in constraint]
        ck, ca = _i32([k for k, _ in c]), _i32([a for _, a in c])
    okind, oaxis = _i32([0] * md), _i32([0] * md)
    cost, order = ctypes.c_double(), ctypes.c_int32()
    _check(_load().rtp_infer_sbp_signature(len(inputs), len(shape), _i64(shape), elem_bytes, md, _i32(kinds),
                                           _i32(axes), ck, ca, okind, oaxis, ctypes.byref(cost), ctypes.byref(order)))
    sig = []
    for d in range(md):
        k = okind[d]
        sig.append(("S", oaxis[d]) if k == SPLIT else {BROADCAST: "B", PARTIAL: "P"}[k])
    return sig, cost.value, order.value


def infer_broadcast(shapes, specs):
    """ONNX broadcast n-ary element-wise rule: (output shape, output Spec) for
    inputs of the given shapes and layouts; RtpError -4 when the inputs are
    sharded incompatibly."""
    n = len(shapes)
    nds = (ctypes.c_int32 * n)(*[len(sh) for sh in shapes])
    arrs = [_i64(sh) for sh in shapes]
    shp = (ctypes.POINTER(ctypes.c_int64) * n)(*[ctypes.cast(a, ctypes.POINTER(ctypes.c_int64)) for a in arrs])
    sp = (Spec * n)(*specs)
    out_nd, oshape, out = ctypes.c_int(), _i64([0] * 8), Spec()
    _check(_load().rtp_infer_broadcast(n, nds, shp, sp, ctypes.byref(out_nd), oshape, ctypes.byref(out)))
    return tuple(oshape[d] for d in range(out_nd.value)), out


# ---- tensor-parallel MLP ------------------------------------------------------------

def tp_mlp(X, A_shards, B_shards, Y=None, partials=None, Z=None, mode: int = 1, chunks: int = 1,
           col_blocks: int = 1, s0=None, s1=None):
    """Z = sum_i GELU(X A_i) B_i on P = len(A_shards) virtual ranks (bf16 in, float32 Z).
    Returns (Z, Y). Buffers not given are allocated with torch."""
    torch = _torch()
    P = len(A_shards)
    M, K = X.shape
    Fp = A_shards[0].shape[1]
    N = B_shards[0].shape[1]
    F = Fp * P
    dev = X.device
    if Y is None:
        Y = [torch.empty((M, Fp), dtype=torch.bfloat16, device=dev) for _ in range(P)]
    if Z is None:
        Z = torch.empty((M, N), dtype=torch.float32, device=dev)
    if mode == 0 and partials is None:
        partials = [torch.empty((M, N), dtype=torch.float32, device=dev) for _ in range(P)]
    bf16, f32 = torch.bfloat16, torch.float32
    _check_buffers("tp_mlp", _device_of(X), [
        ("X", [X], (M, K), bf16), ("A_shards", A_shards, (K, Fp), bf16), ("B_shards", B_shards, [(Fp, N)] * P, bf16),
        ("Y", Y, [(M, Fp)] * P, bf16), ("partials", partials or [], [(M, N)] * (P if partials is not None else 0), f32),
        ("Z", [Z], (M, N), f32)])
    if s0 is None:
        s0 = torch.cuda.current_stream()
    if s1 is None:
        s1 = s0
    pp = _ptrs([p.data_ptr() for p in partials]) if partials is not None else None
    _check(_load().rtp_tp_mlp(P, M, K, F, N, X.data_ptr(), _ptrs([a.data_ptr() for a in A_shards]),
                              _ptrs([b.data_ptr() for b in B_shards]), _ptrs([y.data_ptr() for y in Y]), pp,
                              Z.data_ptr(), mode, chunks, col_blocks, _stream_ptr(s0), _stream_ptr(s1)))
    return Z, Y


def tp_mlp_overlap(sum_in_epilogue: int) -> int:
    """Where mode 0 sums the rank partials, for later calls from this thread:
    0 (the default) in kernels of their own (on s1 beside the next GEMMs when
    given), 1 in the epilogue of the GEMM that writes them. Returns the
    previous setting."""
    prev = ctypes.c_int()
    _check(_load().rtp_tp_mlp_overlap(int(sum_in_epilogue), ctypes.byref(prev)))
    return prev.value


def tp_mlp_train_forward(X, A_shards, B_shards, Y=None, H=None, Z=None, stream=None):
    """The fused forward that also keeps the bf16 pre-activations H_i = X A_i
    for the backward pass. Returns (Z, Y, H)."""
    torch = _torch()
    P = len(A_shards)
    M, K = X.shape
    Fp = A_shards[0].shape[1]
    N = B_shards[0].shape[1]
    dev = X.device
    if Y is None:
        Y = [torch.empty((M, Fp), dtype=torch.bfloat16, device=dev) for _ in range(P)]
    if H is None:
        H = [torch.empty((M, Fp), dtype=torch.bfloat16, device=dev) for _ in range(P)]
    if Z is None:
        Z = torch.empty((M, N), dtype=torch.float32, device=dev)
    bf16, f32 = torch.bfloat16, torch.float32
    _check_buffers("tp_mlp_train_forward", _device_of(X), [
        ("X", [X], (M, K), bf16), ("A_shards", A_shards, (K, Fp), bf16), ("B_shards", B_shards, [(Fp, N)] * P, bf16),
        ("Y", Y, [(M, Fp)] * P, bf16), ("H", H, [(M, Fp)] * P, bf16), ("Z", [Z], (M, N), f32)])
    _check(_load().rtp_tp_mlp_train_forward(P, M, K, Fp * P, N, X.data_ptr(), _ptrs([a.data_ptr() for a in A_shards]),
                                            _ptrs([b.data_ptr() for b in B_shards]), _ptrs([y.data_ptr() for y in Y]),
                                            _ptrs([h.data_ptr() for h in H]), Z.data_ptr(), _stream_ptr(stream)))
    return Z, Y, H


def tp_mlp_backward(X, A_shards, B_shards, H, Y, dZ, dH=None, dX_partials=None, dX=None, dA=None, dB=None,
                    mode: int = 1, s0=None, s1=None):
    """Gradients of Z = sum_i GELU(X A_i) B_i given dZ (bf16 [M, N]):
    returns (dX, dA, dB, dH) with dX float32 [M, K], dA[i] float32 [K, F/P],
    dB[i] float32 [F/P, N] and dH[i] = bf16(dZ B_i^T * GELU'(H_i))."""
    torch = _torch()
    P = len(A_shards)
    M, K = X.shape
    Fp = A_shards[0].shape[1]
    N = B_shards[0].shape[1]
    dev = X.device
    f32, bf16 = torch.float32, torch.bfloat16
    if dH is None:
        dH = [torch.empty((M, Fp), dtype=bf16, device=dev) for _ in range(P)]
    if dX is None:
        dX = torch.empty((M, K), dtype=f32, device=dev)
    if dA is None:
        dA = [torch.empty((K, Fp), dtype=f32, device=dev) for _ in range(P)]
    if dB is None:
        dB = [torch.empty((Fp, N), dtype=f32, device=dev) for _ in range(P)]
    if mode == 0 and dX_partials is None:
        dX_partials = [torch.empty((M, K), dtype=f32, device=dev) for _ in range(P)]
    nparts = P if dX_partials is not None else 0
    _check_buffers("tp_mlp_backward", _device_of(X), [
        ("X", [X], (M, K), bf16), ("A_shards", A_shards, (K, Fp), bf16), ("B_shards", B_shards, [(Fp, N)] * P, bf16),
        ("H", H, [(M, Fp)] * P, bf16), ("Y", Y, [(M, Fp)] * P, bf16), ("dZ", [dZ], (M, N), bf16),
        ("dH", dH, [(M, Fp)] * P, bf16), ("dX_partials", dX_partials or [], [(M, K)] * nparts, f32),
        ("dX", [dX], (M, K), f32), ("dA", dA, [(K, Fp)] * P, f32), ("dB", dB, [(Fp, N)] * P, f32)])
    if s0 is None:
        s0 = torch.cuda.current_stream()
    if s1 is None:
        s1 = s0
    ptrs = lambda ts: _ptrs([t.data_ptr() for t in ts])
    pp = ptrs(dX_partials) if dX_partials is not None else None
    _check(_load().rtp_tp_mlp_backward(P, M, K, Fp * P, N, X.data_ptr(), ptrs(A_shards), ptrs(B_shards), ptrs(H),
                                       ptrs(Y), dZ.data_ptr(), ptrs(dH), pp, dX.data_ptr(), ptrs(dA), ptrs(dB), mode,
                                       _stream_ptr(s0), _stream_ptr(s1)))
    return dX, dA, dB, dH


def tp_mlp_sp(X_shards, A_shards, B_shards, Y=None, Z_shards=None, stream=None):
    """Sequence-parallel TP-MLP: X_shards[r] holds rows r*M/P.. of X; returns
    (Z_shards, Y) with Z_shards[r] the same rows of sum_i GELU(X A_i) B_i."""
    torch = _torch()
    P = len(A_shards)
    Mr, K = X_shards[0].shape
    M = Mr * P
    Fp = A_shards[0].shape[1]
    N = B_shards[0].shape[1]
    dev = X_shards[0].device
    if Y is None:
        Y = [torch.empty((M, Fp), dtype=torch.bfloat16, device=dev) for _ in range(P)]
    if Z_shards is None:
        Z_shards = [torch.empty((Mr, N), dtype=torch.float32, device=dev) for _ in range(P)]
    bf16, f32 = torch.bfloat16, torch.float32
    _check_buffers("tp_mlp_sp", _device_of(X_shards[0]), [
        ("X_shards", X_shards, [(Mr, K)] * P, bf16), ("A_shards", A_shards, (K, Fp), bf16),
        ("B_shards", B_shards, [(Fp, N)] * P, bf16), ("Y", Y, [(M, Fp)] * P, bf16),
        ("Z_shards", Z_shards, [(Mr, N)] * P, f32)])
    _check(_load().rtp_tp_mlp_sp(P, M, K, Fp * P, N, _ptrs([x.data_ptr() for x in X_shards]),
                                 _ptrs([a.data_ptr() for a in A_shards]), _ptrs([b.data_ptr() for b in B_shards]),
                                 _ptrs([y.data_ptr() for y in Y]), _ptrs([z.data_ptr() for z in Z_shards]),
                                 _stream_ptr(stream)))
    return Z_shards, Y


def tp_mlp_noalloc(X, A_shards, B_shards, Z=None, stream=None):
    """Z = sum_i GELU(X A_i) B_i with the activations in the library's static
    device scratch (for callers that cannot allocate). Returns Z.

    Every call shares that one static array (16 MiB per device): calls that
    overlap on the GPU, on several streams or from several threads, race on it
    and must be ordered by the caller. The first call on a device finds the
    array's address; make it before any stream capture, and do not reset the
    device after it."""
    torch = _torch()
    P = len(A_shards)
    M, K = X.shape
    Fp = A_shards[0].shape[1]
    N = B_shards[0].shape[1]
    if Z is None:
        Z = torch.empty((M, N), dtype=torch.float32, device=X.device)
    bf16 = torch.bfloat16
    _check_buffers("tp_mlp_noalloc", _device_of(X), [
        ("X", [X], (M, K), bf16), ("A_shards", A_shards, (K, Fp), bf16), ("B_shards", B_shards, [(Fp, N)] * P, bf16),
        ("Z", [Z], (M, N), torch.float32)])
    _check(_load().rtp_tp_mlp_noalloc(P, M, K, Fp * P, N, X.data_ptr(), _ptrs([a.data_ptr() for a in A_shards]),
                                      _ptrs([b.data_ptr() for b in B_shards]), Z.data_ptr(), _stream_ptr(stream)))
    return Z


# ---- linear layers and the gated feed-forward block -------------------------------------

ACTS = {"none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3, "relu": 4}
_ext = None


def _tables():
    """The Python extension that checks lists of tensors and tabulates their addresses."""
    global _ext
    if _ext is None:
        _load()
        _torch()  # the extension's libraries are torch's
        try:
            from . import _table
        except ImportError as e:
            raise ImportError("_table.so is not built (%s); run `python -c \"import __graft_entry__ as g; g.build()\"`"
                              % e) from e
        _table.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (_lib.rtp_tp_linear, _lib.rtp_tp_glu,
                                                                          _lib.rtp_clip_grad_norm)])
        _ext = _table
    return _ext


def _on_gpu(X) -> bool:
    return getattr(X[0] if type(X) is list and X else X, "is_cuda", False)


def _called(got):
    """The outputs of a call that the extension made whole; None when it did not take the arguments."""
    if type(got) is int:
        _check(got)
    return got


def _table_of(fn: str, name: str, ts, n: int, shape, dtype, device: int) -> bytes:
    """Addresses of the n tensors of a list as one table, each checked against the shape, type and device that the call
    will touch (the library sees addresses only)."""
    if len(ts) != n:
        raise RtpError(-1, "%s: %d %s buffers given, %d expected" % (fn, len(ts), name, n))
    code = F32 if dtype is _torch().float32 else BF16
    got = (_ext or _tables()).table(ts, shape, code, device)
    if type(got) is int:
        t = ts[got]
        if not isinstance(t, _torch().Tensor):
            raise RtpError(-1, "%s: %s[%d] is no tensor" % (fn, name, got))
        _buffer_error(fn, name, got, t, shape, dtype, device)
        raise RtpError(-1, "%s: %s[%d] does not fit" % (fn, name, got))
    return got


def _act_code(act: str) -> int:
    try:
        return ACTS[act]
    except (KeyError, TypeError):
        raise RtpError(-1, "unknown activation %r (one of %s)" % (act, ", ".join(ACTS))) from None


def _out_dtype(given, buffer, default):
    """The type of an output: as asked for, else as the buffer given, else the default."""
    dtype = given or (default if buffer is None else buffer.dtype)
    if dtype is not _torch().float32 and dtype is not _torch().bfloat16:
        raise TypeError("rtp tensors are float32 or bfloat16, got %s" % dtype)
    return dtype


def _listed(t) -> list:
    """A list of rank buffers; one tensor stands for a list of one."""
    if type(t) is list:
        return t
    return list(t) if isinstance(t, tuple) else [t]


def _matrix(fn: str, name: str, t):
    if t.dim() != 2:
        raise RtpError(-2, "%s: %s is %s, expected a matrix" % (fn, name, tuple(t.shape)))
    return t.shape


def _allocating_on(stream):
    """Context in which torch allocates, and launches, on the stream that a call was given (None: the current one).
    Memory that torch hands out again is ordered on its owning stream only, and scratch is dropped when the call
    returns: it has to be owned by the stream that the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    torch = _torch()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _new(n: int, shape, dtype, device: int, stream=None) -> list:
    """n fresh buffers of one shape, owned by the stream the call runs on."""
    code = F32 if dtype is _torch().float32 else BF16
    if stream is None:
        return (_ext or _tables()).buffers(n, shape, code, device)
    with _allocating_on(stream):
        return _tables().buffers(n, shape, code, device)


def _slices(whole, n: int, nbytes: int) -> bytes:
    """Addresses of n equal slices of nbytes each of one allocation (scratch that the caller does not see)."""
    p = whole.data_ptr()
    return struct.pack("%dQ" % n, *[p + i * nbytes for i in range(n)])


def _linear_shapes(fn: str, X, W, split: str):
    """(row?, P, M, K, N, Kp, Np) of a linear layer's arguments (lists)."""
    if split != "column" and split != "row":
        raise RtpError(-1, "%s: split %r is not 'column' or 'row'" % (fn, split))
    if not W or not X:
        raise RtpError(-1, "%s: no weight shards or no X" % fn)
    row, P = split == "row", len(W)
    M, _ = _matrix(fn, "X", X[0])
    Kp, Np = _matrix(fn, "W_shards[0]", W[0])
    return row, P, M, Kp * P if row else Kp, Np if row else Np * P, Kp, Np


def tp_linear(X, W_shards, split: str = "column", bias=None, act: str = "none", residual=None, H=None, out=None,
              out_dtype=None, keep_h: bool = False, stream=None):
    """Linear layer on P = len(W_shards) virtual ranks, bias, activation and residual in the product's epilogue.

    column: out_i = act(X W_i + b_i) + R_i, X one tensor [M, K], W_i [K, N/P];
    row:    out = act(sum_i X_i W_i + b) + R, X a list of P tensors [M, K/P], W_i [K/P, N].
    bias, residual, H and out are lists with one entry per output buffer (P for column, 1 for row; a
    single tensor stands for a list of one). All bf16; out may be float32 (out_dtype, or by `out`).
    Returns the list of outputs, or (outputs, H) with keep_h (or H given): the bf16 pre-activations that
    tp_linear_backward reads."""
    fn = "tp_linear"
    if (out is None and H is None and not keep_h and out_dtype is None and stream is None and
            split in ("column", "row") and _on_gpu(X)):
        got = _called((_ext or _tables()).linear(X, W_shards, split == "row", bias, residual, _act_code(act),
                                                 _torch()._C._cuda_getDevice(), _stream_ptr(None) or 0))
        if got is not None:
            return got
    bf16 = _torch().bfloat16
    X, W = _listed(X), _listed(W_shards)
    row, P, M, K, N, Kp, Np = _linear_shapes(fn, X, W, split)
    outs, code, shape = 1 if row else P, _act_code(act), (M, Np)
    device = _device_of(X[0])
    xp = _table_of(fn, "X", X, P if row else 1, (M, Kp), bf16, device)
    wp = _table_of(fn, "W_shards", W, P, (Kp, Np), bf16, device)
    bp = rp = hp = None
    if bias is not None:
        bp = _table_of(fn, "bias", _listed(bias), outs, (Np,), bf16, device)
    if residual is not None:
        rp = _table_of(fn, "residual", _listed(residual), outs, shape, bf16, device)
    if out is not None:
        out = _listed(out)
    out_dtype = _out_dtype(out_dtype, out[0] if out else None, bf16)
    if out is None:
        out = _new(outs, shape, out_dtype, device, stream)
    op = _table_of(fn, "out", out, outs, shape, out_dtype, device)
    if keep_h or H is not None:
        H = _new(outs, shape, bf16, device, stream) if H is None else _listed(H)
        hp = _table_of(fn, "H", H, outs, shape, bf16, device)
    _check(_lib.rtp_tp_linear(1 if row else 0, P, M, K, N, xp, wp, bp, rp, code, _dtype_code(out[0]), hp, op,
                              _stream_ptr(stream)))
    return (out, H) if hp is not None else out


def tp_linear_backward(X, W_shards, dOut, split: str = "column", H=None, act: str = "none", dH=None, dX=None, dW=None,
                       db=None, bias_grad: bool = True, dx_dtype=None, dw_dtype=None, stream=None):
    """Gradients of tp_linear given dOut (bf16, laid out as its outputs) and, with an activation, the kept H.
    Returns lists (dX, dW, db): dX like X, dW like W_shards (bf16, or float32 by dx_dtype / dw_dtype or by the
    buffers given), db float32 like bias (None without bias_grad). The residual's gradient is dOut."""
    fn = "tp_linear_backward"
    bf16, f32 = _torch().bfloat16, _torch().float32
    X, W = _listed(X), _listed(W_shards)
    row, P, M, K, N, Kp, Np = _linear_shapes(fn, X, W, split)
    outs, ins, code, shape = 1 if row else P, P if row else 1, _act_code(act), (M, Np)
    device = _device_of(X[0])
    xp = _table_of(fn, "X", X, ins, (M, Kp), bf16, device)
    wp = _table_of(fn, "W_shards", W, P, (Kp, Np), bf16, device)
    dop = _table_of(fn, "dOut", _listed(dOut), outs, shape, bf16, device)
    hp = dhp = dbp = None
    if code:
        if H is None:
            raise RtpError(-1, "%s: the kept pre-activation H is needed with act=%r" % (fn, act))
        hp = _table_of(fn, "H", _listed(H), outs, shape, bf16, device)
        dH = _new(outs, shape, bf16, device, stream) if dH is None else _listed(dH)
        dhp = _table_of(fn, "dH", dH, outs, shape, bf16, device)
    dx_dtype = _out_dtype(dx_dtype, None if dX is None else _listed(dX)[0], bf16)
    dw_dtype = _out_dtype(dw_dtype, None if dW is None else _listed(dW)[0], bf16)
    dX = _new(ins, (M, Kp), dx_dtype, device, stream) if dX is None else _listed(dX)
    dW = _new(P, (Kp, Np), dw_dtype, device, stream) if dW is None else _listed(dW)
    dxp = _table_of(fn, "dX", dX, ins, (M, Kp), dx_dtype, device)
    dwp = _table_of(fn, "dW", dW, P, (Kp, Np), dw_dtype, device)
    if db is not None or bias_grad:
        db = _new(outs, (Np,), f32, device, stream) if db is None else _listed(db)
        dbp = _table_of(fn, "db", db, outs, (Np,), f32, device)
    _check(_lib.rtp_tp_linear_backward(1 if row else 0, P, M, K, N, xp, wp, hp, dop, code, dhp, _dtype_code(dX[0]), dxp,
                                       _dtype_code(dW[0]), dwp, dbp, _stream_ptr(stream)))
    return dX, dW, db


def _glu_weights(fn: str, X, Ag, Au, B):
    """(P, M, K, Fp, N, device, tables of X, Ag, Au, B) of the gated block's arguments."""
    bf16 = _torch().bfloat16
    P = len(Ag)
    if not P or not B:
        raise RtpError(-1, "%s: no weight shards" % fn)
    M, K = _matrix(fn, "X", X)
    _, Fp = _matrix(fn, "Ag_shards[0]", Ag[0])
    _, N = _matrix(fn, "B_shards[0]", B[0])
    device = _device_of(X)
    _table_of(fn, "X", [X], 1, (M, K), bf16, device)
    return (P, M, K, Fp, N, device, _table_of(fn, "Ag_shards", Ag, P, (K, Fp), bf16, device),
            _table_of(fn, "Au_shards", Au, P, (K, Fp), bf16, device),
            _table_of(fn, "B_shards", B, P, (Fp, N), bf16, device))


def _glu_forward(fn, X, Ag, Au, B, act, residual, kept, Z, out_dtype, stream):
    """kept: [Y] or [Y, Hg, Hu], each a list of P buffers or None. Returns (Z, kept)."""
    bf16 = _torch().bfloat16
    code = _act_code(act)
    P, M, K, Fp, N, device, agp, aup, bp = _glu_weights(fn, X, Ag, Au, B)
    out_dtype = _out_dtype(out_dtype, Z, bf16)
    if Z is None:
        Z, = _new(1, (M, N), out_dtype, device, stream)
    _table_of(fn, "Z", [Z], 1, (M, N), out_dtype, device)
    rp = None
    if residual is not None:
        _table_of(fn, "residual", [residual], 1, (M, N), bf16, device)
        rp = residual.data_ptr()
    if len(kept) == 1 and kept[0] is None:  # Y as scratch
        scratch, = _new(1, (P, M, Fp), bf16, device, stream)
        kp = [_slices(scratch, P, 2 * M * Fp)]
    else:
        kept = [_new(P, (M, Fp), bf16, device, stream) if k is None else _listed(k) for k in kept]
        kp = [_table_of(fn, name, k, P, (M, Fp), bf16, device) for name, k in zip(("Y", "Hg", "Hu"), kept)]
    call = _lib.rtp_tp_glu if len(kp) == 1 else _lib.rtp_tp_glu_train_forward
    _check(call(P, M, K, Fp * P, N, X.data_ptr(), agp, aup, bp, rp, code, *kp, _dtype_code(Z), Z.data_ptr(),
                _stream_ptr(stream)))
    return Z, kept


def tp_glu(X, Ag_shards, Au_shards, B_shards, act: str = "silu", residual=None, Y=None, Z=None, out_dtype=None,
           stream=None):
    """Gated feed-forward block on P = len(Ag_shards) virtual ranks:
    Z = sum_i (act(X Ag_i) * (X Au_i)) B_i + residual, bf16 [M, N] (or float32: out_dtype, or by `Z`).
    Y: P bf16 [M, F/P] scratch buffers, allocated when not given. Returns Z."""
    if Y is None and Z is None and out_dtype is None and stream is None and _on_gpu(X):
        got = _called((_ext or _tables()).glu(X, Ag_shards, Au_shards, B_shards, residual, _act_code(act),
                                              _torch()._C._cuda_getDevice(), _stream_ptr(None) or 0))
        if got is not None:
            return got
    return _glu_forward("tp_glu", X, _listed(Ag_shards), _listed(Au_shards), _listed(B_shards), act, residual, [Y], Z,
                        out_dtype, stream)[0]


def tp_glu_train_forward(X, Ag_shards, Au_shards, B_shards, act: str = "silu", residual=None, Y=None, Hg=None, Hu=None,
                         Z=None, out_dtype=None, stream=None):
    """tp_glu that keeps the bf16 pre-activations Hg_i = X Ag_i and Hu_i = X Au_i beside Y_i = act(Hg_i) * Hu_i for
    tp_glu_backward. Returns (Z, Y, Hg, Hu)."""
    Z, kept = _glu_forward("tp_glu_train_forward", X, _listed(Ag_shards), _listed(Au_shards), _listed(B_shards), act,
                           residual, [Y, Hg, Hu], Z, out_dtype, stream)
    return (Z, *kept)


def tp_glu_backward(X, Ag_shards, Au_shards, B_shards, Hg, Hu, Y, dZ, act: str = "silu", dHg=None, dHu=None, dX=None,
                    dAg=None, dAu=None, dB=None, dx_dtype=None, dw_dtype=None, stream=None):
    """Gradients of the gated block given dZ (bf16 [M, N]) and what tp_glu_train_forward kept. Returns (dX, dAg, dAu,
    dB): dX [M, K] and lists of P weight gradients, bf16 or float32 (dx_dtype, dw_dtype, or by the buffers given). The
    residual's gradient is dZ. dHg, dHu: P bf16 [M, F/P] scratch buffers each."""
    fn = "tp_glu_backward"
    bf16 = _torch().bfloat16
    code = _act_code(act)
    P, M, K, Fp, N, device, agp, aup, bp = _glu_weights(fn, X, _listed(Ag_shards), _listed(Au_shards), _listed(B_shards))
    if Hg is None or Hu is None or Y is None:
        raise RtpError(-1, "%s: Hg, Hu and Y of the training forward are needed" % fn)
    mid = [(name, _new(P, (M, Fp), bf16, device, stream) if t is None else _listed(t))
           for name, t in (("Hg", Hg), ("Hu", Hu), ("Y", Y), ("dHg", dHg), ("dHu", dHu))]
    hg, hu, y, dhg, dhu = (_table_of(fn, name, t, P, (M, Fp), bf16, device) for name, t in mid)
    _table_of(fn, "dZ", [dZ], 1, (M, N), bf16, device)
    dx_dtype = _out_dtype(dx_dtype, dX, bf16)
    if dX is None:
        dX, = _new(1, (M, K), dx_dtype, device, stream)
    _table_of(fn, "dX", [dX], 1, (M, K), dx_dtype, device)
    given = [t for t in (dAg, dAu, dB) if t is not None]
    dw_dtype = _out_dtype(dw_dtype, _listed(given[0])[0] if given else None, bf16)
    dw = [_new(P, s, dw_dtype, device, stream) if t is None else _listed(t)
          for t, s in ((dAg, (K, Fp)), (dAu, (K, Fp)), (dB, (Fp, N)))]
    dwp = [_table_of(fn, name, t, P, s, dw_dtype, device)
           for name, t, s in (("dAg", dw[0], (K, Fp)), ("dAu", dw[1], (K, Fp)), ("dB", dw[2], (Fp, N)))]
    _check(_lib.rtp_tp_glu_backward(P, M, K, Fp * P, N, X.data_ptr(), agp, aup, bp, hg, hu, y, dZ.data_ptr(), code, dhg,
                                    dhu, _dtype_code(dX), dX.data_ptr(), _dtype_code(dw[0][0]), *dwp,
                                    _stream_ptr(stream)))
    return (dX, *dw)


# ---- global gradient norm and clipping -----------------------------------------------------

def counted_pieces(spec: Spec) -> List[bool]:
    """Which rank pieces of a gradient laid out by `spec` count towards the global norm: under broadcast mesh dims only
    the ranks at coordinate 0 (the others hold replicas). A partial layout has no per-rank norm: reshard it first."""
    md = spec.mesh_ndim
    if any(spec.sbp_kind[d] not in (SPLIT, BROADCAST) for d in range(md)):
        raise RtpError(-3, "counted_pieces: a partial layout must be reshard before its norm is taken")
    flags = [True] * spec.num_ranks
    for p in range(spec.num_ranks):
        rest = p
        for d in reversed(range(md)):
            c, rest = rest % spec.mesh_shape[d], rest // spec.mesh_shape[d]
            if c and spec.sbp_kind[d] == BROADCAST:
                flags[spec.rank_ids[p]] = False
    return flags


class GradGroup:
    """The gradients of a program's tensors (rank pieces, float32 and bf16 mixed), for their global norm and clipping.
    Keeps the tensors, their tables and the workspace, as a training loop keeps its gradient buffers; the values are
    read at each call. counted[i] False: tensor i is a replica (counted_pieces) that is clipped but not counted. Calls
    on one group that may overlap on the GPU share its workspace and must be ordered by the caller. stream: where the
    workspace is allocated and zeroed (default: the current stream)."""

    def __init__(self, grads, counted=None, stream=None):
        self._set_up(grads, counted, stream)
        torch = _torch()
        with _allocating_on(stream):  # when the workspace is zero, for other streams (_join)
            if not torch.cuda.is_current_stream_capturing():
                self._zeroed = torch.cuda.current_stream(self.device).record_event()

    @classmethod
    def _for_one_call(cls, grads, counted, stream):
        """A group for one call on the stream given, which needs no event for other streams (15 us)."""
        group = cls.__new__(cls)
        group._set_up(grads, counted, stream)
        return group

    def _set_up(self, grads, counted, stream):
        torch = _torch()
        self.grads = list(grads)
        n = len(self.grads)
        if n and not self.grads[0].is_cuda:
            raise RtpError(-1, "GradGroup: tensors must live on the GPU")
        self.device = self.grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
        self._tabulate()
        self._counted = None
        if counted is not None:
            counted = [bool(c) for c in counted]
            if len(counted) != n:
                raise RtpError(-1, "GradGroup: %d counted flags for %d tensors" % (len(counted), n))
            self._counted = (ctypes.c_uint8 * max(1, n))(*counted)
        # zero once: every call leaves its counter zero
        with _allocating_on(stream):
            self._ws = torch.zeros((_load().rtp_grad_workspace_bytes(n) // 8,), dtype=torch.float64, device=self.device)
            self._zeroed = None
            self._index = self.device.index
            # handles of the streams that may use the workspace as it is: the one that zeroed it, and those of _join
            self._joined = {torch._C._cuda_getCurrentRawStream(self._index) or None}
        # the arguments that a clipping call passes on: how many, and addresses
        self._at = [n, *self._tables_at, 0 if self._counted is None else ctypes.addressof(self._counted), self._ws.data_ptr()]

    def _tabulate(self):
        self._numels = self._table("grads", self.grads)
        self._dtypes = _i32([_dtype_code(g) for g in self.grads])
        self._ptrs = _ptrs([g.data_ptr() for g in self.grads])
        self._tables_at = [ctypes.addressof(a) for a in (self._dtypes, self._numels, self._ptrs)]

    def _refresh(self):
        """Tables of the tensors as they are now: a tensor's storage can be replaced under it (``g.data = ...``, ``set_``),
        and the one tabulated be freed."""
        if _tables().unchanged(*self._at[:4], self.grads, self._index):
            return
        if len(self.grads) != self._at[0]:
            raise RtpError(-1, "GradGroup: %d tensors, built over %d" % (len(self.grads), self._at[0]))
        self._tabulate()
        self._at[1:4] = self._tables_at

    def _table(self, name, ts):
        for i, t in enumerate(ts):
            _dtype_code(t)
            if not t.is_contiguous():
                raise RtpError(-1, "GradGroup: %s[%d] must be contiguous (row-major)" % (name, i))
            if t.device != self.device:
                raise RtpError(-1, "GradGroup: %s[%d] is on %s, the group on %s" % (name, i, t.device, self.device))
        return _i64([t.numel() for t in ts])

    def _join(self, handle):
        """The first call on another stream than the workspace's own: that stream waits until the workspace is zero, and
        keeps it, should the group be dropped, until its work is done. A capturing stream can do neither: a capture
        begins with all earlier work complete, and its graph is replayed only as long as the group is kept."""
        torch = _torch()
        s = torch.cuda.ExternalStream(handle, self.device) if handle else torch.cuda.default_stream(self.device)
        with torch.cuda.stream(s):
            if torch.cuda.is_current_stream_capturing():
                return
            if self._zeroed is not None:
                s.wait_event(self._zeroed)
        self._ws.record_stream(s)
        self._joined.add(handle)

    def _begin(self, stream):
        """(the norm's buffer, the handle of the stream to run on)"""
        torch = _torch()
        if torch._C._cuda_getDevice() != self.device.index:
            raise RtpError(-1, "GradGroup: tensors are on %s but the current CUDA device is %d" % (
                self.device, torch.cuda.current_device()))
        self._refresh()
        handle = _stream_ptr(stream)
        if handle not in self._joined:
            self._join(handle)
        return _new(1, (), torch.float32, self.device.index, stream)[0], handle

    def norm(self, stream=None):
        """The global norm, a float32 scalar tensor on the GPU."""
        norm, handle = self._begin(stream)
        _check(_load().rtp_grad_norm(len(self.grads), self._dtypes, self._numels, self._ptrs, self._counted,
                                     self._ws.data_ptr(), norm.data_ptr(), handle))
        return norm

    def clip(self, max_norm: float, out=None, stream=None):
        """Scales every tensor by min(1, max_norm / (norm + 1e-6)), in place or into the tensors of `out` (same types
        and sizes). Returns (norm, list of the tensors written)."""
        if stream is None and _torch()._C._cuda_getDevice() == self._index:
            handle = _stream_ptr(None)
            if handle not in self._joined:
                self._join(handle)
            norm = _called((_ext or _tables()).clip(*self._at, max_norm, out, self.grads, self._index, handle or 0))
            if norm is not None:
                return norm, (list(self.grads) if out is None else out)
        norm, handle = self._begin(stream)
        optr = None
        if out is not None:
            out = _listed(out)
            if len(out) != len(self.grads):
                raise RtpError(-1, "GradGroup: %d out tensors for %d gradients" % (len(out), len(self.grads)))
            optr = _tables().like(out, self.grads, self.device.index)
            if type(optr) is int:
                o, g = out[optr], self.grads[optr]
                if not isinstance(o, _torch().Tensor):
                    raise RtpError(-1, "GradGroup: out[%d] is no tensor" % optr)
                raise RtpError(-2, "GradGroup: out[%d] is %s %s on %s, expected contiguous %s %s on %s" % (
                    optr, o.dtype, tuple(o.shape), o.device, g.dtype, tuple(g.shape), self.device))
        _check(_load().rtp_clip_grad_norm(len(self.grads), self._dtypes, self._numels, self._ptrs, self._counted,
                                          float(max_norm), optr, self._ws.data_ptr(), norm.data_ptr(), handle))
        return norm, (list(self.grads) if out is None else out)


def grad_norm(grads, counted=None, stream=None):
    """Global norm of a list of gradients (GradGroup.norm without keeping a group)."""
    return GradGroup._for_one_call(grads, counted, stream).norm(stream)


def clip_grad_norm(grads, max_norm: float, counted=None, out=None, stream=None):
    """Clips a list of gradients by their global norm (GradGroup.clip without keeping a group)."""
    return GradGroup._for_one_call(grads, counted, stream).clip(max_norm, out, stream)


def device_error(stream=None) -> int:
    """Reads and clears the device word set when a tensor-core kernel's bounded wait gave up."""
    code = ctypes.c_uint32()
    _check(_load().rtp_device_error(_stream_ptr(stream), ctypes.byref(code)))
    return code.value


def wait_selftest(limit_ns: int, out=None, stream=None, kernel: int = 0):
    """Runs a bounded-wait self-test kernel (a wait on a barrier that nothing
    completes, given up after limit_ns): kernel 0 the tensor-core kernel's
    wait, 1 the resharding kernel's. Returns the uint32 device tensor of
    outcomes (1 = that waiter gave up)."""
    torch = _torch()
    if out is None:
        out = torch.zeros(4, dtype=torch.int32, device="cuda")
    if out.numel() < 2 or out.element_size() != 4 or out.dtype.is_floating_point:
        raise RtpError(-1, "wait_selftest: out must hold at least 2 int32 values")
    _check_cuda([out], "wait_selftest")
    _check(_load().rtp_wait_selftest(int(kernel), int(limit_ns), out.data_ptr(), _stream_ptr(stream)))
    return out


HOOK_NONE, HOOK_PLAN_SHIFT, HOOK_FAIL_ALLOC, HOOK_NO_CLUSTERS, HOOK_WAIT_LIMIT = 0, 1, 2, 3, 4


def test_hook(hook: int, arg: int = 0) -> None:
    """Arms a one-shot host-side fault for this thread's next reshard plan
    (rtp_test_hook): HOOK_PLAN_SHIFT moves a planned destination offset by
    `arg` elements, HOOK_FAIL_ALLOC fails the planner's next allocation; or,
    HOOK_NO_CLUSTERS, for its next product of more than 128 rows: clusters of
    `arg` or more CTAs find no room; HOOK_WAIT_LIMIT, for its next one of up to
    128 rows: waits give up after `arg` ns."""
    _check(_load().rtp_test_hook(int(hook), int(arg)))


def product_launches() -> dict:
    """Launches of each form by this thread's tp_linear, tp_glu and gradient calls since it last asked: "few" (up to 128
    rows), "whole" (tiles of one SM pair), and 2, 3, 4 (pairs that share a tile's K range)."""
    counts = (ctypes.c_int32 * 5)()
    _check(_load().rtp_product_launches(counts))
    return dict(zip(("few", "whole", 2, 3, 4), counts))


def version() -> str:
    return _load().rtp_version().decode()
