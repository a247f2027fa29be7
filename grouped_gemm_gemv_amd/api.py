"""Python binding of libmoe with the C ABI's names.

Argument marshalling only: tensors are passed as device pointers, the stream
is torch's current HIP stream, and every step of the layer runs in the HIP
kernels of libmoe.  Element types: torch.float32 (MOE_F32) or torch.bfloat16
(MOE_BF16); indices int32; routing weights float32.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import _lib
from ._lib import (MoeBackwardSizes, MoeDispatch, MoeForwardViews, MoeResidual, MoeSaved8, MoeShape, MoeSizes, check, lib)

_DT = {torch.float32: _lib.MOE_F32, torch.bfloat16: _lib.MOE_BF16}
_TORCH_DT = {v: k for k, v in _DT.items()}


@dataclasses.dataclass(frozen=True)
class Shape:
    T: int
    d: int
    E: int
    k: int
    F: int
    capacity: int = 0
    dtype: torch.dtype = torch.bfloat16
    tile_rows: int = 0  # 0: the library chooses
    weight_layout: int = 0  # 0: row-major expert weights; 1: blocked 16-row order (moe_pack_blocked16)

    def c(self) -> MoeShape:
        return MoeShape(self.T, self.d, self.E, self.k, self.F, self.capacity, _DT[self.dtype], self.tile_rows,
                        self.weight_layout)

    def __getstate__(self):
        """The fields alone: the C struct that _c keeps here can be neither pickled nor copied."""
        return {f.name: getattr(self, f.name) for f in dataclasses.fields(self)}


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmoe takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libmoe takes contiguous tensors")
    return t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def query(shape: Shape) -> MoeSizes:
    out = MoeSizes()
    check("moe_query", lib().moe_query(ctypes.byref(shape.c()), ctypes.byref(out)))
    return out


def workspace_size(shape: Shape) -> int:
    """Bytes of workspace moe_forward needs (moe_workspace_size)."""
    n = ctypes.c_size_t()
    check("moe_workspace_size", lib().moe_workspace_size(ctypes.byref(shape.c()), ctypes.byref(n)))
    return n.value


class Dispatch:
    """Device buffer holding one moe_dispatch_t's arrays, with tensor views."""

    def __init__(self, shape: Shape, device="cuda", c: Optional[MoeDispatch] = None,
                 owner: Optional[torch.Tensor] = None):
        self.shape = shape
        if c is None:
            sz = query(shape)
            self.buf = torch.empty(sz.dispatch_bytes + 256, dtype=torch.uint8, device=device)
            base = (self.buf.data_ptr() + 255) // 256 * 256
            c = MoeDispatch()
            check("moe_dispatch_carve",
                  lib().moe_dispatch_carve(ctypes.byref(shape.c()), base, sz.dispatch_bytes, ctypes.byref(c)))
        else:
            self.buf = owner
        self.c = c

    def _view(self, name: str, n: int, dtype=torch.int32) -> torch.Tensor:
        ptr = getattr(self.c, name)
        off = ptr - self.buf.data_ptr()
        esz = torch.tensor([], dtype=dtype).element_size()
        return self.buf[off:off + n * esz].view(dtype)

    def arrays(self) -> dict:
        s, E, Tk = self.shape, self.shape.E, self.shape.T * self.shape.k
        R = _rows(s)
        mt = self.c.max_tiles
        return {
            "counts": self._view("counts", E),
            "offsets": self._view("offsets", E + 1),
            "spill_counts": self._view("spill_counts", E),
            "spill_offsets": self._view("spill_offsets", E + 1),
            "row_of": self._view("row_of", Tk),
            "token_of": self._view("token_of", R),
            "tile_off": self._view("tile_off", 2 * (E + 1)).view(2, E + 1),
            "tile_map": self._view("tile_map", 2 * mt * 4).view(2, mt, 4),
            "n_tiles": self._view("n_tiles", 2),
            "err_flags": self._view("err_flags", 1),
        }


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A device byte buffer whose data pointer is 256-byte aligned."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def moe_route(shape: Shape, x, w_router, bias, topk_ids, topk_w, stream=None):
    check("moe_route", lib().moe_route(ctypes.byref(shape.c()), _p(x), _p(w_router), _p(bias), _p(topk_ids),
                                       _p(topk_w), _stream(stream)))


def moe_permute(shape: Shape, x, topk_ids, disp: Dispatch, x_perm, ws, stream=None):
    check("moe_permute", lib().moe_permute(ctypes.byref(shape.c()), _p(x), _p(topk_ids), ctypes.byref(disp.c),
                                           _p(x_perm), _p(ws), ws.numel(), _stream(stream)))


def moe_ffn_gate_up(shape: Shape, x_perm, w_gate, w_up, disp: Dispatch, pass_idx: int, h, stream=None):
    check("moe_ffn_gate_up", lib().moe_ffn_gate_up(ctypes.byref(shape.c()), _p(x_perm), _p(w_gate), _p(w_up),
                                                   ctypes.byref(disp.c), pass_idx, _p(h), _stream(stream)))


def moe_ffn_gate_up_gather(shape: Shape, x, w_gate, w_up, disp: Dispatch, pass_idx: int, h, stream=None):
    check("moe_ffn_gate_up_gather", lib().moe_ffn_gate_up_gather(
        ctypes.byref(shape.c()), _p(x), _p(w_gate), _p(w_up), ctypes.byref(disp.c), pass_idx, _p(h),
        _stream(stream)))


LAYOUT_ROWS = 0
LAYOUT_BLOCKED16 = 1
# pass argument of the grouped GEMM calls: both passes of the capacity mode in one launch
PASS_BOTH = 2


def moe_pack_blocked16(src, dst=None, stream=None):
    """Re-store a [..., rows, K] weight tensor (rows % 16 == 0, K * itemsize % 64 == 0)
    in the blocked 16-row order; returns dst (allocated like src if None)."""
    if dst is None:
        dst = torch.empty_like(src)
    if src.shape != dst.shape or src.dtype != dst.dtype:
        raise ValueError("dst must match src")
    rows = src.shape[-2]
    row_bytes = src.shape[-1] * src.element_size()
    matrices = src.numel() // (src.shape[-1] * rows)
    check("moe_pack_blocked16", lib().moe_pack_blocked16(_p(src), _p(dst), matrices, rows, row_bytes,
                                                         _stream(stream)))
    return dst


def moe_ffn_gate_up_fp8(shape: Shape, x, w_gate, w_up, s_gate, s_up, disp: Dispatch, pass_idx: int, h,
                        stream=None):
    """Gate+up with E4M3 weight codes (uint8 [E,F,d]) and per-channel fp32 scales [E,F]."""
    check("moe_ffn_gate_up_fp8", lib().moe_ffn_gate_up_fp8(
        ctypes.byref(shape.c()), _p(x), _p(w_gate), _p(w_up), _p(s_gate), _p(s_up), ctypes.byref(disp.c),
        pass_idx, _p(h), _stream(stream)))


def _down_disp(disp: Dispatch, shape: Shape):
    """The C dispatch of a down GEMM call.  Where the call splits K, its partial sums [2][R][d] go to the
    dispatch's own buffer, whose size the library does not know: one carved for fewer or narrower rows is refused."""
    mine = disp.shape
    if (disp.c.kpart and shape.dtype is torch.bfloat16 and shape.F >= 128
            and _rows(mine) * mine.d < _rows(shape) * shape.d):
        raise ValueError(f"disp was made for {mine}: its partial sums of the down GEMM are too small for {shape}")
    return ctypes.byref(disp.c)


def moe_ffn_down_fp8(shape: Shape, h, w_down, s_down, disp: Dispatch, pass_idx: int, y_perm, stream=None):
    """Down projection with E4M3 weight codes (uint8 [E,d,F]) and per-channel fp32 scales [E,d]."""
    d = _down_disp(disp, shape)
    check("moe_ffn_down_fp8", lib().moe_ffn_down_fp8(ctypes.byref(shape.c()), _p(h), _p(w_down), _p(s_down),
                                                     d, pass_idx, _p(y_perm),
                                                     _stream(stream)))


def moe_ffn_down(shape: Shape, h, w_down, disp: Dispatch, pass_idx: int, y_perm, stream=None):
    d = _down_disp(disp, shape)
    check("moe_ffn_down", lib().moe_ffn_down(ctypes.byref(shape.c()), _p(h), _p(w_down), d,
                                             pass_idx, _p(y_perm), _stream(stream)))


def moe_grouped_ffn(shape: Shape, x_perm, w_gate, w_up, w_down, disp: Dispatch, h, y_perm, stream=None):
    d = _down_disp(disp, shape)
    check("moe_grouped_ffn", lib().moe_grouped_ffn(ctypes.byref(shape.c()), _p(x_perm), _p(w_gate), _p(w_up),
                                                   _p(w_down), d, _p(h), _p(y_perm),
                                                   _stream(stream)))


def moe_combine(shape: Shape, y_perm, topk_w, disp: Dispatch, out, stream=None):
    check("moe_combine", lib().moe_combine(ctypes.byref(shape.c()), _p(y_perm), _p(topk_w), ctypes.byref(disp.c),
                                           _p(out), _stream(stream)))


@dataclasses.dataclass
class ForwardViews:
    disp: Dispatch
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    x_perm: Optional[torch.Tensor]  # None: moe_forward reads x through token_of
    h: torch.Tensor
    y_perm: torch.Tensor


def _ws_view(ws: torch.Tensor, ptr: int, n: int, dtype) -> torch.Tensor:
    off = ptr - ws.data_ptr()
    esz = torch.tensor([], dtype=dtype).element_size()
    return ws[off:off + n * esz].view(dtype)


def _forward_views(shape: Shape, v, ws, topk_ids, topk_w) -> ForwardViews:
    R = query(shape).rows
    Tk = shape.T * shape.k
    s = shape
    ids = topk_ids if topk_ids is not None else _ws_view(ws, v.topk_ids, Tk, torch.int32).view(s.T, s.k)
    wts = topk_w if topk_w is not None else _ws_view(ws, v.topk_w, Tk, torch.float32).view(s.T, s.k)
    return ForwardViews(
        disp=Dispatch(shape, c=v.disp, owner=ws),
        topk_ids=ids, topk_w=wts,
        x_perm=None,
        h=_ws_view(ws, v.h, R * s.F, s.dtype).view(R, s.F),
        y_perm=_ws_view(ws, v.y_perm, R * s.d, s.dtype).view(R, s.d),
    )


def moe_forward(shape: Shape, x, w_router, bias, topk_ids, topk_w, w_gate, w_up, w_down, out, ws,
                stream=None) -> ForwardViews:
    """The whole layer; returns views of the intermediates inside `ws`."""
    v = MoeForwardViews()
    check("moe_forward", lib().moe_forward(ctypes.byref(shape.c()), _p(x), _p(w_router), _p(bias), _p(topk_ids),
                                           _p(topk_w), _p(w_gate), _p(w_up), _p(w_down), _p(out), _p(ws),
                                           ws.numel(), ctypes.byref(v), _stream(stream)))
    return _forward_views(shape, v, ws, topk_ids, topk_w)


def moe_forward_fp8(shape: Shape, x, w_router, bias, topk_ids, topk_w, w_gate, w_up, w_down, s_gate, s_up,
                    s_down, out, ws, stream=None) -> ForwardViews:
    """The whole layer with E4M3 expert weight codes and per-channel fp32 scales."""
    v = MoeForwardViews()
    check("moe_forward_fp8", lib().moe_forward_fp8(
        ctypes.byref(shape.c()), _p(x), _p(w_router), _p(bias), _p(topk_ids), _p(topk_w), _p(w_gate), _p(w_up),
        _p(w_down), _p(s_gate), _p(s_up), _p(s_down), _p(out), _p(ws), ws.numel(), ctypes.byref(v),
        _stream(stream)))
    return _forward_views(shape, v, ws, topk_ids, topk_w)


def moe_forward_noalloc(shape: Shape, x, w_router, bias, topk_ids, topk_w, w_gate, w_up, w_down, out,
                        stream=None) -> MoeForwardViews:
    """The whole layer with the library's own device scratch array instead of a
    workspace (for callers that cannot allocate); returns the raw views struct
    (device addresses inside that array, valid until the next call)."""
    v = MoeForwardViews()
    check("moe_forward_noalloc", lib().moe_forward_noalloc(
        ctypes.byref(shape.c()), _p(x), _p(w_router), _p(bias), _p(topk_ids), _p(topk_w), _p(w_gate), _p(w_up),
        _p(w_down), _p(out), ctypes.byref(v), _stream(stream)))
    return v


# ---- backward pass ----


def _in(t: Optional[torch.Tensor], name: str, shape: tuple, dtype: torch.dtype, device) -> Optional[int]:
    """Device address of a tensor that must have this shape and type, contiguous on `device`; None stays None."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {list(shape)} of {dtype}, got {list(t.shape)} of {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return _p(t)  # says what else is wrong


def _c(s: Shape):
    """The C struct of a shape, by reference; made once for each Shape, which is immutable."""
    ref = s.__dict__.get("_cref")
    if ref is None:
        ref = ctypes.byref(s.c())
        object.__setattr__(s, "_cref", ref)
    return ref


def _rows(s: Shape) -> int:
    """R: rows of the dispatch's row space (moe_sizes_t.rows)."""
    Tk = s.T * s.k
    return s.E * s.capacity + max(0, Tk - s.capacity) if s.capacity > 0 else Tk


def _disp(disp: Dispatch, shape: Shape, device):
    """The C dispatch of a Dispatch that was made for this shape (d, F, storage order and tile height aside).
    None of the calls behind it writes the dispatch's partial sums, the only array whose size depends on d."""
    mine, other = disp.shape, shape
    if (mine.T, mine.E, mine.k, mine.capacity) != (other.T, other.E, other.k, other.capacity):
        raise ValueError(f"disp was made for {mine}")
    if disp.buf.device != device:
        raise ValueError(f"disp is on {disp.buf.device}, expected {device}")
    return ctypes.byref(disp.c)


def _weights(shape: Shape, prefix: str, gate, up, down, device):
    s = shape
    return (_in(gate, prefix + "_gate", (s.E, s.F, s.d), s.dtype, device),
            _in(up, prefix + "_up", (s.E, s.F, s.d), s.dtype, device),
            _in(down, prefix + "_down", (s.E, s.d, s.F), s.dtype, device))


def _ws(ws: torch.Tensor, device):
    if ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    return _p(ws), ws.numel() * ws.element_size()


_gpus = set()  # devices that are GPUs


def _call(name: str, device, stream, *args):
    """One entry point on the tensors' device, on `stream` or that device's current stream."""
    if device not in _gpus:  # (the name of its type takes longer to make than all else here)
        if device.type != "cuda":
            raise ValueError("libmoe takes device tensors")
        _gpus.add(device)
    index = device.index
    if stream is None:
        # (the handle alone: a Stream object around it takes longer than the rest of this function)
        s = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    else:
        s = stream.cuda_stream
    fn = getattr(lib(), name)
    if index == torch.cuda.current_device():
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    check(name, status)


def backward_query(shape: Shape) -> MoeBackwardSizes:
    """Bytes of the 8-bit projections and of the backward calls' workspaces (moe_backward_query)."""
    out = MoeBackwardSizes()
    check("moe_backward_query", lib().moe_backward_query(_c(shape), ctypes.byref(out)))
    return out


def backward_workspace_size(shape: Shape) -> int:
    """Bytes of workspace moe_backward needs; enough for every other backward call."""
    return backward_query(shape).backward_ws_bytes


class Saved8:
    """Device buffer of a layer's two projections in 8 bits (moe_saved8_t), with tensor views."""

    def __init__(self, shape: Shape, device="cuda"):
        self.shape = shape
        n = backward_query(shape).saved8_bytes
        self.buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
        base = (self.buf.data_ptr() + 255) // 256 * 256
        self.c = MoeSaved8()
        check("moe_saved8_carve", lib().moe_saved8_carve(_c(shape), base, n, ctypes.byref(self.c)))

    def arrays(self) -> dict:
        """gate, up [R, F] int8 codes; gate_exp, up_exp [R, F / 16] uint8 exponents."""
        R, F = _rows(self.shape), self.shape.F

        def view(ptr, cols, dtype):
            off = ptr - self.buf.data_ptr()
            return self.buf[off:off + R * cols].view(dtype).view(R, cols)

        return {"gate": view(self.c.gate, F, torch.int8), "up": view(self.c.up, F, torch.int8),
                "gate_exp": view(self.c.gate_exp, F // 16, torch.uint8),
                "up_exp": view(self.c.up_exp, F // 16, torch.uint8)}


def _saved(saved: Saved8, shape: Shape, device):
    mine, other = saved.shape, shape
    if (mine.T, mine.E, mine.k, mine.F, mine.capacity) != (other.T, other.E, other.k, other.F, other.capacity):
        raise ValueError(f"saved was made for {mine}")
    if saved.buf.device != device:
        raise ValueError(f"saved is on {saved.buf.device}, expected {device}")
    return ctypes.byref(saved.c)


def moe_ffn_gate_up_save8(shape: Shape, x, w_gate, w_up, disp: Dispatch, pass_idx: int, h, saved: Saved8,
                          stream=None):
    """Gate+up over a pass (x [T, d] read through the dispatch) that also keeps both projections in 8 bits."""
    s, dev = shape, x.device
    wg, wu, _ = _weights(s, "w", w_gate, w_up, None, dev)
    _call("moe_ffn_gate_up_save8", dev, stream, _c(s), _in(x, "x", (s.T, s.d), s.dtype, dev), wg, wu,
          _disp(disp, s, dev), pass_idx, _in(h, "h", (_rows(s), s.F), s.dtype, dev), _saved(saved, s, dev))


def moe_saved8_unpack(shape: Shape, saved: Saved8, disp: Dispatch, gate, up, stream=None):
    """The values the codes stand for, in bf16 (gate, up [R, F]); rows without a token are left as they are."""
    s, dev = shape, gate.device
    R = _rows(s)
    _call("moe_saved8_unpack", dev, stream, _c(s), _saved(saved, s, dev), _disp(disp, s, dev),
          _in(gate, "gate", (R, s.F), torch.bfloat16, dev), _in(up, "up", (R, s.F), torch.bfloat16, dev))


def moe_combine_backward(shape: Shape, dout, y_perm, topk_w, disp: Dispatch, dy_perm, dtopk_w, stream=None):
    """Gradient of moe_combine: dy_perm [R, d] and dtopk_w [T, k] (fp32)."""
    s, dev = shape, dout.device
    R = _rows(s)
    _call("moe_combine_backward", dev, stream, _c(s), _in(dout, "dout", (s.T, s.d), s.dtype, dev),
          _in(y_perm, "y_perm", (R, s.d), s.dtype, dev), _in(topk_w, "topk_w", (s.T, s.k), torch.float32, dev),
          _disp(disp, s, dev), _in(dy_perm, "dy_perm", (R, s.d), s.dtype, dev),
          _in(dtopk_w, "dtopk_w", (s.T, s.k), torch.float32, dev))


def moe_permute_backward(shape: Shape, dx_perm, disp: Dispatch, dx, stream=None):
    """Gradient of moe_permute's gather: dx [T, d] from dx_perm [R, d]."""
    s, dev = shape, dx_perm.device
    _call("moe_permute_backward", dev, stream, _c(s),
          _in(dx_perm, "dx_perm", (_rows(s), s.d), s.dtype, dev), _disp(disp, s, dev),
          _in(dx, "dx", (s.T, s.d), s.dtype, dev))


def moe_route_backward(shape: Shape, x, w_router, topk_ids, topk_w, dtopk_w, dx, dw_router, dbias, ws, stream=None):
    """Gradient of moe_route from the routing weights' gradient; dbias may be None."""
    s, dev = shape, x.device
    tk = (s.T, s.k)
    _call("moe_route_backward", dev, stream, _c(s), _in(x, "x", (s.T, s.d), s.dtype, dev),
          _in(w_router, "w_router", (s.E, s.d), s.dtype, dev), _in(topk_ids, "topk_ids", tk, torch.int32, dev),
          _in(topk_w, "topk_w", tk, torch.float32, dev), _in(dtopk_w, "dtopk_w", tk, torch.float32, dev),
          _in(dx, "dx", (s.T, s.d), s.dtype, dev), _in(dw_router, "dw_router", (s.E, s.d), s.dtype, dev),
          _in(dbias, "dbias", (s.E,), torch.float32, dev), *_ws(ws, dev))


def moe_grouped_ffn_backward(shape: Shape, x, dout, topk_w, w_gate, w_up, w_down, disp: Dispatch, saved: Saved8,
                             dx_perm, dtopk_w, dw_gate, dw_up, dw_down, ws, stream=None):
    """Gradient of the experts' products from the 8-bit projections.  dw_gate and dw_up (both or neither) and
    dw_down may be None: not computed."""
    s, dev = shape, x.device
    tk = (s.T, s.k)
    _call("moe_grouped_ffn_backward", dev, stream, _c(s), _in(x, "x", (s.T, s.d), s.dtype, dev),
          _in(dout, "dout", (s.T, s.d), s.dtype, dev), _in(topk_w, "topk_w", tk, torch.float32, dev),
          *_weights(s, "w", w_gate, w_up, w_down, dev), _disp(disp, s, dev), _saved(saved, s, dev),
          _in(dx_perm, "dx_perm", (_rows(s), s.d), s.dtype, dev),
          _in(dtopk_w, "dtopk_w", tk, torch.float32, dev), *_weights(s, "dw", dw_gate, dw_up, dw_down, dev),
          *_ws(ws, dev))


def moe_forward_save8(shape: Shape, x, w_router, bias, topk_ids, topk_w, w_gate, w_up, w_down, out, disp: Dispatch,
                      saved: Saved8, ws, stream=None):
    """The whole layer for training.  topk_ids and topk_w [T, k] are written where w_router is given, else read;
    disp and saved receive what moe_backward needs."""
    s, dev = shape, x.device
    tk = (s.T, s.k)
    _call("moe_forward_save8", dev, stream, _c(s), _in(x, "x", (s.T, s.d), s.dtype, dev),
          _in(w_router, "w_router", (s.E, s.d), s.dtype, dev), _in(bias, "bias", (s.E,), torch.float32, dev),
          _in(topk_ids, "topk_ids", tk, torch.int32, dev), _in(topk_w, "topk_w", tk, torch.float32, dev),
          *_weights(s, "w", w_gate, w_up, w_down, dev), _in(out, "out", (s.T, s.d), s.dtype, dev),
          _disp(disp, s, dev), _saved(saved, s, dev), *_ws(ws, dev))


def moe_backward(shape: Shape, x, w_router, topk_ids, topk_w, w_gate, w_up, w_down, disp: Dispatch, saved: Saved8,
                 dout, dx, dtopk_w, dw_router, dbias, dw_gate, dw_up, dw_down, ws, stream=None):
    """The whole layer's backward pass after moe_forward_save8.  w_router None: the routing was the caller's, and
    dw_router and dbias are None too."""
    s, dev = shape, x.device
    tk = (s.T, s.k)
    _call("moe_backward", dev, stream, _c(s), _in(x, "x", (s.T, s.d), s.dtype, dev),
          _in(w_router, "w_router", (s.E, s.d), s.dtype, dev), _in(topk_ids, "topk_ids", tk, torch.int32, dev),
          _in(topk_w, "topk_w", tk, torch.float32, dev), *_weights(s, "w", w_gate, w_up, w_down, dev),
          _disp(disp, s, dev), _saved(saved, s, dev), _in(dout, "dout", (s.T, s.d), s.dtype, dev),
          _in(dx, "dx", (s.T, s.d), s.dtype, dev), _in(dtopk_w, "dtopk_w", tk, torch.float32, dev),
          _in(dw_router, "dw_router", (s.E, s.d), s.dtype, dev), _in(dbias, "dbias", (s.E,), torch.float32, dev),
          *_weights(s, "dw", dw_gate, dw_up, dw_down, dev), *_ws(ws, dev))


# ---- the block around the layer ----


@dataclasses.dataclass(frozen=True)
class Residual:
    """What moe_residual does beside its arrays: eps of the norms, the residual branch's scale, dropout's p."""
    eps: float = 1e-6
    scale: float = 1.0
    dropout: float = 0.0

    def c(self, gate: int):
        """The C struct for a kind of gate, by reference; made once for each of the three."""
        refs = self.__dict__.get("_crefs")
        if refs is None:
            refs = tuple(ctypes.byref(MoeResidual(self.eps, self.scale, self.dropout, g)) for g in range(3))
            object.__setattr__(self, "_crefs", refs)
        return refs[gate]

    def __getstate__(self):
        """The fields alone, as Shape's."""
        return {f.name: getattr(self, f.name) for f in dataclasses.fields(self)}


def _gate(gate, s: Shape, name: str, device):
    """moe_gate_t and the address of a gate [T] (one value a token) or [T, d], or None."""
    if gate is None:
        return _lib.GATE_NONE, None
    full = gate.dim() != 1
    want = (s.T, s.d) if full else (s.T,)
    return _lib.GATE_FULL if full else _lib.GATE_TOKEN, _in(gate, name, want, s.dtype, device)


def _rng(rng, device):
    return _in(rng, "rng", (2,), torch.int64, device)


def residual_workspace_size(shape: Shape) -> int:
    """Bytes of workspace of moe_norm_backward and moe_residual_backward."""
    n = ctypes.c_size_t()
    check("moe_residual_workspace_size", lib().moe_residual_workspace_size(_c(shape), ctypes.byref(n)))
    return n.value


def moe_norm(shape: Shape, x, w, n, eps: float = 1e-6, stream=None):
    """n = x / rms(x) w for every row of x [T, d]; w [d]."""
    s, dev = shape, x.device
    _call("moe_norm", dev, stream, _c(s), _in(x, "x", (s.T, s.d), s.dtype, dev), _in(w, "w", (s.d,), s.dtype, dev), eps,
          _in(n, "n", (s.T, s.d), s.dtype, dev))


def moe_norm_backward(shape: Shape, x, w, dn, dres, dx, dw, ws, eps: float = 1e-6, stream=None):
    """Gradient of moe_norm: dx = dres + the norm's (dres may be None, and dx may be dres); dw [d], or None."""
    s, dev = shape, x.device
    Td = (s.T, s.d)
    _call("moe_norm_backward", dev, stream, _c(s), _in(x, "x", Td, s.dtype, dev), _in(w, "w", (s.d,), s.dtype, dev), eps,
          _in(dn, "dn", Td, s.dtype, dev), _in(dres, "dres", Td, s.dtype, dev), _in(dx, "dx", Td, s.dtype, dev),
          _in(dw, "dw", (s.d,), s.dtype, dev), *_ws(ws, dev))


def moe_residual(shape: Shape, r: Residual, res, y, post_w, gate, rng, next_w, out, n, stream=None):
    """out = res + scale sigmoid(gate) dropout(y / rms(y) post_w) and n = out / rms(out) next_w.

    post_w, gate ([T] or [T, d]) and next_w with n may be None; rng int64 [2] on the device (seed, step), None without
    dropout; out may be res."""
    s, dev = shape, y.device
    Td = (s.T, s.d)
    kind, g = _gate(gate, s, "gate", dev)
    _call("moe_residual", dev, stream, _c(s), r.c(kind), _in(res, "res", Td, s.dtype, dev),
          _in(y, "y", Td, s.dtype, dev), _in(post_w, "post_w", (s.d,), s.dtype, dev), g, _rng(rng, dev),
          _in(next_w, "next_w", (s.d,), s.dtype, dev), _in(out, "out", Td, s.dtype, dev), _in(n, "n", Td, s.dtype, dev))


def moe_residual_backward(shape: Shape, r: Residual, out, y, post_w, gate, rng, next_w, dout, dn, dres, dy, dgate,
                          dpost_w, dnext_w, ws, stream=None):
    """Gradient of moe_residual from those of out (or None) and n (with next_w); `out` is what the forward call left.
    dgate, dpost_w and dnext_w may be None: not computed.  dres may be dout."""
    s, dev = shape, y.device
    Td = (s.T, s.d)
    kind, g = _gate(gate, s, "gate", dev)
    if dgate is not None and (gate is None or dgate.shape != gate.shape):
        raise ValueError("dgate must have the gate's shape")
    _call("moe_residual_backward", dev, stream, _c(s), r.c(kind), _in(out, "out", Td, s.dtype, dev),
          _in(y, "y", Td, s.dtype, dev), _in(post_w, "post_w", (s.d,), s.dtype, dev), g, _rng(rng, dev),
          _in(next_w, "next_w", (s.d,), s.dtype, dev), _in(dout, "dout", Td, s.dtype, dev),
          _in(dn, "dn", Td, s.dtype, dev), _in(dres, "dres", Td, s.dtype, dev), _in(dy, "dy", Td, s.dtype, dev),
          _gate(dgate, s, "dgate", dev)[1], _in(dpost_w, "dpost_w", (s.d,), s.dtype, dev),
          _in(dnext_w, "dnext_w", (s.d,), s.dtype, dev), *_ws(ws, dev))


def moe_dropout(x, p: float, rng, out, stream=None):
    """out = x where kept, over 1 - p; any contiguous x of fp32 or bf16, and out like it (or x itself).  The same call
    on a gradient is the gradient.  rng int64 [2] on the device: seed, step."""
    if x.dtype not in _DT:
        raise ValueError(f"x must be fp32 or bf16, got {x.dtype}")
    dev = x.device
    _call("moe_dropout", dev, stream, _in(x, "x", x.shape, x.dtype, dev), x.numel(), _DT[x.dtype], p, _rng(rng, dev),
          _in(out, "out", x.shape, x.dtype, dev))


# ---- the layer for a few tokens ----


def decode_workspace_size(shape: Shape) -> int:
    """Bytes of workspace of moe_decode and moe_decode_fp8."""
    n = ctypes.c_size_t()
    check("moe_decode_workspace_size", lib().moe_decode_workspace_size(_c(shape), ctypes.byref(n)))
    return n.value


def _decode(name, shape: Shape, x, norm_w, w_router, bias, topk_ids, topk_w, weights, res, out, ws, eps, scale, stream):
    s, dev = shape, x.device
    tk = (s.T, s.k)
    _call(name, dev, stream, _c(s), _in(x, "x", (s.T, s.d), s.dtype, dev), _in(norm_w, "norm_w", (s.d,), s.dtype, dev),
          eps, _in(w_router, "w_router", (s.E, s.d), s.dtype, dev), _in(bias, "bias", (s.E,), torch.float32, dev),
          _in(topk_ids, "topk_ids", tk, torch.int32, dev), _in(topk_w, "topk_w", tk, torch.float32, dev), *weights,
          _in(res, "res", (s.T, s.d), s.dtype, dev), scale, _in(out, "out", (s.T, s.d), s.dtype, dev), *_ws(ws, dev))


def moe_decode(shape: Shape, x, norm_w, w_router, bias, topk_ids, topk_w, w_gate, w_up, w_down, res, out, ws,
               eps: float = 1e-6, scale: float = 1.0, stream=None):
    """The layer for up to 16 tokens, with the norm before it (norm_w) and the residual behind it (res; out may be
    res): out = res + scale layer(x / rms(x) norm_w).  norm_w, bias and res may be None.  With w_router the routing is
    computed, and written to topk_ids and topk_w [T, k] where they are given; without it they are read.  9 to 16 wide
    tokens and few, large experts are faster with moe_norm and moe_forward."""
    weights = _weights(shape, "w", w_gate, w_up, w_down, x.device)
    _decode("moe_decode", shape, x, norm_w, w_router, bias, topk_ids, topk_w, weights, res, out, ws, eps, scale, stream)


def moe_decode_fp8(shape: Shape, x, norm_w, w_router, bias, topk_ids, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down,
                   res, out, ws, eps: float = 1e-6, scale: float = 1.0, stream=None):
    """moe_decode with E4M3 expert weight codes (uint8) and per-channel fp32 scales."""
    s, dev = shape, x.device
    up, down = (s.E, s.F, s.d), (s.E, s.d, s.F)
    weights = [_in(w, n, sh, torch.uint8, dev)
               for w, n, sh in ((w_gate, "w_gate", up), (w_up, "w_up", up), (w_down, "w_down", down))]
    weights += [_in(v, n, sh, torch.float32, dev)
                for v, n, sh in ((s_gate, "s_gate", up[:2]), (s_up, "s_up", up[:2]), (s_down, "s_down", down[:2]))]
    _decode("moe_decode_fp8", s, x, norm_w, w_router, bias, topk_ids, topk_w, weights, res, out, ws, eps, scale, stream)
