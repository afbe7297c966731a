"""The operators around and beside the Comba recurrence: short causal convolution,
selective scan, gated norm and residual norm, each with its backward and, where a model
decodes with it, its single-token form.

As in the package's other functions, these check tensors, allocate what the caller does
not pass, and call the C ABI (``include/comba.h``, which states every formula).  Token
tensors are [B, T, C], or packed [total_T, C] with ``cu_seqlens`` (int32 [N + 1] on the
device).  Workspaces come from PyTorch's allocator, one per call, so calls on several
streams and captured graphs do not share them.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

import chunk_delta_rule_b200 as _cdr

__all__ = ["short_conv", "short_conv_bwd", "short_conv_step", "selective_scan", "selective_scan_bwd",
           "selective_scan_step", "gated_norm", "gated_norm_bwd", "residual_norm", "residual_norm_bwd"]

_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
_F32 = torch.float32


def _tensor(t, name: str, dtype, shape, index: int, optional: bool = False) -> None:
    """Refuses ``t`` unless it is a contiguous tensor of this type and shape on CUDA device
    ``index`` (decode steps are short enough for the checks to count: one expression
    passes what is right, and only a wrong tensor is looked at closely)."""
    if t is None and optional:
        return
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.is_cuda and t.get_device() == index):
        return
    _cdr._check(t, name, dtype, shape)
    raise ValueError(f"{name} must be on cuda:{index} (got {t.device})")


def _element(t, name: str) -> torch.dtype:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name} must be bf16 or fp32 (got {t.dtype})")
    return t.dtype


def _device(t, name: str) -> int:
    """The CUDA device of a call, from its first tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    return t.get_device()


class _Call:
    """One call of the library on the device of its first tensor.  Buffers that are
    allocated here for a stream other than the current one come from that stream's memory,
    which nothing on the current one may still be using, and are known to the current
    stream, which is likely to read them."""
    __slots__ = ("first", "index", "stream")

    def __init__(self, first, index: int, stream):
        self.first, self.index, self.stream = first, index, None
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=index)
            if stream.cuda_stream != torch.cuda.current_stream(index).cuda_stream:
                self.stream = stream

    def _alloc(self, make):
        if self.stream is None:
            return make()
        with torch.cuda.stream(self.stream):
            t = make()
        t.record_stream(torch.cuda.current_stream(self.index))
        return t

    def new(self, shape, dtype):
        return self._alloc(lambda: self.first.new_empty(shape, dtype=dtype))

    def like(self, t):
        if self.stream is None:
            return torch.empty_like(t)   # of a contiguous tensor: the quickest allocation
        return self._alloc(lambda: torch.empty_like(t))

    def workspace(self, nbytes: int, given: Optional[torch.Tensor]):
        if given is None:
            return self.new((max(int(nbytes), 16),), torch.uint8)
        if given.dtype != torch.uint8 or not given.is_cuda or given.get_device() != self.index or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{self.index}")
        return given

    def __call__(self, name: str, *args) -> None:
        fn = getattr(_cdr.library(), name)
        args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
        handle = torch._C._cuda_getCurrentRawStream(self.index) if self.stream is None else self.stream.cuda_stream
        if torch.cuda.current_device() == self.index:
            st = fn(*args, handle)
        else:
            with torch.cuda.device(self.index):
                st = fn(*args, handle)
        if st != 0:
            raise _cdr.CombaError(st, name)


_INT_MAX = 0x7FFFFFFF


def _ints(name: str, *sizes: int) -> None:
    """Refuses sizes that the C ABI's ints cannot hold (ctypes would cut them).  A decode
    step asks only once a comparison has found one: a call here is 0.35 us."""
    if max(sizes, default=0) > _INT_MAX:
        raise ValueError(f"{name} must have dimensions below 2^31 (got {sizes})")


def _tokens(x, cu_seqlens, name: str = "x"):
    """(leading shape, N, T, C) of a token tensor: N sequences of T tokens, or T packed."""
    _element(x, name)
    _ints(name, *x.shape)
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError(f"{name} must be [B, T, C]")
        return tuple(x.shape[:2]), x.shape[0], x.shape[1], x.shape[2]
    if x.dim() != 2:
        raise ValueError(f"{name} must be [total_T, C] with cu_seqlens")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N + 1]")
    _ints("cu_seqlens", cu_seqlens.numel() - 1)
    return (x.shape[0],), cu_seqlens.numel() - 1, x.shape[0], x.shape[1]


def _filter(weight, C: int, dev):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    if W > _INT_MAX:
        _ints("weight", W)
    _tensor(weight, "weight", _F32, (C, W), dev)
    return W


def short_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
               silu: bool = True, out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
               return_state: bool = True, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """comba_short_conv_fwd: causal convolution of W (2, 3 or 4) taps per channel, with
    SiLU unless ``silu`` is False.  x [B,T,C] or packed [total_T,C], bf16 or fp32; weight
    [C,W], bias [C] or None fp32; initial_state [N,W-1,C] (the inputs before each
    sequence, oldest first) or None.  Returns (out like x, final_state [N,W-1,C] or None)."""
    lead, N, T, C = _tokens(x, cu_seqlens)
    dt, dev, shape = x.dtype, _device(x, "x"), x.shape
    _tensor(x, "x", dt, shape, dev)
    W = _filter(weight, C, dev)
    _tensor(bias, "bias", _F32, (C,), dev, True)
    _tensor(initial_state, "initial_state", dt, (N, W - 1, C), dev, True)
    _tensor(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev, True)
    call = _Call(x, dev, stream)
    if out is None:
        out = call.like(x)
    else:
        _tensor(out, "out", dt, shape, dev)
    if final_state is None and return_state:
        final_state = call.new((N, W - 1, C), dt)
    _tensor(final_state, "final_state", dt, (N, W - 1, C), dev, True)
    call("comba_short_conv_fwd", x, weight, bias, initial_state, out, final_state, cu_seqlens, N, T, C, W, int(silu),
         _DTYPE[dt])
    return out, final_state


def short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, dout: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, silu: bool = True,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """comba_short_conv_bwd: gradients of <dout, out> + <dfinal_state, final_state> of
    short_conv.  Returns a dict of dx (like x), dweight, dbias (None without bias) in fp32
    and dinitial_state (None without initial_state).  ``workspace``: a uint8 device tensor
    of at least comba_short_conv_bwd_workspace_size bytes, for this call alone."""
    lead, N, T, C = _tokens(x, cu_seqlens)
    dt, dev, shape = x.dtype, _device(x, "x"), x.shape
    _tensor(x, "x", dt, shape, dev)
    W = _filter(weight, C, dev)
    _tensor(dout, "dout", dt, shape, dev)
    _tensor(bias, "bias", _F32, (C,), dev, True)
    _tensor(initial_state, "initial_state", dt, (N, W - 1, C), dev, True)
    _tensor(dfinal_state, "dfinal_state", dt, (N, W - 1, C), dev, True)
    _tensor(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev, True)
    call = _Call(x, dev, stream)
    g = {"dx": call.like(x), "dweight": call.new((C, W), _F32),
         "dbias": None if bias is None else call.new((C,), _F32),
         "dinitial_state": None if initial_state is None else call.new((N, W - 1, C), dt)}
    need = _cdr.library().comba_short_conv_bwd_workspace_size(N, T, C, W, int(cu_seqlens is not None))
    ws = call.workspace(need, workspace)
    call("comba_short_conv_bwd", x, weight, bias, initial_state, dout, dfinal_state, g["dx"], g["dweight"], g["dbias"],
         g["dinitial_state"], cu_seqlens, N, T, C, W, int(silu), _DTYPE[dt], ws, ws.numel())
    return g


def short_conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    silu: bool = True, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """comba_short_conv_step: one token, x [B,C]; ``state`` [B,W-1,C] moves on in place.
    Returns out [B,C]."""
    dt = _element(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [B, C]")
    B, C = x.shape
    if B > _INT_MAX or C > _INT_MAX:
        _ints("x", B, C)
    dev = _device(x, "x")
    _tensor(x, "x", dt, (B, C), dev)
    W = _filter(weight, C, dev)
    _tensor(state, "state", dt, (B, W - 1, C), dev)
    _tensor(bias, "bias", _F32, (C,), dev, True)
    call = _Call(x, dev, stream)
    if out is None:
        out = call.new((B, C), dt)
    _tensor(out, "out", dt, (B, C), dev)
    call("comba_short_conv_step", x, weight, bias, state, out, B, C, W, int(silu), _DTYPE[dt])
    return out


def _groups_states(Bm):
    G, N = Bm.shape[-2:]
    if G > _INT_MAX or N > _INT_MAX:
        _ints("Bm", G, N)
    return G, N


def _scan_inputs(lead, C, x, dt, A_log, Bm, Cm, D, dt_bias, z):
    """(groups, states) of a scan whose token tensors have the leading shape ``lead``."""
    et, dev, shape = x.dtype, _device(x, "x"), x.shape
    _tensor(x, "x", et, shape, dev)
    _tensor(dt, "dt", et, shape, dev)
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != len(lead) + 2:
        raise ValueError("Bm must be [..., G, N]")
    G, N = _groups_states(Bm)
    _tensor(A_log, "A_log", _F32, (C, N), dev)
    _tensor(Bm, "Bm", et, (*lead, G, N), dev)
    _tensor(Cm, "Cm", et, (*lead, G, N), dev)
    _tensor(D, "D", _F32, (C,), dev, True)
    _tensor(dt_bias, "dt_bias", _F32, (C,), dev, True)
    _tensor(z, "z", et, shape, dev, True)
    return G, N


def selective_scan(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                   D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   h_final: Optional[torch.Tensor] = None, return_state: bool = True,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """comba_selective_scan_fwd: h_t = exp(delta A) h_{t-1} + delta x_t B_t, out_t =
    (sum_n h_t C_t + D x_t) silu(z_t), with delta = softplus(dt + dt_bias) and A =
    -exp(A_log).  x, dt, z [B,T,C] or packed [total_T,C], bf16 or fp32; Bm, Cm [...,G,N]
    of the same type (G dividing C; N 8 .. 128, a power of two); A_log [C,N], D and
    dt_bias [C] (or None), h0 [nseq,C,N] (or None) fp32.  Returns (out like x, h_final
    [nseq,C,N] fp32 or None).  ``h_final`` may be passed as ``h0`` itself.  ``workspace``: a
    uint8 device tensor of at least comba_selective_scan_fwd_workspace_size bytes (few long
    sequences run in pieces), for this call alone."""
    lead, nseq, T, C = _tokens(x, cu_seqlens)
    G, N = _scan_inputs(lead, C, x, dt, A_log, Bm, Cm, D, dt_bias, z)
    et, dev, shape = x.dtype, _device(x, "x"), x.shape
    _tensor(h0, "h0", _F32, (nseq, C, N), dev, True)
    _tensor(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), dev, True)
    call = _Call(x, dev, stream)
    if out is None:
        out = call.like(x)
    else:
        _tensor(out, "out", et, shape, dev)
    if h_final is None and return_state:
        h_final = call.new((nseq, C, N), _F32)
    _tensor(h_final, "h_final", _F32, (nseq, C, N), dev, True)
    need = _cdr.library().comba_selective_scan_fwd_workspace_size(nseq, T, C, G, N, int(cu_seqlens is not None))
    ws = call.workspace(need, workspace) if need or workspace is not None else None
    call("comba_selective_scan_fwd", x, dt, A_log, Bm, Cm, D, dt_bias, z, h0, out, h_final, cu_seqlens, nseq, T, C, G, N,
         _DTYPE[et], ws, 0 if ws is None else ws.numel())
    return out, h_final


def selective_scan_bwd(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                       dout: torch.Tensor, D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                       z: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                       dh_final: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """comba_selective_scan_bwd: gradients of <dout, out> + <dh_final, h_final> of
    selective_scan.  Returns a dict of dx, ddt, dBm, dCm, dz (of their inputs' type) and
    dA_log, dD, ddt_bias, dh0 (fp32); dz, dD, ddt_bias and dh0 are None where their input
    is.  ``workspace``: a uint8 device tensor of at least
    comba_selective_scan_bwd_workspace_size bytes, for this call alone."""
    lead, nseq, T, C = _tokens(x, cu_seqlens)
    G, N = _scan_inputs(lead, C, x, dt, A_log, Bm, Cm, D, dt_bias, z)
    et, dev, f32, shape = x.dtype, _device(x, "x"), _F32, x.shape
    _tensor(dout, "dout", et, shape, dev)
    _tensor(h0, "h0", f32, (nseq, C, N), dev, True)
    _tensor(dh_final, "dh_final", f32, (nseq, C, N), dev, True)
    _tensor(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), dev, True)
    call = _Call(x, dev, stream)
    g = {"dx": call.like(x), "ddt": call.like(x), "dA_log": call.new((C, N), f32),
         "dBm": call.new((*lead, G, N), et), "dCm": call.new((*lead, G, N), et),
         "dD": None if D is None else call.new((C,), f32),
         "ddt_bias": None if dt_bias is None else call.new((C,), f32),
         "dz": None if z is None else call.like(x),
         "dh0": None if h0 is None else call.new((nseq, C, N), f32)}
    need = _cdr.library().comba_selective_scan_bwd_workspace_size(nseq, T, C, G, N, int(cu_seqlens is not None))
    ws = call.workspace(need, workspace)
    call("comba_selective_scan_bwd", x, dt, A_log, Bm, Cm, D, dt_bias, z, h0, dout, dh_final, g["dx"], g["ddt"], g["dA_log"],
         g["dBm"], g["dCm"], g["dD"], g["ddt_bias"], g["dz"], g["dh0"], cu_seqlens, nseq, T, C, G, N, _DTYPE[et], ws,
         ws.numel())
    return g


def selective_scan_step(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                        h: torch.Tensor, D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """comba_selective_scan_step: one token, x, dt, z [B,C], Bm, Cm [B,G,N]; the state
    ``h`` [B,C,N] fp32 is updated in place.  Returns out [B,C]."""
    et = _element(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [B, C]")
    B, C = x.shape
    if B > _INT_MAX or C > _INT_MAX:
        _ints("x", B, C)
    dev = _device(x, "x")
    G, N = _scan_inputs((B,), C, x, dt, A_log, Bm, Cm, D, dt_bias, z)
    _tensor(h, "h", _F32, (B, C, N), dev)
    call = _Call(x, dev, stream)
    if out is None:
        out = call.new((B, C), et)
    _tensor(out, "out", et, (B, C), dev)
    call("comba_selective_scan_step", x, dt, A_log, Bm, Cm, D, dt_bias, z, h, out, B, C, G, N, _DTYPE[et])
    return out


def _norm_rows(x, name: str = "x"):
    dt = _element(x, name)
    if x.dim() < 1:
        raise ValueError(f"{name} must be [..., D]")
    D = x.shape[-1]
    if D > _INT_MAX:
        _ints(name, D)
    return dt, D, (x.numel() // D if D else 0)


def gated_norm(x: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """comba_gated_norm_fwd: x / sqrt(mean(x^2) + eps) * weight * silu(gate) over the last
    dimension, e.g. chunk_fwd's out [B,T,H,dv] per head.  x, gate [..., D] bf16 or fp32;
    weight [D] fp32; D <= 8192.  Returns out like x."""
    dt, D, rows = _norm_rows(x)
    dev = _device(x, "x")
    _tensor(x, "x", dt, x.shape, dev)
    _tensor(gate, "gate", dt, x.shape, dev)
    _tensor(weight, "weight", _F32, (D,), dev)
    call = _Call(x, dev, stream)
    if out is None:
        out = call.like(x)
    else:
        _tensor(out, "out", dt, x.shape, dev)
    call("comba_gated_norm_fwd", x, gate, weight, out, rows, D, float(eps), _DTYPE[dt])
    return out


def gated_norm_bwd(x: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, dout: torch.Tensor, eps: float = 1e-6,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """comba_gated_norm_bwd: gradients of <dout, out> of gated_norm, as a dict of dx, dgate
    (like x) and dweight [D] fp32."""
    dt, D, rows = _norm_rows(x)
    dev = _device(x, "x")
    _tensor(x, "x", dt, x.shape, dev)
    _tensor(gate, "gate", dt, x.shape, dev)
    _tensor(weight, "weight", _F32, (D,), dev)
    _tensor(dout, "dout", dt, x.shape, dev)
    call = _Call(x, dev, stream)
    g = {"dx": call.like(x), "dgate": call.like(x), "dweight": call.new((D,), _F32)}
    ws = call.workspace(_cdr.library().comba_gated_norm_bwd_workspace_size(rows, D), workspace)
    call("comba_gated_norm_bwd", x, gate, weight, dout, g["dx"], g["dgate"], g["dweight"], rows, D, float(eps), _DTYPE[dt],
         ws, ws.numel())
    return g


def _residual_inputs(x, stream_t, name, weight, scale, post_weight):
    dt, D, rows = _norm_rows(x)
    dev = _device(x, "x")
    _tensor(x, "x", dt, x.shape, dev)
    rt = _element(stream_t, name)
    if rt not in (dt, _F32):
        raise TypeError(f"{name} must be fp32 or of x's dtype (got {rt})")
    _tensor(stream_t, name, rt, x.shape, dev)
    _tensor(weight, "weight", _F32, (D,), dev)
    _tensor(scale, "scale", _F32, (D,), dev, True)
    _tensor(post_weight, "post_weight", _F32, (D,), dev, True)
    return dt, rt, D, rows, dev


def residual_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, scale: Optional[torch.Tensor] = None,
                  post_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                  h: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """comba_residual_norm_fwd: h = residual + scale * u and out = h / sqrt(mean(h^2) + eps)
    * weight, with u = x, or x's RMS norm times post_weight.  x [..., D] bf16 or fp32;
    residual of x's dtype or fp32; weight, scale, post_weight [D] fp32 (the last two or
    None).  Returns (out like x, h like residual); ``h`` may be ``residual`` itself."""
    dt, rt, D, rows, dev = _residual_inputs(x, residual, "residual", weight, scale, post_weight)
    call = _Call(x, dev, stream)
    if out is None:
        out = call.like(x)
    else:
        _tensor(out, "out", dt, x.shape, dev)
    if h is None:
        h = call.like(residual)
    else:
        _tensor(h, "h", rt, x.shape, dev)
    call("comba_residual_norm_fwd", x, residual, weight, scale, post_weight, out, h, rows, D, float(eps), _DTYPE[dt],
         _DTYPE[rt])
    return out, h


def residual_norm_bwd(x: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor,
                      dh: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                      post_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """comba_residual_norm_bwd: gradients of <dy, out> + <dh, h> of residual_norm, from x
    and the h it returned.  Returns a dict of dx (like x), dresidual (like h), and dweight,
    dscale, dpost_weight [D] fp32 (the last two None where their input is)."""
    dt, rt, D, rows, dev = _residual_inputs(x, h, "h", weight, scale, post_weight)
    _tensor(dy, "dy", dt, x.shape, dev)
    _tensor(dh, "dh", rt, x.shape, dev, True)
    call = _Call(x, dev, stream)
    f32 = _F32
    g = {"dx": call.like(x), "dresidual": call.like(h), "dweight": call.new((D,), f32),
         "dscale": None if scale is None else call.new((D,), f32),
         "dpost_weight": None if post_weight is None else call.new((D,), f32)}
    ws = call.workspace(_cdr.library().comba_residual_norm_bwd_workspace_size(rows, D), workspace)
    call("comba_residual_norm_bwd", x, h, weight, scale, post_weight, dy, dh, g["dx"], g["dresidual"], g["dweight"],
         g["dscale"], g["dpost_weight"], rows, D, float(eps), _DTYPE[dt], _DTYPE[rt], ws, ws.numel())
    return g
