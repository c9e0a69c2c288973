"""The expert layer's calls (include/rnl.h): rows into MXFP8, routing, products
grouped by expert, the weighted sum back.

The rules of _native.py (checks, outputs and workspace of the call's stream),
with the checks written for calls of a few microseconds: one test a tensor,
and the messages of _native._need where it fails.
"""
from __future__ import annotations

import collections
import functools

import torch

from . import _native as nat

_BF16, _U8, _I32, _F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


def _check(t, name, dtype, shape, dev):
    """A contiguous tensor of that type, shape and device; its address."""
    if t is None or t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        nat._need(t, name, dtype, shape, dev)
    return t.data_ptr()


def _output(t, name, dtype, shape, dev, stream):
    """The caller's output, checked, or a new one on the call's stream."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev) if stream is None else nat._new(shape, dtype, dev, stream)
    _check(t, name, dtype, shape, dev)
    return t


def _stream(dev, stream):
    """The raw stream of a call on dev (nat._stream for everything but the current
    stream of the current device, refusals among it)."""
    if stream is None and dev.type == "cuda" and dev.index == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(dev.index)
    return nat._stream(dev, stream)


# a function of the sizes alone; the call itself is 1 us of a small call's 10
_workspace_size = functools.lru_cache(maxsize=256)(nat.workspace_size)


def _space(nbytes, dev, given, stream):
    """(address, bytes) of the workspace and what keeps it alive; none where none is needed."""
    if given is None:
        if nbytes == 0:
            return None, 0, None
        given = nat._workspace(nbytes, dev, None, stream)
    elif given.device != dev:
        raise ValueError(f"workspace must be on {dev}, got {given.device}")
    return given.data_ptr(), given.numel() * given.element_size(), given


def _blocks(K, block):
    """Blocks of a row; sizes that the call refuses have none."""
    return K // block if block > 0 else 0


def rnl_add_rmsnorm_mxfp8(x, gamma=None, residual=None, x_sum_out=None, eps=1e-6, norm_mode=nat.NORM_RSQRT, block=64,
                          codes_out=None, scale_out=None, stream=None):
    """Residual add (optional), RMSNorm and MX quantisation of the rows of x [T, K]
    (bf16): returns (E4M3 codes uint8 [T, K], E8M0 scale bytes uint8
    [T, K / block]), the operand of mxfp8_scaled_mm and rnl_grouped_linear_mxfp8.
    x_sum_out may be x or residual (in-place add)."""
    shape = T, K = x.shape
    dev = x.device
    px = _check(x, "x", _BF16, shape, dev)
    pr = None if residual is None else _check(residual, "residual", _BF16, shape, dev)
    ps = None if x_sum_out is None else _check(x_sum_out, "x_sum_out", _BF16, shape, dev)
    pg = None if gamma is None else _check(gamma, "gamma", _BF16, (K,), dev)
    codes_out = _output(codes_out, "codes_out", _U8, shape, dev, stream)
    scale_out = _output(scale_out, "scale_out", _U8, (T, _blocks(K, block)), dev, stream)
    status = (nat._lib or nat.load()).rnl_add_rmsnorm_mxfp8(px, pr, ps, pg, T, K, eps, norm_mode, block, codes_out.data_ptr(),
                                              scale_out.data_ptr(), _stream(dev, stream))
    if status:
        raise nat.RnlError(status, "rnl_add_rmsnorm_mxfp8")
    return codes_out, scale_out


def rnl_quant_mxfp8(x, block=64, codes_out=None, scale_out=None, stream=None):
    """MX quantisation of the rows of x [T, K] (bf16) as they are; returns (codes, scale bytes)."""
    shape = T, K = x.shape
    dev = x.device
    px = _check(x, "x", _BF16, shape, dev)
    codes_out = _output(codes_out, "codes_out", _U8, shape, dev, stream)
    scale_out = _output(scale_out, "scale_out", _U8, (T, _blocks(K, block)), dev, stream)
    status = (nat._lib or nat.load()).rnl_quant_mxfp8(px, T, K, block, codes_out.data_ptr(), scale_out.data_ptr(),
                                        _stream(dev, stream))
    if status:
        raise nat.RnlError(status, "rnl_quant_mxfp8")
    return codes_out, scale_out


MoeRoute = collections.namedtuple("MoeRoute", "ids weights offsets rows slots")


def rnl_moe_route(logits, top_k, renormalize=True, ids_out=None, weights_out=None, offsets_out=None, rows_out=None,
                  slots_out=None, workspace=None, stream=None):
    """The top_k experts of every token (logits fp32 [T, E]), their softmax weights,
    and the tokens' rows grouped by expert: MoeRoute(ids [T, k], weights [T, k],
    offsets [E + 1], rows [T * k], slots [T, k])."""
    T, E = logits.shape
    dev = logits.device
    pl = _check(logits, "logits", _F32, (T, E), dev)
    k = min(max(top_k, 0), E)  # (the call refuses what is outside)
    ids = _output(ids_out, "ids_out", _I32, (T, k), dev, stream)
    weights = _output(weights_out, "weights_out", _F32, (T, k), dev, stream)
    offsets = _output(offsets_out, "offsets_out", _I32, (E + 1,), dev, stream)
    rows = _output(rows_out, "rows_out", _I32, (T * k,), dev, stream)
    slots = _output(slots_out, "slots_out", _I32, (T, k), dev, stream)
    pw, nw, _keep = _space(_workspace_size(nat.OP_MOE_ROUTE, T, k, E), dev, workspace, stream)
    status = (nat._lib or nat.load()).rnl_moe_route(pl, T, E, top_k, 1 if renormalize else 0, ids.data_ptr(), weights.data_ptr(),
                                      offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), pw, nw,
                                      _stream(dev, stream))
    if status:
        raise nat.RnlError(status, "rnl_moe_route")
    return MoeRoute(ids, weights, offsets, rows, slots)


def _rows_and_output(R, E, N, offsets, rows, swiglu, out, dev, stream):
    """What both grouped products check alike: (M, offsets' and rows' addresses, out)."""
    po = _check(offsets, "offsets", _I32, (E + 1,), dev)
    M, pr = R, None
    if rows is not None:
        M = rows.shape[0]
        pr = _check(rows, "rows", _I32, (M,), dev)
    return M, po, pr, _output(out, "out", _BF16, (M, N // 2 if swiglu else N), dev, stream)


def rnl_grouped_linear_bf16(x, W, offsets, rows=None, swiglu=False, out=None, workspace=None, stream=None):
    """out[i] = x[rows[i]] @ W[e]^T for the rows i of expert e (offsets[e] <= i <
    offsets[e + 1]; rows None: x[i]); with swiglu W[e] holds gate rows, then up
    rows, and out = silu(gate) * up.  x [R, K], W [E, N, K], out [M, N or N / 2]."""
    R, K = x.shape
    E, N = W.shape[0], W.shape[1]
    dev = x.device
    px, pW = _check(x, "x", _BF16, (R, K), dev), _check(W, "W", _BF16, (E, N, K), dev)
    M, po, pr, out = _rows_and_output(R, E, N, offsets, rows, swiglu, out, dev, stream)
    pw, nw, _keep = _space(_workspace_size(nat.OP_GROUPED, M, K, N, E), dev, workspace, stream)
    status = (nat._lib or nat.load()).rnl_grouped_linear_bf16(px, R, pW, E, N, K, po, pr, M, 1 if swiglu else 0, out.data_ptr(), pw,
                                                nw, _stream(dev, stream))
    if status:
        raise nat.RnlError(status, "rnl_grouped_linear_bf16")
    return out


def rnl_grouped_linear_mxfp8(x_codes, x_scale, w_codes, w_scale, offsets, rows=None, swiglu=False, block=64, out=None,
                             workspace=None, stream=None):
    """rnl_grouped_linear_bf16 on MXFP8 operands: codes uint8 [R, K] and [E, N, K],
    scale bytes uint8 [R, K / block] and [E, N, K / block]; bf16 out."""
    R, K = x_codes.shape
    E, N = w_codes.shape[0], w_codes.shape[1]
    dev = x_codes.device
    nb = _blocks(K, block)
    px, pxs = _check(x_codes, "x_codes", _U8, (R, K), dev), _check(x_scale, "x_scale", _U8, (R, nb), dev)
    pW, pWs = _check(w_codes, "w_codes", _U8, (E, N, K), dev), _check(w_scale, "w_scale", _U8, (E, N, nb), dev)
    M, po, pr, out = _rows_and_output(R, E, N, offsets, rows, swiglu, out, dev, stream)
    pw, nw, _keep = _space(_workspace_size(nat.OP_GROUPED, M, K, N, E), dev, workspace, stream)
    status = (nat._lib or nat.load()).rnl_grouped_linear_mxfp8(px, pxs, R, pW, pWs, E, N, K, block, po, pr, M, 1 if swiglu else 0,
                                                 out.data_ptr(), pw, nw, _stream(dev, stream))
    if status:
        raise nat.RnlError(status, "rnl_grouped_linear_mxfp8")
    return out


def rnl_moe_combine(y, slots, weights, residual=None, out=None, stream=None):
    """out[t] = residual[t] + sum_j weights[t, j] * y[slots[t, j]] (slots -1 left
    out); y [M, N] bf16, slots and weights [T, k]; out may be residual."""
    M, N = y.shape
    T, k = slots.shape
    dev = y.device
    py = _check(y, "y", _BF16, (M, N), dev)
    ps, pw = _check(slots, "slots", _I32, (T, k), dev), _check(weights, "weights", _F32, (T, k), dev)
    pr = None if residual is None else _check(residual, "residual", _BF16, (T, N), dev)
    out = _output(out, "out", _BF16, (T, N), dev, stream)
    status = (nat._lib or nat.load()).rnl_moe_combine(py, M, N, ps, pw, T, k, pr, out.data_ptr(), _stream(dev, stream))
    if status:
        raise nat.RnlError(status, "rnl_moe_combine")
    return out
