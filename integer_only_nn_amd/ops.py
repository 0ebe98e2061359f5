"""Thin Python binding of libionn.so: one function per C entry point, same
names, same argument order.  Arguments are torch tensors on a ROCm device
(PyTorch is used only for device memory and streams); this module only
checks dtypes/shapes and passes raw pointers.  Every computation runs in the
library's HIP kernels.  Outputs are caller-provided, as in the C ABI.
"""
import ctypes

import torch

from ._lib import ConvDesc, check, lib


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _p(t, dtype=None, numel=None, name="tensor"):
    """Device pointer of a contiguous tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor (no CPU path exists)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements, has {t.numel()}")
    return ctypes.c_void_p(t.data_ptr())


i8, i16, i32, u32 = torch.int8, torch.int16, torch.int32, torch.int32  # uint32 scalars held as int32


def ionn_fill_u32(dst, value=0, stream=None):
    check(lib().ionn_fill_u32(_p(dst, torch.int32, name="dst"), dst.numel(), value & 0xFFFFFFFF,
                              _stream(stream)), "ionn_fill_u32")


def ionn_absmax_i32(x, absmax, stream=None):
    check(lib().ionn_absmax_i32(_p(x, i32, name="x"), x.numel(), _p(absmax, u32, 1, "absmax"),
                                _stream(stream)), "ionn_absmax_i32")


def int_linear_fwd(X, W, Y, absmax_Y=None, stream=None):
    B, IN = X.shape
    OUT = W.shape[0]
    assert tuple(W.shape) == (OUT, IN) and tuple(Y.shape) == (B, OUT), "shape mismatch"
    check(lib().int_linear_fwd(_p(X, i8, name="X"), _p(W, i8, name="W"), _p(Y, i32, name="Y"),
                               B, IN, OUT, _p(absmax_Y, u32, 1, "absmax_Y"), _stream(stream)),
          "int_linear_fwd")


def int_linear_dgrad(dY, W, dX, relu_act=None, absmax_dX=None, stream=None):
    B, OUT = dY.shape
    IN = W.shape[1]
    assert tuple(W.shape) == (OUT, IN) and tuple(dX.shape) == (B, IN), "shape mismatch"
    if relu_act is not None:
        assert tuple(relu_act.shape) == (B, IN), "relu_act shape mismatch"
    check(lib().int_linear_dgrad(_p(dY, i8, name="dY"), _p(W, i8, name="W"),
                                 _p(relu_act, i8, name="relu_act"), _p(dX, i32, name="dX"), B, IN,
                                 OUT, _p(absmax_dX, u32, 1, "absmax_dX"), _stream(stream)),
          "int_linear_dgrad")


def int_linear_wgrad(dY, X, G, absmax_G=None, stream=None):
    B, OUT = dY.shape
    IN = X.shape[1]
    assert tuple(X.shape) == (B, IN) and tuple(G.shape) == (OUT, IN), "shape mismatch"
    check(lib().int_linear_wgrad(_p(dY, i8, name="dY"), _p(X, i8, name="X"), _p(G, i32, name="G"),
                                 B, IN, OUT, _p(absmax_G, u32, 1, "absmax_G"), _stream(stream)),
          "int_linear_wgrad")


def int_linear_wgrad_workspace_bytes(B, IN, OUT):
    return int(lib().int_linear_wgrad_workspace_bytes(int(B), int(IN), int(OUT)))


def int_linear_wgrad_ws(dY, X, G, workspace, absmax_G=None, stream=None):
    B, OUT = dY.shape
    IN = X.shape[1]
    assert tuple(X.shape) == (B, IN) and tuple(G.shape) == (OUT, IN), "shape mismatch"
    check(lib().int_linear_wgrad_ws(_p(dY, i8, name="dY"), _p(X, i8, name="X"), _p(G, i32, name="G"),
                                    B, IN, OUT, _p(absmax_G, u32, 1, "absmax_G"),
                                    _p(workspace, None, name="workspace"),
                                    workspace.numel() * workspace.element_size() if workspace is not None else 0,
                                    _stream(stream)), "int_linear_wgrad_ws")


def niti_quantize(acc, absmax, target_bits, relu, out, shift_out=None, stream=None):
    assert acc.numel() == out.numel()
    check(lib().niti_quantize(_p(acc, i32, name="acc"), acc.numel(), _p(absmax, u32, 1, "absmax"),
                              int(target_bits), int(bool(relu)), _p(out, i8, name="out"),
                              _p(shift_out, i32, 1, "shift_out"), _stream(stream)),
          "niti_quantize")


def niti_quantize_update(G, absmax, target_bits, mu_weight, W, shifts_out=None, gq_out=None,
                         stream=None):
    assert G.numel() == W.numel()
    check(lib().niti_quantize_update(_p(G, i32, name="G"), G.numel(), _p(absmax, u32, 1, "absmax"),
                                     int(target_bits), int(mu_weight), _p(W, i8, name="W"),
                                     _p(shifts_out, i32, 2, "shifts_out"),
                                     _p(gq_out, i32, G.numel(), "gq_out"), _stream(stream)),
          "niti_quantize_update")


def int_linear_step_small_fits(B, IN, OUT):
    return bool(lib().int_linear_step_small_fits(int(B), int(IN), int(OUT)))


def int_linear_step_small(X, W, dY, tb_w, mu_weight, tb_d, Y, dX, delta, G, maxima, shifts, gq=None,
                          stream=None):
    B, IN = X.shape
    OUT = W.shape[0]
    assert tuple(W.shape) == (OUT, IN) and tuple(dY.shape) == (B, OUT), "shape mismatch"
    assert tuple(Y.shape) == (B, OUT) and tuple(dX.shape) == (B, IN) and tuple(delta.shape) == (B, IN)
    assert tuple(G.shape) == (OUT, IN) and (gq is None or tuple(gq.shape) == (OUT, IN))
    check(lib().int_linear_step_small(_p(X, i8, name="X"), _p(W, i8, name="W"), _p(dY, i8, name="dY"), B, IN,
                                      OUT, int(tb_w), int(mu_weight), int(tb_d), _p(Y, i32, name="Y"),
                                      _p(dX, i32, name="dX"), _p(delta, i8, name="delta"), _p(G, i32, name="G"),
                                      _p(gq, i32, OUT * IN, "gq"), _p(maxima, u32, 3, "maxima"),
                                      _p(shifts, i32, 3, "shifts"), _stream(stream)),
          "int_linear_step_small")


def niti_quantize_update_clear(G, absmax, target_bits, mu_weight, W, clear, shifts_out=None, gq_out=None,
                               stream=None):
    assert G.numel() == W.numel()
    check(lib().niti_quantize_update_clear(_p(G, i32, name="G"), G.numel(), _p(absmax, u32, 1, "absmax"),
                                           int(target_bits), int(mu_weight), _p(W, i8, name="W"),
                                           _p(shifts_out, i32, 2, "shifts_out"),
                                           _p(gq_out, i32, G.numel(), "gq_out"),
                                           _p(clear, u32, None, "clear"), clear.numel() if clear is not None else 0,
                                           _stream(stream)),
          "niti_quantize_update_clear")


def ionn_oss_requant(acc, offset, mult, k, out, relu=False, stream=None):
    M, C = acc.shape
    assert tuple(out.shape) == (M, C) and offset.numel() == C and mult.numel() == C and k.numel() == C
    check(lib().ionn_oss_requant(_p(acc, i32, name="acc"), _p(offset, i32, name="offset"),
                                 _p(mult, i32, name="mult"), _p(k, i8, name="k"), M, C, int(bool(relu)),
                                 _p(out, i8, name="out"), _stream(stream)), "ionn_oss_requant")


def int_linear_fwd_oss_workspace_bytes(B, IN, OUT):
    return int(lib().int_linear_fwd_oss_workspace_bytes(int(B), int(IN), int(OUT)))


def int_linear_fwd_oss(X, W, offset, mult, k, Y, relu=False, workspace=None, stream=None):
    B, IN = X.shape
    OUT = W.shape[0]
    assert tuple(W.shape) == (OUT, IN) and tuple(Y.shape) == (B, OUT), "shape mismatch"
    assert offset.numel() == OUT and mult.numel() == OUT and k.numel() == OUT
    check(lib().int_linear_fwd_oss(_p(X, i8, name="X"), _p(W, i8, name="W"), _p(offset, i32, name="offset"),
                                   _p(mult, i32, name="mult"), _p(k, i8, name="k"), int(bool(relu)),
                                   _p(Y, i8, name="Y"), B, IN, OUT, _p(workspace, None, name="workspace"),
                                   workspace.numel() * workspace.element_size() if workspace is not None else 0,
                                   _stream(stream)), "int_linear_fwd_oss")


def ionn_bias_grad_workspace_bytes(M, C):
    return int(lib().ionn_bias_grad_workspace_bytes(int(M), int(C)))


def ionn_bias_grad_noalloc(d, gb, stream=None):
    M, C = d.shape
    assert gb.numel() == C
    check(lib().ionn_bias_grad_noalloc(_p(d, i8, name="d"), M, C, _p(gb, i32, name="gb"), _stream(stream)),
          "ionn_bias_grad_noalloc")


def ionn_bias_grad(d, gb, workspace, stream=None):
    M, C = d.shape
    assert gb.numel() == C
    check(lib().ionn_bias_grad(_p(d, i8, name="d"), M, C, _p(gb, i32, name="gb"),
                               _p(workspace, None, name="workspace"),
                               workspace.numel() * workspace.element_size() if workspace is not None else 0,
                               _stream(stream)), "ionn_bias_grad")


def niti_quantize_update_i32(G, absmax, target_bits, mu, P, shifts_out=None, gq_out=None, stream=None):
    assert G.numel() == P.numel()
    check(lib().niti_quantize_update_i32(_p(G, i32, name="G"), G.numel(), _p(absmax, u32, 1, "absmax"),
                                         int(target_bits), int(mu), _p(P, i32, name="P"),
                                         _p(shifts_out, i32, 2, "shifts_out"),
                                         _p(gq_out, i32, G.numel(), "gq_out"), _stream(stream)),
          "niti_quantize_update_i32")


def ionn_mse_grad_targets(out, labels, tmc, tmw, g, absmax_g=None, stream=None):
    B, C = out.shape
    assert tuple(g.shape) == (B, C) and labels.numel() == B and tmc.numel() == C and tmw.numel() == C
    check(lib().ionn_mse_grad_targets(_p(out, i8, name="out"), _p(labels, i32, name="labels"), B, C,
                                      _p(tmc, i8, name="tmc"), _p(tmw, i8, name="tmw"), _p(g, i32, name="g"),
                                      _p(absmax_g, u32, 1, "absmax_g"), _stream(stream)), "ionn_mse_grad_targets")


def ionn_relu_mask_i32(d, act, absmax_d=None, stream=None):
    assert d.numel() == act.numel()
    check(lib().ionn_relu_mask_i32(_p(d, i32, name="d"), _p(act, i8, name="act"), d.numel(),
                                   _p(absmax_d, u32, 1, "absmax_d"), _stream(stream)), "ionn_relu_mask_i32")


def layer_array(layers):
    """ctypes array of ionn_layer from dicts with type, KH, KW, pad, H, W, Cin,
    Cout and device tensors weight (int8), offset (int32), mult (int32), k (int8)."""
    from ._lib import Layer
    arr = (Layer * len(layers))()
    for i, L in enumerate(layers):
        arr[i] = Layer(int(L["type"]), int(L.get("KH", 1)), int(L.get("KW", 1)), int(L.get("pad", 0)),
                       int(L["H"]), int(L["W"]), int(L["Cin"]), int(L["Cout"]),
                       _p(L["weight"], i8, name="weight"), _p(L["offset"], i32, name="offset"),
                       _p(L["mult"], i32, name="mult"), _p(L["k"], i8, name="k"))
    return arr


def ionn_model_workspace_bytes(larr, B):
    n = int(lib().ionn_model_workspace_bytes(larr, len(larr), int(B)))
    if n == 0:
        check(2, "ionn_model_workspace_bytes")
    return n


def ionn_model_forward(larr, X, workspace, out=None, stream=None):
    check(lib().ionn_model_forward(larr, len(larr), _p(X, i8, name="X"), X.shape[0], _p(out, i8, name="out"),
                                   _p(workspace, None, name="workspace"), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "ionn_model_forward")


def ionn_model_backward(larr, X, labels, tmc, tmw, workspace, tb_delta=7, tb_weight=8, mu=2, shifts_out=None,
                        stream=None):
    check(lib().ionn_model_backward(larr, len(larr), _p(X, i8, name="X"), X.shape[0],
                                    _p(labels, i32, name="labels"), _p(tmc, i8, name="tmc"), _p(tmw, i8, name="tmw"),
                                    int(tb_delta), int(tb_weight), int(mu), _p(workspace, None, name="workspace"),
                                    workspace.numel() * workspace.element_size(),
                                    _p(shifts_out, i32, 1 + 5 * len(larr), "shifts_out"), _stream(stream)),
          "ionn_model_backward")


def int_output_error(out, labels, target_mag, e, absmax_e=None, stream=None):
    B, C = out.shape
    assert tuple(e.shape) == (B, C) and labels.numel() == B
    check(lib().int_output_error(_p(out, i8, name="out"), _p(labels, i32, name="labels"), B, C,
                                 int(target_mag), _p(e, i32, name="e"),
                                 _p(absmax_e, u32, 1, "absmax_e"), _stream(stream)),
          "int_output_error")


def conv_desc(N, H, W, Cin, Cout, KH=3, KW=3, stride=1, pad=1, dilation=1, groups=1):
    return ConvDesc(N, H, W, Cin, Cout, KH, KW, stride, pad, dilation, groups)


def _conv_numels(desc):
    """Elements of X [N][H][W][Cin], W [Cout][KH][KW][Cin] and the output
    [N][Ho][Wo][Cout] (Ho = H + 2 pad - KH + 1, stride 1) that a call with
    this descriptor touches."""
    ho = max(desc.H + 2 * desc.pad - desc.KH + 1, 0)
    wo = max(desc.W + 2 * desc.pad - desc.KW + 1, 0)
    return (desc.N * desc.H * desc.W * desc.Cin, desc.Cout * desc.KH * desc.KW * desc.Cin,
            desc.N * ho * wo * desc.Cout)


def int_conv_fwd(X, Wt, Y, desc, absmax_Y=None, stream=None):
    nx, nw, ny = _conv_numels(desc)
    check(lib().int_conv_fwd(_p(X, i8, nx, "X"), _p(Wt, i8, nw, "W"), _p(Y, i32, ny, "Y"),
                             ctypes.byref(desc), _p(absmax_Y, u32, 1, "absmax_Y"), _stream(stream)),
          "int_conv_fwd")


def int_conv_dgrad(dY, Wt, dX, desc, absmax_dX=None, stream=None):
    nx, nw, ny = _conv_numels(desc)
    check(lib().int_conv_dgrad(_p(dY, i8, ny, "dY"), _p(Wt, i8, nw, "W"), _p(dX, i32, nx, "dX"),
                               ctypes.byref(desc), _p(absmax_dX, u32, 1, "absmax_dX"),
                               _stream(stream)), "int_conv_dgrad")




def int_conv_requant_workspace_bytes(desc):
    return int(lib().int_conv_requant_workspace_bytes(ctypes.byref(desc)))


def _ws(workspace):
    return (_p(workspace, None, name="workspace"),
            workspace.numel() * workspace.element_size() if workspace is not None else 0)


def int_conv_fwd_requant(X, Wt, Y8, desc, target_bits, relu, absmax_Y, shift_out=None, workspace=None,
                         stream=None):
    nx, nw, ny = _conv_numels(desc)
    check(lib().int_conv_fwd_requant(_p(X, i8, nx, "X"), _p(Wt, i8, nw, "W"), _p(Y8, i8, ny, "Y8"),
                                     ctypes.byref(desc), int(target_bits), int(bool(relu)),
                                     _p(absmax_Y, u32, 1, "absmax_Y"), _p(shift_out, i32, 1, "shift_out"),
                                     *_ws(workspace), _stream(stream)), "int_conv_fwd_requant")


def int_conv_dgrad_requant(dY, Wt, dX8, desc, target_bits, absmax_dX, shift_out=None, workspace=None,
                           stream=None):
    nx, nw, ny = _conv_numels(desc)
    check(lib().int_conv_dgrad_requant(_p(dY, i8, ny, "dY"), _p(Wt, i8, nw, "W"), _p(dX8, i8, nx, "dX8"),
                                       ctypes.byref(desc), int(target_bits), _p(absmax_dX, u32, 1, "absmax_dX"),
                                       _p(shift_out, i32, 1, "shift_out"), *_ws(workspace), _stream(stream)),
          "int_conv_dgrad_requant")


def int_conv_wgrad_workspace_bytes(desc):
    return int(lib().int_conv_wgrad_workspace_bytes(ctypes.byref(desc)))


def int_conv_wgrad(dY, X, G, desc, absmax_G=None, workspace=None, stream=None):
    nx, nw, ny = _conv_numels(desc)
    check(lib().int_conv_wgrad(_p(dY, i8, ny, "dY"), _p(X, i8, nx, "X"), _p(G, i32, nw, "G"),
                               ctypes.byref(desc), _p(absmax_G, u32, 1, "absmax_G"),
                               _p(workspace, None, name="workspace"),
                               workspace.numel() * workspace.element_size() if workspace is not None else 0,
                               _stream(stream)), "int_conv_wgrad")


def dfp16_workspace_bytes(M, K, N, which):
    return int(lib().dfp16_workspace_bytes(M, K, N, which))


def _dfp(fn, name, A, eA, B, eB, out, eout, M, K, N, chunk, workspace, status_out, stream):
    check(fn(_p(A, i16, name="A"), _p(eA, i32, 1, "eA"), _p(B, i16, name="B"),
             _p(eB, i32, 1, "eB"), _p(out, i16, name="out"), _p(eout, i32, 1, "e_out"), M, K, N,
             int(chunk), _p(workspace, None, name="workspace"),
             workspace.numel() * workspace.element_size() if workspace is not None else 0,
             _p(status_out, i32, 1, "status_out"), _stream(stream)), name)


def dfp16_gemm_fwd(X, eX, W, eW, Y, eY, workspace, chunk=64, status_out=None, stream=None):
    M, K = X.shape
    N = W.shape[0]
    assert tuple(W.shape) == (N, K) and tuple(Y.shape) == (M, N)
    _dfp(lib().dfp16_gemm_fwd, "dfp16_gemm_fwd", X, eX, W, eW, Y, eY, M, K, N, chunk, workspace,
         status_out, stream)


def dfp16_gemm_dgrad(dY, edY, W, eW, dX, edX, workspace, chunk=64, status_out=None, stream=None):
    M, N = dY.shape
    K = W.shape[1]
    assert tuple(W.shape) == (N, K) and tuple(dX.shape) == (M, K)
    _dfp(lib().dfp16_gemm_dgrad, "dfp16_gemm_dgrad", dY, edY, W, eW, dX, edX, M, K, N, chunk,
         workspace, status_out, stream)


def dfp16_gemm_wgrad(dY, edY, X, eX, G, eG, workspace, chunk=64, status_out=None, stream=None):
    M, N = dY.shape
    K = X.shape[1]
    assert tuple(X.shape) == (M, K) and tuple(G.shape) == (N, K)
    _dfp(lib().dfp16_gemm_wgrad, "dfp16_gemm_wgrad", dY, edY, X, eX, G, eG, M, K, N, chunk,
         workspace, status_out, stream)


# ---- DFP as the DFP page runs it: FP32 partials, conversions, SGD -----------

f32 = torch.float32


def dfp16_f32_splits(M, K, N, which):
    return int(lib().dfp16_f32_splits(M, K, N, which))


def dfp16_f32_workspace_bytes(M, K, N, which, nsplit=0):
    return int(lib().dfp16_f32_workspace_bytes(M, K, N, which, nsplit))


def _dfp_f32(fn, name, A, eA, B, eB, out, M, K, N, input_shift, nsplit, workspace, stream):
    check(fn(_p(A, i16, name="A"), _p(eA, i32, 1, "eA"), _p(B, i16, name="B"), _p(eB, i32, 1, "eB"),
             _p(out, f32, name="out"), M, K, N, int(input_shift), int(nsplit), _p(workspace, None, name="workspace"),
             workspace.numel() * workspace.element_size() if workspace is not None else 0, _stream(stream)), name)


def dfp16_gemm_fwd_f32(X, eX, W, eW, Y, workspace, input_shift=1, nsplit=0, stream=None):
    M, K = X.shape
    N = W.shape[0]
    assert tuple(W.shape) == (N, K) and tuple(Y.shape) == (M, N)
    _dfp_f32(lib().dfp16_gemm_fwd_f32, "dfp16_gemm_fwd_f32", X, eX, W, eW, Y, M, K, N, input_shift, nsplit,
             workspace, stream)


def dfp16_gemm_dgrad_f32(dY, edY, W, eW, dX, workspace, input_shift=1, nsplit=0, stream=None):
    M, N = dY.shape
    K = W.shape[1]
    assert tuple(W.shape) == (N, K) and tuple(dX.shape) == (M, K)
    _dfp_f32(lib().dfp16_gemm_dgrad_f32, "dfp16_gemm_dgrad_f32", dY, edY, W, eW, dX, M, K, N, input_shift, nsplit,
             workspace, stream)


def dfp16_gemm_wgrad_f32(dY, edY, X, eX, G, workspace, input_shift=1, nsplit=0, stream=None):
    M, N = dY.shape
    K = X.shape[1]
    assert tuple(X.shape) == (M, K) and tuple(G.shape) == (N, K)
    _dfp_f32(lib().dfp16_gemm_wgrad_f32, "dfp16_gemm_wgrad_f32", dY, edY, X, eX, G, M, K, N, input_shift, nsplit,
             workspace, stream)


def dfp16_gemm_fwd_f32_blocked(X, eX, W, eW, Y, workspace, input_shift=1, nsplit=0, stream=None):
    """eX: int32 [M][ceil(K/64)], eW: int32 [N][ceil(K/64)] (device)."""
    M, K = X.shape
    N = W.shape[0]
    nch = (K + 63) // 64
    assert tuple(W.shape) == (N, K) and tuple(Y.shape) == (M, N)
    check(lib().dfp16_gemm_fwd_f32_blocked(
        _p(X, i16, name="X"), _p(eX, i32, M * nch, "eX"), _p(W, i16, name="W"), _p(eW, i32, N * nch, "eW"),
        _p(Y, f32, name="Y"), M, K, N, int(input_shift), int(nsplit), _p(workspace, None, name="workspace"),
        workspace.numel() * workspace.element_size() if workspace is not None else 0, _stream(stream)),
        "dfp16_gemm_fwd_f32_blocked")


def dfp_convert_workspace_bytes():
    return int(lib().dfp_convert_workspace_bytes())


def dfp_from_f32(x, out, e_out, workspace, P=16, status_out=None, stream=None):
    assert x.numel() == out.numel()
    check(lib().dfp_from_f32(_p(x, f32, name="x"), x.numel(), int(P), _p(out, i16, name="out"),
                             _p(e_out, i32, 1, "e_out"), _p(status_out, i32, 1, "status_out"),
                             _p(workspace, None, name="workspace"),
                             workspace.numel() * workspace.element_size(), _stream(stream)), "dfp_from_f32")


def dfp_to_f32(I, e, out, stream=None):
    assert I.numel() == out.numel()
    check(lib().dfp_to_f32(_p(I, i16, name="I"), I.numel(), _p(e, i32, 1, "e"), _p(out, f32, name="out"),
                           _stream(stream)), "dfp_to_f32")


def dfp_from_f32_blocked(x, out, e_out, B=64, P=16, status_out=None, stream=None):
    rows, K = x.shape
    nb = (K + B - 1) // B
    assert tuple(out.shape) == (rows, K) and e_out.numel() >= rows * nb
    check(lib().dfp_from_f32_blocked(_p(x, f32, name="x"), rows, K, int(B), int(P), _p(out, i16, name="out"),
                                     _p(e_out, i32, rows * nb, "e_out"), _p(status_out, i32, 1, "status_out"),
                                     _stream(stream)), "dfp_from_f32_blocked")


def dfp16_sgd_update(W32, G32, lr, W16, eW, workspace, status_out=None, stream=None):
    n = W32.numel()
    assert G32.numel() == n and W16.numel() == n
    check(lib().dfp16_sgd_update(_p(W32, f32, name="W32"), _p(G32, f32, name="G32"), n, float(lr),
                                 _p(W16, i16, name="W16"), _p(eW, i32, 1, "eW"), _p(status_out, i32, 1, "status_out"),
                                 _p(workspace, None, name="workspace"), workspace.numel() * workspace.element_size(),
                                 _stream(stream)), "dfp16_sgd_update")


def dfp16_gavg(G, eG, eW, gavg_out, stream=None):
    check(lib().dfp16_gavg(_p(G, i16, name="G"), _p(eG, i32, 1, "eG"), _p(eW, i32, 1, "eW"),
                           G.numel(), _p(gavg_out, torch.float64, 1, "gavg_out"), _stream(stream)),
          "dfp16_gavg")


# ---- adaptive per-layer precision -------------------------------------------

def _ptr_array(ts, dtype, name):
    return (ctypes.c_void_p * len(ts))(*[_p(t, dtype, name=f"{name}[{l}]").value for l, t in enumerate(ts)])


def _sizes(ts):
    return (ctypes.c_int64 * len(ts))(*[t.numel() for t in ts])


def apt_workspace_bytes(sizes):
    return lib().apt_workspace_bytes(len(sizes), (ctypes.c_int64 * len(sizes))(*[int(n) for n in sizes]))


def apt_update(Ws, Gs, k, e_w, e_g, lr_shift, gavg_sum=None, gavg_count=None, workspace=None, stream=None):
    """One step's k-bit update of every layer (lists of int16 device tensors);
    k, e_w, e_g: int32 [L]; gavg_sum (float64 [L]) and gavg_count (int32 [L])
    given together make it a sampling step."""
    L = len(Ws)
    if len(Gs) != L or any(w.numel() != g.numel() for w, g in zip(Ws, Gs)):
        raise ValueError("Ws and Gs must pair up with equal sizes")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib().apt_update(L, _ptr_array(Ws, i16, "W"), _ptr_array(Gs, i16, "G"), _sizes(Ws),
                           _p(k, i32, L, "k"), _p(e_w, i32, L, "e_w"), _p(e_g, i32, L, "e_g"), int(lr_shift),
                           _p(gavg_sum, torch.float64, L, "gavg_sum"), _p(gavg_count, i32, L, "gavg_count"),
                           _p(workspace, name="workspace"), ws_bytes, _stream(stream)), "apt_update")


def _wbytes(Ws):
    """Host int32 array of bytes per weight (1 for int8 tensors, 2 for int16)."""
    out = []
    for l, w in enumerate(Ws):
        if w.dtype not in (torch.int8, torch.int16):
            raise TypeError(f"W[{l}] must be int8 or int16, not {w.dtype}")
        out.append(1 if w.dtype == torch.int8 else 2)
    return (ctypes.c_int32 * len(Ws))(*out)


def apt_update_mixed(Ws, Gs, k, e_w, e_g, lr_shift, gavg_sum=None, gavg_count=None, workspace=None, stream=None):
    """apt_update over layers held in int8 (k in [2, 8]) or int16."""
    L = len(Ws)
    if len(Gs) != L or any(w.numel() != g.numel() for w, g in zip(Ws, Gs)):
        raise ValueError("Ws and Gs must pair up with equal sizes")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib().apt_update_mixed(L, _ptr_array(Ws, None, "W"), _wbytes(Ws), _ptr_array(Gs, i16, "G"), _sizes(Ws),
                                 _p(k, i32, L, "k"), _p(e_w, i32, L, "e_w"), _p(e_g, i32, L, "e_g"), int(lr_shift),
                                 _p(gavg_sum, torch.float64, L, "gavg_sum"), _p(gavg_count, i32, L, "gavg_count"),
                                 _p(workspace, name="workspace"), ws_bytes, _stream(stream)), "apt_update_mixed")


def apt_adjust_mixed(Ws, k, e_w, gavg_sum, gavg_count, t_min, t_max, k_min=2, k_max=16, dk_out=None, stream=None):
    """apt_adjust over layers held in int8 (never raised past 8 bits) or int16."""
    L = len(Ws)
    check(lib().apt_adjust_mixed(L, _ptr_array(Ws, None, "W"), _wbytes(Ws), _sizes(Ws), _p(k, i32, L, "k"),
                                 _p(e_w, i32, L, "e_w"), _p(gavg_sum, torch.float64, L, "gavg_sum"),
                                 _p(gavg_count, i32, L, "gavg_count"), float(t_min), float(t_max), int(k_min),
                                 int(k_max), _p(dk_out, i32, L, "dk_out"), _stream(stream)), "apt_adjust_mixed")


def apt_adjust(Ws, k, e_w, gavg_sum, gavg_count, t_min, t_max, k_min=2, k_max=16, dk_out=None, stream=None):
    """Between epochs: one bit more or less per layer on its mean Gavg."""
    L = len(Ws)
    check(lib().apt_adjust(L, _ptr_array(Ws, i16, "W"), _sizes(Ws), _p(k, i32, L, "k"), _p(e_w, i32, L, "e_w"),
                           _p(gavg_sum, torch.float64, L, "gavg_sum"), _p(gavg_count, i32, L, "gavg_count"),
                           float(t_min), float(t_max), int(k_min), int(k_max), _p(dk_out, i32, L, "dk_out"),
                           _stream(stream)), "apt_adjust")


# ---- floating-point operations around the DFP-8 products ---------------------

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
ADAMW_BLOCK = 256  # elements of an 8-bit optimiser state that share an exponent
_FLOATS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _dtype(t, name):
    """The library's number of a floating tensor's type."""
    d = _FLOATS.get(getattr(t, "dtype", None))
    if d is None:
        raise TypeError(f"{name}: expected a float32, bfloat16 or float16 tensor")
    return d


# The calls below serve single tokens too, where the host's share of a call
# counts (a launch takes 2.8 us of it): a tensor that is in order costs _m or
# _v a few attribute reads, _refuse has the messages, and the current stream
# is read without building a Stream object.

def _refuse(t, dtype, shape, name):
    """Raises what is wrong with an argument."""
    if isinstance(t, torch.Tensor):
        have = t.numel() if isinstance(shape, int) else tuple(t.shape)
        need = shape if isinstance(shape, int) else tuple(shape)
        if have != need:
            raise ValueError(f"shape mismatch: {name} has {have}, needs {need}")
    _p(t, dtype, name=name)
    raise ValueError(f"{name}: not accepted")


def _m(t, dtype, shape, name):
    """Address of a contiguous device tensor of this type and shape (None -> NULL)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, shape, name)


def _v(t, dtype, n, name):
    """The same for a tensor of n elements in any shape."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.is_cuda and t.numel() == n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, n, name)


def _s(t, dtype, name):
    """The same for a scalar held in a tensor of at least one element."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.is_cuda and t.numel() >= 1:
            return t.data_ptr()
    except AttributeError:
        pass
    return _p(t, dtype, 1, name).value


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(stream, t):
    """The stream's handle: by default the current one of t's device."""
    if stream is None and _raw_stream is not None and t.is_cuda:
        return _raw_stream(t.get_device())
    return _stream(stream)


def _act(act):
    """The library's number of an activation, given by number or name."""
    return ACTIVATIONS[act] if isinstance(act, str) else int(act)


def _same(cond, what):
    if not cond:
        raise ValueError(f"shape mismatch: {what}")


def _reduced(X, W):
    """Columns of a layer's input and weights; 0 where neither is given (no gradient of either is asked for)."""
    for t in (X, W):
        if t is not None:
            return t.shape[1]
    return 0


def _space(workspace):
    """Address and bytes of a workspace (None: NULL and 0)."""
    if workspace is None:
        return None, 0
    if workspace.is_cuda and workspace.is_contiguous():
        return workspace.data_ptr(), workspace.nbytes
    return _p(workspace, name="workspace").value, workspace.nbytes


def dfp8_from_float_workspace_bytes():
    return int(lib().dfp8_from_float_workspace_bytes())


def dfp8_from_float(x, out, e_out, absmax=None, workspace=None, status_out=None, stream=None):
    ws, nws = _space(workspace)
    rc = lib().dfp8_from_float(_v(x, x.dtype, x.numel(), "x"), _dtype(x, "x"), x.numel(), _s(absmax, u32, "absmax"),
                               _v(out, i8, x.numel(), "out"), _s(e_out, i32, "e_out"),
                               _s(status_out, i32, "status_out"), ws, nws, _on(stream, x))
    if rc:
        check(rc, "dfp8_from_float")


def dfp8_linear_fwd_workspace_bytes(B, IN, OUT):
    return int(lib().dfp8_linear_fwd_workspace_bytes(int(B), int(IN), int(OUT)))


def dfp8_linear_fwd(X, eX, W, eW, Y, bias=None, act=0, residual=None, Z=None, absmax_Y=None, workspace=None,
                    stream=None):
    xs, dt = X.shape, Y.dtype
    B, IN = xs
    OUT = W.shape[0]
    ys = (B, OUT)
    ws, nws = _space(workspace)
    rc = lib().dfp8_linear_fwd(_m(X, i8, xs, "X"), _s(eX, i32, "eX"), _m(W, i8, (OUT, IN), "W"), _s(eW, i32, "eW"),
                               _v(bias, f32, OUT, "bias"), _act(act), _m(residual, dt, ys, "residual"),
                               _m(Z, dt, ys, "Z"), _m(Y, dt, ys, "Y"), _dtype(Y, "Y"), B, IN, OUT,
                               _s(absmax_Y, u32, "absmax_Y"), ws, nws, _on(stream, Y))
    if rc:
        check(rc, "dfp8_linear_fwd")


def dfp8_linear_bwd_workspace_bytes(B, IN, OUT):
    return int(lib().dfp8_linear_bwd_workspace_bytes(int(B), int(IN), int(OUT)))


def dfp8_linear_bwd(dY, Z, act, X, eX, W, eW, dZ8, edZ, dX=None, G=None, gb=None, workspace=None, status_out=None,
                    stream=None):
    """Z may be None for no activation; X and eX are read for G, W and eW for dX (and may be None without)."""
    ys, dt = dY.shape, dY.dtype
    B, OUT = ys
    IN = _reduced(X, W)
    xs, gs = (B, IN), (OUT, IN)
    ws, nws = _space(workspace)
    rc = lib().dfp8_linear_bwd(_m(dY, dt, ys, "dY"), _m(Z, dt, ys, "Z"), _act(act), _dtype(dY, "dY"),
                               _m(X, i8, xs, "X"), _s(eX, i32, "eX"), _m(W, i8, gs, "W"), _s(eW, i32, "eW"),
                               _m(dZ8, i8, ys, "dZ8"), _s(edZ, i32, "edZ"), _m(dX, dt, xs, "dX"), _m(G, dt, gs, "G"),
                               _v(gb, f32, OUT, "gb"), B, IN, OUT, _s(status_out, i32, "status_out"), ws, nws,
                               _on(stream, dY))
    if rc:
        check(rc, "dfp8_linear_bwd")


def dfp8_gated_fwd_workspace_bytes(B, IN, H):
    return int(lib().dfp8_gated_fwd_workspace_bytes(int(B), int(IN), int(H)))


def dfp8_gated_fwd(X, eX, W, eW, Y, bias=None, act="silu", Z=None, absmax_Y=None, workspace=None, stream=None):
    """W: [2 H][IN], the gate's rows and then the up projection's; Z: [B][2 H]."""
    xs, dt = X.shape, Y.dtype
    B, IN = xs
    H = W.shape[0] // 2
    ws, nws = _space(workspace)
    rc = lib().dfp8_gated_fwd(_m(X, i8, xs, "X"), _s(eX, i32, "eX"), _m(W, i8, (2 * H, IN), "W"), _s(eW, i32, "eW"),
                              _v(bias, f32, 2 * H, "bias"), _act(act), _m(Z, dt, (B, 2 * H), "Z"),
                              _m(Y, dt, (B, H), "Y"), _dtype(Y, "Y"), B, IN, H, _s(absmax_Y, u32, "absmax_Y"), ws, nws,
                              _on(stream, Y))
    if rc:
        check(rc, "dfp8_gated_fwd")


def dfp8_gated_bwd_workspace_bytes(B, IN, H):
    return int(lib().dfp8_gated_bwd_workspace_bytes(int(B), int(IN), int(H)))


def dfp8_gated_bwd(dY, Z, act, X, eX, W, eW, dZ8, edZ, dX=None, G=None, gb=None, workspace=None, status_out=None,
                   stream=None):
    """X and eX are read for G, W and eW for dX (and may be None without)."""
    ys, dt = dY.shape, dY.dtype
    B, H = ys
    IN = _reduced(X, W)
    xs, zs, gs = (B, IN), (B, 2 * H), (2 * H, IN)
    ws, nws = _space(workspace)
    rc = lib().dfp8_gated_bwd(_m(dY, dt, ys, "dY"), _m(Z, dt, zs, "Z"), _act(act), _dtype(dY, "dY"),
                              _m(X, i8, xs, "X"), _s(eX, i32, "eX"), _m(W, i8, gs, "W"), _s(eW, i32, "eW"),
                              _m(dZ8, i8, zs, "dZ8"), _s(edZ, i32, "edZ"), _m(dX, dt, xs, "dX"), _m(G, dt, gs, "G"),
                              _v(gb, f32, 2 * H, "gb"), B, IN, H, _s(status_out, i32, "status_out"), ws, nws,
                              _on(stream, dY))
    if rc:
        check(rc, "dfp8_gated_bwd")


def dfp8_linear_path(product, B, IN, OUT):
    """"rows", "tiles 256", "tiles 128", "tiles" or "narrow", for product "fwd", "dX" or "G"."""
    p = lib().dfp8_linear_path(("fwd", "dX", "G").index(product), int(B), int(IN), int(OUT))
    if p < 0:
        raise ValueError(f"B = {B}, IN = {IN}, OUT = {OUT}")
    return ("rows", "tiles 256", "tiles 128", "tiles", "narrow")[p]


def ionn_layer_norm_fwd(x, y, gamma=None, beta=None, eps=1e-5, mean=None, rstd=None, absmax_y=None, stream=None):
    xs, dt = x.shape, x.dtype
    rows, cols = xs
    rc = lib().ionn_layer_norm_fwd(_m(x, dt, xs, "x"), _v(gamma, f32, cols, "gamma"), _v(beta, f32, cols, "beta"), eps,
                                   _m(y, dt, xs, "y"), _v(mean, f32, rows, "mean"), _v(rstd, f32, rows, "rstd"),
                                   _dtype(x, "x"), rows, cols, _s(absmax_y, u32, "absmax_y"), _on(stream, x))
    if rc:
        check(rc, "ionn_layer_norm_fwd")


def ionn_layer_norm_bwd_workspace_bytes(rows, cols):
    return int(lib().ionn_layer_norm_bwd_workspace_bytes(int(rows), int(cols)))


def ionn_layer_norm_bwd(dy, x, mean, rstd, dx, gamma=None, dres=None, dgamma=None, dbeta=None, workspace=None,
                        stream=None):
    xs, dt = x.shape, x.dtype
    rows, cols = xs
    ws, nws = _space(workspace)
    rc = lib().ionn_layer_norm_bwd(_m(dy, dt, xs, "dy"), _m(x, dt, xs, "x"), _v(mean, f32, rows, "mean"),
                                   _v(rstd, f32, rows, "rstd"), _v(gamma, f32, cols, "gamma"),
                                   _m(dres, dt, xs, "dres"), _m(dx, dt, xs, "dx"), _v(dgamma, f32, cols, "dgamma"),
                                   _v(dbeta, f32, cols, "dbeta"), _dtype(x, "x"), rows, cols, ws, nws, _on(stream, x))
    if rc:
        check(rc, "ionn_layer_norm_bwd")


NORMS = {"none": 0, "layer": 1, "rms": 2}


def _norm(kind):
    """The library's number of a norm, given by number or name."""
    return NORMS[kind] if isinstance(kind, str) else int(kind)


def _gate_groups(gate, gate_rows, rows):
    """Rows of the gate tensor."""
    if gate is None:
        return 0
    return -(-rows // gate_rows) if 0 < gate_rows < rows else 1


def ionn_residual_norm_fwd(a, x, y, n, norm_a="rms", gamma_a=None, beta_a=None, gate=None, gate_rows=0, alpha=1.0,
                           norm_y="rms", gamma_y=None, beta_y=None, eps=1e-5, mean_a=None, rstd_a=None, mean_y=None,
                           rstd_y=None, absmax_n=None, stream=None):
    """a None (with norm_a "none"): the norm of alpha x alone; y or n None: not written."""
    xs, dt = x.shape, x.dtype
    rows, cols = xs
    rc = lib().ionn_residual_norm_fwd(
        _m(a, dt, xs, "a"), _m(x, dt, xs, "x"), _norm(norm_a), _v(gamma_a, f32, cols, "gamma_a"),
        _v(beta_a, f32, cols, "beta_a"), _v(gate, f32, _gate_groups(gate, gate_rows, rows) * cols, "gate"), gate_rows,
        alpha, _norm(norm_y), _v(gamma_y, f32, cols, "gamma_y"), _v(beta_y, f32, cols, "beta_y"), eps,
        _m(y, dt, xs, "y"), _m(n, dt, xs, "n"), _v(mean_a, f32, rows, "mean_a"), _v(rstd_a, f32, rows, "rstd_a"),
        _v(mean_y, f32, rows, "mean_y"), _v(rstd_y, f32, rows, "rstd_y"), _dtype(x, "x"), rows, cols,
        _s(absmax_n, u32, "absmax_n"), _on(stream, x))
    if rc:
        check(rc, "ionn_residual_norm_fwd")


def ionn_residual_norm_bwd_workspace_bytes(rows, cols, gate_rows=0):
    return int(lib().ionn_residual_norm_bwd_workspace_bytes(int(rows), int(cols), int(gate_rows)))


def ionn_residual_norm_bwd(dy, dn, a, y, da, dx, norm_a="rms", gamma_a=None, beta_a=None, gate=None, gate_rows=0,
                           alpha=1.0, norm_y="rms", gamma_y=None, mean_a=None, rstd_a=None, mean_y=None, rstd_y=None,
                           dgamma_a=None, dbeta_a=None, dgate=None, dgamma_y=None, dbeta_y=None, workspace=None,
                           stream=None):
    """dy or dn None: no such error; every output may be None."""
    err = dy if dy is not None else dn
    xs, dt = err.shape, err.dtype
    rows, cols = xs
    gates = _gate_groups(gate, gate_rows, rows) * cols
    ws, nws = _space(workspace)
    rc = lib().ionn_residual_norm_bwd(
        _m(dy, dt, xs, "dy"), _m(dn, dt, xs, "dn"), _m(a, dt, xs, "a"), _m(y, dt, xs, "y"), _norm(norm_a),
        _v(gamma_a, f32, cols, "gamma_a"), _v(beta_a, f32, cols, "beta_a"), _v(gate, f32, gates, "gate"), gate_rows,
        alpha, _norm(norm_y), _v(gamma_y, f32, cols, "gamma_y"), _v(mean_a, f32, rows, "mean_a"),
        _v(rstd_a, f32, rows, "rstd_a"), _v(mean_y, f32, rows, "mean_y"), _v(rstd_y, f32, rows, "rstd_y"),
        _m(da, dt, xs, "da"), _m(dx, dt, xs, "dx"), _v(dgamma_a, f32, cols, "dgamma_a"),
        _v(dbeta_a, f32, cols, "dbeta_a"), _v(dgate, f32, gates, "dgate"), _v(dgamma_y, f32, cols, "dgamma_y"),
        _v(dbeta_y, f32, cols, "dbeta_y"), _dtype(err, "dy"), rows, cols, ws, nws, _on(stream, err))
    if rc:
        check(rc, "ionn_residual_norm_bwd")


def _state_ptrs(ts, bits, name):
    """Pointers of optimiser states: float32, or one byte per element (uint8,
    int8 or float8_e4m3fn tensors of codes)."""
    if bits == 8 and any(t.element_size() != 1 for t in ts):
        raise TypeError(f"{name}: 8-bit states are held in tensors of one byte per element")
    return _ptr_array(ts, f32 if bits == 32 else None, name)


def ionn_adamw_step(Ps, Gs, Ms, Vs, t, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, Ss=None, step=None,
                    lr_dev=None, grad_scale=None, absmax_P=None, stream=None, Rs=None):
    """One step of every tensor (lists of device tensors); 8-bit states where
    Ss (int8 [blocks][2] per tensor) is given, with the roots' remainders
    (ionn_adamw_step_carried) where Rs (int8 per element) is."""
    L = len(Ps)
    bits = 32 if Ss is None else 8
    _same(len(Gs) == L and len(Ms) == L and len(Vs) == L and (Ss is None or len(Ss) == L), "lists of tensors")
    _same(all(p.numel() == x.numel() for xs in (Gs, Ms, Vs) for p, x in zip(Ps, xs)), "P, G, M and V of a tensor")
    _same(Ss is None or all(s.numel() == 2 * -(-p.numel() // ADAMW_BLOCK) for p, s in zip(Ps, Ss)), "S of a tensor")
    _same(Rs is None or (Ss is not None and len(Rs) == L and all(r.numel() == p.numel() for p, r in zip(Ps, Rs))),
          "R of a tensor")
    if L == 0:
        return
    head = (L, _ptr_array(Ps, f32, "P"), _ptr_array(Gs, Gs[0].dtype, "G"), _dtype(Gs[0], "G"),
            _state_ptrs(Ms, bits, "M"), _state_ptrs(Vs, bits, "V"), None if Ss is None else _ptr_array(Ss, i8, "S"))
    tail = (_sizes(Ps), int(t), lr, beta1, beta2, eps, weight_decay, _s(step, i32, "step"), _s(lr_dev, f32, "lr_dev"),
            _s(grad_scale, f32, "grad_scale"), _v(absmax_P, u32, L, "absmax_P"), _on(stream, Ps[0]))
    if Rs is None:
        rc = lib().ionn_adamw_step(*head, bits, *tail)
    else:
        rc = lib().ionn_adamw_step_carried(*head, _ptr_array(Rs, i8, "R"), *tail)
    if rc:
        check(rc, "ionn_adamw_step" if Rs is None else "ionn_adamw_step_carried")


def _shapes(ts):
    """Rows and columns of matrices, as host arrays."""
    return tuple((ctypes.c_int64 * len(ts))(*[int(t.shape[d]) for t in ts]) for d in (0, 1))


def ionn_muon_workspace_bytes(shapes):
    """shapes: (rows, columns) of each matrix."""
    rows, cols = ((ctypes.c_int64 * len(shapes))(*[int(s[d]) for s in shapes]) for d in (0, 1))
    return int(lib().ionn_muon_workspace_bytes(len(shapes), rows, cols))


def ionn_muon_tile(shapes, l=0):
    """Side of the tiles that matrix l of these shapes is worked in."""
    rows, cols = ((ctypes.c_int64 * len(shapes))(*[int(s[d]) for s in shapes]) for d in (0, 1))
    side = lib().ionn_muon_tile(len(shapes), rows, cols, int(l))
    if side < 0:
        raise ValueError(f"shapes = {shapes}, l = {l}")
    return side


def ionn_muon_step(Ps, Gs, Ms, lr, workspace, momentum=0.95, nesterov=True, eps=1e-7, weight_decay=0.0, ns_steps=5,
                   scale=None, lr_dev=None, grad_scale=None, absmax_P=None, stream=None):
    """One step of every matrix (lists of 2-d device tensors); scale: a number
    for each (None: sqrt(max(1, rows / columns)))."""
    L = len(Ps)
    _same(len(Gs) == L and len(Ms) == L and (scale is None or len(scale) == L), "lists of matrices")
    _same(all(p.dim() == 2 and p.shape == g.shape == m.shape for p, g, m in zip(Ps, Gs, Ms)), "P, G and M of a matrix")
    if L == 0:
        return
    rows, cols = _shapes(Ps)
    ws, nws = _space(workspace)
    rc = lib().ionn_muon_step(
        L, _ptr_array(Ps, f32, "P"), _ptr_array(Gs, Gs[0].dtype, "G"), _dtype(Gs[0], "G"), _ptr_array(Ms, f32, "M"), rows,
        cols, lr, momentum, int(nesterov), eps, weight_decay, int(ns_steps),
        None if scale is None else (ctypes.c_double * L)(*[float(v) for v in scale]), _s(lr_dev, f32, "lr_dev"),
        _s(grad_scale, f32, "grad_scale"), _v(absmax_P, u32, L, "absmax_P"), ws, nws, _on(stream, Ps[0]))
    if rc:
        check(rc, "ionn_muon_step")
