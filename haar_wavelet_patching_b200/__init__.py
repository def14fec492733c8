"""B200 Haar patcher / unpatcher, FSQ quantizer and operators of a model over the tokens (embedding of codes, rotary
positions, cross attention, a paged cache with its attention, drawing codes, verifying drafts): Python binding of libtok.so.

The functions named like the C ABI (``tok_haar_fwd`` ...) marshal torch CUDA
tensors into the C calls of ``include/tok.h`` and nothing else: every step of
the computation runs in the library's sm_100a kernels.  There is no CPU path;
a missing library or a CPU tensor raises.

Convenience wrappers (``haar_fwd``, ``haar_inv``, ``fsq_encode``,
``fsq_decode``, ``cross_attention``, ``sample_codes`` ...) allocate outputs with torch and call the same entry points.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtok.so")

(TOK_OK, TOK_ERR_NULL, TOK_ERR_SHAPE, TOK_ERR_ALIGN, TOK_ERR_DTYPE, TOK_ERR_ALIAS, TOK_ERR_CUDA,
 TOK_ERR_TIMEOUT, TOK_ERR_TOO_LARGE) = range(9)
TOK_F32, TOK_BF16 = 0, 1
FSQ_CODEBOOK = 64000
FSQ_DIM = 6

# Every symbol include/tok.h declares.
ABI_SYMBOLS = ("tok_abi_version", "tok_status_str", "tok_last_cuda_error", "tok_check_device",
               "tok_selftest_wait_timeout", "tok_haar_fwd",
               "tok_haar_inv", "tok_haar_fwd_adjoint", "tok_haar_inv_adjoint", "tok_haar_fwd_windows",
               "tok_haar_inv_windows", "tok_haar_fwd_single", "tok_haar_inv_single", "tok_haar_fwd_channels_last", "tok_haar_padded_extents", "tok_haar_fwd_padded", "tok_haar_inv_cropped",
               "tok_haar_fwd_chunk", "tok_haar_inv_chunk", "tok_conv_spatial", "tok_conv_temporal_causal",
               "tok_conv_factorized", "tok_patch_embed_pack_weights", "tok_patch_embed_spatial", "tok_fsq_encode", "tok_fsq_decode", "tok_fsq_backward_workspace_size",
               "tok_fsq_encode_backward", "tok_fsq_encode_backward_noalloc", "tok_fsq_decode_backward",
               "tok_rope_table", "tok_rope_grid", "tok_rope_grid_adjoint", "tok_rope_positions",
               "tok_rope_positions_adjoint", "tok_sample_codes", "tok_cross_attention_workspace_size",
               "tok_cross_attention", "tok_cross_attention_backward_workspace_size", "tok_cross_attention_backward",
               "tok_embed_codes", "tok_embed_codes_backward_workspace_size", "tok_embed_codes_backward",
               "tok_page_tables", "tok_page_release", "tok_paged_write", "tok_paged_attention_workspace_size",
               "tok_paged_attention", "tok_verify_codes_workspace_size", "tok_verify_codes")

_lib = None


class _Heads(ctypes.Structure):
    """tok_heads: a [B, N, H, D] tensor with dense channels."""
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class _Pages(ctypes.Structure):
    """tok_pages: a [P, page_size, H, D] tensor with dense channels."""
    _fields_ = [("ptr", ctypes.c_void_p), ("page", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class TokError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = lib().tok_status_str(status).decode()
        if status == TOK_ERR_CUDA:
            msg += f" (cudaError {lib().tok_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")


def lib():
    """The loaded libtok.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m haar_wavelet_patching_b200.build` "
                              "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.tok_abi_version.restype = i32
        L.tok_abi_version.argtypes = []
        L.tok_status_str.restype = ctypes.c_char_p
        L.tok_status_str.argtypes = [i32]
        L.tok_last_cuda_error.restype = i32
        L.tok_last_cuda_error.argtypes = []
        L.tok_check_device.restype = i32
        L.tok_check_device.argtypes = [vp]
        L.tok_selftest_wait_timeout.restype = i32
        L.tok_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp]
        for f in (L.tok_haar_fwd, L.tok_haar_inv, L.tok_haar_fwd_adjoint, L.tok_haar_inv_adjoint,
                  L.tok_haar_fwd_single, L.tok_haar_inv_single, L.tok_haar_fwd_channels_last):
            f.restype = i32
            f.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, vp]
        L.tok_fsq_backward_workspace_size.restype = i64
        L.tok_fsq_backward_workspace_size.argtypes = [i64, i64, i64]
        for f in (L.tok_fsq_encode_backward, L.tok_fsq_decode_backward):
            f.restype = i32
            f.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp]
        L.tok_fsq_encode_backward_noalloc.restype = i32
        L.tok_fsq_encode_backward_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        for f in (L.tok_haar_fwd_windows, L.tok_haar_inv_windows):
            f.restype = i32
            f.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, i64, i64, vp]
        i64p = ctypes.POINTER(ctypes.c_int64)
        L.tok_haar_padded_extents.restype = i32
        L.tok_haar_padded_extents.argtypes = [i64, i64, i64, i64, i64, i64p, i64p, i64p]
        for f in (L.tok_haar_fwd_padded, L.tok_haar_inv_cropped):
            f.restype = i32
            f.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, i64, i64, vp]
        for f in (L.tok_haar_fwd_chunk, L.tok_haar_inv_chunk):
            f.restype = i32
            f.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, i32, vp]
        for f in (L.tok_conv_spatial, L.tok_conv_temporal_causal):
            f.restype = i32
            f.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, vp]
        L.tok_patch_embed_pack_weights.restype = i32
        L.tok_patch_embed_pack_weights.argtypes = [vp, vp, i64, i64, vp]
        L.tok_patch_embed_spatial.restype = i32
        L.tok_patch_embed_spatial.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64, vp]
        L.tok_conv_factorized.restype = i32
        L.tok_conv_factorized.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64, vp]
        L.tok_fsq_encode.restype = i32
        L.tok_fsq_encode.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        f64 = ctypes.c_double
        L.tok_rope_table.restype = i32
        L.tok_rope_table.argtypes = [vp] + [i64] * 6 + [f64] * 6 + [vp]
        for f in (L.tok_rope_grid, L.tok_rope_grid_adjoint):
            f.restype = i32
            f.argtypes = [vp, vp, vp, i32] + [i64] * 19 + [i32, vp]
        for f in (L.tok_rope_positions, L.tok_rope_positions_adjoint):
            f.restype = i32
            f.argtypes = [vp] * 5 + [i32] + [i64] * 13 + [i32, vp]
        f32 = ctypes.c_float
        for f in (L.tok_cross_attention_workspace_size, L.tok_cross_attention_backward_workspace_size):
            f.restype = i64
            f.argtypes = [i64] * 6
        hp = ctypes.POINTER(_Heads)
        L.tok_cross_attention.restype = i32
        L.tok_cross_attention.argtypes = [hp] * 4 + [vp, vp] + [i64] * 6 + [f32, vp, i64, vp]
        L.tok_cross_attention_backward.restype = i32
        L.tok_cross_attention_backward.argtypes = [hp] * 4 + [vp, hp, vp] + [hp] * 3 + [i64] * 6 + [f32, vp, i64, vp]
        L.tok_sample_codes.restype = i32
        L.tok_sample_codes.argtypes = [vp, i32, i64, i64, i64, vp, vp, f32, vp, i32, vp, f32, vp, f32, vp, vp, vp]
        L.tok_fsq_decode.restype = i32
        L.tok_fsq_decode.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        L.tok_embed_codes.restype = i32
        L.tok_embed_codes.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, i64, i64, f32, vp]
        L.tok_embed_codes_backward_workspace_size.restype = i64
        L.tok_embed_codes_backward_workspace_size.argtypes = [i64] * 3
        L.tok_embed_codes_backward.restype = i32
        L.tok_embed_codes_backward.argtypes = [vp, vp, vp, i32, i32] + [i64] * 5 + [f32, vp, i64, vp]
        L.tok_page_tables.restype = i32
        L.tok_page_tables.argtypes = [vp] * 10 + [i64] * 6 + [vp]
        L.tok_page_release.restype = i32
        L.tok_page_release.argtypes = [vp] * 8 + [i64] * 5 + [vp]
        pp = ctypes.POINTER(_Pages)
        L.tok_paged_write.restype = i32
        L.tok_paged_write.argtypes = [hp, hp, vp, pp, pp, vp] + [i64] * 6 + [vp]
        L.tok_paged_attention_workspace_size.restype = i64
        L.tok_paged_attention_workspace_size.argtypes = [i64] * 5
        L.tok_paged_attention.restype = i32
        L.tok_paged_attention.argtypes = [hp, pp, pp, vp, vp, vp, hp, vp] + [i64] * 9 + [f32, vp, i64, vp]
        L.tok_verify_codes.restype = i32
        L.tok_verify_codes.argtypes = [vp, vp, i32, vp, vp, vp, vp, f32, vp, vp] + [i64] * 7 + [vp, i64, vp]
        L.tok_verify_codes_workspace_size.restype = i64
        L.tok_verify_codes_workspace_size.argtypes = [i64] * 3
        _lib = L
    return _lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TOK_F32
    if t.dtype == torch.bfloat16:
        return TOK_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: the patcher takes float32 or bfloat16")


def _cuda(t: torch.Tensor, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(t: torch.Tensor, stream):
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _check(status, what):
    if status != TOK_OK:
        raise TokError(status, what)


# ---------------------------------------------------------------------------
# Shape rules (host logic).
# ---------------------------------------------------------------------------
def latent_frames(T: int) -> int:
    """1 + (T-1)/4 latent frames for T = 1 + 4k video frames; 1 for an image."""
    if T == 1:
        return 1
    if T < 1 or T % 4 != 1:
        raise ValueError(f"T={T}: the causal two-level patcher needs T == 1 or T % 4 == 1")
    return 1 + (T - 1) // 4


def haar_coeff_shape(B, C, T, H, W):
    if H % 4 or W % 4:
        raise ValueError(f"H={H}, W={W} must be multiples of 4")
    return (B, (16 if T == 1 else 64) * C, latent_frames(T), H // 4, W // 4)


# ---------------------------------------------------------------------------
# C-ABI calls.
# ---------------------------------------------------------------------------
def tok_check_device(device=None, stream=None):
    """Synchronize the stream; raise TokError if a kernel stopped after a bounded wait ran out."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    _check(lib().tok_check_device(ctypes.c_void_p(stream.cuda_stream)), "tok_check_device")


def tok_selftest_wait_timeout(polls: int, device=None, stream=None):
    """Launch the failure-channel self-test: a kernel whose barrier wait runs out after
    `polls` polls and counts a timeout (the next tok_check_device raises TOK_ERR_TIMEOUT)."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    _check(lib().tok_selftest_wait_timeout(polls, ctypes.c_void_p(stream.cuda_stream)), "tok_selftest_wait_timeout")


def tok_haar_fwd(x: torch.Tensor, y: torch.Tensor, stream=None):
    """x [B,C,T,H,W] -> y [B,64C,T',H/4,W/4] (T == 1: [B,16C,1,H/4,W/4]); same dtype."""
    _cuda(x, "x"), _cuda(y, "y")
    if x.dim() != 5:
        raise ValueError("x must be [B, C, T, H, W]")
    if y.dtype != x.dtype:
        raise TypeError("x and y must have the same dtype")
    B, C, T, H, W = x.shape
    if tuple(y.shape) != haar_coeff_shape(B, C, T, H, W):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {haar_coeff_shape(B, C, T, H, W)}")
    _check(lib().tok_haar_fwd(_ptr(x), _ptr(y), _dtype_code(x), B, C, T, H, W, _stream(x, stream)), "tok_haar_fwd")
    return y


def tok_haar_inv(y: torch.Tensor, x: torch.Tensor, stream=None):
    """Coefficients y -> x [B,C,T,H,W] (the output's shape gives T, H, W)."""
    _cuda(x, "x"), _cuda(y, "y")
    if x.dim() != 5:
        raise ValueError("x must be [B, C, T, H, W]")
    if y.dtype != x.dtype:
        raise TypeError("x and y must have the same dtype")
    B, C, T, H, W = x.shape
    if tuple(y.shape) != haar_coeff_shape(B, C, T, H, W):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {haar_coeff_shape(B, C, T, H, W)}")
    _check(lib().tok_haar_inv(_ptr(y), _ptr(x), _dtype_code(x), B, C, T, H, W, _stream(x, stream)), "tok_haar_inv")
    return x


def _haar_windows(fwd, x, y, t_begin, t_end, stream):
    _cuda(x, "x"), _cuda(y, "y")
    if x.dim() != 5 or y.dtype != x.dtype:
        raise ValueError("x must be [B, C, T, H, W] and y of the same dtype")
    B, C, T, H, W = x.shape
    if tuple(y.shape) != haar_coeff_shape(B, C, T, H, W):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {haar_coeff_shape(B, C, T, H, W)}")
    f = lib().tok_haar_fwd_windows if fwd else lib().tok_haar_inv_windows
    src, dst = (x, y) if fwd else (y, x)
    _check(f(_ptr(src), _ptr(dst), _dtype_code(x), B, C, T, H, W, int(t_begin), int(t_end), _stream(x, stream)),
           "tok_haar_fwd_windows" if fwd else "tok_haar_inv_windows")


def tok_haar_fwd_windows(x: torch.Tensor, y: torch.Tensor, t_begin: int, t_end: int, stream=None):
    """Forward restricted to latent frames [t_begin, t_end) of the full tensors x, y."""
    _haar_windows(True, x, y, t_begin, t_end, stream)
    return y


def tok_haar_inv_windows(y: torch.Tensor, x: torch.Tensor, t_begin: int, t_end: int, stream=None):
    """Inverse restricted to latent frames [t_begin, t_end): writes only those windows' pixel frames."""
    _haar_windows(False, x, y, t_begin, t_end, stream)
    return x


def channels_last_shape(B, C, T, H, W):
    """tok_haar_fwd_channels_last's output: [B, T', H/4, W/4, 64C] (images [B, 1, H/4, W/4, 16C])."""
    b, k, t, h, w = haar_coeff_shape(B, C, T, H, W)
    return (b, t, h, w, k)


def tok_haar_fwd_channels_last(x: torch.Tensor, y: torch.Tensor, stream=None):
    """x [B,C,T,H,W] -> y [B,T',H/4,W/4,64C]: the patcher's coefficients, channels last."""
    _cuda(x, "x"), _cuda(y, "y")
    if x.dim() != 5 or y.dtype != x.dtype:
        raise ValueError("x must be [B, C, T, H, W] and y of the same dtype")
    B, C, T, H, W = x.shape
    if tuple(y.shape) != channels_last_shape(B, C, T, H, W):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {channels_last_shape(B, C, T, H, W)}")
    _check(lib().tok_haar_fwd_channels_last(_ptr(x), _ptr(y), _dtype_code(x), B, C, T, H, W, _stream(x, stream)),
           "tok_haar_fwd_channels_last")
    return y


def haar_fwd_channels_last(x: torch.Tensor, stream=None) -> torch.Tensor:
    y = torch.empty(channels_last_shape(*x.shape), dtype=x.dtype, device=x.device)
    return tok_haar_fwd_channels_last(x, y, stream)


def single_coeff_shape(B, C, T, H, W):
    """The single-level patcher's output: [B, 8C, (T+1)/2, H/2, W/2], images [B, 4C, 1, H/2, W/2]."""
    return (B, 4 * C, 1, H // 2, W // 2) if T == 1 else (B, 8 * C, (T + 1) // 2, H // 2, W // 2)


def _haar_single(fwd, x, y, stream):
    _cuda(x, "x"), _cuda(y, "y")
    if x.dim() != 5 or y.dtype != x.dtype:
        raise ValueError("x must be [B, C, T, H, W] and y of the same dtype")
    B, C, T, H, W = x.shape
    if tuple(y.shape) != single_coeff_shape(B, C, T, H, W):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {single_coeff_shape(B, C, T, H, W)}")
    f = lib().tok_haar_fwd_single if fwd else lib().tok_haar_inv_single
    src, dst = (x, y) if fwd else (y, x)
    _check(f(_ptr(src), _ptr(dst), _dtype_code(x), B, C, T, H, W, _stream(x, stream)),
           "tok_haar_fwd_single" if fwd else "tok_haar_inv_single")


def tok_haar_fwd_single(x: torch.Tensor, y: torch.Tensor, stream=None):
    """The single-level patcher (patch_size=2): x [B,C,T,H,W] -> y (single_coeff_shape)."""
    _haar_single(True, x, y, stream)
    return y


def tok_haar_inv_single(y: torch.Tensor, x: torch.Tensor, stream=None):
    _haar_single(False, x, y, stream)
    return x


def padded_extents(T: int, H: int, W: int, spatial_multiple: int = 4, temporal_multiple: int = 4):
    """(Tp, Hp, Wp) of tok_haar_fwd_padded: zeros in space, a mirrored tail in time."""
    Tp, Hp, Wp = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().tok_haar_padded_extents(T, H, W, spatial_multiple, temporal_multiple, ctypes.byref(Tp),
                                         ctypes.byref(Hp), ctypes.byref(Wp)), "tok_haar_padded_extents")
    return Tp.value, Hp.value, Wp.value


def padded_coeff_shape(B, C, T, H, W, spatial_multiple=4, temporal_multiple=4):
    Tp, Hp, Wp = padded_extents(T, H, W, spatial_multiple, temporal_multiple)
    return haar_coeff_shape(B, C, Tp, Hp, Wp)


def tok_haar_fwd_padded(x: torch.Tensor, y: torch.Tensor, spatial_multiple: int = 4, temporal_multiple: int = 4,
                        stream=None):
    """x [B,C,T,H,W] of any extents -> y, the patcher of the padded clip (see padded_coeff_shape)."""
    _cuda(x, "x"), _cuda(y, "y")
    if x.dim() != 5 or y.dtype != x.dtype:
        raise ValueError("x must be [B, C, T, H, W] and y of the same dtype")
    B, C, T, H, W = x.shape
    if tuple(y.shape) != padded_coeff_shape(B, C, T, H, W, spatial_multiple, temporal_multiple):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected "
                         f"{padded_coeff_shape(B, C, T, H, W, spatial_multiple, temporal_multiple)}")
    _check(lib().tok_haar_fwd_padded(_ptr(x), _ptr(y), _dtype_code(x), B, C, T, H, W, spatial_multiple,
                                     temporal_multiple, _stream(x, stream)), "tok_haar_fwd_padded")
    return y


def tok_haar_inv_cropped(y: torch.Tensor, x: torch.Tensor, spatial_multiple: int = 4, temporal_multiple: int = 4,
                         stream=None):
    """Coefficients of a padded clip -> x [B,C,T,H,W], the unpatcher cropped to x's extents."""
    _cuda(x, "x"), _cuda(y, "y")
    if x.dim() != 5 or y.dtype != x.dtype:
        raise ValueError("x must be [B, C, T, H, W] and y of the same dtype")
    B, C, T, H, W = x.shape
    if tuple(y.shape) != padded_coeff_shape(B, C, T, H, W, spatial_multiple, temporal_multiple):
        raise ValueError("y does not have the padded coefficient shape of x")
    _check(lib().tok_haar_inv_cropped(_ptr(y), _ptr(x), _dtype_code(x), B, C, T, H, W, spatial_multiple,
                                      temporal_multiple, _stream(x, stream)), "tok_haar_inv_cropped")
    return x


def chunk_coeff_shape(B, C, T, H, W, first):
    """Streaming chunks are video: 64C channels, (T + 3) // 4 latent frames (first) or T // 4."""
    return (B, 64 * C, (T + 3) // 4 if first else T // 4, H // 4, W // 4)


def _haar_chunk(fwd, x, y, first, stream):
    _cuda(x, "x"), _cuda(y, "y")
    if x.dim() != 5 or y.dtype != x.dtype:
        raise ValueError("x must be [B, C, T, H, W] and y of the same dtype")
    B, C, T, H, W = x.shape
    if tuple(y.shape) != chunk_coeff_shape(B, C, T, H, W, first):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {chunk_coeff_shape(B, C, T, H, W, first)}")
    f = lib().tok_haar_fwd_chunk if fwd else lib().tok_haar_inv_chunk
    src, dst = (x, y) if fwd else (y, x)
    _check(f(_ptr(src), _ptr(dst), _dtype_code(x), B, C, T, H, W, int(bool(first)), _stream(x, stream)),
           "tok_haar_fwd_chunk" if fwd else "tok_haar_inv_chunk")


def tok_haar_fwd_chunk(x: torch.Tensor, y: torch.Tensor, first: bool, stream=None):
    """A chunk of a video: first -> T = 1 + 4k frames with the frame-0 replicas; else 4k frames, none."""
    _haar_chunk(True, x, y, first, stream)
    return y


def tok_haar_inv_chunk(y: torch.Tensor, x: torch.Tensor, first: bool, stream=None):
    _haar_chunk(False, x, y, first, stream)
    return x


def _conv_dims(x, name):
    _cuda(x, name)
    if x.dim() != 5 or x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a channels-last bf16 tensor [B, T, h, w, C]")
    return x.shape


def tok_conv_spatial(x: torch.Tensor, ws: torch.Tensor, y: torch.Tensor, stream=None):
    """1 x k x k convolution, 'same' zero padding: x [B,T,h,w,Cin], ws [Cout,k,k,Cin] -> y [B,T,h,w,Cout]."""
    B, T, h, w, Cin = _conv_dims(x, "x")
    _conv_dims(y, "y"), _cuda(ws, "ws")
    Cout, k = ws.shape[0], ws.shape[1]
    if tuple(ws.shape) != (Cout, k, k, Cin) or tuple(y.shape) != (B, T, h, w, Cout) or ws.dtype != torch.bfloat16:
        raise ValueError("ws must be bf16 [Cout, k, k, Cin] and y [B, T, h, w, Cout]")
    _check(lib().tok_conv_spatial(_ptr(x), _ptr(ws), _ptr(y), B, T, h, w, Cin, Cout, k, _stream(x, stream)),
           "tok_conv_spatial")
    return y


def tok_conv_temporal_causal(x: torch.Tensor, wt: torch.Tensor, y: torch.Tensor, stream=None):
    """k x 1 x 1 convolution over time, frame t reading t-k+1 .. t: wt [Cout, k, Cin]."""
    B, T, h, w, Cin = _conv_dims(x, "x")
    _conv_dims(y, "y"), _cuda(wt, "wt")
    Cout, k = wt.shape[0], wt.shape[1]
    if tuple(wt.shape) != (Cout, k, Cin) or tuple(y.shape) != (B, T, h, w, Cout) or wt.dtype != torch.bfloat16:
        raise ValueError("wt must be bf16 [Cout, k, Cin] and y [B, T, h, w, Cout]")
    _check(lib().tok_conv_temporal_causal(_ptr(x), _ptr(wt), _ptr(y), B, T, h, w, Cin, Cout, k,
                                          _stream(x, stream)), "tok_conv_temporal_causal")
    return y


def tok_conv_factorized(x, ws, wt, mid, y, stream=None):
    """The spatial convolution into mid, then the causal temporal convolution into y."""
    B, T, h, w, Cin = _conv_dims(x, "x")
    _conv_dims(mid, "mid"), _conv_dims(y, "y"), _cuda(ws, "ws"), _cuda(wt, "wt")
    Cmid, k, Cout = ws.shape[0], ws.shape[1], wt.shape[0]
    if (tuple(ws.shape) != (Cmid, k, k, Cin) or tuple(wt.shape) != (Cout, k, Cmid)
            or tuple(mid.shape) != (B, T, h, w, Cmid) or tuple(y.shape) != (B, T, h, w, Cout)):
        raise ValueError("shapes: ws [Cmid,k,k,Cin], wt [Cout,k,Cmid], mid [B,T,h,w,Cmid], y [B,T,h,w,Cout]")
    _check(lib().tok_conv_factorized(_ptr(x), _ptr(ws), _ptr(wt), _ptr(mid), _ptr(y), B, T, h, w, Cin, Cmid, Cout,
                                     k, _stream(x, stream)), "tok_conv_factorized")
    return y


def tok_patch_embed_pack_weights(ws: torch.Tensor, wp: torch.Tensor, stream=None):
    """Reorder the spatial filter ws [Cmid, 3, 3, 64C] for the fused call: wp [Cmid, 9C, 64]."""
    _cuda(ws, "ws"), _cuda(wp, "wp")
    Cmid, C = ws.shape[0], ws.shape[3] // 64
    if (ws.dim() != 4 or tuple(ws.shape[1:3]) != (3, 3) or ws.shape[3] != 64 * C or ws.dtype != torch.bfloat16
            or tuple(wp.shape) != (Cmid, 9 * C, 64) or wp.dtype != torch.bfloat16):
        raise ValueError("ws must be bf16 [Cmid, 3, 3, 64C] and wp bf16 [Cmid, 9C, 64]")
    _check(lib().tok_patch_embed_pack_weights(_ptr(ws), _ptr(wp), C, Cmid, _stream(ws, stream)),
           "tok_patch_embed_pack_weights")
    return wp


def tok_patch_embed_spatial(x: torch.Tensor, wp: torch.Tensor, y: torch.Tensor, stream=None):
    """The patcher fused into the 1 x 3 x 3 convolution: x [B,C,T,H,W] bf16 pixels, wp the packed
    filter [Cmid, 9C, 64] -> y [B, T', H/4, W/4, Cmid] bf16."""
    _cuda(x, "x"), _cuda(wp, "wp"), _cuda(y, "y")
    if x.dim() != 5 or x.dtype != torch.bfloat16 or wp.dtype != torch.bfloat16 or y.dtype != torch.bfloat16:
        raise ValueError("x [B, C, T, H, W], wp and y must be bf16")
    B, C, T, H, W = x.shape
    Cmid = wp.shape[0]
    if tuple(wp.shape) != (Cmid, 9 * C, 64) or tuple(y.shape) != (B, latent_frames(T), H // 4, W // 4, Cmid):
        raise ValueError("wp must be [Cmid, 9C, 64] and y [B, T', H/4, W/4, Cmid]")
    _check(lib().tok_patch_embed_spatial(_ptr(x), _ptr(wp), _ptr(y), B, C, T, H, W, Cmid, _stream(x, stream)),
           "tok_patch_embed_spatial")
    return y


def patch_embed_pack_weights(ws, stream=None):
    Cmid, C = ws.shape[0], ws.shape[3] // 64
    wp = torch.empty((Cmid, 9 * C, 64), dtype=torch.bfloat16, device=ws.device)
    return tok_patch_embed_pack_weights(ws, wp, stream)


def patch_embed_spatial(x, wp, stream=None):
    B, C, T, H, W = x.shape
    y = torch.empty((B, latent_frames(T), H // 4, W // 4, wp.shape[0]), dtype=torch.bfloat16, device=x.device)
    return tok_patch_embed_spatial(x, wp, y, stream)


def conv_factorized(x, ws, wt, stream=None):
    B, T, h, w, _ = x.shape
    mid = torch.empty((B, T, h, w, ws.shape[0]), dtype=torch.bfloat16, device=x.device)
    y = torch.empty((B, T, h, w, wt.shape[0]), dtype=torch.bfloat16, device=x.device)
    return tok_conv_factorized(x, ws, wt, mid, y, stream)


def tok_haar_fwd_adjoint(gy: torch.Tensor, gx: torch.Tensor, stream=None):
    """Gradient of the patcher: gy (coefficient shape) -> gx [B,C,T,H,W]."""
    _cuda(gx, "gx"), _cuda(gy, "gy")
    B, C, T, H, W = gx.shape
    if gy.dtype != gx.dtype or tuple(gy.shape) != haar_coeff_shape(B, C, T, H, W):
        raise ValueError("gy must have the coefficient shape and dtype of gx")
    _check(lib().tok_haar_fwd_adjoint(_ptr(gy), _ptr(gx), _dtype_code(gx), B, C, T, H, W, _stream(gx, stream)),
           "tok_haar_fwd_adjoint")
    return gx


def tok_haar_inv_adjoint(gx: torch.Tensor, gy: torch.Tensor, stream=None):
    """Gradient of the unpatcher: gx [B,C,T,H,W] -> gy (coefficient shape)."""
    _cuda(gx, "gx"), _cuda(gy, "gy")
    B, C, T, H, W = gx.shape
    if gy.dtype != gx.dtype or tuple(gy.shape) != haar_coeff_shape(B, C, T, H, W):
        raise ValueError("gy must have the coefficient shape and dtype of gx")
    _check(lib().tok_haar_inv_adjoint(_ptr(gx), _ptr(gy), _dtype_code(gx), B, C, T, H, W, _stream(gx, stream)),
           "tok_haar_inv_adjoint")
    return gy


def _latent_dims(u: torch.Tensor):
    if u.dim() < 2:
        raise ValueError("latent must be [B, C, ...]")
    B, C = u.shape[0], u.shape[1]
    S = 1
    for d in u.shape[2:]:
        S *= d
    return B, C, S


def tok_fsq_encode(u: torch.Tensor, w: torch.Tensor, idx: torch.Tensor, codes: torch.Tensor = None, stream=None):
    """u [B,C,...] fp32, w [6,C] fp32 -> idx [B,...] int32 (+ codes [B,6,...] fp32)."""
    for t, n in ((u, "u"), (w, "w"), (idx, "idx"), (codes, "codes")):
        _cuda(t, n)
    B, C, S = _latent_dims(u)
    if u.dtype != torch.float32 or w.dtype != torch.float32 or idx.dtype != torch.int32:
        raise TypeError("u and w must be float32, idx int32")
    if tuple(w.shape) != (FSQ_DIM, C):
        raise ValueError(f"w must be [6, {C}]")
    if idx.numel() != B * S or (codes is not None and (codes.numel() != B * FSQ_DIM * S or codes.dtype != torch.float32)):
        raise ValueError("idx must hold B*S int32 and codes B*6*S float32")
    _check(lib().tok_fsq_encode(_ptr(u), _ptr(w), _ptr(idx), _ptr(codes), B, C, S, _stream(u, stream)),
           "tok_fsq_encode")
    return idx, codes


def tok_fsq_decode(idx: torch.Tensor, w: torch.Tensor, out: torch.Tensor, bad_count: torch.Tensor = None,
                   stream=None):
    """idx [B,...] int32, w [6,C] -> out [B,C,...] fp32; bad_count: optional 1-element int32 CUDA tensor."""
    for t, n in ((idx, "idx"), (w, "w"), (out, "out"), (bad_count, "bad_count")):
        _cuda(t, n)
    B, C, S = _latent_dims(out)
    if idx.dtype != torch.int32 or w.dtype != torch.float32 or out.dtype != torch.float32:
        raise TypeError("idx must be int32, w and out float32")
    if tuple(w.shape) != (FSQ_DIM, C) or idx.numel() != B * S:
        raise ValueError(f"w must be [6, {C}] and idx hold B*S = {B * S} indices")
    if bad_count is not None and (bad_count.dtype != torch.int32 or bad_count.numel() < 1):
        raise ValueError("bad_count must be an int32 CUDA tensor")
    _check(lib().tok_fsq_decode(_ptr(idx), _ptr(w), _ptr(out), _ptr(bad_count), B, C, S, _stream(idx, stream)),
           "tok_fsq_decode")
    return out


def fsq_backward_workspace_size(B: int, C: int, S: int) -> int:
    n = int(lib().tok_fsq_backward_workspace_size(B, C, S))
    if n < 0:
        raise ValueError(f"no FSQ backward for B={B}, C={C}, S={S} (1 <= C <= 16)")
    return n


def tok_fsq_encode_backward(u, w, grad_codes, grad_u, grad_w, workspace, stream=None):
    """Straight-through encode backward into grad_u [B,C,...] and grad_w [6,C]; workspace: uint8 CUDA tensor."""
    for t, n in ((u, "u"), (w, "w"), (grad_codes, "grad_codes"), (grad_u, "grad_u"), (grad_w, "grad_w"),
                 (workspace, "workspace")):
        _cuda(t, n)
    B, C, S = _latent_dims(u)
    if grad_u.shape != u.shape or grad_codes.numel() != B * FSQ_DIM * S or tuple(grad_w.shape) != (FSQ_DIM, C):
        raise ValueError("shapes: grad_u like u, grad_codes [B,6,...], grad_w [6,C]")
    _check(lib().tok_fsq_encode_backward(_ptr(u), _ptr(w), _ptr(grad_codes), _ptr(grad_u), _ptr(grad_w),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(), B, C, S,
                                         _stream(u, stream)), "tok_fsq_encode_backward")
    return grad_u, grad_w


def tok_fsq_encode_backward_noalloc(u, w, grad_codes, grad_u, grad_w, stream=None):
    """tok_fsq_encode_backward using the library's fixed scratch instead of a workspace (allocates nothing;
    its 3 MB scratch holds at most 8,388,608 tokens at C = 16; concurrent calls must be serialized by the caller)."""
    for t, n in ((u, "u"), (w, "w"), (grad_codes, "grad_codes"), (grad_u, "grad_u"), (grad_w, "grad_w")):
        _cuda(t, n)
    B, C, S = _latent_dims(u)
    if grad_u.shape != u.shape or grad_codes.numel() != B * FSQ_DIM * S or tuple(grad_w.shape) != (FSQ_DIM, C):
        raise ValueError("shapes: grad_u like u, grad_codes [B,6,...], grad_w [6,C]")
    _check(lib().tok_fsq_encode_backward_noalloc(_ptr(u), _ptr(w), _ptr(grad_codes), _ptr(grad_u), _ptr(grad_w),
                                                 B, C, S, _stream(u, stream)), "tok_fsq_encode_backward_noalloc")
    return grad_u, grad_w


def tok_fsq_decode_backward(idx, w, grad_out, grad_codes, grad_w, workspace, stream=None):
    """Decode backward into grad_codes [B,6,...] and grad_w [6,C]; workspace: uint8 CUDA tensor."""
    for t, n in ((idx, "idx"), (w, "w"), (grad_out, "grad_out"), (grad_codes, "grad_codes"), (grad_w, "grad_w"),
                 (workspace, "workspace")):
        _cuda(t, n)
    B, C, S = _latent_dims(grad_out)
    if idx.numel() != B * S or grad_codes.numel() != B * FSQ_DIM * S or tuple(grad_w.shape) != (FSQ_DIM, C):
        raise ValueError("shapes: idx [B,...], grad_codes [B,6,...], grad_w [6,C]")
    _check(lib().tok_fsq_decode_backward(_ptr(idx), _ptr(w), _ptr(grad_out), _ptr(grad_codes), _ptr(grad_w),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(), B, C, S,
                                         _stream(idx, stream)), "tok_fsq_decode_backward")
    return grad_codes, grad_w


# ---------------------------------------------------------------------------
# Calls of the token-model operators: on the tensors' device, whichever is current.
# ---------------------------------------------------------------------------
def _call(name, device, stream, *args):
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        s = stream.cuda_stream
    if torch.cuda.current_device() == device.index:
        status = getattr(_lib or lib(), name)(*args, s)
    else:
        with torch.cuda.device(device):
            status = getattr(_lib or lib(), name)(*args, s)
    if status != TOK_OK:
        raise TokError(status, name)


# ---------------------------------------------------------------------------
# Rotary positions of the axes (time, height, width).
# ---------------------------------------------------------------------------
def _triple(v):
    return tuple(v) if isinstance(v, (tuple, list)) else (v, v, v)


def rope_table(sizes, dims, base=10000.0, scale=1.0, device="cuda", stream=None) -> torch.Tensor:
    """cos and sin of positions [0, sizes[a]) and the dims[a] / 2 pairs of each axis (t, h, w), for the
    rope_* calls: float32 [sum sizes[a] * dims[a]].  base, scale: one number or one per axis."""
    (nt, nh, nw), (dt, dh, dw) = sizes, dims
    if min(nt, nh, nw, dt, dh, dw) < 0:
        raise ValueError("sizes and dims must not be negative")
    if torch.device(device).type != "cuda":
        raise ValueError("the table must be on a CUDA device (there is no CPU path)")
    table = _new(torch.empty(0, device=device), nt * dt + nh * dh + nw * dw, torch.float32, stream)
    _call("tok_rope_table", table.device, stream, table.data_ptr(), nt, nh, nw, dt, dh, dw, *_triple(base),
          *_triple(scale))
    return table


def _rope_check(x, y, table, sizes, dims):
    dev = x.device
    if dev.type != "cuda" or y.device != dev or table.device != dev:
        raise ValueError("x, y and table must be CUDA tensors on one device (there is no CPU path)")
    if x.shape != y.shape or x.dtype != y.dtype:
        raise ValueError("x and y must have the same shape and dtype")
    if table.dtype != torch.float32 or table.numel() != sizes[0] * dims[0] + sizes[1] * dims[1] + sizes[2] * dims[2] \
            or not table.is_contiguous():
        raise ValueError("table must be the float32 rope_table of these sizes and dims")
    if x.shape[-1] > 1 and (x.stride(-1) != 1 or y.stride(-1) != 1):
        raise ValueError("the channels of x and y must be dense")


def _token_stride(t: torch.Tensor, name: str) -> int:
    """The one stride of the leading dimensions of [..., heads, D] taken as one index."""
    if t.is_contiguous():
        return t.shape[-1] * t.shape[-2]
    stride = None
    for n, s in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if n != 1:
            if stride is None:
                first, stride = s, s
            elif s != stride:
                raise ValueError(f"the leading dimensions of {name} must have one common stride")
            stride *= n
    return 0 if stride is None else first


def _rope_grid(name, x, y, table, sizes, dims, origin, interleaved, stream):
    _rope_check(x, y, table, sizes, dims)
    if x.dim() != 6:
        raise ValueError("the tensors must be [B, T, h, w, heads, D]")
    B, T, h, w, H, D = x.shape
    _call(name, x.device, stream, x.data_ptr(), y.data_ptr(), table.data_ptr(), _dtype_code(x), B, T, h, w, H, D,
          _token_stride(x, "x"), x.stride(4), _token_stride(y, "y"), y.stride(4), *origin, *sizes, *dims,
          bool(interleaved))
    return y


def tok_rope_grid(x, y, table, sizes, dims, origin=(0, 0, 0), interleaved=False, stream=None):
    """Rotary positions of every token of a grid: x [B,T,h,w,heads,D] -> y, token (t, i, j) at position
    origin + (t, i, j).  x and y may be strided (dense channels, one token stride); y may be x."""
    return _rope_grid("tok_rope_grid", x, y, table, sizes, dims, origin, interleaved, stream)


def tok_rope_grid_adjoint(gy, gx, table, sizes, dims, origin=(0, 0, 0), interleaved=False, stream=None):
    """Gradient of tok_rope_grid: gy -> gx."""
    return _rope_grid("tok_rope_grid_adjoint", gy, gx, table, sizes, dims, origin, interleaved, stream)


def _rope_positions(name, x, y, pos, table, sizes, dims, interleaved, bad_count, stream):
    _rope_check(x, y, table, sizes, dims)
    if x.dim() < 3:
        raise ValueError("the tensors must be [..., heads, D]")
    if pos.device != x.device or pos.dtype != torch.int32 or not pos.is_contiguous() \
            or pos.shape != x.shape[:-2] + (3,):
        raise ValueError("pos must be a contiguous int32 CUDA tensor [..., 3] of (t, h, w)")
    if bad_count is not None and (bad_count.device != x.device or bad_count.dtype != torch.int32 or bad_count.numel() < 1):
        raise ValueError("bad_count must be an int32 CUDA tensor")
    H, D = x.shape[-2:]
    N = 1
    for n in x.shape[:-2]:
        N *= n
    _call(name, x.device, stream, x.data_ptr(), y.data_ptr(), pos.data_ptr(), table.data_ptr(),
          None if bad_count is None else bad_count.data_ptr(), _dtype_code(x), N, H, D, _token_stride(x, "x"),
          x.stride(-2), _token_stride(y, "y"), y.stride(-2), *sizes, *dims, bool(interleaved))
    return y


def tok_rope_positions(x, y, pos, table, sizes, dims, interleaved=False, bad_count=None, stream=None):
    """Rotary positions of tokens at given places: x [..., heads, D], pos [..., 3] int32 -> y.  A position
    outside the table gives NaN in the rotated channels and adds 1 to bad_count (int32 CUDA tensor)."""
    return _rope_positions("tok_rope_positions", x, y, pos, table, sizes, dims, interleaved, bad_count, stream)


def tok_rope_positions_adjoint(gy, gx, pos, table, sizes, dims, interleaved=False, bad_count=None, stream=None):
    """Gradient of tok_rope_positions: gy -> gx."""
    return _rope_positions("tok_rope_positions_adjoint", gy, gx, pos, table, sizes, dims, interleaved, bad_count,
                           stream)


# ---------------------------------------------------------------------------
# Drawing codes from logits.
# ---------------------------------------------------------------------------
def _setting(v, name, dtype, rows, device):
    """A sampling setting: (device pointer or None, value for every row)."""
    if not isinstance(v, torch.Tensor):
        return None, v
    if v.device != device or v.dtype != dtype or v.numel() != rows or not v.is_contiguous():
        raise ValueError(f"{name} must be a number or a contiguous {dtype} CUDA tensor with one value per row")
    return v.data_ptr(), 0


def tok_sample_codes(logits, u, idx, logprob=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """Draw one code per row: logits [..., V] (float32 or bfloat16), u [...] fp32 in [0, 1) -> idx [...] int32
    (-1 for a row of -inf) and, if given, logprob [...] fp32 under the filtered distribution.  The settings
    are numbers or tensors with one value per row (float32; top_k int32).  Filters: top_k largest, then the
    top_p nucleus, then weight >= min_p of the largest; ties to the lower index; temperature 0 is greedy."""
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError("logits must be a CUDA tensor (there is no CPU path)")
    if logits.dim() < 1 or logits.shape[-1] < 1:
        raise ValueError("logits must be [..., V] with V >= 1")
    lead, V = logits.shape[:-1], logits.shape[-1]
    if V > 1 and logits.stride(-1) != 1:
        raise ValueError("the last dimension of logits must be dense")
    for t, name, dtype in ((u, "u", torch.float32), (idx, "idx", torch.int32), (logprob, "logprob", torch.float32)):
        if t is not None and (t.device != dev or t.dtype != dtype or t.shape != lead or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor with one value per row")
    R = u.numel()
    tp, ta = _setting(temperature, "temperature", torch.float32, R, dev)
    kp, ka = _setting(top_k, "top_k", torch.int32, R, dev)
    pp, pa = _setting(top_p, "top_p", torch.float32, R, dev)
    mp, ma = _setting(min_p, "min_p", torch.float32, R, dev)
    stride = V if logits.is_contiguous() else _token_stride(logits.unsqueeze(-2), "logits")
    _call("tok_sample_codes", dev, stream, logits.data_ptr(), _dtype_code(logits), R, V, stride, u.data_ptr(), tp, ta,
          kp, max(-1, min(ka, 2 ** 31 - 1)), pp, pa, mp, ma, idx.data_ptr(),
          None if logprob is None else logprob.data_ptr())
    return idx, logprob


# ---------------------------------------------------------------------------
# Cross attention.
# ---------------------------------------------------------------------------
def _heads(t: torch.Tensor) -> _Heads:
    b, n, h, _ = t.stride()
    return _Heads(t.data_ptr(), b, n, h)


def _attn_dims(q, k, v, k_lens, others):
    """(B, Nq, Nk, Hq, Hkv, D) of checked tensors; others: (tensor, name, like q or like k)."""
    dev = q.device
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, Nq, Hq, D], k and v [B, Nk, Hkv, D]")
    B, Nq, Hq, D = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    sq, sk = q.shape, torch.Size((B, Nk, Hkv, D))
    if dev.type != "cuda":
        raise ValueError("q must be a CUDA tensor (there is no CPU path)")
    for t, name, shape in ((q, "q", sq), (k, "k", sk), (v, "v", sk), *((t, n, sq if lq else sk) for t, n, lq in others)):
        if t.dtype != torch.bfloat16 or t.device != dev:
            raise ValueError(f"{name} must be a bfloat16 CUDA tensor on the device of q")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.stride(3) != 1:
            raise ValueError(f"the channels of {name} must be dense")
    if k_lens is not None and (k_lens.device != dev or k_lens.dtype != torch.int32
                               or k_lens.shape != (B,) or not k_lens.is_contiguous()):
        raise ValueError("k_lens must be a contiguous int32 CUDA tensor [B]")
    return B, Nq, Nk, Hq, Hkv, D


def _stats(t, name, dims, device):
    B, Nq, _, Hq, _, _ = dims
    if t is not None and (t.device != device or t.dtype != torch.float32 or t.shape != (B, Hq, Nq) or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor [B, Hq, Nq]")


def _attn_workspace(f, dims, workspace, like, stream):
    need = f(*dims)
    if need < 0:
        raise ValueError(f"no cross attention for (B, Nq, Nk, Hq, Hkv, D) = {dims}: D a multiple of 8, at most 128; "
                         "Hq a multiple of Hkv")
    if workspace is None:
        return _new(like, need, torch.uint8, stream) if need else None
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the device of q")
    return workspace


def _bytes(t):
    return (None, 0) if t is None else (t.data_ptr(), t.numel() * t.element_size())


def cross_attention_workspace_size(B, Nq, Nk, Hq, Hkv, D) -> int:
    return int(lib().tok_cross_attention_workspace_size(B, Nq, Nk, Hq, Hkv, D))


def cross_attention_backward_workspace_size(B, Nq, Nk, Hq, Hkv, D) -> int:
    return int(lib().tok_cross_attention_backward_workspace_size(B, Nq, Nk, Hq, Hkv, D))


def tok_cross_attention(q, k, v, o, lse=None, k_lens=None, scale=None, workspace=None, stream=None):
    """o = softmax(scale q k^T) v over the first k_lens[b] keys: q, o [B,Nq,Hq,D], k, v [B,Nk,Hkv,D] bf16 (dense
    channels, other strides free), lse [B,Hq,Nq] fp32 or None, k_lens [B] int32 or None; scale: 1/sqrt(D) by
    default; workspace: cross_attention_workspace_size bytes, allocated if None."""
    dims = _attn_dims(q, k, v, k_lens, ((o, "o", True),))
    _stats(lse, "lse", dims, q.device)
    ws = _attn_workspace(lib().tok_cross_attention_workspace_size, dims, workspace, q, stream)
    _call("tok_cross_attention", q.device, stream, _heads(q), _heads(k), _heads(v), _heads(o),
          None if lse is None else lse.data_ptr(), None if k_lens is None else k_lens.data_ptr(), *dims,
          dims[5] ** -0.5 if scale is None else scale, *_bytes(ws))
    return o


def tok_cross_attention_backward(q, k, v, o, lse, grad_o, grad_q, grad_k, grad_v, k_lens=None, scale=None,
                                 workspace=None, stream=None):
    """Gradients of tok_cross_attention into grad_q, grad_k, grad_v, from its inputs, o and lse."""
    dims = _attn_dims(q, k, v, k_lens, ((o, "o", True), (grad_o, "grad_o", True), (grad_q, "grad_q", True),
                                        (grad_k, "grad_k", False), (grad_v, "grad_v", False)))
    if lse is None:
        raise ValueError("lse must be what tok_cross_attention gave (with_lse)")
    _stats(lse, "lse", dims, q.device)
    ws = _attn_workspace(lib().tok_cross_attention_backward_workspace_size, dims, workspace, q, stream)
    _call("tok_cross_attention_backward", q.device, stream, _heads(q), _heads(k), _heads(v), _heads(o), lse.data_ptr(),
          _heads(grad_o), None if k_lens is None else k_lens.data_ptr(), _heads(grad_q), _heads(grad_k), _heads(grad_v),
          *dims, dims[5] ** -0.5 if scale is None else scale, *_bytes(ws))
    return grad_q, grad_k, grad_v


# ---------------------------------------------------------------------------
# A step over the codes, token by token.  These calls are short, so their checks are one expression each where all is
# well; what is wrong is found out afterwards.
# ---------------------------------------------------------------------------
_i32, _f32, _bf16 = torch.int32, torch.float32, torch.bfloat16
_raw_stream, _device_now = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _enqueue(name, dev, stream, *args):
    """_call for a device index."""
    s = _raw_stream(dev) if stream is None else stream.cuda_stream
    f = getattr(_lib or lib(), name)
    if _device_now() == dev:
        status = f(*args, s)
    else:
        with torch.cuda.device(dev):
            status = f(*args, s)
    if status != TOK_OK:
        raise TokError(status, name)


def _device_of(t, name):
    """The index of a CUDA tensor's device."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return t.get_device()


def _is(t, dtype, dev, shape):
    return t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous()


def _need(t, name, dtype, dev, shape):
    """A contiguous tensor of this dtype and shape on this device, or None."""
    if t is not None and not _is(t, dtype, dev, shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on cuda:{dev}")


def _counter(t, dev):
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not _i32 or t.numel() < 1:
        raise ValueError("bad_count must be an int32 CUDA tensor on the device of the inputs")
    return t.data_ptr()


def _row_stride(t, name):
    """The stride of the rows of [..., D], dense in D, its leading dimensions taken as one index."""
    if t.is_contiguous():
        return t.shape[-1]
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be dense")
    return _token_stride(t.unsqueeze(-2), name)


def _workspace_of(need, workspace, like, stream, what):
    if need < 0:
        raise ValueError(what)
    if workspace is None:
        return _new(like, need, torch.uint8, stream) if need else None
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the device of the inputs")
    return workspace


# ---------------------------------------------------------------------------
# Embedding of codes.
# ---------------------------------------------------------------------------
def _codes_check(codes, dev, rows, name):
    if codes.dtype is not _i32 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous int32 CUDA tensor")
    if rows.get_device() != dev or rows.dim() < 1 or rows.shape[:-1] != codes.shape:
        raise ValueError(f"{name} must be [..., D] on the device of codes [...]")


def tok_embed_codes(codes, table, y, scale=1.0, bad_count=None, stream=None):
    """y[..., :] = scale * table[codes]: codes [...] int32, table [V, D], y [..., D] (float32 or bfloat16, rows
    strided).  A code outside the table gives a row of NaN and adds 1 to bad_count (int32 CUDA tensor)."""
    dev = _device_of(codes, "codes")
    _codes_check(codes, dev, y, "y")
    if table.dim() != 2 or table.get_device() != dev or table.dtype is not y.dtype or table.shape[1] != y.shape[-1]:
        raise ValueError("table must be [V, D] with the dtype, device and D of y")
    V, D = table.shape
    _enqueue("tok_embed_codes", dev, stream, codes.data_ptr(), table.data_ptr(), y.data_ptr(),
             _counter(bad_count, dev), _dtype_code(y), codes.numel(), V, D, _row_stride(table, "table"),
             _row_stride(y, "y"), scale)
    return y


def embed_codes_backward_workspace_size(N, V, D) -> int:
    return int(lib().tok_embed_codes_backward_workspace_size(N, V, D))


def tok_embed_codes_backward(grad_y, codes, grad_table, scale=1.0, workspace=None, stream=None):
    """Gradient of tok_embed_codes into grad_table [V, D] (overwritten): grad_y [..., D], codes [...]; the two
    gradients' dtypes are their own.  workspace: embed_codes_backward_workspace_size bytes, allocated if None."""
    dev = _device_of(codes, "codes")
    _codes_check(codes, dev, grad_y, "grad_y")
    if grad_table.dim() != 2 or grad_table.get_device() != dev or grad_table.shape[1] != grad_y.shape[-1]:
        raise ValueError("grad_table must be [V, D] with the device and D of grad_y")
    N, (V, D) = codes.numel(), grad_table.shape
    ws = _workspace_of(embed_codes_backward_workspace_size(N, V, D), workspace, codes, stream,
                       f"no embedding for (N, V, D) = {(N, V, D)}: V at most 2^18, D at most 65536")
    _enqueue("tok_embed_codes_backward", dev, stream, codes.data_ptr(), grad_y.data_ptr(), grad_table.data_ptr(),
             _dtype_code(grad_y), _dtype_code(grad_table), N, V, D, _row_stride(grad_y, "grad_y"),
             _row_stride(grad_table, "grad_table"), scale, *_bytes(ws))
    return grad_table


# ---------------------------------------------------------------------------
# Pages of a cache of keys and values.
# ---------------------------------------------------------------------------
_ONE = torch.Size((1,))


def _table_check(table, dev, B):
    """The table's row stride."""
    if table.dtype is not _i32 or table.get_device() != dev or table.dim() != 2 or table.shape[0] != B \
            or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be an int32 CUDA tensor [B, M] with dense rows")
    return table.stride(0) if B > 1 else table.shape[1]


def _counts_check(dev, lens, held, free, pages, held_out, free_out):
    shape = lens.shape
    if not (len(shape) == 1 and pages.dim() == 1 and _is(lens, _i32, dev, shape) and _is(held, _i32, dev, shape)
            and _is(held_out, _i32, dev, shape) and _is(free, _i32, dev, _ONE) and _is(free_out, _i32, dev, _ONE)
            and _is(pages, _i32, dev, pages.shape)):
        raise ValueError("lens, held and held_out must be [B], free and free_out [1], pages [F], all contiguous int32 "
                         "tensors on one CUDA device")


def tok_page_tables(lens, fresh, held, free, pages, table, slots, held_out, free_out, page_size, bad_count=None,
                    stream=None):
    """Room for new tokens: stream b has lens[b] tokens and gets fresh[b] more (None: all of slots' columns).  Pages
    come off the end of pages[:free] in the order of streams and go into table [B, M]; slots [B, N] gets
    page * page_size + row of each new token (-1 behind them), held_out and free_out the new counts (they may be
    held and free).  A stream without room gets slots of -1 and adds 1 to bad_count.  All int32."""
    dev = _device_of(lens, "lens")
    _counts_check(dev, lens, held, free, pages, held_out, free_out)
    B = lens.shape[0]
    row = _table_check(table, dev, B)
    if slots.dim() != 2 or slots.shape[0] != B or not _is(slots, _i32, dev, slots.shape):
        raise ValueError("slots must be a contiguous int32 CUDA tensor [B, N]")
    _need(fresh, "fresh", _i32, dev, lens.shape)
    _enqueue("tok_page_tables", dev, stream, lens.data_ptr(), None if fresh is None else fresh.data_ptr(),
             held.data_ptr(), free.data_ptr(), pages.data_ptr(), table.data_ptr(), slots.data_ptr(),
             held_out.data_ptr(), free_out.data_ptr(), _counter(bad_count, dev), B, slots.shape[1], table.shape[1],
             pages.shape[0], page_size, row)
    return slots


def tok_page_release(lens, held, free, pages, table, held_out, free_out, page_size, bad_count=None, stream=None):
    """Give back the pages that lens[b] tokens do not need: onto pages[free:], their table entries become -1; held_out and
    free_out get the new counts (they may be held and free)."""
    dev = _device_of(lens, "lens")
    _counts_check(dev, lens, held, free, pages, held_out, free_out)
    B = lens.shape[0]
    row = _table_check(table, dev, B)
    _enqueue("tok_page_release", dev, stream, lens.data_ptr(), held.data_ptr(), free.data_ptr(), pages.data_ptr(),
             table.data_ptr(), held_out.data_ptr(), free_out.data_ptr(), _counter(bad_count, dev), B, table.shape[1],
             pages.shape[0], page_size, row)


def _view4(t, name, dev):
    """Strides of a bfloat16 tensor of four dimensions with dense channels."""
    if t.dtype is not _bf16 or t.get_device() != dev or t.dim() != 4:
        raise ValueError(f"{name} must be a bfloat16 tensor of four dimensions on cuda:{dev}")
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"the channels of {name} must be dense")
    return s


def _heads_of(t, name, dev):
    s = _view4(t, name, dev)
    return _Heads(t.data_ptr(), s[0], s[1], s[2])


def _pool_of(t, name, dev):
    s = _view4(t, name, dev)
    return _Pages(t.data_ptr(), s[0], s[1], s[2])


def paged_write(k, v, k_pages, v_pages, slots, bad_count=None, stream=None):
    """Keys and values k, v [B, N, H, D] (dense channels, other strides free) into the pages [P, page_size, H, D] at
    slots [B, N] int32 (page * page_size + row; below 0: left out), all bfloat16.  A slot behind the pool is left
    out and adds 1 to bad_count.  Slots must differ."""
    dev = _device_of(k, "k")
    shape, pool = k.shape, k_pages.shape
    args = (_heads_of(k, "k", dev), _heads_of(v, "v", dev), slots.data_ptr(), _pool_of(k_pages, "k_pages", dev),
            _pool_of(v_pages, "v_pages", dev))
    if v.shape != shape or v_pages.shape != pool or pool[2:] != shape[2:]:
        raise ValueError("k and v must be [B, N, H, D], alike, k_pages and v_pages [P, page_size, H, D], alike")
    _need(slots, "slots", _i32, dev, shape[:2])
    _enqueue("tok_paged_write", dev, stream, *args, _counter(bad_count, dev), *shape, pool[0], pool[1])


tok_paged_write = paged_write


def paged_attention_workspace_size(B, Nq, Hq, Hkv, D) -> int:
    return int(lib().tok_paged_attention_workspace_size(B, Nq, Hq, Hkv, D))


def tok_paged_attention(q, k_pages, v_pages, table, k_lens, o, lse=None, q_lens=None, scale=None, workspace=None,
                        stream=None):
    """Attention of new tokens over pages: q, o [B, Nq, Hq, D], pages [P, page_size, Hkv, D] bfloat16 (dense
    channels, other strides free), table [B, M], k_lens [B], q_lens [B] or None (Nq) int32.  Query i < q_lens[b] is token
    k_lens[b] - q_lens[b] + i of its stream and sees the tokens up to itself; the others get o = 0, lse = -inf.
    lse [B, Hq, Nq] fp32 or None; scale: 1/sqrt(D) by default; workspace: paged_attention_workspace_size bytes,
    allocated if None."""
    dev = _device_of(q, "q")
    args = (_heads_of(q, "q", dev), _pool_of(k_pages, "k_pages", dev), _pool_of(v_pages, "v_pages", dev))
    out = _heads_of(o, "o", dev)
    B, Nq, Hq, D = q.shape
    P, page_size, Hkv, _ = pool = k_pages.shape
    if o.shape != q.shape or v_pages.shape != pool or pool[3] != D:
        raise ValueError("q and o must be [B, Nq, Hq, D], alike, k_pages and v_pages [P, page_size, Hkv, D], alike")
    row = _table_check(table, dev, B)
    if k_lens is None:
        raise ValueError("k_lens must be a contiguous int32 CUDA tensor [B]")
    _need(k_lens, "k_lens", _i32, dev, q.shape[:1])
    _need(q_lens, "q_lens", _i32, dev, q.shape[:1])
    _need(lse, "lse", _f32, dev, (B, Hq, Nq))
    ws = _workspace_of((_lib or lib()).tok_paged_attention_workspace_size(B, Nq, Hq, Hkv, D), workspace, q, stream,
                       f"no paged attention for (B, Nq, Hq, Hkv, D) = {(B, Nq, Hq, Hkv, D)}: D a multiple of 8, at "
                       "most 128; Hq a multiple of Hkv; Nq at most 64")
    _enqueue("tok_paged_attention", dev, stream, *args, table.data_ptr(), k_lens.data_ptr(),
             None if q_lens is None else q_lens.data_ptr(), out, None if lse is None else lse.data_ptr(), B, Nq, Hq, Hkv, D,
             P, page_size, table.shape[1], row, D ** -0.5 if scale is None else scale, *_bytes(ws))
    return o


# ---------------------------------------------------------------------------
# Verifying drafted codes.
# ---------------------------------------------------------------------------
def verify_codes_workspace_size(B, K, V) -> int:
    return int(lib().tok_verify_codes_workspace_size(B, K, V))


def tok_verify_codes(logits, codes, u, out, accepted, draft_logits=None, n_draft=None, temperature=1.0, workspace=None,
                     stream=None):
    """Which drafted codes stand, and the code behind them: logits [B, K + 1, V] (float32 or bfloat16), draft_logits
    [B, K, V] or None (each draft was certain), codes [B, K] int32, u [B, K + 1] fp32 in [0, 1), n_draft [B] int32 or
    None (K), temperature a number or fp32 [B] -> out [B, K + 1] int32 (the codes that stand, the drawn one, then -1),
    accepted [B] int32.  Draft i stands if u q(x) < p(x); the code behind is drawn with u[:, K] from max(p - q, 0), or
    from p behind all drafts.  workspace: verify_codes_workspace_size bytes, allocated if None."""
    dev = _device_of(logits, "logits")
    if logits.dim() != 3 or logits.shape[1] < 1 or logits.shape[2] < 1:
        raise ValueError("logits must be [B, K + 1, V] with V >= 1")
    B, rows, V = logits.shape
    K, one, strides = rows - 1, (B,), logits.stride()
    drafted = draft_logits is not None and K > 0
    d = draft_logits.stride() if drafted else (0, 0, 1)
    if V > 1 and (strides[2] != 1 or d[2] != 1):
        raise ValueError("the last dimension of logits and draft_logits must be dense")
    if draft_logits is not None and (draft_logits.get_device() != dev or draft_logits.dtype is not logits.dtype
                                     or draft_logits.shape != (B, K, V)):
        raise ValueError(f"draft_logits must be {(B, K, V)} with the dtype and device of logits")
    if not (_is(codes, _i32, dev, (B, K)) and _is(u, _f32, dev, (B, rows)) and _is(out, _i32, dev, (B, rows))
            and _is(accepted, _i32, dev, one)):
        raise ValueError("codes must be [B, K] int32, u [B, K + 1] float32, out [B, K + 1] and accepted [B] int32, all "
                         "contiguous on the device of logits")
    _need(n_draft, "n_draft", _i32, dev, one)
    ws = _workspace_of((_lib or lib()).tok_verify_codes_workspace_size(B, K, V), workspace, logits, stream,
                       f"no verification for (B, K, V) = {(B, K, V)}: K at most 63, V at most 2^18")
    tp, ta = (None, temperature) if not isinstance(temperature, torch.Tensor) else \
        _setting(temperature, "temperature", _f32, B, logits.device)
    _enqueue("tok_verify_codes", dev, stream, logits.data_ptr(), draft_logits.data_ptr() if drafted else None,
             _dtype_code(logits), codes.data_ptr(), u.data_ptr(), None if n_draft is None else n_draft.data_ptr(), tp, ta,
             out.data_ptr(), accepted.data_ptr(), B, K, V, strides[0], strides[1], d[0], d[1], *_bytes(ws))
    return out, accepted


# ---------------------------------------------------------------------------
# Allocating wrappers.
# ---------------------------------------------------------------------------
def haar_fwd(x: torch.Tensor, stream=None) -> torch.Tensor:
    y = torch.empty(haar_coeff_shape(*x.shape), dtype=x.dtype, device=x.device)
    return tok_haar_fwd(x, y, stream)


def haar_inv(y: torch.Tensor, T: int, H: int, W: int, stream=None) -> torch.Tensor:
    B = y.shape[0]
    C = y.shape[1] // (16 if T == 1 else 64)
    x = torch.empty((B, C, T, H, W), dtype=y.dtype, device=y.device)
    return tok_haar_inv(y, x, stream)


def fsq_encode(u: torch.Tensor, w: torch.Tensor, with_codes: bool = False, stream=None):
    B = u.shape[0]
    idx = torch.empty((B,) + tuple(u.shape[2:]), dtype=torch.int32, device=u.device)
    codes = torch.empty((B, FSQ_DIM) + tuple(u.shape[2:]), dtype=torch.float32, device=u.device) if with_codes else None
    tok_fsq_encode(u, w, idx, codes, stream)
    return (idx, codes) if with_codes else idx


def fsq_decode(idx: torch.Tensor, w: torch.Tensor, bad_count: torch.Tensor = None, stream=None) -> torch.Tensor:
    out = torch.empty((idx.shape[0], w.shape[1]) + tuple(idx.shape[1:]), dtype=torch.float32, device=idx.device)
    return tok_fsq_decode(idx, w, out, bad_count, stream)


def haar_fwd_single(x: torch.Tensor, stream=None) -> torch.Tensor:
    y = torch.empty(single_coeff_shape(*x.shape), dtype=x.dtype, device=x.device)
    return tok_haar_fwd_single(x, y, stream)


def haar_inv_single(y: torch.Tensor, T: int, H: int, W: int, stream=None) -> torch.Tensor:
    x = torch.empty((y.shape[0], y.shape[1] // (4 if T == 1 else 8), T, H, W), dtype=y.dtype, device=y.device)
    return tok_haar_inv_single(y, x, stream)


def haar_fwd_padded(x: torch.Tensor, spatial_multiple: int = 4, temporal_multiple: int = 4,
                    stream=None) -> torch.Tensor:
    y = torch.empty(padded_coeff_shape(*x.shape, spatial_multiple, temporal_multiple), dtype=x.dtype, device=x.device)
    return tok_haar_fwd_padded(x, y, spatial_multiple, temporal_multiple, stream)


def haar_inv_cropped(y: torch.Tensor, T: int, H: int, W: int, spatial_multiple: int = 4, temporal_multiple: int = 4,
                     stream=None) -> torch.Tensor:
    B = y.shape[0]
    C = y.shape[1] // (16 if T == 1 else 64)
    x = torch.empty((B, C, T, H, W), dtype=y.dtype, device=y.device)
    return tok_haar_inv_cropped(y, x, spatial_multiple, temporal_multiple, stream)


def haar_fwd_chunk(x: torch.Tensor, first: bool, stream=None) -> torch.Tensor:
    y = torch.empty(chunk_coeff_shape(*x.shape, first), dtype=x.dtype, device=x.device)
    return tok_haar_fwd_chunk(x, y, first, stream)


def haar_inv_chunk(y: torch.Tensor, T: int, H: int, W: int, first: bool, stream=None) -> torch.Tensor:
    x = torch.empty((y.shape[0], y.shape[1] // 64, T, H, W), dtype=y.dtype, device=y.device)
    return tok_haar_inv_chunk(y, x, first, stream)


def haar_fwd_adjoint(gy: torch.Tensor, T: int, H: int, W: int, stream=None) -> torch.Tensor:
    B = gy.shape[0]
    C = gy.shape[1] // (16 if T == 1 else 64)
    gx = torch.empty((B, C, T, H, W), dtype=gy.dtype, device=gy.device)
    return tok_haar_fwd_adjoint(gy, gx, stream)


def haar_inv_adjoint(gx: torch.Tensor, stream=None) -> torch.Tensor:
    gy = torch.empty(haar_coeff_shape(*gx.shape), dtype=gx.dtype, device=gx.device)
    return tok_haar_inv_adjoint(gx, gy, stream)


def _workspace(B, C, S, device):
    return torch.empty(max(fsq_backward_workspace_size(B, C, S), 1), dtype=torch.uint8, device=device)


def fsq_encode_backward(u: torch.Tensor, w: torch.Tensor, grad_codes: torch.Tensor, stream=None):
    B, C, S = _latent_dims(u)
    grad_u = torch.empty_like(u)
    grad_w = torch.empty_like(w)
    return tok_fsq_encode_backward(u, w, grad_codes, grad_u, grad_w, _workspace(B, C, S, u.device), stream)


def fsq_decode_backward(idx: torch.Tensor, w: torch.Tensor, grad_out: torch.Tensor, stream=None):
    B, C, S = _latent_dims(grad_out)
    grad_codes = torch.empty((B, FSQ_DIM) + tuple(grad_out.shape[2:]), dtype=torch.float32, device=idx.device)
    grad_w = torch.empty_like(w)
    return tok_fsq_decode_backward(idx, w, grad_out, grad_codes, grad_w, _workspace(B, C, S, idx.device), stream)


def _new(like, shape, dtype, stream):
    """A tensor on the device of `like` for work on `stream` (memory that no other stream may still be using)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _dense(x, stream):
    if stream is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(x, memory_format=torch.contiguous_format)


def rope_grid(x, table, sizes, dims, origin=(0, 0, 0), interleaved=False, stream=None) -> torch.Tensor:
    return tok_rope_grid(x, _dense(x, stream), table, sizes, dims, origin, interleaved, stream)


def rope_grid_adjoint(gy, table, sizes, dims, origin=(0, 0, 0), interleaved=False, stream=None) -> torch.Tensor:
    return tok_rope_grid_adjoint(gy, _dense(gy, stream), table, sizes, dims, origin, interleaved, stream)


def rope_positions(x, pos, table, sizes, dims, interleaved=False, bad_count=None, stream=None) -> torch.Tensor:
    return tok_rope_positions(x, _dense(x, stream), pos, table, sizes, dims, interleaved, bad_count, stream)


def rope_positions_adjoint(gy, pos, table, sizes, dims, interleaved=False, bad_count=None,
                           stream=None) -> torch.Tensor:
    return tok_rope_positions_adjoint(gy, _dense(gy, stream), pos, table, sizes, dims, interleaved, bad_count, stream)


def sample_codes(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, with_logprob=False, stream=None):
    """idx, or (idx, logprob): see tok_sample_codes.  idx feeds fsq_decode where V is the FSQ codebook."""
    idx = _new(logits, logits.shape[:-1], torch.int32, stream)
    logprob = _new(logits, logits.shape[:-1], torch.float32, stream) if with_logprob else None
    tok_sample_codes(logits, u, idx, logprob, temperature, top_k, top_p, min_p, stream)
    return (idx, logprob) if with_logprob else idx


def cross_attention(q, k, v, k_lens=None, scale=None, with_lse=False, stream=None):
    """o, or (o, lse): see tok_cross_attention."""
    o = _dense(q, stream)
    lse = _new(q, (q.shape[0], q.shape[2], q.shape[1]), torch.float32, stream) if with_lse else None
    tok_cross_attention(q, k, v, o, lse, k_lens, scale, None, stream)
    return (o, lse) if with_lse else o


def cross_attention_backward(q, k, v, o, lse, grad_o, k_lens=None, scale=None, stream=None):
    """(grad_q, grad_k, grad_v): see tok_cross_attention_backward."""
    return tok_cross_attention_backward(q, k, v, o, lse, grad_o, _dense(q, stream), _dense(k, stream),
                                        _dense(v, stream), k_lens, scale, None, stream)


def embed_codes(codes, table, scale=1.0, bad_count=None, stream=None) -> torch.Tensor:
    """y [..., D]: see tok_embed_codes."""
    y = _new(table, codes.shape + table.shape[1:], table.dtype, stream)
    return tok_embed_codes(codes, table, y, scale, bad_count, stream)


def embed_codes_backward(grad_y, codes, V, scale=1.0, dtype=None, stream=None) -> torch.Tensor:
    """grad_table [V, D] of `dtype` (that of grad_y by default): see tok_embed_codes_backward."""
    grad = _new(grad_y, (V, grad_y.shape[-1]), grad_y.dtype if dtype is None else dtype, stream)
    return tok_embed_codes_backward(grad_y, codes, grad, scale, None, stream)


def page_tables(lens, fresh, n, held, free, pages, table, page_size, bad_count=None, stream=None) -> torch.Tensor:
    """slots [B, n]; held, free and table are updated in place: see tok_page_tables."""
    slots = _new(lens, (lens.shape[0], n), torch.int32, stream)
    return tok_page_tables(lens, fresh, held, free, pages, table, slots, held, free, page_size, bad_count, stream)


def page_release(lens, held, free, pages, table, page_size, bad_count=None, stream=None):
    """held, free, pages and table are updated in place: see tok_page_release."""
    tok_page_release(lens, held, free, pages, table, held, free, page_size, bad_count, stream)


def paged_attention(q, k_pages, v_pages, table, k_lens, q_lens=None, scale=None, with_lse=False, stream=None):
    """o, or (o, lse): see tok_paged_attention."""
    o = _dense(q, stream)
    lse = _new(q, (q.shape[0], q.shape[2], q.shape[1]), torch.float32, stream) if with_lse else None
    tok_paged_attention(q, k_pages, v_pages, table, k_lens, o, lse, q_lens, scale, None, stream)
    return (o, lse) if with_lse else o


def verify_codes(logits, codes, u, draft_logits=None, n_draft=None, temperature=1.0, stream=None):
    """(out, accepted): see tok_verify_codes.  out feeds embed_codes where V is the table's."""
    out = _new(logits, logits.shape[:2], torch.int32, stream)
    accepted = _new(logits, logits.shape[:1], torch.int32, stream)
    return tok_verify_codes(logits, codes, u, out, accepted, draft_logits, n_draft, temperature, None, stream)
