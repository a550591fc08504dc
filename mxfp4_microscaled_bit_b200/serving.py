"""Binding of the serving operators (include/fp4lin_serving.h): the norm in front of a linear
layer with its 8-bit output, products of a few rows with 4-bit weights, and the paged 8-bit KV
cache with its block tables, append and attention.

Argument marshalling only, as in the package: every tensor is checked before its pointer crosses
the C ABI, and nothing falls back to PyTorch.  These calls sit in a decoding loop, where a step of
Python costs as much as the kernel, so the checks ask each tensor only what the call depends on.

Every call takes `stream=` (default: the current stream).  Outputs and workspaces that are not given are
made in the current stream's memory, and a call on another stream then first waits for all that the
current stream has pending; one whose outputs and workspace are all given waits for nothing.

A paged cache is a pair (codes uint8 [num_pages, H, P, D], scales uint8 [num_pages, H]), one for K
and one for V.
"""
from __future__ import annotations

import ctypes

import torch

_i64, _sz, _vp, _int, _f32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SERVING_EXPORTS = {
    "rmsnorm_mxfp8": (_int, [_vp, _i64, _vp, _i64, _vp, _f32, _int, _i64, _i64, _vp, _vp, _vp, _i64, _vp]),
    "nvfp4_matvec": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _i64, _i64, _vp]),
    "mxfp4_matvec": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp, _vp, _vp, _i64, _i64, _vp]),
    "kv_block_tables": (_int, [_vp, _i64, _int, _vp, _vp, _int, _vp, _int, _vp, _int, _int, _vp, _vp, _vp, _vp]),
    "kv_fp8_store": (_int, [_vp, _i64, _vp, _i64, _vp, _int, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _vp]),
    "kv_fp8_attention_workspace_bytes": (_sz, [_int, _int, _int, _int, _i64, _int]),
    "kv_fp8_attention": (_int, [_vp, _i64, _int, _vp, _vp, _vp, _vp, _int, _int, _vp, _i64, _int, _vp, _vp, _int,
                                _i64, _f32, _vp, _int, _int, _int, _int, _vp, _sz, _vp]),
}

_BF16, _U8, _F32, _I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32

try:  # torch.empty on the current CUDA device in a third of the time
    from torch._C._dynamo.guards import _empty_strided_cuda as _empty_strided
except ImportError:
    def _empty_strided(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


_library = None


def _lib():
    global _library
    if _library is None:
        from . import lib
        _library = lib()
    return _library


def _fail(fn: str, status: int):
    from . import Fp4LinError
    raise Fp4LinError(fn, status)


def _refuse(fn: str, name: str, t, dtype, dev: int) -> None:
    """Raise for what _arg and _rows have in common, if that is what is wrong with t."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a torch.Tensor, not {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{fn}: {name} must be {dtype}, not {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor, not on {t.device}")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} is on {t.device}; the library works on the current device cuda:{dev}")


def _arg(fn: str, name: str, t, dtype, count: int, dev: int) -> int:
    """t: a contiguous `dtype` tensor of at least `count` values on device `dev`; its address."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev:
        if t.is_contiguous() and t.numel() >= count:
            return t.data_ptr()
    _refuse(fn, name, t, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous")
    raise ValueError(f"{fn}: {name} holds {t.numel()} values, the call needs {count}")


def _rows(fn: str, name: str, t, dtype, shape: tuple, row: int, dev: int) -> int:
    """t: a `dtype` tensor of this shape whose rows (all dimensions but the first, `row` values) are
    contiguous; its first dimension's stride."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape:
        if t.is_contiguous():
            return row
        stride = t.stride()
        # a row's dimensions of one value may have any stride: those go the long way
        if len(shape) == 2 and stride[1] == 1 or len(shape) == 3 and stride[2] == 1 and stride[1] == shape[2]:
            if stride[0] >= row:
                return stride[0]
    _refuse(fn, name, t, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} must be {list(shape)}, not {list(t.shape)}")
    want = 1
    for n, s in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n > 1 and s != want:
            raise ValueError(f"{fn}: {name} must have contiguous rows (strides {t.stride()})")
        want *= n
    if shape[0] > 1 and t.stride(0) < want:
        raise ValueError(f"{fn}: {name}'s rows overlap (strides {t.stride()})")
    return t.stride(0) if shape[0] > 1 else want


def _device(fn: str, name: str, t) -> int:
    if isinstance(t, torch.Tensor) and t.is_cuda:
        return torch.cuda.current_device()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a torch.Tensor, not {type(t).__name__}")
    raise ValueError(f"{fn}: {name} must be a CUDA tensor, not on {t.device}")


def _raw_stream(stream, dev: int, made=()) -> int:
    """The stream's handle.  made: tensors that this call took from the current stream's memory.  Another
    stream first waits for what that memory may still serve, and it is not given out again before that
    stream is done with it."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)  # current_stream() without making a Stream object
    raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if made and raw != torch._C._cuda_getCurrentRawStream(dev):
        s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(raw, device=dev)
        s.wait_stream(torch.cuda.current_stream(dev))
        for t in made:
            t.record_stream(s)
    return raw


def _scale_bytes(rows: int, cols: int) -> int:
    return (rows + 127) // 128 * 128 * ((cols + 3) // 4 * 4)


# ------------------------------------------------------------------ norm
def _apart(fn, s, ld_s, others, rows, cols):
    """summed [rows, cols] at s is another's memory, or shares none with it (rows may lie between rows: two
    column slices of one buffer)."""
    for name, lo, ld in others:
        if s < lo + ((rows - 1) * ld + cols) * 2 and lo < s + ((rows - 1) * ld_s + cols) * 2:
            if ld_s == ld or rows == 1:
                if s == lo:
                    continue
                # row i of summed begins this many bytes behind row i + n of the other; n = near, near + 1 come closest
                near = (s - lo) // (2 * ld)
                if all(abs(n) >= rows or abs(s - lo - 2 * n * ld) >= 2 * cols for n in (near, near + 1)):
                    continue
            raise ValueError(f"{fn}: summed overlaps {name} without being it")


def rmsnorm_mxfp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
                  hadamard: int = 0, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                  summed: torch.Tensor | None = None, stream=None):
    """RMS norm of bf16 x [rows, cols] (+ residual), rotated when hadamard is 16 or 32, in MXFP8.

    The output is what weight_only_linear takes for up to 16 rows.

    Returns (codes uint8 [rows, cols] of E4M3 bytes, scales uint8 [scale_bytes(rows, cols/32)] of
    E8M0 bytes in the tensor-core layout, s): s = bf16(x + residual), in `summed` if given (which
    may be the residual or x itself, or share no memory with them), or x where there is no residual."""
    fn = "rmsnorm_mxfp8"
    dev = _device(fn, "x", x)
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be 2-D, not {x.dim()}-D")
    rows, cols = x.shape
    ld_x = _rows(fn, "x", x, _BF16, (rows, cols), cols, dev)
    w = _arg(fn, "weight", weight, _BF16, cols, dev)
    r = s = None
    ld_r = ld_s = cols
    made = []
    if residual is not None:
        ld_r = _rows(fn, "residual", residual, _BF16, (rows, cols), cols, dev)
        r = residual.data_ptr()
        if summed is None:
            summed = _empty_strided((rows, cols), (cols, 1), _BF16)
            made.append(summed)
        else:
            ld_s = _rows(fn, "summed", summed, _BF16, (rows, cols), cols, dev)
            _apart(fn, summed.data_ptr(), ld_s, (("residual", r, ld_r), ("x", x.data_ptr(), ld_x)), rows, cols)
        s = summed.data_ptr()
    elif summed is not None:
        raise ValueError(f"{fn}: summed is the sum with a residual, and there is none")
    if codes is None:
        codes = _empty_strided((rows, cols), (cols, 1), _U8)
        made.append(codes)
    else:
        _arg(fn, "codes", codes, _U8, rows * cols, dev)
    need = _scale_bytes(rows, cols // 32)
    if scales is None:
        scales = _empty_strided((need,), (1,), _U8)
        made.append(scales)
    else:
        _arg(fn, "scales", scales, _U8, need, dev)
    st = _lib().rmsnorm_mxfp8(x.data_ptr(), ld_x, r, ld_r, w, eps, hadamard, rows, cols, codes.data_ptr(),
                              scales.data_ptr(), s, ld_s, _raw_stream(stream, dev, made))
    if st:
        _fail(fn, st)
    return codes, scales, x if residual is None else summed


# ------------------------------------------------------------------ matvec
def _matvec(fn, nv, x, w_codes, w_scales, g_w, x_scales, hadamard, out, stream):
    dev = _device(fn, "x", x)
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be 2-D, not {x.dim()}-D")
    M, K = x.shape
    ld_x = _rows(fn, "x", x, _BF16 if x_scales is None else _U8, (M, K), K, dev)
    xs = None if x_scales is None else _arg(fn, "x_scales", x_scales, _U8, _scale_bytes(M, K // 32), dev)
    if not isinstance(w_codes, torch.Tensor) or w_codes.dim() != 2:
        raise ValueError(f"{fn}: w_codes must be a 2-D codes tensor [N, K/2]")
    N = w_codes.shape[0]
    if w_codes.shape[1] * 2 != K:
        raise ValueError(f"{fn}: w_codes holds {w_codes.shape[1] * 2} values a row, x {K}")
    w = _arg(fn, "w_codes", w_codes, _U8, 0, dev)
    ws = _arg(fn, "w_scales", w_scales, _U8, _scale_bytes(N, K // (16 if nv else 32)), dev)
    ldy = N
    made = ()
    if out is None:
        out = _empty_strided((M, N), (N, 1), _BF16)
        made = (out,)
    else:
        ldy = _rows(fn, "out", out, _BF16, (M, N), N, dev)
    if nv:
        st = _lib().nvfp4_matvec(x.data_ptr(), xs, M, K, ld_x, hadamard, w, ws, _arg(fn, "g_w", g_w, _F32, 1, dev),
                                 out.data_ptr(), N, ldy, _raw_stream(stream, dev, made))
    else:
        st = _lib().mxfp4_matvec(x.data_ptr(), xs, M, K, ld_x, hadamard, w, ws, out.data_ptr(), N, ldy,
                                 _raw_stream(stream, dev, made))
    if st:
        _fail(fn, st)
    return out


def nvfp4_matvec(x, w_codes, w_scales, g_w, *, x_scales=None, hadamard: int = 0, out=None, stream=None):
    """y [M, N] bf16 = x W^T for NVFP4 weights and M <= 16 rows of x: bf16 [M, K] (rotated on the
    way in when hadamard = 16), or MXFP8 codes uint8 [M, K] with x_scales (rmsnorm_mxfp8).  out must
    not overlap the inputs."""
    return _matvec("nvfp4_matvec", True, x, w_codes, w_scales, g_w, x_scales, hadamard, out, stream)


def mxfp4_matvec(x, w_codes, w_scales, *, x_scales=None, hadamard: int = 0, out=None, stream=None):
    """nvfp4_matvec for MXFP4 weights (hadamard = 32)."""
    return _matvec("mxfp4_matvec", False, x, w_codes, w_scales, None, x_scales, hadamard, out, stream)


def weight_only_linear(x, weight, *, x_scales=None, out=None, stream=None):
    """y = x W^T for a prepared weight (prepare_weight, prepare_weight_gptq) and M <= 16 rows whose
    activations stay in 16 bits, or in the 8 bits of rmsnorm_mxfp8 (which must have rotated them by
    weight.hadamard).  More rows are refused: their products are the W4A4 ones, nvfp4_linear and
    mxfp4_linear, of bf16 activations."""
    had = weight.hadamard if x_scales is None else 0
    if weight.fmt == "nvfp4":
        return nvfp4_matvec(x, weight.codes, weight.scales, weight.g, x_scales=x_scales, hadamard=had, out=out,
                            stream=stream)
    return mxfp4_matvec(x, weight.codes, weight.scales, x_scales=x_scales, hadamard=had, out=out, stream=stream)


# ------------------------------------------------------------------ paged KV cache
def kv_block_tables(block_table, lens, new_lens, free_pages, free_head, page: int, *, max_tokens: int, cu_new=None,
                    slots=None, next_head=None, stream=None):
    """Pages for new tokens and the slot of each, from request lengths on the device.

    block_table int32 [B, width] (rows contiguous) is updated in place; lens, new_lens int32 [B];
    free_pages int32 [F], taken from index free_head[0] on; max_tokens: the slots to write, at
    least the new tokens' sum.  Returns (cu_new int32 [B + 1], slots int32 [max_tokens] with -1
    behind the last token, next_head int32 [1])."""
    fn = "kv_block_tables"
    dev = _device(fn, "block_table", block_table)
    if block_table.dim() != 2:
        raise ValueError(f"{fn}: block_table must be 2-D, not {block_table.dim()}-D")
    B, width = block_table.shape
    ld = _rows(fn, "block_table", block_table, _I32, (B, width), width, dev)
    pl = _arg(fn, "lens", lens, _I32, B, dev)
    pn = _arg(fn, "new_lens", new_lens, _I32, B, dev)
    pf = _arg(fn, "free_pages", free_pages, _I32, 1, dev)
    ph = _arg(fn, "free_head", free_head, _I32, 1, dev)
    made = []
    if not 1 <= max_tokens < 2 ** 31:
        raise ValueError(f"{fn}: max_tokens must be at least 1 and below 2^31, not {max_tokens}")
    if cu_new is None:
        cu_new = _empty_strided((B + 1,), (1,), _I32)
        made.append(cu_new)
    else:
        _arg(fn, "cu_new", cu_new, _I32, B + 1, dev)
    if slots is None:
        slots = _empty_strided((max_tokens,), (1,), _I32)
        made.append(slots)
    else:
        _arg(fn, "slots", slots, _I32, max_tokens, dev)
    if next_head is None:
        next_head = _empty_strided((1,), (1,), _I32)
        made.append(next_head)
    else:
        _arg(fn, "next_head", next_head, _I32, 1, dev)
    st = _lib().kv_block_tables(block_table.data_ptr(), ld, width, pl, pn, B, pf, free_pages.numel(), ph, page,
                                max_tokens, cu_new.data_ptr(), slots.data_ptr(), next_head.data_ptr(),
                                _raw_stream(stream, dev, made))
    if st:
        _fail(fn, st)
    return cu_new, slots, next_head


def _paged(fn, side, cache, dev):
    """Addresses and shape of a paged cache (codes [num_pages, H, P, D], scales [num_pages, H])."""
    if not isinstance(cache, (tuple, list)) or len(cache) != 2:
        raise TypeError(f"{fn}: {side}_cache must be a pair (codes, scales)")
    codes, scales = cache
    if not isinstance(codes, torch.Tensor) or codes.dim() != 4:
        raise ValueError(f"{fn}: {side}_cache's codes must be [num_pages, H, P, D]")
    shape = codes.shape
    pc = _arg(fn, f"{side}_cache's codes", codes, _U8, 0, dev)
    ps = _arg(fn, f"{side}_cache's scales", scales, _U8, shape[0] * shape[1], dev)
    return pc, ps, shape


def kv_fp8_store(k_new, v_new, slots, k_cache, v_cache, *, stream=None) -> None:
    """Append k_new and v_new (bf16 [T, H, D], a token's heads contiguous) to the paged caches at
    slots int32 [T] (kv_block_tables; -1: skipped)."""
    fn = "kv_fp8_store"
    dev = _device(fn, "k_new", k_new)
    kc, ks, shape = _paged(fn, "k", k_cache, dev)
    vc, vs, vshape = _paged(fn, "v", v_cache, dev)
    if shape != vshape:
        raise ValueError(f"{fn}: the K and V caches must have the same shape")
    NP, H, P, D = shape
    T = slots.shape[0] if isinstance(slots, torch.Tensor) and slots.dim() == 1 else -1
    if T < 1:
        raise ValueError(f"{fn}: slots must be a 1-D tensor of at least one slot")
    ps = _arg(fn, "slots", slots, _I32, T, dev)
    ld_k = _rows(fn, "k_new", k_new, _BF16, (T, H, D), H * D, dev)
    ld_v = _rows(fn, "v_new", v_new, _BF16, (T, H, D), H * D, dev)
    st = _lib().kv_fp8_store(k_new.data_ptr(), ld_k, v_new.data_ptr(), ld_v, ps, T, kc, ks, vc, vs, NP, H, P, D,
                             _raw_stream(stream, dev))
    if st:
        _fail(fn, st)


def kv_fp8_attention(q, k_cache, v_cache, block_table, lens, cu_new, *, max_new: int, max_len: int,
                     scale: float | None = None, out=None, workspace=None, stream=None):
    """Causal attention of a step's new tokens over the paged caches (their rows stored already).

    q bf16 [T, HQ, D] (a token's heads contiguous), HQ a multiple of the cache's H; block_table
    int32 [B, width]; lens int32 [B], rows before the step; cu_new int32 [B + 1] (kv_block_tables);
    max_new, max_len: bounds that the host knows on a request's new tokens and on lens + new.
    scale defaults to D ** -0.5.  Returns out, bf16 [T, HQ, D]; rows of no request are not written."""
    fn = "kv_fp8_attention"
    dev = _device(fn, "q", q)
    kc, ks, shape = _paged(fn, "k", k_cache, dev)
    vc, vs, vshape = _paged(fn, "v", v_cache, dev)
    if shape != vshape:
        raise ValueError(f"{fn}: the K and V caches must have the same shape")
    NP, H, P, D = shape
    if q.dim() != 3 or H < 1 or q.shape[1] % H or q.shape[2] != D:
        raise ValueError(f"{fn}: q must be [T, a multiple of {H} heads, {D}], not {list(q.shape)}")
    T, HQ = q.shape[0], q.shape[1]
    ld_q = _rows(fn, "q", q, _BF16, (T, HQ, D), HQ * D, dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError(f"{fn}: block_table must be a 2-D tensor")
    B, width = block_table.shape
    ld_t = _rows(fn, "block_table", block_table, _I32, (B, width), width, dev)
    pl = _arg(fn, "lens", lens, _I32, B, dev)
    pcu = _arg(fn, "cu_new", cu_new, _I32, B + 1, dev)
    made = []
    if out is None:
        out = _empty_strided((T, HQ, D), (HQ * D, D, 1), _BF16)
        made.append(out)
    else:
        _arg(fn, "out", out, _BF16, T * HQ * D, dev)
    if not (1 <= max_new < 2 ** 31 and 1 <= max_len < 2 ** 31):
        raise ValueError(f"{fn}: max_new and max_len must be at least 1 and below 2^31, not {max_new} and {max_len}")
    L, G = _lib(), HQ // H
    if workspace is None:
        need = L.kv_fp8_attention_workspace_bytes(B, H, G, max_new, max_len, D)
        pw = None
        if need:
            workspace = _empty_strided((need,), (1,), _U8)
            made.append(workspace)
            pw = workspace.data_ptr()
    else:
        pw, need = _arg(fn, "workspace", workspace, getattr(workspace, "dtype", None), 0, dev), workspace.numel() * workspace.element_size()
    st = L.kv_fp8_attention(q.data_ptr(), ld_q, T, kc, ks, vc, vs, NP, P, block_table.data_ptr(), ld_t, width, pl, pcu,
                            max_new, max_len, D ** -0.5 if scale is None else scale, out.data_ptr(), B, H, G, D, pw,
                            need, _raw_stream(stream, dev, made))
    if st:
        _fail(fn, st)
    return out
