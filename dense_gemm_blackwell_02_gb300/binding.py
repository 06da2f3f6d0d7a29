"""ctypes binding of libgemm.so (include/gemm.h): argument marshalling only.

Every step of the GEMM runs inside the library's CUDA kernels; this module
passes pointers, sizes, dtype codes and the caller's CUDA stream.  If the
library is missing it raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import struct

F16, BF16, F32, E4M3, E5M2 = 0, 1, 2, 3, 4
STATUS_NAMES = {0: "GEMM_OK", 1: "GEMM_ERR_INVALID_ARG", 2: "GEMM_ERR_UNSUPPORTED",
                3: "GEMM_ERR_CUDA", 4: "GEMM_ERR_OOM", 5: "GEMM_ERR_TIMEOUT",
                6: "GEMM_ERR_BAD_INDEX"}
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgemm.so")

# Every function include/gemm.h declares (checked against the header by the tests).
EXPORTS = ("gemm_run_adapters_packed", "gemm_rotary_packed", "gemm_adjust_logits_packed",
           "gemm_create", "gemm_destroy", "gemm_run", "gemm_run_epilogue", "gemm_run_blockwise",
           "gemm_run_grouped", "gemm_run_host",
           "gemm_set_config",
           "gemm_last_config", "gemm_device_status", "gemm_set_wait_limit",
           "gemm_set_test_stall", "gemm_sm_count", "gemm_status_string", "gemm_run_noalloc",
           "gemm_last_cuda_error", "gemm_plan",
           "gemm_run_adapters", "gemm_rotary", "gemm_adjust_logits")


class GemmConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("variant", "block_n", "splits", "stages",
                                                "group_m", "max_ctas", "chain_kblocks",
                                                "dp_tiles", "prefetch_kblocks", "epilogue",
                                                "l2_hint", "swap_ab", "swap_rows", "scheduler")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


ACT_NONE, ACT_RELU = 0, 1


class GemmEpilogue(ctypes.Structure):
    """gemm_epilogue_t: C = act(alpha * A . B^T + beta * C_prev + bias)."""
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("bias", ctypes.c_void_p),
                ("activation", ctypes.c_int32)]


class GemmBlockScales(ctypes.Structure):
    """gemm_block_scales_t: FP8 block scales, sfa per (block_m rows, 128 of K) of A and
    sfb per (128 rows, 128 of K) of B."""
    _fields_ = [("sfa", ctypes.c_void_p), ("sfb", ctypes.c_void_p), ("block_m", ctypes.c_int32),
                ("block_n", ctypes.c_int32)]


class GemmAdapters(ctypes.Structure):
    """gemm_adapters_t: a pool of low-rank adapters, down count x rank x K and up
    count x N x rank, with a factor for each."""
    _fields_ = [("down", ctypes.c_void_p), ("up", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("count", ctypes.c_int32), ("rank", ctypes.c_int32)]


PAIRS_HALF, PAIRS_NEIGHBOURS = 0, 1


class GemmRotary(ctypes.Structure):
    """gemm_rotary_t: the tables, the tokens' positions along every axis, and which axis
    turns which pair."""
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("pair_axis", ctypes.c_char_p),
                ("num_positions", ctypes.c_int64), ("axes", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("pairs", ctypes.c_int32),
                ("inverse", ctypes.c_int32)]


class GemmLogits(ctypes.Structure):
    """gemm_logits_t: histories and penalties, biases and masks of a batch of rows."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("tokens", "token_start", "prompt_len", "repetition",
                                                "frequency", "presence", "bias_tokens",
                                                "bias_values", "bias_start", "mask")]
                + [("mask_stride", ctypes.c_int64), ("mask_count", ctypes.c_int64),
                   ("mask_row", ctypes.c_void_p)])


class GemmProblem(ctypes.Structure):
    """gemm_problem_t: one problem of a grouped launch, C = A . B^T."""
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class GemmError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{STATUS_NAMES.get(code, code)}{': ' + what if what else ''}")


class GemmDeviceModel(ctypes.Structure):
    """gemm_device_model_t: a GPU described for gemm_plan (SMs, resident CTA pairs,
    resident clusters of four CTAs)."""
    _fields_ = [("sms", ctypes.c_int32), ("pairs", ctypes.c_int32), ("clusters4", ctypes.c_int32)]


GB300_MODEL = (152, 76, 36)  # a full GB300: 152 SMs, 76 pairs, 36 clusters of four


def plan(M, N, K, dtype_in=F16, dtype_out=F16, fused=False, blockwise=False, config=None,
         device=GB300_MODEL) -> dict:
    """The configuration the library would launch for this product on the described
    device (gemm_plan): the host's decisions only, no GPU needed.  Raises GemmError with
    the call's status when it refuses."""
    cfg = None
    if config:
        cfg = GemmConfig(**{**{n: 0 for n, _ in GemmConfig._fields_}, **config})
    dev = GemmDeviceModel(*device)
    out = GemmConfig()
    _check(lib().gemm_plan(ctypes.byref(dev), ctypes.byref(cfg) if cfg is not None else None,
                           M, N, K, dtype_in, dtype_out, 1 if fused else 0,
                           1 if blockwise else 0, ctypes.byref(out)), "gemm_plan")
    return out.as_dict()


_lib = None


def lib():
    """Load libgemm.so (built in-tree) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run "
                           "`python -m dense_gemm_blackwell_02_gb300.build` first")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, u32, u64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32,
                              ctypes.c_uint64)
    L.gemm_create.argtypes = [ctypes.POINTER(vp)]
    L.gemm_destroy.argtypes = [vp]
    L.gemm_run.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
    L.gemm_run_host.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
    L.gemm_set_config.argtypes = [vp, ctypes.POINTER(GemmConfig)]
    L.gemm_last_config.argtypes = [vp, ctypes.POINTER(GemmConfig)]
    L.gemm_device_status.argtypes = [vp, vp, ctypes.POINTER(u32)]
    L.gemm_set_wait_limit.argtypes = [vp, u64]
    L.gemm_set_test_stall.argtypes = [vp, i32]
    L.gemm_sm_count.argtypes = [vp]
    L.gemm_sm_count.restype = i32
    L.gemm_run_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, i32, i32, vp]
    L.gemm_run_epilogue.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32,
                                    ctypes.POINTER(GemmEpilogue), vp]
    L.gemm_run_blockwise.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32,
                                     ctypes.POINTER(GemmBlockScales), vp]
    L.gemm_run_grouped.argtypes = [vp, ctypes.POINTER(GemmProblem), i32, i32, i32, vp]
    L.gemm_run_adapters.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32,
                                    ctypes.POINTER(GemmAdapters), vp, vp]
    L.gemm_rotary.argtypes = [vp, vp, vp] + [i64] * 7 + [i32, ctypes.POINTER(GemmRotary), vp]
    L.gemm_adjust_logits.argtypes = [vp, vp, vp] + [i64] * 4 + [i32, i32,
                                                                ctypes.POINTER(GemmLogits), vp]
    for name in ("gemm_run_adapters_packed", "gemm_rotary_packed", "gemm_adjust_logits_packed"):
        getattr(L, name).argtypes = [ctypes.c_char_p]
    L.gemm_status_string.argtypes = [i32]
    L.gemm_status_string.restype = ctypes.c_char_p
    L.gemm_plan.argtypes = [ctypes.POINTER(GemmDeviceModel), ctypes.POINTER(GemmConfig), i64, i64,
                            i64, i32, i32, i32, i32, ctypes.POINTER(GemmConfig)]
    L.gemm_last_cuda_error.argtypes = [vp]
    L.gemm_last_cuda_error.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name not in ("gemm_sm_count", "gemm_status_string", "gemm_last_cuda_error"):
            getattr(L, name).restype = i32
    _lib = L
    return L


def _check(code: int, what: str = "", h=None):
    if code != 0:
        if code == 3 and h is not None:  # GEMM_ERR_CUDA: name the CUDA error behind it
            detail = lib().gemm_last_cuda_error(h).decode()
            if detail:
                what = f"{what} ({detail})" if what else detail
        raise GemmError(code, what)


def torch_float32():
    import torch
    return torch.float32


_torch = None        # torch, and its dtypes' codes: set when the first handle is made
_DTYPE_CODE = None


def _use_torch():
    global _torch, _DTYPE_CODE
    if _torch is None:
        import torch
        _torch = torch
        _DTYPE_CODE = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32,
                       torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}


def torch_dtype_code(dt) -> int:
    _use_torch()
    return _DTYPE_CODE[dt]


def _need(t, name, dtype, shape, index):
    """Check an auxiliary tensor on CUDA device `index` and give its address (0 for None)."""
    if t is None:
        return 0
    if (t.get_device() != index or t.dtype is not dtype or not t.is_contiguous()
            or (shape is not None and t.shape != shape)):
        want = "" if shape is None else f" of shape {tuple(shape)}"
        raise ValueError(f"{name} must be a contiguous {dtype} tensor{want} on cuda:{index}")
    return t.data_ptr()


def _vec(t, name, dtype, n, index):
    """_need for a vector of n values; 0 for None."""
    if t is None:
        return 0
    if (t.dtype is not dtype or t.shape != (n,) or t.get_device() != index
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape ({n},) on cuda:{index}")
    return t.data_ptr()


# The blocks of the packed calls (gemm_adapters_call_t, gemm_rotary_call_t,
# gemm_logits_call_t).  A block costs a microsecond; a dozen arguments through ctypes and a
# structure, three.
_ADAPTERS_CALL = struct.Struct("PPPPqqqPPiiPPPii")
_ROTARY_CALL = struct.Struct("PPPqqqqqqqP" "PPPPqiiii" "ii")
_LOGITS_CALL = struct.Struct("PPPqqqqPii" "PPPPPPPPPPqqP")


def pair_axes(sections, interleaved=False):
    """The axis that turns each rotary pair, from the number of pairs of every axis: axis
    after axis ([2, 1] -> 0 0 1), or dealt out in turn until an axis has its pairs
    (interleaved; [2, 1] -> 0 1 0)."""
    left = [int(n) for n in sections]
    if not left or min(left) < 0:
        raise ValueError("sections must be numbers of pairs, one for each axis")
    if not interleaved:
        return [a for a, n in enumerate(left) for _ in range(n)]
    axes = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                left[a] -= 1
                axes.append(a)
    return axes


def _stream_ptr(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_of(stream, index):
    """_stream_ptr for a CUDA device given by its index, by the raw handle (a Stream object
    around it costs 2 us of a 20 us call)."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Gemm:
    """One library handle (workspace, status word, tensor-map cache)."""

    def __init__(self):
        _use_torch()
        h = ctypes.c_void_p()
        _check(lib().gemm_create(ctypes.byref(h)), "gemm_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            lib().gemm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def sm_count(self) -> int:
        return lib().gemm_sm_count(self._h)

    # ------------------------------------------------------------ raw pointers --
    def run_ptr(self, a_ptr, b_ptr, c_ptr, M, N, K, dtype_in, dtype_out, stream_ptr=0) -> int:
        """gemm_run on raw device pointers; returns the status code."""
        return lib().gemm_run(self._h, a_ptr, b_ptr, c_ptr, M, N, K, dtype_in, dtype_out,
                              stream_ptr)

    # ----------------------------------------------------------- torch tensors --
    def run(self, A, B, C, stream=None):
        """C = A @ B.T for CUDA tensors A (M,K), B (N,K), C (M,N), all contiguous."""
        if not (A.is_cuda and B.is_cuda and C.is_cuda):
            raise ValueError("A, B and C must be CUDA tensors")
        if not (A.is_contiguous() and B.is_contiguous() and C.is_contiguous()):
            raise ValueError("A, B and C must be contiguous (row-major, K-major operands)")
        if A.dim() != 2 or B.dim() != 2 or C.dim() != 2:
            raise ValueError("A, B and C must be 2-D")
        M, K = A.shape
        N, K2 = B.shape
        if K != K2 or tuple(C.shape) != (M, N):
            raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, "
                             f"C {tuple(C.shape)}")
        if A.dtype != B.dtype:
            raise ValueError("A and B must share a dtype")
        code = self.run_ptr(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                            torch_dtype_code(A.dtype), torch_dtype_code(C.dtype),
                            _stream_ptr(stream, A.device))
        _check(code, f"gemm_run M={M} N={N} K={K}", self._h)
        return C

    def run_epilogue(self, A, B, C, alpha=1.0, beta=0.0, bias=None, relu=False, stream=None):
        """C = act(alpha * A @ B.T + beta * C + bias) in the GEMM's epilogue: bias a CUDA
        float32 tensor of N values (or None), act ReLU when relu."""
        M, K = A.shape
        N = B.shape[0]
        if bias is not None:
            if not (bias.is_cuda and bias.dtype == torch_float32() and bias.is_contiguous()
                    and bias.numel() == N):
                raise ValueError("bias must be a contiguous float32 CUDA tensor of N values")
        if not (A.is_cuda and B.is_cuda and C.is_cuda and A.is_contiguous() and B.is_contiguous()
                and C.is_contiguous() and B.shape[1] == K and tuple(C.shape) == (M, N)
                and A.dtype == B.dtype):
            raise ValueError("A (M,K), B (N,K), C (M,N): contiguous CUDA tensors, A and B of one dtype")
        epi = GemmEpilogue(float(alpha), float(beta), None if bias is None else bias.data_ptr(),
                           ACT_RELU if relu else ACT_NONE)
        code = lib().gemm_run_epilogue(self._h, A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                                       torch_dtype_code(A.dtype), torch_dtype_code(C.dtype),
                                       ctypes.byref(epi), _stream_ptr(stream, A.device))
        _check(code, f"gemm_run_epilogue M={M} N={N} K={K}", self._h)
        return C

    def run_blockwise(self, A, B, C, sfa, sfb, block_m, block_n=128, stream=None):
        """C = sum_kb sfa[kb, i // block_m] * sfb[kb, j // block_n] * (A @ B.T over the kb-th
        128 columns of K), A and B FP8 CUDA tensors; sfa and sfb contiguous float32 CUDA
        tensors stored K-block-major, ceil(K / 128) x ceil(M / block_m) and
        ceil(K / 128) x ceil(N / block_n)."""
        M, K = A.shape
        N = B.shape[0]
        nkb = -(-K // 128)
        for t, rows, name in ((sfa, -(-M // max(block_m, 1)), "sfa"), (sfb, -(-N // max(block_n, 1)), "sfb")):
            if not (t.is_cuda and t.dtype == torch_float32() and t.is_contiguous()
                    and tuple(t.shape) == (nkb, rows)):
                raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of {nkb} x {rows}")
        if not (A.is_cuda and B.is_cuda and C.is_cuda and A.is_contiguous() and B.is_contiguous()
                and C.is_contiguous() and B.shape[1] == K and tuple(C.shape) == (M, N)
                and A.dtype == B.dtype):
            raise ValueError("A (M,K), B (N,K), C (M,N): contiguous CUDA tensors, A and B of one dtype")
        sc = GemmBlockScales(sfa.data_ptr(), sfb.data_ptr(), int(block_m), int(block_n))
        code = lib().gemm_run_blockwise(self._h, A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                                        torch_dtype_code(A.dtype), torch_dtype_code(C.dtype),
                                        ctypes.byref(sc), _stream_ptr(stream, A.device))
        _check(code, f"gemm_run_blockwise M={M} N={N} K={K}", self._h)
        return C

    def run_grouped(self, problems, stream=None):
        """C_g = A_g @ B_g.T for every (A_g, B_g, C_g) in `problems`, in one launch: CUDA
        tensors, contiguous, one input dtype and one output dtype for all."""
        if not problems:
            return
        din, dout = problems[0][0].dtype, problems[0][2].dtype
        arr = (GemmProblem * len(problems))()
        for i, (A, B, C) in enumerate(problems):
            M, K = A.shape
            N = B.shape[0]
            if not (A.is_cuda and B.is_cuda and C.is_cuda and A.is_contiguous()
                    and B.is_contiguous() and C.is_contiguous() and B.shape[1] == K
                    and tuple(C.shape) == (M, N) and A.dtype == din and B.dtype == din
                    and C.dtype == dout):
                raise ValueError(f"problem {i}: A (M,K), B (N,K), C (M,N) contiguous CUDA tensors "
                                 "with the group's dtypes")
            arr[i] = GemmProblem(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K)
        code = lib().gemm_run_grouped(self._h, arr, len(problems), torch_dtype_code(din),
                                      torch_dtype_code(dout),
                                      _stream_ptr(stream, problems[0][0].device))
        _check(code, f"gemm_run_grouped count={len(problems)}", self._h)

    # ------------------------------------------ operators around the projections --
    def run_adapters(self, X, W, Y, down, up, row_adapter, scale=None, stream=None):
        """Y[i] = W @ X[i] + scale[a] * up[a] @ (down[a] @ X[i]) with a = row_adapter[i]
        (no second term where a is negative): CUDA tensors X (M,K), W (N,K), Y (M,N), down
        (adapters, rank, K), up (adapters, N, rank) of X's dtype, row_adapter int32 (M),
        scale float32 (adapters) or None; all contiguous."""
        if not X.is_cuda:
            raise ValueError("X must be a CUDA tensor")
        if X.dim() != 2 or W.dim() != 2 or down.dim() != 3:
            raise ValueError("X and W must be 2-D, down and up 3-D")
        M, K = X.shape
        N = W.shape[0]
        count, rank, _ = down.shape
        dev, dt, out = X.get_device(), X.dtype, Y.dtype
        code = _lib.gemm_run_adapters_packed(_ADAPTERS_CALL.pack(
            self._h.value or 0, _need(X, "X", dt, None, dev), _need(W, "W", dt, (N, K), dev),
            _need(Y, "Y", out, (M, N), dev), M, N, K,
            _vec(row_adapter, "row_adapter", _torch.int32, M, dev), _stream_of(stream, dev),
            _DTYPE_CODE[dt], _DTYPE_CODE[out], _need(down, "down", dt, (count, rank, K), dev),
            _need(up, "up", dt, (count, N, rank), dev),
            _vec(scale, "scale", _torch.float32, count, dev), count, rank))
        if code:
            _check(code, f"gemm_run_adapters M={M} N={N} K={K} rank={rank}", self._h)
        return Y

    def rotary(self, x, y, cos, sin, positions, pair_axis=None, neighbours=False, inverse=False,
               stream=None):
        """Turn the pairs of every head by their tokens' positions: CUDA tensors x and y
        (tokens, heads, dim) of one dtype, values of a head contiguous, any other strides,
        y possibly x; cos and sin float32 (positions, pairs); positions int32 (axes, tokens)
        or (tokens,); pair_axis the axis of every pair (see pair_axes; None: the first).
        Pairs are (i, i + pairs), or neighbouring values.  inverse turns back (the
        gradient)."""
        dev, dt = x.get_device(), x.dtype
        if not (x.is_cuda and y.get_device() == dev and y.dtype is dt and x.dim() == 3
                and y.shape == x.shape):
            raise ValueError("x and y must be CUDA tensors (tokens, heads, dim) of one device and dtype")
        T, H, D = x.shape
        xt, xh, xd = x.stride()
        yt, yh, yd = y.stride()
        if D > 1 and (xd != 1 or yd != 1):
            raise ValueError("the values of a head must be contiguous")
        if positions.dim() == 1:
            positions = positions[None]
        if cos.dim() != 2 or positions.dim() != 2:
            raise ValueError("cos and sin must be (positions, pairs), positions (axes, tokens)")
        P, half = cos.shape
        axes = positions.shape[0]
        follow = b""
        if pair_axis is not None:
            if len(pair_axis) != half:
                raise ValueError(f"pair_axis must name an axis for each of the {half} pairs")
            follow = bytes(pair_axis)
        f32 = _torch.float32
        code = _lib.gemm_rotary_packed(_ROTARY_CALL.pack(
            self._h.value or 0, x.data_ptr(), y.data_ptr(), T, H, D, xt, xh, yt, yh,
            _stream_of(stream, dev), _need(cos, "cos", f32, None, dev),
            _need(sin, "sin", f32, (P, half), dev),
            _need(positions, "positions", _torch.int32, (axes, T), dev), 0, P, axes, 2 * half,
            PAIRS_NEIGHBOURS if neighbours else PAIRS_HALF, 1 if inverse else 0, _DTYPE_CODE[dt],
            1 if follow else 0) + follow)
        if code:
            if follow and max(follow) >= axes:
                raise ValueError(f"pair_axis must hold axes below {axes}")
            _check(code, f"gemm_rotary tokens={T} heads={H} dim={D}", self._h)
        return y

    def adjust_logits(self, logits, out, tokens=None, token_start=None, prompt_len=None,
                      repetition=None, frequency=None, presence=None, bias_tokens=None,
                      bias_values=None, bias_start=None, mask=None, mask_row=None, stream=None):
        """Penalties for repeated tokens, biases and grammar masks (gemm_adjust_logits):
        CUDA tensors logits and out (rows, vocab), rows of any stride, out possibly logits.
        tokens (int32) and token_start (int64, rows + 1) are the rows' histories, the first
        prompt_len (int32) of each the prompt; repetition, frequency and presence float32
        (rows); bias_tokens (int32, fastest when ascending within a row), bias_values
        (float32) and bias_start (int64, rows + 1) the biases; mask int32 (masks, words) with bit
        v % 32 of word v // 32 set where token v may follow, mask_row int32 (rows),
        negative for no mask, or None for one mask per row."""
        dev = logits.get_device()
        if not (logits.is_cuda and out.get_device() == dev and logits.dim() == 2
                and out.shape == logits.shape):
            raise ValueError("logits and out must be CUDA tensors (rows, vocab) of one device")
        B, V = logits.shape
        sl, cl = logits.stride()
        so, co = out.stride()
        if V > 1 and (cl != 1 or co != 1):
            raise ValueError("the logits of a row must be contiguous")
        if B > 1 and (sl < V or so < V):
            raise ValueError("rows must not overlap")
        if B == 1:  # a single row's stride says nothing
            sl = so = V
        f32, i32, i64 = _torch.float32, _torch.int32, _torch.int64
        masks = words = 0
        if mask is not None:
            if mask.dim() != 2:
                raise ValueError("mask must be (masks, words)")
            masks, words = mask.shape
            # (an empty tensor has no address, which would say that there are no masks)
            if masks * words == 0 and B and V:
                raise ValueError("mask holds no mask")
        code = _lib.gemm_adjust_logits_packed(_LOGITS_CALL.pack(
            self._h.value or 0, logits.data_ptr(), out.data_ptr(), B, V, sl, so,
            _stream_of(stream, dev), _DTYPE_CODE[logits.dtype], _DTYPE_CODE[out.dtype],
            _need(tokens, "tokens", i32, None, dev),
            _vec(token_start, "token_start", i64, B + 1, dev),
            _vec(prompt_len, "prompt_len", i32, B, dev),
            _vec(repetition, "repetition", f32, B, dev),
            _vec(frequency, "frequency", f32, B, dev),
            _vec(presence, "presence", f32, B, dev),
            _need(bias_tokens, "bias_tokens", i32, None, dev),
            _need(bias_values, "bias_values", f32,
                  None if bias_tokens is None else bias_tokens.shape, dev),
            _vec(bias_start, "bias_start", i64, B + 1, dev),
            _need(mask, "mask", i32, None, dev), words, masks,
            _vec(mask_row, "mask_row", i32, B, dev)))
        if code:
            _check(code, f"gemm_adjust_logits rows={B} vocab={V}", self._h)
        return out

    def run_host(self, A, B, C, dtype_in, dtype_out, stream=None):
        """gemm_run_host on CPU tensors (pinned for asynchronous copies)."""
        M, K = A.shape
        N = B.shape[0]
        sp = 0 if stream is None else _stream_ptr(stream, None)
        code = lib().gemm_run_host(self._h, A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                                   dtype_in, dtype_out, sp)
        _check(code, "gemm_run_host", self._h)
        return C

    # ----------------------------------------------------------------- control --
    def set_config(self, variant=0, block_n=0, splits=0, stages=0, group_m=0, max_ctas=0,
                   chain_kblocks=0, prefetch_kblocks=0, epilogue=0, l2_hint=0, swap_ab=0,
                   swap_rows=0, scheduler=0):
        cfg = GemmConfig(variant, block_n, splits, stages, group_m, max_ctas, chain_kblocks, 0,
                         prefetch_kblocks, epilogue, l2_hint, swap_ab, swap_rows, scheduler)
        _check(lib().gemm_set_config(self._h, ctypes.byref(cfg)), "gemm_set_config")

    def reset_config(self):
        _check(lib().gemm_set_config(self._h, None), "gemm_set_config")

    def last_config(self) -> dict:
        cfg = GemmConfig()
        _check(lib().gemm_last_config(self._h, ctypes.byref(cfg)), "gemm_last_config")
        return cfg.as_dict()

    def device_status(self, stream=None):
        """(status code, raw device word) after synchronising the stream."""
        import torch
        detail = ctypes.c_uint32(0)
        sp = _stream_ptr(stream, torch.cuda.current_device())
        code = lib().gemm_device_status(self._h, sp, ctypes.byref(detail))
        return code, detail.value

    def set_wait_limit(self, ns: int):
        _check(lib().gemm_set_wait_limit(self._h, int(ns)), "gemm_set_wait_limit")

    def set_test_stall(self, enable: bool):
        _check(lib().gemm_set_test_stall(self._h, 1 if enable else 0), "gemm_set_test_stall")


def status_string(code: int) -> str:
    return lib().gemm_status_string(code).decode()
