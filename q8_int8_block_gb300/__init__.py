"""Python binding of libq8 (include/q8.h): the Q8_0 block-quantized linear layer on GB300.

Argument marshalling only: every step of the layer runs in the CUDA library.  Tensors
are torch tensors on the current CUDA device (torch provides device memory and streams);
each function passes raw pointers, sizes and the current stream to the C ABI and raises
Q8Error on a non-OK status.  There is no CPU fallback: if libq8.so is missing, importing
this package fails.

    Wq, Wd = q8_quantize_weights(W)              # W float32 [N,K] -> int8 [N,K], fp16 bits [N,K/32]
    xq, xd = q8_quantize_act(x)                  # x bf16/float32 [M,K] -> int8 [M,K], float32 [M,K/32]
    y = q8_linear(x, Wq, Wd)                     # x bf16 [M,K] -> float32 [M,N]
    y = q8_linear_ex(x, Wq, Wd, path="tensor", workspace=ws)
    y = q8_linear_fused(x, Wq, Wd, epi="silu_mul", aux=gate, out_dtype=torch.bfloat16)
    y = q8_linear_fused(h, Wq, Wd, norm_weight=g, norm_eps=1e-6)   # RMSNorm(h) . W^T
    xq, xd, r = q8_quantize_act_rmsnorm(h, g, 1e-6)
    B16 = q8_weights_to_f16(Wq)                        # once per weight matrix
    y = q8_linear_prepared(x, B16, Wd)                 # tensor-core path, no per-call widening
    o = q8_bsa_attention(q, k, v, row_ptr, col_idx)    # block-sparse causal attention
    q, k = q8_qk_norm_rope(q, k, positions, inv_freq, q_weight=wq, k_weight=wk)  # heads' norm + rotation
    o = q8_prompt_attention(q, k, v, cu_q)             # causal, packed sequences of any lengths
    o = q8_prefix_attention(q, kp, vp, ko, vo, n)      # one new token a request, shared prefix
    tab = q8_rope_table(positions, inv_freq)           # a step's rotations, for all layers
    cache = torch.zeros(q8_kv4_cache_shape(pages, page, Hkv, d), dtype=torch.uint8, device="cuda")
    qr = q8_kv4_append(k, v, cache, slots, table=tab, q=q, q_weight=wq, k_weight=wk)  # 4-bit paged cache
    o = q8_kv4_attention(qr, cache, block_table, kv_len)  # newest tokens over their caches
    k, v = q8_kv4_gather(cache, block_table, cu, tokens)  # the cache read back
    codes, scales = q8_kv3_encode(kv)                  # kv [..., 128] -> 3-bit codes + scales
    kv_hat = q8_kv3_decode(codes, scales, torch.bfloat16)
    isum = q8_block_sums(xq, Wq, path="decode")  # int32 [M,N,K/32]
"""
import ctypes
import os
import struct

import torch

__all__ = ["Q8Error", "q8_quantize_weights", "q8_quantize_act", "q8_quantize_act_rmsnorm",
           "q8_linear", "q8_linear_ex", "q8_kv3_encode", "q8_kv3_decode", "KV3_GROUP",
           "q8_weights_to_f16", "q8_linear_prepared", "q8_linear_prepared_workspace_size",
           "q8_bsa_attention", "q8_qk_norm_rope", "q8_prompt_attention",
           "q8_prompt_attention_workspace_size", "q8_prefix_attention",
           "q8_prefix_attention_workspace_size", "q8_rope_table", "q8_kv4_cache_shape", "q8_kv4_append",
           "q8_kv4_gather", "q8_kv4_attention", "q8_kv4_attention_workspace_size", "KV4_TILE",
           "q8_linear_fused", "EPILOGUES",
           "q8_linear_workspace_size", "q8_block_sums", "q8_device_error", "q8_release",
           "q8_set_timing_events", "q8_linear_noalloc", "NOALLOC_SCRATCH_BYTES",
           "q8_version", "lib_path", "QK", "PATHS"]

QK = 32
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libq8.so")

STATUS = {0: "Q8_OK", 1: "Q8_ERR_NULL", 2: "Q8_ERR_SHAPE", 3: "Q8_ERR_ALIGN", 4: "Q8_ERR_DTYPE",
          5: "Q8_ERR_NOMEM", 6: "Q8_ERR_CUDA", 7: "Q8_ERR_DEVICE", 8: "Q8_ERR_CAPTURE",
          9: "Q8_ERR_VALUE"}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}
PATHS = {"auto": 0, "decode": 1, "tensor": 2, "batch": 3, "dp4a": 4}
EPILOGUES = {"none": 0, "add": 1, "silu_mul": 2}


class Q8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = _L.q8_status_string(status).decode()
        if status == 6:
            msg += ": " + _L.q8_last_cuda_error().decode()
        super().__init__(f"{what}: {STATUS.get(status, status)} ({msg})")


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libq8.so is not built ({_LIB_PATH}); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(_LIB_PATH)
    p, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    sigs = {
        "q8_quantize_weights": [p, p, p, i64, i64, p],
        "q8_quantize_act": [p, i32, p, p, i64, i64, p],
        "q8_linear": [p, p, p, p, i64, i64, i64, p],
        "q8_linear_ex": [p, i32, p, p, p, i64, i64, i64, i32, p, sz, p],
        "q8_block_sums": [p, p, p, i64, i64, i64, i32, p],
        "q8_linear_noalloc": [p, i32, p, p, p, i64, i64, i64, p],
        "q8_linear_fused": [p, i32, p, f32, p, p, i32, p, p, i32, i64, i64, i64, i32, p, sz, p],
        "q8_quantize_act_rmsnorm": [p, i32, p, f32, p, p, p, i64, i64, p],
        "q8_kv3_encode": [p, i32, p, p, i64, p],
        "q8_kv3_decode": [p, p, p, i32, i64, p],
        "q8_weights_to_f16": [p, p, i64, i64, p],
        "q8_bsa_attention": [p, p, p, p, p, i64, p, i32, i64, i64, i64, i64, p],
        "q8_qk_norm_rope": [p, p, i32, i64, i64, p, p, f32, p, p, i64, i32, p, p, i64, i64, i64, i64, i64, i64, p],
        "q8_prompt_attention": [p, p, p, p, p, p, i64, i64, i64, i64, i64, i64, f32, p, p, sz, p],
        "q8_prefix_attention": [p, p, p, p, p, p, p, i64, i64, i64, i64, i64, i64, f32, p, p, sz, p],
        "q8_rope_table": [p, i64, p, p, p, i64, i64, p],
        "q8_kv4_append": [p, p, p, i32, p, p, p, f32, p, i64, i32, p, p, i64, i64, i64, p, i64, i64, i64, i64, p],
        "q8_kv4_gather": [p, i64, i64, i64, p, i64, p, p, p, p, i32, i64, i64, i64, i64, p],
        "q8_kv4_attention": [p, p, i64, i64, i64, p, i64, p, p, p, i64, i64, i64, i64, i64, f32, p, p, sz, p],
        "q8_linear_prepared": [p, i32, p, f32, p, p, i32, p, p, i32, i64, i64, i64, p, sz, p],
    }
    for name, args in sigs.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = i32
    L.q8_set_timing_events.argtypes = [p, p, i32]
    L.q8_set_timing_events.restype = i32
    L.q8_linear_workspace_size.argtypes = [i64, i64, i64, i32]
    L.q8_linear_workspace_size.restype = sz
    L.q8_linear_prepared_workspace_size.argtypes = [i64, i64, i64]
    L.q8_linear_prepared_workspace_size.restype = sz
    for name in ("q8_prompt_attention_workspace_size", "q8_prefix_attention_workspace_size"):
        getattr(L, name).argtypes = [i64] * 6
        getattr(L, name).restype = sz
    L.q8_kv4_attention_workspace_size.argtypes = [i64] * 6 + [i32]
    L.q8_kv4_attention_workspace_size.restype = sz
    L.q8_device_error.argtypes = [ctypes.POINTER(i32)]
    L.q8_device_error.restype = ctypes.c_uint32
    L.q8_status_string.argtypes = [i32]
    L.q8_status_string.restype = ctypes.c_char_p
    L.q8_last_cuda_error.argtypes = []
    L.q8_last_cuda_error.restype = ctypes.c_char_p
    L.q8_release.argtypes = []
    L.q8_release.restype = None
    L.q8_version.argtypes = []
    L.q8_version.restype = ctypes.c_char_p
    return L


_L = _load()


def lib_path() -> str:
    return _LIB_PATH


def lib():
    return _L


def _check(status: int, what: str):
    if status != 0:
        raise Q8Error(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without building a torch Stream object (a few microseconds per
# call otherwise); torch has long provided the query, the fallback covers a build without it
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _RAW_STREAM is not None:
            return ctypes.c_void_p(_RAW_STREAM(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _stream_on(stream, d):
    """_stream for a caller that has looked the current device d up already."""
    if stream is None and _RAW_STREAM is not None:
        return _RAW_STREAM(d)
    return _stream(stream)


def _key(table, key, name):
    """table[key], or a ValueError naming the accepted keys."""
    if key not in table:
        raise ValueError(f"{name}: expected one of {sorted(table)}, got {key!r}")
    return table[key]


def _need(t, dtype, shape, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: must be a contiguous CUDA tensor")


def _on_device(**tensors):
    """Every tensor given (None skipped) is a contiguous CUDA tensor on the current device:
    the library launches there, so a pointer into host memory or another GPU's memory must
    not reach its kernels.  One device query per call."""
    d = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}: must be a contiguous CUDA tensor")
        if d is None:
            d = torch.cuda.current_device()
        if t.get_device() != d:
            raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{d} "
                             "(use torch.cuda.device)")


def q8_quantize_weights(W, Wq=None, Wd=None, stream=None):
    """W float32 [N,K] -> (Wq int8 [N,K], Wd int16-stored binary16 bits [N,K/32])."""
    N, K = W.shape
    _need(W, torch.float32, (N, K), "W")
    if Wq is None:
        Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    if Wd is None:
        Wd = torch.empty((N, K // QK), dtype=torch.int16, device=W.device)
    _need(Wq, torch.int8, (N, K), "Wq")
    _need(Wd, torch.int16, (N, K // QK), "Wd")
    _on_device(W=W, Wq=Wq, Wd=Wd)
    _check(_L.q8_quantize_weights(_ptr(W), _ptr(Wq), _ptr(Wd), N, K, _stream(stream)),
           "q8_quantize_weights")
    return Wq, Wd


def q8_quantize_act(x, xq=None, xd=None, stream=None):
    """x bf16 or float32 [M,K] -> (xq int8 [M,K], xd float32 [M,K/32])."""
    M, K = x.shape
    if x.dtype not in DTYPES:
        raise TypeError(f"x: expected bfloat16 or float32, got {x.dtype}")
    _need(x, x.dtype, (M, K), "x")
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if xd is None:
        xd = torch.empty((M, K // QK), dtype=torch.float32, device=x.device)
    _need(xq, torch.int8, (M, K), "xq")
    _need(xd, torch.float32, (M, K // QK), "xd")
    _on_device(x=x, xq=xq, xd=xd)
    _check(_L.q8_quantize_act(_ptr(x), DTYPES[x.dtype], _ptr(xq), _ptr(xd), M, K, _stream(stream)),
           "q8_quantize_act")
    return xq, xd


def q8_quantize_act_rmsnorm(x, gamma, eps, xq=None, xd=None, r=None, stream=None):
    """RMSNorm fused into the activation quantizer: x bf16/float32 [M,K], gamma float32 [K]
    -> (xq int8 [M,K]: codes of x * gamma, xd float32 [M,K/32]: their scales times r,
    r float32 [M] = 1 / sqrt(mean(x^2) + eps))."""
    M, K = x.shape
    if x.dtype not in DTYPES:
        raise TypeError(f"x: expected bfloat16 or float32, got {x.dtype}")
    _need(x, x.dtype, (M, K), "x")
    _need(gamma, torch.float32, (K,), "gamma")
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if xd is None:
        xd = torch.empty((M, K // QK), dtype=torch.float32, device=x.device)
    if r is None:
        r = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(xq, torch.int8, (M, K), "xq")
    _need(xd, torch.float32, (M, K // QK), "xd")
    _need(r, torch.float32, (M,), "r")
    _on_device(x=x, gamma=gamma, xq=xq, xd=xd, r=r)
    _check(_L.q8_quantize_act_rmsnorm(_ptr(x), DTYPES[x.dtype], _ptr(gamma), float(eps), _ptr(xq),
                                      _ptr(xd), _ptr(r), M, K, _stream(stream)),
           "q8_quantize_act_rmsnorm")
    return xq, xd, r


def _lin_check(x, Wq, Wd, y):
    M, K = x.shape
    N = Wq.shape[0]
    _need(Wq, torch.int8, (N, K), "Wq")
    _need(Wd, torch.int16, (N, K // QK), "Wd")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _need(y, torch.float32, (M, N), "y")
    return M, N, K, y


def q8_linear(x, Wq, Wd, y=None, stream=None):
    """y float32 [M,N] = Q8_0 linear of bf16 x [M,K] (library-owned scratch)."""
    _need(x, torch.bfloat16, tuple(x.shape), "x")
    M, N, K, y = _lin_check(x, Wq, Wd, y)
    _on_device(x=x, Wq=Wq, Wd=Wd, y=y)
    _check(_L.q8_linear(_ptr(x), _ptr(Wq), _ptr(Wd), _ptr(y), M, N, K, _stream(stream)),
           "q8_linear")
    return y


def q8_linear_workspace_size(M, N, K, path="auto") -> int:
    return int(_L.q8_linear_workspace_size(M, N, K, _key(PATHS, path, "path")))


def q8_linear_ex(x, Wq, Wd, y=None, path="auto", workspace=None, stream=None):
    """q8_linear with activation type (bf16/float32), kernel family and caller scratch.
    workspace: a uint8 CUDA tensor of at least q8_linear_workspace_size() bytes, or None
    (then one is allocated here with torch)."""
    if x.dtype not in DTYPES:
        raise TypeError(f"x: expected bfloat16 or float32, got {x.dtype}")
    path_id = _key(PATHS, path, "path")
    _need(x, x.dtype, tuple(x.shape), "x")
    M, N, K, y = _lin_check(x, Wq, Wd, y)
    need = q8_linear_workspace_size(M, N, K, path)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _on_device(x=x, Wq=Wq, Wd=Wd, y=y, workspace=workspace)
    _check(_L.q8_linear_ex(_ptr(x), DTYPES[x.dtype], _ptr(Wq), _ptr(Wd), _ptr(y), M, N, K,
                           path_id, _ptr(workspace), nbytes, _stream(stream)), "q8_linear_ex")
    return y


def q8_linear_fused(x, Wq, Wd, epi="none", aux=None, y=None, out_dtype=torch.float32,
                    path="auto", workspace=None, stream=None, norm_weight=None, norm_eps=1e-6):
    """The linear layer with its neighbours fused into it.  norm_weight (float32 [K]): the
    input is RMSNorm(x) with that weight and norm_eps, applied inside the layer's quantizer.
    epi "none": y = x.W^T; "add": y = x.W^T + aux (residual); "silu_mul":
    y = silu(aux) * x.W^T (aux the gate projection's output).  aux float32 [M,N];
    y float32 or bfloat16 [M,N].  workspace None uses the library-owned scratch."""
    if x.dtype not in DTYPES:
        raise TypeError(f"x: expected bfloat16 or float32, got {x.dtype}")
    if out_dtype not in DTYPES:
        raise TypeError(f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
    epi_id, path_id = _key(EPILOGUES, epi, "epi"), _key(PATHS, path, "path")
    if epi_id != 0 and aux is None:
        raise ValueError(f"epi {epi!r} needs aux")
    _need(x, x.dtype, tuple(x.shape), "x")
    M, K = x.shape
    N = Wq.shape[0]
    _need(Wq, torch.int8, (N, K), "Wq")
    _need(Wd, torch.int16, (N, K // QK), "Wd")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _need(y, out_dtype, (M, N), "y")
    if epi_id != 0:
        _need(aux, torch.float32, (M, N), "aux")
    if norm_weight is not None:
        _need(norm_weight, torch.float32, (K,), "norm_weight")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _on_device(x=x, norm_weight=norm_weight, Wq=Wq, Wd=Wd, aux=aux, y=y, workspace=workspace)
    _check(_L.q8_linear_fused(_ptr(x), DTYPES[x.dtype], _ptr(norm_weight), float(norm_eps),
                              _ptr(Wq), _ptr(Wd), epi_id,
                              _ptr(aux), _ptr(y), DTYPES[out_dtype], M, N, K, path_id,
                              _ptr(workspace), nbytes, _stream(stream)), "q8_linear_fused")
    return y


def q8_weights_to_f16(Wq, B16=None, stream=None):
    """Wq int8 [N,K] -> B16 int16-stored binary16 codes [N,K], for q8_linear_prepared."""
    N, K = Wq.shape
    _need(Wq, torch.int8, (N, K), "Wq")
    if B16 is None:
        B16 = torch.empty((N, K), dtype=torch.int16, device=Wq.device)
    _need(B16, torch.int16, (N, K), "B16")
    _on_device(Wq=Wq, B16=B16)
    _check(_L.q8_weights_to_f16(_ptr(Wq), _ptr(B16), N, K, _stream(stream)), "q8_weights_to_f16")
    return B16


def q8_linear_prepared_workspace_size(M, N, K) -> int:
    return int(_L.q8_linear_prepared_workspace_size(M, N, K))


def q8_linear_prepared(x, B16, Wd, epi="none", aux=None, y=None, out_dtype=torch.float32,
                       workspace=None, stream=None, norm_weight=None, norm_eps=1e-6):
    """q8_linear_fused on the tensor-core path with weights widened once by
    q8_weights_to_f16 (no per-call widening)."""
    if x.dtype not in DTYPES:
        raise TypeError(f"x: expected bfloat16 or float32, got {x.dtype}")
    if out_dtype not in DTYPES:
        raise TypeError(f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
    epi_id = _key(EPILOGUES, epi, "epi")
    if epi_id != 0 and aux is None:
        raise ValueError(f"epi {epi!r} needs aux")
    _need(x, x.dtype, tuple(x.shape), "x")
    M, K = x.shape
    N = B16.shape[0]
    _need(B16, torch.int16, (N, K), "B16")
    _need(Wd, torch.int16, (N, K // QK), "Wd")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _need(y, out_dtype, (M, N), "y")
    if epi_id != 0:
        _need(aux, torch.float32, (M, N), "aux")
    if norm_weight is not None:
        _need(norm_weight, torch.float32, (K,), "norm_weight")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _on_device(x=x, norm_weight=norm_weight, B16=B16, Wd=Wd, aux=aux, y=y, workspace=workspace)
    _check(_L.q8_linear_prepared(_ptr(x), DTYPES[x.dtype], _ptr(norm_weight), float(norm_eps),
                                 _ptr(B16), _ptr(Wd), epi_id, _ptr(aux), _ptr(y),
                                 DTYPES[out_dtype], M, N, K, _ptr(workspace), nbytes,
                                 _stream(stream)), "q8_linear_prepared")
    return y


def q8_bsa_attention(q, k, v, row_ptr, col_idx, out_dtype=torch.float32, o=None, stream=None):
    """Block-sparse causal attention: q [H,T,128], k and v [Hkv,T,128] bfloat16; row_ptr
    int32 [H*T/64+1], col_idx int32 [nnz] (the listed 64-token key blocks of each head's
    64-token query block) -> o [H,T,128] of out_dtype."""
    H, T, d = q.shape
    Hkv = k.shape[0]
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, (H if name == "q" else Hkv, T, d), name)
    _need(row_ptr, torch.int32, (H * (T // 64) + 1,), "row_ptr")
    if col_idx.dim() != 1:
        raise ValueError("col_idx: a 1-D int32 CUDA tensor")
    _need(col_idx, torch.int32, (col_idx.numel(),), "col_idx")
    if out_dtype not in DTYPES:
        raise TypeError(f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
    if o is None:
        o = torch.empty((H, T, d), dtype=out_dtype, device=q.device)
    _need(o, out_dtype, (H, T, d), "o")
    _on_device(q=q, k=k, v=v, row_ptr=row_ptr, col_idx=col_idx, o=o)
    _check(_L.q8_bsa_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr), _ptr(col_idx),
                               col_idx.numel(), _ptr(o), DTYPES[out_dtype], H, Hkv, T, d,
                               _stream(stream)), "q8_bsa_attention")
    return o


def _heads(name, t, dtype, shape, d):
    """The strides of t, a tensor on CUDA device d of this type and shape whose innermost
    dimension (a head's channels) is contiguous."""
    st = t.stride()
    if t.dtype is dtype and t.shape == shape and t.get_device() == d and (st[-1] == 1 or shape[-1] <= 1):
        return st
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != d:
        raise ValueError(f"{name}: must be a CUDA tensor on the current device (cuda:{d})")
    raise ValueError(f"{name}: the channels of a head must be contiguous")


def _vector(name, t, dtype, n, d):
    """The address of t, a contiguous vector of n elements on CUDA device d."""
    if t.dtype is dtype and t.shape == (n,) and t.get_device() == d and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != (n,):
        raise ValueError(f"{name}: expected shape {(n,)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: must be a contiguous CUDA tensor on the current device (cuda:{d})")


_STRIDES8, _STRIDES14 = struct.Struct("8q").pack, struct.Struct("14q").pack


def _empty(shape, dtype, device, stream):
    """A new tensor for work on `stream`: torch hands its memory on in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(workspace, need, device, d, stream):
    """(tensor or None, address or None, bytes): the caller's workspace, else one from torch."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _empty(need, torch.uint8, device, stream)
        return workspace, workspace.data_ptr(), need
    if workspace.get_device() != d or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be a contiguous CUDA tensor on the current device (cuda:{d})")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def q8_qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                    interleaved=False, q_out=None, k_out=None, stream=None):
    """RMSNorm of every query and key head and the rotation of its first channels by position:
    q [T,H,d], k [T,Hkv,d] bfloat16 or float32 (views of a projection's rows are fine),
    positions int32 [T], inv_freq float64 [rot/2], weights float32 [d] or None (no norm)
    -> (q_out, k_out) bfloat16.  q_out=q, k_out=k work in place (bfloat16)."""
    dev = torch.cuda.current_device()
    (T, H, d), (_, Hkv, _), (half,) = q.shape, k.shape, inv_freq.shape
    dtype, bf16, f32 = q.dtype, torch.bfloat16, torch.float32
    xtype = DTYPES.get(dtype)
    if xtype is None:
        raise TypeError(f"q: expected bfloat16 or float32, got {dtype}")
    sq, sk = _heads("q", q, dtype, (T, H, d), dev), _heads("k", k, dtype, (T, Hkv, d), dev)
    if q_out is None:
        q_out, sqo = _empty((T, H, d), bf16, q.device, stream), (H * d, d)
    else:
        sqo = _heads("q_out", q_out, bf16, (T, H, d), dev)
    if k_out is None:
        k_out, sko = _empty((T, Hkv, d), bf16, q.device, stream), (Hkv * d, d)
    else:
        sko = _heads("k_out", k_out, bf16, (T, Hkv, d), dev)
    if (H > 1 and (sq[1] != d or sqo[1] != d)) or (Hkv > 1 and (sk[1] != d or sko[1] != d)):
        raise ValueError("q, k, q_out, k_out: the heads of a token must be contiguous")
    if T <= 1:  # a single token: its stride says nothing
        sq, sk, sqo, sko = (H * d,), (Hkv * d,), (H * d,), (Hkv * d,)
    status = _L.q8_qk_norm_rope(
        q.data_ptr(), k.data_ptr(), xtype, sq[0], sk[0],
        None if q_weight is None else _vector("q_weight", q_weight, f32, d, dev),
        None if k_weight is None else _vector("k_weight", k_weight, f32, d, dev), eps,
        _vector("positions", positions, torch.int32, T, dev), _vector("inv_freq", inv_freq, torch.float64, half, dev),
        2 * half, 1 if interleaved else 0, q_out.data_ptr(), k_out.data_ptr(), sqo[0], sko[0], T, H, Hkv, d,
        _stream_on(stream, dev))
    if status:
        raise Q8Error(status, "q8_qk_norm_rope")
    return q_out, k_out


def q8_prompt_attention_workspace_size(B, Tq, Tk, H, Hkv, d) -> int:
    return int(_L.q8_prompt_attention_workspace_size(B, Tq, Tk, H, Hkv, d))


def q8_prompt_attention(q, k, v, cu_q, cu_k=None, scale=None, o=None, workspace=None, stream=None):
    """Causal attention over packed sequences: q [Tq,H,d], k and v [Tk,Hkv,d] bfloat16 (d 64 or
    128; strided views are fine), cu_q and cu_k int32 [B+1] on the device: sequence s holds the
    queries cu_q[s]:cu_q[s+1], the last ones of its keys cu_k[s]:cu_k[s+1] (None: cu_q)
    -> o [Tq,H,d] bfloat16 (a new o is not initialised outside the sequences).  scale None:
    1/sqrt(d).  workspace None: allocated here with torch (as a new o, on `stream`)."""
    dev = torch.cuda.current_device()
    (Tq, H, d), (Tk, Hkv, _) = q.shape, k.shape
    sq, sk, sv = (_heads("q", q, torch.bfloat16, (Tq, H, d), dev), _heads("k", k, torch.bfloat16, (Tk, Hkv, d), dev),
                  _heads("v", v, torch.bfloat16, (Tk, Hkv, d), dev))
    n = cu_q.numel()
    if n < 1:
        raise ValueError("cu_q: expected at least one entry")
    pq = _vector("cu_q", cu_q, torch.int32, n, dev)
    pk = pq if cu_k is None else _vector("cu_k", cu_k, torch.int32, n, dev)
    if o is None:
        o = _empty((Tq, H, d), torch.bfloat16, q.device, stream)
        so = (H * d, d)
    else:
        so = _heads("o", o, torch.bfloat16, (Tq, H, d), dev)
    workspace, pw, nbytes = _workspace(
        workspace, _L.q8_prompt_attention_workspace_size(n - 1, Tq, Tk, H, Hkv, d), q.device, dev, stream)
    status = _L.q8_prompt_attention(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), pq, pk, o.data_ptr(), n - 1, Tq, Tk, H, Hkv, d,
        (d or 1) ** -0.5 if scale is None else scale,
        _STRIDES8(sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1]), pw, nbytes, _stream_on(stream, dev))
    if status:
        raise Q8Error(status, "q8_prompt_attention")
    return o


def q8_prefix_attention_workspace_size(B, P, cap, H, Hkv, d) -> int:
    return int(_L.q8_prefix_attention_workspace_size(B, P, cap, H, Hkv, d))


def q8_prefix_attention(q, k_prefix, v_prefix, k_own, v_own, own_len, scale=None, o=None,
                        workspace=None, stream=None):
    """One query for each of B requests behind a shared prefix: q [B,H,d], k_prefix and
    v_prefix [P,Hkv,d], k_own and v_own [B,cap,Hkv,d] bfloat16 (d 64 or 128; strided views are
    fine), own_len int32 [B] on the device: request b sees the prefix and its first own_len[b]
    own keys -> o [B,H,d] bfloat16.  scale None: 1/sqrt(d).  workspace None: allocated here with
    torch (as a new o, on `stream`)."""
    dev = torch.cuda.current_device()
    (B, H, d), (P, Hkv, _), (_, cap, _, _) = q.shape, k_prefix.shape, k_own.shape
    bf16, shared, own = torch.bfloat16, (P, Hkv, d), (B, cap, Hkv, d)
    sq = _heads("q", q, bf16, (B, H, d), dev)
    skp, svp = _heads("k_prefix", k_prefix, bf16, shared, dev), _heads("v_prefix", v_prefix, bf16, shared, dev)
    sko, svo = _heads("k_own", k_own, bf16, own, dev), _heads("v_own", v_own, bf16, own, dev)
    pn = _vector("own_len", own_len, torch.int32, B, dev)
    if o is None:
        o = _empty((B, H, d), bf16, q.device, stream)
        so = (H * d, d)
    else:
        so = _heads("o", o, bf16, (B, H, d), dev)
    workspace, pw, nbytes = _workspace(
        workspace, _L.q8_prefix_attention_workspace_size(B, P, cap, H, Hkv, d), q.device, dev, stream)
    status = _L.q8_prefix_attention(
        q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k_own.data_ptr(), v_own.data_ptr(), pn, o.data_ptr(),
        B, P, cap, H, Hkv, d, (d or 1) ** -0.5 if scale is None else scale,
        _STRIDES14(sq[0], sq[1], skp[0], skp[1], svp[0], svp[1], sko[0], sko[1], sko[2], svo[0], svo[1], svo[2],
                   so[0], so[1]), pw, nbytes, _stream_on(stream, dev))
    if status:
        raise Q8Error(status, "q8_prefix_attention")
    return o


KV4_TILE = 32  # tokens of a tile


def q8_kv4_cache_shape(pages, page, Hkv, d):
    """The shape of a paged 4-bit cache (uint8): [pages, Hkv, page/32, 36 d], page a multiple of 32."""
    if page % KV4_TILE or page < KV4_TILE or d not in (64, 128, 256):
        raise ValueError(f"page: a multiple of {KV4_TILE}, d: 64, 128 or 256; got {page} and {d}")
    return pages, Hkv, page // KV4_TILE, 36 * d


def _kv4_cache(cache, d, dev):
    """(page stride in bytes, pages, page, Hkv): cache is a uint8 tensor of q8_kv4_cache_shape on CUDA
    device dev whose pages are contiguous (but may lie apart from one another)."""
    if cache.dtype is not torch.uint8:
        raise TypeError(f"cache: expected torch.uint8, got {cache.dtype}")
    shape = cache.shape
    if len(shape) != 4 or shape[3] != 36 * d:
        raise ValueError(f"cache: expected shape (pages, Hkv, page/32, {36 * d}), got {tuple(shape)}")
    if cache.get_device() != dev:
        raise ValueError(f"cache: must be a CUDA tensor on the current device (cuda:{dev})")
    pages, Hkv, tiles, size = shape
    if cache.is_contiguous():
        return Hkv * tiles * size, pages, KV4_TILE * tiles, Hkv
    st = cache.stride()
    if (st[3] != 1 and size > 1) or (st[2] != size and tiles > 1) or (st[1] != tiles * size and Hkv > 1):
        raise ValueError("cache: the bytes of a page must be contiguous")
    return (st[0] if pages > 1 else Hkv * tiles * size), pages, KV4_TILE * tiles, Hkv


def _block_table(block_table, B, dev):
    """(address, width) of a contiguous int32 [B, width] on CUDA device dev."""
    shape = block_table.shape
    if block_table.dtype is not torch.int32:
        raise TypeError(f"block_table: expected torch.int32, got {block_table.dtype}")
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"block_table: expected shape ({B}, width), got {tuple(shape)}")
    if block_table.get_device() != dev or not block_table.is_contiguous():
        raise ValueError(f"block_table: must be a contiguous CUDA tensor on the current device (cuda:{dev})")
    return block_table.data_ptr(), shape[1]


def q8_rope_table(positions, inv_freq, axis=None, table=None, stream=None):
    """A step's rotations, for all its layers: positions int32 [T], or [axes, T] with axis int32 [half]
    (which axis turns a pair; None: the first), inv_freq float64 [half] -> float32 [T, 2, half],
    cosines then sines."""
    dev = torch.cuda.current_device()
    if positions.dtype is not torch.int32:
        raise TypeError(f"positions: expected torch.int32, got {positions.dtype}")
    if positions.dim() not in (1, 2):
        raise ValueError(f"positions: expected shape (T,) or (axes, T), got {tuple(positions.shape)}")
    if positions.get_device() != dev or not positions.is_contiguous():
        raise ValueError(f"positions: must be a contiguous CUDA tensor on the current device (cuda:{dev})")
    axes, T = (1, positions.shape[0]) if positions.dim() == 1 else positions.shape
    (half,) = inv_freq.shape
    if table is None:
        table = _empty((T, 2, half), torch.float32, positions.device, stream)
    elif table.dtype is not torch.float32:
        raise TypeError(f"table: expected torch.float32, got {table.dtype}")
    elif table.shape != (T, 2, half) or table.get_device() != dev or not table.is_contiguous():
        raise ValueError(f"table: a contiguous CUDA tensor of shape {(T, 2, half)} on the current device (cuda:{dev})")
    status = _L.q8_rope_table(positions.data_ptr(), axes, _vector("inv_freq", inv_freq, torch.float64, half, dev),
                              None if axis is None else _vector("axis", axis, torch.int32, half, dev),
                              table.data_ptr(), T, half, _stream_on(stream, dev))
    if status:
        raise Q8Error(status, "q8_rope_table")
    return table


_STRIDES4 = struct.Struct("4q").pack


def q8_kv4_append(k, v, cache, slots, table=None, q=None, q_weight=None, k_weight=None, eps=1e-6,
                  interleaved=False, q_out=None, stream=None):
    """A step's keys and values into the paged 4-bit cache, and its queries made ready: RMSNorm of the
    query and key heads (weights float32 [d], None: none), their rotation by table (float32
    [T, 2, rot/2] from q8_rope_table, None: none), and the quantiser.  k, v [T,Hkv,d] and q [T,H,d]
    bfloat16 or float32 (views of a projection's rows are fine), cache uint8 of
    q8_kv4_cache_shape, slots int32 [T] (page * index + offset; negative: not kept)
    -> q_out [T,H,d] bfloat16 (None without q)."""
    dev = torch.cuda.current_device()
    T, Hkv, d = k.shape
    dtype, f32 = k.dtype, torch.float32
    xtype = DTYPES.get(dtype)
    if xtype is None:
        raise TypeError(f"k: expected bfloat16 or float32, got {dtype}")
    sk, sv = _heads("k", k, dtype, (T, Hkv, d), dev), _heads("v", v, dtype, (T, Hkv, d), dev)
    if Hkv > 1 and (sk[1] != d or sv[1] != d):
        raise ValueError("k, v: the heads of a token must be contiguous")
    H, sq, sqo, pq, po = 0, (0,), (0,), None, None
    if q is not None:
        H = q.shape[1]
        sq = _heads("q", q, dtype, (T, H, d), dev)
        if q_out is None:
            q_out, sqo = _empty((T, H, d), torch.bfloat16, q.device, stream), (H * d, d)
        else:
            sqo = _heads("q_out", q_out, torch.bfloat16, (T, H, d), dev)
        if H > 1 and (sq[1] != d or sqo[1] != d):
            raise ValueError("q, q_out: the heads of a token must be contiguous")
        pq, po = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out: given without q")
    rot, pt = 0, None
    if table is not None:
        shape = table.shape
        if table.dtype is not f32:
            raise TypeError(f"table: expected torch.float32, got {table.dtype}")
        if len(shape) != 3 or shape[0] != T or shape[1] != 2:
            raise ValueError(f"table: expected shape ({T}, 2, rot/2), got {tuple(shape)}")
        if table.get_device() != dev or not table.is_contiguous():
            raise ValueError(f"table: must be a contiguous CUDA tensor on the current device (cuda:{dev})")
        rot, pt = 2 * shape[2], table.data_ptr()
    page_stride, pages, page, heads = _kv4_cache(cache, d, dev)
    if heads != Hkv:
        raise ValueError(f"cache: expected {Hkv} key/value heads, got {heads}")
    status = _L.q8_kv4_append(
        pq, k.data_ptr(), v.data_ptr(), xtype, _STRIDES4(sq[0], sk[0], sv[0], sqo[0]),
        None if q_weight is None else _vector("q_weight", q_weight, f32, d, dev),
        None if k_weight is None else _vector("k_weight", k_weight, f32, d, dev), eps, pt, rot,
        1 if interleaved else 0, _vector("slots", slots, torch.int32, T, dev), cache.data_ptr(), page_stride, pages,
        page, po, T, H, Hkv, d, _stream_on(stream, dev))
    if status:
        raise Q8Error(status, "q8_kv4_append")
    return q_out


def _rows(name, t, dtype, shape, dev):
    """t, a contiguous tensor of this type and shape on CUDA device dev."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous CUDA tensor of shape {shape} on the current device (cuda:{dev})")
    return t


def q8_kv4_gather(cache, block_table, cu, tokens, first=None, out_dtype=torch.bfloat16, k=None, v=None, stream=None):
    """The cache read back: row cu[b] + i of k and v [tokens,Hkv,d] (out_dtype bfloat16 or float32) is
    token first[b] + i (None: i) of request b; cu int32 [B+1], first int32 [B], block_table int32
    [B, width].  New k and v are not initialised outside the sequences."""
    dev = torch.cuda.current_device()
    if out_dtype not in DTYPES:
        raise TypeError(f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
    d = cache.shape[-1] // 36
    page_stride, pages, page, Hkv = _kv4_cache(cache, d, dev)
    n = cu.numel()
    if n < 1:
        raise ValueError("cu: expected at least one entry")
    pc, (pb, width) = _vector("cu", cu, torch.int32, n, dev), _block_table(block_table, n - 1, dev)
    shape = (tokens, Hkv, d)
    k = _empty(shape, out_dtype, cache.device, stream) if k is None else _rows("k", k, out_dtype, shape, dev)
    v = _empty(shape, out_dtype, cache.device, stream) if v is None else _rows("v", v, out_dtype, shape, dev)
    status = _L.q8_kv4_gather(
        cache.data_ptr(), page_stride, pages, page, pb, width,
        None if first is None else _vector("first", first, torch.int32, n - 1, dev), pc, k.data_ptr(),
        v.data_ptr(), DTYPES[out_dtype], n - 1, tokens, Hkv, d, _stream_on(stream, dev))
    if status:
        raise Q8Error(status, "q8_kv4_gather")
    return k, v


def q8_kv4_attention_workspace_size(B, width, page, H, Hkv, d, one_query=True) -> int:
    return int(_L.q8_kv4_attention_workspace_size(B, width, page, H, Hkv, d, 1 if one_query else 0))


def q8_kv4_attention(q, cache, block_table, kv_len, cu_q=None, scale=None, o=None, workspace=None, stream=None):
    """Attention of each request's newest tokens over its cache: q [Tq,H,d] bfloat16 (strided views are
    fine), cache uint8 of q8_kv4_cache_shape, block_table int32 [B, width], kv_len int32 [B] tokens
    of each request (the queries' own among them), cu_q int32 [B+1], rising (None: one query each,
    Tq = B, and faster):
    query i of lq sees the keys j <= i + kv_len - lq -> o [Tq,H,d] bfloat16 (a new o is not
    initialised outside the sequences).  scale None: 1/sqrt(d).  workspace None: allocated here with
    torch (as a new o, on `stream`).  For chunks of a prompt q8_kv4_gather and q8_prompt_attention are
    faster (heads of 64 or 128 channels; of 256 this is the only way)."""
    dev = torch.cuda.current_device()
    Tq, H, d = q.shape
    sq = _heads("q", q, torch.bfloat16, (Tq, H, d), dev)
    page_stride, pages, page, Hkv = _kv4_cache(cache, d, dev)
    B = Tq if cu_q is None else cu_q.numel() - 1
    if B < 0:
        raise ValueError("cu_q: expected at least one entry")
    pc = None if cu_q is None else _vector("cu_q", cu_q, torch.int32, B + 1, dev)
    (pb, width), pn = _block_table(block_table, B, dev), _vector("kv_len", kv_len, torch.int32, B, dev)
    if o is None:
        o = _empty((Tq, H, d), torch.bfloat16, q.device, stream)
        so = (H * d, d)
    else:
        so = _heads("o", o, torch.bfloat16, (Tq, H, d), dev)
    workspace, pw, nbytes = _workspace(
        workspace, _L.q8_kv4_attention_workspace_size(B, width, page, H, Hkv, d, 1 if cu_q is None else 0), q.device, dev,
        stream)
    status = _L.q8_kv4_attention(
        q.data_ptr(), cache.data_ptr(), page_stride, pages, page, pb, width, pn, pc, o.data_ptr(), B, Tq, H, Hkv, d,
        (d or 1) ** -0.5 if scale is None else scale, _STRIDES4(sq[0], sq[1], so[0], so[1]), pw, nbytes,
        _stream_on(stream, dev))
    if status:
        raise Q8Error(status, "q8_kv4_attention")
    return o


KV3_GROUP = 128


def q8_kv3_encode(x, codes=None, scales=None, stream=None):
    """3-bit KV-cache codec, encoder: x bf16/float32 [..., 128*k] (contiguous) ->
    (codes int32 [groups, 12] holding the uint32 code words, scales float32 [groups]), one
    group per 128 consecutive elements.  Reinterpret codes with .view(torch.int32) as needed."""
    if x.dtype not in DTYPES:
        raise TypeError(f"x: expected bfloat16 or float32, got {x.dtype}")
    if x.numel() % KV3_GROUP:
        raise ValueError("x: a contiguous CUDA tensor of whole 128-element groups")
    _need(x, x.dtype, tuple(x.shape), "x")
    n = x.numel() // KV3_GROUP
    if codes is None:
        codes = torch.empty((n, 12), dtype=torch.int32, device=x.device)
    if scales is None:
        scales = torch.empty((n,), dtype=torch.float32, device=x.device)
    _need(codes, torch.int32, (n, 12), "codes")
    _need(scales, torch.float32, (n,), "scales")
    _on_device(x=x, codes=codes, scales=scales)
    _check(_L.q8_kv3_encode(_ptr(x), DTYPES[x.dtype], _ptr(codes), _ptr(scales), n, _stream(stream)),
           "q8_kv3_encode")
    return codes, scales


def q8_kv3_decode(codes, scales, out_dtype=torch.bfloat16, out=None, stream=None):
    """3-bit KV-cache codec, decoder: (codes int32 [groups, 12], scales float32 [groups]) ->
    out [groups, 128] of out_dtype (bfloat16 or float32)."""
    n = codes.shape[0]
    _need(codes, torch.int32, (n, 12), "codes")
    _need(scales, torch.float32, (n,), "scales")
    if out_dtype not in DTYPES:
        raise TypeError(f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
    if out is None:
        out = torch.empty((n, KV3_GROUP), dtype=out_dtype, device=codes.device)
    _need(out, out_dtype, (n, KV3_GROUP), "out")
    _on_device(codes=codes, scales=scales, out=out)
    _check(_L.q8_kv3_decode(_ptr(codes), _ptr(scales), _ptr(out), DTYPES[out_dtype], n,
                            _stream(stream)), "q8_kv3_decode")
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20


def q8_linear_noalloc(x, Wq, Wd, y=None, stream=None):
    """Tensor-core Q8_0 linear that allocates no device memory: its scratch is a static
    device array of NOALLOC_SCRATCH_BYTES in the library (see include/q8.h).  For callers
    whose memory is owned by a fixed pool or whose step must not allocate.  Calls that
    overlap on the GPU share that array and race; make the first call on a device before
    any stream capture."""
    if x.dtype not in DTYPES:
        raise TypeError(f"x: expected bfloat16 or float32, got {x.dtype}")
    _need(x, x.dtype, tuple(x.shape), "x")
    M, N, K, y = _lin_check(x, Wq, Wd, y)
    _on_device(x=x, Wq=Wq, Wd=Wd, y=y)
    _check(_L.q8_linear_noalloc(_ptr(x), DTYPES[x.dtype], _ptr(Wq), _ptr(Wd), _ptr(y), M, N, K,
                                _stream(stream)), "q8_linear_noalloc")
    return y


def q8_block_sums(xq, Wq, isum=None, path="auto", stream=None):
    """Exact int32 block sums isum [M,N,K/32] of int8 codes, by the kernel of `path`."""
    path_id = _key(PATHS, path, "path")
    M, K = xq.shape
    N = Wq.shape[0]
    _need(xq, torch.int8, (M, K), "xq")
    _need(Wq, torch.int8, (N, K), "Wq")
    if isum is None:
        isum = torch.empty((M, N, K // QK), dtype=torch.int32, device=xq.device)
    _need(isum, torch.int32, (M, N, K // QK), "isum")
    _on_device(xq=xq, Wq=Wq, isum=isum)
    _check(_L.q8_block_sums(_ptr(xq), _ptr(Wq), _ptr(isum), M, N, K, path_id, _stream(stream)),
           "q8_block_sums")
    return isum


def q8_device_error() -> int:
    """Synchronizes the device and returns (and clears) the device error word (0 = none)."""
    st = ctypes.c_int(0)
    word = _L.q8_device_error(ctypes.byref(st))
    _check(st.value, "q8_device_error")
    return int(word)


def q8_set_timing_events(starts=None, stops=None):
    """Timing hook: events (torch.cuda.Event(enable_timing=True)) recorded around the main
    kernel of each later q8_linear / q8_linear_ex call, cycling through the list; under
    graph capture they become event nodes.  No arguments: switch off."""
    if not starts:
        _check(_L.q8_set_timing_events(None, None, 0), "q8_set_timing_events")
        return
    assert len(starts) == len(stops)
    for e in list(starts) + list(stops):  # make sure the CUDA events exist
        if e.cuda_event == 0:
            e.record()
    arr = ctypes.c_void_p * len(starts)
    a = arr(*[e.cuda_event for e in starts])
    b = arr(*[e.cuda_event for e in stops])
    _check(_L.q8_set_timing_events(a, b, len(starts)), "q8_set_timing_events")


def q8_release():
    _L.q8_release()


def q8_version() -> str:
    return _L.q8_version().decode()
