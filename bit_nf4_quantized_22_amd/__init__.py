"""QLoRA NF4 hot path on MI355X (gfx950): thin Python binding over the C ABI.

The functions here have the names of the C entry points in
``include/qlora_nf4.h`` and only marshal arguments: they check that tensors
are contiguous device tensors of the right dtype and size, allocate outputs
with torch when the caller passes none, and call the library on torch's
current stream.  Every step of the computation runs in the HIP kernels of
``lib/libqlora_nf4.so``; there is no other code path.  If the library is not
built, every call raises.

The library is loaded lazily so that ``bit_nf4_quantized_22_amd.synth`` can
be imported without it.
"""

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libqlora_nf4.so")

QN_OK, QN_ERR_NULL, QN_ERR_SHAPE, QN_ERR_ALIGN = 0, -1, -2, -3
QN_ERR_UNSUPPORTED, QN_ERR_WORKSPACE, QN_ERR_HIP = -4, -5, -6
QN_F32, QN_BF16 = 0, 1
QN_OP_FWD, QN_OP_BWD_DX, QN_OP_LORA_GRADS, QN_OP_BWD_DX_DROPOUT = 0, 1, 2, 3
QN_OP_FP8_FWD, QN_OP_FP8_BWD_DX = 4, 5
QN_OP_MXFP4_FWD, QN_OP_MXFP4_BWD_DX = 6, 7
QN_STATE_F32, QN_STATE_8BIT = 0, 1
QN_MUON_ORIGINAL, QN_MUON_MATCH_RMS = 0, 1
FP8_BLOCK, STATE_BLOCK, MXFP4_GROUP = 128, 256, 32
BLOCKSIZE, GROUP = 64, 256

EXPORTS = ("qn_status_string", "nf4_codebook", "nf4_quantize", "dq_quantize_scales",
           "nf4_dequant", "qn_workspace_bytes", "qlora_linear_fwd", "qlora_linear_bwd_dx",
           "lora_grads", "qlora_merge", "lora_adamw_step", "lora_dropout",
           "qlora_linear_fwd_dropout", "qlora_linear_bwd_dx_dropout", "fp4_codebook",
           "fp4_quantize", "dq_quantize_scales_fp8", "qlora_linear_fwd_noalloc",
           "dq_quantize_scales_centred", "nf4_quantize_dq", "nf4_quantize_dq_batch",
           "qn_hbm_read_probe", "fp8_quantize_blocks", "fp8_quantize_rows", "fp8_dequant",
           "fp8_matmul", "fp8_linear_fwd", "fp8_linear_bwd_dx", "lora_adamw_table_bytes",
           "lora_adamw_table", "lora_grad_norm_workspace_bytes", "lora_grad_norm",
           "lora_adamw_multi_step", "mxfp4_scale_bytes", "mxfp4_quantize", "mxfp4_dequant",
           "mxfp4_pack_scales", "mxfp4_unpack_scales", "mxfp4_matmul", "mxfp4_linear_fwd",
           "mxfp4_linear_bwd_dx", "lora_muon_table_bytes", "lora_muon_table",
           "lora_muon_workspace_bytes", "lora_muon_multi_step")


class QnError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


class qn_weight(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("qscale", ctypes.c_void_p),
                ("gscale", ctypes.c_void_p), ("absmax", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("blocksize", ctypes.c_int32), ("group", ctypes.c_int32),
                ("quant_type", ctypes.c_int32), ("scale_type", ctypes.c_int32),
                ("offset", ctypes.c_void_p)]


class qn_fp8_weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class qn_mxfp4_weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class qn_adamw_tensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("p_bf16", ctypes.c_void_p),
                ("n", ctypes.c_int64)]


class qn_adamw_plan(ctypes.Structure):
    _fields_ = [("chunks", ctypes.c_int64), ("bytes", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("state", ctypes.c_int32)]


class qn_muon_tensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("p_bf16", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class qn_muon_plan(ctypes.Structure):
    _fields_ = [("matrices", ctypes.c_int64 * 4), ("chunks", ctypes.c_int64 * 4),
                ("spans", ctypes.c_int64 * 4), ("bytes", ctypes.c_int64), ("ws_bytes", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32)]


class qn_muon_step(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("eps", ctypes.c_float),
                ("ns", ctypes.c_double * 3), ("ns_steps", ctypes.c_int32),
                ("nesterov", ctypes.c_int32), ("adjust", ctypes.c_int32)]


_lib = None


def load_library():
    """Load lib/libqlora_nf4.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing "
                           "(run python -m bit_nf4_quantized_22_amd.build)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz, u64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                  ctypes.c_float, ctypes.c_size_t, ctypes.c_uint64)
    wp = ctypes.POINTER(qn_weight)
    sig = {
        "qn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "nf4_codebook": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float)]),
        "fp4_codebook": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float)]),
        "nf4_quantize": (ctypes.c_int, [vp, i32, i64, i32, vp, vp, vp]),
        "fp4_quantize": (ctypes.c_int, [vp, i32, i64, i32, vp, vp, vp]),
        "dq_quantize_scales": (ctypes.c_int, [vp, i64, i32, vp, vp, vp]),
        "dq_quantize_scales_fp8": (ctypes.c_int, [vp, i64, i32, vp, vp, vp]),
        "dq_quantize_scales_centred": (ctypes.c_int, [vp, i64, i32, vp, vp, vp, vp]),
        "nf4_quantize_dq": (ctypes.c_int, [vp, i32, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp]),
        "nf4_quantize_dq_batch": (ctypes.c_int, [i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp,
                                                 vp, vp]),
        "qn_hbm_read_probe": (ctypes.c_int, [vp, i64, vp, vp]),
        "nf4_dequant": (ctypes.c_int, [wp, i32, vp, vp]),
        "qn_workspace_bytes": (sz, [i32, i64, i64, i64, i32]),
        "qlora_linear_fwd": (ctypes.c_int, [wp, vp, i64, vp, vp, i32, f32, vp, vp, vp, sz, vp]),
        "qlora_linear_bwd_dx": (ctypes.c_int, [wp, vp, i64, vp, vp, i32, f32, vp, vp, vp, sz, vp]),
        "lora_grads": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, f32, vp, vp,
                                      vp, sz, vp]),
        "qlora_merge": (ctypes.c_int, [wp, vp, vp, i32, f32, vp, vp]),
        "lora_adamw_step": (ctypes.c_int, [vp, vp, vp, vp, vp, i64, f32, f32, f32, f32, f32, i32,
                                           vp]),
        "lora_dropout": (ctypes.c_int, [vp, i64, i64, f32, u64, vp, vp]),
        "qlora_linear_fwd_noalloc": (ctypes.c_int, [wp, vp, i64, vp, vp, i32, f32, vp, vp, vp]),
        "qlora_linear_fwd_dropout": (ctypes.c_int, [wp, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp,
                                                    sz, vp]),
        "qlora_linear_bwd_dx_dropout": (ctypes.c_int, [wp, vp, i64, vp, vp, i32, f32, f32, u64, vp,
                                                       vp, vp, sz, vp]),
    }
    fp, ap, pp = (ctypes.POINTER(c) for c in (qn_fp8_weight, qn_adamw_tensor, qn_adamw_plan))
    lin = [fp, vp, i64, vp, vp, i32, f32, vp, vp, vp, sz, vp]
    sig.update({
        "fp8_quantize_blocks": (ctypes.c_int, [vp, i32, i64, i64, vp, vp, vp]),
        "fp8_quantize_rows": (ctypes.c_int, [vp, i64, i64, vp, vp, vp]),
        "fp8_dequant": (ctypes.c_int, [fp, i32, vp, vp]),
        "fp8_matmul": (ctypes.c_int, [fp, vp, vp, i64, i32, vp, vp, sz, vp]),
        "fp8_linear_fwd": (ctypes.c_int, lin),
        "fp8_linear_bwd_dx": (ctypes.c_int, lin),
        "lora_adamw_table_bytes": (sz, [ap, i32]),
        "lora_adamw_table": (ctypes.c_int, [ap, i32, i32, i32, vp, sz, pp]),
        "lora_grad_norm_workspace_bytes": (sz, [pp]),
        "lora_grad_norm": (ctypes.c_int, [pp, vp, f32, vp, vp, sz, vp]),
        "lora_adamw_multi_step": (ctypes.c_int, [pp, vp, vp, f32, f32, f32, f32, f32, i32, vp]),
    })
    mp = ctypes.POINTER(qn_mxfp4_weight)
    lin = [mp, vp, i64, vp, vp, i32, f32, vp, vp, vp, sz, vp]
    sig.update({
        "mxfp4_scale_bytes": (sz, [i64, i64]),
        "mxfp4_quantize": (ctypes.c_int, [vp, i32, i64, i64, vp, vp, vp]),
        "mxfp4_dequant": (ctypes.c_int, [vp, vp, i64, i64, i32, vp, vp]),
        "mxfp4_pack_scales": (ctypes.c_int, [vp, i64, i64, vp, vp]),
        "mxfp4_unpack_scales": (ctypes.c_int, [vp, i64, i64, vp, vp]),
        "mxfp4_matmul": (ctypes.c_int, [mp, vp, vp, i64, vp, vp, sz, vp]),
        "mxfp4_linear_fwd": (ctypes.c_int, lin),
        "mxfp4_linear_bwd_dx": (ctypes.c_int, lin),
    })
    tp, pp, sp = (ctypes.POINTER(c) for c in (qn_muon_tensor, qn_muon_plan, qn_muon_step))
    sig.update({
        "lora_muon_table_bytes": (sz, [tp, i32]),
        "lora_muon_table": (ctypes.c_int, [tp, i32, i32, vp, sz, pp]),
        "lora_muon_workspace_bytes": (sz, [pp]),
        "lora_muon_multi_step": (ctypes.c_int, [pp, vp, sp, vp, sz, vp]),
    })
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(fn, status):
    if status != QN_OK:
        msg = load_library().qn_status_string(status).decode()
        raise QnError(fn, status, msg)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, dtype, numel=None, name="tensor"):
    torch = _torch()
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous() or t.dtype != dtype:
        raise ValueError(f"{name}: need a contiguous {dtype} device tensor")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
    return t


QN_NF4, QN_FP4 = 0, 1
QN_SCALE_U8, QN_SCALE_FP8, QN_SCALE_CENTRED = 0, 1, 2
_QUANT_TYPES = {"nf4": QN_NF4, "fp4": QN_FP4}
_SCALE_TYPES = {"u8": QN_SCALE_U8, "fp8": QN_SCALE_FP8, "centred": QN_SCALE_CENTRED}


class QuantWeight:
    """Device tensors of a 4-bit weight W[N, K] (+ double-quantised constants).

    packed uint8[N*K/2]; qscale uint8[N*K/64] and gscale fp32[ceil(N*K/64/256)]
    when double-quantised, else absmax fp32[N*K/64].  quant_type "nf4" or
    "fp4" (the code table), scale_type "u8", "fp8" or "centred" (the level-2
    code; "centred" also carries offset, fp32[1], the subtracted mean).
    """

    def __init__(self, packed, N, K, qscale=None, gscale=None, absmax=None, quant_type="nf4",
                 scale_type="u8", offset=None):
        self.packed, self.qscale, self.gscale, self.absmax = packed, qscale, gscale, absmax
        self.N, self.K = int(N), int(K)
        self.quant_type, self.scale_type = quant_type, scale_type
        self.offset = offset

    def c_struct(self):
        return qn_weight(self.packed.data_ptr(),
                         None if self.qscale is None else self.qscale.data_ptr(),
                         None if self.gscale is None else self.gscale.data_ptr(),
                         None if self.absmax is None else self.absmax.data_ptr(),
                         self.N, self.K, BLOCKSIZE, GROUP, _QUANT_TYPES[self.quant_type],
                         _SCALE_TYPES[self.scale_type],
                         None if self.offset is None else self.offset.data_ptr())


def nf4_codebook():
    """The 16 fp32 NF4 code points (host call), as a list of floats."""
    out = (ctypes.c_float * 16)()
    _check("nf4_codebook", load_library().nf4_codebook(out))
    return list(out)


def fp4_codebook():
    """The 16 fp32 FP4 code points (host call), as a list of floats."""
    out = (ctypes.c_float * 16)()
    _check("fp4_codebook", load_library().fp4_codebook(out))
    return list(out)


def nf4_quantize(w, packed=None, absmax=None, stream=None):
    """Blockwise NF4 quantisation of a fp32 or bf16 device tensor (flattened).

    Returns (packed uint8[numel/2], absmax fp32[ceil(numel/64)]).
    """
    return _quantize("nf4_quantize", w, packed, absmax, stream)


def fp4_quantize(w, packed=None, absmax=None, stream=None):
    """nf4_quantize with the FP4 code table."""
    return _quantize("fp4_quantize", w, packed, absmax, stream)


def nf4_quantize_dq(w, quant_type="nf4", scale_type="u8", packed=None, qscale=None, gscale=None,
                    absmax=None, stream=None):
    """Quantisation and double quantisation in one launch: returns (packed,
    qscale, gscale); the block constants are written to absmax only when a
    tensor is given for them."""
    torch = _torch()
    lib = load_library()
    if quant_type not in _QUANT_TYPES or scale_type not in ("u8", "fp8"):
        raise ValueError("quant_type must be 'nf4' or 'fp4', scale_type 'u8' or 'fp8'")
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("nf4_quantize_dq: weights must be float32 or bfloat16")
    _dev(w, w.dtype, name="w")
    n = w.numel()
    nb = -(-n // BLOCKSIZE)
    ng = -(-nb // GROUP)
    dev = w.device
    packed = torch.empty(n // 2, dtype=torch.uint8, device=dev) if packed is None else packed
    qscale = torch.empty(nb, dtype=torch.uint8, device=dev) if qscale is None else qscale
    gscale = torch.empty(ng, dtype=torch.float32, device=dev) if gscale is None else gscale
    _dev(packed, torch.uint8, n // 2, "packed")
    _dev(qscale, torch.uint8, nb, "qscale")
    _dev(gscale, torch.float32, ng, "gscale")
    _dev(absmax, torch.float32, nb, "absmax")
    dt = QN_F32 if w.dtype == torch.float32 else QN_BF16
    _check("nf4_quantize_dq", lib.nf4_quantize_dq(
        _ptr(w), dt, n, BLOCKSIZE, GROUP, _QUANT_TYPES[quant_type], _SCALE_TYPES[scale_type],
        _ptr(packed), _ptr(absmax), _ptr(qscale), _ptr(gscale), _stream(stream)))
    return packed, qscale, gscale


def nf4_quantize_dq_batch(ws, quant_type="nf4", scale_type="u8", outs=None, absmax=None,
                          stream=None):
    """nf4_quantize_dq over up to 8 weights of one dtype in one launch:
    returns a list of (packed, qscale, gscale), one per weight.  outs, if
    given, holds such triples to write into; absmax, if given, a list of
    fp32 tensors (or None entries) for the block constants."""
    torch = _torch()
    lib = load_library()
    if quant_type not in _QUANT_TYPES or scale_type not in ("u8", "fp8"):
        raise ValueError("quant_type must be 'nf4' or 'fp4', scale_type 'u8' or 'fp8'")
    n = len(ws)
    if n == 0:
        return []
    dtypes = {w.dtype for w in ws}
    if len(dtypes) != 1 or dtypes.pop() not in (torch.float32, torch.bfloat16):
        raise ValueError("nf4_quantize_dq_batch: weights must all be float32 or all bfloat16")
    res = []
    for i, w in enumerate(ws):
        _dev(w, w.dtype, name="w")
        m = w.numel()
        nb = -(-m // BLOCKSIZE)
        ng = -(-nb // GROUP)
        dev = w.device
        if outs is not None:
            packed, qscale, gscale = outs[i]
        else:
            packed = torch.empty(m // 2, dtype=torch.uint8, device=dev)
            qscale = torch.empty(nb, dtype=torch.uint8, device=dev)
            gscale = torch.empty(ng, dtype=torch.float32, device=dev)
        _dev(packed, torch.uint8, m // 2, "packed")
        _dev(qscale, torch.uint8, nb, "qscale")
        _dev(gscale, torch.float32, ng, "gscale")
        if absmax is not None:
            _dev(absmax[i], torch.float32, nb, "absmax")
        res.append((packed, qscale, gscale))
    vpa = ctypes.c_void_p * n
    wa = vpa(*[_ptr(w) for w in ws])
    na = (ctypes.c_int64 * n)(*[w.numel() for w in ws])
    pa = vpa(*[_ptr(r[0]) for r in res])
    qa = vpa(*[_ptr(r[1]) for r in res])
    ga = vpa(*[_ptr(r[2]) for r in res])
    aa = vpa(*[_ptr(a) for a in absmax]) if absmax is not None else None
    dt = QN_F32 if ws[0].dtype == torch.float32 else QN_BF16
    _check("nf4_quantize_dq_batch", lib.nf4_quantize_dq_batch(
        n, wa, na, dt, BLOCKSIZE, GROUP, _QUANT_TYPES[quant_type], _SCALE_TYPES[scale_type],
        pa, aa, qa, ga, _stream(stream)))
    return res


def quantize_weights(ws, stream=None, quant_type="nf4", scale_type="u8"):
    """Double-quantised QuantWeight of each [N, K] tensor in ws (one dtype),
    at most 8 per launch (nf4_quantize_dq_batch)."""
    out = []
    for i in range(0, len(ws), 8):
        part = ws[i:i + 8]
        for w, (packed, qscale, gscale) in zip(part, nf4_quantize_dq_batch(
                part, quant_type, scale_type, stream=stream)):
            out.append(QuantWeight(packed, w.shape[0], w.shape[1], qscale=qscale, gscale=gscale,
                                   quant_type=quant_type, scale_type=scale_type))
    return out


def _quantize(fn, w, packed, absmax, stream):
    torch = _torch()
    lib = load_library()
    if w.dtype == torch.float32:
        dt = QN_F32
    elif w.dtype == torch.bfloat16:
        dt = QN_BF16
    else:
        raise ValueError(f"{fn}: weights must be float32 or bfloat16")
    _dev(w, w.dtype, name="w")
    n = w.numel()
    nb = -(-n // BLOCKSIZE)
    if packed is None:
        packed = torch.empty(n // 2, dtype=torch.uint8, device=w.device)
    if absmax is None:
        absmax = torch.empty(nb, dtype=torch.float32, device=w.device)
    _dev(packed, torch.uint8, n // 2, "packed")
    _dev(absmax, torch.float32, nb, "absmax")
    _check(fn, getattr(lib, fn)(_ptr(w), dt, n, BLOCKSIZE, _ptr(packed), _ptr(absmax),
                                _stream(stream)))
    return packed, absmax


def dq_quantize_scales(absmax, qscale=None, gscale=None, stream=None, fp8=False):
    """Double quantisation: returns (qscale uint8[nb], gscale fp32[ceil(nb/256)]);
    fp8 selects the E4M3 level-2 code (dq_quantize_scales_fp8)."""
    torch = _torch()
    lib = load_library()
    _dev(absmax, torch.float32, name="absmax")
    nb = absmax.numel()
    ng = -(-nb // GROUP)
    if qscale is None:
        qscale = torch.empty(nb, dtype=torch.uint8, device=absmax.device)
    if gscale is None:
        gscale = torch.empty(ng, dtype=torch.float32, device=absmax.device)
    _dev(qscale, torch.uint8, nb, "qscale")
    _dev(gscale, torch.float32, ng, "gscale")
    fn = "dq_quantize_scales_fp8" if fp8 else "dq_quantize_scales"
    _check(fn, getattr(lib, fn)(_ptr(absmax), nb, GROUP, _ptr(qscale), _ptr(gscale),
                                _stream(stream)))
    return qscale, gscale


def dq_quantize_scales_centred(absmax, qscale=None, gscale=None, offset=None, stream=None):
    """Mean-centred double quantisation: returns (qscale uint8[nb] (signed
    codes), gscale fp32[ceil(nb/256)], offset fp32[1])."""
    torch = _torch()
    lib = load_library()
    _dev(absmax, torch.float32, name="absmax")
    nb = absmax.numel()
    ng = -(-nb // GROUP)
    dev = absmax.device
    qscale = torch.empty(nb, dtype=torch.uint8, device=dev) if qscale is None else qscale
    gscale = torch.empty(ng, dtype=torch.float32, device=dev) if gscale is None else gscale
    offset = torch.empty(1, dtype=torch.float32, device=dev) if offset is None else offset
    _dev(qscale, torch.uint8, nb, "qscale")
    _dev(gscale, torch.float32, ng, "gscale")
    _dev(offset, torch.float32, 1, "offset")
    _check("dq_quantize_scales_centred", lib.dq_quantize_scales_centred(
        _ptr(absmax), nb, GROUP, _ptr(qscale), _ptr(gscale), _ptr(offset), _stream(stream)))
    return qscale, gscale, offset


def quantize_weight(w, double_quant=True, stream=None, quant_type="nf4", scale_type="u8"):
    """4-bit quantisation (+ double quantisation) of a [N, K] tensor -> QuantWeight.

    quant_type "nf4" (nf4_quantize) or "fp4" (fp4_quantize); scale_type "u8"
    (dq_quantize_scales), "fp8" (dq_quantize_scales_fp8) or "centred"
    (dq_quantize_scales_centred)."""
    if quant_type not in _QUANT_TYPES or scale_type not in _SCALE_TYPES:
        raise ValueError("quant_type must be 'nf4' or 'fp4', scale_type 'u8', 'fp8' or "
                         "'centred'")
    N, K = w.shape
    if double_quant and scale_type != "centred":
        packed, qscale, gscale = nf4_quantize_dq(w, quant_type, scale_type, stream=stream)
        return QuantWeight(packed, N, K, qscale=qscale, gscale=gscale, quant_type=quant_type,
                           scale_type=scale_type)
    quant = fp4_quantize if quant_type == "fp4" else nf4_quantize
    packed, absmax = quant(w, stream=stream)
    if not double_quant:
        return QuantWeight(packed, N, K, absmax=absmax, quant_type=quant_type)
    qscale, gscale, offset = dq_quantize_scales_centred(absmax, stream=stream)
    return QuantWeight(packed, N, K, qscale=qscale, gscale=gscale, quant_type=quant_type,
                       scale_type=scale_type, offset=offset)


def nf4_dequant(qw, out_dtype=None, out=None, stream=None):
    """Materialise W[N, K] as fp32 or bf16."""
    torch = _torch()
    lib = load_library()
    out_dtype = out_dtype or torch.bfloat16
    dt = QN_BF16 if out_dtype == torch.bfloat16 else QN_F32
    if out is None:
        out = torch.empty((qw.N, qw.K), dtype=out_dtype, device=qw.packed.device)
    _dev(out, out_dtype, qw.N * qw.K, "out")
    cw = qw.c_struct()
    _check("nf4_dequant", lib.nf4_dequant(ctypes.byref(cw), dt, _ptr(out), _stream(stream)))
    return out


def qn_workspace_bytes(op, M, N, K, r):
    return int(load_library().qn_workspace_bytes(op, M, N, K, r))


def workspace(nbytes, device):
    """A uint8 device workspace of nbytes for the linear ops."""
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device)


def _workspace(op, M, N, K, r, ws, device):
    need = qn_workspace_bytes(op, M, N, K, r)
    if ws is None and need > 0:
        ws = workspace(need, device)
    return ws, (0 if ws is None else ws.numel())


def qlora_linear_fwd(qw, x, A, B, r, alpha, y=None, u_out=None, ws=None, stream=None):
    """y = x W^T + (alpha/r) (x A^T) B^T  (bf16 in/out)."""
    return _fwd(qw, x, None, A, B, r, alpha, y, u_out, ws, stream)


def qlora_linear_fwd_dropout(qw, x, x_drop, A, B, r, alpha, y=None, u_out=None, ws=None,
                             stream=None):
    """y = x W^T + (alpha/r) (x_drop A^T) B^T, x_drop from lora_dropout."""
    return _fwd(qw, x, x_drop, A, B, r, alpha, y, u_out, ws, stream)


def hbm_read_probe(buf, sink, stream=None):
    """Streaming read of a contiguous device tensor (a measurement aid);
    sink is a device tensor of at least 4 bytes."""
    if not buf.is_cuda or not buf.is_contiguous() or not sink.is_cuda:
        raise ValueError("hbm_read_probe: contiguous device tensors required")
    nbytes = buf.numel() * buf.element_size()
    _check("qn_hbm_read_probe", load_library().qn_hbm_read_probe(
        _ptr(buf), nbytes - nbytes % 16, _ptr(sink), _stream(stream)))


def qlora_linear_fwd_noalloc(qw, x, A, B, r, alpha, y, u_out=None, stream=None):
    """qlora_linear_fwd on the library's own scratch array: y (and u_out)
    must be given; the call allocates nothing."""
    torch = _torch()
    lib = load_library()
    M = x.shape[0]
    _dev(x, torch.bfloat16, M * qw.K, "x")
    if r:
        _dev(A, torch.bfloat16, r * qw.K, "A")
        _dev(B, torch.bfloat16, qw.N * r, "B")
    if y is None:
        raise ValueError("y: the allocation-free forward writes into a given tensor")
    _dev(y, torch.bfloat16, M * qw.N, "y")
    _dev(u_out, torch.bfloat16, M * r, "u_out")
    cw = qw.c_struct()
    a, b = (_ptr(A), _ptr(B)) if r else (None, None)
    _check("qlora_linear_fwd_noalloc", lib.qlora_linear_fwd_noalloc(
        ctypes.byref(cw), _ptr(x), M, a, b, r, float(alpha), _ptr(y), _ptr(u_out),
        _stream(stream)))
    return y


def _fwd(qw, x, x_drop, A, B, r, alpha, y, u_out, ws, stream):
    torch = _torch()
    lib = load_library()
    M = x.shape[0]
    _dev(x, torch.bfloat16, M * qw.K, "x")
    _dev(x_drop, torch.bfloat16, M * qw.K, "x_drop")
    if r:
        _dev(A, torch.bfloat16, r * qw.K, "A")
        _dev(B, torch.bfloat16, qw.N * r, "B")
    if y is None:
        y = torch.empty((M, qw.N), dtype=torch.bfloat16, device=x.device)
    _dev(y, torch.bfloat16, M * qw.N, "y")
    _dev(u_out, torch.bfloat16, M * r, "u_out")
    ws, wsb = _workspace(QN_OP_FWD, M, qw.N, qw.K, r, ws, x.device)
    cw = qw.c_struct()
    a, b = (_ptr(A), _ptr(B)) if r else (None, None)
    if x_drop is None:
        _check("qlora_linear_fwd", lib.qlora_linear_fwd(
            ctypes.byref(cw), _ptr(x), M, a, b, r, float(alpha), _ptr(y), _ptr(u_out), _ptr(ws),
            wsb, _stream(stream)))
    else:
        _check("qlora_linear_fwd_dropout", lib.qlora_linear_fwd_dropout(
            ctypes.byref(cw), _ptr(x), _ptr(x_drop), M, a, b, r, float(alpha), _ptr(y),
            _ptr(u_out), _ptr(ws), wsb, _stream(stream)))
    return y


def qlora_linear_bwd_dx(qw, dy, A, B, r, alpha, dx=None, t_out=None, ws=None, stream=None):
    """dx = dy W + (alpha/r) (dy B) A  (bf16 in/out)."""
    return _bwd(qw, dy, A, B, r, alpha, None, 0, dx, t_out, ws, stream)


def qlora_linear_bwd_dx_dropout(qw, dy, A, B, r, alpha, p, seed, dx=None, t_out=None, ws=None,
                                stream=None):
    """dx = dy W + keep/(1-p) * ((alpha/r) (dy B) A), the mask of lora_dropout(p, seed)."""
    return _bwd(qw, dy, A, B, r, alpha, p, seed, dx, t_out, ws, stream)


def _bwd(qw, dy, A, B, r, alpha, p, seed, dx, t_out, ws, stream):
    torch = _torch()
    lib = load_library()
    M = dy.shape[0]
    _dev(dy, torch.bfloat16, M * qw.N, "dy")
    if r:
        _dev(A, torch.bfloat16, r * qw.K, "A")
        _dev(B, torch.bfloat16, qw.N * r, "B")
    if dx is None:
        dx = torch.empty((M, qw.K), dtype=torch.bfloat16, device=dy.device)
    _dev(dx, torch.bfloat16, M * qw.K, "dx")
    _dev(t_out, torch.bfloat16, M * r, "t_out")
    ws, wsb = _workspace(QN_OP_BWD_DX if p is None else QN_OP_BWD_DX_DROPOUT, M, qw.N, qw.K, r,
                         ws, dy.device)
    cw = qw.c_struct()
    a, b = (_ptr(A), _ptr(B)) if r else (None, None)
    if p is None:
        _check("qlora_linear_bwd_dx", lib.qlora_linear_bwd_dx(
            ctypes.byref(cw), _ptr(dy), M, a, b, r, float(alpha), _ptr(dx), _ptr(t_out),
            _ptr(ws), wsb, _stream(stream)))
    else:
        _check("qlora_linear_bwd_dx_dropout", lib.qlora_linear_bwd_dx_dropout(
            ctypes.byref(cw), _ptr(dy), M, a, b, r, float(alpha), float(p), int(seed), _ptr(dx),
            _ptr(t_out), _ptr(ws), wsb, _stream(stream)))
    return dx


def lora_dropout(x, p, seed, out=None, stream=None):
    """The LoRA branch's dropped input bf16[M, K]: x * keep / (1 - p), Philox mask."""
    torch = _torch()
    lib = load_library()
    M, K = x.shape
    _dev(x, torch.bfloat16, M * K, "x")
    if out is None:
        out = torch.empty_like(x)
    _dev(out, torch.bfloat16, M * K, "out")
    _check("lora_dropout", lib.lora_dropout(_ptr(x), M, K, float(p), int(seed), _ptr(out),
                                            _stream(stream)))
    return out


def lora_grads(x, dy, A, B, r, alpha, u=None, t=None, dA=None, dB=None, ws=None, stream=None):
    """(dA fp32[r, K], dB fp32[N, r]) = ((alpha/r) (dy B)^T x, (alpha/r) dy^T (x A^T))."""
    torch = _torch()
    lib = load_library()
    M, K = x.shape
    N = dy.shape[1]
    _dev(x, torch.bfloat16, M * K, "x")
    _dev(dy, torch.bfloat16, M * N, "dy")
    _dev(A, torch.bfloat16, r * K, "A")
    _dev(B, torch.bfloat16, N * r, "B")
    _dev(u, torch.bfloat16, M * r, "u")
    _dev(t, torch.bfloat16, M * r, "t")
    if dA is None:
        dA = torch.empty((r, K), dtype=torch.float32, device=x.device)
    if dB is None:
        dB = torch.empty((N, r), dtype=torch.float32, device=x.device)
    _dev(dA, torch.float32, r * K, "dA")
    _dev(dB, torch.float32, N * r, "dB")
    ws, wsb = _workspace(QN_OP_LORA_GRADS, M, N, K, r, ws, x.device)
    _check("lora_grads", lib.lora_grads(
        _ptr(x), _ptr(dy), _ptr(u), _ptr(t), _ptr(A), _ptr(B), M, N, K, r, float(alpha),
        _ptr(dA), _ptr(dB), _ptr(ws), wsb, _stream(stream)))
    return dA, dB


def qlora_merge(qw, A, B, r, alpha, out=None, stream=None):
    """Merged 16-bit weight bf16[N, K] = bf16(dequant(W) + (alpha/r) B A)."""
    torch = _torch()
    lib = load_library()
    N, K = qw.N, qw.K
    if r:
        _dev(A, torch.bfloat16, r * K, "A")
        _dev(B, torch.bfloat16, N * r, "B")
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=qw.packed.device)
    _dev(out, torch.bfloat16, N * K, "out")
    cw = qw.c_struct()
    _check("qlora_merge", lib.qlora_merge(ctypes.byref(cw), _ptr(A) if r else None,
                                          _ptr(B) if r else None, r, float(alpha), _ptr(out),
                                          _stream(stream)))
    return out


def lora_adamw_step(p, g, m, v, step, lr=2e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                    p_bf16=None, stream=None):
    """In-place AdamW step on fp32 p, m, v with gradient g; optionally writes
    bf16(p) to p_bf16.  Returns p."""
    torch = _torch()
    lib = load_library()
    n = p.numel()
    for t, name in ((p, "p"), (g, "g"), (m, "m"), (v, "v")):
        _dev(t, torch.float32, n, name)
    if p_bf16 is not None:
        _dev(p_bf16, torch.bfloat16, n, "p_bf16")
    _check("lora_adamw_step", lib.lora_adamw_step(
        _ptr(p), _ptr(g), _ptr(m), _ptr(v), _ptr(p_bf16), n, float(lr), float(betas[0]),
        float(betas[1]), float(eps), float(weight_decay), int(step), _stream(stream)))
    return p


# --- block-scaled FP8 ------------------------------------------------------


def _fit(t, dtype, numel, dev, name):
    """_dev, and on the device dev (one pass: these checks run on every call of
    a decode step)."""
    if t.dtype is not dtype or t.numel() != numel or t.device != dev or not t.is_contiguous():
        _dev(t, dtype, numel, name)
        raise ValueError(f"{name}: on {t.device}, other tensors of the call on {dev}")


def _call(fn, dev, stream, *args):
    """Call a library function with dev current, on the given stream of dev
    or on its current one."""
    torch = _torch()
    f = getattr(load_library(), fn)
    at = dev.index
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(at)
    elif stream.device != dev:
        raise ValueError(f"{fn}: the stream belongs to {stream.device}, the tensors to {dev}")
    else:
        s = stream.cuda_stream
    if torch._C._cuda_getDevice() == at:
        status = f(*args, s)
    else:
        with torch.cuda.device(dev):
            status = f(*args, s)
    if status != QN_OK:
        _check(fn, status)


def _new(stream, dtype, dev, *shape):
    """A tensor for a call on the given stream: in that stream's memory, so
    that neither earlier nor later work of the current stream shares it."""
    torch = _torch()
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=dev)


def _addr(t):
    return None if t is None else t.data_ptr()


class Fp8Weight:
    """Device tensors of an 8-bit weight W[N, K]: codes float8_e4m3fn[N, K]
    and scale fp32[ceil(N/128), ceil(K/128)], one per 128 x 128 block."""

    def __init__(self, codes, scale):
        torch = _torch()
        if codes.dim() != 2:
            raise ValueError("codes: need a matrix [N, K]")
        N, K = self.N, self.K = codes.shape
        dev = self.device = codes.device
        _dev(codes, torch.float8_e4m3fn, name="codes")
        _fit(scale, torch.float32, -(-N // FP8_BLOCK) * -(-K // FP8_BLOCK), dev, "scale")
        self.codes, self.scale = codes, scale

    def c_struct(self):
        return qn_fp8_weight(self.codes.data_ptr(), self.scale.data_ptr(), self.N, self.K)


def fp8_quantize_blocks(w, codes=None, scale=None, stream=None):
    """E4M3 codes float8_e4m3fn[N, K] and the scale of each 128 x 128 block,
    fp32[ceil(N/128), ceil(K/128)], of a fp32 or bf16 matrix."""
    torch = _torch()
    if w.dim() != 2 or w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("fp8_quantize_blocks: need a float32 or bfloat16 matrix")
    _dev(w, w.dtype, name="w")
    N, K = w.shape
    nb, kb = -(-N // FP8_BLOCK), -(-K // FP8_BLOCK)
    if codes is None:
        codes = _new(stream, torch.float8_e4m3fn, w.device, N, K)
    else:
        _fit(codes, torch.float8_e4m3fn, N * K, w.device, "codes")
    if scale is None:
        scale = _new(stream, torch.float32, w.device, nb, kb)
    else:
        _fit(scale, torch.float32, nb * kb, w.device, "scale")
    _call("fp8_quantize_blocks", w.device, stream, w.data_ptr(),
          QN_F32 if w.dtype == torch.float32 else QN_BF16, N, K, codes.data_ptr(),
          scale.data_ptr())
    return codes, scale


def fp8_quantize_weight(w, stream=None):
    """The Fp8Weight of a fp32 or bf16 matrix [N, K] (fp8_quantize_blocks)."""
    return Fp8Weight(*fp8_quantize_blocks(w, stream=stream))


def fp8_quantize_rows(x, codes=None, scale=None, stream=None):
    """E4M3 codes float8_e4m3fn[M, K] and scales fp32[ceil(K/128), M] of a
    bf16 matrix, one scale per 128 columns of a row."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x: need a matrix [M, K]")
    M, K = x.shape
    kb = -(-K // FP8_BLOCK)
    _dev(x, torch.bfloat16, name="x")
    if codes is None:
        codes = _new(stream, torch.float8_e4m3fn, x.device, M, K)
    else:
        _fit(codes, torch.float8_e4m3fn, M * K, x.device, "codes")
    if scale is None:
        scale = _new(stream, torch.float32, x.device, kb, M)
    else:
        _fit(scale, torch.float32, kb * M, x.device, "scale")
    _call("fp8_quantize_rows", x.device, stream, x.data_ptr(), M, K, codes.data_ptr(),
          scale.data_ptr())
    return codes, scale


def fp8_dequant(fw, out_dtype=None, out=None, stream=None):
    """Materialise an Fp8Weight as fp32 or bf16 [N, K]."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("fp8_dequant: out_dtype must be float32 or bfloat16")
    dev = fw.device
    if out is None:
        out = _new(stream, out_dtype, dev, fw.N, fw.K)
    else:
        _fit(out, out_dtype, fw.N * fw.K, dev, "out")
    _call("fp8_dequant", dev, stream, fw.c_struct(),
          QN_BF16 if out_dtype == torch.bfloat16 else QN_F32, out.data_ptr())
    return out


def fp8_matmul(fw, codes, scale, transposed=False, out=None, ws=None, stream=None):
    """x W^T (bf16[M, N]) of x [M, K] from fp8_quantize_rows, or with
    transposed x W (bf16[M, K]) of x [M, N]."""
    torch = _torch()
    L, n = (fw.N, fw.K) if transposed else (fw.K, fw.N)
    if codes.dim() != 2 or codes.shape[1] != L:
        raise ValueError(f"codes: need [M, {L}]")
    M = codes.shape[0]
    dev = fw.device
    _fit(codes, torch.float8_e4m3fn, M * L, dev, "codes")
    _fit(scale, torch.float32, -(-L // FP8_BLOCK) * M, dev, "scale")
    if out is None:
        out = _new(stream, torch.bfloat16, dev, M, n)
    else:
        _fit(out, torch.bfloat16, M * n, dev, "out")
    if ws is None:
        op = QN_OP_FP8_BWD_DX if transposed else QN_OP_FP8_FWD
        ws = _new(stream, torch.uint8, dev, qn_workspace_bytes(op, M, fw.N, fw.K, 0))
    else:
        _fit(ws, torch.uint8, ws.numel(), dev, "ws")
    _call("fp8_matmul", dev, stream, fw.c_struct(), codes.data_ptr(), scale.data_ptr(), M,
          int(bool(transposed)), out.data_ptr(), ws.data_ptr(), ws.numel())
    return out


def fp8_linear_fwd(fw, x, A, B, r, alpha, y=None, u_out=None, ws=None, stream=None):
    """y = Q(x) W^T + (alpha/r) (x A^T) B^T on an Fp8Weight (bf16 in/out)."""
    return _scaled_linear("fp8_linear_fwd", QN_OP_FP8_FWD, fw, x, fw.K, fw.N, A, B, r, alpha, y,
                          u_out, ws, stream)


def fp8_linear_bwd_dx(fw, dy, A, B, r, alpha, dx=None, t_out=None, ws=None, stream=None):
    """dx = Q(dy) W + (alpha/r) (dy B) A on an Fp8Weight (bf16 in/out)."""
    return _scaled_linear("fp8_linear_bwd_dx", QN_OP_FP8_BWD_DX, fw, dy, fw.N, fw.K, A, B, r, alpha,
                          dx, t_out, ws, stream)


def _scaled_linear(fn, op, fw, x, L, n, A, B, r, alpha, out, low, ws, stream):
    """A layer on an Fp8Weight or an Mxfp4Weight."""
    torch = _torch()
    bf16, dev = torch.bfloat16, fw.device
    M = x.shape[0]
    fwd = op in (QN_OP_FP8_FWD, QN_OP_MXFP4_FWD)
    _fit(x, bf16, M * L, dev, "x" if fwd else "dy")
    a = b = None
    if r and A is not None:
        _fit(A, bf16, r * fw.K, dev, "A")
        a = A.data_ptr()
    if r and B is not None:
        _fit(B, bf16, fw.N * r, dev, "B")
        b = B.data_ptr()
    if out is None:
        out = _new(stream, bf16, dev, M, n)
    else:
        _fit(out, bf16, M * n, dev, "y" if fwd else "dx")
    if low is not None:
        _fit(low, bf16, M * r, dev, "u_out" if fwd else "t_out")
    if ws is None:
        ws = _new(stream, torch.uint8, dev, qn_workspace_bytes(op, M, fw.N, fw.K, r))
    else:
        _fit(ws, torch.uint8, ws.numel(), dev, "ws")
    _call(fn, dev, stream, fw.c_struct(), x.data_ptr(), M, a, b, r, alpha, out.data_ptr(),
          _addr(low), ws.data_ptr(), ws.numel())
    return out


# --- microscaled 4-bit ------------------------------------------------------


def mxfp4_scale_bytes(R, K):
    """Bytes of the scales of an MXFP4 matrix [R, K]."""
    return int(load_library().mxfp4_scale_bytes(R, K))


class Mxfp4Weight:
    """Device tensors of a microscaled 4-bit weight W[N, K]: codes
    uint8[N, K/2] (E2M1, the even column in the low half of a byte) and scale
    uint8[mxfp4_scale_bytes(N, K)], in tiles (mxfp4_pack_scales)."""

    def __init__(self, codes, scale):
        torch = _torch()
        if codes.dim() != 2:
            raise ValueError("codes: need a matrix [N, K / 2]")
        N, K = self.N, self.K = codes.shape[0], 2 * codes.shape[1]
        dev = self.device = codes.device
        _dev(codes, torch.uint8, name="codes")
        _fit(scale, torch.uint8, mxfp4_scale_bytes(N, K), dev, "scale")
        self.codes, self.scale = codes, scale

    def c_struct(self):
        return qn_mxfp4_weight(self.codes.data_ptr(), self.scale.data_ptr(), self.N, self.K)


def mxfp4_quantize(x, codes=None, scale=None, stream=None):
    """E2M1 codes uint8[R, K/2] and scales uint8[mxfp4_scale_bytes(R, K)] of a
    fp32 or bf16 matrix [R, K], one power of two per 32 columns of a row."""
    torch = _torch()
    if x.dim() != 2 or x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("mxfp4_quantize: need a float32 or bfloat16 matrix")
    _dev(x, x.dtype, name="x")
    R, K = x.shape
    if codes is None:
        codes = _new(stream, torch.uint8, x.device, R, K // 2)
    else:
        _fit(codes, torch.uint8, R * K // 2, x.device, "codes")
    size = mxfp4_scale_bytes(R, K)
    if scale is None:
        scale = _new(stream, torch.uint8, x.device, size)
    else:
        _fit(scale, torch.uint8, size, x.device, "scale")
    _call("mxfp4_quantize", x.device, stream, x.data_ptr(),
          QN_F32 if x.dtype == torch.float32 else QN_BF16, R, K, codes.data_ptr(),
          scale.data_ptr())
    return codes, scale


def mxfp4_quantize_weight(w, stream=None):
    """The Mxfp4Weight of a fp32 or bf16 matrix [N, K] (mxfp4_quantize)."""
    return Mxfp4Weight(*mxfp4_quantize(w, stream=stream))


def mxfp4_pack_scales(rows, scale=None, stream=None):
    """Scales uint8[R, K/32], a byte per 32 columns of a row, as tiles."""
    torch = _torch()
    if rows.dim() != 2:
        raise ValueError("rows: need a matrix [R, K / 32]")
    _dev(rows, torch.uint8, name="rows")
    R, K = rows.shape[0], rows.shape[1] * MXFP4_GROUP
    size = mxfp4_scale_bytes(R, K)
    if scale is None:
        scale = _new(stream, torch.uint8, rows.device, size)
    else:
        _fit(scale, torch.uint8, size, rows.device, "scale")
    _call("mxfp4_pack_scales", rows.device, stream, rows.data_ptr(), R, K, scale.data_ptr())
    return scale


def mxfp4_unpack_scales(scale, R, K, rows=None, stream=None):
    """Scales uint8[R, K/32], a byte per 32 columns of a row, of tiles."""
    torch = _torch()
    dev = scale.device
    _dev(scale, torch.uint8, mxfp4_scale_bytes(R, K), "scale")
    if rows is None:
        rows = _new(stream, torch.uint8, dev, R, K // MXFP4_GROUP)
    else:
        _fit(rows, torch.uint8, R * (K // MXFP4_GROUP), dev, "rows")
    _call("mxfp4_unpack_scales", dev, stream, scale.data_ptr(), R, K, rows.data_ptr())
    return rows


def mxfp4_dequant(mw, out_dtype=None, out=None, stream=None):
    """The values of an Mxfp4Weight as bf16 or fp32 [N, K]."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("mxfp4_dequant: out_dtype must be float32 or bfloat16")
    dev = mw.device
    if out is None:
        out = _new(stream, out_dtype, dev, mw.N, mw.K)
    else:
        _fit(out, out_dtype, mw.N * mw.K, dev, "out")
    _call("mxfp4_dequant", dev, stream, mw.codes.data_ptr(), mw.scale.data_ptr(), mw.N, mw.K,
          QN_BF16 if out_dtype == torch.bfloat16 else QN_F32, out.data_ptr())
    return out


def mxfp4_matmul(mw, codes, scale, out=None, ws=None, stream=None):
    """x W^T (bf16[M, N]) of x [M, K] from mxfp4_quantize."""
    torch = _torch()
    if codes.dim() != 2 or 2 * codes.shape[1] != mw.K:
        raise ValueError(f"codes: need [M, {mw.K // 2}]")
    M, dev = codes.shape[0], mw.device
    _fit(codes, torch.uint8, M * mw.K // 2, dev, "codes")
    _fit(scale, torch.uint8, mxfp4_scale_bytes(M, mw.K), dev, "scale")
    if out is None:
        out = _new(stream, torch.bfloat16, dev, M, mw.N)
    else:
        _fit(out, torch.bfloat16, M * mw.N, dev, "out")
    if ws is None:
        ws = _new(stream, torch.uint8, dev, qn_workspace_bytes(QN_OP_MXFP4_FWD, M, mw.N, mw.K, 0))
    else:
        _fit(ws, torch.uint8, ws.numel(), dev, "ws")
    _call("mxfp4_matmul", dev, stream, mw.c_struct(), codes.data_ptr(), scale.data_ptr(), M,
          out.data_ptr(), ws.data_ptr(), ws.numel())
    return out


def mxfp4_linear_fwd(mw, x, A, B, r, alpha, y=None, u_out=None, ws=None, stream=None):
    """y = Q(x) W^T + (alpha/r) (x A^T) B^T on an Mxfp4Weight (bf16 in/out)."""
    return _scaled_linear("mxfp4_linear_fwd", QN_OP_MXFP4_FWD, mw, x, mw.K, mw.N, A, B, r, alpha, y,
                          u_out, ws, stream)


def mxfp4_linear_bwd_dx(mw, dy, A, B, r, alpha, dx=None, t_out=None, ws=None, stream=None):
    """dx = Q8(dy) W + (alpha/r) (dy B) A on an Mxfp4Weight (bf16 in/out)."""
    return _scaled_linear("mxfp4_linear_bwd_dx", QN_OP_MXFP4_BWD_DX, mw, dy, mw.N, mw.K, A, B, r,
                          alpha, dx, t_out, ws, stream)


# --- AdamW over many matrices ----------------------------------------------


class AdamwTable:
    """The device table of lora_adamw_multi_step and lora_grad_norm over the
    given matrices, which it keeps alive (their memory is updated in place)."""

    def __init__(self, plan, table, device, tensors):
        self.plan, self.table, self.device, self.tensors = plan, table, device, tensors


def lora_adamw_table(ps, gs, ms, vs, m_scales=None, v_scales=None, p_bf16s=None):
    """Table over matrices p (fp32) with gradients g (all fp32 or all bf16).

    States: m and v fp32, or m float8_e4m3fn and v float8_e5m2 with
    m_scales and v_scales fp32[ceil(n/256)] each (start all of them from
    zeros).  p_bf16s, if given, holds bf16 tensors (or None) that receive the
    new p.  Build it once; changed addresses or sizes need a new one."""
    torch = _torch()
    lib = load_library()
    n = len(ps)
    if not n:
        raise ValueError("lora_adamw_table: no matrices")
    for col, name in zip((ps, gs, ms, vs), ("p", "g", "m", "v")):
        if any(t is None for t in col):
            raise ValueError(f"{name}: missing")
    eight = ms[0].dtype != torch.float32
    none = [None] * n
    if eight and (m_scales is None or v_scales is None):
        raise ValueError("lora_adamw_table: 8-bit states need m_scales and v_scales")
    if not eight:
        m_scales = v_scales = none
    p_bf16s = none if p_bf16s is None else p_bf16s
    cols = [list(c) for c in (ps, gs, ms, vs, m_scales, v_scales, p_bf16s)]
    if any(len(c) != n for c in cols):
        raise ValueError("lora_adamw_table: lists of different lengths")
    gt = gs[0].dtype
    if gt not in (torch.float32, torch.bfloat16):
        raise ValueError("lora_adamw_table: gradients must be float32 or bfloat16")
    mt, vt = (torch.float8_e4m3fn, torch.float8_e5m2) if eight else (torch.float32,) * 2
    dev = ps[0].device
    _dev(ps[0], torch.float32, name="p")
    arr = (qn_adamw_tensor * n)()
    for i, row in enumerate(zip(*cols)):
        k = row[0].numel()
        blocks = -(-k // STATE_BLOCK)
        for t, dt, size, name in zip(row, (torch.float32, gt, mt, vt, torch.float32,
                                           torch.float32, torch.bfloat16),
                                     (k, k, k, k, blocks, blocks, k),
                                     ("p", "g", "m", "v", "m_scale", "v_scale", "p_bf16")):
            if t is None and eight and name in ("m_scale", "v_scale"):
                raise ValueError(f"{name}: missing")
            if t is not None:
                _fit(t, dt, size, dev, name)
        arr[i] = qn_adamw_tensor(*[_addr(t) for t in row], k)
    size = lib.lora_adamw_table_bytes(arr, n)
    host = torch.empty(max(size, 1), dtype=torch.uint8)
    plan = qn_adamw_plan()
    _check("lora_adamw_table", lib.lora_adamw_table(
        arr, n, QN_F32 if gt == torch.float32 else QN_BF16,
        QN_STATE_8BIT if eight else QN_STATE_F32, host.data_ptr(), size, ctypes.byref(plan)))
    return AdamwTable(plan, host.to(dev), dev, cols)


def lora_grad_norm_workspace_bytes(table):
    return int(load_library().lora_grad_norm_workspace_bytes(table.plan))


def lora_grad_norm(table, max_norm, out=None, ws=None, stream=None):
    """fp32[2]: the L2 norm of all gradients of a table and the coefficient
    min(1, max_norm / (norm + 1e-6)) (NaN if the norm is not finite)."""
    torch = _torch()
    dev = table.device
    if out is None:
        out = _new(stream, torch.float32, dev, 2)
    else:
        _fit(out, torch.float32, 2, dev, "out")
    if ws is None:
        ws = _new(stream, torch.uint8, dev, lora_grad_norm_workspace_bytes(table))
    else:
        _fit(ws, torch.uint8, ws.numel(), dev, "ws")
    _call("lora_grad_norm", dev, stream, table.plan, table.table.data_ptr(),
          max_norm, out.data_ptr(), ws.data_ptr(), ws.numel())
    return out


def lora_adamw_multi_step(table, step, lr=2e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                          grad_scale=None, stream=None):
    """One in-place AdamW step on every matrix of a table.  grad_scale, a
    device fp32[1] (lora_grad_norm's out[1:]), multiplies the gradients; a
    step with one that is not finite does nothing."""
    torch = _torch()
    dev = table.device
    if grad_scale is not None:
        _fit(grad_scale, torch.float32, 1, dev, "grad_scale")
    _call("lora_adamw_multi_step", dev, stream, table.plan, table.table.data_ptr(),
          _addr(grad_scale), lr, betas[0], betas[1], eps, weight_decay, step)


# --- Muon over many matrices -------------------------------------------------


class MuonTable:
    """The device table of lora_muon_multi_step over the given matrices, which it
    keeps alive (their memory is updated in place)."""

    def __init__(self, plan, table, device, tensors):
        self.plan, self.table, self.device, self.tensors = plan, table, device, tensors


def lora_muon_table(ps, gs, ms, p_bf16s=None):
    """Table over matrices p (fp32, the smaller side at most 128) with gradients g
    (all fp32 or all bf16) and momenta m (fp32, zeros at the start).  p_bf16s, if
    given, holds bf16 matrices (or None) that receive the new p.  Build it once;
    changed addresses or sizes need a new one."""
    torch = _torch()
    lib = load_library()
    n = len(ps)
    if not n:
        raise ValueError("lora_muon_table: no matrices")
    for col, name in zip((ps, gs, ms), ("p", "g", "m")):
        if any(t is None for t in col):
            raise ValueError(f"{name}: missing")
    cols = [list(c) for c in (ps, gs, ms, [None] * n if p_bf16s is None else p_bf16s)]
    if any(len(c) != n for c in cols):
        raise ValueError("lora_muon_table: lists of different lengths")
    gt = gs[0].dtype
    if gt not in (torch.float32, torch.bfloat16):
        raise ValueError("lora_muon_table: gradients must be float32 or bfloat16")
    dev = ps[0].device
    _dev(ps[0], torch.float32, name="p")
    arr = (qn_muon_tensor * n)()
    for i, row in enumerate(zip(*cols)):
        if row[0].dim() != 2:
            raise ValueError("p: need matrices")
        for t, dt, name in zip(row, (torch.float32, gt, torch.float32, torch.bfloat16),
                               ("p", "g", "m", "p_bf16")):
            if t is not None:
                _fit(t, dt, row[0].numel(), dev, name)
                if t.shape != row[0].shape:
                    raise ValueError(f"{name}: shape {tuple(t.shape)}, p has "
                                     f"{tuple(row[0].shape)}")
        arr[i] = qn_muon_tensor(*[_addr(t) for t in row], *row[0].shape)
    size = lib.lora_muon_table_bytes(arr, n)
    host = torch.empty(max(size, 1), dtype=torch.uint8)
    plan = qn_muon_plan()
    _check("lora_muon_table", lib.lora_muon_table(
        arr, n, QN_F32 if gt == torch.float32 else QN_BF16, host.data_ptr(), size,
        ctypes.byref(plan)))
    return MuonTable(plan, host.to(dev), dev, cols)


def lora_muon_workspace_bytes(table):
    return int(load_library().lora_muon_workspace_bytes(table.plan))


def lora_muon_multi_step(table, lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.1, eps=1e-7,
                         adjust="original", ns_coefficients=(3.4445, -4.775, 2.0315), ns_steps=5,
                         ws=None, stream=None):
    """One in-place Muon step on every matrix of a table.  adjust: "original"
    multiplies the orthogonal update by sqrt(max(1, rows / cols)),
    "match_rms_adamw" by 0.2 sqrt(max(rows, cols)).  abs(ns_coefficients[0]) ** (2 *
    ns_steps) may reach 2**43: 12 steps of the default."""
    torch = _torch()
    dev = table.device
    kinds = {"original": QN_MUON_ORIGINAL, "match_rms_adamw": QN_MUON_MATCH_RMS}
    if adjust not in kinds:
        raise ValueError(f"adjust: one of {sorted(kinds)}")
    if len(ns_coefficients) != 3:
        raise ValueError("ns_coefficients: need three")
    step = qn_muon_step(lr, momentum, weight_decay, eps,
                        (ctypes.c_double * 3)(*ns_coefficients), ns_steps, int(bool(nesterov)),
                        kinds[adjust])
    if ws is None:
        ws = _new(stream, torch.uint8, dev, lora_muon_workspace_bytes(table))
    else:
        _fit(ws, torch.uint8, ws.numel(), dev, "ws")
    _call("lora_muon_multi_step", dev, stream, table.plan, table.table.data_ptr(), step,
          ws.data_ptr(), ws.numel())
