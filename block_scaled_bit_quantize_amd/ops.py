"""PyTorch-facing wrappers of the bsq_* entry points (argument marshalling
only: shapes, output allocation, device pointers, the current stream)."""
import functools

import torch

from ._lib import BsqError, check, load_library

F32, BF16 = 0, 1
OUTER_TENSOR, OUTER_ROW, OUTER_GIVEN = 0, 1, 2
FOUR_OVER_SIX = 16  # flag OR-ed into the NVFP4 quantize mode
RN, SR = 0, 1
NVFP4, MXFP8 = 0, 1

_OUTER = {"tensor": OUTER_TENSOR, "row": OUTER_ROW, "given": OUTER_GIVEN}
_RND = {"rn": RN, "sr": SR}
_FMT = {"nvfp4": NVFP4, "mxfp8": MXFP8}


def _enum(v, table):
    return table[v] if isinstance(v, str) else int(v)


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object: 0.2 us where current_stream() takes 2.8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream():
    if _raw_stream is None or _raw_device is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_raw_device())


def _dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise BsqError("expected contiguous device tensors")


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=4096)
def _ws_bytes(name, index, *sizes):
    """A workspace query's answer for these sizes on device `index` (a decode loop asks the same again and again)."""
    if _raw_device is not None and _raw_device() == index:
        return getattr(load_library(), name)(*sizes)
    with torch.cuda.device(index):
        return getattr(load_library(), name)(*sizes)


def _run(name, first, others, *args):
    """Calls entry point `name` with args and the current stream of the tensors'
    device, which is made the current one for it; all tensors must be on it."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise BsqError("all tensors must be on one device")
    fn = getattr(load_library(), name)
    if _raw_device is not None and _raw_stream is not None and _raw_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _stream())
    if status:
        check(status, name)


def quantize_nvfp4(x, mode="tensor", outer_in=None, four_over_six=False):
    """Round-to-nearest NVFP4 of x [B, R, C] or [R, C] (float32 or bfloat16);
    four_over_six picks each block's scale from the 6- and 4-mapping candidates.
    Returns (codes u8 [..., C/2], scales u8 [..., C/16], outer f32 [B] or [B*R])."""
    lib = load_library()
    _dev(x, outer_in)
    squeeze = x.dim() == 2
    x3 = x.unsqueeze(0) if squeeze else x
    B, R, C = x3.shape
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(x.dtype)
    if dt is None:
        raise BsqError("x must be float32 or bfloat16")
    m = _enum(mode, _OUTER)
    flags = m | (FOUR_OVER_SIX if four_over_six else 0)
    codes = torch.empty((B, R, C // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((B, R, C // 16), dtype=torch.uint8, device=x.device)
    outer = torch.empty((B * R,) if m == OUTER_ROW else (B,), dtype=torch.float32, device=x.device)
    wsb = lib.bsq_quantize_nvfp4_workspace(B, R, C, flags)
    ws = _ws(wsb, x.device) if wsb else None
    check(lib.bsq_quantize_nvfp4(x3.data_ptr(), dt, B, R, C, flags, _ptr(outer_in), codes.data_ptr(),
                                 scales.data_ptr(), outer.data_ptr(), _ptr(ws), wsb, _stream()),
          "bsq_quantize_nvfp4")
    if squeeze:
        return codes[0], scales[0], outer
    return codes, scales, outer


def swiglu_quantize_nvfp4(h13, four_over_six=True):
    """The expert chain's quantization step: h13 [M, 2F] (float32 or bfloat16,
    gate columns first) -> NVFP4 of silu(gate) * up with per-row outer scales:
    (codes u8 [M, F/2], scales u8 [M, F/16], outer f32 [M])."""
    lib = load_library()
    _dev(h13)
    M, F2 = h13.shape
    F = F2 // 2
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(h13.dtype)
    if dt is None:
        raise BsqError("h13 must be float32 or bfloat16")
    codes = torch.empty((M, F // 2), dtype=torch.uint8, device=h13.device)
    scales = torch.empty((M, F // 16), dtype=torch.uint8, device=h13.device)
    outer = torch.empty((M,), dtype=torch.float32, device=h13.device)
    check(lib.bsq_swiglu_quantize_nvfp4(h13.data_ptr(), dt, M, F, FOUR_OVER_SIX if four_over_six else 0,
                                        codes.data_ptr(), scales.data_ptr(), outer.data_ptr(), _stream()),
          "bsq_swiglu_quantize_nvfp4")
    return codes, scales, outer


def quantize_nvfp4_square(x, mode="tensor", outer_in=None, transpose=True):
    """Square-tile NVFP4 (one scale per 16x16 tile) of x [B, R, C] or [R, C]
    (float32 or bfloat16; R and C multiples of 16); mode "tensor" or "given".
    Returns (codes [..., R, C/2], scales [..., R, C/16], outer f32 [B],
    codes_t [..., C, R/2], scales_t [..., C, R/16]); the transposed pair is
    None when transpose is False."""
    lib = load_library()
    _dev(x, outer_in)
    squeeze = x.dim() == 2
    x3 = x.unsqueeze(0) if squeeze else x
    B, R, C = x3.shape
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(x.dtype)
    if dt is None:
        raise BsqError("x must be float32 or bfloat16")
    m = _enum(mode, _OUTER)
    dev = x.device
    codes = torch.empty((B, R, C // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((B, R, C // 16), dtype=torch.uint8, device=dev)
    codes_t = torch.empty((B, C, R // 2), dtype=torch.uint8, device=dev) if transpose else None
    scales_t = torch.empty((B, C, R // 16), dtype=torch.uint8, device=dev) if transpose else None
    outer = torch.empty((B,), dtype=torch.float32, device=dev)
    wsb = lib.bsq_quantize_nvfp4_square_workspace(B, R, C, m)
    ws = _ws(wsb, dev) if wsb else None
    check(lib.bsq_quantize_nvfp4_square(x3.data_ptr(), dt, B, R, C, m, _ptr(outer_in), codes.data_ptr(),
                                        scales.data_ptr(), _ptr(codes_t), _ptr(scales_t), outer.data_ptr(),
                                        _ptr(ws), wsb, _stream()), "bsq_quantize_nvfp4_square")
    if squeeze:
        return (codes[0], scales[0], outer, codes_t[0] if transpose else None,
                scales_t[0] if transpose else None)
    return codes, scales, outer, codes_t, scales_t


def padded_segment_layout(seg_offsets_host, cols):
    """Host helper: (padded length of each segment, total elements) of the padded
    per-segment transposed layout for a host list/array of segment offsets."""
    seg = [int(v) for v in seg_offsets_host]
    mp = [(seg[e + 1] - seg[e] + 31) // 32 * 32 for e in range(len(seg) - 1)]
    return mp, cols * sum(mp)


def _segmented_capacity(rows, nseg, cols):
    # upper bound of cols * sum(pad32(M_e)); the exact size needs the offsets on the host
    return cols * (rows + 31 * nseg)


def quantize_mxfp8(x, rnd="sr", seed=0, stream_id=0, transpose=False, seg_offsets=None, out_elems=None):
    """MXFP8 of x [R, C] (float32 or bfloat16). transpose=False: codes [R, C],
    scales [R, C/32]. transpose=True: flat codes / scales in the padded
    per-segment transposed layout (seg_offsets: int64 device [E+1] or None for
    one segment); out_elems (optional) sets the exact output length."""
    lib = load_library()
    _dev(x, seg_offsets)
    R, C = x.shape
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(x.dtype)
    if dt is None:
        raise BsqError("x must be float32 or bfloat16")
    r = _enum(rnd, _RND)
    if not transpose:
        codes = torch.empty((R, C), dtype=torch.uint8, device=x.device)
        scales = torch.empty((R, C // 32), dtype=torch.uint8, device=x.device)
        check(lib.bsq_quantize_mxfp8(x.data_ptr(), dt, R, C, 0, None, 0, r, seed, stream_id, codes.data_ptr(),
                                     scales.data_ptr(), None, 0, _stream()), "bsq_quantize_mxfp8")
        return codes, scales
    nseg = seg_offsets.numel() - 1 if seg_offsets is not None else 1
    n = out_elems if out_elems is not None else _segmented_capacity(R, nseg, C)
    codes = torch.empty((n,), dtype=torch.uint8, device=x.device)
    scales = torch.empty((n // 32,), dtype=torch.uint8, device=x.device)
    wsb = lib.bsq_quantize_mxfp8_workspace(R, 1, nseg)
    ws = _ws(wsb, x.device)
    check(lib.bsq_quantize_mxfp8(x.data_ptr(), dt, R, C, 1, _ptr(seg_offsets), nseg if seg_offsets is not None else 0,
                                 r, seed, stream_id, codes.data_ptr(), scales.data_ptr(), ws.data_ptr(), wsb,
                                 _stream()), "bsq_quantize_mxfp8")
    return codes, scales


def quantize_mxfp8_dual(x, rnd="sr", seed=0, stream_rows=0, stream_t=0, seg_offsets=None, out_elems=None):
    """Both MXFP8 quantizations of x [R, C] from one read: ((codes [R, C],
    scales [R, C/32]) as quantize_mxfp8(transpose=False, stream_id=stream_rows),
    (codes_t, scales_t) as quantize_mxfp8(transpose=True, stream_id=stream_t))."""
    lib = load_library()
    _dev(x, seg_offsets)
    R, C = x.shape
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(x.dtype)
    if dt is None:
        raise BsqError("x must be float32 or bfloat16")
    r = _enum(rnd, _RND)
    nseg = seg_offsets.numel() - 1 if seg_offsets is not None else 1
    n = out_elems if out_elems is not None else _segmented_capacity(R, nseg, C)
    codes = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    scales = torch.empty((R, C // 32), dtype=torch.uint8, device=x.device)
    codes_t = torch.empty((n,), dtype=torch.uint8, device=x.device)
    scales_t = torch.empty((n // 32,), dtype=torch.uint8, device=x.device)
    wsb = lib.bsq_quantize_mxfp8_workspace(R, 1, nseg)
    ws = _ws(wsb, x.device)
    check(lib.bsq_quantize_mxfp8_dual(x.data_ptr(), dt, R, C, _ptr(seg_offsets),
                                      nseg if seg_offsets is not None else 0, r, seed, stream_rows, stream_t,
                                      codes.data_ptr(), scales.data_ptr(), codes_t.data_ptr(), scales_t.data_ptr(),
                                      ws.data_ptr(), wsb, _stream()), "bsq_quantize_mxfp8_dual")
    return (codes, scales), (codes_t, scales_t)


def requant_transpose_sr(codes, scales, outer, in_mode, out_fmt="mxfp8", seed=0, stream_id=0, rnd="sr",
                         row_gather=None, seg_offsets=None, out_elems=None):
    """Dequantize -> transpose -> requantize.
    Batch mode: codes [B, R, C/2] (or [R, C/2]) -> output [B, C, R] codes
    (MXFP8 [B, C, R] bytes, NVFP4 [B, C, R/2]) and scales; NVFP4 also returns
    the new outer scales [B].
    Gather mode (row_gather int32 [rows], seg_offsets int64 [E+1]): input
    [T, C/2], output flat padded per-segment transposed MXFP8."""
    lib = load_library()
    _dev(codes, scales, outer, row_gather, seg_offsets)
    im = _enum(in_mode, _OUTER)
    fmt = _enum(out_fmt, _FMT)
    r = _enum(rnd, _RND)
    dev = codes.device
    if row_gather is not None:
        T, C2 = codes.shape
        C = 2 * C2
        rows = row_gather.numel()
        nseg = seg_offsets.numel() - 1
        n = out_elems if out_elems is not None else _segmented_capacity(rows, nseg, C)
        oc = torch.empty((n,), dtype=torch.uint8, device=dev)
        osc = torch.empty((n // 32,), dtype=torch.uint8, device=dev)
        wsb = lib.bsq_requant_workspace(1, rows, nseg, fmt, 1)
        ws = _ws(wsb, dev)
        check(lib.bsq_requant_transpose_sr(codes.data_ptr(), scales.data_ptr(), outer.data_ptr(), im, 1, rows, C, T,
                                           row_gather.data_ptr(), seg_offsets.data_ptr(), nseg, fmt, r, seed,
                                           stream_id, oc.data_ptr(), osc.data_ptr(), None, ws.data_ptr(), wsb,
                                           _stream()), "bsq_requant_transpose_sr")
        return oc, osc
    squeeze = codes.dim() == 2
    c3 = codes.unsqueeze(0) if squeeze else codes
    B, R, C2 = c3.shape
    C = 2 * C2
    if fmt == MXFP8:
        oc = torch.empty((B, C, R), dtype=torch.uint8, device=dev)
        osc = torch.empty((B, C, R // 32), dtype=torch.uint8, device=dev)
        oo = None
    else:
        oc = torch.empty((B, C, R // 2), dtype=torch.uint8, device=dev)
        osc = torch.empty((B, C, R // 16), dtype=torch.uint8, device=dev)
        oo = torch.empty((B,), dtype=torch.float32, device=dev)
    wsb = lib.bsq_requant_workspace(B, R, 0, fmt, 0)
    ws = _ws(wsb, dev) if wsb else None
    check(lib.bsq_requant_transpose_sr(c3.data_ptr(), scales.data_ptr(), outer.data_ptr(), im, B, R, C, B * R, None,
                                       None, 0, fmt, r, seed, stream_id, oc.data_ptr(), osc.data_ptr(), _ptr(oo),
                                       _ptr(ws), wsb, _stream()), "bsq_requant_transpose_sr")
    if squeeze:
        oc, osc = oc[0], osc[0]
    return (oc, osc) if fmt == MXFP8 else (oc, osc, oo)


_OUT = {torch.bfloat16: BF16, torch.float32: F32}


def grouped_gemm_nvfp4(a_codes, a_scales, a_outer, b_codes, b_scales, b_outer, seg_offsets, M_total,
                       row_index=None, out=None, out_dtype=torch.bfloat16):
    """y [M_total, N] = per expert, gathered x_q rows times w_q^T with both
    outer scales (bf16 or float32 output). a_*: [T, K/2], [T, K/16], a_outer
    [T] (per token) or [1]; b_*: [E, N, K/2], [E, N, K/16], b_outer [E]."""
    lib = load_library()
    _dev(a_codes, a_scales, a_outer, b_codes, b_scales, b_outer, seg_offsets, row_index)
    T, K2 = a_codes.shape
    E, N, _ = b_codes.shape
    per_row = 1 if a_outer.numel() == T and T > 1 else 0
    if out is None:
        out = torch.empty((M_total, N), dtype=out_dtype, device=a_codes.device)
    check(lib.bsq_grouped_gemm_nvfp4(a_codes.data_ptr(), a_scales.data_ptr(), a_outer.data_ptr(), per_row, T,
                                     _ptr(row_index), b_codes.data_ptr(), b_scales.data_ptr(), b_outer.data_ptr(),
                                     seg_offsets.data_ptr(), E, M_total, N, 2 * K2, out.data_ptr(), _OUT[out.dtype],
                                     _stream()), "bsq_grouped_gemm_nvfp4")
    return out


def grouped_gemm_nvfp4_s2f6(a_codes, a_scales, a_outer, b_codes, b_scales, b_outer, seg_offsets, M_total, signs,
                            row_index=None):
    """The w2 GEMM with the combine codec in its epilogue: the product of
    grouped_gemm_nvfp4, RHT-rotated and S2F6-quantized per 32 columns ->
    (codes u8 [M_total, N], scales u8 [M_total, N/32])."""
    lib = load_library()
    _dev(a_codes, a_scales, a_outer, b_codes, b_scales, b_outer, seg_offsets, row_index)
    T, K2 = a_codes.shape
    E, N, _ = b_codes.shape
    per_row = 1 if a_outer.numel() == T and T > 1 else 0
    codes = torch.empty((M_total, N), dtype=torch.uint8, device=a_codes.device)
    scales = torch.empty((M_total, N // 32), dtype=torch.uint8, device=a_codes.device)
    check(lib.bsq_grouped_gemm_nvfp4_s2f6(a_codes.data_ptr(), a_scales.data_ptr(), a_outer.data_ptr(), per_row, T,
                                          _ptr(row_index), b_codes.data_ptr(), b_scales.data_ptr(),
                                          b_outer.data_ptr(), seg_offsets.data_ptr(), E, M_total, N, 2 * K2,
                                          signs & 0xFFFFFFFF, codes.data_ptr(), scales.data_ptr(), _stream()),
          "bsq_grouped_gemm_nvfp4_s2f6")
    return codes, scales


def grouped_gemm_mxfp8(wgrad, a_codes, a_scales, b_codes, b_scales, seg_offsets, M, N, K=0, out=None,
                       out_dtype=None):
    """wgrad=False (DGRAD): a [M_total(=M), K], b [E, N, K] -> [M, N] (bf16
    by default). wgrad=True (WGRAD): a, b flat padded per-segment transposed
    layouts with M and N rows per expert -> [E, M, N] (float32 by default)."""
    lib = load_library()
    _dev(a_codes, a_scales, b_codes, b_scales, seg_offsets)
    E = seg_offsets.numel() - 1
    if out is None:
        dt = out_dtype or (torch.float32 if wgrad else torch.bfloat16)
        shape = (E, M, N) if wgrad else (M, N)
        out = torch.empty(shape, dtype=dt, device=a_codes.device)
    check(lib.bsq_grouped_gemm_mxfp8(1 if wgrad else 0, a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(),
             seg_offsets.data_ptr(), E, M, N, K, out.data_ptr(), _OUT[out.dtype], _stream()), "bsq_grouped_gemm_mxfp8")
    return out


def gemm_nvfp4_inreg_scale(a_codes, a_scales, a_outer, b_codes, b_scales, b_outer):
    """Dense NVFP4 product with the block scales applied in registers (FP8
    MFMA per 16-value block, fp32 scaling): a_* [M, K/2], [M, K/16], [M];
    b_* [N, K/2], [N, K/16], [1] -> float32 [M, N]. The alternative to the
    exact 16-bit decode of grouped_gemm_nvfp4, kept for comparison."""
    lib = load_library()
    _dev(a_codes, a_scales, a_outer, b_codes, b_scales, b_outer)
    M, N, K = a_codes.shape[0], b_codes.shape[0], 2 * a_codes.shape[1]
    out = torch.empty((M, N), dtype=torch.float32, device=a_codes.device)
    check(lib.bsq_gemm_nvfp4_inreg_scale(a_codes.data_ptr(), a_scales.data_ptr(), a_outer.data_ptr(),
                                         b_codes.data_ptr(), b_scales.data_ptr(), b_outer.data_ptr(), M, N, K,
                                         out.data_ptr(), _stream()), "bsq_gemm_nvfp4_inreg_scale")
    return out


def route(topk_ids, num_experts):
    """topk_ids int32 [T, k] -> (row_index int32 [T*k], seg_offsets int64 [E+1], pair_row int32 [T*k])."""
    lib = load_library()
    _dev(topk_ids)
    T, k = topk_ids.shape
    dev = topk_ids.device
    row_index = torch.empty((T * k,), dtype=torch.int32, device=dev)
    pair_row = torch.empty((T * k,), dtype=torch.int32, device=dev)
    seg = torch.empty((num_experts + 1,), dtype=torch.int64, device=dev)
    wsb = lib.bsq_route_workspace(T, num_experts)
    ws = _ws(wsb, dev) if wsb else None
    check(lib.bsq_route(topk_ids.data_ptr(), T, k, num_experts, row_index.data_ptr(), seg.data_ptr(),
                        pair_row.data_ptr(), _ptr(ws), wsb, _stream()), "bsq_route")
    return row_index, seg, pair_row


def route_noalloc(topk_ids, num_experts, row_index, seg_offsets, pair_row):
    """route() into caller-provided outputs with no device allocation: the
    library's own per-GPU array holds the per-chunk counts (tokens x E up to
    the 1 MiB limit of BSQ_ROUTE_NOALLOC_MAX_BYTES). Calls on one GPU that
    overlap in time race."""
    lib = load_library()
    _dev(topk_ids, row_index, seg_offsets, pair_row)
    T, k = topk_ids.shape
    if row_index.numel() != T * k or pair_row.numel() != T * k or seg_offsets.numel() != num_experts + 1:
        raise BsqError("route_noalloc: output sizes do not match topk_ids and num_experts")
    check(lib.bsq_route_noalloc(topk_ids.data_ptr(), T, k, num_experts, row_index.data_ptr(), seg_offsets.data_ptr(),
                                pair_row.data_ptr(), _stream()), "bsq_route_noalloc")
    return row_index, seg_offsets, pair_row


def _need(cond, what):
    if not cond:
        raise BsqError(what)


def _dtype(t, what):
    dt = _OUT.get(t.dtype)
    if dt is None:
        raise BsqError(f"{what} must be float32 or bfloat16")
    return dt


def moe_gate(logits, k, renormalize=True):
    """The k experts of each token: logits [T, E] (float32 or bfloat16) ->
    (weights f32 [T, k], topk_ids int32 [T, k]), largest first, ties to the
    lowest index. The weights are a softmax over the selected logits, or with
    renormalize=False over all of them. Logits of -inf (and NaN) are masked; a
    slot that finds no unmasked logit left gets id -1 and weight 0. Not recorded
    by autograd, as no operator here: moe_gate_backward is the gradient."""
    lib = load_library()
    _dev(logits)
    _need(logits.dim() == 2, "moe_gate: logits must be [tokens, experts]")
    T, E = logits.shape
    dt = _dtype(logits, "logits")
    _need(1 <= k <= min(E, 64), "moe_gate: k must be in [1, min(experts, 64)]")
    weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    check(lib.bsq_moe_gate(logits.data_ptr(), dt, T, E, k, 1 if renormalize else 0, weights.data_ptr(),
                           ids.data_ptr(), _stream()), "bsq_moe_gate")
    return weights, ids


def moe_gate_backward(dweights, weights, topk_ids, logits, renormalize=True):
    """Gradient of moe_gate's weights to its logits, the selection held fixed:
    dweights f32 [T, k] with moe_gate's outputs and input -> dlogits [T, E] of
    logits' type (every element written)."""
    lib = load_library()
    _dev(dweights, weights, topk_ids, logits)
    _need(logits.dim() == 2 and weights.dim() == 2, "moe_gate_backward: logits [tokens, experts], weights [tokens, k]")
    T, E = logits.shape
    k = weights.shape[1]
    dt = _dtype(logits, "logits")
    _need(weights.shape == (T, k) and dweights.shape == (T, k) and topk_ids.shape == (T, k),
          "moe_gate_backward: dweights, weights and topk_ids must be [tokens, k]")
    _need(dweights.dtype == torch.float32 and weights.dtype == torch.float32 and topk_ids.dtype == torch.int32,
          "moe_gate_backward: dweights and weights must be float32, topk_ids int32")
    dlogits = torch.empty_like(logits)
    check(lib.bsq_moe_gate_backward(dweights.data_ptr(), weights.data_ptr(), topk_ids.data_ptr(), logits.data_ptr(),
                                    dt, T, E, k, 1 if renormalize else 0, dlogits.data_ptr(), _stream()),
          "bsq_moe_gate_backward")
    return dlogits


_SCORE = {"sigmoid": 0, "softmax": 1}


def _score(score, what):
    _need(score in _SCORE, what + ": score must be 'sigmoid' or 'softmax'")
    return _SCORE[score]


def moe_gate_grouped(logits, k, bias=None, groups=1, group_k=None, group_top=2, score="sigmoid", renormalize=True,
                     scale=1.0):
    """The k experts of each token by scores s, a balancing bias and groups:
    logits [T, E] (float32 or bfloat16) -> (weights f32 [T, k], topk_ids int32
    [T, k]). s is the sigmoid of the logits or their softmax; the keys s + bias
    (f32 [E] or None) choose: the group_k groups (all unless given) of E / groups
    neighbouring experts with the largest sums of their group_top best keys,
    then the k largest keys in them, largest first, ties to the lowest index.
    weights: scale * s, with renormalize divided by the selected scores' sum.
    Logits of -inf (and NaN) are masked; a slot that finds no expert left gets
    id -1 and weight 0. moe_gate_grouped_backward is the gradient."""
    _dev(logits, bias)
    _need(logits.dim() == 2, "moe_gate_grouped: logits must be [tokens, experts]")
    T, E = logits.shape
    dt = _dtype(logits, "logits")
    group_k = groups if group_k is None else group_k
    _need(1 <= groups <= 64 and E % groups == 0 and 1 <= group_k <= groups,
          "moe_gate_grouped: groups must divide the experts (64 at most), 1 <= group_k <= groups")
    _need(1 <= k <= min(64, group_k * (E // groups)), "moe_gate_grouped: k must be in [1, min(64, experts of group_k groups)]")
    _need(bias is None or (bias.dtype == torch.float32 and bias.numel() == E),
          "moe_gate_grouped: bias must be float32 [experts]")
    sc = _score(score, "moe_gate_grouped")
    weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    _run("bsq_moe_gate_grouped", logits, (bias,), logits.data_ptr(), dt, _ptr(bias), T, E, k, groups, group_k,
         group_top, sc, 1 if renormalize else 0, scale, weights.data_ptr(), ids.data_ptr())
    return weights, ids


def moe_gate_grouped_backward(dweights, weights, topk_ids, logits, score="sigmoid", renormalize=True, scale=1.0):
    """Gradient of moe_gate_grouped's weights to its logits, the selection held
    fixed: dweights f32 [T, k] with moe_gate_grouped's outputs, input, score,
    renormalize and scale -> dlogits [T, E] of logits' type (every element
    written). The bias only selects and has no gradient."""
    _dev(dweights, weights, topk_ids, logits)
    _need(logits.dim() == 2 and weights.dim() == 2,
          "moe_gate_grouped_backward: logits [tokens, experts], weights [tokens, k]")
    T, E = logits.shape
    k = weights.shape[1]
    dt = _dtype(logits, "logits")
    _need(weights.shape == (T, k) and dweights.shape == (T, k) and topk_ids.shape == (T, k),
          "moe_gate_grouped_backward: dweights, weights and topk_ids must be [tokens, k]")
    _need(dweights.dtype == torch.float32 and weights.dtype == torch.float32 and topk_ids.dtype == torch.int32,
          "moe_gate_grouped_backward: dweights and weights must be float32, topk_ids int32")
    sc = _score(score, "moe_gate_grouped_backward")
    dlogits = torch.empty_like(logits)
    _run("bsq_moe_gate_grouped_backward", logits, (dweights, weights, topk_ids), dweights.data_ptr(),
         weights.data_ptr(), topk_ids.data_ptr(), logits.data_ptr(), dt, T, E, k, sc, 1 if renormalize else 0, scale,
         dlogits.data_ptr())
    return dlogits


def moe_few_tokens_nvfp4(x, topk_ids, topk_weights, w13_codes, w13_scales, w13_outer, w2_codes, w2_scales, w2_outer):
    """A whole expert layer for a few tokens (decode): y [T, H] of x's type =
    sum over a token's experts of weight * W2 (silu(gate) * up), (gate; up) =
    W13 x, from x [T, H] (float32 or bfloat16, not quantized), topk_ids int32
    [T, k] and topk_weights f32 [T, k] as moe_gate returns them (ids outside
    [0, E) add nothing) and NVFP4 weights with one outer scale per expert: w13
    [E, 2F, H] (gate rows first), w2 [E, H, F]. T * k <= 2048."""
    lib = load_library()
    _dev(x, topk_ids, topk_weights, w13_codes, w13_scales, w13_outer, w2_codes, w2_scales, w2_outer)
    _need(x.dim() == 2 and topk_ids.dim() == 2 and w13_codes.dim() == 3 and w2_codes.dim() == 3,
          "moe_few_tokens_nvfp4: x [T, H], topk_ids [T, k], w13 and w2 codes [E, rows, cols / 2]")
    T, H = x.shape
    k = topk_ids.shape[1]
    E, F = w2_codes.shape[0], 2 * w2_codes.shape[2]
    dt = _dtype(x, "x")
    _need(topk_ids.shape == (T, k) and topk_weights.shape == (T, k) and topk_ids.dtype == torch.int32
          and topk_weights.dtype == torch.float32,
          "moe_few_tokens_nvfp4: topk_ids must be int32 [T, k] and topk_weights float32 [T, k]")
    _need(w13_codes.shape == (E, 2 * F, H // 2) and w2_codes.shape == (E, H, F // 2)
          and w13_scales.shape == (E, 2 * F, H // 16) and w2_scales.shape == (E, H, F // 16)
          and w13_outer.numel() == E and w2_outer.numel() == E,
          "moe_few_tokens_nvfp4: w13 must be [E, 2F, H] and w2 [E, H, F] (codes, scales, outer [E])")
    _need(w13_codes.dtype == w2_codes.dtype == w13_scales.dtype == w2_scales.dtype == torch.uint8
          and w13_outer.dtype == w2_outer.dtype == torch.float32,
          "moe_few_tokens_nvfp4: codes and scales must be uint8, outer scales float32")
    out = torch.empty_like(x)
    wsb = lib.bsq_moe_few_nvfp4_workspace(T, H, F, E, k)
    ws = _ws(wsb, x.device)
    check(lib.bsq_moe_few_nvfp4(x.data_ptr(), dt, T, H, F, E, k, topk_ids.data_ptr(), topk_weights.data_ptr(),
                                w13_codes.data_ptr(), w13_scales.data_ptr(), w13_outer.data_ptr(),
                                w2_codes.data_ptr(), w2_scales.data_ptr(), w2_outer.data_ptr(), out.data_ptr(),
                                ws.data_ptr(), wsb, _stream()), "bsq_moe_few_nvfp4")
    return out


def quantize_int8(x):
    """Rows of x [R, C] (float32 or bfloat16, C % 16 == 0) in 8-bit integers
    with a scale each: (codes int8 [R, C], scales f32 [R]). A row with a NaN or
    an infinity gets the scale NaN, and NaN in every output made from it."""
    lib = load_library()
    _dev(x)
    _need(x.dim() == 2, "quantize_int8: x must be [rows, cols]")
    R, C = x.shape
    dt = _dtype(x, "x")
    codes = torch.empty((R, C), dtype=torch.int8, device=x.device)
    scales = torch.empty((R,), dtype=torch.float32, device=x.device)
    check(lib.bsq_quantize_int8(x.data_ptr(), dt, R, C, codes.data_ptr(), scales.data_ptr(), _stream()),
          "bsq_quantize_int8")
    return codes, scales


def swiglu_quantize_int8(h13):
    """quantize_int8 of silu(gate) * up, from h13 [R, 2F] (gate columns first)."""
    lib = load_library()
    _dev(h13)
    _need(h13.dim() == 2 and h13.shape[1] % 2 == 0, "swiglu_quantize_int8: h13 must be [rows, 2 * ffn]")
    R, F = h13.shape[0], h13.shape[1] // 2
    dt = _dtype(h13, "h13")
    codes = torch.empty((R, F), dtype=torch.int8, device=h13.device)
    scales = torch.empty((R,), dtype=torch.float32, device=h13.device)
    check(lib.bsq_swiglu_quantize_int8(h13.data_ptr(), dt, R, F, codes.data_ptr(), scales.data_ptr(), _stream()),
          "bsq_swiglu_quantize_int8")
    return codes, scales


def _int8_operand(codes, scales, what):
    if not (codes.dim() == 2 and codes.dtype == torch.int8 and scales.dtype == torch.float32
            and scales.numel() == codes.shape[0]):
        raise BsqError(what + ": int8 codes [rows, K] with float32 scales [rows]")


def gemm_int8(a_codes, a_scales, b_codes, b_scales, bias=None, out_dtype=torch.bfloat16):
    """y [M, N] = (sum_k a[m, k] b[n, k]) a_scales[m] b_scales[n] + bias[n] of
    int8 codes a [M, K] and b [N, K] (K % 16 == 0), exact integer sums; bias
    float32 [N] or None; bfloat16 or float32 output."""
    lib = load_library()
    _dev(a_codes, a_scales, b_codes, b_scales, bias)
    _int8_operand(a_codes, a_scales, "gemm_int8: a")
    _int8_operand(b_codes, b_scales, "gemm_int8: b")
    M, K = a_codes.shape
    N = b_codes.shape[0]
    _need(b_codes.shape[1] == K, "gemm_int8: a and b must share K")
    _need(bias is None or (bias.dtype == torch.float32 and bias.numel() == N), "gemm_int8: bias must be float32 [N]")
    _need(out_dtype in _OUT, "out_dtype must be float32 or bfloat16")
    out = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    check(lib.bsq_gemm_int8(a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(),
                            _ptr(bias), M, N, K, out.data_ptr(), _OUT[out_dtype], _stream()), "bsq_gemm_int8")
    return out


def linear_int8(x, b_codes, b_scales, bias=None, out_dtype=None):
    """gemm_int8 of quantize_int8(x) in one call: x [M, K] (float32 or bfloat16,
    K <= 32768), weights int8 [N, K] with float32 scales [N]; out_dtype is x's
    unless given. The same bits as the two calls."""
    lib = load_library()
    _dev(x, b_codes, b_scales, bias)
    _need(x.dim() == 2, "linear_int8: x must be [M, K]")
    dt = _dtype(x, "x")
    _int8_operand(b_codes, b_scales, "linear_int8: b")
    M, K = x.shape
    N = b_codes.shape[0]
    out_dtype = out_dtype or x.dtype
    _need(b_codes.shape[1] == K, "linear_int8: x and b must share K")
    _need(bias is None or (bias.dtype == torch.float32 and bias.numel() == N), "linear_int8: bias must be float32 [N]")
    _need(out_dtype in _OUT, "out_dtype must be float32 or bfloat16")
    out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    wsb = lib.bsq_linear_int8_workspace(M, K)
    ws = _ws(wsb, x.device) if wsb else None
    check(lib.bsq_linear_int8(x.data_ptr(), dt, b_codes.data_ptr(), b_scales.data_ptr(), _ptr(bias), M, N, K,
                              out.data_ptr(), _OUT[out_dtype], _ptr(ws), wsb, _stream()), "bsq_linear_int8")
    return out


def quantize_int4(w, group=128, symmetric=False):
    """Weights w [N, K] (float32 or bfloat16) in 4-bit integers with a scale and
    a zero point for each group (32, 64 or 128) of neighbours along K:
    (codes u8 [N, K/2], scales bf16 [N, K/group], zeros u8 [N, K/group] or, with
    symmetric, None). They stand for (q - z) * s, z = 8 without zeros."""
    _dev(w)
    _need(w.dim() == 2, "quantize_int4: w must be [N, K]")
    N, K = w.shape
    dt = _dtype(w, "w")
    _need(group in (32, 64, 128) and K >= group and K % group == 0,
          "quantize_int4: group must be 32, 64 or 128 and divide K")
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((N, K // group), dtype=torch.bfloat16, device=w.device)
    zeros = None if symmetric else torch.empty((N, K // group), dtype=torch.uint8, device=w.device)
    _run("bsq_quantize_int4", w, (), w.data_ptr(), dt, N, K, group, 1 if symmetric else 0, codes.data_ptr(),
         scales.data_ptr(), _ptr(zeros))
    return codes, scales, zeros


def _int4_group(codes, scales, zeros, what):
    """(N, K, group) of 4-bit weights."""
    _need(codes.dim() == 2 and codes.dtype == torch.uint8 and scales.dim() == 2 and scales.dtype == torch.bfloat16
          and scales.shape[0] == codes.shape[0] and scales.shape[1] > 0,
          what + ": uint8 codes [N, K/2] with bfloat16 scales [N, K/group]")
    _need(zeros is None or (zeros.dtype == torch.uint8 and zeros.shape == scales.shape),
          what + ": zeros must be uint8 [N, K/group]")
    N, K = codes.shape[0], 2 * codes.shape[1]
    group = K // scales.shape[1]
    _need(group in (32, 64, 128) and group * scales.shape[1] == K, what + ": groups must be of 32, 64 or 128")
    return N, K, group


def dequantize_int4(codes, scales, zeros=None, out_dtype=torch.float32):
    """The values [N, K] that 4-bit groups stand for, (q - z) * s."""
    _dev(codes, scales, zeros)
    N, K, group = _int4_group(codes, scales, zeros, "dequantize_int4")
    _need(out_dtype in _OUT, "out_dtype must be float32 or bfloat16")
    out = torch.empty((N, K), dtype=out_dtype, device=codes.device)
    _run("bsq_dequantize_int4", codes, (scales, zeros), codes.data_ptr(), scales.data_ptr(), _ptr(zeros), N, K, group,
         out.data_ptr(), _OUT[out_dtype])
    return out


def linear_int4(x, codes, scales, zeros=None, bias=None, out_dtype=None):
    """y [M, N] = x W^T + bias of unquantized activations x [M, K] (float32 or
    bfloat16) and weights in 4-bit groups as quantize_int4 returns them; bias
    float32 [N] or None; out_dtype is x's unless given. float32 x enters with 22
    significant bits (the limits are bsq.h's). One token or few: bound by reading
    the codes once."""
    _dev(x, codes, scales, zeros, bias)
    _need(x.dim() == 2, "linear_int4: x must be [M, K]")
    dt = _dtype(x, "x")
    N, K, group = _int4_group(codes, scales, zeros, "linear_int4")
    M = x.shape[0]
    out_dtype = out_dtype or x.dtype
    _need(x.shape[1] == K, "linear_int4: x and the weights must share K")
    _need(bias is None or (bias.dtype == torch.float32 and bias.numel() == N), "linear_int4: bias must be float32 [N]")
    _need(out_dtype in _OUT, "out_dtype must be float32 or bfloat16")
    out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    wsb = _ws_bytes("bsq_linear_int4_workspace", x.get_device(), M, N, K, group, dt)
    ws = _ws(wsb, x.device) if wsb else None
    _run("bsq_linear_int4", x, (codes, scales, zeros, bias), x.data_ptr(), dt, codes.data_ptr(), scales.data_ptr(),
         _ptr(zeros), group, _ptr(bias), M, N, K, out.data_ptr(), _OUT[out_dtype], _ptr(ws), wsb)
    return out


def token_logprobs(logits, targets, top=0):
    """Log probabilities of given tokens: logits [T, V] (float32 or bfloat16,
    -inf masked), targets int64 [T] (outside [0, V): padding, log probability 0)
    -> (logprobs f32 [T], entropy f32 [T], stats f32 [T, 2], top_logprobs f32
    [T, top], top_ids int32 [T, top]), the last two None without `top`: the
    largest alternatives, ties to the lowest index, id -1 where no unmasked
    logit is left. stats (the row's maximum and log sum e^(x - maximum), which
    add up to the log-sum-exp) is for token_logprobs_backward, the gradient."""
    _dev(logits, targets)
    _need(logits.dim() == 2, "token_logprobs: logits must be [tokens, vocabulary]")
    T, V = logits.shape
    dt = _dtype(logits, "logits")
    _need(targets.dtype == torch.int64 and targets.shape == (T,), "token_logprobs: targets must be int64 [tokens]")
    _need(1 <= V <= 1 << 20 and 0 <= top <= min(V, 64), "token_logprobs: 1 <= vocabulary <= 2^20, 0 <= top <= min(vocabulary, 64)")
    f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=logits.device)
    logprobs, entropy, stats = f32(T), f32(T), f32(T, 2)
    top_lp = f32(T, top) if top else None
    top_ids = torch.empty((T, top), dtype=torch.int32, device=logits.device) if top else None
    wsb = _ws_bytes("bsq_token_logprobs_workspace", logits.get_device(), T, V, top, dt)
    ws = _ws(wsb, logits.device) if wsb else None
    _run("bsq_token_logprobs", logits, (targets,), logits.data_ptr(), dt, targets.data_ptr(), T, V, top,
         logprobs.data_ptr(), entropy.data_ptr(), stats.data_ptr(), _ptr(top_lp), _ptr(top_ids), _ptr(ws), wsb)
    return logprobs, entropy, stats, top_lp, top_ids


def token_logprobs_backward(dlogprobs, dentropy, logits, targets, stats, entropy):
    """Gradient of token_logprobs' logprobs and entropy to its logits: dlogprobs
    and dentropy f32 [T] (either may be None) with token_logprobs' inputs and
    outputs -> dlogits [T, V] of logits' type (every element written, 0 at
    masked logits)."""
    _dev(dlogprobs, dentropy, logits, targets, stats, entropy)
    _need(logits.dim() == 2, "token_logprobs_backward: logits must be [tokens, vocabulary]")
    T, V = logits.shape
    dt = _dtype(logits, "logits")
    _need(dlogprobs is not None or dentropy is not None, "token_logprobs_backward: dlogprobs or dentropy must be given")
    for t, shape in ((dlogprobs, (T,)), (dentropy, (T,)), (stats, (T, 2)), (entropy, (T,))):
        _need(t is None or (t.dtype == torch.float32 and t.shape == shape),
              "token_logprobs_backward: dlogprobs, dentropy and entropy must be float32 [tokens], stats [tokens, 2]")
    _need(targets.dtype == torch.int64 and targets.shape == (T,),
          "token_logprobs_backward: targets must be int64 [tokens]")
    _need(1 <= V <= 1 << 20, "token_logprobs_backward: 1 <= vocabulary <= 2^20")
    dlogits = torch.empty_like(logits)
    _run("bsq_token_logprobs_backward", logits, (dlogprobs, dentropy, targets, stats, entropy), _ptr(dlogprobs),
         _ptr(dentropy), logits.data_ptr(), dt, targets.data_ptr(), stats.data_ptr(), entropy.data_ptr(), T, V,
         dlogits.data_ptr())
    return dlogits


def rht_s2f6_encode(x, signs):
    """Combine-codec sender: x [R, C] (float32 or bfloat16, C % 32 == 0) ->
    (codes u8 [R, C] two's-complement S2F6, scales u8 [R, C/32] UE8M0) of the
    rows rotated by the 32-point Hadamard transform with sign mask `signs`."""
    lib = load_library()
    _dev(x)
    R, C = x.shape
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(x.dtype)
    if dt is None:
        raise BsqError("x must be float32 or bfloat16")
    codes = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    scales = torch.empty((R, C // 32), dtype=torch.uint8, device=x.device)
    check(lib.bsq_rht_s2f6_encode(x.data_ptr(), dt, R, C, signs & 0xFFFFFFFF, codes.data_ptr(), scales.data_ptr(),
                                  _stream()), "bsq_rht_s2f6_encode")
    return codes, scales


def rht_s2f6_combine(codes, scales, pair_row, k, signs, out_dtype=torch.bfloat16):
    """Combine-codec receiver: token t sums the dequantized rows
    pair_row[t*k + j] (int32 [T*k]) and inverts the transform -> [T, C]."""
    lib = load_library()
    _dev(codes, scales, pair_row)
    R, C = codes.shape
    T = pair_row.numel() // k
    od = {torch.float32: F32, torch.bfloat16: BF16}.get(out_dtype)
    if od is None:
        raise BsqError("out_dtype must be float32 or bfloat16")
    out = torch.empty((T, C), dtype=out_dtype, device=codes.device)
    check(lib.bsq_rht_s2f6_combine(codes.data_ptr(), scales.data_ptr(), R, C, pair_row.data_ptr(), T, k,
                                   signs & 0xFFFFFFFF, out.data_ptr(), od, _stream()), "bsq_rht_s2f6_combine")
    return out


def dequantize_nvfp4(codes, scales, outer, mode="tensor"):
    lib = load_library()
    _dev(codes, scales, outer)
    squeeze = codes.dim() == 2
    c3 = codes.unsqueeze(0) if squeeze else codes
    B, R, C2 = c3.shape
    out = torch.empty((B, R, 2 * C2), dtype=torch.float32, device=codes.device)
    check(lib.bsq_dequantize_nvfp4(c3.data_ptr(), scales.data_ptr(), outer.data_ptr(), _enum(mode, _OUTER), B, R,
                                   2 * C2, out.data_ptr(), _stream()), "bsq_dequantize_nvfp4")
    return out[0] if squeeze else out


def dequantize_mxfp8(codes, scales):
    lib = load_library()
    _dev(codes, scales)
    R, C = codes.shape
    out = torch.empty((R, C), dtype=torch.float32, device=codes.device)
    check(lib.bsq_dequantize_mxfp8(codes.data_ptr(), scales.data_ptr(), R, C, out.data_ptr(), _stream()),
          "bsq_dequantize_mxfp8")
    return out


def rng_bits16(seed, stream_id, first, n, device="cuda"):
    lib = load_library()
    out = torch.empty((n,), dtype=torch.int16, device=device)
    check(lib.bsq_rng_bits16(seed, stream_id, first, n, out.data_ptr(), _stream()), "bsq_rng_bits16")
    return out


def mfma_rate_probe(kind, data, iters, workgroups, device="cuda"):
    """Launch the per-instruction MFMA throughput probe (see bsq.h) and
    return its output tensor [workgroups * 256]; the caller times the launch."""
    lib = load_library()
    out = torch.empty((workgroups * 256,), dtype=torch.float32, device=device)
    check(lib.bsq_mfma_rate_probe(kind, data, iters, workgroups, out.data_ptr(), _stream()), "bsq_mfma_rate_probe")
    return out
