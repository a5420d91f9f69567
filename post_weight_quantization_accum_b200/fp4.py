"""4-bit floating point: quantisation, product and product grouped by expert.

A quantised matrix is a dict: ``packed`` uint8 [rows, 16 * ceil(n / 32)] (two
E2M1 codes a byte), ``scales`` uint8 [bands, quads, 512] (scale tiles of 128
rows x 4 blocks), ``tensor_scale`` fp32 [groups] ("nvfp4") or None ("mxfp4"),
``offsets`` (the int32 tensor that the rows' groups came from, not a copy of
it, or None: one group, or groups of one size) and the plain values ``rows``,
``n``, ``format``, ``groups``.  include/gptq.h defines the formats and layouts;
the functions here check arguments, get outputs and workspaces from torch and
call the library.  (A dict that a program lays out itself may leave ``offsets``
out: how its rows are grouped is then not checked.)

A call runs on ``stream`` or, without one, on the current stream of the
tensors' device (which need not be the current device); outputs belong to that
stream.
"""
import torch

from ._lib import GPTQ_BF16, GPTQ_F32, GPTQ_MXFP4, GPTQ_NVFP4, LIB, aligned_workspace, check, check_workspace

FP4_FORMATS = {"mxfp4": GPTQ_MXFP4, "nvfp4": GPTQ_NVFP4}
FP4_BLOCK = {"mxfp4": 32, "nvfp4": 16}
MAX_GROUPS = 512  # of an offsets tensor
_DTYPES = {torch.float32: GPTQ_F32, torch.bfloat16: GPTQ_BF16}
# the handle of a device's current stream, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _enter(device, stream):
    """(stream handle, guard): the tensors' device and the stream are current
    until guard (None: they were) is left, so that what is allocated belongs to
    them."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, not on {device}")
    index = device.index
    if stream is None and index == torch.cuda.current_device():
        return _raw_stream(index), None
    if stream is None:
        guard = torch.cuda.device(device)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    else:
        guard = torch.cuda.stream(stream)
    guard.__enter__()
    return _raw_stream(index), guard


def _leave(guard):
    if guard is not None:
        guard.__exit__(None, None, None)


def _need(ok, why):
    if not ok:
        raise ValueError(why)


def _vector(t, name, dtype, length, device):
    """An argument that is a contiguous vector (length None: any)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 1 or not t.is_contiguous() or (length is not None and shape[0] != length):
        raise ValueError(f"{name} must be a contiguous vector{'' if length is None else f' of {length}'}, "
                         f"got {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


def _check_format(format):
    if format not in FP4_FORMATS:
        raise ValueError(f"format must be one of {sorted(FP4_FORMATS)}, got {format!r}")


def _bands(rows, groups, ragged):
    """Bands of 128 rows that the scales need (ragged: for any offsets)."""
    return rows // 128 + groups if ragged else groups * ((rows // groups + 127) // 128)


def fp4_check_quantize_args(X, format, tensor_scale=None, row_index=None, offsets=None, ws=None):
    """The checks gptq_fp4_quantize makes before it touches the device; they
    need no GPU.  Returns (rows, groups) of the result."""
    _check_format(format)
    if X.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {X.dtype}: fp32 or bf16")
    shape = X.shape
    if len(shape) not in (2, 3):
        raise ValueError(f"X must be [rows, n] or [groups, rows, n], got {tuple(shape)}")
    if not 1 <= shape[-1] <= 65535:
        raise ValueError(f"X must have 1 to 65535 columns, got {shape[-1]}")
    if len(shape) == 3:
        _need(X.is_contiguous(), "a stack of matrices must be contiguous")
        _need(row_index is None and offsets is None, "row_index and offsets go with a matrix, not with a stack")
        _need(shape[0] >= 1, "a stack needs at least one matrix")
        rows, groups = shape[0] * shape[1], shape[0]
    else:
        if not X.is_contiguous():
            _need(X.stride(1) == 1 or shape[1] == 1, "X's rows must be contiguous")
            _need(X.stride(0) >= shape[1] or shape[0] <= 1, "X's rows must not overlap")
        rows, groups = shape[0], 1
    device = X.device
    if row_index is not None:
        _vector(row_index, "row_index", torch.int32, None, device)
        rows = row_index.shape[0]
    if offsets is not None:
        _vector(offsets, "offsets", torch.int32, None, device)
        groups = offsets.shape[0] - 1
        if not 1 <= groups <= MAX_GROUPS:
            raise ValueError(f"offsets must have 2 to {MAX_GROUPS + 1} entries, got {groups + 1}")
    if tensor_scale is not None:
        _need(format == "nvfp4", "mxfp4 has no tensor scale")
        _vector(tensor_scale, "tensor_scale", torch.float32, groups, device)
    check_workspace(ws, device)
    return rows, groups


def _output(X, out, name, shape, dtype):
    t = out.get(name) if out else None
    if t is None:
        return X.new_empty(*shape, dtype=dtype)
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != X.device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {X.device}")
    return t


def gptq_fp4_quantize(X, format="nvfp4", tensor_scale=None, row_index=None, offsets=None, want_deq=False, out=None,
                      ws=None, stream=None):
    """Quantise X [rows, n] (or a stack [groups, rows, n], one group a matrix)
    to 4-bit floating point; returns the dict that the products take (and
    ``deq``, fp32 [rows, n], with ``want_deq``).

    row_index (int32): row i of the result is X's row row_index[i].  offsets
    (int32 [groups + 1]): the result's rows in groups, each with a tensor scale
    of its own.  tensor_scale: use these (fp32 [groups], positive) instead of
    the rows' own maxima.  out: dict of outputs to write into.
    """
    rows, groups = fp4_check_quantize_args(X, format, tensor_scale, row_index, offsets, ws)
    shape, ragged, code = X.shape, offsets is not None, FP4_FORMATS[format]
    n = shape[-1]
    block = 4 * FP4_BLOCK[format]
    stack = len(shape) == 3
    x_rows, ldx = (rows, n) if stack else (shape[0], max(X.stride(0), n))

    where, guard = _enter(X.device, stream)
    try:
        packed = _output(X, out, "packed", (rows, 16 * ((n + 31) // 32)), torch.uint8)
        scales = _output(X, out, "scales", (_bands(rows, groups, ragged), (n + block - 1) // block, 512), torch.uint8)
        t, wp, wbytes, deq = tensor_scale, None, 0, None
        if code == GPTQ_NVFP4 and t is None:
            t = _output(X, out, "tensor_scale", (groups,), torch.float32)
            wbytes = LIB.gptq_fp4_quantize_workspace_size(rows, n, code, groups, ragged)
            if wbytes > 0:
                keep = ws if ws is not None else X.new_empty(wbytes + 256, dtype=torch.uint8)
                wp, wbytes = aligned_workspace(keep)
        q = {"packed": packed, "scales": scales, "tensor_scale": t, "rows": rows, "n": n, "format": format,
             "groups": groups, "offsets": offsets}
        if want_deq:
            q["deq"] = deq = _output(X, out, "deq", (rows, n), torch.float32)
        check("gptq_fp4_quantize",
              LIB.gptq_fp4_quantize(X.data_ptr(), _DTYPES[X.dtype], x_rows, n, ldx,
                                    None if row_index is None else row_index.data_ptr(), rows,
                                    None if offsets is None else offsets.data_ptr(), groups, code,
                                    tensor_scale is not None, None if t is None else t.data_ptr(), packed.data_ptr(),
                                    scales.data_ptr(), None if deq is None else deq.data_ptr(), wp, wbytes, where))
        return q
    finally:
        _leave(guard)


def fp4_check_matrix(q, name, ragged=False):
    """That the dict q holds a quantised matrix as include/gptq.h lays it out
    (ragged: its groups came from offsets)."""
    try:
        p, s, t, rows, n, format, groups = (q["packed"], q["scales"], q["tensor_scale"], q["rows"], q["n"],
                                            q["format"], q["groups"])
    except KeyError as e:
        raise ValueError(f"{name} is no quantised matrix: it lacks {e}") from None
    _check_format(format)
    if groups < 1:
        raise ValueError(f"{name} must have at least one group, got {groups}")
    if not ragged and rows % groups != 0:
        raise ValueError(f"{name} has {rows} rows, which is no multiple of its {groups} groups")
    if p.dtype != torch.uint8 or s.dtype != torch.uint8:
        raise TypeError(f"{name}'s codes and scales must be uint8")
    pitch = 16 * ((n + 31) // 32)
    if p.shape != (rows, pitch) or not p.is_contiguous():
        raise ValueError(f"{name}['packed'] must be contiguous of shape {(rows, pitch)}, got {tuple(p.shape)}")
    bands, block, shape = _bands(rows, groups, ragged), 4 * FP4_BLOCK[format], s.shape
    if len(shape) != 3 or shape[0] < bands or shape != (shape[0], (n + block - 1) // block, 512) or not s.is_contiguous():
        raise ValueError(f"{name}['scales'] must be contiguous of shape {(bands, (n + block - 1) // block, 512)}, "
                         f"got {tuple(shape)}")
    device = p.device
    if s.device != device:
        raise ValueError(f"{name}'s tensors are on different devices")
    if format == "mxfp4":
        if t is not None:
            raise ValueError(f"{name}: mxfp4 has no tensor scales")
    elif t is None:
        raise ValueError(f"{name}: nvfp4 has tensor scales")
    else:
        _vector(t, "a matrix's tensor_scale", torch.float32, groups, device)


def _check_even(offsets, rows, groups, why, stream):
    """That these offsets cut `rows` rows into `groups` groups of one size, in
    which case the scales lie as without offsets.  Reads them (and so waits for
    the stream): only where a matrix is used in another way than it was made."""
    if offsets.is_cuda:
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(offsets.device)):
            if torch.cuda.is_current_stream_capturing():
                raise ValueError(f"{why}, and these cannot be read during a capture")
            at = offsets.tolist()
    else:
        at = offsets.tolist()
    if at != [rows // groups * g for g in range(groups + 1)]:
        raise ValueError(f"{why}, and these are not groups of one size from row 0 on")


def _check_stack(q, name, stream):
    """That q is one group of all its rows, or groups of one size."""
    if q.get("offsets") is not None:
        _check_even(q["offsets"], q["rows"], q["groups"], f"{name}'s rows were grouped by offsets", stream)


def _check_y(y, dtype, tokens, rows, device):
    if y is None:
        if dtype not in _DTYPES:
            raise TypeError(f"unsupported output dtype {dtype}: fp32 or bf16")
        return
    if y.dtype not in _DTYPES:
        raise TypeError(f"unsupported output dtype {y.dtype}: fp32 or bf16")
    if (y.shape != (tokens, rows) or (y.stride(1) != 1 and rows != 1) or (y.stride(0) < rows and tokens > 1) or
            y.device != device):
        raise ValueError(f"y must be {(tokens, rows)} with contiguous rows on {device}")


def _check_experts(w, offsets):
    _vector(offsets, "offsets", torch.int32, w["groups"] + 1, w["packed"].device)
    if w["groups"] > MAX_GROUPS:
        raise ValueError(f"at most {MAX_GROUPS} groups, w has {w['groups']}")


def _product(w, x, offsets, dtype, y, stream):
    fp4_check_matrix(w, "w")
    if offsets is not None:
        _check_experts(w, offsets)
    fp4_check_matrix(x, "x", offsets is not None)
    for key in ("format", "n", "groups"):
        if w[key] != x[key]:
            raise ValueError(f"w and x differ in {key}: {w[key]} and {x[key]}")
    wp, xp, groups, tokens, n = w["packed"], x["packed"], w["groups"], x["rows"], w["n"]
    if xp.device != wp.device:
        raise ValueError(f"w is on {wp.device}, x on {xp.device}")
    rows = w["rows"] // groups
    _check_y(y, dtype, tokens, rows, wp.device)
    _check_stack(w, "w", stream)
    if offsets is None:
        _check_stack(x, "x", stream)
    elif "offsets" in x and x["offsets"] is None:
        _check_even(offsets, tokens, groups, "x was quantised without the product's offsets", stream)

    where, guard = _enter(wp.device, stream)
    try:
        o = y if y is not None else wp.new_empty(tokens, rows, dtype=dtype)
        wt, xt = w["tensor_scale"], x["tensor_scale"]
        wt, xt = (None, None) if wt is None else (wt.data_ptr(), xt.data_ptr())
        ldy = rows if y is None else max(y.stride(0), rows)
        if offsets is None:
            check("gptq_fp4_matmul",
                  LIB.gptq_fp4_matmul(FP4_FORMATS[w["format"]], wp.data_ptr(), w["scales"].data_ptr(), wt, rows, n,
                                      xp.data_ptr(), x["scales"].data_ptr(), xt, tokens, o.data_ptr(),
                                      _DTYPES[o.dtype], ldy, where))
        else:
            check("gptq_fp4_grouped_matmul",
                  LIB.gptq_fp4_grouped_matmul(FP4_FORMATS[w["format"]], wp.data_ptr(), w["scales"].data_ptr(), wt,
                                              groups, rows, n, xp.data_ptr(), x["scales"].data_ptr(), xt, tokens,
                                              offsets.data_ptr(), o.data_ptr(), _DTYPES[o.dtype], ldy, where))
        return o
    finally:
        _leave(guard)


def gptq_fp4_matmul(w, x, dtype=torch.float32, y=None, stream=None):
    """y[i, r] = sum_c W[r, c] X[i, c] of two quantised matrices (dicts of
    gptq_fp4_quantize, same format and width, one group of all rows each): [x
    rows, w rows] in `dtype` (fp32 or bf16), or written into y in its own."""
    if w.get("groups") != 1:
        raise ValueError(f"w has {w.get('groups')} groups: gptq_fp4_grouped_matmul takes them")
    return _product(w, x, None, dtype, y, stream)


def gptq_fp4_grouped_matmul(w, x, offsets, dtype=torch.float32, y=None, stream=None):
    """The product of each group of x's rows (the offsets that x was quantised
    with) with its own matrix of the stack w ([groups, rows, n] quantised): y
    [x rows, rows].  Rows of y outside the offsets are left as they were.

    A matrix whose dict says that it was grouped otherwise (x without offsets,
    w with some) is taken where the offsets make groups of one size, which are
    read back for that: such a call waits for the stream, and is refused during
    a capture."""
    if offsets is None:
        raise ValueError("gptq_fp4_grouped_matmul needs the rows' offsets")
    return _product(w, x, offsets, dtype, y, stream)


def fp4_linear(w, X, dtype=None, tensor_scale=None, row_index=None, offsets=None, y=None, ws=None, stream=None):
    """A 4-bit layer on X [tokens, n] (fp32 or bf16): X is quantised to w's
    format and multiplied with w, in `dtype` (default: X's).  With offsets (and
    a row_index that gathers the rows), each group of rows goes through its own
    matrix of the stack w, as a layer of experts does.  The same result as
    gptq_fp4_quantize and a product, in one call of the library."""
    fp4_check_matrix(w, "w")
    wp, n, groups, format = w["packed"], w["n"], w["groups"], w["format"]
    if X.dim() != 2 or X.shape[1] != n:
        raise ValueError(f"X must be [tokens, {n}], got {tuple(X.shape)}")
    tokens, x_groups = fp4_check_quantize_args(X, format, tensor_scale, row_index, offsets, ws)
    if offsets is not None:
        _check_experts(w, offsets)
    if x_groups != groups:
        raise ValueError(f"w has {groups} groups: give the rows' offsets")
    if X.device != wp.device:
        raise ValueError(f"w is on {wp.device}, X on {X.device}")
    rows = w["rows"] // groups
    if dtype is None:
        dtype = X.dtype
    _check_y(y, dtype, tokens, rows, wp.device)
    _check_stack(w, "w", stream)
    code = FP4_FORMATS[format]
    where, guard = _enter(wp.device, stream)
    try:
        o = y if y is not None else X.new_empty(tokens, rows, dtype=dtype)
        nbytes, base = LIB.gptq_fp4_linear_workspace_size(tokens, rows, n, code, groups, offsets is not None), None
        if nbytes > 0:
            keep = ws if ws is not None else X.new_empty(nbytes + 256, dtype=torch.uint8)
            base, nbytes = aligned_workspace(keep)
        wt = w["tensor_scale"]
        check("gptq_fp4_linear",
              LIB.gptq_fp4_linear(code, wp.data_ptr(), w["scales"].data_ptr(), None if wt is None else wt.data_ptr(),
                                  groups, rows, n, X.data_ptr(), _DTYPES[X.dtype], X.shape[0], max(X.stride(0), n),
                                  None if row_index is None else row_index.data_ptr(), tokens,
                                  None if offsets is None else offsets.data_ptr(),
                                  None if tensor_scale is None else tensor_scale.data_ptr(), o.data_ptr(),
                                  _DTYPES[o.dtype], rows if y is None else max(y.stride(0), rows), base, nbytes, where))
        return o
    finally:
        _leave(guard)
