"""4-bit floating point: quantisation, product and product grouped by expert.

A quantised matrix is a dict: ``packed`` uint8 [rows, 16 * ceil(n / 32)] (two
E2M1 codes a byte), ``scales`` uint8 [bands, quads, 512] (scale tiles of 128
rows x 4 blocks), ``tensor_scale`` fp32 [groups] ("nvfp4") or None ("mxfp4"),
and the plain values ``rows``, ``n``, ``format``, ``groups``.  include/gptq.h
defines the formats and layouts; the functions here check arguments, get
outputs and workspaces from torch and call the library.
"""
import torch

from ._lib import GPTQ_BF16, GPTQ_F32, GPTQ_MXFP4, GPTQ_NVFP4, LIB, check

FP4_FORMATS = {"mxfp4": GPTQ_MXFP4, "nvfp4": GPTQ_NVFP4}
FP4_BLOCK = {"mxfp4": 32, "nvfp4": 16}
MAX_GROUPS = 512  # of an offsets tensor
_DTYPES = {torch.float32: GPTQ_F32, torch.bfloat16: GPTQ_BF16}


def _ptr(t):
    return None if t is None else t.data_ptr()


class _Place:
    """Makes the tensors' device and the stream current while outputs are
    allocated and the library is called; ``where`` is the stream's handle."""

    def __init__(self, device, stream):
        self.guard = None
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            self.guard = torch.cuda.stream(stream)
        elif device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        self.where = torch.cuda.current_stream().cuda_stream
        return self

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)


def _need(ok, why):
    if not ok:
        raise ValueError(why)


def _vector(t, name, dtype, length, device):
    """An argument that is a contiguous vector (length None: any)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _need(t.dim() == 1 and t.is_contiguous() and (length is None or t.numel() == length),
          f"{name} must be a contiguous vector{'' if length is None else f' of {length}'}, got {tuple(t.shape)}")
    _need(t.device == device, f"{name} is on {t.device}, the other tensors on {device}")


def _check_format(format):
    if format not in FP4_FORMATS:
        raise ValueError(f"format must be one of {sorted(FP4_FORMATS)}, got {format!r}")


def fp4_check_quantize_args(X, format, tensor_scale=None, row_index=None, offsets=None):
    """The checks gptq_fp4_quantize makes before it touches the device; they
    need no GPU.  Returns (rows, groups) of the result."""
    _check_format(format)
    if X.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {X.dtype}: fp32 or bf16")
    _need(X.dim() in (2, 3), f"X must be [rows, n] or [groups, rows, n], got {tuple(X.shape)}")
    _need(1 <= X.shape[-1] <= 65535, f"X must have 1 to 65535 columns, got {X.shape[-1]}")
    if X.dim() == 3:
        _need(X.is_contiguous(), "a stack of matrices must be contiguous")
        _need(row_index is None and offsets is None, "row_index and offsets go with a matrix, not with a stack")
        _need(X.shape[0] >= 1, "a stack needs at least one matrix")
        rows, groups = X.shape[0] * X.shape[1], X.shape[0]
    else:
        _need(X.stride(1) == 1 or X.shape[1] == 1, "X's rows must be contiguous")
        _need(X.stride(0) >= X.shape[1] or X.shape[0] <= 1, "X's rows must not overlap")
        rows, groups = X.shape[0], 1
    if row_index is not None:
        _vector(row_index, "row_index", torch.int32, None, X.device)
        rows = row_index.numel()
    if offsets is not None:
        _vector(offsets, "offsets", torch.int32, None, X.device)
        groups = offsets.numel() - 1
        _need(1 <= groups <= MAX_GROUPS, f"offsets must have 2 to {MAX_GROUPS + 1} entries, got {offsets.numel()}")
    if tensor_scale is not None:
        _need(format == "nvfp4", "mxfp4 has no tensor scale")
        _vector(tensor_scale, "tensor_scale", torch.float32, groups, X.device)
    return rows, groups


def _output(out, name, shape, dtype, device):
    t = out.get(name)
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t.dtype == dtype and tuple(t.shape) == tuple(shape) and t.is_contiguous() and t.device == device,
          f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
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
    rows, groups = fp4_check_quantize_args(X, format, tensor_scale, row_index, offsets)
    dev = X.device
    _need(dev.type == "cuda", f"X must be on a CUDA device, not on {dev}")
    n, code, ragged = X.shape[-1], FP4_FORMATS[format], offsets is not None
    nv = format == "nvfp4"
    out = out or {}
    block = 4 * FP4_BLOCK[format]
    size = rows // groups
    bands = rows // 128 + groups if ragged else groups * ((size + 127) // 128)
    x_rows, ldx = (rows, n) if X.dim() == 3 else (X.shape[0], max(X.stride(0), n))
    with _Place(dev, stream) as place:
        q = {"packed": _output(out, "packed", (rows, 16 * ((n + 31) // 32)), torch.uint8, dev),
             "scales": _output(out, "scales", (bands, (n + block - 1) // block, 512), torch.uint8, dev),
             "tensor_scale": None, "rows": rows, "n": n, "format": format, "groups": groups}
        if nv:
            q["tensor_scale"] = tensor_scale if tensor_scale is not None else _output(
                out, "tensor_scale", (groups,), torch.float32, dev)
        if want_deq:
            q["deq"] = _output(out, "deq", (rows, n), torch.float32, dev)
        wp, wbytes = None, 0
        if nv and tensor_scale is None:
            wbytes = LIB.gptq_fp4_quantize_workspace_size(rows, n, code, groups, int(ragged))
            if wbytes > 0:
                ws = ws if ws is not None else torch.empty(wbytes + 256, dtype=torch.uint8, device=dev)
                wp = (ws.data_ptr() + 255) & ~255
                wbytes = ws.numel() - (wp - ws.data_ptr())
        check("gptq_fp4_quantize",
              LIB.gptq_fp4_quantize(_ptr(X), _DTYPES[X.dtype], x_rows, n, ldx, _ptr(row_index), rows, _ptr(offsets),
                                    groups, code, int(tensor_scale is not None), _ptr(q["tensor_scale"]),
                                    _ptr(q["packed"]), _ptr(q["scales"]), _ptr(q.get("deq")), wp, wbytes,
                                    place.where))
    return q


def fp4_check_matrix(q, name, ragged=False):
    """That the dict q holds a quantised matrix as include/gptq.h lays it out
    (ragged: its groups came from offsets)."""
    missing = [k for k in ("packed", "scales", "tensor_scale", "rows", "n", "format", "groups") if k not in q]
    _need(not missing, f"{name} is no quantised matrix: it lacks {missing}")
    _check_format(q["format"])
    rows, n, groups = q["rows"], q["n"], q["groups"]
    block = 4 * FP4_BLOCK[q["format"]]
    p, s, t = q["packed"], q["scales"], q["tensor_scale"]
    bands = rows // 128 + groups if ragged else groups * ((rows // groups + 127) // 128)
    _need(ragged or rows % groups == 0, f"{name} has {rows} rows, which is no multiple of its {groups} groups")
    if p.dtype != torch.uint8 or s.dtype != torch.uint8:
        raise TypeError(f"{name}'s codes and scales must be uint8")
    _need(tuple(p.shape) == (rows, 16 * ((n + 31) // 32)) and p.is_contiguous(),
          f"{name}['packed'] must be contiguous of shape {(rows, 16 * ((n + 31) // 32))}, got {tuple(p.shape)}")
    _need(s.dim() == 3 and s.shape[0] >= bands and tuple(s.shape[1:]) == ((n + block - 1) // block, 512) and
          s.is_contiguous(), f"{name}['scales'] must be contiguous of shape {(bands, (n + block - 1) // block, 512)}, "
                             f"got {tuple(s.shape)}")
    _need(s.device == p.device, f"{name}'s tensors are on different devices")
    _need((t is not None) == (q["format"] == "nvfp4"), f"{name}: nvfp4 has tensor scales, mxfp4 none")
    if t is not None:
        _vector(t, f"{name}['tensor_scale']", torch.float32, groups, p.device)


def _product(w, x, offsets, dtype, y, stream):
    fp4_check_matrix(w, "w")
    fp4_check_matrix(x, "x", ragged=offsets is not None)
    _need(w["format"] == x["format"], f"w is {w['format']}, x is {x['format']}")
    _need(w["n"] == x["n"], f"w has {w['n']} columns, x has {x['n']}")
    _need(w["groups"] == x["groups"], f"w has {w['groups']} groups, x has {x['groups']}")
    dev = w["packed"].device
    _need(x["packed"].device == dev, f"w is on {dev}, x on {x['packed'].device}")
    groups, tokens = w["groups"], x["rows"]
    rows = w["rows"] // groups
    if y is None:
        if dtype not in _DTYPES:
            raise TypeError(f"unsupported output dtype {dtype}: fp32 or bf16")
    else:
        if y.dtype not in _DTYPES or (dtype is not None and y.dtype != dtype):
            raise TypeError(f"unsupported output dtype {y.dtype}")
        _need(tuple(y.shape) == (tokens, rows) and (y.stride(1) == 1 or rows == 1) and
              (y.stride(0) >= rows or tokens <= 1) and y.device == dev,
              f"y must be {(tokens, rows)} with contiguous rows on {dev}")
    _need(dev.type == "cuda", f"the matrices must be on a CUDA device, not on {dev}")
    with _Place(dev, stream) as place:
        if y is None:
            y = torch.empty((tokens, rows), dtype=dtype, device=dev)
        ldy = max(y.stride(0), rows)
        if offsets is None:
            check("gptq_fp4_matmul",
                  LIB.gptq_fp4_matmul(FP4_FORMATS[w["format"]], _ptr(w["packed"]), _ptr(w["scales"]),
                                      _ptr(w["tensor_scale"]), rows, w["n"], _ptr(x["packed"]), _ptr(x["scales"]),
                                      _ptr(x["tensor_scale"]), tokens, _ptr(y), _DTYPES[y.dtype], ldy, place.where))
        else:
            check("gptq_fp4_grouped_matmul",
                  LIB.gptq_fp4_grouped_matmul(FP4_FORMATS[w["format"]], _ptr(w["packed"]), _ptr(w["scales"]),
                                              _ptr(w["tensor_scale"]), groups, rows, w["n"], _ptr(x["packed"]),
                                              _ptr(x["scales"]), _ptr(x["tensor_scale"]), tokens, _ptr(offsets),
                                              _ptr(y), _DTYPES[y.dtype], ldy, place.where))
    return y


def gptq_fp4_matmul(w, x, dtype=torch.float32, y=None, stream=None):
    """y[i, r] = sum_c W[r, c] X[i, c] of two quantised matrices (dicts of
    gptq_fp4_quantize, same format and width): [x rows, w rows] in `dtype`
    (fp32 or bf16), or written into y."""
    _need(w.get("groups") == 1, f"w has {w.get('groups')} groups: gptq_fp4_grouped_matmul takes them")
    return _product(w, x, None, dtype if y is None else None, y, stream)


def gptq_fp4_grouped_matmul(w, x, offsets, dtype=torch.float32, y=None, stream=None):
    """The product of each group of x's rows (offsets as x was quantised with)
    with its own matrix of the stack w ([groups, rows, n] quantised): y
    [x rows, rows].  Rows of y outside the offsets are left as they were."""
    _vector(offsets, "offsets", torch.int32, None, w["packed"].device)
    _need(offsets.numel() == w["groups"] + 1, f"offsets has {offsets.numel()} entries for {w['groups']} groups")
    _need(w["groups"] <= MAX_GROUPS, f"at most {MAX_GROUPS} groups, w has {w['groups']}")
    return _product(w, x, offsets, dtype if y is None else None, y, stream)


def fp4_linear(w, X, dtype=None, tensor_scale=None, row_index=None, offsets=None, y=None, stream=None):
    """A 4-bit layer on X [tokens, n] (fp32 or bf16): X is quantised to w's
    format and multiplied with w, in `dtype` (default: X's).  With offsets (and
    a row_index that gathers the rows), each group of rows goes through its own
    matrix of the stack w, as a layer of experts does."""
    x = gptq_fp4_quantize(X, w["format"], tensor_scale=tensor_scale, row_index=row_index, offsets=offsets,
                          stream=stream)
    dtype = X.dtype if dtype is None else dtype
    if offsets is None:
        return gptq_fp4_matmul(w, x, dtype=dtype, y=y, stream=stream)
    return gptq_fp4_grouped_matmul(w, x, offsets, dtype=dtype, y=y, stream=stream)
