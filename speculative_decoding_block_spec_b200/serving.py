"""The serving operators: logit rules, token history, paged-cache tables.

The calls around a verify step that depend on lengths and tokens which only
the device knows (include/specv.h, "Serving state"):

  dvl_allocate_pack -> spec_kv_map -> target forward -> spec_logit_rules
  -> spec_verify_* -> spec_history_add, spec_kv_release

State lives in tables with one row per seat, the place a request keeps from
its first to its last token. History and KvPages hold those tables; they are
ordinary tensors that a program reads and writes in place.
"""
import ctypes

import torch

from . import SpecError, Workspace, _dtype_code, lib

_I32, _F32, _I64 = torch.int32, torch.float32, torch.int64
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}  # spec_dtype


class _CHistory(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("counts", "seen", "repetition", "frequency", "presence", "bias_tokens",
                                               "bias_values")] + \
               [("n_bias", ctypes.c_int32), ("seats", ctypes.c_int32), ("V", ctypes.c_int64)]


class _CPages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("page_table", "owned", "free_pages", "free_count")] + \
               [(n, ctypes.c_int32) for n in ("seats", "max_pages", "n_pages", "page_size")]


def _check(t, name, dtype, shape, device=None):
    """Raises unless t is a contiguous tensor of `dtype` and `shape` (a number: that many dimensions of any size; None
    in it: any size) on device number `device` (-1: host); returns its address. Shapes come first, so a mis-sized
    tensor is named even where there is no CUDA device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    s = t.shape
    if shape.__class__ is int:
        if len(s) != shape:
            raise ValueError("%s has shape %s, expected %d dimensions" % (name, tuple(s), shape))
    elif s != shape:
        if len(s) != len(shape) or any(w is not None and g != w for g, w in zip(s, shape)):
            raise ValueError("%s has shape %s, expected %s"
                             % (name, tuple(s), tuple("*" if w is None else w for w in shape)))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.get_device() != device:
        raise ValueError("%s is on %s, the call's other tensors on device %d" % (name, t.device, device))
    return t.data_ptr()


class History:
    """The token history of `seats` requests, and their penalties and biases.

    counts [seats, V] int32 (output tokens), seen [seats, ceil(V/32)] int32
    (bit v%32 of word v//32: prompt or output holds v), repetition, frequency,
    presence [seats] fp32 (None: off), bias_tokens [seats, n] int32 (negative:
    unused) with bias_values [seats, n] fp32. History.empty allocates them."""

    def __init__(self, counts, seen, repetition=None, frequency=None, presence=None, bias_tokens=None,
                 bias_values=None):
        c = _CHistory()
        c.counts = _check(counts, "counts", _I32, (None, None))
        seats, V = counts.shape
        dev = counts.get_device()
        c.seen = _check(seen, "seen", _I32, (seats, (V + 31) // 32), dev)
        c.repetition = None if repetition is None else _check(repetition, "repetition", _F32, (seats,), dev)
        c.frequency = None if frequency is None else _check(frequency, "frequency", _F32, (seats,), dev)
        c.presence = None if presence is None else _check(presence, "presence", _F32, (seats,), dev)
        if (bias_tokens is None) != (bias_values is None):
            raise ValueError("bias_tokens and bias_values go together")
        n = 0
        if bias_tokens is not None:
            c.bias_tokens = _check(bias_tokens, "bias_tokens", _I32, (seats, None), dev)
            n = bias_tokens.shape[1]
            c.bias_values = _check(bias_values, "bias_values", _F32, (seats, n), dev)
        c.n_bias, c.seats, c.V = n, seats, V
        self._c, self._ref, self._dev, self.seats, self.V = c, ctypes.byref(c), dev, seats, V
        self._tensors = (counts, seen, repetition, frequency, presence, bias_tokens, bias_values)

    @classmethod
    def empty(cls, seats, V, n_bias=0, device="cuda"):
        """Empty histories with neutral penalties (r = 1, f = p = 0) and n_bias unused bias entries a seat."""
        z = dict(device=device)
        bias = (None, None) if n_bias == 0 else (torch.full((seats, n_bias), -1, dtype=_I32, **z),
                                                 torch.zeros((seats, n_bias), dtype=_F32, **z))
        return cls(torch.zeros((seats, V), dtype=_I32, **z), torch.zeros((seats, (V + 31) // 32), dtype=_I32, **z),
                   torch.ones(seats, dtype=_F32, **z), torch.zeros(seats, dtype=_F32, **z),
                   torch.zeros(seats, dtype=_F32, **z), *bias)

    counts = property(lambda self: self._tensors[0])
    seen = property(lambda self: self._tensors[1])
    repetition = property(lambda self: self._tensors[2])
    frequency = property(lambda self: self._tensors[3])
    presence = property(lambda self: self._tensors[4])
    bias_tokens = property(lambda self: self._tensors[5])
    bias_values = property(lambda self: self._tensors[6])


class KvPages:
    """The pages of a paged cache: page_table [seats, max_pages] int32, owned
    [seats] int32, free_pages [n_pages] int32 (a stack) and free_count [1]
    int32. KvPages.empty allocates them with every page free."""

    def __init__(self, page_table, owned, free_pages, free_count, page_size):
        c = _CPages()
        c.page_table = _check(page_table, "page_table", _I32, (None, None))
        dev = page_table.get_device()
        c.seats, c.max_pages = page_table.shape
        c.owned = _check(owned, "owned", _I32, (c.seats,), dev)
        c.free_pages = _check(free_pages, "free_pages", _I32, (None,), dev)
        c.free_count = _check(free_count, "free_count", _I32, (1,), dev)
        if not 1 <= int(page_size) <= 0x7fffffff:
            raise ValueError("page_size must be positive")
        c.n_pages, c.page_size = free_pages.shape[0], int(page_size)
        self._c, self._ref, self._dev, self.page_size = c, ctypes.byref(c), dev, int(page_size)
        self.seats, self.max_pages, self.n_pages = c.seats, c.max_pages, c.n_pages
        self._tensors = (page_table, owned, free_pages, free_count)

    @classmethod
    def empty(cls, seats, max_pages, n_pages, page_size, device="cuda"):
        """Nobody holds a page; page 0 is handed out first."""
        return cls(torch.full((seats, max_pages), -1, dtype=_I32, device=device),
                   torch.zeros(seats, dtype=_I32, device=device),
                   torch.arange(n_pages - 1, -1, -1, dtype=_I32, device=device),
                   torch.full((1,), n_pages, dtype=_I32, device=device), page_size)

    page_table = property(lambda self: self._tensors[0])
    owned = property(lambda self: self._tensors[1])
    free_pages = property(lambda self: self._tensors[2])
    free_count = property(lambda self: self._tensors[3])


def _raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# the same handle without a Stream object made for it, and the current device without a check for CUDA (the tensors
# are on it), where torch offers them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(device, workspace, nbytes, name, *args):
    """The library call on the current stream of device number `device`, with that device current. Without a
    workspace, the call gets one of its own."""
    if device < 0:
        raise TypeError("%s: tensors must be CUDA tensors" % name)
    if _current_device() != device:
        with torch.cuda.device(device):
            return _launch(device, workspace, nbytes, name, *args)
    if workspace is None:
        workspace = Workspace(nbytes, torch.device("cuda", device))
    buf = workspace.buf
    if buf.get_device() != device:
        raise ValueError("workspace is on %s, the call's other tensors on device %d" % (buf.device, device))
    st = getattr(lib(), name)(*args, buf.data_ptr(), buf.numel(), _raw_stream(device))
    if st != 0:
        raise SpecError(name, st)


def rules_workspace_size(B):
    return int(lib().spec_rules_workspace_size(B))


def kv_workspace_size(B):
    return int(lib().spec_kv_workspace_size(B))


def spec_logit_rules(logits, history=None, *, seats=None, draft_tokens=None, verify_len=None, target_row_off=None,
                     mask=None, mask_rows=None, out=None, workspace=None):
    """Penalties, biases and grammar masks on the rows of a verify step: on the
    target rows, and on draft rows only where the drafter drew each token from
    the row edited in the same way (a block drafter's rows, which it drew from
    unedited, stay as they are; include/specv.h says why).

    logits  target rows [B, L+1, V], or packed [n, V] with target_row_off [B]
            (or [B + 1]), or draft rows [B, L, V] / [B, K, L, V]; bf16 or fp32.
            L is draft_tokens' [B, L]; without draft_tokens the rows are
            target rows of L = rows - 1 (a decoding step: [B, 1, V]).
    history History with the requests' penalties (None: mask only);
    seats   [B] int32, the request's seat (None: request b sits in seat b,
            negative: none).
    mask    [M, >= rows, ceil(V/32)] int32, bit v%32 of word v//32 set where
            token v is allowed; mask_rows [B] int32, the request's mask or
            negative (None: mask b).
    out     None: in place. Returns the edited rows."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a tensor")
    dev, shape, K = logits.get_device(), logits.shape, 1
    dims = len(shape)
    V = shape[-1] if dims else 0
    L = tp = None
    if draft_tokens is not None:
        tp = _check(draft_tokens, "draft_tokens", _I32, 2, dev)
        B, L = draft_tokens.shape
    if target_row_off is not None:
        if L is None:
            raise ValueError("packed rows need draft_tokens [B, L]")
        if dims != 2:
            raise ValueError("logits has shape %s, expected packed rows [*, V]" % (tuple(shape),))
        if target_row_off.dim() != 1 or target_row_off.shape[0] not in (B, B + 1):
            raise ValueError("target_row_off must be [B] or [B + 1] with B = %d" % B)
        rows = L + 1
    else:
        if dims == 4:
            K = shape[1]
        elif dims != 3:
            raise ValueError("logits has shape %s, expected [B, rows, V] or [B, K, rows, V]" % (tuple(shape),))
        rows = shape[-2]
        if L is None:
            B, L = shape[0], max(rows - 1, 0)
            if history is not None and L > 0:
                raise ValueError("draft_tokens [B, L]: the history of row i holds the drafted tokens before it")
        if shape[0] != B or rows not in (L, L + 1):
            raise ValueError("logits has shape %s, expected %d requests of %d (draft) or %d (target) rows"
                             % (tuple(shape), B, L, L + 1))
    dtype = logits.dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        dt = _dtype_code(logits)  # raises
    xp = _check(logits, "logits", dtype, shape, dev)
    op = xp if out is None else _check(out, "out", dtype, shape, dev)
    rp = None if target_row_off is None else _check(target_row_off, "target_row_off", _I32, 1, dev)
    vp = None if verify_len is None else _check(verify_len, "verify_len", _I32, (B,), dev)
    sp = None if seats is None else _check(seats, "seats", _I32, (B,), dev)
    hp = None
    if history is not None:
        if history._dev != dev or history.V != V:
            raise ValueError("history holds V = %d on device %d, logits V = %d on device %d"
                             % (history.V, history._dev, V, dev))
        if seats is None and B > history.seats:
            raise ValueError("seats: %d requests for %d seats" % (B, history.seats))
        hp = history._ref
    n_masks = mask_len = 0
    mp = np_ = None
    if mask is not None:
        mp = _check(mask, "mask", _I32, (None, None, (V + 31) // 32), dev)
        n_masks, mask_len = mask.shape[0], mask.shape[1]
        if mask_len < rows or n_masks < 1:
            raise ValueError("mask has shape %s, expected at least %d rows a mask" % (tuple(mask.shape), rows))
        np_ = None if mask_rows is None else _check(mask_rows, "mask_rows", _I32, (B,), dev)
        if mask_rows is None and n_masks < B:
            raise ValueError("mask_rows: %d requests for %d masks" % (B, n_masks))
    elif mask_rows is not None:
        raise ValueError("mask_rows needs mask")
    n_rows = shape[0] if target_row_off is not None else B * K * rows
    _launch(dev, workspace, 256, "spec_logit_rules", xp, op, dt, rp, n_rows, B, K, rows, L, V, tp, vp, hp, sp, mp,
            n_masks, mask_len, np_)
    return logits if out is None else out


def spec_history_add(history, tokens, *, seats=None, offsets=None, output=True, workspace=None):
    """Tokens enter the history of their requests' seats: tokens [B, M] int32
    (negative: padding; the out_tokens of a verify call), or [N] with offsets
    [B + 1] int32. output: generated tokens (counted), else prompt tokens."""
    dev = history._dev
    if offsets is None:
        tp = _check(tokens, "tokens", _I32, 2, dev)
        B = tokens.shape[0]
        op = None
    else:
        tp = _check(tokens, "tokens", _I32, 1, dev)
        op = _check(offsets, "offsets", _I32, 1, dev)
        B = offsets.shape[0] - 1
    sp = None if seats is None else _check(seats, "seats", _I32, (B,), dev)
    if seats is None and B > history.seats:
        raise ValueError("seats: %d requests for %d seats" % (B, history.seats))
    _launch(dev, workspace, 256, "spec_history_add", history._ref, sp, B, tp, tokens.numel(), op, 1 if output else 0)


def spec_history_clear(history, seats, *, workspace=None):
    """Empties the history of seats [B] int32 (negative: skipped)."""
    dev = history._dev
    sp = _check(seats, "seats", _I32, 1, dev)
    _launch(dev, workspace, 256, "spec_history_clear", history._ref, sp, seats.shape[0])


def spec_kv_map(pages, ctx_len, offsets, n_tokens, *, seats=None, block_table=None, out=None, workspace=None):
    """Pages, cache slots and block table for a step that appends tokens
    offsets[b] .. offsets[b+1] ([B + 1] int32, e.g. from dvl_allocate_pack)
    behind the ctx_len [B] int32 tokens of each request. n_tokens: capacity of
    the outputs. block_table [B, max_pages] int32 (None: not written).
    Returns (kv_slots [n_tokens] int64, positions [n_tokens] int32, seq_len [B] int32)."""
    dev = pages._dev
    cp = _check(ctx_len, "ctx_len", _I32, 1, dev)
    B, N = ctx_len.shape[0], int(n_tokens)
    fp = _check(offsets, "offsets", _I32, (B + 1,), dev)
    sp = None if seats is None else _check(seats, "seats", _I32, (B,), dev)
    if seats is None and B > pages.seats:
        raise ValueError("seats: %d requests for %d seats" % (B, pages.seats))
    bp = None if block_table is None else _check(block_table, "block_table", _I32, (B, pages.max_pages), dev)
    if out is None:
        on = ctx_len.device
        out = (torch.empty(N, dtype=_I64, device=on), torch.empty(N, dtype=_I32, device=on),
               torch.empty(B, dtype=_I32, device=on))
    slots, positions, seq_len = out
    kp = _check(slots, "kv_slots", _I64, (N,), dev)
    pp = None if positions is None else _check(positions, "positions", _I32, (N,), dev)
    qp = _check(seq_len, "seq_len", _I32, (B,), dev)
    _launch(dev, workspace, 512, "spec_kv_map", pages._ref, sp, B, cp, fp, N, kp, pp, qp, bp)
    return out


def spec_kv_release(pages, seats, *, keep_len=None, workspace=None):
    """Requests in seats [B] int32 (negative: skipped) give back the pages
    behind their first keep_len [B] int32 tokens (None: all of them)."""
    dev = pages._dev
    sp = _check(seats, "seats", _I32, 1, dev)
    B = seats.shape[0]
    kp = None if keep_len is None else _check(keep_len, "keep_len", _I32, (B,), dev)
    _launch(dev, workspace, 512, "spec_kv_release", pages._ref, sp, B, kp)
