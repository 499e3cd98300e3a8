"""Operators on caller tensors: token sampling and the 8-bit K/V cache of one
attention layer.  Names follow the C entry points: ``sample`` ->
``dory_sample``, ``KV8Pages.append`` -> ``dory_kv8_append``,
``KV8Pages.attend`` -> ``dory_kv8_attend``.

Tensors live on one CUDA device; work goes to ``stream`` (default: that
device's current stream).  Arguments that do not fit raise ``ValueError``
before anything is enqueued.
"""
import ctypes
import threading

import torch

from . import _lib
from ._lib import DoryKv8, check

PAGE = 64                 # tokens per page
BLOCK = 32                # tokens per scale
LIMIT = 2 ** 31           # sizes are 32-bit in the library

_I64x3 = ctypes.c_int64 * 3
_I64x2 = ctypes.c_int64 * 2
_F32, _I32, _BF16 = torch.float32, torch.int32, torch.bfloat16


def _refuse(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed, got {type(t).__name__}")
    raise ValueError(f"{name}: contiguous {dtype} {tuple(shape)} on {device} is "
                     f"needed, got {t.dtype} {tuple(t.shape)}, strides "
                     f"{t.stride()}, on {t.device}")


def _dense(t, name, dtype, shape, device):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype
            and t.shape == shape and t.device == device and t.is_contiguous()):
        _refuse(t, name, dtype, shape, device)
    return t


def _rows(t, name, n):
    """Element strides of the first n dims of a tensor whose last dim is
    contiguous and whose rows are 16-byte aligned (the strides of dims of
    length 1 do not matter)."""
    s = [0 if size == 1 else st for size, st in zip(t.shape[:n], t.stride())]
    if t.stride(-1) != 1 or t.data_ptr() % 16 or any(x % 8 for x in s):
        raise ValueError(f"{name}: the last dim must be contiguous and every "
                         "row 16-byte aligned")
    return s


def _on_other_rows(out, q):
    """Whether contiguous `out` [B, H, d] shares memory with q [B, H, d] (equal
    sizes, last dim contiguous) and is not q itself."""
    (B, H, d), (sb, sh, _) = q.shape, q.stride()
    at, lo, hi = q.data_ptr(), out.data_ptr(), out.data_ptr() + 2 * out.numel()
    if lo >= at + 2 * ((B - 1) * sb + (H - 1) * sh + d) or hi <= at:
        return False
    if at == lo and q.is_contiguous():
        return False
    rows = (at + 2 * (b * sb + h * sh) for b in range(B) for h in range(H))
    return any(lo < r + 2 * d and r < hi for r in rows)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name}: a CUDA tensor is needed")
    return t.device


def _here(device):
    """The device's current stream if the device is the current one, else
    None (then work is enqueued inside _On)."""
    if torch.cuda.current_device() == device.index:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return None


class _On:
    """The device made current, and `stream` (None: the device's current one),
    so that outputs allocated inside belong to the stream the work goes to."""

    def __init__(self, device, stream):
        if stream is None:
            self.ctx = torch.cuda.device(device)
        elif stream.device != device:
            raise ValueError(f"stream: on {stream.device}, the tensors are on "
                             f"{device}")
        else:
            self.ctx = torch.cuda.stream(stream)
        self.device = device

    def __enter__(self):
        self.ctx.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


def sample(logits, uniform, temperature=None, top_k=None, top_p=None,
           min_p=None, tokens=None, logprobs=False, stream=None):
    """Draw one token per row of logits f32 [B, V] (rows may be strided) from
    uniforms f32 [B] in [0, 1); see dory_sample for the rule.

    temperature, top_p, min_p f32 [B] and top_k int32 [B] are device tensors,
    one value per row, or None.  tokens: int32 [B] to write, or None.
    logprobs: True, or an f32 [B] tensor to write.  Returns (tokens, logprobs
    or None)."""
    dev = _cuda(logits, "logits")
    if logits.dtype is not _F32 or logits.dim() != 2:
        raise ValueError("logits: float32 [B, V] is needed, got "
                         f"{logits.dtype} {tuple(logits.shape)}")
    B, V = row = logits.shape
    ld, step = logits.stride()
    if B <= 1:
        ld = V
    if V < 1 or (V > 1 and step != 1) or ld < V:
        raise ValueError("logits: rows must be contiguous and apart")
    if B >= LIMIT or V >= LIMIT:
        raise ValueError("logits: fewer than 2^31 rows and columns are needed")
    row = row[:1]
    _dense(uniform, "uniform", _F32, row, dev)
    T = k = p = m = None
    if temperature is not None:
        T = _dense(temperature, "temperature", _F32, row, dev).data_ptr()
    if top_k is not None:
        k = _dense(top_k, "top_k", _I32, row, dev).data_ptr()
    if top_p is not None:
        p = _dense(top_p, "top_p", _F32, row, dev).data_ptr()
    if min_p is not None:
        m = _dense(min_p, "min_p", _F32, row, dev).data_ptr()
    if tokens is not None:
        _dense(tokens, "tokens", _I32, row, dev)
    lp = None
    if logprobs is not False and logprobs is not True:
        lp = _dense(logprobs, "logprobs", _F32, row, dev)

    def enqueue(st, tokens, lp):
        if tokens is None:
            tokens = torch.empty_like(uniform, dtype=_I32)
        if logprobs is True:
            lp = torch.empty_like(uniform)
        rc = _lib.load().dory_sample(
            logits.data_ptr(), ld, B, V, T, k, p, m, uniform.data_ptr(),
            tokens.data_ptr(), None if lp is None else lp.data_ptr(), st)
        if rc:
            check("dory_sample", rc)
        return tokens, lp

    st = _here(dev) if stream is None else None
    if st is not None:
        return enqueue(st, tokens, lp)
    with _On(dev, stream) as st:
        return enqueue(st, tokens, lp)


class _Workspaces(threading.local):
    """A thread's workspaces by (stream, heads).  An attention is two launches,
    the second of which reads what the first left in the workspace, and the
    interpreter lock is let go meanwhile: another thread on the same stream
    needs a workspace of its own."""

    def __init__(self):
        self.kept = {}


class KV8Pages:
    """One attention layer's K/V entries in 8 bits (dory_kv8): E4M3 codes in
    64-token pages behind a block table, one power-of-two scale per 32 tokens
    and KV head.  The tensors are the caller's and are only referred to:

    k, v             uint8 [n_pages, n_kv_heads, 64, head_dim]
    k_scale, v_scale float32 [n_pages, n_kv_heads, 2]
    block_table      int32 [batch, pages_per_seq]
    """

    def __init__(self, k, v, k_scale, v_scale, block_table):
        dev = _cuda(k, "k")
        if k.dim() != 4 or k.shape[2] != PAGE or k.shape[3] not in (64, 128, 160):
            raise ValueError("k: uint8 [n_pages, n_kv_heads, 64, head_dim] with "
                             "head_dim 64, 128 or 160 is needed, got "
                             f"{tuple(k.shape)}")
        shape = tuple(k.shape)
        _dense(k, "k", torch.uint8, shape, dev)
        _dense(v, "v", torch.uint8, shape, dev)
        _dense(k_scale, "k_scale", torch.float32, (shape[0], shape[1], 2), dev)
        _dense(v_scale, "v_scale", torch.float32, (shape[0], shape[1], 2), dev)
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
            raise ValueError("block_table: int32 [batch, pages_per_seq] is needed")
        _dense(block_table, "block_table", torch.int32,
               tuple(block_table.shape), dev)
        if 0 in shape or 0 in block_table.shape:
            raise ValueError("an empty cache")
        if max(*shape, *block_table.shape) >= LIMIT:
            raise ValueError("fewer than 2^31 pages and sequences are needed")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.block_table, self.device = block_table, dev
        self.n_kv_heads, self.head_dim = shape[1], shape[3]
        self.batch, self.pages_per_seq = block_table.shape
        self._room = self.pages_per_seq * PAGE           # tokens of a sequence
        self.c = DoryKv8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                         v_scale.data_ptr(), block_table.data_ptr(), shape[0],
                         self.pages_per_seq, self.batch, shape[1], shape[3])
        self._ref = ctypes.byref(self.c)
        # the TMA maps of the pages, built once
        self._plan = ctypes.create_string_buffer(_lib.KV8_PLAN_BYTES + 64)
        plan = -(-ctypes.addressof(self._plan) // 64) * 64
        check("dory_kv8_plan", _lib.load().dory_kv8_plan(self._ref, plan))
        self.c.plan = plan
        self._ws = _Workspaces()
        self._rows = self._q_rows = (None,)
        self._q_heads = [g * shape[1] for g in (1, 2, 4, 8)]

    @classmethod
    def empty(cls, batch, max_ctx, n_kv_heads, head_dim, device="cuda"):
        """A cache of its own: every sequence owns ceil(max_ctx / 64) pages."""
        P = -(-max_ctx // PAGE)
        n = batch * P
        dev = torch.device(device)
        z = dict(dtype=torch.uint8, device=dev)
        o = dict(dtype=torch.float32, device=dev)
        return cls(torch.zeros((n, n_kv_heads, PAGE, head_dim), **z),
                   torch.zeros((n, n_kv_heads, PAGE, head_dim), **z),
                   torch.ones((n, n_kv_heads, 2), **o),
                   torch.ones((n, n_kv_heads, 2), **o),
                   torch.arange(n, dtype=torch.int32, device=dev).view(batch, P))

    def append(self, k, v, pos, n=None, stream=None):
        """Append the first n[b] (None: all) of the rows k, v bf16 [batch, T,
        n_kv_heads, head_dim] (any strides with 16-byte aligned rows) behind
        the pos[b] tokens that sequence b holds; pos, n int32 [batch]."""
        dev, B = self.device, self.batch
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k: bf16 [batch, T, n_kv_heads, head_dim] is needed")
        T = k.shape[1]
        shape = (B, T, self.n_kv_heads, self.head_dim)
        for t, name in ((k, "k"), (v, "v")):
            if not (isinstance(t, torch.Tensor) and t.dtype is _BF16
                    and t.shape == shape and t.device == dev):
                _refuse(t, name, _BF16, shape, dev)
        if T > self.pages_per_seq * PAGE:
            raise ValueError(f"{T} rows, a sequence holds "
                             f"{self.pages_per_seq * PAGE}")
        _dense(pos, "pos", _I32, (B,), dev)
        if n is not None:
            n = _dense(n, "n", _I32, (B,), dev).data_ptr()
        if T == 0:
            return
        # the stride arrays of the last call (of any thread), if the strides are
        # the same
        key = (T, k.stride(), v.stride())
        pk, pv = k.data_ptr(), v.data_ptr()
        rows = self._rows
        if key != rows[0] or pk % 16 or pv % 16:
            rows = self._rows = (key, _I64x3(*_rows(k, "k", 3)),
                                 _I64x3(*_rows(v, "v", 3)))
        args = (self._ref, pk, pv, rows[1], rows[2], T, pos.data_ptr(), n)
        st = _here(dev) if stream is None else None
        if st is not None:
            rc = _lib.load().dory_kv8_append(*args, st)
        else:
            with _On(dev, stream) as st:
                rc = _lib.load().dory_kv8_append(*args, st)
        if rc:
            check("dory_kv8_append", rc)

    def workspace(self, n_q_heads):
        """A workspace for attend with n_q_heads query heads; one
        call at a time may use it."""
        nb = ctypes.c_int64()
        with torch.cuda.device(self.device):
            check("dory_kv8_workspace_bytes",
                  _lib.load().dory_kv8_workspace_bytes(self._ref, n_q_heads,
                                                       ctypes.byref(nb)))
        return torch.empty(nb.value, dtype=torch.uint8, device=self.device)

    def attend(self, q, lens, window=0, scale=None, out=None, ws=None,
               stream=None):
        """Attention of one query per sequence, q bf16 [batch, n_q_heads,
        head_dim], over the lens[b] (int32 [batch]) cached tokens, the last
        `window` of them if window > 0; scale defaults to 1 / sqrt(head_dim).
        Returns bf16 [batch, n_q_heads, head_dim] (`out`, if given, which may
        be a contiguous q itself).  Without
        `ws` this object keeps one workspace per stream and thread, and a
        captured graph gets one of its own; a `ws` given is for one thread and
        one stream at a time."""
        dev, B, hd = self.device, self.batch, self.head_dim
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q: bf16 [batch, n_q_heads, head_dim] is needed")
        Hq = q.shape[1]
        shape = (B, Hq, hd)
        if not (q.dtype is _BF16 and q.shape == shape and q.device == dev):
            _refuse(q, "q", _BF16, shape, dev)
        if Hq not in self._q_heads:
            raise ValueError(f"{Hq} query heads on {self.n_kv_heads} KV heads: "
                             "1, 2, 4 or 8 per KV head are needed")
        _dense(lens, "lens", _I32, (B,), dev)
        if window < 0:
            raise ValueError("window: 0 (off) or more is needed")
        if window > self._room:
            window = self._room
        key, pq = (Hq, q.stride()), q.data_ptr()
        rows = self._q_rows
        if key != rows[0] or pq % 16:
            rows = self._q_rows = (key, _I64x2(*_rows(q, "q", 2)))
        if out is not None:
            _dense(out, "out", _BF16, shape, dev)
            if _on_other_rows(out, q):
                raise ValueError("out: overlaps other rows of q")
        if ws is not None and not (isinstance(ws, torch.Tensor) and ws.dtype is torch.uint8
                                   and ws.device == dev and ws.is_contiguous()):
            raise ValueError(f"ws: contiguous uint8 on {dev} is needed (workspace())")
        if scale is None:
            scale = hd ** -0.5
        st = _here(dev) if stream is None else None
        if st is not None:
            return self._attend(st, pq, rows[1], q, lens, window, scale, out, ws)
        with _On(dev, stream) as st:
            return self._attend(st, pq, rows[1], q, lens, window, scale, out, ws)

    def _attend(self, st, pq, strides, q, lens, window, scale, out, ws):
        Hq = q.shape[1]
        if out is None:
            out = (torch.empty_like(q) if q.is_contiguous()
                   else torch.empty(q.shape, dtype=_BF16, device=self.device))
        if ws is None and torch.cuda.is_current_stream_capturing():
            ws = self.workspace(Hq)          # the graph's own
        elif ws is None:
            ws = self._ws.kept.get((st, Hq))
            if ws is None:
                ws = self._ws.kept[st, Hq] = self.workspace(Hq)
        rc = _lib.load().dory_kv8_attend(
            self._ref, pq, strides, Hq, lens.data_ptr(), window, scale,
            out.data_ptr(), ws.data_ptr(), ws.numel(), st)
        if rc:
            check("dory_kv8_attend", rc)
        return out
