"""The decode loop's operators next to the verify step (``specdecode.h``):
beam selection over beams and vocabulary, the reordering of beam states, and
the block tables, slot maps and moves of a paged cache.

As in the package itself, the classes bind a call's buffers once, for loops,
and the functions of the same name make one call.  Buffers that a call does
not get are allocated on its stream (`stream`, by default the current one when
the call is bound), every call enqueues kernels only, and ``error_word``
collects SV_ERR_* bits until the caller clears it.  A bound object is one call
at a time: two that may overlap need two objects with buffers of their own.
Tensors of a call live on one GPU, which need not be the current one.
"""
from __future__ import annotations

import ctypes

import torch

SV_ERR_SCORE = 128
SV_ERR_PARENT = 256
SV_ERR_LENGTH = 512
SV_ERR_PAGES = 1024
SV_ERR_PAGE = 2048
MAX_BEAMS = 32
MAX_CANDIDATES = 64
MAX_POOLS = 1024


def bind_library(lib: ctypes.CDLL) -> None:
    """Declare the entry points of specdecode.h on the loaded library."""
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.spec_beam_select_workspace_size.argtypes = [i32] * 5
    lib.spec_beam_select_workspace_size.restype = sz
    lib.spec_beam_select.argtypes = [P, i32, i32, i32, i32, i64, i64, P, P, P, i32, i32, P, P, P, P, P, P, sz, P]
    lib.spec_beam_reorder.argtypes = [P, i32, i32, i32, i32, i32, i64, P, P, P, P]
    lib.spec_beam_reorder_paged.argtypes = [P, i32, i32, i32, i32, i32, i64, i32, P, i32, P, P, P, i32, P, P]
    lib.spec_cache_extend.argtypes = [P, P, i32, i32, P, i32, i32, P, i32, P, P, i32, P, P, P, P, P, P, P, P]
    lib.spec_cache_commit.argtypes = [P, P, P, i32, P, i32, P, i32, i32, P, i32, P, P, P, P, P, P]
    lib.spec_cache_compact.argtypes = [P, i32, i32, i32, i32, i64, i32, P, i32, P, i32, P, P, i32, P, P]
    for name in ("spec_beam_select", "spec_beam_reorder", "spec_beam_reorder_paged", "spec_cache_extend",
                 "spec_cache_commit", "spec_cache_compact"):
        getattr(lib, name).restype = i32


def _need(name: str, t, shape, dtype=torch.int32, device=None) -> torch.Tensor:
    """`t` if it is a contiguous GPU tensor of this shape and type."""
    if not torch.is_tensor(t) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, the device of the call's other tensors")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {str(dtype).replace('torch.', '')} tensor")
    return t


def _overlap(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether two contiguous tensors share memory."""
    x0, y0 = x.data_ptr(), y.data_ptr()
    return (x0 < y0 + y.numel() * y.element_size() and y0 < x0 + x.numel() * x.element_size()
            and x.numel() > 0 and y.numel() > 0)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


class _Bound:
    """A call of one entry point: function, arguments, device and stream."""

    def _bind(self, device, stream):
        from . import _check, load_library
        self._lib = load_library()
        self._check = _check
        self._device = device
        self._stream = torch.cuda.current_stream(device) if stream is None else stream
        if self._stream.device != device:
            raise ValueError(f"the stream must be one of {device}, the device of the call's tensors")
        return self._lib

    def _new(self, shape, dtype=torch.int32, zero=False):
        with torch.cuda.stream(self._stream):
            return (torch.zeros if zero else torch.empty)(shape, dtype=dtype, device=self._device)

    def _run(self) -> None:
        if torch.cuda.current_device() == self._device.index:
            status = self._fn(*self._args)
        else:
            with torch.cuda.device(self._device):
                status = self._fn(*self._args)
        if status:
            self._check(status)


class BeamSelector(_Bound):
    """Beam search's selection (spec_beam_select): the M best continuations
    of every sequence over its W beams and the vocabulary.

    logits [B, W, V] float32 or bfloat16, the last dimension contiguous, the
    others at any stride (expanded ones too); scores [B, W] float32, the beams'
    cumulative log-probabilities (-inf: a dead beam, whose logits have no effect); temperature
    None (1), a float or a [B] float32 tensor; finished [B, W] int32: beams
    whose only continuation is `eos` at their score.  Each call returns
    (scores [B, M], parent [B, M], tokens [B, M], finished [B, M],
    error_word [1]), best first, -inf and -1 past the last candidate.  The
    outputs are allocated unless passed in; with M == W out_scores may be
    `scores` and out_finished may be `finished`.
    """

    def __init__(self, logits: torch.Tensor, scores: torch.Tensor, M: int, *, temperature=None,
                 finished: torch.Tensor | None = None, eos: int = -1, workspace: torch.Tensor | None = None,
                 out_scores: torch.Tensor | None = None, out_parent: torch.Tensor | None = None,
                 out_tokens: torch.Tensor | None = None, out_finished: torch.Tensor | None = None, stream=None):
        from . import SpecVerifyError, _dtype_code
        if logits.dim() != 3:
            raise ValueError("logits must be [B, W, V]")
        B, W, V = logits.shape
        code = _dtype_code(logits)
        if not logits.is_cuda:
            raise ValueError("logits must be a CUDA tensor")
        if V > 1 and logits.stride(2) != 1:
            raise ValueError("the vocabulary must be contiguous in logits")
        if not 1 <= W <= MAX_BEAMS or not 1 <= M <= MAX_CANDIDATES:
            raise ValueError(f"W must be in [1, {MAX_BEAMS}] and M in [1, {MAX_CANDIDATES}]")
        if not -1 <= eos < V or (finished is not None and eos < 0):
            raise ValueError("eos must be a token, or -1 when no beam is finished")
        dev = logits.device
        lib = self._bind(dev, stream)
        _need("scores", scores, (B, W), torch.float32, dev)
        if finished is not None:
            _need("finished", finished, (B, W), torch.int32, dev)
        if temperature is not None and not torch.is_tensor(temperature):
            value, temperature = float(temperature), self._new((B,), torch.float32)
            with torch.cuda.stream(self._stream):
                temperature.fill_(value)
        if temperature is not None:
            _need("temperature", temperature, (B,), torch.float32, dev)
        n = int(lib.spec_beam_select_workspace_size(B, W, V, code, M))
        if n == 0:
            raise SpecVerifyError("invalid sizes for a workspace")
        if workspace is None:
            workspace = self._new((n,), torch.uint8)
        elif not workspace.is_cuda or workspace.device != dev:
            raise ValueError("workspace must be a CUDA tensor of the logits' device")
        out = []
        for name, t, dtype, own in (("out_scores", out_scores, torch.float32, scores),
                                    ("out_parent", out_parent, torch.int32, None),
                                    ("out_tokens", out_tokens, torch.int32, None),
                                    ("out_finished", out_finished, torch.int32, finished)):
            t = self._new((B, M), dtype) if t is None else _need(name, t, (B, M), dtype, dev)
            if own is not None and _overlap(t, own) and not (M == W and t.data_ptr() == own.data_ptr()):
                raise ValueError(f"{name} can share memory with the call's input only as that input, when M == W")
            out.append(t)
        self.error_word = self._new((1,), zero=True)
        self._out = (*out, self.error_word)
        self._keep = (logits, scores, temperature, finished, workspace)
        self._fn = lib.spec_beam_select
        self._args = (logits.data_ptr(), B, W, V, code, logits.stride(0), logits.stride(1), _ptr(scores),
                      _ptr(temperature), _ptr(finished), int(eos), int(M), *(_ptr(t) for t in out),
                      _ptr(self.error_word), _ptr(workspace), workspace.numel() * workspace.element_size(),
                      self._stream.cuda_stream)

    def __call__(self):
        self._run()
        return self._out


def beam_select(logits: torch.Tensor, scores: torch.Tensor, M: int, **kw):
    """One call of BeamSelector."""
    return BeamSelector(logits, scores, M, **kw)()


def _pools(pools, ndim: int, what: str):
    """The caches of a call, a tensor with a leading dimension of caches or a
    sequence of tensors, as (device pointers, common shape, row bytes, device)."""
    stack = torch.is_tensor(pools)
    every = [pools] if stack and pools.dim() == ndim else list(pools)
    if not 1 <= len(every) <= MAX_POOLS:
        raise ValueError(f"between 1 and {MAX_POOLS} caches, each {what}")
    first = every[0]
    for p in every:
        if not torch.is_tensor(p) or not p.is_cuda or p.dim() != ndim or not p.is_contiguous():
            raise ValueError(f"every cache must be a contiguous CUDA tensor {what}")
        if p.shape != first.shape or p.dtype != first.dtype or p.device != first.device:
            raise ValueError("the caches of a call must have one shape, type and device")
    size = first.numel() * first.element_size()
    at = sorted(p.data_ptr() for p in every)
    if size and any(y - x < size for x, y in zip(at, at[1:])):
        raise ValueError("the caches of a call may not overlap")
    ptrs = (ctypes.c_void_p * len(every))(*(p.data_ptr() for p in every))
    return ptrs, every, first.shape, first.shape[-1] * first.element_size(), first.device


class BeamReorder(_Bound):
    """Beam states after a selection, in place: beam j of sequence b takes
    over the state of beam parent[b, j] (-1: keeps its own) at positions
    below length[b].

    Dense caches are [B * W, G, S, D] tensors of any type (G: heads before
    positions, or 1; length None: all S positions).  With block_table
    [B * W, max_blocks] int32 they are pools [num_pages, G, page_size, D]
    (spec_beam_reorder_paged), length is needed, and positions below start[b]
    (None: 0), which beams may share, are left alone; max_length bounds
    length (default: what a block table holds).  `pools` is one cache, a
    sequence of them, or a tensor with a leading dimension of caches: all move
    in one launch per 128.
    """

    def __init__(self, pools, parent: torch.Tensor, *, length: torch.Tensor | None = None,
                 block_table: torch.Tensor | None = None, start: torch.Tensor | None = None,
                 max_length: int | None = None, stream=None):
        paged = block_table is not None
        what = "[num_pages, G, page_size, D]" if paged else "[B * W, G, S, D]"
        ptrs, every, shape, row, dev = _pools(pools, 4, what)
        if parent.dim() != 2 or not 1 <= parent.shape[1] <= MAX_BEAMS:
            raise ValueError(f"parent must be [B, W] with W in [1, {MAX_BEAMS}]")
        B, W = parent.shape
        lib = self._bind(dev, stream)
        _need("parent", parent, (B, W), torch.int32, dev)
        if length is not None:
            _need("length", length, (B,), torch.int32, dev)
        if shape[1] < 1 or row < 1:
            raise ValueError("a cache needs heads and row elements")
        self.error_word = self._new((1,), zero=True)
        self._keep = (every, parent, length, block_table, start, ptrs)
        tail = (_ptr(self.error_word), self._stream.cuda_stream)
        if not paged:
            if start is not None or max_length is not None:
                raise ValueError("start and max_length go with a block table")
            if shape[0] != B * W:
                raise ValueError("a dense cache must be [B * W, G, S, D]")
            self._fn = lib.spec_beam_reorder
            self._args = (ptrs, len(every), B, W, shape[1], shape[2], row, _ptr(parent), _ptr(length), *tail)
            return
        if length is None:
            raise ValueError("length is needed with a block table")
        if block_table.dim() != 2 or shape[2] < 1:
            raise ValueError("block_table must be [B * W, max_blocks] and pages hold at least one position")
        blocks = block_table.shape[1]
        _need("block_table", block_table, (B * W, blocks), torch.int32, dev)
        if start is not None:
            _need("start", start, (B,), torch.int32, dev)
        most = blocks * shape[2] if max_length is None else int(max_length)
        self._fn = lib.spec_beam_reorder_paged
        self._args = (ptrs, len(every), B, W, shape[1], shape[2], row, shape[0], _ptr(block_table), blocks,
                      _ptr(parent), _ptr(start), _ptr(length), most, *tail)

    def __call__(self) -> None:
        self._run()


def beam_reorder(pools, parent: torch.Tensor, **kw) -> None:
    """One call of BeamReorder."""
    BeamReorder(pools, parent, **kw)()


class CacheExtend(_Bound):
    """Pages, block tables and slot maps for the new tokens of a batch
    (spec_cache_extend): sequence b holds seq_len[b] tokens and gets
    new_len[b] + extra more (new_len None: extra), with pages from the end of
    free_list [num_pages], whose length is free_count [1] (int32 all).

    Each call extends block_table [B, max_blocks] in place, writes what is
    left to free_count_out (default: free_count) and returns (slots
    [max_tokens] int64, positions, seq_ids [max_tokens], query_start [B + 1],
    granted [B]); slots are -1 behind the last token and for sequences that
    were not granted their pages.
    """

    def __init__(self, seq_len: torch.Tensor, block_table: torch.Tensor, free_list: torch.Tensor,
                 free_count: torch.Tensor, page_size: int, max_tokens: int, *, new_len: torch.Tensor | None = None,
                 extra: int = 0, free_count_out: torch.Tensor | None = None, granted: torch.Tensor | None = None,
                 error_word: torch.Tensor | None = None, stream=None):
        if block_table.dim() != 2 or free_list.dim() != 1:
            raise ValueError("block_table must be [B, max_blocks] and free_list [num_pages]")
        B, blocks = block_table.shape
        dev = block_table.device
        _need("block_table", block_table, (B, blocks))
        lib = self._bind(dev, stream)
        _need("seq_len", seq_len, (B,), torch.int32, dev)
        _need("free_list", free_list, free_list.shape, torch.int32, dev)
        _need("free_count", free_count, (1,), torch.int32, dev)
        if new_len is not None:
            _need("new_len", new_len, (B,), torch.int32, dev)
        free_count_out = free_count if free_count_out is None else _need("free_count_out", free_count_out, (1,),
                                                                         torch.int32, dev)
        n = int(max_tokens)
        if n < 0:
            raise ValueError("max_tokens must not be negative")
        self.slots = self._new((n,), torch.int64)
        self.positions, self.seq_ids = self._new((n,)), self._new((n,))
        self.query_start, self.page_start = self._new((B + 1,), zero=True), self._new((B + 1,), zero=True)
        self.granted = self._new((B,)) if granted is None else _need("granted", granted, (B,), torch.int32, dev)
        self.error_word = (self._new((1,), zero=True) if error_word is None
                           else _need("error_word", error_word, (1,), torch.int32, dev))
        if B == 0:  # no sequence: nothing is enqueued that would write them
            with torch.cuda.stream(self._stream):
                self.slots.fill_(-1), self.positions.zero_(), self.seq_ids.fill_(-1)
        self._out = (self.slots, self.positions, self.seq_ids, self.query_start, self.granted)
        self._keep = (seq_len, new_len, block_table, free_list, free_count, free_count_out)
        self._fn = lib.spec_cache_extend
        self._args = (_ptr(seq_len), _ptr(new_len), int(extra), B, _ptr(block_table), blocks, int(page_size),
                      _ptr(free_list), free_list.numel(), _ptr(free_count), _ptr(free_count_out), n,
                      _ptr(self.slots), _ptr(self.positions), _ptr(self.seq_ids), _ptr(self.query_start),
                      _ptr(self.granted), _ptr(self.page_start), _ptr(self.error_word), self._stream.cuda_stream)

    def __call__(self):
        self._run()
        return self._out


def cache_extend(*args, **kw):
    """One call of CacheExtend."""
    return CacheExtend(*args, **kw)()


class CacheCommit(_Bound):
    """Lengths after a verify step (spec_cache_commit): of its reserved[b]
    new tokens sequence b keeps accepted_len[b] + extra, and the pages behind
    them go back to the free list; finished[b] != 0 gives all its pages back
    and makes its length 0.  Each call returns (seq_len_out, free_count_out),
    by default seq_len and free_count themselves.
    """

    def __init__(self, seq_len: torch.Tensor, reserved: torch.Tensor, accepted_len: torch.Tensor,
                 block_table: torch.Tensor, free_list: torch.Tensor, free_count: torch.Tensor, page_size: int, *,
                 extra: int = 1, finished: torch.Tensor | None = None, seq_len_out: torch.Tensor | None = None,
                 free_count_out: torch.Tensor | None = None, error_word: torch.Tensor | None = None, stream=None):
        if block_table.dim() != 2 or free_list.dim() != 1:
            raise ValueError("block_table must be [B, max_blocks] and free_list [num_pages]")
        B, blocks = block_table.shape
        dev = block_table.device
        _need("block_table", block_table, (B, blocks))
        lib = self._bind(dev, stream)
        for name, t in (("seq_len", seq_len), ("reserved", reserved), ("accepted_len", accepted_len)):
            _need(name, t, (B,), torch.int32, dev)
        _need("free_list", free_list, free_list.shape, torch.int32, dev)
        _need("free_count", free_count, (1,), torch.int32, dev)
        if finished is not None:
            _need("finished", finished, (B,), torch.int32, dev)
        seq_len_out = seq_len if seq_len_out is None else _need("seq_len_out", seq_len_out, (B,), torch.int32, dev)
        free_count_out = free_count if free_count_out is None else _need("free_count_out", free_count_out, (1,),
                                                                         torch.int32, dev)
        self.page_start = self._new((B + 1,), zero=True)
        self.error_word = (self._new((1,), zero=True) if error_word is None
                           else _need("error_word", error_word, (1,), torch.int32, dev))
        self._out = (seq_len_out, free_count_out)
        self._keep = (seq_len, reserved, accepted_len, finished, block_table, free_list, free_count)
        self._fn = lib.spec_cache_commit
        self._args = (_ptr(seq_len), _ptr(reserved), _ptr(accepted_len), int(extra), _ptr(finished), B,
                      _ptr(block_table), blocks, int(page_size), _ptr(free_list), free_list.numel(),
                      _ptr(free_count), _ptr(free_count_out), _ptr(seq_len_out), _ptr(self.page_start),
                      _ptr(self.error_word), self._stream.cuda_stream)

    def __call__(self):
        self._run()
        return self._out


def cache_commit(*args, **kw):
    """One call of CacheCommit."""
    return CacheCommit(*args, **kw)()


class CacheCompact(_Bound):
    """Cache entries of a token tree's accepted path moved behind each other,
    in place (spec_cache_compact): the rows of node path[b, i], written at
    position seq_len[b] + first + path[b, i], go to seq_len[b] + first + i for
    i < accepted_len[b].  `pools` as for BeamReorder with a block table
    [B, max_blocks]; path [B, N] and accepted_len [B] as spec_verify_tree
    gives them."""

    def __init__(self, pools, block_table: torch.Tensor, seq_len: torch.Tensor, path: torch.Tensor,
                 accepted_len: torch.Tensor, *, first: int = 1, error_word: torch.Tensor | None = None, stream=None):
        ptrs, every, shape, row, dev = _pools(pools, 4, "[num_pages, G, page_size, D]")
        if block_table.dim() != 2 or path.dim() != 2:
            raise ValueError("block_table must be [B, max_blocks] and path [B, N]")
        B, blocks = block_table.shape
        N = path.shape[1]
        if min(shape[1:]) < 1:
            raise ValueError("a cache needs heads, positions and row elements")
        lib = self._bind(dev, stream)
        _need("block_table", block_table, (B, blocks), torch.int32, dev)
        _need("seq_len", seq_len, (B,), torch.int32, dev)
        _need("path", path, (B, N), torch.int32, dev)
        _need("accepted_len", accepted_len, (B,), torch.int32, dev)
        self.error_word = (self._new((1,), zero=True) if error_word is None
                           else _need("error_word", error_word, (1,), torch.int32, dev))
        self._keep = (every, block_table, seq_len, path, accepted_len, ptrs)
        self._fn = lib.spec_cache_compact
        self._args = (ptrs, len(every), B, shape[1], shape[2], row, shape[0], _ptr(block_table), blocks,
                      _ptr(seq_len), int(first), _ptr(path), _ptr(accepted_len), N, _ptr(self.error_word),
                      self._stream.cuda_stream)

    def __call__(self) -> None:
        self._run()


def cache_compact(*args, **kw) -> None:
    """One call of CacheCompact."""
    CacheCompact(*args, **kw)()


class PagedCache:
    """The bookkeeping of a paged cache for a batch of B sequences, all on
    the GPU: seq_len [B], block_table [B, max_blocks], free_list [num_pages]
    and free_count [1], reserved [B] (the tokens granted by the last extend)
    and one error_word for every call.  `extender` binds the call before a
    forward pass, `committer` and `compactor` the calls after a verify step,
    in turn: an extend is committed before the next one;
    Verifier and TreeVerifier make the latter themselves when they are given
    the cache."""

    def __init__(self, B: int, max_blocks: int, num_pages: int, page_size: int, device="cuda"):
        dev = torch.device(device)
        self.page_size, self.num_pages = int(page_size), int(num_pages)
        self.seq_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.reserved = torch.zeros(B, dtype=torch.int32, device=dev)
        self.block_table = torch.full((B, max_blocks), -1, dtype=torch.int32, device=dev)
        self.free_list = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=dev)
        self.free_count = torch.full((1,), num_pages, dtype=torch.int32, device=dev)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=dev)

    def extender(self, max_tokens: int, *, new_len: torch.Tensor | None = None, extra: int = 0,
                 stream=None) -> CacheExtend:
        return CacheExtend(self.seq_len, self.block_table, self.free_list, self.free_count, self.page_size,
                           max_tokens, new_len=new_len, extra=extra, granted=self.reserved,
                           error_word=self.error_word, stream=stream)

    def committer(self, accepted_len: torch.Tensor, *, extra: int = 1, finished: torch.Tensor | None = None,
                  stream=None) -> CacheCommit:
        return CacheCommit(self.seq_len, self.reserved, accepted_len, self.block_table, self.free_list,
                           self.free_count, self.page_size, extra=extra, finished=finished,
                           error_word=self.error_word, stream=stream)

    def compactor(self, pools, path: torch.Tensor, accepted_len: torch.Tensor, *, first: int = 1,
                  stream=None) -> CacheCompact:
        return CacheCompact(pools, self.block_table, self.seq_len, path, accepted_len, first=first,
                            error_word=self.error_word, stream=stream)
