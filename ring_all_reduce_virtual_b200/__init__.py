"""Ring all-reduce over N virtual ranks on one B200: the Python binding.

Each "virtual rank" is one CUDA tensor (one buffer in the GPU's HBM).  These
functions only marshal tensors, enums and the current stream into the C ABI
of ``librr_virtual.so`` (declared in ``include/rr.h``); every step of every
collective runs in that library's CUDA kernels.  If the library is missing,
the first call raises: there is no fallback.

Sources: [P4] "Collective communication primitives" (ai-infra-handbooks);
[P3] "Training gradient sync and collective communication" (geek-doc.cn);
[P1] "How all-reduce keeps every card identical" (mhpq.cn); [P2] "AllReduce
from principle to tuning" (xxqk.cn).  ``include/rr.h`` states each call's
semantics with its passage.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Sequence

from ._lib import MAX_RANKS, Cost, RingEvent, RRError, Stats, TensorList, check, lib

__all__ = [
    "all_reduce", "all_reduce_wire", "all_reduce_host", "all_reduce_host_noalloc", "ring_step", "ring_schedule", "reduce_scatter", "all_gather", "all_to_all",
    "RankSet", "BucketPlan", "GradSet", "Reducer", "GradList", "grad_norm", "clip_grads",
    "embedding", "embedding_grad", "cost_model", "pick_algo", "set_picker_params", "last_stats",
    "check_timeouts", "RRError",
    "OPS", "ALGOS", "MAX_RANKS",
]

OPS = {"sum": 0, "avg": 1, "max": 2, "min": 3, "prod": 4}
ALGOS = {"auto": 0, "ring": 1, "oneshot": 2, "tree": 3, "tree_oneshot": 4, "two_shot": 5, "double_ring": 6}
ALGO_NAMES = {v: k for k, v in ALGOS.items()}
PHASES = {"reduce_scatter": 0, "all_gather": 1}
_DTYPE_NAMES = {"f32": 0, "bf16": 1, "i32": 2, "f16": 3}


def _dtype_code(dtype) -> int:
    import torch

    codes = {torch.float32: 0, torch.bfloat16: 1, torch.int32: 2, torch.float16: 3}
    if isinstance(dtype, str):
        return _DTYPE_NAMES[dtype]
    if dtype not in codes:
        raise TypeError(f"unsupported dtype {dtype}; use float32, bfloat16, float16 or int32")
    return codes[dtype]


def _ptr_array(tensors: Sequence) -> ctypes.Array:
    arr = (ctypes.c_void_p * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        arr[i] = t.data_ptr()
    return arr


def _ranks(tensors: Sequence, what: str):
    """Check that the rank tensors are CUDA, contiguous and alike."""
    if len(tensors) < 1 or len(tensors) > MAX_RANKS:
        raise ValueError(f"{what}: need 1..{MAX_RANKS} rank tensors, got {len(tensors)}")
    t0 = tensors[0]
    for t in tensors:
        if not t.is_cuda:
            raise ValueError(f"{what}: rank tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError(f"{what}: rank tensors must be contiguous")
        if t.dtype != t0.dtype or t.numel() != t0.numel() or t.device != t0.device:
            raise ValueError(f"{what}: rank tensors must share dtype, size and device")
    return t0.numel(), _dtype_code(t0.dtype), t0.device


class RankSet:
    """The N rank tensors of an all-reduce, checked and marshalled once.

    ``all_reduce``, ``all_reduce_wire`` and ``ring_step`` accept either this
    or a list of tensors.  A list is checked (CUDA, contiguous, same dtype,
    size and device) and its pointers copied into a ctypes array on every
    call, which costs several microseconds for 8 ranks -- as much as the
    kernel of a small message.  A RankSet does that once: it keeps the tensors
    alive and stays valid while they keep their storage (in-place updates are
    fine; ``resize_`` or ``set_`` on a member is not)."""

    def __init__(self, tensors: Sequence):
        self.count, self.dtype, self.device = _ranks(tensors, "RankSet")
        self.nranks = len(tensors)
        self.ptrs = _ptr_array(tensors)
        self.tensors = list(tensors)
        self._rows = None  # what the embedding calls make of it, kept by the first

    def __len__(self) -> int:
        return self.nranks

    def bind(self, op="sum", algo="auto", stream=None):
        """A callable that runs ``all_reduce(self, op, algo, stream)`` with
        every argument converted to its C type once, so each call costs one
        ctypes call: for small messages, repeated from Python, whose per-call
        host cost is otherwise several microseconds of argument handling."""
        f = lib().rr_allreduce
        args = (self.ptrs, ctypes.c_int(self.nranks), ctypes.c_size_t(self.count), ctypes.c_int(self.dtype),
                ctypes.c_int(_op(op)), ctypes.c_int(_algo(algo)), _stream(stream, self.device))

        def call() -> None:
            st = f(*args)
            if st:
                check(st, "all_reduce")
        return call


def _rank_args(tensors, what: str):
    """(pointer array, nranks, count, dtype code, device) of a list or a RankSet."""
    if isinstance(tensors, RankSet):
        return tensors.ptrs, tensors.nranks, tensors.count, tensors.dtype, tensors.device
    count, d, dev = _ranks(tensors, what)
    return _ptr_array(tensors), len(tensors), count, d, dev


_torch_calls = None  # (torch, current stream's handle by device index, current device's index), at first use


def _calls():
    """PyTorch's calls that every norm, clipping and embedding call makes: a
    stream's handle without building a Stream object (2 us) where PyTorch
    offers that, the current device's index without its initialisation check."""
    global _torch_calls
    if _torch_calls is None:
        import torch

        torch.cuda.current_device()  # initialises CUDA, once
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
        _torch_calls = torch, raw, getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _torch_calls


def _stream(stream, device):
    if stream is None:
        return ctypes.c_void_p(_calls()[1](device.index))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _op(op) -> int:
    return OPS[op] if isinstance(op, str) else int(op)


def _algo(algo) -> int:
    return ALGOS[algo] if isinstance(algo, str) else int(algo)


def all_reduce(tensors, op="sum", algo="auto", stream=None) -> None:
    """In-place all-reduce over the rank tensors, a list or a ``RankSet``
    (``rr_allreduce``)."""
    ptrs, n, count, d, dev = _rank_args(tensors, "all_reduce")
    check(lib().rr_allreduce(ptrs, n, count, d, _op(op), _algo(algo), _stream(stream, dev)), "all_reduce")


def all_reduce_wire(tensors, op="sum", wire="bf16", algo="auto", stream=None) -> None:
    """In-place all-reduce of fp32 rank tensors whose transfers are rounded
    to the bf16 wire format while the folds stay fp32 (``rr_allreduce_wire``)."""
    ptrs, n, count, d, dev = _rank_args(tensors, "all_reduce_wire")
    if d != _DTYPE_NAMES["f32"]:
        raise TypeError("all_reduce_wire: the rank tensors must be float32 (the wire format is bf16)")
    check(lib().rr_allreduce_wire(ptrs, n, count, _op(op), _dtype_code(wire), _algo(algo), _stream(stream, dev)),
          "all_reduce_wire")


def all_reduce_host(host: Sequence, device: Sequence, op="sum", algo="auto", stream=None) -> None:
    """All-reduce of host tensors through device staging tensors
    (``rr_allreduce_host``): copy in, reduce, copy back, all enqueued on
    ``stream``.  ``host`` should be pinned; it holds the result once the
    stream is synchronised."""
    count, d, dev = _ranks(device, "all_reduce_host")
    if len(host) != len(device):
        raise ValueError("all_reduce_host: one host tensor per device tensor")
    for h in host:
        if h.is_cuda or not h.is_contiguous() or h.numel() != count or _dtype_code(h.dtype) != d:
            raise ValueError("all_reduce_host: host tensors must be contiguous CPU tensors like the device ones")
    check(lib().rr_allreduce_host(_ptr_array(host), _ptr_array(device), len(device), count, d, _op(op),
                                  _algo(algo), _stream(stream, dev)), "all_reduce_host")


def all_reduce_host_noalloc(host: Sequence, op="sum", algo="auto", stream=None) -> None:
    """All-reduce of host tensors for callers that cannot allocate device
    memory (``rr_allreduce_host_noalloc``): the values are staged in the
    library's static device region (``RR_NOALLOC_MAX_BYTES`` in all), so the
    call allocates nothing.  ``host`` should be pinned; it holds the result
    once the stream is synchronised."""
    import torch

    if len(host) < 1 or len(host) > MAX_RANKS:
        raise ValueError(f"all_reduce_host_noalloc: need 1..{MAX_RANKS} host tensors")
    h0 = host[0]
    for h in host:
        if h.is_cuda or not h.is_contiguous() or h.numel() != h0.numel() or h.dtype != h0.dtype:
            raise ValueError("all_reduce_host_noalloc: host tensors must be contiguous CPU tensors alike")
    dev = torch.device("cuda", torch.cuda.current_device())
    check(lib().rr_allreduce_host_noalloc(_ptr_array(host), len(host), h0.numel(), _dtype_code(h0.dtype), _op(op),
                                          _algo(algo), _stream(stream, dev)), "all_reduce_host_noalloc")


def ring_step(tensors, op, phase, step: int, stream=None) -> None:
    """One ring step for all ranks at once (``rr_ring_step``)."""
    ptrs, n, count, d, dev = _rank_args(tensors, "ring_step")
    ph = PHASES[phase] if isinstance(phase, str) else int(phase)
    check(lib().rr_ring_step(ptrs, n, count, d, _op(op), ph, step, _stream(stream, dev)), "ring_step")


def ring_schedule(nranks: int, count: int, dtype="f32") -> list[dict]:
    """The ring schedule as a list of transfers (``rr_ring_schedule``)."""
    total = 2 * max(nranks - 1, 0) * nranks
    ev = (RingEvent * max(total, 1))()
    got = ctypes.c_size_t(0)
    check(lib().rr_ring_schedule(nranks, count, _dtype_code(dtype), ev, total, ctypes.byref(got)),
          "ring_schedule")
    return [{k: int(getattr(ev[i], k)) for k, _ in RingEvent._fields_} for i in range(got.value)]


def reduce_scatter(send: Sequence, recv: Sequence, op="sum", algo="auto", stream=None) -> None:
    """``recv[r]`` = part r of the reduction of all ``send`` (``rr_reduce_scatter``)."""
    count, d, dev = _ranks(send, "reduce_scatter")
    rcount, rd, rdev = _ranks(recv, "reduce_scatter")
    if len(recv) != len(send) or rd != d or rdev != dev or rcount * len(send) != count:
        raise ValueError("reduce_scatter: recv must be N tensors of count/N elements of the same dtype and device")
    check(lib().rr_reduce_scatter(_ptr_array(send), _ptr_array(recv), len(send), rcount, d, _op(op),
                                  _algo(algo), _stream(stream, dev)), "reduce_scatter")


def all_gather(send: Sequence, recv: Sequence, algo="auto", stream=None) -> None:
    """``recv[r]`` = concatenation of all ``send`` parts (``rr_all_gather``)."""
    scount, d, dev = _ranks(send, "all_gather")
    rcount, rd, rdev = _ranks(recv, "all_gather")
    if len(recv) != len(send) or rd != d or rdev != dev or rcount != scount * len(send):
        raise ValueError("all_gather: recv must be N tensors of N*count elements of the same dtype and device")
    check(lib().rr_all_gather(_ptr_array(send), _ptr_array(recv), len(send), scount, d, _algo(algo),
                              _stream(stream, dev)), "all_gather")


def all_to_all(send: Sequence, recv: Sequence, stream=None) -> None:
    """Block transpose across ranks (``rr_all_to_all``)."""
    count, d, dev = _ranks(send, "all_to_all")
    rcount, rd, rdev = _ranks(recv, "all_to_all")
    n = len(send)
    if len(recv) != n or rd != d or rdev != dev or rcount != count or count % n:
        raise ValueError("all_to_all: recv must match send (size, dtype, device), and N must divide the count")
    check(lib().rr_all_to_all(_ptr_array(send), _ptr_array(recv), n, count // n, d, _stream(stream, dev)),
          "all_to_all")


class GradSet:
    """The gradient tensors of all ranks (``grads[r][t]``), checked and with
    their device pointers marshalled once.  Bucket calls accept either this or
    the nested lists; a DDP step reuses the same gradient buffers every step,
    so building the pointer array once keeps the per-bucket host cost to a
    few microseconds.  Every rank must hold the same tensor sizes, all
    contiguous CUDA tensors of one dtype on one device."""

    def __init__(self, grads: Sequence[Sequence]):
        import weakref

        if not grads or not grads[0]:
            raise ValueError("GradSet: no gradients")
        first = grads[0][0]
        numels = [int(g.numel()) for g in grads[0]]
        for rank in grads:
            if len(rank) != len(numels):
                raise ValueError("GradSet: every rank needs the same number of tensors")
            for t, g in enumerate(rank):
                if not g.is_cuda or not g.is_contiguous() or g.device != first.device or g.dtype != first.dtype:
                    raise ValueError("GradSet: gradients must be contiguous CUDA tensors of one dtype and device")
                if g.numel() != numels[t]:
                    raise ValueError(f"GradSet: tensor {t} has different sizes on different ranks")
        self.nranks = len(grads)
        self.numels = numels
        self.dtype = _dtype_code(first.dtype)
        self.device = first.device
        self.ptrs = _ptr_array([g for rank in grads for g in rank])
        self._keep = [list(rank) for rank in grads]  # the tensors must outlive the pointers
        self._plans = weakref.WeakSet()  # plans this set was checked against
        self._list = None  # this set as a GradList, made when a norm or a clipping first asks for it

    @classmethod
    def _of(cls, grads) -> "GradSet":
        """``grads`` as a GradSet; a GradList's is made once and kept with it."""
        if not isinstance(grads, GradList):
            return cls([grads] if len(grads) and hasattr(grads[0], "data_ptr") else grads)
        if grads._set is None:
            grads._set = cls(grads._keep)
        return grads._set


class GradList:
    """The gradient tensors whose global norm is taken and that are clipped,
    checked and with their device pointers marshalled once: a list of tensors
    (one rank), or one list per rank (``grads[r][t]``) whose ranks hold the
    same sizes and types.  Unlike a ``GradSet`` a list may mix float32,
    bfloat16 and float16 tensors.  ``grad_norm``, ``clip_grads`` and
    ``BucketPlan.all_reduce_clip`` (for its gradients, which are of one type,
    and for ``synced``) accept this, a ``GradSet`` or the lists; it keeps the
    tensors alive and stays valid while they keep their storage."""

    def __init__(self, grads):
        grads = list(grads)
        if grads and hasattr(grads[0], "data_ptr"):
            grads = [grads]
        ranks = [list(rank) for rank in grads] or [[]]
        if len(ranks) > MAX_RANKS:
            raise ValueError(f"GradList: need 1..{MAX_RANKS} ranks, got {len(ranks)}")
        flat = [g for rank in ranks for g in rank]
        for rank in ranks:
            if len(rank) != len(ranks[0]):
                raise ValueError("GradList: every rank needs the same number of tensors")
            for g, g0 in zip(rank, ranks[0]):
                if not g.is_cuda or not g.is_contiguous() or g.device != flat[0].device:
                    raise ValueError("GradList: gradients must be contiguous CUDA tensors on one device")
                if g.numel() != g0.numel() or g.dtype != g0.dtype:
                    raise ValueError("GradList: a tensor has different sizes or dtypes on different ranks")
        codes = [_dtype_code(g.dtype) for g in ranks[0]]
        if _DTYPE_NAMES["i32"] in codes:
            raise TypeError("GradList: gradients must be float32, bfloat16 or float16")
        self._marshal(_ptr_array(flat), [int(g.numel()) for g in ranks[0]], codes, len(ranks))
        self.device = flat[0].device if flat else None
        self._keep = ranks  # the tensors must outlive the pointers
        self._set = None  # this list as a GradSet, made when a bucket call first asks for it

    def _marshal(self, ptrs, numels, codes, nranks):
        n = len(numels)
        self.nranks = nranks
        self._arrays = (ptrs, (ctypes.c_size_t * max(n, 1))(*numels), (ctypes.c_int * max(n, 1))(*codes))
        self._c = TensorList(*[ctypes.cast(a, t) for a, (_, t) in zip(self._arrays, TensorList._fields_)], n, nranks)
        self._ref = ctypes.byref(self._c)
        self._scratch_bytes = None

    @classmethod
    def _of(cls, grads) -> "GradList":
        """``grads`` as a GradList; a GradSet's is made once and kept with it."""
        if isinstance(grads, GradList):
            return grads
        if not isinstance(grads, GradSet):
            return cls(grads)
        if grads._list is None:
            one = cls.__new__(cls)
            one._marshal(grads.ptrs, grads.numels, [grads.dtype] * len(grads.numels), grads.nranks)
            one.device = grads.device
            one._keep, one._set = grads._keep, None
            grads._list = one
        return grads._list

    def _workspace(self) -> int:
        """Bytes of device workspace that a call on this list needs."""
        if self._scratch_bytes is None:
            b = ctypes.c_size_t()
            check(lib().rr_clip_workspace(None, 0, 0, 0, self._ref, ctypes.byref(b)), "clip_workspace")
            self._scratch_bytes = b.value
        return self._scratch_bytes


@contextlib.contextmanager
def _placed(stream, device):
    """Run with ``device`` current (kernels are launched from there) and the
    caching allocator serving ``stream``: scratch memory of a call is taken
    there, so that its next user on that stream is ordered behind the call.
    A stream of another device is refused: making it current would leave it."""
    import torch

    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device)
            with torch.cuda.stream(stream):
                yield


def _with_norm(what: str, fn, args: tuple, device, need: int, out, stream):
    """Run ``fn(*args, norm pointer, workspace pointer, bytes, stream)``; the norm's tensor."""
    torch, raw, current = _calls()
    index = device.index
    if stream is not None or index != current():
        with _placed(stream, device):
            return _with_norm(what, fn, args, device, need, out, None)
    if out is None:  # memory of its own: a norm that is kept, in a log say, does not keep the workspace
        out = torch.empty_strided((), (), dtype=torch.float32, device=device)  # 0.9 us less than empty(())
    elif not out.is_cuda or out.dtype != torch.float32 or out.numel() != 1 or out.device != device:
        raise ValueError("out must be one float32 element on the gradients' device")
    mem = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=device)
    st = fn(*args, out.data_ptr(), mem.data_ptr(), need, raw(index))
    if st:
        check(st, what)
    return out


def _norm_call(what: str, fn, args: tuple, gl: GradList, out, stream):
    """``_with_norm`` for a list."""
    device = gl.device
    if device is None:
        torch = _calls()[0]
        device = out.device if out is not None else torch.device("cuda", torch.cuda.current_device())
    return _with_norm(what, fn, args, device, gl._workspace(), out, stream)


def grad_norm(grads, out=None, stream=None):
    """The global 2-norm of rank 0's gradients (``rr_grad_norm``): a float32
    scalar on the device, ``out`` where it is given.  ``grads``: a list of
    tensors, one list per rank, a ``GradList`` or a ``GradSet``."""
    gl = GradList._of(grads)
    return _norm_call("grad_norm", lib().rr_grad_norm, (gl._ref,), gl, out, stream)


def clip_grads(grads, max_norm: float, eps: float = 1e-6, out=None, stream=None):
    """Scale gradients so that their global norm is at most ``max_norm``
    (``rr_clip_grads``): in place for one rank; for several, rank 0's
    gradients, scaled, go to every rank.  Returns the norm before clipping as
    a float32 scalar on the device (``out`` where it is given); nothing waits
    for the GPU."""
    gl = GradList._of(grads)
    return _norm_call("clip_grads", lib().rr_clip_grads, (gl._ref, float(max_norm), float(eps)), gl, out, stream)


def _id_set(tokens, what: str):
    """(pointer array, id type, ranks, tokens per rank, device) of the ranks'
    token ids: a list of int32 or int64 tensors, or a RankSet (int32)."""
    if isinstance(tokens, RankSet):
        if tokens.dtype != 2:
            raise TypeError(f"{what}: token ids must be int32 or int64")
        return tokens.ptrs, 0, tokens.nranks, tokens.count, tokens.device
    n = len(tokens)
    if n < 1 or n > MAX_RANKS:
        raise ValueError(f"{what}: need 1..{MAX_RANKS} token tensors, got {n}")
    t0 = tokens[0]
    dtype, count, device = t0.dtype, t0.numel(), t0.device
    id_type = _ID_TYPES.get(str(dtype))
    if id_type is None:
        raise TypeError(f"{what}: token ids must be int32 or int64")
    for t in tokens:
        if not t.is_cuda or not t.is_contiguous() or t.dtype != dtype or t.numel() != count or t.device != device:
            raise ValueError(f"{what}: token tensors must be contiguous CUDA tensors alike")
    return _ptr_array(tokens), id_type, n, count, device


_ID_TYPES = {"torch.int32": 0, "torch.int64": 1}


def _row_set(tensors, what: str):
    """(pointer array, ranks, rows, row width, dtype code, device) of 2-D (or
    more) tensors whose last axis is a row: a list, or a RankSet (which keeps
    the answer)."""
    is_set = isinstance(tensors, RankSet)
    if is_set and tensors._rows is not None:
        return tensors._rows
    ptrs, n, count, d, dev = _rank_args(tensors, what)
    width = 0
    for t in tensors.tensors if is_set else tensors:
        shape = t.shape
        if len(shape) < 2 or shape[-1] == 0 or shape[-1] != (width or shape[-1]):
            raise ValueError(f"{what}: need tensors of rows (two axes or more, rows not empty, of one width on every rank)")
        width = shape[-1]
    rows = ptrs, n, count // width, width, d, dev
    if is_set:
        tensors._rows = rows
    return rows


def embedding(tokens, tables, outs, scale: float = 1.0, stream=None) -> None:
    """``outs[r][t] = scale * tables[r][tokens[r][t]]`` for every rank in one
    launch (``rr_embedding``).  Lists of one tensor per rank, or RankSets;
    ids int32 or int64, rows float32, bfloat16 or float16.  An id outside the
    table gives a row of zeros."""
    ids, id_type, n, T, dev = _id_set(tokens, "embedding")
    w, wn, V, D, d, wdev = _row_set(tables, "embedding")
    o, on, rows, od, odt, odev = _row_set(outs, "embedding")
    if wn != n or on != n or rows != T or od != D or odt != d or wdev != dev or odev != dev:
        raise ValueError("embedding: need one table [V, D] and one output [tokens, D] per rank, alike and on the "
                         "tokens' device")
    args = (ids, id_type, w, o, n, T, V, D, d, float(scale))
    _, raw, current = _calls()
    if stream is None and dev.index == current():
        st = lib().rr_embedding(*args, raw(dev.index))
        if st:
            check(st, "embedding")
        return
    with _placed(stream, dev):
        check(lib().rr_embedding(*args, raw(dev.index)), "embedding")


_embed_bytes: dict = {}  # workspace bytes of embedding_grad by (ranks, tokens, rows, width)


def embedding_grad(tokens, grad_out, grads, op="avg", scale: float = 1.0, accumulate: bool = False,
                   padding_idx: int | None = None, stream=None) -> None:
    """The gradient of the embedding table over the tokens of all ranks
    (``rr_embedding_grad``): ``grads[o][v] = f * sum of grad_out[r][t] over
    tokens[r][t] == v`` with ``f = scale`` (``op="sum"``) or ``scale / ranks``
    (``"avg"``), into every tensor of ``grads`` (each rank's replica, or one);
    with ``accumulate`` added to what is there.  ``grads`` may be float32
    beside 16-bit rows.  Ids outside the table and ``padding_idx`` add nothing."""
    ids, id_type, n, T, dev = _id_set(tokens, "embedding_grad")
    g, gn, rows, D, d, gdev = _row_set(grad_out, "embedding_grad")
    w, wn, V, wd, wdt, wdev = _row_set(grads, "embedding_grad")
    if gn != n or rows != T or wd != D or gdev != dev or wdev != dev:
        raise ValueError("embedding_grad: need one output gradient [tokens, D] per rank and table gradients [V, D], on "
                         "the tokens' device")
    key = (n, T, V, D)
    need = _embed_bytes.get(key)
    if need is None:
        b = ctypes.c_size_t()
        check(lib().rr_embedding_grad_workspace(n, T, V, D, ctypes.byref(b)), "embedding_grad_workspace")
        if len(_embed_bytes) >= 4096:  # token counts that change from call to call
            _embed_bytes.clear()
        need = _embed_bytes[key] = max(b.value, 256)

    args = (ids, id_type, g, n, T, V, D, d, _op(op), float(scale), -1 if padding_idx is None else int(padding_idx), w, wn,
            wdt, 1 if accumulate else 0)
    torch, raw, current = _calls()
    with contextlib.nullcontext() if stream is None and dev.index == current() else _placed(stream, dev):
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        check(lib().rr_embedding_grad(*args, ws.data_ptr(), need, raw(dev.index)), "embedding_grad")


class BucketPlan:
    """DDP-style bucket plan over a list of gradient sizes (``rr_bucket_plan``)."""

    def __init__(self, numels: Sequence[int], grad_dtype="bf16", cap_bytes: int = 25 * (1 << 20)):
        arr = (ctypes.c_size_t * max(len(numels), 1))(*[int(m) for m in numels])
        handle = ctypes.c_void_p()
        check(lib().rr_bucket_plan(arr, len(numels), _dtype_code(grad_dtype), int(cap_bytes),
                                   ctypes.byref(handle)), "bucket_plan")
        self._h = handle
        self._free = lib().rr_bucket_plan_free  # held: module globals may be gone when __del__ runs at exit
        self.numels = [int(m) for m in numels]
        self.grad_dtype = _dtype_code(grad_dtype)
        self._clip_bytes = {}  # workspace bytes of all_reduce_clip by bucket range, ranks and synced list

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._free(h)
            self._h = None

    @property
    def num_buckets(self) -> int:
        return int(lib().rr_bucket_count(self._h))

    def info(self, bucket: int) -> tuple[int, int, int]:
        """(first tensor, number of tensors, fp32 elements) of a bucket."""
        f, c, m = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
        check(lib().rr_bucket_info(self._h, bucket, ctypes.byref(f), ctypes.byref(c), ctypes.byref(m)),
              "bucket_info")
        return f.value, c.value, m.value

    def tensor(self, t: int) -> tuple[int, int]:
        """(bucket, element offset in it) of a tensor."""
        b, o = ctypes.c_int(), ctypes.c_size_t()
        check(lib().rr_bucket_tensor(self._h, t, ctypes.byref(b), ctypes.byref(o)), "bucket_tensor")
        return b.value, o.value

    def _grads(self, grads):
        """(pointers, nranks, device) of gradients that match this plan's
        tensor sizes and dtype (checked once per GradSet and plan)."""
        gs = grads if isinstance(grads, GradSet) else GradSet._of(grads)
        if self not in gs._plans:
            if gs.numels != self.numels or gs.dtype != self.grad_dtype:
                raise ValueError("gradients do not match the bucket plan (tensor count, sizes or dtype)")
            gs._plans.add(self)
        return gs.ptrs, gs.nranks, gs.device

    def _buckets(self, bucket: int, buckets: Sequence, n: int, device):
        """Pointer array of the fp32 bucket buffers, checked against the bucket's size."""
        numel = self.info(bucket)[2]
        if len(buckets) != n:
            raise ValueError("one fp32 bucket buffer per rank")
        for t in buckets:
            if (not t.is_cuda or not t.is_contiguous() or t.device != device or _dtype_code(t.dtype) != 0
                    or t.numel() < numel):
                raise ValueError(f"bucket buffers must be contiguous fp32 CUDA tensors of at least {numel} elements")
        return _ptr_array(buckets)

    def flat_buffers(self, nranks: int, device=None, dtype=None):
        """Gradients laid out as views into one flat buffer per bucket and
        rank (DDP's ``gradient_as_bucket_view``): returns ``(flats, grads)``
        with ``flats[b][r]`` the bucket's buffer on rank r and ``grads[r][t]``
        a view of tensor t inside it.  A bucket sync on this layout is
        ``all_reduce(flats[b], op, "oneshot")``, with the same bits as
        ``all_reduce(b, grads, op)`` and no gather or scatter at all.  (The
        buffers are allocated by PyTorch here, not by the library.)"""
        import torch

        dtype = dtype or torch.bfloat16
        flats, grads = [], [[None] * len(self.numels) for _ in range(nranks)]
        for b in range(self.num_buckets):
            first, cnt, numel = self.info(b)
            row = [torch.zeros(numel, dtype=dtype, device=device) for _ in range(nranks)]
            flats.append(row)
            for t in range(first, first + cnt):
                off = self.tensor(t)[1]
                for r in range(nranks):
                    grads[r][t] = row[r][off:off + self.numels[t]]
        return flats, grads

    def pack(self, bucket: int, grads: Sequence[Sequence], buckets: Sequence, stream=None) -> None:
        """``grads[r][t]`` -> fp32 ``buckets[r]`` for the bucket's tensors."""
        g, n, dev = self._grads(grads)
        check(lib().rr_bucket_pack(self._h, bucket, g, self._buckets(bucket, buckets, n, dev), n,
                                   _stream(stream, dev)), "bucket_pack")

    def unpack(self, bucket: int, buckets: Sequence, grads: Sequence[Sequence], op="avg", stream=None) -> None:
        """fp32 ``buckets[r]`` -> ``grads[r][t]`` (AVG divides by N)."""
        g, n, dev = self._grads(grads)
        check(lib().rr_bucket_unpack(self._h, bucket, self._buckets(bucket, buckets, n, dev), g, n, _op(op),
                                     _stream(stream, dev)), "bucket_unpack")

    def all_reduce(self, bucket: int, grads: Sequence[Sequence], op="avg", stream=None) -> None:
        """Fused pack + ring-order all-reduce + unpack, in place on ``grads``."""
        g, n, dev = self._grads(grads)
        check(lib().rr_bucket_allreduce(self._h, bucket, g, n, _op(op), _stream(stream, dev)),
              "bucket_allreduce")

    def all_reduce_range(self, first: int, count: int, grads: Sequence[Sequence], op="avg", stream=None) -> None:
        """Fused sync of buckets ``first .. first + count - 1`` in a few shared
        launches, with the bits of ``all_reduce`` on each of them
        (``rr_bucket_allreduce_range``)."""
        g, n, dev = self._grads(grads)
        check(lib().rr_bucket_allreduce_range(self._h, first, count, g, n, _op(op), _stream(stream, dev)),
              "bucket_allreduce_range")


    def all_reduce_clip(self, grads, max_norm: float, op="avg", first: int = 0, count: int | None = None, synced=None,
                        eps: float = 1e-6, out=None, stream=None):
        """Fused sync of buckets ``first .. first + count - 1`` (default: all)
        and clipping by the global norm of the result
        (``rr_bucket_allreduce_clip``): the average (``op``) is formed in
        fp32, scaled there and then rounded.  ``synced`` adds gradients that are
        already alike on every rank (rank 0's count: a ``GradList`` or one list
        per rank; ``[]`` is none) to the norm and to the clipping.  Returns the norm before
        clipping as a float32 scalar on the device (``out`` where it is given)."""
        g, n, dev = self._grads(grads)
        rest = GradList._of(synced) if synced is not None else None
        if rest is not None and rest.device not in (None, dev):
            raise ValueError("the synced gradients must be on the gradients' device")
        count = self.num_buckets - first if count is None else count
        ref = rest._ref if rest is not None else None
        key = (first, count, n, rest._workspace() if rest is not None else 0)
        need = self._clip_bytes.get(key)
        if need is None:
            b = ctypes.c_size_t()
            check(lib().rr_clip_workspace(self._h, first, count, n, ref, ctypes.byref(b)), "clip_workspace")
            need = self._clip_bytes[key] = b.value
        args = (self._h, first, count, g, n, _op(op), ref, float(max_norm), float(eps))
        return _with_norm("bucket_allreduce_clip", lib().rr_bucket_allreduce_clip, args, dev, need, out, stream)


class Reducer:
    """DDP-style overlapped bucket sync (``rr_reducer_*``): mark each
    gradient ready on the stream that produced it; every bucket's fused sync
    starts on ``comm`` as soon as its last gradient is ready; ``finish``
    joins the step.  Keep ``plan`` and the gradients alive while in use."""

    def __init__(self, plan: BucketPlan, grads, op="avg", comm=None, max_ctas: int = 0):
        import torch

        g = grads if isinstance(grads, GradSet) else GradSet(grads)
        plan._grads(g)  # the gradients must match the plan
        # a high-priority stream lets bucket syncs start as soon as SMs free up
        self.comm = comm if comm is not None else torch.cuda.Stream(g.device, priority=-1)
        self._plan, self._grads = plan, g
        handle = ctypes.c_void_p()
        check(lib().rr_reducer_create(plan._h, g.ptrs, g.nranks, _op(op), _stream(self.comm, g.device),
                                      int(max_ctas), ctypes.byref(handle)), "reducer_create")
        self._h = handle
        self._free = lib().rr_reducer_free  # held: module globals may be gone when __del__ runs at exit
        self._device = g.device

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._free(h)
            self._h = None

    def ready(self, tensor: int, stream=None) -> None:
        check(lib().rr_reducer_ready(self._h, tensor, _stream(stream, self._device)), "reducer_ready")

    def finish(self, stream=None, max_norm: float | None = None, eps: float = 1e-6):
        """Join the step on ``stream``; with ``max_norm``, then clip the synced
        gradients there (``clip_grads``) and return their norm."""
        check(lib().rr_reducer_finish(self._h, _stream(stream, self._device)), "reducer_finish")
        if max_norm is not None:
            return clip_grads(self._grads, max_norm, eps, stream=stream)
        return None


def cost_model(algo, nranks: int, bytes_per_rank: float, alpha_s: float, beta_bytes_per_s: float) -> dict:
    """The alpha-beta model terms (``rr_cost_model``)."""
    c = Cost()
    check(lib().rr_cost_model(_algo(algo), nranks, float(bytes_per_rank), float(alpha_s),
                              float(beta_bytes_per_s), ctypes.byref(c)), "cost_model")
    return {k: float(getattr(c, k)) for k, _ in Cost._fields_}


def pick_algo(nranks: int, count: int, dtype="f32") -> str:
    """The algorithm AUTO runs for this shape (``rr_pick_algo``)."""
    return ALGO_NAMES[int(lib().rr_pick_algo(nranks, count, _dtype_code(dtype)))]


def set_picker_params(launch_s: float, hbm_bytes_per_s: float) -> None:
    check(lib().rr_set_picker_params(float(launch_s), float(hbm_bytes_per_s)), "set_picker_params")


def last_stats() -> dict:
    """What the last call on this thread did (``rr_get_stats``)."""
    s = Stats()
    check(lib().rr_get_stats(ctypes.byref(s)), "get_stats")
    out = {k: int(getattr(s, k)) for k, _ in Stats._fields_}
    out["algo"] = ALGO_NAMES.get(out["algo"], out["algo"])
    return out


def check_timeouts() -> None:
    """Synchronise the device and raise ``RRError`` (status RR_ERR_TIMEOUT)
    if any bounded device wait ran out since the last check
    (``rr_check_timeouts``)."""
    check(lib().rr_check_timeouts(), "check_timeouts")
