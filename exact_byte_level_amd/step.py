"""The operators around the model in a serving step: keys and values written to the slots of a paged cache, the attention of
new tokens over it, and the choice of the next token (C ABI in include/tt_step.h; the meaning of every argument is described
there).

Calls behave as those of ``serve``: the ``*_into`` calls write into the caller's tensors and only enqueue on the current
stream (or ``stream``), so they can be captured into a HIP graph; arguments of a wrong type, shape or device raise ValueError;
nothing is differentiated, and what is written counts as modified.  None of these calls waits for the device.

    slots, positions, rows = table.plan()                     # a BlockTable: one new token for each row in use
    layer = tt.KeyValueCache(table, heads=8, dim=128)         # of one layer
    layer.write(k, v, slots)
    y = layer.attend(q)                                       # [R, query heads, 128]
    tokens = tt.sample_tokens(tt.shape_logits(logits, ...), u, temperature=t, top_p=p)
"""
import ctypes
import math

from . import _check, lib as _base_lib
from . import serve as _serve

_bind = None   # checks tensors and calls the library
_torch = None
_lib = None


def _start():
    """The library's calls of a step and their binding, once."""
    global _bind, _torch, _lib
    bind = _serve._bind or _serve._start()
    L = _base_lib()
    bind.connect_step(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
        "tt_write_cache", "tt_attend_cache", "tt_attend_workspace", "tt_sample_tokens", "tt_sample_workspace")))
    for name, n in (("tt_attend_workspace", 4), ("tt_sample_workspace", 2)):
        getattr(L, name).argtypes = [ctypes.c_int64] * n
        getattr(L, name).restype = ctypes.c_int64
    _torch, _lib = _serve._torch, L
    _bind = bind
    return bind


def _on(stream):
    return _serve._on(stream)


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def _needs(x, name, dims):
    """What a call takes sizes from before the binding has looked at it."""
    if not isinstance(x, _torch.Tensor):
        raise ValueError("%s: a tensor is needed" % name)
    if x.dim() != dims:
        raise ValueError("%s: a %d-d tensor is needed, got a %d-d one" % (name, dims, x.dim()))


def _space(bytes, where, device):
    if bytes < 0:
        _check(bytes, where)
    return _torch.empty(bytes, dtype=_torch.uint8, device=device) if bytes else None


# -------------------------------------------------------------------- cache

def write_cache_into(keys, values, slots, key_cache, value_cache, key_scale=None, value_scale=None, stream=None):
    """Enqueue tt_write_cache: ``keys`` and ``values`` [N, heads, dim] (float32, float16 or bfloat16) go to ``slots``
    (int64 [N], as BlockTable.plan gives them; negative: passed over) of the caches [blocks, block_size, heads, dim]
    (float16, bfloat16 or float8_e4m3fn; any strides with the elements of a head one behind the other), divided by
    ``key_scale`` and ``value_scale`` (float32 [heads])."""
    rc = (_bind or _start()).write_cache(keys, values, slots, key_cache, value_cache, key_scale, value_scale, _handle(stream))
    if rc:
        _check(rc, "tt_write_cache")


def attend_workspace(query, key_cache):
    """A workspace for attend_cache_into with tensors of these shapes, or None where none is needed."""
    if _bind is None:
        _start()
    _needs(query, "query", 3)
    _needs(key_cache, "key_cache", 4)
    return _space(_lib.tt_attend_workspace(query.shape[0], query.shape[1], key_cache.shape[2], key_cache.shape[3]),
                  "tt_attend_workspace", query.device)


def attend_cache_into(query, key_cache, value_cache, table, lengths, out, rows=None, scale=None, window=0, softcap=0.0,
                      key_scale=None, value_scale=None, lse=None, workspace=None, stream=None):
    """Enqueue tt_attend_cache: each ``query`` [N, heads, dim] (float16 or bfloat16) attends to the first ``lengths`` (int32 [N];
    not above 0: none) tokens of its row of ``table`` (int32 [R, width]), row ``rows[i]`` (int32 [N]) or, without them, row
    i; ``out`` is like the query.

    Several queries of a row read its tokens together only where there are more queries than rows of ``table``, 512 at most: a table that is
    cut to the rows in use serves them better.

    ``scale``: of the scores, by default ``1 / sqrt(dim)``; ``window``: above 0, only the last so many tokens are seen;
    ``softcap``: 0, or 1e-6 .. 1e20, by which scores are capped through a tanh; ``key_scale``, ``value_scale``: what write_cache_into divided by; ``lse``
    (float32 [N, heads]): receives the logarithm of each sum of weights.  ``workspace``: from attend_workspace; without it
    one is made."""
    bind = _bind or _start()
    if workspace is None:
        with _on(stream):
            workspace = _workspace_for(query, key_cache)
    rc = bind.attend_cache(query, key_cache, value_cache, table, lengths, out, rows, _scale(query) if scale is None else scale,
                           window, softcap, key_scale, value_scale, lse, workspace, _handle(stream))
    if rc:
        _check(rc, "tt_attend_cache")


def _scale(query):
    shape = getattr(query, "shape", ())
    return 1.0 / math.sqrt(shape[-1]) if len(shape) and shape[-1] else 1.0


def _workspace_for(query, key_cache):
    """As attend_workspace; of what is no query or no cache nothing, so that the call says what is wrong."""
    q, c = getattr(query, "shape", ()), getattr(key_cache, "shape", ())
    if len(q) != 3 or len(c) != 4:
        return None
    n = _lib.tt_attend_workspace(q[0], q[1], c[2], c[3])
    return _space(n, "tt_attend_workspace", query.device) if n > 0 else None


def attend_cache(query, key_cache, value_cache, table, lengths, lse=False, stream=None, **options):
    """The attention's output as a new tensor like ``query``, with ``lse`` a pair of it and the logarithms of the sums; options
    as in attend_cache_into."""
    if _bind is None:
        _start()
    _needs(query, "query", 3)
    with _on(stream):
        out = _torch.empty(query.shape, dtype=query.dtype, device=query.device)
        sums = _torch.empty(query.shape[:2], dtype=_torch.float32, device=query.device) if lse else None
        attend_cache_into(query, key_cache, value_cache, table, lengths, out, lse=sums, stream=stream, **options)
    return (out, sums) if lse else out


class KeyValueCache:
    """The keys and values of one layer, for the blocks of a BlockTable: ``keys`` and ``values`` [blocks, block_size, heads,
    dim], zeros at first, with ``key_scale`` and ``value_scale`` where the type has 8 bits.

        layer.write(k, v, slots)          # slots of table.plan()
        y = layer.attend(q)               # a query for each row of the table
        y = layer.attend(q, positions + 1, rows)   # several new tokens of a row: each sees what stands before it
    """

    def __init__(self, table, heads, dim, dtype=None, key_scale=None, value_scale=None):
        if _bind is None:
            _start()
        self.table = table
        shape = (table.free_blocks.numel(), table.block_size, heads, dim)
        make = dict(dtype=_torch.bfloat16 if dtype is None else dtype, device=table.table.device)
        self.keys, self.values = _torch.zeros(shape, **make), _torch.zeros(shape, **make)
        self.key_scale, self.value_scale = key_scale, value_scale

    def write(self, keys, values, slots, stream=None):
        write_cache_into(keys, values, slots, self.keys, self.values, self.key_scale, self.value_scale, stream)

    def attend_into(self, query, out, lengths=None, rows=None, stream=None, **options):
        attend_cache_into(query, self.keys, self.values, self.table.table, self.table.lengths if lengths is None else lengths, out,
                          rows=rows, key_scale=self.key_scale, value_scale=self.value_scale, stream=stream, **options)

    def attend(self, query, lengths=None, rows=None, lse=False, stream=None, **options):
        return attend_cache(query, self.keys, self.values, self.table.table, self.table.lengths if lengths is None else lengths,
                            lse=lse, rows=rows, key_scale=self.key_scale, value_scale=self.value_scale, stream=stream, **options)


# ------------------------------------------------------------------- sampling

def sample_workspace(logits):
    """A workspace for sample_tokens_into with logits of this shape, or None where none is needed."""
    if _bind is None:
        _start()
    _needs(logits, "logits", 2)
    return _space(_lib.tt_sample_workspace(logits.shape[0], logits.shape[1]), "tt_sample_workspace", logits.device)


def sample_tokens_into(logits, uniform, tokens, temperature=None, top_k=None, top_p=None, min_p=None, logprobs=None,
                       workspace=None, stream=None):
    """Enqueue tt_sample_tokens: ``tokens`` (int32 [R]) receives the token that each row of ``logits`` [R, V] (float32, float16
    or bfloat16) draws by its random number ``uniform`` (float32 [R], from 0 to below 1): -1 where no logit is above -infinity.

    ``temperature`` (float32 [R]; not above 0: the likeliest token), ``top_k`` (int32 [R]; not above 0: not limited), ``top_p`` and
    ``min_p`` (float32 [R]; from 1 on, up to 0: not limited) say which tokens are kept, ``logprobs`` (float32 [R])
    receives the logarithm of the drawn one's share of them.  ``workspace``: from sample_workspace; without it one is made.
    Logits that shape_logits has divided by a temperature need none here."""
    bind = _bind or _start()
    if workspace is None:
        shape = getattr(logits, "shape", ())
        n = _lib.tt_sample_workspace(*shape) if len(shape) == 2 else 0
        if n > 0:
            with _on(stream):
                workspace = _space(n, "tt_sample_workspace", logits.device)
    rc = bind.sample_tokens(logits, uniform, tokens, temperature, top_k, top_p, min_p, logprobs, workspace, _handle(stream))
    if rc:
        _check(rc, "tt_sample_tokens")


def sample_tokens(logits, uniform, logprobs=False, stream=None, **options):
    """The drawn tokens (int32 [R]), with ``logprobs`` a pair of them and the logarithms of their shares; options as in
    sample_tokens_into."""
    if _bind is None:
        _start()
    _needs(logits, "logits", 2)
    with _on(stream):
        tokens = _torch.empty(logits.shape[0], dtype=_torch.int32, device=logits.device)
        shares = _torch.empty(logits.shape[0], dtype=_torch.float32, device=logits.device) if logprobs else None
        sample_tokens_into(logits, uniform, tokens, logprobs=shares, stream=stream, **options)
    return (tokens, shares) if logprobs else tokens
