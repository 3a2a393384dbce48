"""What a serving step needs next to the tokenizer: block tables of a paged
cache, token sets, grammar masks and the shaping of logits (C ABI in
include/tt_serve.h; the meaning of every argument is described there).

The ``*_into`` calls write into the caller's tensors and only enqueue on the
current stream (or ``stream``), so they can be captured into a HIP graph; the
others make their results and, where the device may report a data error, wait
for it.  Arguments of a wrong type, shape or device raise ValueError.

    ids, offsets = tt.encode_batch(prompts, starts)           # offsets: int64 [B + 1]
    cache = tt.BlockTable(rows=B, width=256, blocks=4096, block_size=16)
    slots, positions, rows = cache.plan(offsets.cuda())
    seen = tt.token_bits(ids, vocab, offsets=offsets.cuda())
    out = tt.shape_logits(logits, seen=seen, repetition=rho, temperature=t)
"""
import contextlib
import ctypes
import struct

import numpy as np

from . import TTError, TT_OK, _check, _stream, lib as _base_lib

F32, F16, BF16 = 0, 1, 2
STATE_DEAD, STATE_FREE = -1, -2

_PLAN = struct.Struct("=17q")
_GRAMMAR = struct.Struct("=10q")
_SHAPE = struct.Struct("=26q")

_lib = None
_types = None  # torch element type -> code
_torch = None


def _start():
    """The library with the argument types of the serving calls, set once."""
    global _lib, _types, _torch
    import torch
    L = _base_lib()
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.tt_plan_blocks.argtypes = [vp, vp]
    L.tt_release_blocks.argtypes = [vp, vp, i64, i64, vp, i64, i64, vp, i64, vp, vp, vp, vp, vp]
    L.tt_token_bits.argtypes = [vp, i64, vp, i64, i64, vp, i64, i32, vp]
    L.tt_grammar_bits.argtypes = [vp, vp, i64, vp, i64, i64, vp]
    L.tt_grammar_advance.argtypes = [vp, vp, vp, i64, vp, vp]
    L.tt_shape_logits.argtypes = [vp, vp]
    L.tt_vocab_size.argtypes = [vp, vp]
    L.tt_vocab_strings.argtypes = [vp, vp]
    for f in ("tt_plan_blocks", "tt_release_blocks", "tt_token_bits", "tt_grammar_bits", "tt_grammar_advance",
              "tt_shape_logits", "tt_vocab_size", "tt_vocab_strings"):
        getattr(L, f).restype = ctypes.c_int
    _types = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    _torch = torch
    _lib = L
    return L


def _device(t, name):
    """Index of the tensor's device, which has to be the current one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s is not on a GPU" % name)
    if dev != _torch.cuda.current_device():
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, dev, _torch.cuda.current_device()))
    return dev


def _vec(t, name, dtype, dev, size=None):
    """Address of a 1-d tensor without gaps."""
    if t.dtype is not dtype or t.dim() != 1 or t.get_device() != dev:
        raise ValueError("%s: a 1-d %s tensor on cuda:%d is needed, got %s %s on %s"
                         % (name, dtype, dev, tuple(t.shape), t.dtype, t.device))
    n = t.numel()
    if size is not None and n != size:
        raise ValueError("%s has %d entries, not %d" % (name, n, size))
    if n > 1 and t.stride(0) != 1:
        raise ValueError("%s has gaps between its entries" % name)
    return t.data_ptr()


def _mat(t, name, dtype, dev, rows=None, least=0):
    """Address and row stride of a 2-d tensor whose rows are without gaps."""
    if t.dtype is not dtype or t.dim() != 2 or t.get_device() != dev:
        raise ValueError("%s: a 2-d %s tensor on cuda:%d is needed, got %s %s on %s"
                         % (name, dtype, dev, tuple(t.shape), t.dtype, t.device))
    n, m = t.shape
    if rows is not None and n != rows:
        raise ValueError("%s has %d rows, not %d" % (name, n, rows))
    if m < least:
        raise ValueError("%s has rows of %d entries, %d are needed" % (name, m, least))
    if m > 1 and n and t.stride(1) != 1:
        raise ValueError("%s has gaps within its rows" % name)
    return t.data_ptr(), t.stride(0)


def _on(stream):
    """What is allocated inside belongs to the stream it is used on."""
    return contextlib.nullcontext() if stream is None else _torch.cuda.stream(stream)


def _words(vocab):
    return (vocab + 31) // 32


def _raise_count(out_n, where):
    n = int(out_n.item())
    if n < 0:
        raise TTError(n, where)
    return n


# ------------------------------------------------------------- block tables

def plan_blocks_into(lengths, table, free_blocks, n_free, block_size, slots, out_n, offsets=None, positions=None,
                     rows=None, out_lengths=None, out_n_free=None, stream=None):
    """Enqueue tt_plan_blocks: blocks for the new tokens of every row of ``table`` (int32 [R, width]), and the
    slot, position and row of each token.

    ``offsets`` (int64 [R + 1], as encode_batch gives them) says how many new tokens each row has; without
    it every row in use (length >= 0) gets one.  ``slots`` (int64), ``positions`` and ``rows`` (int32) have one
    entry per place; places without a token receive -1.  ``lengths`` and ``n_free`` are brought up to date in
    place unless ``out_lengths`` / ``out_n_free`` are given.  ``out_n`` (int64 [1]) receives the number of
    tokens or an error code, and then nothing else has changed.
    """
    L = _lib or _start()
    dev = _device(lengths, "lengths")
    i32, i64 = _torch.int32, _torch.int64
    n, places = lengths.numel(), slots.numel()
    t, ts = _mat(table, "table", i32, dev, n)
    args = _PLAN.pack(
        _vec(lengths, "lengths", i32, dev), 0 if offsets is None else _vec(offsets, "offsets", i64, dev, n + 1),
        n, places, int(block_size), t, ts, table.shape[1], _vec(free_blocks, "free_blocks", i32, dev),
        free_blocks.numel(), _vec(n_free, "n_free", i32, dev, 1), _vec(slots, "slots", i64, dev),
        0 if positions is None else _vec(positions, "positions", i32, dev, places),
        0 if rows is None else _vec(rows, "rows", i32, dev, places),
        lengths.data_ptr() if out_lengths is None else _vec(out_lengths, "out_lengths", i32, dev, n),
        n_free.data_ptr() if out_n_free is None else _vec(out_n_free, "out_n_free", i32, dev, 1),
        _vec(out_n, "out_n", i64, dev, 1))
    rc = L.tt_plan_blocks(args, _stream(stream, dev))
    if rc != TT_OK:
        _check(rc, "tt_plan_blocks")


def release_blocks_into(lengths, done, table, free_blocks, n_free, block_size, out_n, out_lengths=None,
                        out_n_free=None, stream=None):
    """Enqueue tt_release_blocks: rows with ``done`` (bool or uint8 [R]) give their blocks back to the end of the
    free list and become rows not in use (length -1)."""
    L = _lib or _start()
    dev = _device(lengths, "lengths")
    i32 = _torch.int32
    n = lengths.numel()
    t, ts = _mat(table, "table", i32, dev, n)
    if done.dtype is not _torch.bool and done.dtype is not _torch.uint8:
        raise ValueError("done: truth values are needed, got %s" % done.dtype)
    rc = L.tt_release_blocks(
        _vec(lengths, "lengths", i32, dev), _vec(done, "done", done.dtype, dev, n), n, int(block_size), t, ts,
        table.shape[1], _vec(free_blocks, "free_blocks", i32, dev), free_blocks.numel(),
        _vec(n_free, "n_free", i32, dev, 1),
        lengths.data_ptr() if out_lengths is None else _vec(out_lengths, "out_lengths", i32, dev, n),
        n_free.data_ptr() if out_n_free is None else _vec(out_n_free, "out_n_free", i32, dev, 1),
        _vec(out_n, "out_n", _torch.int64, dev, 1), _stream(stream, dev))
    if rc != TT_OK:
        _check(rc, "tt_release_blocks")


class BlockTable:
    """The block table of ``rows`` requests of up to ``width`` blocks each, over a cache of ``blocks`` blocks:
    ``lengths`` (-1: row not in use), ``table``, ``free_blocks`` and ``n_free``, all on the GPU.

        slots, positions, rows = cache.plan(offsets)   # prompts: offsets int64 [rows + 1]
        slots, positions, rows = cache.plan()          # a step: one token for each row in use
        cache.release(done)
    """

    def __init__(self, rows, width, blocks, block_size, device="cuda"):
        if _lib is None:
            _start()
        make = dict(dtype=_torch.int32, device=device)
        self.block_size = int(block_size)
        self.lengths = _torch.full((rows,), -1, **make)
        self.table = _torch.full((rows, width), -1, **make)
        self.free_blocks = _torch.arange(blocks - 1, -1, -1, **make)  # the last entry is taken first
        self.n_free = _torch.full((1,), blocks, **make)

    def plan_into(self, slots, out_n, offsets=None, positions=None, rows=None, stream=None):
        plan_blocks_into(self.lengths, self.table, self.free_blocks, self.n_free, self.block_size, slots, out_n,
                         offsets=offsets, positions=positions, rows=rows, stream=stream)

    def plan(self, offsets=None, stream=None):
        """(slots, positions, rows) of the new tokens; raises if the device reports an error."""
        with _on(stream):
            places = self.lengths.numel() if offsets is None else int(offsets[-1].item())
            dev = self.lengths.device
            slots = _torch.empty(max(places, 0), dtype=_torch.int64, device=dev)
            positions, rows = (_torch.empty(max(places, 0), dtype=_torch.int32, device=dev) for _ in range(2))
            out_n = _torch.empty(1, dtype=_torch.int64, device=dev)
            self.plan_into(slots, out_n, offsets, positions, rows, stream)
            _raise_count(out_n, "tt_plan_blocks")
        return slots, positions, rows

    def release_into(self, done, out_n, stream=None):
        release_blocks_into(self.lengths, done, self.table, self.free_blocks, self.n_free, self.block_size, out_n,
                            stream=stream)

    def release(self, done, stream=None):
        """The rows of ``done`` end; returns how many blocks came back."""
        with _on(stream):
            out_n = _torch.empty(1, dtype=_torch.int64, device=self.lengths.device)
            self.release_into(done, out_n, stream)
            return _raise_count(out_n, "tt_release_blocks")


# --------------------------------------------------------------- token sets

def token_bits_into(ids, bits, vocab, offsets=None, add=False, stream=None):
    """Enqueue tt_token_bits: ``bits`` (int32 [R, words]) receives (``add``: is joined with) the sets of the ids
    of each text, ``ids[offsets[r]:offsets[r + 1]]``; without ``offsets`` all ids are one text."""
    L = _lib or _start()
    dev = _device(bits, "bits")
    rows = 1 if offsets is None else offsets.numel() - 1
    b, bs = _mat(bits, "bits", _torch.int32, dev, rows, _words(vocab))
    n = ids.numel()
    rc = L.tt_token_bits(_vec(ids, "ids", _torch.int32, dev) if n else None, n,
                         None if offsets is None else _vec(offsets, "offsets", _torch.int64, dev), rows, int(vocab),
                         b, bs, 1 if add else 0, _stream(stream, dev))
    if rc != TT_OK:
        _check(rc, "tt_token_bits")


def token_bits(ids, vocab, offsets=None, stream=None):
    """The token sets (int32 [R, words]) of the ids of each text."""
    if _lib is None:
        _start()
    with _on(stream):
        bits = _torch.empty((1 if offsets is None else offsets.numel() - 1, _words(vocab)), dtype=_torch.int32,
                            device=ids.device)
        token_bits_into(ids, bits, vocab, offsets=offsets, stream=stream)
    return bits


class TokenStrings:
    """The byte strings of a vocabulary on the GPU: token v is ``strings[offsets[v]:offsets[v + 1]]`` (uint8
    and whole numbers, on the host).  A token without bytes is one that no grammar allows."""

    def __init__(self, strings, offsets, device="cuda"):
        if _lib is None:
            _start()
        strings = np.ascontiguousarray(np.asarray(strings, dtype=np.uint8).reshape(-1))
        offsets = np.asarray(offsets).reshape(-1)
        if not len(offsets) or offsets[0] < 0 or offsets[-1] > len(strings) or np.any(offsets[1:] < offsets[:-1]):
            raise ValueError("offsets: one more than there are tokens, in order and inside the strings")
        if len(strings) > 0x7FFFFFFF or len(offsets) > (1 << 24) + 1:
            raise ValueError("strings of at most 2^31 - 1 bytes and 2^24 tokens")
        self.n_tokens = len(offsets) - 1
        self.strings = _torch.from_numpy(strings.copy()).to(device)
        self.offsets = _torch.from_numpy(offsets.astype(np.int32)).to(device)

    @classmethod
    def of_tokenizer(cls, device="cuda"):
        """The strings of the loaded tokenizer."""
        L = _lib or _start()
        n, size = ctypes.c_int64(), ctypes.c_int64()
        _check(L.tt_vocab_size(ctypes.byref(n), ctypes.byref(size)), "tt_vocab_size")
        strings, offsets = np.empty(size.value, np.uint8), np.empty(n.value + 1, np.int32)
        _check(L.tt_vocab_strings(strings.ctypes.data, offsets.ctypes.data), "tt_vocab_strings")
        return cls(strings, offsets, device)


class Grammar:
    """An automaton over bytes on the GPU: ``next`` [S, 256] gives the state after each byte, -1 where there is none;
    ``accept`` [S] the states in which an answer may end.  ``end_id`` is the token that ends it (-1: none).
    Bytes that no state tells apart are put into one class, which makes the table small enough for LDS."""

    def __init__(self, next, accept=None, end_id=-1, device="cuda"):
        if _lib is None:
            _start()
        table = np.asarray(next)
        if table.ndim != 2 or table.shape[1] != 256 or not 1 <= table.shape[0] <= 32767:
            raise ValueError("next: [S, 256] with 1 <= S <= 32767 is needed, got %s" % (table.shape,))
        n = table.shape[0]
        if not np.issubdtype(table.dtype, np.integer) or table.min() < -1 or table.max() >= n:
            raise ValueError("next: whole numbers from -1 to %d are needed" % (n - 1))
        accept = np.zeros(n, bool) if accept is None else np.asarray(accept)
        if accept.shape != (n,):
            raise ValueError("accept: one entry for each of %d states is needed" % n)
        columns, classes = np.unique(table.astype(np.int16), axis=1, return_inverse=True)
        self.n_states, self.n_classes, self.end_id = n, columns.shape[1], int(end_id)
        self.classes = _torch.from_numpy(classes.reshape(-1).astype(np.uint8)).to(device)
        self.next = _torch.from_numpy(np.ascontiguousarray(columns)).to(device)
        self.accept = _torch.from_numpy((accept != 0).astype(np.uint8)).to(device)

    def _args(self, tokens):
        return _GRAMMAR.pack(self.classes.data_ptr(), self.next.data_ptr(), self.accept.data_ptr(), self.n_states,
                             self.n_classes, self.end_id, tokens.strings.data_ptr(), tokens.strings.numel(),
                             tokens.offsets.data_ptr(), tokens.n_tokens)


def _same_device(grammar, tokens, dev):
    if grammar.next.get_device() != dev or tokens.strings.get_device() != dev:
        raise ValueError("the grammar, the token strings and the states have to be on one device")


def grammar_bits_into(grammar, tokens, states, bits, vocab=None, stream=None):
    """Enqueue tt_grammar_bits: ``bits`` (int32 [R, words]) receives the tokens (a TokenStrings) that may follow
    each of ``states`` (int32 [R]; STATE_DEAD: none, STATE_FREE: all).  ``vocab`` is the model's, by default the
    strings'."""
    L = _lib or _start()
    dev = _device(states, "states")
    _same_device(grammar, tokens, dev)
    vocab = tokens.n_tokens if vocab is None else int(vocab)
    n = states.numel()
    b, bs = _mat(bits, "bits", _torch.int32, dev, n, _words(vocab))
    rc = L.tt_grammar_bits(grammar._args(tokens), _vec(states, "states", _torch.int32, dev), n, b, bs, vocab,
                           _stream(stream, dev))
    if rc != TT_OK:
        _check(rc, "tt_grammar_bits")


def grammar_bits(grammar, tokens, states=None, vocab=None, stream=None):
    """The token sets that may follow ``states``; without them the set of every state, row q for state q, which is
    what shape_logits takes as ``allowed`` with the states as ``allowed_rows``."""
    if _lib is None:
        _start()
    with _on(stream):
        if states is None:
            states = _torch.arange(grammar.n_states, dtype=_torch.int32, device=grammar.next.device)
        bits = _torch.empty((states.numel(), _words(tokens.n_tokens if vocab is None else int(vocab))),
                            dtype=_torch.int32, device=states.device)
        grammar_bits_into(grammar, tokens, states, bits, vocab, stream)
    return bits


def grammar_advance_into(grammar, tokens, states, chosen, out_states=None, stream=None):
    """Enqueue tt_grammar_advance: the states after the ``chosen`` tokens (int32 [R]), in place unless
    ``out_states`` is given."""
    L = _lib or _start()
    dev = _device(states, "states")
    _same_device(grammar, tokens, dev)
    n = states.numel()
    s = _vec(states, "states", _torch.int32, dev)
    rc = L.tt_grammar_advance(grammar._args(tokens), s, _vec(chosen, "chosen", _torch.int32, dev, n), n,
                              s if out_states is None else _vec(out_states, "out_states", _torch.int32, dev, n),
                              _stream(stream, dev))
    if rc != TT_OK:
        _check(rc, "tt_grammar_advance")


# ------------------------------------------------------------------- logits

def shape_logits_into(logits, out, seen=None, generated=None, n_generated=None, repetition=None, frequency=None,
                      presence=None, bias_offsets=None, bias_ids=None, bias_values=None, allowed=None,
                      allowed_rows=None, temperature=None, stream=None):
    """Enqueue tt_shape_logits: penalties for repeated tokens, biases, the allowed sets and the temperature,
    applied to ``logits`` [R, V] (float32, float16 or bfloat16) and rounded once to ``out`` (the same type or float32;
    it may be ``logits``).

    ``seen``: token sets int32 [R, words] of the prompts; ``generated`` int32 [R, cap] with ``n_generated`` int32 [R];
    ``repetition``, ``frequency``, ``presence``, ``temperature``: float32 [R]; ``bias_offsets`` int64 [R + 1],
    ``bias_ids`` int32 and ``bias_values`` float32 [N]; ``allowed``: token sets int32 [S, words], row r going by
    ``allowed_rows[r]`` (int32; STATE_FREE: everything allowed) or, without it, by set r.
    """
    L = _lib or _start()
    dev = _device(logits, "logits")
    i32, f32 = _torch.int32, _torch.float32
    kind, okind = _types.get(logits.dtype), _types.get(out.dtype)
    if kind is None or okind is None or (okind != kind and okind != F32):
        raise ValueError("logits %s to %s: float32, float16 or bfloat16 to itself or to float32 is needed"
                         % (logits.dtype, out.dtype))
    x, xs = _mat(logits, "logits", logits.dtype, dev)
    n, vocab = logits.shape
    y, ys = _mat(out, "out", out.dtype, dev, n)
    if out.shape[1] != vocab:
        raise ValueError("out has rows of %d entries, not %d" % (out.shape[1], vocab))
    words = (vocab + 31) // 32
    s, ss = (0, 0) if seen is None else _mat(seen, "seen", i32, dev, n, words)
    g, gs, cap = 0, 0, 0
    if generated is not None:
        g, gs = _mat(generated, "generated", i32, dev, n)
        cap = generated.shape[1]
    a, as_, count = 0, 0, 0
    if allowed is not None:
        count = n if allowed_rows is None else None
        a, as_ = _mat(allowed, "allowed", i32, dev, count, words)
        count = allowed.shape[0]
        a = a or x  # without a single set there is no address, but the rows still go by them
    elif allowed_rows is not None:
        raise ValueError("allowed_rows without allowed")
    n_bias = 0
    if bias_offsets is not None:
        if bias_ids is None or bias_values is None:
            raise ValueError("bias_offsets without bias_ids and bias_values")
        n_bias = bias_ids.numel()
    elif bias_ids is not None or bias_values is not None:
        raise ValueError("bias_ids and bias_values without bias_offsets")
    args = _SHAPE.pack(
        x, xs, y, ys, n, vocab, kind, okind, s, ss, g, gs, cap,
        0 if n_generated is None else _vec(n_generated, "n_generated", i32, dev, n),
        0 if repetition is None else _vec(repetition, "repetition", f32, dev, n),
        0 if frequency is None else _vec(frequency, "frequency", f32, dev, n),
        0 if presence is None else _vec(presence, "presence", f32, dev, n),
        0 if bias_offsets is None else _vec(bias_offsets, "bias_offsets", _torch.int64, dev, n + 1),
        0 if bias_offsets is None else _vec(bias_ids, "bias_ids", i32, dev),
        0 if bias_offsets is None else _vec(bias_values, "bias_values", f32, dev, n_bias), n_bias,
        a, as_, count, 0 if allowed_rows is None else _vec(allowed_rows, "allowed_rows", i32, dev, n),
        0 if temperature is None else _vec(temperature, "temperature", f32, dev, n))
    rc = L.tt_shape_logits(args, _stream(stream, dev))
    if rc != TT_OK:
        _check(rc, "tt_shape_logits")


def shape_logits(logits, dtype=None, stream=None, **options):
    """The shaped logits as a new tensor of ``dtype`` (default: float32); options as in shape_logits_into."""
    if _lib is None:
        _start()
    with _on(stream):
        out = _torch.empty(logits.shape, dtype=_torch.float32 if dtype is None else dtype, device=logits.device)
        shape_logits_into(logits, out, stream=stream, **options)
    return out
