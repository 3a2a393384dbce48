"""What a serving step needs next to the tokenizer: block tables of a paged
cache, token sets, grammar masks and the shaping of logits (C ABI in
include/tt_serve.h; the meaning of every argument is described there).

The ``*_into`` calls write into the caller's tensors and only enqueue on the
current stream (or ``stream``), so they can be captured into a HIP graph; the
others make their results and, where the device may report a data error, wait
for it.  Arguments of a wrong type, shape or device raise ValueError.

Nothing is differentiated: results carry no gradient, whatever the logits carry.  What is written in place counts as
modified, so that a gradient which needs the value from before raises.

    ids, offsets = tt.encode_batch(prompts, starts)           # offsets: int64 [B + 1]
    cache = tt.BlockTable(rows=B, width=256, blocks=4096, block_size=16)
    slots, positions, rows = cache.plan(offsets.cuda())
    seen = tt.token_bits(ids, vocab, offsets=offsets.cuda())
    out = tt.shape_logits(logits, seen=seen, repetition=rho, temperature=t)
"""
import contextlib
import ctypes
import importlib.util
import os
import struct

import numpy as np

from . import TTError, TT_ESTALE, TT_ETOOBIG, TT_OK, _check, lib as _base_lib

STATE_DEAD, STATE_FREE = -1, -2

BIND_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_bind.so")

_bind = None   # checks tensors and calls the library
_torch = None


def _start():
    """Load the library's serving calls and their binding, once."""
    global _bind, _torch
    import torch
    L = _base_lib()
    if not os.path.exists(BIND_PATH):
        raise RuntimeError("_bind.so not built (%s); run exact_byte_level_amd.build.build()" % BIND_PATH)
    spec = importlib.util.spec_from_file_location("_bind", BIND_PATH)
    bind = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bind)
    bind.connect(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
        "tt_plan_blocks", "tt_release_blocks", "tt_token_bits", "tt_grammar_bits", "tt_grammar_advance",
        "tt_shape_logits")))
    L.tt_vocab_size.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    L.tt_vocab_strings.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64]
    _torch = torch
    _bind = bind
    return bind


def _on(stream):
    """What is allocated inside belongs to the stream it is used on."""
    return contextlib.nullcontext() if stream is None else _torch.cuda.stream(stream)


def _handle(stream):
    return None if stream is None else stream.cuda_stream


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
    rc = (_bind or _start()).plan(lengths, table, free_blocks, n_free, block_size, slots, out_n, offsets, positions, rows,
                                  out_lengths, out_n_free, _handle(stream))
    if rc != TT_OK:
        _check(rc, "tt_plan_blocks")


def release_blocks_into(lengths, done, table, free_blocks, n_free, block_size, out_n, out_lengths=None,
                        out_n_free=None, stream=None):
    """Enqueue tt_release_blocks: rows with ``done`` (bool or uint8 [R]) give their blocks back to the end of the
    free list and become rows not in use (length -1)."""
    rc = (_bind or _start()).release(lengths, done, table, free_blocks, n_free, block_size, out_n, out_lengths,
                                     out_n_free, _handle(stream))
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
        if _bind is None:
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
            places, dev = self.lengths.numel(), self.lengths.device
            if offsets is not None:
                if offsets.shape != (places + 1,):
                    raise ValueError("offsets: [%d] is needed, got %s" % (places + 1, list(offsets.shape)))
                places = int(offsets[-1].item())
                if places > 0x7FFFFFFF:
                    raise TTError(TT_ETOOBIG, "tt_plan_blocks")
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
    rc = (_bind or _start()).token_bits(ids, bits, vocab, offsets, add, _handle(stream))
    if rc != TT_OK:
        _check(rc, "tt_token_bits")


def token_bits(ids, vocab, offsets=None, stream=None):
    """The token sets (int32 [R, words]) of the ids of each text."""
    if _bind is None:
        _start()
    with _on(stream):
        bits = _torch.empty((1 if offsets is None else max(offsets.numel() - 1, 0), _words(vocab)), dtype=_torch.int32,
                            device=ids.device)
        token_bits_into(ids, bits, vocab, offsets=offsets, stream=stream)
    return bits


class _OnDevice:
    """Tensors whose addresses the calls take from ``_fields``, packed once.  They stay alive with the object, also where an
    attribute is set to another tensor (which the calls do not see); a copy points to its own."""

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_fields"}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._point(*self._tensors)


class TokenStrings(_OnDevice):
    """The byte strings of a vocabulary on the GPU: token v is ``strings[offsets[v]:offsets[v + 1]]`` (uint8
    and whole numbers, on the host).  A token without bytes is one that no grammar allows."""

    def __init__(self, strings, offsets, device="cuda"):
        if _bind is None:
            _start()
        strings, offsets = np.asarray(strings).reshape(-1), np.asarray(offsets).reshape(-1)
        if strings.dtype != np.uint8 and len(strings):
            whole = strings.dtype.kind in "biuf" and np.all(strings == np.floor(strings))
            if not whole or strings.min() < 0 or strings.max() > 255:
                raise ValueError("strings: bytes, as whole numbers from 0 to 255, are needed")
        if offsets.dtype.kind not in "iu" and np.any(offsets != np.floor(offsets)):
            raise ValueError("offsets: whole numbers are needed")
        strings = np.ascontiguousarray(strings.astype(np.uint8, copy=False))
        if not len(offsets) or offsets[0] < 0 or offsets[-1] > len(strings) or np.any(offsets[1:] < offsets[:-1]):
            raise ValueError("offsets: one more than there are tokens, in order and inside the strings")
        if len(strings) > 0x7FFFFFFF or len(offsets) > (1 << 24) + 1:
            raise ValueError("strings of at most 2^31 - 1 bytes and 2^24 tokens")
        self.n_tokens = len(offsets) - 1
        self.strings = _torch.from_numpy(strings.copy()).to(device)
        self.offsets = _torch.from_numpy(offsets.astype(np.int32)).to(device)
        self._point(self.strings, self.offsets)

    def _point(self, strings, offsets):
        self._tensors = strings, offsets
        self._device = strings.get_device()
        # the last fields of tt_grammar
        self._fields = struct.pack("=4q", strings.data_ptr(), strings.numel(), offsets.data_ptr(), self.n_tokens)

    @classmethod
    def of_tokenizer(cls, device="cuda"):
        """The strings of the loaded tokenizer."""
        if _bind is None:
            _start()
        L = _base_lib()
        n, size = ctypes.c_int64(), ctypes.c_int64()
        rc = TT_ESTALE
        while rc == TT_ESTALE:  # another thread has loaded another tokenizer in between
            _check(L.tt_vocab_size(ctypes.byref(n), ctypes.byref(size)), "tt_vocab_size")
            strings, offsets = np.empty(size.value, np.uint8), np.empty(n.value + 1, np.int32)
            rc = L.tt_vocab_strings(strings.ctypes.data, offsets.ctypes.data, n, size)
        _check(rc, "tt_vocab_strings")
        return cls(strings, offsets, device)


class Grammar(_OnDevice):
    """An automaton over bytes on the GPU: ``next`` [S, 256] gives the state after each byte, -1 where there is none;
    ``accept`` [S] the states in which an answer may end.  ``end_id`` is the token that ends it (-1: none).
    Bytes that no state tells apart are put into one class, which makes the table small enough for LDS."""

    def __init__(self, next, accept=None, end_id=-1, device="cuda"):
        if _bind is None:
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
        by_byte = np.ascontiguousarray(table.astype(np.int16).T)
        seen = {}  # a byte's column -> its class
        classes = np.array([seen.setdefault(column.tobytes(), len(seen)) for column in by_byte], np.uint8)
        first = np.unique(classes, return_index=True)[1]
        self.n_states, self.n_classes, self.end_id = n, len(seen), int(end_id)
        self.classes = _torch.from_numpy(classes).to(device)
        self.next = _torch.from_numpy(np.ascontiguousarray(by_byte[first].T)).to(device)
        self.accept = _torch.from_numpy((accept != 0).astype(np.uint8)).to(device)
        self._point(self.classes, self.next, self.accept)

    def _point(self, classes, next, accept):
        self._tensors = classes, next, accept
        self._device = next.get_device()
        # the first fields of tt_grammar
        self._fields = struct.pack("=6q", classes.data_ptr(), next.data_ptr(), accept.data_ptr(), self.n_states,
                                   self.n_classes, self.end_id)


def _shared_device(grammar, tokens):
    return grammar._device if grammar._device == tokens._device else -1


def grammar_bits_into(grammar, tokens, states, bits, vocab=None, stream=None):
    """Enqueue tt_grammar_bits: ``bits`` (int32 [R, words]) receives the tokens (a TokenStrings) that may follow
    each of ``states`` (int32 [R]; STATE_DEAD: none, STATE_FREE: all).  ``vocab`` is the model's, by default the
    strings'."""
    rc = (_bind or _start()).grammar_bits(grammar._fields + tokens._fields, _shared_device(grammar, tokens), states, bits,
                                          tokens.n_tokens if vocab is None else vocab, _handle(stream))
    if rc != TT_OK:
        _check(rc, "tt_grammar_bits")


def grammar_bits(grammar, tokens, states=None, vocab=None, stream=None):
    """The token sets that may follow ``states``; without them the set of every state, row q for state q, which is
    what shape_logits takes as ``allowed`` with the states as ``allowed_rows``."""
    if _bind is None:
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
    rc = (_bind or _start()).grammar_advance(grammar._fields + tokens._fields, _shared_device(grammar, tokens), states,
                                             chosen, out_states, _handle(stream))
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
    rc = (_bind or _start()).shape(logits, out, seen, generated, n_generated, repetition, frequency, presence,
                                   bias_offsets, bias_ids, bias_values, allowed, allowed_rows, temperature,
                                   _handle(stream))
    if rc != TT_OK:
        _check(rc, "tt_shape_logits")


def shape_logits(logits, dtype=None, stream=None, **options):
    """The shaped logits as a new tensor of ``dtype`` (default: float32); options as in shape_logits_into."""
    if _bind is None:
        _start()
    with _on(stream):
        out = _torch.empty(logits.shape, dtype=_torch.float32 if dtype is None else dtype, device=logits.device)
        shape_logits_into(logits, out, stream=stream, **options)
    return out
