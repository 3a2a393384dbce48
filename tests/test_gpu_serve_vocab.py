"""Token strings of the loaded tokenizer: sizes that no longer hold, and a tokenizer that is replaced in between."""
import ctypes
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from exact_byte_level_amd import serve  # noqa: E402

MERGES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "data", "vocab_c1.npy")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("more_tokens, more_bytes", [(-1, 0), (1, 0), (0, -1), (0, 1), (-200, 50)])
def test_strings_are_not_written_to_other_sizes(more_tokens, more_bytes):
    tt.load(np.load(MERGES)[:300])
    serve.TokenStrings.of_tokenizer()  # declares the calls' arguments
    n, size = ctypes.c_int64(), ctypes.c_int64()
    L = tt.lib()
    assert L.tt_vocab_size(ctypes.byref(n), ctypes.byref(size)) == tt.TT_OK and n.value == 556
    strings, offsets = np.full(size.value, 7, np.uint8), np.full(n.value + 1, 7, np.int32)
    args = strings.ctypes.data, offsets.ctypes.data, n.value + more_tokens, size.value + more_bytes
    assert L.tt_vocab_strings(*args) == tt.TT_ESTALE
    assert (strings == 7).all() and (offsets == 7).all()
    assert L.tt_vocab_strings(*args[:2], n, size) == tt.TT_OK
    assert offsets[0] == 0 and offsets[-1] == size.value and (strings[:256] == np.arange(256)).all()


@pytest.mark.parametrize("first, then", [(50, 400), (400, 50)])
def test_a_tokenizer_loaded_in_between(monkeypatch, first, then):
    """As if another thread loaded it right after the sizes were read."""
    merges = np.load(MERGES)
    tt.load(merges[:then])
    want = tt.TokenStrings.of_tokenizer()
    tt.load(merges[:first])
    real = tt.lib()

    class Between:
        tt_vocab_strings = staticmethod(real.tt_vocab_strings)
        turns = 0

        def tt_vocab_size(self, *sizes):
            rc = real.tt_vocab_size(*sizes)
            if not self.turns:
                tt.load(merges[:then])
            self.turns += 1
            return rc

    between = Between()
    monkeypatch.setattr(serve, "_base_lib", lambda: between)
    got = tt.TokenStrings.of_tokenizer()
    assert between.turns == 2 and got.n_tokens == 256 + then
    assert torch.equal(got.strings, want.strings) and torch.equal(got.offsets, want.offsets)
