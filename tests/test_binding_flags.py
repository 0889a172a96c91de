"""The calls' flags (causal, pairs) take what int() takes, as the ctypes binding's
did: numpy's truth values and floats among them. The other whole numbers do not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _util import ensure_library  # noqa: E402

ensure_library()
import decode_dsa_kv_gb300 as d  # noqa: E402
from decode_dsa_kv_gb300 import _abi  # noqa: E402

A = 0x10000          # a fake, aligned address (never dereferenced: no token, no row)
FLAGS = [True, 0, 7, np.bool_(True), np.bool_(False), np.int64(1), np.float32(1), 1.0, 0.5, "1",
         torch.tensor(True), torch.tensor(1.0)]


def chunk(T=0, causal=True):
    return d.sfa_mla_chunk(A, 16 * 576, A, T, 1, 16, A, 64, _abi.DSA_CACHE_BF16, A, 4, 16, A, causal,
                           1 / 24, A, None, A, 1 << 30, None, 0)


def append(n=0, pairs=True):
    return d.dsa_cache_append(A, 512, A, 64, A, A, n, A, pairs, A, 64, _abi.DSA_CACHE_BF16, None, 0, 0,
                              0, None, 0, None, 0)


@pytest.mark.parametrize("flag", FLAGS, ids=lambda x: f"{type(x).__name__}:{x}")
def test_flags(flag):
    assert chunk(causal=flag) == _abi.TS_OK
    assert append(pairs=flag) == _abi.TS_OK


@pytest.mark.parametrize("flag, error", [(None, TypeError), ("yes", ValueError), ([], TypeError),
                                         (float("nan"), ValueError)])
def test_what_int_refuses(flag, error):
    for call in (lambda: chunk(causal=flag), lambda: append(pairs=flag)):
        with pytest.raises(error):
            call()


def test_the_other_numbers_are_whole():
    for bad in (1.0, np.float32(0), "0"):
        with pytest.raises(TypeError):
            chunk(T=bad)
        with pytest.raises(TypeError):
            append(n=bad)
    assert chunk(T=np.int32(0)) == append(n=np.int64(0)) == _abi.TS_OK
