"""CPU tests of what the binding of the cache and window operators refuses, and
how it names it."""
import ctypes

import pytest
import torch

import token_level_top_hs2_b200 as hs2
from token_level_top_hs2_b200 import build as hs2_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    hs2_build.build()
    return hs2.load()


def test_a_misaligned_tensor_is_named():
    """lengths[1:] of a batch's lengths: the library would say only that some
    argument is invalid."""
    lengths = torch.zeros(9, dtype=torch.int32)
    assert hs2._dense(lengths[:8], "lengths", (torch.int32,), (8,), -1) == lengths.data_ptr()
    assert hs2._dense(lengths[4:8], "lengths", (torch.int32,), (4,), -1) == lengths.data_ptr() + 16
    with pytest.raises(ValueError, match="lengths: must start on a 16-byte boundary"):
        hs2._dense(lengths[1:], "lengths", (torch.int32,), (8,), -1)
    with pytest.raises(ValueError, match="start: must start on a 16-byte boundary"):
        hs2._dense_or_none(lengths[2:], "start", (torch.int32,), (7,), -1)


class Said(Exception):
    pass


def test_windows_and_sinks_beyond_32_bits_are_not_wrapped(monkeypatch):
    """-2^32 + 5 is no window of 5."""
    seen = {}

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                ints = [a for a in args if isinstance(a, int)]
                shape = args[0]
                seen[name] = ((shape.window, shape.n_sink) if isinstance(shape, hs2.WindowShape)
                              else tuple(ctypes.c_int(i).value for i in ints[1:3]))
                assert name != "hs2_paged_decode" or seen[name] == tuple(ints[1:3])
                return hs2.HS2_ERR_INVALID_ARG
            return call

    monkeypatch.setattr(hs2, "load", Lib)
    monkeypatch.setattr(hs2, "_current_device", lambda: -1)
    monkeypatch.setattr(hs2, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(hs2, "_paged_workspace", lambda *a: 16)
    monkeypatch.setattr(hs2, "_rank", lambda t, name, rank: t.shape)
    bf = torch.bfloat16
    q, kv = torch.zeros(1, 4, 2, 64, dtype=bf), torch.zeros(1, 4, 1, 64, dtype=bf)
    qd, pages = torch.zeros(1, 2, 64, dtype=bf), torch.zeros(2, 1, 16, 64, dtype=torch.uint8)
    table, lengths, sc = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, 1)
    ws, big = torch.zeros(64, dtype=torch.uint8), 2**32
    for window, n_sink, want in ((5, 4, (5, 4)), (5 - big, 4, (-1, 4)), (5, 4 - big, (5, -1)),
                                 (big + 5, big + 4, (2**31 - 1, 2**31 - 1)), (0, 0, (0, 0))):
        for name, call in (
            ("hs2_window_attn", lambda: hs2.hs2_window_attn(q, kv, kv, window, n_sink, o=q,
                                                            lse=torch.zeros(1, 4, 2))),
            ("hs2_paged_decode", lambda: hs2.hs2_paged_decode(qd, pages, pages, sc, sc, table, lengths, window=window,
                                                              n_sink=n_sink, o=qd, lse=torch.zeros(1, 2),
                                                              workspace=ws))):
            monkeypatch.setattr(hs2, "_check", lambda st, what: (_ for _ in ()).throw(Said()))
            with pytest.raises(Said):
                call()
            assert seen[name] == want, (name, window, n_sink)
