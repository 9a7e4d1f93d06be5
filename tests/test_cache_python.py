"""PagedCache's own checks without a GPU: a cache over CPU memory whose calls end where
something would be enqueued."""
import contextlib

import pytest
import torch

import kv_cache_compression_04_b200 as kvc
from kv_cache_compression_04_b200 import build

ENQUEUED = kvc.KVC_ERR_CUDA  # what a call that passes its checks ends with here


class HostCache(kvc.PagedCache):
    """A cache whose pool, status word and workspaces are CPU memory."""

    def __init__(self, layers=1, heads=2, d=128, pages=4, page=16, group=64):
        self.status = torch.zeros(1, dtype=torch.int32)
        self._ws, self._lock, self._calls = {}, kvc.threading.Lock(), (None, None, None, {})
        desc = kvc.kvc_cache_desc(layers, heads, d, 4, group, 0, 0, 0, 3, page, 0, pages)
        block = kvc.kvc_cache_block_bytes(desc)
        self._set(desc, torch.zeros(layers, pages, 2, heads, block, dtype=torch.uint8))

    def _here(self, stream, *tensors):
        return 0


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would be enqueued on CPU pointers")
    build.build()
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())


def load(c, lens, nbytes=64):
    n = sum(lens)
    c.load(torch.zeros(64, dtype=torch.uint8), nbytes, torch.zeros(n, dtype=torch.int64), lens)


def status(call):
    with pytest.raises(kvc.KvcError) as e:
        call()
    return e.value.status


@pytest.mark.parametrize("refused", [[1] * 1025, [3, -1], [2 ** 31 - 1, 1 - 2 ** 31]])
def test_a_refused_load_leaves_the_stream_usable(refused):
    """The first call on a stream: nothing of it is kept."""
    c = HostCache()
    assert status(lambda: load(c, refused)) == kvc.KVC_ERR_INVALID_ARG
    assert status(lambda: load(c, [5])) == ENQUEUED
    assert status(lambda: load(c, refused)) == kvc.KVC_ERR_INVALID_ARG
    assert status(lambda: load(c, [500])) == ENQUEUED


@pytest.mark.parametrize("nbytes", [-1, -2 ** 63, 65, 2 ** 64])
def test_load_refuses_a_size_that_the_buffer_does_not_have(nbytes):
    """A negative one would reach the library as a size near 2^64."""
    with pytest.raises(ValueError):
        load(HostCache(), [5], nbytes)


def test_load_noting_checks_its_status_word():
    """kvc_cache_load's checks, and the status word's alignment."""
    fake, c, seq = 0x7F0000000000, HostCache().desc, [5, 0, 9]
    c.pool = fake
    size = kvc.kvc_cache_load_workspace_bytes(c, seq)

    def call(status, ws=size, lens=seq):
        return kvc.kvc_cache_load_noting(fake, 4096, c, lens, fake, fake, ws, status, None)

    assert call(fake + 4) == call(None) == ENQUEUED
    assert call(fake + 2) == kvc.KVC_ERR_INVALID_ARG
    assert call(fake, size - 1) == kvc.KVC_ERR_CAPACITY
    assert call(fake, size, [5, -1]) == kvc.KVC_ERR_INVALID_ARG


def test_attention_of_too_many_rows_is_refused():
    """2^31 rows of out in all: refused with the arguments, not after two kernels."""
    fake, c = 0x7F0000000000, kvc.kvc_cache_desc(64, 8, 128, 4, 128, 0, 0, 0, 0, 16, 0, 4, 0x7F0000000000)
    for tokens, starts, max_q in ((1 << 20, fake, 1), (1 << 20, fake, 500)):
        for n, want in ((tokens - 1, ENQUEUED), (tokens, kvc.KVC_ERR_UNSUPPORTED)):
            t = kvc.kvc_cache_attn(0, 4, 3, max_q, 1, 0, 0.1, 0, n, starts, fake, fake, 10, 10, fake,
                                   n * 4096, 4096, 128, fake, n * 4096, 4096, 128, None)
            assert (kvc.kvc_cache_attend_workspace_bytes(c, t) == 0) == (n == tokens)
            assert kvc.kvc_cache_attend(c, t, fake, 1 << 60, None, None) == want


def test_waiting_calls_refuse_a_capture(monkeypatch):
    """Before anything is enqueued, on the current stream and on one that is given."""
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: True)
    c = HostCache()
    for stream in (None, object()):
        with pytest.raises(ValueError):
            c.check(stream=stream)
        with pytest.raises(ValueError):
            c.load(torch.zeros(64, dtype=torch.uint8), 64, torch.zeros(5, dtype=torch.int64), [5], stream=stream, check=True)
    assert status(lambda: load(c, [5])) == ENQUEUED and not c._ws
