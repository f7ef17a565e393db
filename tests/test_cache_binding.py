"""The binding's own checks (no GPU): what must not reach the library."""
import numpy as np
import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg


class NoLibrary:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(cg, "lib", NoLibrary)


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


@pytest.mark.parametrize("n,m", [(3, 2), (2, 3), (1, 0), (0, 1)])
def test_lists_of_pairs_have_one_length(no_library, n, m):
    """An extension, a fork or a copy whose two lists differ in length would read past the shorter one."""
    cache, pages, ws = cg.Cache(1, 1, 8, 4, 8), cg.Pages(i32(8), i32(8).view(4, 2), i32(4)), i32(256)
    ptrs = torch.zeros(2, dtype=torch.int64)
    assert cg.cg_pages_extend(cache, pages, i32(n), i32(m), ws, 0) == cg.CG_ERR_INVALID_ARG
    assert cg.cg_pages_fork(cache, pages, ptrs, ptrs, i32(n), i32(m), ws, 0) == cg.CG_ERR_INVALID_ARG
    assert cg.cg_pages_copy(cache, ptrs, ptrs, i32(n), i32(m), ws, 0) == cg.CG_ERR_INVALID_ARG


@pytest.mark.parametrize("x", [3.7, "7", b"7", np.int64(4096), np.zeros(1, np.int64), [4096], object()])
def test_what_is_no_address_is_not_made_one(x):
    with pytest.raises(AttributeError):
        cg._ptr(x)


def test_addresses():
    t = i32(4)
    assert (cg._ptr(t), cg._ptr(None), cg._ptr(4096), cg._ptr(0)) == (t.data_ptr(), 0, 4096, 0)


def test_the_current_stream_before_cuda_is_initialised(monkeypatch):
    """Until torch has initialised CUDA in this process, the current stream is asked for by torch's public call, which
    initialises it or says why it cannot."""
    class Stream:
        cuda_stream = 0x1230

    def cannot():
        raise RuntimeError("no CUDA here")

    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    assert cg._stream(None) == 0x1230
    monkeypatch.setattr(torch.cuda, "current_stream", cannot)
    with pytest.raises(RuntimeError, match="no CUDA here"):
        cg._stream(None)


def test_streams_by_object_and_handle():
    class Stream:
        cuda_stream = 0x1230

    assert (cg._stream(Stream()), cg._stream(0x1240), cg._stream(0)) == (0x1230, 0x1240, None)
