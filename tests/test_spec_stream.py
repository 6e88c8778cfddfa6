"""The `stream` argument of the speculative-decoding calls (CPU)."""
import contextlib
import types

import pytest
import torch


@pytest.fixture(scope="module")
def fd():
    from decode_attention_decoding_gb300 import build
    build.build()
    import decode_attention_decoding_gb300 as fd
    return fd


class FakeTensor:
    """Says which GPU it is on; any other use is an AttributeError."""
    def get_device(self):
        return 0


@pytest.mark.parametrize("name,n", [("fd_build_tables", 8), ("fd_cache_write", 5), ("fd_cache_compact", 6), ("fd_tree_decode", 3),
                                    ("fd_tree_decode_paged", 5)])
def test_a_stream_of_another_gpu_is_refused(fd, monkeypatch, name, n):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        getattr(fd, name)(*[FakeTensor()] * n, stream=stream)
