"""Numbers that the C types of the 4-bit cache and window calls do not hold: ctypes would pass other ones."""
import pytest
import torch


@pytest.fixture(scope="module")
def fd():
    from decode_attention_decoding_gb300 import build
    build.build()
    import decode_attention_decoding_gb300 as fd
    return fd


def attend(fd, monkeypatch, window=8, sinks=0, status=0, **kw):
    """The binding's common part on CPU tensors: the arguments that the library would get."""
    from decode_attention_decoding_gb300 import longcontext
    got = []
    monkeypatch.setattr(longcontext, "_call", lambda gpu, f, *a: got.append(a) or status)
    args = dict(seq_lens_host=None, scale=None, out=None, lse=None, workspace=torch.zeros(256, dtype=torch.uint8), num_ctas=0,
                split_events=None, check=True, kv=0, k_scale=1.0, v_scale=1.0)
    args.update(kw)
    longcontext._attend("f", None, torch.zeros(1, 8, 64, dtype=torch.bfloat16), -1, (0, 0), 1, 16, 8, None, None, window, sinks, **args)
    return got[0]


@pytest.mark.parametrize("window,sinks", [(-2 ** 32 + 5, 0), (5, -2 ** 32 + 1), (-2 ** 31 - 1, 0), (-2 ** 40, -2 ** 40)])
def test_negative_windows_that_an_int_does_not_hold(fd, monkeypatch, window, sinks):
    """Their low 32 bits may be a window."""
    with pytest.raises(ValueError, match="2\\^31"):
        attend(fd, monkeypatch, window, sinks)


@pytest.mark.parametrize("window,sinks", [(-1, 0), (8, -1), (-2 ** 31, -2 ** 31)])
def test_other_negative_windows_are_the_library_s_to_refuse(fd, monkeypatch, window, sinks):
    with pytest.raises(fd.FdError):
        attend(fd, monkeypatch, window, sinks, status=fd.FD_ERR_INVALID_ARG)
    a = attend(fd, monkeypatch, window, sinks)
    assert (window, sinks) in zip(a, a[1:])
    a = attend(fd, monkeypatch, 2 ** 31 - 1, 2 ** 31 - 1)
    assert (2 ** 31 - 1,) * 2 in zip(a, a[1:])
