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


class Event:
    cuda_event = 1


@pytest.mark.parametrize("events", [None, (Event(), Event())])
@pytest.mark.parametrize("bad", [dict(num_ctas=2 ** 32 + 7), dict(num_ctas=2 ** 32), dict(num_ctas=-2 ** 32 + 7), dict(k_scale=1e-46),
                                 dict(v_scale=1e-46), dict(k_scale=-1e-46)])
def test_options_that_the_library_would_read_as_others(fd, monkeypatch, events, bad):
    """2^32 + 7 CTAs as 7, and a scale that fp32 does not hold as 0, which stands for 1."""
    with pytest.raises(ValueError):
        attend(fd, monkeypatch, split_events=events, **bad)
    for good in (dict(k_scale=1e-45), dict(v_scale=0.0), dict(num_ctas=160)):   # 1e-45: fp32's least number
        attend(fd, monkeypatch, split_events=events, **good)


def test_row_scales_that_fp32_does_not_hold(fd, monkeypatch):
    from decode_attention_decoding_gb300 import longcontext
    with pytest.raises(ValueError):
        longcontext._opts(0, 0, 0, 1e-50, 1.0, 1)
    with pytest.raises(ValueError):
        longcontext._opts(0, 0, 0, 1.0, 1e-50, 1)


@pytest.mark.parametrize("shape", [(2 ** 32 + 1, 8, 8, 128, 1), (1, 2 ** 32 + 8, 8, 128, 1), (1, 8, 2 ** 32 + 8, 128, 1),
                                   (1, 8, 8, 2 ** 32 + 128, 1), (1, 8, 8, 128, 2 ** 32 + 1), (-2 ** 32 + 1, 8, 8, 128, 1)])
def test_workspaces_of_shapes_that_no_call_accepts(fd, shape):
    assert fd.fd_window_workspace_size(*shape) == 0
    with pytest.raises(fd.FdError):
        fd.make_window_workspace(*shape[:4], q_len=shape[4])
