"""The native side of the binding without a GPU: its module objects' own state, and what is refused
before a device is touched."""
import ctypes
import importlib.util

import pytest

from causal_video_diffusion_b200 import binding
from causal_video_diffusion_b200 import build as cuda_build


@pytest.fixture(scope="module")
def host():
    cuda_build.build()
    return cuda_build.build_host()


def load(path):
    spec = importlib.util.spec_from_file_location("_host_calls", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def entry_points():
    return [ctypes.cast(getattr(binding.lib(), n), ctypes.c_void_p).value for n in (
        "unstep_norm_modulate", "unstep_gate_residual_norm", "unstep_q8_rope_kv_append",
        "unstep_q8_window_attn", "unstep_q8_cache_read")]


def test_module_objects_keep_their_own_binding(host):
    """A status becomes the exception that this module object was bound to, whatever another was."""
    class First(binding.UnstepError):
        pass

    class Second(binding.UnstepError):
        pass

    cache = binding.unstep_q8_cache_t()
    at = ctypes.addressof(cache)
    one, two = load(host), load(host)
    one.bind(First, *entry_points())
    two.bind(Second, *entry_points())
    for m, error in ((one, First), (two, Second), (one, First)):
        with pytest.raises(binding.UnstepError) as e:
            m.q8_read(at, 0, 0, 0, None, None, None)          # no frames: refused ahead of the call
        assert type(e.value) is error and e.value.status == binding.UNSTEP_ERR_ARG
    two.bind(First, *entry_points())
    with pytest.raises(First):
        two.q8_read(at, 0, 0, 0, None, None, None)


def test_calls_before_bind_are_refused(host):
    m = load(host)
    for f, n in ((m.norm_modulate, 4), (m.gate_residual_norm, 9), (m.q8_append, 9), (m.q8_attn, 6),
                 (m.q8_read, 7)):
        with pytest.raises(ValueError, match="bind"):
            f(*[None] * n)
    with pytest.raises(TypeError):
        m.bind(RuntimeError)
    with pytest.raises(ValueError):
        m.bind(RuntimeError, 0, 0, 0, 0, 0)


def test_another_torch_or_python_rebuilds(host, monkeypatch):
    """The module built for this torch and Python is kept, and not for others: its next load would
    meet another ABI."""
    import subprocess
    import sys
    import types

    import torch
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return types.SimpleNamespace(returncode=1, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    assert cuda_build.build_host() == host and not ran
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", torch.__version__ + ".1")
        with pytest.raises(RuntimeError):
            cuda_build.build_host()
    with monkeypatch.context() as m:
        m.setattr(sys, "implementation", types.SimpleNamespace(cache_tag="cpython-399"))
        with pytest.raises(RuntimeError):
            cuda_build.build_host()
    assert len(ran) == 2
    assert torch.__version__ in load(host).__doc__
