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
