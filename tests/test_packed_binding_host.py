"""The packed operators' Python extension without a GPU: arguments are looked at before the device is."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from mla_latent_kv_fp8_gb300 import build
    build.build()
    from mla_latent_kv_fp8_gb300 import _lib
    return _lib


def test_extension_refuses_its_arguments_by_kind(L):
    """What is no tensor or number, and too few or too many arguments: TypeError, on any machine."""
    b = L._bound()
    for f in (b.append_rotated, b.rotate_query, b.gather_latent, b.prefill_ragged):
        for args in ((), ("no tensor",), (3,), (None,) * 30):
            with pytest.raises(TypeError):
                f(*args)


def test_extension_refuses_host_tensors(L):
    """A tensor in host memory is refused as such, without asking for a device."""
    b = L._bound()
    t = torch.zeros((2, 576), dtype=torch.bfloat16)
    for f in (b.append_rotated, b.rotate_query, b.gather_latent, b.prefill_ragged):
        with pytest.raises(L.MlaError, match="CUDA device"):
            f(*[t] * 20)
