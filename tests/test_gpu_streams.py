"""Streams of the decode-step calls: torch's, and objects that only have a handle."""

import types

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def test_a_stream_that_only_has_a_handle(pm):
    x = torch.randn((3, 1000), device="cuda")
    u = torch.rand(3, device="cuda")
    want = pm.moe_sample_tokens(x, u)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for s in (stream, torch.cuda.ExternalStream(stream.cuda_stream), types.SimpleNamespace(cuda_stream=stream.cuda_stream)):
        ids = torch.full((3,), -1, dtype=torch.int32, device="cuda")
        stream.wait_stream(torch.cuda.current_stream())
        pm.moe_sample_tokens(x, u, ids_out=ids, stream=s)
        stream.synchronize()
        assert torch.equal(ids, want)


def test_a_stream_without_a_handle_is_an_error(pm):
    x, u, ids = torch.zeros((1, 8), device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(AttributeError):
        pm.moe_sample_tokens(x, u, ids_out=ids, stream=object())
