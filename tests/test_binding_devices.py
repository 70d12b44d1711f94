"""The devices of a call, without a GPU: tensors on several devices and a stream of another
device are refused before anything of CUDA's is touched (the tensors here have a device but no
memory)."""

import types

import pytest

torch = pytest.importorskip("torch")
fake = pytest.importorskip("torch._subclasses.fake_tensor")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up devices are checked where there are real ones")
BF16, I32, F32 = torch.bfloat16, torch.int32, torch.float32


@pytest.fixture(scope="module")
def pm():
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def at(device, *size, dt):
    with fake.FakeTensorMode():
        return torch.empty(size, dtype=dt, device=device)


APPEND = dict(k_cache=(4, 2, 16, 64, BF16), v_cache=(4, 2, 16, 64, BF16), q=(3, 4, 64, BF16), k=(3, 2, 64, BF16),
              v=(3, 2, 64, BF16), positions=(3, I32), slots=(3, I32), inv_freq=(32, F32), pair_axis=(32, I32),
              q_norm=(64, BF16), k_norm=(64, BF16), k_scale=(2, F32), v_scale=(2, F32), q_out=(3, 4, 64, BF16),
              err_out=(1, I32))
ATTEND = dict(k_cache=(4, 2, 16, 64, BF16), v_cache=(4, 2, 16, 64, BF16), q=(3, 4, 64, BF16), prefix_pages=(2, I32),
              page_table=(3, 1, I32), suffix_len=(3, I32), row_seq=(3, I32), k_scale=(2, F32), v_scale=(2, F32),
              out=(3, 4, 64, BF16), lse_out=(3, 4, F32), scratch=(1 << 20, torch.uint8), err_out=(1, I32))
SAMPLE = dict(logits=(3, 100, F32), u=(3, F32), temperature=(3, F32), top_k=(3, I32), top_p=(3, F32), min_p=(3, F32),
              ids_out=(3, I32), logprob_out=(3, F32))
CALLS = {"moe_kv_append": (APPEND, {}), "moe_prefix_attention": (ATTEND, dict(prefix_len=20, max_suffix=16)),
         "moe_sample_tokens": (SAMPLE, {})}


def args(call, **where):
    tensors, more = CALLS[call]
    made = {n: at(where.get(n, "cuda:0"), *d[:-1], dt=d[-1]) for n, d in tensors.items()}
    return {**made, **more}


@pytest.mark.parametrize("call,name", [(c, n) for c, (d, _) in CALLS.items() for n in list(d)[1:]])
@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
def test_a_tensor_elsewhere_is_refused(pm, call, name, device):
    first = next(iter(CALLS[call][0]))
    with pytest.raises(AssertionError, match=f"{name}: on {device}, {first} on cuda:0"):
        getattr(pm, call)(**args(call, **{name: device}))


@pytest.mark.parametrize("call", list(CALLS))
def test_a_first_tensor_on_the_host_is_refused(pm, call):
    first = next(iter(CALLS[call][0]))
    with pytest.raises(AssertionError, match=f"{first}: not a CUDA tensor"):
        getattr(pm, call)(**args(call, **{first: "cpu"}))


@pytest.mark.parametrize("call", list(CALLS))
def test_a_stream_of_another_device_is_refused(pm, call):
    stream = types.SimpleNamespace(cuda_stream=0, device_index=1)
    with pytest.raises(AssertionError, match="stream: of cuda:1, .* on cuda:0"):
        getattr(pm, call)(**args(call), stream=stream)
