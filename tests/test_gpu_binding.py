"""What the binding of moe_kv_append, moe_prefix_attention and moe_sample_tokens refuses: tensors
of another type, shape, layout or place raise AssertionError before anything is launched; what
only the library sees raises PmoeError with its status."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def pm():
    import paged_expert_moe_gb300 as pm
    return pm


def zeros(*size, dt=torch.bfloat16):
    return torch.zeros(size, dtype=dt, device="cuda")


def append_args(**change):
    a = dict(k_cache=zeros(4, 2, 16, 64), v_cache=zeros(4, 2, 16, 64), q=zeros(3, 4, 64), k=zeros(3, 2, 64), v=zeros(3, 2, 64),
             positions=zeros(3, dt=torch.int32), slots=zeros(3, dt=torch.int32), inv_freq=zeros(32, dt=torch.float32))
    a.update(change)
    return a


def attend_args(**change):
    a = dict(k_cache=zeros(4, 2, 16, 64), v_cache=zeros(4, 2, 16, 64), q=zeros(3, 4, 64), prefix_pages=zeros(2, dt=torch.int32),
             prefix_len=20, page_table=zeros(3, 1, dt=torch.int32), suffix_len=zeros(3, dt=torch.int32), max_suffix=16)
    a.update(change)
    return a


def sample_args(**change):
    a = dict(logits=zeros(3, 100, dt=torch.float32), u=zeros(3, dt=torch.float32))
    a.update(change)
    return a


I32, F32, E4M3 = torch.int32, torch.float32, torch.float8_e4m3fn

CACHES = [
    dict(k_cache=lambda: zeros(4, 2, 16, 64, dt=F32)), dict(v_cache=lambda: zeros(4, 2, 16, 64, dt=E4M3)),
    dict(v_cache=lambda: zeros(5, 2, 16, 64)), dict(k_cache=lambda: zeros(4, 16, 64)),
    dict(k_cache=lambda: zeros(4, 2, 16, 64).transpose(1, 2), v_cache=lambda: zeros(4, 2, 16, 64).transpose(1, 2)),
    dict(k_cache=lambda: zeros(4, 2, 16, 64, dt=E4M3), v_cache=lambda: zeros(4, 2, 16, 64, dt=E4M3)),  # no scales
    dict(k_cache=lambda: torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)),  # on the host
]


def made(change):
    return {k: f() if callable(f) else f for k, f in change.items()}


@pytest.mark.parametrize("change", CACHES + [
    dict(q=lambda: zeros(3, 4, 64, dt=F32)), dict(q=lambda: zeros(3, 4, 128)), dict(q=lambda: zeros(3, 64)),
    dict(k=lambda: zeros(2, 2, 64)), dict(v=lambda: zeros(3, 3, 64)), dict(k=lambda: zeros(3, 2, 128)[..., ::2]),
    dict(positions=lambda: zeros(3, dt=torch.int64)), dict(positions=lambda: zeros(2, dt=I32)),
    dict(slots=lambda: zeros(4, dt=I32)), dict(slots=lambda: zeros(6, dt=I32)[::2]), dict(inv_freq=lambda: zeros(32)),
    dict(pair_axis=lambda: zeros(16, dt=I32)), dict(q_norm=lambda: zeros(32)), dict(k_norm=lambda: zeros(64, dt=F32)),
    dict(q_out=lambda: zeros(3, 4, 32)), dict(err_out=lambda: zeros(1, dt=F32)),
])
def test_append_refuses(pm, change):
    pm.moe_kv_append(**append_args())
    with pytest.raises(AssertionError):
        pm.moe_kv_append(**append_args(**made(change)))


@pytest.mark.parametrize("change", CACHES + [
    dict(q=lambda: zeros(3, 4, 64, dt=F32)), dict(q=lambda: zeros(3, 4, 128)), dict(prefix_pages=lambda: zeros(1, dt=I32)),
    dict(prefix_pages=lambda: zeros(2, dt=torch.int64)), dict(page_table=lambda: zeros(3, dt=I32)),
    dict(page_table=lambda: zeros(3, 2, dt=I32)[:, :1]), dict(suffix_len=lambda: zeros(2, dt=I32)),
    dict(row_seq=lambda: zeros(4, dt=I32)), dict(out=lambda: zeros(3, 4, 64, dt=F32)), dict(out=lambda: zeros(3, 2, 64)),
    dict(lse_out=lambda: zeros(3, dt=F32)), dict(scratch=lambda: zeros(1 << 20, dt=F32)), dict(prefix_len=1 << 40),
])
def test_attention_refuses(pm, change):
    pm.moe_prefix_attention(**attend_args())
    with pytest.raises(AssertionError):
        pm.moe_prefix_attention(**attend_args(**made(change)))


@pytest.mark.parametrize("change", [
    dict(logits=lambda: zeros(3, 100, dt=torch.float16)), dict(logits=lambda: zeros(100, dt=F32)),
    dict(logits=lambda: zeros(100, 3, dt=F32).T), dict(logits=lambda: torch.zeros(3, 100)), dict(u=None),
    dict(u=lambda: zeros(2, dt=F32)), dict(u=lambda: zeros(3, dt=torch.float64)), dict(temperature=lambda: zeros(1, dt=F32)),
    dict(top_k=lambda: zeros(3, dt=torch.int64)), dict(top_p=lambda: zeros(3)), dict(min_p=lambda: zeros(6, dt=F32)[::2]),
    dict(ids_out=lambda: zeros(3, dt=torch.int64)), dict(logprob_out=lambda: zeros(3, 1)),
])
def test_sampling_refuses(pm, change):
    pm.moe_sample_tokens(**sample_args())
    with pytest.raises(AssertionError):
        pm.moe_sample_tokens(**sample_args(**made(change)))


def test_statuses_of_the_library_are_raised(pm):
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_prefix_attention(**attend_args(scratch=zeros(16, dt=torch.uint8)))
    assert e.value.status == pm.PMOE_EINVAL
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_kv_append(**append_args(inv_freq=zeros(12, dt=F32)))  # rotary_dim 24
    assert e.value.status == pm.PMOE_EINVAL
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_sample_tokens(zeros(1, 262145, dt=F32), zeros(1, dt=F32))
    assert e.value.status == pm.PMOE_EINVAL
    torch.cuda.synchronize()
