"""The attention and sampling calls' argument checks, which need no GPU."""

import ctypes

import pytest

EINVAL, EUNSUPPORTED, OK = -1, -5, 0


@pytest.fixture(scope="module")
def pm():
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def desc(pm, **change):
    d = dict(k=0x10000, v=0x20000, page_stride=2 * 16 * 64, k_scale=0, v_scale=0, num_pages=4, page_size=16, kv_heads=2,
             head_dim=64, dtype=0)
    d.update(change)
    return pm._lib.pmoe_kv_desc(**d)


BAD_CACHES = [
    (dict(k=0), EINVAL), (dict(v=0x20008), EINVAL), (dict(page_stride=2 * 16 * 64 - 8), EINVAL),
    (dict(page_stride=2 * 16 * 64 + 4), EINVAL), (dict(num_pages=0), EINVAL), (dict(kv_heads=0), EINVAL),
    (dict(num_pages=1 << 28), EINVAL), (dict(dtype=1), EINVAL), (dict(dtype=1, k_scale=0x30002, v_scale=0x30000), EINVAL),
    (dict(page_size=8), EUNSUPPORTED), (dict(page_size=24), EUNSUPPORTED), (dict(page_size=512), EUNSUPPORTED),
    (dict(head_dim=96), EUNSUPPORTED), (dict(dtype=2), EUNSUPPORTED),
]


def append(pm, d, **change):
    a = dict(q=0x40000, qs=256, k=0x50000, ks=128, v=0x60000, vs=128, T=3, hq=4, pos=0x70000, axes=1, pa=0, freq=0x80000,
             rot=64, inter=0, qn=0, kn=0, eps=1e-6, slots=0x90000, out=0xa0000, err=0, stream=0)
    a.update(change)
    return pm.load().moe_kv_append(ctypes.byref(d) if d is not None else None, *a.values())


def attend(pm, d, **change):
    a = dict(q=0x40000, qs=256, T=3, hq=4, scale=0.125, pp=0x50000, L=40, pt=0x60000, width=2, seqs=3, rs=0, lens=0x70000,
             S=20, out=0x80000, lse=0, scratch=0, nbytes=0, err=0, stream=0)
    a.update(change)
    return pm.load().moe_prefix_attention(ctypes.byref(d) if d is not None else None, *a.values())


def sample(pm, **change):
    a = dict(x=0x40000, bf16=0, T=2, V=100, stride=100, temp=0, k=0, p=0, m=0, u=0x50000, ids=0x60000, lp=0, stream=0)
    a.update(change)
    return pm.load().moe_sample_tokens(*a.values())


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(pm, change, status):
    d = desc(pm, **change)
    assert append(pm, d) == status
    assert attend(pm, d) == status
    assert pm.load().moe_prefix_attention_scratch_bytes(ctypes.byref(d), 3, 4, 40, 20) == 0


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(hq=0), dict(q=0), dict(k=0), dict(v=0), dict(slots=0), dict(out=0), dict(out=0x40000), dict(pos=0),
    dict(freq=0), dict(rot=24), dict(rot=80), dict(rot=-16), dict(axes=0), dict(axes=9), dict(axes=2), dict(eps=-1.0),
    dict(eps=float("nan")), dict(qs=248), dict(ks=120), dict(vs=132), dict(q=0x40008), dict(qn=0x40002), dict(kn=0x40004),
    dict(pos=0x70001), dict(slots=0x90002), dict(err=0xb0001), dict(out=0xa0008),
])
def test_append_refuses(pm, change):
    assert append(pm, desc(pm), **change) == EINVAL


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(hq=3), dict(hq=0), dict(q=0), dict(out=0), dict(qs=248), dict(qs=260), dict(q=0x40008),
    dict(out=0x80008), dict(L=-1), dict(S=-1), dict(pp=0), dict(pp=0x50002), dict(pt=0), dict(lens=0), dict(width=1),
    dict(seqs=2), dict(rs=0x70000, seqs=0), dict(scale=float("inf")), dict(lse=0x90001), dict(err=0x90002),
    dict(scratch=0x90008), dict(T=1 << 22),
])
def test_attention_refuses(pm, change):
    assert attend(pm, desc(pm), **change) == EINVAL


def test_attention_refuses_large_groups(pm):
    assert attend(pm, desc(pm), hq=130, qs=130 * 64) == EUNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(V=0), dict(V=262145, stride=262145), dict(stride=99), dict(x=0), dict(u=0), dict(ids=0),
    dict(x=0x40002), dict(bf16=1, x=0x40001), dict(temp=0x50001), dict(k=0x50002), dict(p=0x50001), dict(m=0x50002),
    dict(u=0x50001), dict(ids=0x60002), dict(lp=0x60001),
])
def test_sampling_refuses(pm, change):
    assert sample(pm, **change) == EINVAL


def test_nothing_to_do(pm):
    assert append(pm, desc(pm), T=0) == OK
    assert attend(pm, desc(pm), T=0) == OK
    assert sample(pm, T=0) == OK
    assert append(pm, None) == EINVAL and attend(pm, None) == EINVAL
