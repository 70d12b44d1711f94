"""Argument checks of the calls of a step over unequal requests, which need no GPU: at the C entry, and of
the binding's devices (tensors that have a device but no memory)."""

import ctypes
import types

import pytest

from tests.test_serving_abi import BAD_CACHES, desc

EINVAL, EUNSUPPORTED, OK = -1, -5, 0


@pytest.fixture(scope="module")
def pm():
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def tables(pm, **change):
    a = dict(table=0x10000, stride=4, page=16, pages=9, free=0x20000, cap=9, count=0x30000, lens=0x40000, new=0x50000, R=3, T=5,
             lens_out=0x60000, count_out=0x70000, start=0x80000, pos=0x90000, slots=0xa0000, seq=0xb0000, seen=0, err=0, stream=0)
    a.update(change)
    return pm.load().moe_batch_tables(*a.values())


def attend(pm, d, **change):
    a = dict(q=0x40000, qs=256, T=3, hq=4, scale=0.125, start=0x50000, lens=0x60000, R=2, pt=0x70000, width=2, window=0, sinks=0,
             out=0x80000, lse=0, scratch=0, nbytes=0, err=0, stream=0)
    a.update(change)
    return pm.load().moe_chunk_attention(ctypes.byref(d) if d is not None else None, *a.values())


def select(pm, **change):
    a = dict(x=0x10000, bf16=0, T=2, E=64, stride=64, k=4, scoring=0, bias=0, groups=8, top=2, gtop=1, renorm=1, scale=1.0,
             ids=0x20000, w=0x30000, stream=0)
    a.update(change)
    return pm.load().moe_router_select(*a.values())


def adjust(pm, **change):
    a = dict(x=0x10000, bf16=0, T=2, V=100, stride=100, hist=0x20000, hs=8, H=8, pl=0, hl=0x30000, rep=0, freq=0, pres=0,
             bi=0x40000, b=0x50000, B=3, mask=0x60000, ms=4, out=0x70000, obf=0, os=100, err=0, stream=0)
    a.update(change)
    return pm.load().moe_adjust_logits(*a.values())


@pytest.mark.parametrize("change", [
    dict(R=-1), dict(R=8193), dict(T=-1), dict(T=(1 << 24) + 1), dict(stride=0), dict(pages=0), dict(cap=-1), dict(pages=1 << 27),
    dict(table=0), dict(free=0), dict(count=0), dict(lens=0), dict(new=0), dict(lens_out=0), dict(count_out=0), dict(start=0),
    dict(pos=0), dict(slots=0), dict(seq=0), dict(table=0x10002), dict(seen=0x10001), dict(err=0x10001), dict(lens_out=0x50000),
    dict(new=0x40000)])
def test_tables_refuse(pm, change):
    assert tables(pm, **change) == EINVAL


@pytest.mark.parametrize("page", [0, 8, 24, 512])
def test_tables_refuse_page_sizes(pm, page):
    assert tables(pm, page=page) == EUNSUPPORTED


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_attention_refuses_bad_caches(pm, change, status):
    d = desc(pm, **change)
    assert attend(pm, d) == status
    assert pm.load().moe_chunk_attention_scratch_bytes(ctypes.byref(d), 3, 4, 2) == 0


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(R=-1), dict(R=(1 << 20) + 1), dict(hq=3), dict(hq=0), dict(q=0), dict(out=0), dict(qs=248), dict(qs=260),
    dict(q=0x40008), dict(out=0x80008), dict(start=0), dict(lens=0), dict(pt=0), dict(start=0x50002), dict(lens=0x60001),
    dict(pt=0x70002), dict(width=0), dict(width=(1 << 26) + 1), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(lse=0x90001), dict(err=0x90002), dict(scratch=0x90008), dict(T=1 << 22)])
def test_attention_refuses(pm, change):
    assert attend(pm, desc(pm), **change) == EINVAL


def test_attention_refuses_its_queries_as_outputs(pm):
    assert attend(pm, desc(pm), out=0x40000) == EINVAL


def test_attention_refuses_large_groups(pm):
    assert attend(pm, desc(pm), hq=130, qs=130 * 64) == EUNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(E=0), dict(E=1025, stride=1025), dict(stride=63), dict(k=0), dict(k=33), dict(k=17), dict(scoring=2),
    dict(groups=0), dict(groups=7), dict(groups=64), dict(top=0), dict(top=9), dict(gtop=0), dict(gtop=3), dict(scale=float("nan")),
    dict(x=0), dict(x=0x10002), dict(bf16=1, x=0x10001), dict(ids=0), dict(w=0), dict(ids=0x20001), dict(w=0x30002), dict(bias=0x10001)])
def test_selection_refuses(pm, change):
    assert select(pm, **change) == EINVAL


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(V=0), dict(V=262145, stride=262145, os=262145, ms=9000), dict(stride=99), dict(os=99), dict(H=-1),
    dict(H=1 << 19, hs=1 << 19), dict(hs=7), dict(hist=0), dict(hl=0), dict(B=-1), dict(B=4096), dict(bi=0), dict(b=0), dict(ms=3),
    dict(x=0), dict(out=0), dict(x=0x10002), dict(out=0x70002), dict(mask=0x60001), dict(hist=0x20002), dict(rep=0x1), dict(err=0x3),
    dict(out=0x10000, obf=1), dict(out=0x10000, os=104)])
def test_adjusting_refuses(pm, change):
    assert adjust(pm, **change) == EINVAL


def test_nothing_to_do(pm):
    assert attend(pm, desc(pm), T=0) == OK and attend(pm, desc(pm), R=0) == OK and attend(pm, None) == EINVAL
    assert select(pm, T=0) == OK and adjust(pm, T=0) == OK


# ---------------------------------------------------------------------------- devices

torch = pytest.importorskip("torch")
fake = pytest.importorskip("torch._subclasses.fake_tensor")
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up devices are checked where there are real ones")
BF16, I32, F32 = torch.bfloat16, torch.int32, torch.float32

CALLS = {
    "moe_batch_tables": (dict(page_table=(3, 4, I32), free_pages=(9, I32), free_count=(1, I32), lens=(3, I32), new_len=(3, I32),
                              lens_out=(3, I32), free_count_out=(1, I32), q_start=(4, I32), positions=(5, I32), slots=(5, I32),
                              row_seq=(5, I32), row_len=(5, I32), err_out=(1, I32)), dict(T=5, page_size=16, num_pages=9)),
    "moe_chunk_attention": (dict(k_cache=(4, 2, 16, 64, BF16), v_cache=(4, 2, 16, 64, BF16), q=(3, 4, 64, BF16), q_start=(3, I32),
                                 kv_len=(2, I32), page_table=(2, 2, I32), k_scale=(2, F32), v_scale=(2, F32), out=(3, 4, 64, BF16),
                                 lse_out=(3, 4, F32), scratch=(1 << 20, torch.uint8), err_out=(1, I32)), {}),
    "moe_router_select": (dict(logits=(3, 64, F32), bias=(64, F32), ids_out=(3, 4, I32), w_out=(3, 4, F32)), dict(top_k=4)),
    "moe_adjust_logits": (dict(logits=(3, 100, F32), history=(3, 8, I32), prompt_len=(3, I32), history_len=(3, I32),
                               repetition=(3, F32), frequency=(3, F32), presence=(3, F32), bias_ids=(3, 2, I32), bias=(3, 2, F32),
                               mask=(3, 4, I32), out=(3, 100, F32), err_out=(1, I32)), {}),
}


def args(call, **where):
    tensors, more = CALLS[call]
    with fake.FakeTensorMode():
        made = {n: torch.empty(d[:-1], dtype=d[-1], device=where.get(n, "cuda:0")) for n, d in tensors.items()}
    return {**made, **more}


@no_gpu
@pytest.mark.parametrize("call,name", [(c, n) for c, (d, _) in CALLS.items() for n in list(d)[1:]])
@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
def test_a_tensor_elsewhere_is_refused(pm, call, name, device):
    first = next(iter(CALLS[call][0]))
    with pytest.raises(AssertionError, match=f"{name}: on {device}, {first} on cuda:0"):
        getattr(pm, call)(**args(call, **{name: device}))


@no_gpu
@pytest.mark.parametrize("call", list(CALLS))
def test_a_first_tensor_on_the_host_and_another_devices_stream_are_refused(pm, call):
    first = next(iter(CALLS[call][0]))
    with pytest.raises(AssertionError, match=f"{first}: not a CUDA tensor"):
        getattr(pm, call)(**args(call, **{first: "cpu"}))
    with pytest.raises(AssertionError, match="stream: of cuda:1, .* on cuda:0"):
        getattr(pm, call)(**args(call), stream=types.SimpleNamespace(cuda_stream=0, device_index=1))
