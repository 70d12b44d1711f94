"""Caches whose tensors have strides of no meaning, those of dimensions of size 1: they are the same
cache, whatever torch keeps there."""

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


def one_head_by_token(x):
    """[pages, 1, page, D] as a view of [pages, page, 1, D]."""
    y = torch.empty_like(x.transpose(1, 2), memory_format=torch.contiguous_format)
    y = y.as_strided(y.shape, (y.shape[1] * y.shape[3], y.shape[3], y.shape[3], 1))
    return y.copy_(x.transpose(1, 2)).transpose(1, 2)


def one_page_of_many(x):
    """[1, heads, page, D] as the middle page of a cache with gaps."""
    wide = torch.zeros((3, x[0].numel() + 64), dtype=x.dtype, device="cuda")
    wide[1, :-64] = x.flatten()
    return wide[:, :-64].unflatten(1, x.shape[1:])[1:2]


def one_page_with_an_odd_stride(x):
    return x.as_strided(x.shape, (5, *x.stride()[1:]))


@pytest.mark.parametrize("shape,view", [((6, 1, 16, 64), one_head_by_token), ((1, 3, 32, 128), one_page_of_many),
                                        ((1, 1, 64, 64), one_page_with_an_odd_stride), ((1, 1, 16, 128), one_head_by_token)])
@pytest.mark.parametrize("which", [(True, True), (False, True), (True, False)])
def test_strides_of_single_dimensions_do_not_matter(pm, shape, view, which):
    pages, heads, page, D = shape
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = new(7, 2 * heads, D), new(7, heads, D), new(7, heads, D)
    slots = torch.arange(7, dtype=torch.int32, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(7, 1)
    lens = torch.arange(7, dtype=torch.int32, device="cuda") + 1
    results = []
    for views in ((False, False), which):
        caches = [view(c) if w else c for c, w in zip((torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
                                                       for _ in range(2)), views)]
        pm.moe_kv_append(*caches, q, k, v, None, slots, None)
        need = pm.moe_prefix_attention_scratch_bytes(*caches, 7, 2 * heads, 0, page)
        scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
        out = pm.moe_prefix_attention(*caches, q, None, 0, table, lens, page, scratch=scratch)
        results.append([*caches, out])
    assert all(torch.equal(a, b) for a, b in zip(*results)) and bool(results[0][0].any())
