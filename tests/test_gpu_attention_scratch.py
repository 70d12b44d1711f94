"""One scratch buffer for a batch that shrinks: the size for its largest call serves every smaller
one, with the same bits as scratch of its own."""

import pytest

from tests.test_gpu_prefix_attention import make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


@pytest.mark.parametrize("T,Hq,Hkv,D,e4m3,prefix,suffix", [(8, 32, 4, 128, False, 60000, 100), (256, 32, 4, 128, False, 1000, 64),
                                                           (40, 16, 1, 64, True, 9000, 700)])
def test_one_buffer_for_all_smaller_calls(pm, T, Hq, Hkv, D, e4m3, prefix, suffix):
    c = make(T + prefix, T, Hq, Hkv, D, 16, e4m3, prefix, suffix)
    up = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    pages, table, lens = up(c["pp"]), up(c["pt"]), up(c["lens"])
    scratch = torch.empty(pm.moe_prefix_attention_scratch_bytes(c["k"], c["v"], T, Hq, prefix, suffix), dtype=torch.uint8,
                          device="cuda")

    def call(t, p, s, **more):
        return pm.moe_prefix_attention(c["k"], c["v"], c["q"][:t], pages, p, table, lens[:t].clamp(max=s), s,
                                       k_scale=c["ks"], v_scale=c["vs"], **more)

    for t in sorted({1, 2, 3, 4, 5, T // 6, T // 2, T - 42 if T > 42 else 1, T - 1, T} - {0}):
        for p, s in ((prefix, suffix), (prefix // 2, suffix), (0, suffix), (prefix, 1), (prefix // 7, 0)):
            assert torch.equal(call(t, p, s, scratch=scratch), call(t, p, s)), (t, p, s)
