"""The readme's example of a step over requests, run as it stands."""

import os
import re

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example(word):
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    found = [b for b in blocks if word in b]
    assert len(found) == 1
    return found[0]


def test_names_of_the_tables():
    import paged_expert_moe_gb300 as pm
    named = set(re.findall(r"\bbt\.(\w+)", example("moe_batch_tables")))
    assert named and named <= set(pm.BatchTables._fields)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
def test_step_over_requests():
    """Two requests with a piece of a prompt, one that generates, one that rests, one that has ended."""
    import paged_expert_moe_gb300 as pm
    g = torch.Generator(device="cuda").manual_seed(0)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    R, T, page_size, num_pages, Hq, Hkv, D, E, V = 5, 64, 16, 40, 8, 2, 64, 64, 1000
    lens = ints(0, 20, 33, 5, 40)
    page_table = torch.zeros((R, 8), dtype=torch.int32, device="cuda")
    at = 0
    for r, have in enumerate((0, 2, 3, 1, 3)):
        page_table[r, :have] = torch.arange(at, at + have)
        at += have
    free_pages = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    free_pages[:num_pages - at] = torch.arange(at, num_pages)
    k_cache, v_cache = (n(num_pages, Hkv, page_size, D).bfloat16() for _ in range(2))
    q, k, v = n(T, Hq + 2 * Hkv, D).bfloat16().split([Hq, Hkv, Hkv], dim=1)
    names = dict(pm=pm, page_table=page_table, free_pages=free_pages, free_count=ints(num_pages - at), lens=lens,
                 new_len=ints(30, 20, 1, 0, -1), T=T, page_size=page_size, num_pages=num_pages, k_cache=k_cache,
                 v_cache=v_cache, q=q, k=k, v=v, inv_freq=1e4 ** (-torch.arange(0, D, 2, device="cuda") / D), logits=n(T, E),
                 b=n(E) * 0.1, l=n(R, V), h=torch.randint(0, V, (R, 12), generator=g, device="cuda", dtype=torch.int32),
                 pl=ints(0, 1, 2, 3, 4), hl=ints(0, 5, 12, 3, 9), r=torch.full((R,), 1.2, device="cuda"),
                 m=torch.full((R, -(-V // 32)), -1, dtype=torch.int32, device="cuda"))
    exec(compile(example("moe_batch_tables"), "README.md", "exec"), names)
    assert names["bt"].lens.tolist() == [30, 40, 34, 5, 0] and names["bt"].q_start.tolist() == [0, 30, 50, 51, 51, 51]
    assert torch.isfinite(names["o"][:51]).all() and names["ids"].shape == (T, 8) and names["l"].shape == (R, V)
