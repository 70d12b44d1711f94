"""The calls of a step over requests where their paths meet: attention segments of every kind
in one CTA's run, maxima that grow from tile to tile, two captured graphs at once, and a whole
step captured and replayed while requests come and end.

Attention's tolerance is that of test_gpu_chunk_attention; all else is equal bits or whole numbers.
"""

import numpy as np
import pytest

from tests import test_gpu_batch_tables as tables
from tests import test_gpu_router_select as selection
from tests.test_gpu_chunk_attention import check, make, poison_unseen, run, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


KINDS = [(64, False), (128, False), (64, True), (128, True)]


@pytest.mark.parametrize("D,e4m3", KINDS)
@pytest.mark.parametrize("fall", [False, True])
def test_maxima_that_move_with_every_tile(pm, D, e4m3, fall):
    """Keys that grow (or fall) along a request by 2^12 over 3,000 keys: few rows, one query tile, two."""
    c = make(D + e4m3, [1, 1, 3, 40, 200], [3000, 2950, 700, 1500, 1300], 8, 2, D, 32, e4m3, qscale=4.0)
    for r, n in enumerate(c["lens"]):
        for i in range(-(-int(n) // 32)):
            at = c["table"][r][i]
            j = torch.arange(i * 32, i * 32 + 32, device="cuda") / 3000
            ramp = torch.exp2(12 * (1 - j if fall else j) - 10)[:, None]
            x = (c["k"][at].float() * ramp).clamp(-448, 448)
            c["k"][at] = x.to(c["k"].dtype)
    out, lse = run(pm, c)
    check(c, out, lse)


@pytest.mark.parametrize("D,e4m3", KINDS)
@pytest.mark.parametrize("window,sinks,page", [(0, 0, 64), (300, 5, 16), (130, 200, 128)])
def test_segments_of_all_kinds_in_one_run(pm, D, e4m3, window, sinks, page):
    """Far more items than CTAs, of one query tile and of two, of one key tile and of many, in any order."""
    rng = np.random.default_rng(D + window + e4m3)
    news = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 9, 33, 70], 200)]
    lens = [n + int(x) for n, x in zip(news, rng.choice([0, 5, 120, 130, 250, 260, 400, 700, 1200], 200))]
    c = make(9, news, lens, 16, 4, D, page, e4m3, window, sinks, pad=3)
    poison_unseen(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(pm, c, err_out=err)
    assert int(err) == 0
    check(c, out, lse)


@pytest.mark.parametrize("D,e4m3", KINDS)
def test_values_that_are_not_finite_in_any_tile(pm, D, e4m3):
    """One NaN value far back, in a tile that all rows see: every row that sees it has it, in its column alone."""
    c = make(12, [1, 20, 150], [900, 1000, 700], 8, 2, D, 16, e4m3)
    want, _ = run(pm, c)
    for r in range(3):
        page = c["table"][r][100 // 16]
        (c["v"].view(torch.uint8) if e4m3 else c["v"])[page, 1, 100 % 16, 7] = 0x7f if e4m3 else float("nan")
    got, _ = run(pm, c)
    hit = torch.zeros_like(want, dtype=torch.bool)
    hit[:, 4:, 7] = True
    assert torch.all(torch.isnan(got[hit])) and torch.equal(got[~hit], want[~hit])


def test_two_captured_graphs_at_once(pm):
    """Each call of a captured graph has scratch of its own, whether two graphs run at once or in turn."""
    cases = [make(21, [1] * 30, [900] * 30, 16, 2, 64, 16, False), make(22, [300, 1, 90], [2000, 700, 95], 16, 2, 64, 16, False)]
    want = [run(pm, c)[0] for c in cases]
    held, graphs, streams, keep = [torch.zeros_like(w) for w in want], [], [torch.cuda.Stream(), torch.cuda.Stream()], []
    for c, out in zip(cases, held):
        args = (c["k"], c["v"], c["q"], up(c["start"]), up(c["lens"]), up(c["table"]))
        keep.append(args)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pm.moe_chunk_attention(*args, out=out)
        graphs.append(g)
    for _ in range(20):
        for out in held:
            out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


class Step:
    """A step of all calls on its own state; every row is padded to a fixed count."""

    R, T, page, pages, width, Hq, Hkv, D, E, V = 6, 96, 16, 60, 20, 8, 2, 64, 32, 3001

    def __init__(self, pm):
        self.pm = pm
        g = torch.Generator(device="cuda").manual_seed(5)
        i32 = dict(dtype=torch.int32, device="cuda")
        n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.table = torch.zeros((self.R, self.width), **i32)
        self.free, self.count = torch.arange(self.pages, **i32), torch.tensor([self.pages], **i32)
        self.lens, self.new = torch.zeros(self.R, **i32), torch.zeros(self.R, **i32)
        self.k, self.v = (torch.zeros((self.pages, self.Hkv, self.page, self.D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.qkv = torch.zeros((self.T, (self.Hq + 2 * self.Hkv) * self.D), dtype=torch.bfloat16, device="cuda")
        self.inv_freq = 10000.0 ** (-torch.arange(0, self.D, 2, device="cuda") / self.D)
        self.route, self.head = n(self.Hq * self.D, self.E) * 0.05, n(self.Hq * self.D, self.V) * 0.05
        self.bias, self.u = n(self.E) * 0.05, torch.rand(self.T, generator=g, device="cuda")
        self.history = torch.zeros((self.T, 8), **i32)
        self.history_len = torch.full((self.T,), 8, **i32)
        self.repetition = torch.full((self.T,), 1.3, device="cuda")
        self.err = torch.zeros(1, **i32)
        self.out = torch.zeros((self.T, self.Hq, self.D), dtype=torch.bfloat16, device="cuda")

    def __call__(self):
        pm = self.pm
        t = pm.moe_batch_tables(self.table, self.free, self.count, self.lens, self.new, self.T, self.page, self.pages,
                                lens_out=self.lens, free_count_out=self.count, err_out=self.err)
        q, k, v = self.qkv.view(self.T, -1, self.D).split([self.Hq, self.Hkv, self.Hkv], dim=1)
        q = pm.moe_kv_append(self.k, self.v, q, k, v, t.positions, t.slots, self.inv_freq, err_out=self.err)
        self.out.zero_()
        pm.moe_chunk_attention(self.k, self.v, q, t.q_start, t.lens, self.table, out=self.out, err_out=self.err)
        x = self.out.view(self.T, -1).float()
        ids, w = pm.moe_router_select(x @ self.route, 4, scoring="sigmoid", bias=self.bias, groups=4, top_groups=2)
        logits = pm.moe_adjust_logits(x @ self.head, history=self.history, history_len=self.history_len,
                                      repetition=self.repetition, err_out=self.err)
        self.result = (t.positions, t.slots, t.row_seq, self.lens, self.count, self.table, self.out, ids, w, logits,
                       pm.moe_sample_tokens(logits, self.u))


def test_a_captured_step_follows_requests_that_come_and_end(pm):
    eager, captured = Step(pm), Step(pm)
    captured()  # (a step of nothing, so that all is set up)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    rng = np.random.default_rng(1)
    live = np.zeros(Step.R, bool)
    for _ in range(12):
        new = np.where(live, rng.choice([-1, 0, 1, 1, 1, 13], Step.R), rng.choice([0, 20, 33], Step.R))
        while new[new > 0].sum() > Step.T:
            new[rng.integers(Step.R)] = 0
        inputs = torch.randn((Step.T, eager.qkv.shape[1]), device="cuda").to(torch.bfloat16)
        history = torch.randint(0, Step.V, (Step.T, 8), device="cuda", dtype=torch.int32)
        for s in (eager, captured):
            s.new.copy_(up(new.astype(np.int32)))
            s.qkv.copy_(inputs)
            s.history.copy_(history)
        eager()
        graph.replay()
        torch.cuda.synchronize()
        assert int(eager.err) == 0 and int(captured.err) == 0
        assert all(torch.equal(a, b) for a, b in zip(eager.result, captured.result))
        now = eager.lens.cpu().numpy()
        live = now > 0
        assert live.any()


@pytest.mark.parametrize("R,T,page,most", [(40, 50, 16, 9000), (1500, 4000, 16, 700), (3000, 40, 256, 3000)])
def test_long_requests_end_together(pm, R, T, page, most):
    """Hundreds of pages come back from one request, from requests of several turns of the block."""
    c = tables.make(R, R, T, page, 2, most, done=0.5)
    got, err = tables.run(pm, c)
    tables.check(c, got, err)


def test_a_stack_without_room_for_what_comes_back(pm):
    """Pages beyond the stack's capacity are lost and reported; the ones that fit are where they belong."""
    c = tables.make(3, 30, 40, 16, 3, 900, done=1.0, rest=0.0, spare=0)
    whole = c["free"].size
    c["free"] = c["free"][:whole // 2].copy()
    got, err = tables.run(pm, c)
    have = -(-c["lens"] // 16)
    back = np.concatenate([c["table"][r, :have[r]] for r in range(30)])
    assert err == 128 and int(got[3]) == whole // 2
    assert np.array_equal(got[1].cpu().numpy(), back[:whole // 2])


@pytest.mark.parametrize("E,groups,top_groups,k", [(96, 1, 1, 5), (96, 8, 3, 7), (160, 8, 3, 8), (160, 4, 2, 6), (192, 6, 2, 10),
                                                   (192, 32, 9, 8), (384, 1, 1, 32), (384, 12, 4, 6), (512, 16, 4, 8), (1024, 32, 8, 32)])
@pytest.mark.parametrize("bf16", [False, True])
def test_selection_with_any_share_of_a_lane(pm, E, groups, top_groups, k, bf16):
    """Experts a lane 3, 5, 6, 12, 16 and 32, in groups of whole lanes and of others; rows aligned or not."""
    g = torch.Generator(device="cuda").manual_seed(E + groups)
    T = 700
    wide = torch.randn((T, E + 8), generator=g, device="cuda").to(torch.bfloat16 if bf16 else torch.float32)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    for logits in (wide[:, :E].contiguous(), wide[:, 1:E + 1]):
        for scoring in ("sigmoid", "softmax"):
            selection.check(pm, logits, k, scoring, bias, groups, top_groups, 2)
