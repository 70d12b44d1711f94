"""moe_batch_tables against the oracle: whole numbers, so every one is equal."""

import numpy as np
import pytest

from oracle import steps

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def make(seed, R, T, page, chunk=3, most=200, spare=None, width=None, done=0.2, rest=0.2, dtype=np.int32):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most + 1, R)
    new = np.where(rng.random(R) < 0.3, rng.integers(1, chunk + 1, R), 1)
    u = rng.random(R)
    new[u < rest] = 0
    new[(u >= rest) & (u < rest + done)] = -1
    have = -(-lens // page)
    width = width or int(-(-(most + chunk) // page))
    lens = np.minimum(lens, width * page)
    have = -(-lens // page)
    total = int(have.sum())
    spare = total + R * (chunk // page + 1) if spare is None else spare
    pages = total + spare
    order = rng.permutation(pages).astype(dtype)
    table = np.full((R, width), -9, dtype)
    at = 0
    for r in range(R):
        table[r, :have[r]] = order[at:at + have[r]]
        at += have[r]
    free = np.full(pages, -5, dtype)
    free[:spare] = order[total:]
    return dict(table=table, free=free, count=spare, lens=lens.astype(dtype), new=new.astype(dtype), T=T, page=page, pages=pages)


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(pm, c, in_place=False, **more):
    table, free, count, lens = up(c["table"]), up(c["free"]), up(np.array([c["count"]], np.int32)), up(c["lens"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if in_place:
        more.update(lens_out=lens, free_count_out=count)
    r = pm.moe_batch_tables(table, free, count, lens, up(c["new"]), c["T"], c["page"], c["pages"], err_out=err, **more)
    torch.cuda.synchronize()
    return [table, free, *r], int(err)


def check(c, got, err):
    want = steps.batch_tables(c["table"], c["free"], c["count"], c["lens"], c["new"], c["T"], c["page"], c["pages"])
    table, free, lens, count, start, positions, slots, row_seq, row_len = [x.cpu().numpy() for x in got]
    for name, a, b in (("table", table, want[0]), ("free", free, want[1]), ("lens", lens, want[3]), ("q_start", start, want[4]),
                       ("positions", positions, want[5]), ("slots", slots, want[6]), ("row_seq", row_seq, want[7]),
                       ("row_len", row_len, want[8])):
        assert np.array_equal(a, b), name
    assert int(count[0]) == want[2]
    assert err == (256 if want[9].any() else 0)
    return want


@pytest.mark.parametrize("R,T,page,chunk,most", [
    (1, 1, 16, 1, 0), (1, 5, 16, 3, 40), (3, 20, 32, 4, 100), (40, 60, 16, 3, 90), (256, 256, 64, 1, 500),
    (256, 300, 256, 2, 2000), (1000, 3000, 16, 9, 200), (1025, 5000, 128, 9, 3000), (2500, 9000, 16, 5, 50),
    (8192, 10000, 16, 2, 60), (5, 20000, 64, 6000, 1000), (1, 30000, 16, 30000, 3), (70, 2047, 32, 60, 100)])
def test_tables_match_oracle(pm, R, T, page, chunk, most):
    c = make(R + T, R, T, page, chunk, most)
    got, err = run(pm, c)
    check(c, got, err)
    inside, err2 = run(pm, c, in_place=True)
    assert err == err2 and all(torch.equal(a, b) for a, b in zip(got, inside))


def test_too_few_pages(pm):
    """Requests are served in order until the pages run out; from there on those that need none."""
    for spare in (0, 1, 4, 7):
        c = make(3, 60, 400, 16, 20, 100, spare=spare, done=0.0)
        got, err = run(pm, c)
        want = check(c, got, err)
        assert want[9].any() and (want[6] >= 0).any()


def test_too_few_rows_and_entries(pm):
    c = make(4, 60, 25, 16, 20, 100)
    got, err = run(pm, c)
    assert check(c, got, err)[9].any()
    c = make(5, 60, 600, 16, 40, 100, width=5)
    got, err = run(pm, c)
    assert check(c, got, err)[9].any()


def test_pages_of_ended_requests_serve_the_same_step(pm):
    c = make(6, 30, 200, 16, 40, 60, spare=0, done=0.6, rest=0.0)
    got, err = run(pm, c)
    want = check(c, got, err)
    assert (want[6] >= 0).any()


def test_empty_steps(pm):
    for new in (0, -1):
        c = make(7, 20, 8, 16, 3, 100)
        c["new"][:] = new
        got, err = run(pm, c)
        check(c, got, err)
    c = make(8, 4, 0, 16, 3, 100)
    c["new"][:] = 0
    got, err = run(pm, c)
    check(c, got, err)
    c = make(9, 1, 7, 16, 3, 50)
    c.update(table=c["table"][:0], lens=c["lens"][:0], new=c["new"][:0])
    got, err = run(pm, c)
    assert got[6].tolist() == [-1] * 7 and got[4].tolist() == [0] and int(got[3]) == c["count"] and err == 0


def test_a_run_of_steps_loses_no_page(pm):
    """Requests that come, grow and end over many steps, in place: pages are never shared nor lost."""
    rng = np.random.default_rng(2)
    R, page, width, pages, T = 12, 16, 9, 70, 64
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    free = up(rng.permutation(pages).astype(np.int32))
    count = up(np.array([pages], np.int32))
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    live = np.zeros(R, bool)
    for _ in range(60):
        new = np.where(live, np.where(rng.random(R) < 0.1, -1, rng.integers(0, 9, R)), rng.choice([0, 25], R))
        pm.moe_batch_tables(table, free, count, lens, up(new.astype(np.int32)), T, page, pages, lens_out=lens, free_count_out=count)
        now, n = lens.cpu().numpy(), int(count)
        live = now > 0
        held = [int(p) for r in range(R) for p in table[r, :-(-int(now[r]) // page)].tolist()]
        assert sorted(held + free[:n].tolist()) == list(range(pages))


def test_bad_inputs_are_reported(pm):
    c = make(10, 6, 20, 16, 3, 60, done=0.0, rest=0.0)
    for name, at, value, bit in (("lens", 2, -3, 128), ("lens", 2, 1 << 20, 128), ("new", 2, -2, 128), ("free", slice(None), 1 << 20, 64)):
        bad = {k: (x.copy() if isinstance(x, np.ndarray) else x) for k, x in c.items()}
        bad[name][at] = value
        if name == "free":
            bad["new"][:] = 17
            bad["T"] = 200
        got, err = run(pm, bad)
        assert err & bit
        slots = got[6].cpu().numpy()
        assert slots.max() < c["pages"] * 16 and slots.min() >= -1
    for count in (-1, c["pages"] + 1):
        got, err = run(pm, {**c, "count": count})
        assert err & 128
    full = make(11, 6, 20, 16, 3, 60, done=1.0, rest=0.0)  # a stack without room for what comes back
    got, err = run(pm, {**full, "count": full["pages"]})
    assert err == 128 and int(got[3]) == full["pages"]


def test_graph_replay_with_other_lengths(pm):
    c = make(12, 50, 120, 16, 5, 100)
    table, free, count, lens, new = up(c["table"]), up(c["free"]), up(np.array([c["count"]], np.int32)), up(c["lens"]), up(c["new"])
    g = torch.cuda.CUDAGraph()
    outs = None
    pm.moe_batch_tables(table.clone(), free.clone(), count, lens, new, 120, 16, c["pages"])
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        outs = pm.moe_batch_tables(table, free, count, lens, new, 120, 16, c["pages"])
    g.replay()
    torch.cuda.synchronize()
    check(c, [table, free, *outs], 256 if steps.batch_tables(c["table"], c["free"], c["count"], c["lens"], c["new"], 120, 16,
                                                             c["pages"])[9].any() else 0)
    new.fill_(1)
    table.copy_(up(c["table"])), free.copy_(up(c["free"]))
    g.replay()
    torch.cuda.synchronize()
    c["new"][:] = 1
    check(c, [table, free, *outs], 0)


def test_refusals(pm):
    c = make(13, 3, 9, 16)
    a = dict(page_table=up(c["table"]), free_pages=up(c["free"]), free_count=up(np.array([1], np.int32)), lens=up(c["lens"]),
             new_len=up(c["new"]), T=9, page_size=16, num_pages=c["pages"])
    for change, status in ((dict(page_size=24), pm.PMOE_EUNSUPPORTED), (dict(T=-1), None), (dict(num_pages=0), pm.PMOE_EINVAL),
                           (dict(lens_out=a["new_len"]), pm.PMOE_EINVAL)):
        with pytest.raises((pm.PmoeError, RuntimeError)) as e:
            pm.moe_batch_tables(**{**a, **change})
        assert status is None or e.value.status == status
    for change, name in ((dict(lens=a["lens"][:2]), "lens"), (dict(new_len=a["new_len"].long()), "new_len"),
                         (dict(page_table=a["page_table"].t()), "page_table"), (dict(slots=a["lens"]), "slots")):
        with pytest.raises(AssertionError, match=name):
            pm.moe_batch_tables(**{**a, **change})
