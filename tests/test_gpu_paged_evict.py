"""Eviction from the paged cache on the GPU, exactly as oracle/paged.py does it key by key."""
import numpy as np
import pytest
import torch

from oracle import paged as op

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
BF16, F32 = torch.bfloat16, torch.float32


def _rp():
    import relative_position_representations_gb300 as rp
    return rp


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def _status_is_clear():
    assert _rp().relattn_get_device_error() == 0
    yield
    torch.cuda.synchronize()


def masses(rng, shape, kind):
    if kind == "spread":
        return np.exp(rng.standard_normal(shape) * 3)
    if kind == "ties":       # a handful of values, zeros of both signs among them
        return rng.choice([0.0, -0.0, 1.0, 2.0, 2.0, 0.5], shape)
    if kind == "equal":
        return np.ones(shape)
    if kind == "wild":       # negative ones, infinities, NaN, subnormals
        x = rng.standard_normal(shape) * 10.0 ** rng.integers(-42, 30, shape)
        pick = rng.random(shape)
        x[pick < 0.1], x[pick > 0.95], x[(pick > 0.45) & (pick < 0.5)] = np.inf, -np.inf, np.nan
        return x
    raise ValueError(kind)


def make(lens, Hkv, d, P, dtype=BF16, kind="spread", seed=0, extra=3, M=None):
    rng = np.random.default_rng(seed)
    used = [-(-max(0, n) // P) for n in lens]
    M = M or max(1, max(used))
    N = sum(used) + extra
    perm = rng.permutation(N)
    table, at = np.full((len(lens), M), 2 ** 30), 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    t = lambda: torch.from_numpy(rng.standard_normal((N, Hkv, P, d))).to(dtype)
    return dict(table=table, k=t(), v=t(), mass=torch.from_numpy(masses(rng, (N, Hkv, P), kind)).to(F32),
                free=perm.copy(), head=at)


def run(x, lens, budget, limit, sinks, recent, in_place=False, spaced=False, workspace=None):
    rp = _rp()
    f = lambda t: t.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = op.evict(lens, x["table"], f(x["k"]), f(x["v"]), f(x["mass"]), budget, limit, sinks, recent,
                        x["free"], x["head"])
    both = torch.stack([x["k"], x["v"]], 1).to(DEV) if spaced else None      # a joint pool
    k, v = (both[:, 0], both[:, 1]) if spaced else (x["k"].to(DEV), x["v"].to(DEV))
    mass = x["mass"].to(DEV)
    if spaced:
        mass = torch.zeros((mass.shape[0], mass.shape[1] + 1, mass.shape[2]), device=DEV)
        mass[:, :-1] = x["mass"].to(DEV)
        mass = mass[:, :-1]
    kv, table, free, head = i32(lens), i32(x["table"]), i32(x["free"]), i32([x["head"]])
    kw = dict(kv_len_out=kv, free_head_out=head) if in_place else {}
    got_len, got_head = rp.relattn_paged_evict(kv, table, k, v, mass, budget, limit=limit, sinks=sinks,
                                               recent=recent, free_pages=free, free_head=head,
                                               workspace=workspace, **kw)
    assert rp.relattn_get_device_error() == 0
    if in_place:
        assert got_len is kv and got_head is head
    assert np.array_equal(got_len.cpu().numpy(), want[0])
    assert np.array_equal(table.cpu().numpy(), x["table"])
    assert np.array_equal(free.cpu().numpy(), want[4]) and int(got_head) == want[5]
    for name, got, ref in (("k", k, want[1]), ("v", v, want[2]), ("mass", mass, want[3])):
        assert np.array_equal(f(got), ref, equal_nan=True), name
    return k, v, mass


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "wild"])
@pytest.mark.parametrize("P,Hkv,d", [(16, 2, 64), (8, 1, 128), (1, 3, 64), (2, 1, 64), (128, 2, 64)])
def test_a_batch_of_lengths(kind, P, Hkv, d):
    lens = [300, 130, 129, 128, 7, 0, 511, 1000, 64]
    run(make(lens, Hkv, d, P, kind=kind, seed=P), lens, 128, 128, 4, 30, in_place=P == 16)


@pytest.mark.parametrize("budget,limit,sinks,recent", [
    (1, 1, 0, 0), (1, 1, 1, 0), (1, 1, 0, 1), (2, 2, 1, 1), (100, 100, 100, 0), (100, 100, 0, 100),
    (100, 100, 60, 40), (100, 170, 3, 5), (127, 127, 0, 0), (129, 130, 7, 0), (255, 255, 0, 64), (299, 299, 0, 0),
    (300, 300, 0, 0)])
def test_budgets(budget, limit, sinks, recent):
    lens = [300, 171, 101, 2, 1, 257]
    for kind in ("spread", "ties"):
        run(make(lens, 2, 64, 16, kind=kind, seed=budget), lens, budget, limit, sinks, recent)


@pytest.mark.parametrize("dtype,d,spaced", [(BF16, 64, True), (BF16, 80, False), (BF16, 33, False), (BF16, 7, True),
                                            (BF16, 2, False), (F32, 64, False), (F32, 128, True), (F32, 127, False),
                                            (F32, 1, False), (BF16, 127, False), (BF16, 128, True)])
def test_rows_of_any_kind(dtype, d, spaced):
    lens = [500, 260, 40]
    run(make(lens, 3, d, 8, dtype=dtype, kind="ties", seed=d), lens, 200, 230, 2, 16, spaced=spaced)


@pytest.mark.parametrize("n,budget,kind", [(16384, 9000, "spread"), (16385, 100, "ties"), (20000, 19999, "ties"),
                                           (40000, 20000, "spread"), (40000, 15000, "equal")])
def test_long_requests_use_clusters(n, budget, kind):
    lens = [n, n // 3]
    run(make(lens, 1, 8, 64, kind=kind, seed=n), lens, budget, budget, 5, 70)


def test_keys_past_the_registers_of_a_cluster():
    """Past 131072 keys the weights are read again in each pass. (The oracle's lists are slow here, so
    the kept keys come from one sort.)"""
    rp = _rp()
    rng = np.random.default_rng(3)
    n, P, budget, sinks, recent = 150001, 64, 70000, 3, 500
    M = -(-n // P)
    for w in (rng.random(n).astype(np.float32), np.ones(n, np.float32), np.round(rng.random(n) * 20).astype(np.float32)):
        table = rng.permutation(M)
        mass = np.zeros((M, 1, P), np.float32)
        j = np.arange(n)
        mass[table[j // P], 0, j % P] = w
        k = torch.zeros((M, 1, P, 4), dtype=F32)
        k[table[j // P], 0, j % P] = torch.from_numpy(j[:, None] + np.zeros((1, 4))).to(F32)
        always = (j < sinks) | (j >= n - recent)
        kept = np.sort(np.lexsort((j, -w, ~always))[:budget])
        kd, vd, md = k.to(DEV), (-k).to(DEV), torch.from_numpy(mass).to(DEV)
        out, _ = rp.relattn_paged_evict(i32([n]), i32(table[None]), kd, vd, md, budget, sinks=sinks, recent=recent)
        assert rp.relattn_get_device_error() == 0 and out.tolist() == [budget]
        r = np.arange(budget)
        rows = kd[torch.from_numpy(table[r // P]), 0, torch.from_numpy(r % P)].cpu().numpy()
        assert np.array_equal(rows[:, 0], kept) and np.array_equal(rows[:, 3], kept)
        assert torch.equal(vd, -kd)
        assert np.array_equal(md[torch.from_numpy(table[r // P]), 0, torch.from_numpy(r % P)].cpu().numpy(), w[kept])


def test_many_requests_and_idle_slots():
    rng = np.random.default_rng(5)
    lens = np.where(rng.random(1500) < 0.1, rng.integers(20, 60, 1500), rng.integers(0, 20, 1500)).tolist()
    run(make(lens, 2, 8, 4, kind="ties", M=16), lens, 16, 24, 1, 3, in_place=True)
    run(make(lens, 2, 8, 4, kind="ties", M=16), lens, 64, 64, 1, 3)      # nothing to cut


def test_a_table_wider_than_its_requests_and_lengths_past_it():
    lens = [90, 1000, -4]           # the second is taken as the 128 keys that its row holds
    x = make([90, 128, 0], 1, 64, 8, M=16)
    run(x, lens, 40, 60, 2, 8)


def test_shared_first_pages_are_left_alone():
    """Two requests share pages whose keys all lie below `sinks`."""
    x = make([300, 280], 2, 64, 16, seed=9)
    x["table"][1, :4] = x["table"][0, :4]
    before = x["k"].clone()
    k, v, mass = run(x, [300, 280], 128, 128, 64, 20)
    pages = torch.from_numpy(x["table"][0, :4])
    assert torch.equal(k.cpu()[pages], before[pages])


def test_without_a_free_list():
    rp = _rp()
    x = make([100, 20], 1, 64, 16)
    k, v, mass = x["k"].to(DEV), x["v"].to(DEV), x["mass"].to(DEV)
    out, head = rp.relattn_paged_evict(i32([100, 20]), i32(x["table"]), k, v, mass, 50)
    assert out.tolist() == [50, 20] and head is None
    assert rp.relattn_get_device_error() == 0


@pytest.mark.parametrize("head", [-1, 2, 1000])
def test_a_free_list_that_the_pages_did_not_come_from(head):
    """Reported; the cut itself stands, nothing is given back."""
    rp = _rp()
    x = make([100], 1, 64, 16)
    free = i32(np.arange(50, 60))
    k, v, mass = x["k"].to(DEV), x["v"].to(DEV), x["mass"].to(DEV)
    out, got = rp.relattn_paged_evict(i32([100]), i32(x["table"]), k, v, mass, 50, free_pages=free,
                                      free_head=i32([head]))
    assert rp.relattn_get_device_error() == 1
    assert out.tolist() == [50] and got.tolist() == [head] and free.tolist() == list(range(50, 60))


def test_pages_outside_the_cache_are_reported():
    rp = _rp()
    x = make([100], 1, 64, 16)
    x["table"][0, 2] = 2 ** 30
    x["table"][0, 4] = -1
    k, v, mass = x["k"].to(DEV), x["v"].to(DEV), x["mass"].to(DEV)
    rp.relattn_paged_evict(i32([100]), i32(x["table"]), k, v, mass, 50)
    assert rp.relattn_get_device_error() == 1


def test_replayed_with_pages_taken_in_between():
    """A captured cut, replayed after the requests have grown again through the plan: lengths and the
    free list advance in place."""
    rp = _rp()
    P, M, B = 8, 12, 3
    free, head = i32(np.arange(100)), i32([0])
    kv, table = i32([0] * B), torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn((100, 2, P, 64), device=DEV, generator=g).to(BF16) for _ in range(2))
    mass = torch.rand((100, 2, P), device=DEV, generator=g)
    new = i32([70, 20, 61])
    ws = torch.empty(rp.relattn_paged_evict_workspace_size(B, 2, M * P), dtype=torch.uint8, device=DEV)

    def step():
        rp.relattn_paged_plan(kv, new, table, free, head, P, 200, kv_len=kv, free_head_out=head)
        rp.relattn_paged_evict(kv, table, k, v, mass, 32, limit=40, sinks=2, recent=8, free_pages=free,
                               free_head=head, kv_len_out=kv, free_head_out=head, workspace=ws)

    step()
    assert kv.tolist() == [32, 20, 32] and int(head) == 4 + 3 + 4
    graph = torch.cuda.CUDAGraph()
    new.copy_(i32([9, 25, 7]))
    with torch.cuda.graph(graph):
        step()
    lens = [32, 20, 32]
    for _ in range(6):
        before = (k.clone(), v.clone(), mass.clone(), table.clone())
        graph.replay()
        lens = [a + b for a, b in zip(lens, [9, 25, 7])]
        f = lambda t: t.double().cpu().numpy()
        t = table.cpu().numpy()
        want = op.evict(lens, t, f(before[0]), f(before[1]), f(before[2]), 32, 40, 2, 8)
        assert np.array_equal(f(k), want[1]) and np.array_equal(f(v), want[2]) and np.array_equal(f(mass), want[3])
        lens = want[0].tolist()
        assert kv.tolist() == lens
        held = [int(x) for b in range(B) for x in t[b, :-(-lens[b] // P)]]
        assert int(head) == len(held) == len(set(held))
        assert sorted(held + free.tolist()[int(head):]) == list(range(100))
    assert rp.relattn_get_device_error() == 0


def test_on_another_stream_and_twice_at_once():
    rp = _rp()
    lens = [3000, 2500]
    xs = [make(lens, 2, 64, 16, seed=s) for s in range(2)]
    f = lambda t: t.double().cpu().numpy()
    want = [op.evict(lens, x["table"], f(x["k"]), f(x["v"]), f(x["mass"]), 1000, 1000, 0, 9) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    on = [[x["k"].to(DEV), x["v"].to(DEV), x["mass"].to(DEV), i32(x["table"]), i32(lens)] for x in xs]
    torch.cuda.synchronize()
    for _ in range(1):
        outs = [rp.relattn_paged_evict(o[4], o[3], o[0], o[1], o[2], 1000, recent=9, stream=s)[0]
                for o, s in zip(on, streams)]
    torch.cuda.synchronize()
    for o, w, n in zip(on, want, outs):
        assert n.tolist() == [1000, 1000]
        assert np.array_equal(f(o[0]), w[1]) and np.array_equal(f(o[1]), w[2]) and np.array_equal(f(o[2]), w[3])
    assert rp.relattn_get_device_error() == 0


@pytest.mark.parametrize("lens,budget,bad", [
    ([100], 50, [(0, 4)]),                                          # the only page that a budget leaves: none of it
    ([100, 90, 20, 97], 50, [(0, 6), (1, 4), (1, 5), (3, 5)]),      # all of a request's, some of the others'
    ([100, 3000, 90], 50, [(1, 4), (1, 69), (1, 187), (2, 1)]),     # of hundreds; one in front of the budget too
    ([5000], 40, [(0, i) for i in range(3, 313, 2)])])
def test_numbers_of_no_page_do_not_get_onto_the_list(lens, budget, bad):
    """Table entries outside the cache are reported and left out of what is given back."""
    rp = _rp()
    P = 16
    x = make(lens, 2, 64, P, seed=4)
    N = x["mass"].shape[0]
    for i, (b, e) in enumerate(bad):
        x["table"][b, e] = (-1, N, 2 ** 30, -2 ** 31)[i % 4]
    gone = [int(p) for b, n in enumerate(lens) if n > budget for p in x["table"][b, -(-budget // P):-(-n // P)]]
    gone = [p for p in gone if 0 <= p < N]
    want, head = x["free"].copy(), x["head"] - len(gone)
    want[head:head + len(gone)] = gone
    free = i32(x["free"])
    out, got = rp.relattn_paged_evict(i32(lens), i32(x["table"]), x["k"].to(DEV), x["v"].to(DEV), x["mass"].to(DEV), budget,
                                      free_pages=free, free_head=i32([x["head"]]))
    assert rp.relattn_get_device_error() == 1
    assert out.tolist() == [min(n, budget) for n in lens]
    assert int(got) == head and np.array_equal(free.cpu().numpy(), want)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 128), (BF16, 33)])
def test_a_wait_that_runs_out(dtype, d):
    """A block of rows that is never said to have been read: those that would overwrite them give up and say so; lengths, the
    free list and the request that is not cut are as they should be, and the next call is right."""
    rp = _rp()
    lens, budget = [600, 100, 700], 256
    x = make(lens, 2, d, 16, dtype=dtype, seed=d)
    want = op.evict(lens, x["table"], *(x[n].double().numpy() for n in ("k", "v", "mass")), budget, budget, 0, 100, x["free"],
                    x["head"])
    k, v, mass, free = x["k"].to(DEV), x["v"].to(DEV), x["mass"].to(DEV), i32(x["free"])
    try:
        rp.relattn_set_wait_limit(2_000_000)
        rp.relattn_debug_withhold_first_load(1)
        out, head = rp.relattn_paged_evict(i32(lens), i32(x["table"]), k, v, mass, budget, recent=100, free_pages=free,
                                           free_head=i32([x["head"]]))
        assert rp.relattn_get_device_error() == 4
    finally:
        rp.relattn_debug_withhold_first_load(0)
        rp.relattn_set_wait_limit(2_000_000_000)
    assert out.tolist() == want[0].tolist() == [256, 100, 256]
    assert int(head) == want[5] and np.array_equal(free.cpu().numpy(), want[4])
    cut = torch.from_numpy(np.concatenate([x["table"][0], x["table"][2]]))
    rest = torch.ones(len(x["k"]), dtype=torch.bool)
    rest[cut[cut < len(rest)]] = False
    for got, was in ((k, x["k"]), (v, x["v"]), (mass, x["mass"])):
        assert torch.equal(got.cpu()[rest], was[rest])
    run(x, lens, budget, budget, 0, 100)


@pytest.mark.parametrize("bad", [False, True])
def test_more_requests_are_cut_than_a_block_has_threads(bad):
    """Their pages go back in several turns, in the requests' order."""
    rp = _rp()
    rng = np.random.default_rng(6)
    P, budget = 4, 18
    lens = rng.integers(10, 70, 1300).tolist()
    x = make(lens, 1, 8, P, kind="ties", seed=6)
    if not bad:
        run(x, lens, budget, budget, 1, 3, in_place=True)
        return
    N, first = x["mass"].shape[0], -(-budget // P)
    for b in range(0, 1300, 7):
        if lens[b] > budget:
            x["table"][b, int(rng.integers(first, -(-lens[b] // P) + 1)) - 1] = -3   # (some in front of the budget)
    gone = [int(p) for b, n in enumerate(lens) if n > budget for p in x["table"][b, first:-(-n // P)]]
    assert sum(n > budget for n in lens) > 1000 and min(gone) < 0
    gone = [p for p in gone if 0 <= p < N]
    want, head = x["free"].copy(), x["head"] - len(gone)
    want[head:head + len(gone)] = gone
    free = i32(x["free"])
    _, got = rp.relattn_paged_evict(i32(lens), i32(x["table"]), x["k"].to(DEV), x["v"].to(DEV), x["mass"].to(DEV), budget,
                                    sinks=1, recent=3, free_pages=free, free_head=i32([x["head"]]))
    assert rp.relattn_get_device_error() == 1
    assert int(got) == head and np.array_equal(free.cpu().numpy(), want)
