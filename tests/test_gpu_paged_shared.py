"""Attention of requests that share prefixes, on the GPU, against oracle/paged.py in 64 bits: the definition is
that of relattn_paged_fwd, every key fetched through the request's own row of the table."""
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


def f64(t):
    return None if t is None else t.double().cpu().numpy()


@pytest.fixture(autouse=True)
def _status_is_clear():
    assert _rp().relattn_get_device_error() == 0
    yield
    torch.cuda.synchronize()


def make(groups, H, Hkv, d, P, dtype=BF16, clip_k=0, key=False, value=False, shared_tables=False, seed=0, before=(), after=(),
         extra_rows=0):
    """groups: [(prefix, [(cached behind the prefix's pages, new), ...]), ...]; before, after: (cached, new) of requests
    outside the groups. A group's requests share the prefix's whole pages; rows that no token sees hold NaN, table
    entries behind the last page a wild number."""
    rng = np.random.default_rng(seed)
    reqs, start, prefix = [(0, c, n, None) for c, n in before], [len(before)], []
    for i, (L, members) in enumerate(groups):
        reqs += [(L // P, L // P * P + c, n, i) for c, n in members]
        start.append(start[-1] + len(members))
        prefix.append(L // P * P)
    reqs += [(0, c, n, None) for c, n in after]
    kv = np.array([c + n for _, c, n, _ in reqs])
    M = max(1, int(-(-kv.max() // P)))
    own = [max(0, -(-int(c) // P) - h) for c, (h, _, _, _) in zip(kv, reqs)]
    heads = [L // P for L, _ in groups]
    N = sum(own) + sum(heads) + 3
    perm, at = rng.permutation(N), 0
    first = []
    for h in heads:
        first.append(perm[at:at + h])
        at += h
    table = np.full((len(reqs), M), 2 ** 30)
    for b, ((h, c, n, i), u) in enumerate(zip(reqs, own)):
        if i is not None:
            table[b, :h] = first[i][:M]
        table[b, h:h + u] = perm[at:at + u]
        at += u
    t = lambda *s, sd=1.0: (torch.from_numpy(rng.standard_normal(s)) * sd).to(dtype)
    kp, vp = t(N, Hkv, P, d), t(N, Hkv, P, d)
    live = torch.zeros((N, P), dtype=torch.bool)
    for b in range(len(reqs)):
        for j in range(kv[b] if reqs[b][2] else 0):
            live[table[b, j // P], j % P] = True
    kp.transpose(1, 2)[~live] = float("nan")
    vp.transpose(1, 2)[~live] = float("nan")
    new = [n for _, _, n, _ in reqs]
    Ht = 1 if shared_tables else Hkv
    return dict(q=t(sum(new) + extra_rows, H, d), k_pages=kp, v_pages=vp, table=table,
                q_start=np.concatenate([[0], np.cumsum(new)]), kv_len=kv,
                aK=t(Ht, 2 * clip_k + 1, d, sd=0.5) if key else None, aV=t(Ht, 2 * clip_k + 1, d, sd=0.5) if value else None,
                group_start=np.array(start), prefix_len=np.array(prefix))


def check(x, clip_k=0, window=0, sinks=0, scale=None, max_new=0, weight_step=2.0 ** -8, **kw):
    rp = _rp()
    T, H, d = x["q"].shape
    scale = d ** -0.5 if scale is None else scale
    args = (f64(x["q"]), f64(x["k_pages"]), f64(x["v_pages"]), x["table"], x["q_start"], x["kv_len"], f64(x["aK"]), f64(x["aV"]),
            clip_k, window, sinks, scale)
    z, mass, size = op.attend(*args)
    lse, _ = op.log_sum(args[0], args[1], *args[3:7], *args[8:])
    g = {k: x[k].to(DEV) if x[k] is not None else None for k in ("q", "k_pages", "v_pages", "aK", "aV")}
    wide = torch.zeros((T, H + 1, d), dtype=x["q"].dtype, device=DEV)    # a slice of a joint projection
    wide[:, :H] = g["q"]
    q = g["q"] if T == 0 else wide[:, :H]
    got_lse = torch.full((T, H), 5.0, device=DEV)
    out = torch.full((T, H, d), 5.0, dtype=x["q"].dtype, device=DEV)
    call = (q, g["k_pages"], g["v_pages"], i32(x["table"]), i32(x["q_start"]), i32(x["kv_len"]), i32(x["group_start"]),
            i32(x["prefix_len"]))
    kw = dict(kw, aK=g["aK"], aV=g["aV"], clip_k=clip_k, window=window, sinks=sinks, scale=scale, max_new=max_new)
    assert rp.relattn_paged_shared_fwd(*call, **kw, out=out, lse=got_lse) is out
    assert rp.relattn_get_device_error() == 0
    rows = int(x["q_start"][-1])
    keys = int(max(x["kv_len"].max(), 1))
    u = 2.0 ** -24
    half = 2.0 ** -8 if x["q"].dtype == BF16 else u
    known = np.where(np.isinf(lse), 0, np.abs(lse))
    # the parts' weights go by their log-sum-exps: three rounded numbers of at most that size, two exponentials
    tol = op.tolerance(z, mass, size, keys, d, half, weight_step if x["q"].dtype == BF16 else u) + \
        2.0 * (12.0 * u * (size + known) + 2.0 ** -20)[..., None] * mass
    got = f64(out)
    bad = ~(np.abs(got - z) <= tol)[:rows]
    assert not bad.any(), (int(bad.sum()), np.abs(got - z)[:rows][bad].max(), np.argwhere(bad)[:4])
    g_lse = f64(got_lse)
    assert (got[rows:] == 5.0).all() and (g_lse[rows:] == 5.0).all()   # no request's
    tol = 4.0 * (d + 6) * u * size + 2.0 ** -20 + 2.0 * keys * u + 12.0 * u * known
    with np.errstate(invalid="ignore"):
        assert ((g_lse == lse) | (np.abs(g_lse - lse) <= tol))[:rows].all()
    assert torch.equal(rp.relattn_paged_shared_fwd(*call, **kw), rp.relattn_paged_shared_fwd(*call, **kw)) or extra_nan(out, rows)
    again = rp.relattn_paged_shared_fwd(*call, **kw)
    assert torch.equal(again[:rows], out[:rows])
    return out


def extra_nan(out, rows):
    return rows < out.shape[0]


TERMS = [(0, False, False), (16, True, True), (16, True, False), (16, False, True), (1, True, True), (127, True, True)]


@pytest.mark.parametrize("H,Hkv,d,P", [(4, 4, 64, 16), (8, 2, 128, 8), (6, 2, 64, 128), (16, 1, 128, 32)])
@pytest.mark.parametrize("clip_k,key,value", TERMS)
def test_one_group_of_single_tokens(H, Hkv, d, P, clip_k, key, value):
    members = [(5, 1), (0, 1), (130, 1), (300, 1), (17, 1), (128, 1)]
    x = make([(520, members)], H, Hkv, d, P, clip_k=clip_k, key=key, value=value, seed=P)
    check(x, clip_k, max_new=1)
    check(make([(384, members * 4)], H, Hkv, d, P, clip_k=clip_k, key=key, value=value, shared_tables=True, seed=P), clip_k)


@pytest.mark.parametrize("H,Hkv,d", [(4, 4, 64), (8, 2, 128), (5, 1, 64)])
@pytest.mark.parametrize("clip_k,key,value", TERMS[:3])
def test_groups_among_others(H, Hkv, d, clip_k, key, value):
    """Requests outside every group, groups of one, groups whose prefix is too short, idle requests in and
    between the groups, several tokens a request."""
    groups = [(300, [(20, 3), (0, 2), (9, 0), (200, 5)]), (1000, [(1, 1)]), (100, [(40, 2), (3, 1)]), (0, [(50, 1), (5, 4)]),
              (256, [(0, 0), (30, 0)]), (640, [(0, 0), (7, 1), (90, 2)])]
    x = make(groups, H, Hkv, d, 16, clip_k=clip_k, key=key, value=value, before=[(200, 1), (0, 3)], after=[(50, 2), (400, 1)],
             extra_rows=3)
    check(x, clip_k, max_new=5)
    check(x, clip_k)


def test_the_row_of_an_idle_request_is_not_used():
    x = make([(512, [(0, 0), (40, 1), (70, 1)])], 2, 2, 64, 16)
    x["table"][0] = 2 ** 30
    check(x, max_new=1)


@pytest.mark.parametrize("clip_k", [0, 4, 100])
def test_new_tokens_inside_the_prefix_and_short_requests(clip_k):
    """prefix_len past some requests' own length: they share up to where their tokens stand."""
    x = make([(512, [(40, 1), (70, 2)])], 4, 2, 64, 16, clip_k=clip_k, key=clip_k > 0, value=clip_k > 0)
    for short in (512, 511, 300, 128, 127, 1, 0):
        y = dict(x, kv_len=np.array([short, x["kv_len"][1]]))
        check(y, clip_k)
    check(dict(x, prefix_len=np.array([511])), clip_k)
    check(dict(x, prefix_len=np.array([-5])), clip_k)


@pytest.mark.parametrize("dtype,H,Hkv,d,P", [(F32, 4, 2, 64, 16), (F32, 3, 3, 33, 8), (BF16, 4, 2, 80, 16), (BF16, 4, 1, 64, 4),
                                             (F32, 40, 1, 128, 1), (BF16, 3, 1, 7, 2)])
@pytest.mark.parametrize("clip_k,key,value", TERMS[:2] + [(200, True, True)])
def test_simt(dtype, H, Hkv, d, P, clip_k, key, value):
    groups = [(300, [(20, 3), (0, 1), (9, 0), (90, 2)]), (130, [(1, 1), (30, 1)])]
    x = make(groups, H, Hkv, d, P, dtype=dtype, clip_k=clip_k, key=key, value=value, before=[(20, 1)])
    check(x, clip_k)


def test_chunks_and_prompts_behind_a_prefix():
    groups = [(256, [(0, 150), (30, 1), (200, 300)]), (128, [(0, 40), (5, 129)])]
    for d, H, Hkv in ((64, 4, 4), (128, 6, 2)):
        check(make(groups, H, Hkv, d, 32, clip_k=20, key=True, value=True, after=[(0, 77)]), 20)


@pytest.mark.parametrize("d", [64, 128])
def test_requests_that_fill_a_tile_run_as_without_groups(d):
    rp = _rp()
    x = make([(256, [(0, 150), (30, 120)])], 4, 2, d, 16, clip_k=7, key=True, value=True)
    out = check(x, 7)
    g = {k: x[k].to(DEV) for k in ("q", "k_pages", "v_pages", "aK", "aV")}
    assert torch.equal(out, rp.relattn_paged_fwd(g["q"], g["k_pages"], g["v_pages"], i32(x["table"]), i32(x["q_start"]),
                                                 i32(x["kv_len"]), aK=g["aK"], aV=g["aV"], clip_k=7))


def test_long_prefixes_are_cut_into_pieces():
    x = make([(8192, [(i * 37 % 200, 1) for i in range(40)])], 8, 2, 128, 64, clip_k=8, key=True, value=True)
    check(x, 8, max_new=1)
    x = make([(5000, [(i * 37 % 100, 1 + i % 3) for i in range(9)]), (3000, [(1, 1), (200, 1)])], 2, 1, 64, 16)
    check(x)


def test_few_rows_in_all():
    """At most 16 rows per key head in the whole call: both parts on the kernel for generated tokens."""
    x = make([(700, [(3, 1), (100, 1)])], 4, 1, 64, 16, clip_k=5, key=True, value=True)
    check(x, 5, max_new=1, weight_step=2.0 ** -16)


@pytest.mark.parametrize("window,sinks", [(64, 3), (400, 0), (10 ** 6, 0)])
def test_under_a_window(window, sinks):
    x = make([(512, [(40, 1), (70, 2)])], 4, 2, 64, 16, clip_k=4, key=True, value=True)
    check(x, 4, window=window, sinks=sinks)


def test_no_groups_no_tokens():
    rp = _rp()
    x = make([(512, [(40, 1), (70, 2)])], 4, 2, 64, 16)
    check(dict(x, group_start=np.array([0]), prefix_len=np.zeros(0, dtype=int)))
    g = {k: x[k].to(DEV) for k in ("q", "k_pages", "v_pages")}
    out = rp.relattn_paged_shared_fwd(g["q"][:0], g["k_pages"], g["v_pages"], i32(x["table"]), i32([0, 0, 0]), i32(x["kv_len"]),
                                      i32([0, 2]), i32([512]))
    assert out.shape == (0, 4, 64)


def test_many_groups():
    groups = [(128 + 16 * (i % 9), [(i % 40, 1)] * (1 + i % 4)) for i in range(150)]
    check(make(groups, 2, 1, 64, 16, clip_k=3, key=True), 3, max_new=1)


def test_offsets_that_are_not_ascending_stay_within_the_arrays():
    rp = _rp()
    x = make([(300, [(20, 3), (0, 2), (200, 5)]), (256, [(3, 1), (4, 1)])], 4, 2, 64, 16)
    g = {k: x[k].nan_to_num().to(DEV) for k in ("q", "k_pages", "v_pages")}
    room = torch.full((40, 4, 64), 3.0, dtype=BF16, device=DEV)
    for starts, qs in (([4, 1, 9], x["q_start"]), ([-3, 2, 100], x["q_start"]), ([0, 3, 5], np.array([0, 12, 3, 9, -4, 12])),
                       ([0, 5, 0], np.array([12, 0, 12, 0, 12, 0]))):
        out = room[10:22]
        rp.relattn_paged_shared_fwd(g["q"], g["k_pages"], g["v_pages"], i32(np.clip(x["table"], 0, 5)), i32(qs), i32(x["kv_len"]),
                                    i32(starts), i32([300, 256]), out=out)
        assert rp.relattn_get_device_error() == 0
        assert bool((room[:10] == 3).all()) and bool((room[22:] == 3).all())


def test_pages_outside_the_cache_are_reported():
    rp = _rp()
    x = make([(512, [(20, 1), (30, 1)])], 2, 2, 64, 16)
    x["table"][:, 3] = -7
    g = {k: x[k].to(DEV) for k in ("q", "k_pages", "v_pages")}
    rp.relattn_paged_shared_fwd(g["q"], g["k_pages"], g["v_pages"], i32(x["table"]), i32(x["q_start"]), i32(x["kv_len"]),
                                i32(x["group_start"]), i32(x["prefix_len"]))
    assert rp.relattn_get_device_error() == 1


def test_replayed_with_other_lengths_and_groups():
    rp = _rp()
    a = make([(512, [(40, 1), (70, 1), (5, 1)]), (256, [(3, 1), (9, 1)])], 4, 2, 64, 16, clip_k=6, key=True, value=True, seed=1)
    b = make([(256, [(40, 1), (100, 1)]), (384, [(3, 1), (9, 1), (90, 1)])], 4, 2, 64, 16, clip_k=6, key=True, value=True, seed=2)
    N, M = max(x["k_pages"].shape[0] for x in (a, b)), max(x["table"].shape[1] for x in (a, b))
    kp, vp = (torch.zeros((N, 2, 16, 64), dtype=BF16, device=DEV) for _ in range(2))
    q, table = torch.zeros((5, 4, 64), dtype=BF16, device=DEV), torch.zeros((5, M), dtype=torch.int32, device=DEV)
    qs, kv, gs, pl = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (6, 5, 3, 2))
    tabs = [a["aK"].to(DEV), a["aV"].to(DEV)]
    ws = torch.empty(rp.relattn_paged_shared_workspace_size(5, 4, 2, 64), dtype=torch.uint8, device=DEV)
    run = lambda: rp.relattn_paged_shared_fwd(q, kp, vp, table, qs, kv, gs, pl, aK=tabs[0], aV=tabs[1], clip_k=6, max_new=1,
                                              workspace=ws)

    def put(x):
        kp[:x["k_pages"].shape[0]] = x["k_pages"].to(DEV)
        vp[:x["k_pages"].shape[0]] = x["v_pages"].to(DEV)
        q.copy_(x["q"])
        table[:, :x["table"].shape[1]] = i32(x["table"])
        for t, k in ((qs, "q_start"), (kv, "kv_len"), (gs, "group_start"), (pl, "prefix_len")):
            t.copy_(i32(x[k]))
        for t, k in zip(tabs, ("aK", "aV")):
            t.copy_(x[k])

    put(a)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for x in (a, b, a):
        put(x)
        graph.replay()
        want = check(x, 6, max_new=1)
        assert torch.equal(out, want)


def test_a_wait_that_runs_out():
    """Queries that never come, in both parts: the call ends and says so, and the next one is right."""
    rp = _rp()
    x = make([(640, [(i * 11, 1) for i in range(20)])], 8, 2, 64, 16)
    g = [x[k].to(DEV) for k in ("q", "k_pages", "v_pages")] + [i32(x[k]) for k in ("table", "q_start", "kv_len", "group_start",
                                                                                 "prefix_len")]
    try:
        rp.relattn_set_wait_limit(2_000_000)
        rp.relattn_debug_withhold_first_load(1)
        rp.relattn_paged_shared_fwd(*g, max_new=1)
        assert rp.relattn_get_device_error() == 4
    finally:
        rp.relattn_debug_withhold_first_load(0)
        rp.relattn_set_wait_limit(2_000_000_000)
    check(x, max_new=1)


def test_a_step_that_is_cut_and_goes_on():
    """A group's requests behind a shared prefix, cut by their weights (the prefix lies below `sinks`), attended again: the
    prefix stays as it is for all of them."""
    rp = _rp()
    x = make([(256, [(150, 1), (90, 1), (200, 1)])], 4, 2, 64, 16, clip_k=5, key=True, value=True)
    N = x["k_pages"].shape[0]
    g = {k: x[k].to(DEV) for k in ("q", "k_pages", "v_pages", "aK", "aV")}
    table, qs, kv, gs, pl = (i32(x[k]) for k in ("table", "q_start", "kv_len", "group_start", "prefix_len"))
    lse = torch.empty((3, 4), device=DEV)
    mass = torch.rand((N, 2, 16), device=DEV)
    kw = dict(aK=g["aK"], aV=g["aV"], clip_k=5, max_new=1)
    rp.relattn_paged_shared_fwd(g["q"], g["k_pages"], g["v_pages"], table, qs, kv, gs, pl, lse=lse, **kw)
    # (the shared pages' masses hold no defined number afterwards; below `sinks` none is looked at)
    rp.relattn_paged_weights(g["q"], g["k_pages"], table, qs, kv, lse, mass, aK=g["aK"], clip_k=5, max_new=1)
    kv2, _ = rp.relattn_paged_evict(kv, table, g["k_pages"], g["v_pages"], mass, 320, limit=350, sinks=256, recent=16)
    assert kv2.tolist() == [320, 346 + 1, 320]
    shared = torch.from_numpy(x["table"][0, :16])
    assert torch.equal(g["k_pages"][shared].cpu(), x["k_pages"][shared])
    y = dict(x, k_pages=g["k_pages"].cpu(), v_pages=g["v_pages"].cpu(), kv_len=np.array(kv2.tolist()))
    check(y, 5, max_new=1)


def test_two_streams_at_once():
    rp = _rp()
    xs = [make([(4096, [(i * 11, 1) for i in range(20)])], 8, 2, 128, 16, seed=s) for s in range(2)]
    gs = [[x[k].to(DEV) for k in ("q", "k_pages", "v_pages")] + [i32(x[k]) for k in ("table", "q_start", "kv_len", "group_start",
                                                                                    "prefix_len")] for x in xs]
    want = [rp.relattn_paged_shared_fwd(*g, max_new=1) for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [rp.relattn_paged_shared_fwd(*g, max_new=1, stream=s) for g, s in zip(gs, streams)]
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
