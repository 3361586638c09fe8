"""The paged key/value cache on the GPU against oracle/paged.py in 64 bits: plans and copies
exactly, attention within the bound that oracle.paged.tolerance derives from the types."""
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


# ------------------------------------------------------------------------------------ plan
def run_plan(cached, new, P, M, free, head, max_tokens, in_place=False, table=None):
    rp = _rp()
    rng = np.random.default_rng(len(cached) + P)
    if table is None:
        table = rng.integers(1000, 2000, (len(cached), M))
    ref = op.plan(cached, new, table, free, head, P, max_tokens)
    bt, c, h = i32(table), i32(cached), i32([head])
    kw = dict(kv_len=c, free_head_out=h) if in_place else {}
    kv, qs, sl, ho = rp.relattn_paged_plan(c, i32(new), bt, i32(free), h, P, max_tokens, **kw)
    err = rp.relattn_get_device_error()
    for got, want in zip((bt, kv, qs, sl, ho), ref[:4] + (np.array([ref[4]]),)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert err == (0 if ref[5] else 1)
    return ref


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,P,lo,hi,cmax", [
    (1, 16, 1, 1, 0), (1, 1, 5, 5, 3), (3, 8, 0, 9, 40), (33, 16, 1, 1, 100), (64, 64, 0, 300, 200),
    (1000, 16, 0, 3, 50), (1025, 8, 1, 1, 20), (2500, 32, 0, 7, 10), (40, 16, 200, 700, 900),
    (1, 1024, 20000, 20000, 5), (2, 128, 9000, 9001, 127)])
def test_plan_matches_the_allocator(B, P, lo, hi, cmax, in_place):
    rng = np.random.default_rng(B * 7 + P)
    cached, new = rng.integers(0, cmax + 1, B), rng.integers(lo, hi + 1, B)
    M = int(-(-(cached + new).max() // P)) + 1
    need = int((-(-(cached + new) // P) - -(-cached // P)).sum())
    free = rng.permutation(need + 10)
    run_plan(cached, new, P, M, free, 4, int(new.sum()) + 5, in_place)


def test_plan_leaves_out_what_does_not_fit():
    free = np.arange(100, 110)
    # the third request finds too few pages: it and the fifth stay out, the fourth needs none
    run_plan([0, 5, 3, 3, 8], [33, 4, 90, 2, 9], 8, 16, free, 0, 200)
    # a table row that is too short; negative lengths; more new tokens than slots
    run_plan([0, 120, 0], [8, 9, 8], 8, 16, free, 0, 64)
    run_plan([-1, 0, 4], [3, 8, 2], 8, 16, free, 0, 64)
    run_plan([0, 0, 4], [3, -8, 2], 8, 16, free, 0, 64)
    run_plan([0, 0, 0], [30, 20, 8], 8, 16, free, 0, 40)
    run_plan([0, 0, 0], [30, 41, 8], 8, 16, free, 0, 40)
    run_plan([0, 0], [8, 8], 8, 4, np.zeros(0, dtype=np.int64), 0, 16)
    run_plan([4, 9], [4, 7], 8, 4, np.zeros(0, dtype=np.int64), 0, 16)   # no page needed
    run_plan([2 ** 31 - 1, 0], [5, 5], 8, 4, free, 0, 16)
    # a free-list head that is no index: nothing is handed out
    run_plan([4, 8], [4, 7], 8, 4, free, -3, 16)
    run_plan([4, 8], [4, 7], 8, 4, free, 1000, 16)
    # nothing new at all, and no slots
    run_plan([4, 9, 0], [0, 0, 0], 8, 4, free, 10, 0)


def test_plan_spaced_table_rows():
    rp = _rp()
    wide = torch.full((3, 12), -7, dtype=torch.int32, device=DEV)
    rp.relattn_paged_plan(i32([0, 3, 8]), i32([9, 1, 8]), wide[:, 2:6], i32(np.arange(20, 30)), i32([1]), 4, 18)
    want = np.full((3, 12), -7)
    want[0, 2:5] = [21, 22, 23]
    want[2, 4:6] = [24, 25]
    assert np.array_equal(wide.cpu().numpy(), want)


# ------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,Hkv,d,P,odd", [(1, 1, 64, 16, False), (33, 3, 80, 8, False), (7, 2, 33, 4, False),
                                           (1500, 2, 128, 32, False), (1025, 5, 8, 1, False), (40, 4, 64, 16, True)])
def test_append_writes_the_slots_and_nothing_else(dtype, T, Hkv, d, P, odd):
    rp = _rp()
    g = torch.Generator().manual_seed(T + d)
    N = T // P + 5
    rng = np.random.default_rng(T)
    slots = rng.permutation(N * P)[:T]
    if T > 3:
        slots[1], slots[3] = -1, -5
    off = 1 if odd else 0   # an odd offset: rows that no wide load may touch
    kv = torch.randn((T, 2 * Hkv * d + 3), generator=g).to(dtype).to(DEV)
    k = kv[:, off:off + Hkv * d].unflatten(1, (Hkv, d))
    v = kv[:, Hkv * d + off:2 * Hkv * d + off].unflatten(1, (Hkv, d))
    both = torch.randn((N, 2, Hkv, P, d), generator=g).to(dtype).to(DEV)   # a joint pool
    kp, vp = both[:, 0], both[:, 1]
    f = lambda t: t.double().cpu().numpy()
    wk, wv = op.append(f(k), f(v), slots, f(kp), f(vp))
    rp.relattn_paged_append(k, v, i32(slots), kp, vp)
    assert rp.relattn_get_device_error() == 0
    assert np.array_equal(f(kp), wk) and np.array_equal(f(vp), wv)


def test_append_reports_a_slot_outside_the_cache():
    rp = _rp()
    kp, vp = torch.zeros((2, 1, 8, 64), device=DEV), torch.zeros((2, 1, 8, 64), device=DEV)
    k = torch.ones((3, 1, 64), device=DEV)
    rp.relattn_paged_append(k, k, i32([3, 16, 2 ** 31 - 1]), kp, vp)
    assert rp.relattn_get_device_error() == 1
    assert float(kp.sum()) == 64 and float(vp.sum()) == 64
    rp.relattn_paged_append(k[:0], k[:0], i32([]), kp, vp)   # no token
    assert rp.relattn_get_device_error() == 0


# ------------------------------------------------------------------------------------ attention
def make(new, kv, H, Hkv, d, P, dtype, clip_k=0, key=False, value=False, shared=False, std=1.0,
         table_std=0.5, seed=0, stale=True, extra_rows=0):
    """Inputs for the GPU and, in float64, for the oracle. Rows that no token sees hold NaN, table
    entries behind the last page a wild number."""
    rng = np.random.default_rng(seed)
    new, kv = np.asarray(new), np.asarray(kv)
    M = max(1, int(-(-kv.max() // P)))
    used = [int(-(-max(0, c) // P)) for c in kv]
    N = sum(used) + 3
    perm = rng.permutation(N)
    table = np.full((len(kv), M), 2 ** 30, dtype=np.int64)
    at = 0
    t = lambda *s, sd=1.0: (torch.from_numpy(rng.standard_normal(s)) * sd).to(dtype)
    kp, vp = t(N, Hkv, P, d, sd=std), t(N, Hkv, P, d)
    live = torch.zeros((N, P), dtype=torch.bool)
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
        for j in range(max(0, int(kv[b]))):
            live[table[b, j // P], j % P] = True
    if stale:
        kp.transpose(1, 2)[~live] = float("nan")
        vp.transpose(1, 2)[~live] = float("nan")
    T = int(new.sum()) + extra_rows
    q = t(T, H, d, sd=std)
    Ht = 1 if shared else Hkv
    aK = t(Ht, 2 * clip_k + 1, d, sd=table_std) if key else None
    aV = t(Ht, 2 * clip_k + 1, d, sd=table_std) if value else None
    return dict(q=q, k_pages=kp, v_pages=vp, table=table, q_start=np.concatenate([[0], np.cumsum(new)]),
                kv_len=kv, aK=aK, aV=aV)


def call(x, clip_k, window=0, sinks=0, scale=None, max_new=0, **kw):
    rp = _rp()
    g = lambda t: None if t is None else t.to(DEV)
    T, H, d = x["q"].shape
    ws = torch.full((rp.relattn_paged_workspace_size(H, x["k_pages"].shape[1], d),), 0xFF, dtype=torch.uint8,
                    device=DEV)   # scratch contents must not matter
    out = torch.full((T, H, d), float("nan"), dtype=x["q"].dtype, device=DEV)
    return rp.relattn_paged_fwd(g(x["q"]), g(x["k_pages"]), g(x["v_pages"]), i32(x["table"]), i32(x["q_start"]),
                                i32(x["kv_len"]), aK=g(x["aK"]), aV=g(x["aV"]), clip_k=clip_k, window=window,
                                sinks=sinks, scale=scale, max_new=max_new, out=out, workspace=ws, **kw)


def check(x, got, clip_k, window=0, sinks=0, scale=None):
    d = x["q"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    f = lambda t: None if t is None else t.double().numpy()
    z, mass, size = op.attend(f(x["q"]), np.nan_to_num(f(x["k_pages"])), np.nan_to_num(f(x["v_pages"])), x["table"],
                              x["q_start"], x["kv_len"], f(x["aK"]), f(x["aV"]), clip_k, window, sinks, scale)
    got = got.double().cpu().numpy()
    n = int(x["q_start"][-1])
    assert np.isnan(got[n:]).all()          # rows behind the last request stay
    got, z, mass, size = got[:n], z[:n], mass[:n], size[:n]
    bf = x["q"].dtype == BF16
    half = 2.0 ** -8 if bf else 2.0 ** -24
    tol = op.tolerance(z, mass, size, float(np.max(x["kv_len"])), d, half, half)
    assert np.isfinite(got).all()
    bad = np.abs(got - z) - tol
    at = np.unravel_index(np.argmax(bad), bad.shape)
    assert bad[at] <= 0, (at, got[at], z[at], tol[at])


CASES = [
    # name, new, kv, H, Hkv, d, P, clip_k, key, value, kw
    ("one_key", [1], [1], 1, 1, 64, 16, 2, True, True, {}),
    ("plain_decode", [1, 1, 1], [300, 17, 129], 4, 4, 64, 16, 0, False, False, {}),
    ("decode_terms", [1, 1, 1, 1], [700, 1, 16, 385], 4, 4, 64, 16, 16, True, True, {}),
    ("decode_terms_d128", [1, 1], [515, 257], 8, 2, 128, 32, 64, True, True, {}),
    ("decode_grouped", [1, 1, 1], [1000, 511, 64], 16, 2, 128, 8, 4, False, True, {}),
    ("decode_long", [1], [9001], 16, 2, 64, 64, 16, True, True, {}),
    ("decode_group_16", [1, 1], [333, 90], 16, 1, 64, 16, 5, True, False, {}),
    ("decode_group_48", [1, 1], [200, 90], 48, 1, 64, 16, 5, True, True, {}),
    ("few_tokens", [3, 2, 4], [333, 2, 200], 8, 2, 64, 16, 16, True, True, {}),
    ("few_tokens_d128", [7, 5], [400, 129], 6, 2, 128, 16, 16, True, True, {}),
    ("no_new_tokens", [0, 2, 0, 1, 0], [50, 40, 0, 30, 7], 2, 2, 64, 16, 3, True, True, {}),
    ("empty_rows", [5, 9, 1], [3, 0, 0], 4, 2, 64, 16, 3, True, True, {}),
    ("prompt", [129, 257], [129, 257], 2, 2, 64, 16, 16, True, True, {}),
    ("prompt_d128", [200, 65], [200, 65], 4, 1, 128, 16, 64, True, False, {}),
    ("prompt_group_3", [150], [150], 6, 2, 64, 8, 4, True, True, {}),
    ("prompt_group_5", [140, 3], [170, 400], 10, 2, 128, 64, 16, True, True, {}),
    ("prompt_group_128", [3], [150], 128, 1, 64, 16, 4, True, True, {}),
    ("chunk", [100, 1, 37], [700, 500, 37], 4, 4, 64, 16, 16, True, True, {}),
    ("chunk_d128", [130, 1], [600, 900], 4, 2, 128, 128, 16, True, True, {}),
    ("chunk_plain", [300], [1100], 2, 1, 128, 256, 0, False, False, {}),
    ("clip_0", [40, 1], [90, 300], 2, 2, 64, 16, 0, True, True, {}),
    ("clip_over_length", [60, 1], [60, 90], 2, 2, 64, 16, 127, True, True, {}),
    ("clip_256", [20, 1], [300, 290], 2, 1, 64, 16, 256, True, True, {}),
    ("shared_tables", [70, 1], [100, 200], 4, 2, 64, 16, 8, True, True, dict(shared=True)),
    ("value_only", [90, 2], [200, 400], 2, 2, 128, 16, 16, False, True, {}),
    ("window", [1, 100], [900, 700], 4, 2, 64, 16, 0, False, False, dict(window=200)),
    ("window_1", [1, 30], [500, 100], 2, 2, 64, 16, 4, True, True, dict(window=1)),
    ("window_sinks", [1, 130, 1], [1500, 900, 40], 4, 2, 64, 16, 16, True, True, dict(window=129, sinks=4)),
    ("window_sinks_d128", [200, 1], [1000, 1300], 8, 2, 128, 16, 16, True, True, dict(window=300, sinks=130)),
    ("window_in_clip", [50, 1], [400, 300], 2, 1, 64, 8, 64, True, True, dict(window=20, sinks=3)),
    ("sinks_over_all", [50, 1], [400, 300], 2, 1, 64, 8, 4, True, True, dict(window=20, sinks=10000)),
    ("window_over_all", [50, 1], [400, 300], 2, 1, 64, 8, 4, True, True, dict(window=10000, sinks=3)),
    ("page_1", [9, 1], [40, 70], 2, 2, 64, 1, 4, True, True, {}),
    ("page_4", [150], [200], 2, 2, 64, 4, 4, True, True, {}),
    ("page_1024", [150, 1], [200, 1025], 2, 2, 64, 1024, 4, True, True, {}),
    ("d_80", [40, 1], [90, 300], 4, 2, 80, 16, 4, True, True, {}),
    ("d_96", [40, 1], [90, 300], 4, 2, 96, 16, 4, True, True, {}),
    ("d_33", [20, 1], [50, 70], 2, 1, 33, 16, 4, True, True, {}),
    ("d_1", [20, 1], [50, 70], 2, 1, 1, 16, 4, True, True, {}),
    ("negative_scale", [40, 1], [90, 300], 2, 2, 64, 16, 4, True, True, dict(scale=-0.2)),
    ("zero_scale", [40, 1], [90, 300], 2, 2, 64, 16, 4, True, True, dict(scale=0.0)),
    ("big_scores", [40, 1, 130], [90, 300, 400], 2, 2, 64, 16, 4, True, True, dict(std=4.0)),
    ("many", [1] * 40, list(range(1, 40 * 7, 7)), 3, 3, 64, 16, 16, True, True, {}),
    ("many_mixed", [1, 90, 1, 1, 200, 1, 0, 33], [64, 90, 300, 129, 400, 2, 77, 500], 8, 2, 64, 16, 16, True, True, {}),
    ("past_capacity", [5], [64], 2, 2, 64, 16, 4, True, True, dict(kv=[200])),
]


@pytest.mark.parametrize("hint", [False, True], ids=["", "max_new"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_attention_matches_the_definition(case, dtype, hint):
    name, new, kv, H, Hkv, d, P, k, key, value, kw = case
    kw = dict(kw)
    shared, std = kw.pop("shared", False), kw.pop("std", 1.0)
    x = make(new, kv, H, Hkv, d, P, dtype, k, key, value, shared, std, seed=len(name) + d, extra_rows=2)
    x["kv_len"] = np.asarray(kw.pop("kv", kv))
    got = call(x, k, max_new=max(new) if hint else 0, **kw)
    assert _rp().relattn_get_device_error() == 0
    check(x, got, k, **kw)


@pytest.mark.parametrize("new,kv,H,Hkv,d,k,key,value,kw", [
    # several tiles of a request per CTA and requests that end inside a CTA's share: pieces of both
    # kinds (the end of one request's keys, the beginning of the next's), one and two tiles of rows
    ([24, 3], [5000, 4100], 8, 8, 128, 0, False, False, {}),
    ([24, 3], [5000, 4100], 8, 8, 128, 64, True, False, {}),
    ([20, 9], [6100, 3000], 8, 8, 64, 16, True, True, {}),
    ([131], [3300], 8, 8, 128, 64, True, True, {}),
    ([131], [3300], 8, 8, 64, 16, True, True, dict(window=2000, sinks=200)),
    ([37], [4000], 32, 8, 128, 0, False, False, {}),
    ([1, 1, 1], [9000, 100, 7000], 16, 8, 128, 16, True, True, {}),
    ([1, 1, 1], [9000, 100, 7000], 8, 8, 64, 16, True, True, dict(window=3500, sinks=4))])
def test_long_keys_in_pieces(new, kv, H, Hkv, d, k, key, value, kw):
    x = make(new, kv, H, Hkv, d, 16, BF16, k, key, value, seed=sum(kv) + k)
    got = call(x, k, max_new=max(new), **kw)
    assert _rp().relattn_get_device_error() == 0
    check(x, got, k, **kw)


@pytest.mark.parametrize("new,kv,H,d", [([1] * 5, [700, 3, 90, 2000, 128], 4, 64), ([300, 20], [900, 40], 2, 128)])
def test_equal_calls_give_equal_bits(new, kv, H, d):
    x = make(new, kv, H, H, d, 16, BF16, 16, True, True)
    a = call(x, 16)
    for _ in range(3):
        assert torch.equal(call(x, 16), a)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,H,Hkv,d", [([1, 1], 4, 2, 64), ([150, 40], 4, 2, 64), ([1, 140], 2, 2, 128)])
def test_pages_behind_the_window_may_be_gone(new, H, Hkv, d, dtype):
    """Table entries that no token sees are not read: they hold wild numbers, and rows of seen
    pages that no token sees hold NaN."""
    kv, P, window, sinks = [1000, 777], 16, 100, 5
    x = make(new, kv, H, Hkv, d, P, dtype, 8, True, True)
    want = call(x, 8, window=window, sinks=sinks)
    y = dict(x)
    y["table"], y["k_pages"], y["v_pages"] = x["table"].copy(), x["k_pages"].clone(), x["v_pages"].clone()
    for b in range(2):
        first = kv[b] - new[b] + 1 - window      # the first key that the first token sees
        for pg in range(-(-kv[b] // P)):
            lo, hi = pg * P, pg * P + P
            for j in range(max(lo, sinks), min(hi, first)):
                y["k_pages"][x["table"][b, pg], :, j % P] = float("nan")
                y["v_pages"][x["table"][b, pg], :, j % P] = float("nan")
            if lo >= sinks and hi <= first:
                y["table"][b, pg] = -3 if pg % 2 else 2 ** 31 - 1
    assert torch.equal(call(y, 8, window=window, sinks=sinks), want)
    assert _rp().relattn_get_device_error() == 0
    check(x, want, 8, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [[1, 1], [150, 1]])
def test_a_page_outside_the_cache_counts_as_zeros(new, dtype):
    x = make(new, [300, 200], 2, 2, 64, 16, dtype, 4, True, True)
    x["table"][0, 3] = x["k_pages"].shape[0]
    x["table"][1, 0] = -1
    got = call(x, 4)
    assert _rp().relattn_get_device_error() == 1
    check(x, got, 4)


@pytest.mark.parametrize("new,H,Hkv,d", [([1, 1, 1], 8, 2, 64), ([140, 30, 1], 4, 2, 128)])
def test_spaced_queries_and_pages(new, H, Hkv, d):
    """Queries sliced out of a joint projection, keys and values out of a joint pool."""
    x = make(new, [300, 90, 700], H, Hkv, d, 16, BF16, 8, True, True)
    want = call(x, 8)
    T = x["q"].shape[0]
    wide = torch.full((T, H + 2 * Hkv, d), float("nan"), dtype=BF16, device=DEV)
    wide[:, :H] = x["q"].to(DEV)
    pool = torch.stack([x["k_pages"], x["v_pages"]], 1).to(DEV)
    wt = torch.full((3, x["table"].shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wt[:, :x["table"].shape[1]] = i32(x["table"])
    rp = _rp()
    got = rp.relattn_paged_fwd(wide[:, :H], pool[:, 0], pool[:, 1], wt[:, :x["table"].shape[1]], i32(x["q_start"]),
                               i32(x["kv_len"]), aK=x["aK"].to(DEV), aV=x["aV"].to(DEV), clip_k=8)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_lengths_that_lie_are_kept_in_bounds(dtype):
    """Offsets past the rows, descending offsets, negative lengths: nothing outside the arrays is
    touched, and requests with sound lengths are right."""
    x = make([4, 6], [50, 60], 2, 2, 64, 16, dtype, 4, True, True)
    x["kv_len"] = np.array([50, -5])
    got = call(x, 4).double().cpu().numpy()
    assert np.isfinite(got).all() and not got[4:].any()
    x["kv_len"] = np.array([50, 60])
    x["q_start"] = np.array([0, 4, 4000])          # 10 rows: the second request is given 6
    y = dict(x, q_start=np.array([0, 4, 10]))
    assert torch.equal(call(x, 4), call(y, 4))
    x["q_start"] = np.array([0, 4, 2])
    got = call(x, 4).double().cpu().numpy()
    assert np.isnan(got[4:]).all() and np.isfinite(got[:4]).all()


@pytest.mark.parametrize("new,kv,H,Hkv,d", [([9, 1, 40], [300, 90, 40], 8, 2, 64), ([20, 3], [900, 3], 4, 4, 128)])
def test_max_new_is_a_hint_only(new, kv, H, Hkv, d):
    """Requests with more new tokens than the hint says."""
    x = make(new, kv, H, Hkv, d, 16, BF16, 8, True, True)
    for hint in (1, 2, 5, 10 ** 6):
        check(x, call(x, 8, max_new=hint), 8)


@pytest.mark.parametrize("new,kv,H,d", [([1, 1], [700, 90], 4, 64), ([200, 3], [900, 40], 2, 128)])
def test_a_wait_that_runs_out_is_reported(new, kv, H, d):
    """The first queries are announced and never loaded, with the bound at 10^6 cycles: the kernels give
    up in order and say so, and the next call is right."""
    rp = _rp()
    x = make(new, kv, H, H, d, 16, BF16, 8, True, True)
    want = call(x, 8, max_new=max(new))
    rp.relattn_set_wait_limit(1000000)
    rp.relattn_debug_withhold_first_load(True)
    try:
        call(x, 8, max_new=max(new))
        torch.cuda.synchronize()
    finally:
        rp.relattn_debug_withhold_first_load(False)
        rp.relattn_set_wait_limit(2000000000)
    assert rp.relattn_get_device_error() == 4
    assert torch.equal(call(x, 8, max_new=max(new)), want)
    assert rp.relattn_get_device_error() == 0


# ------------------------------------------------------------------------------------ a server's steps
def test_steps_of_a_server_match_dense_attention():
    """Prompts, chunks and generated tokens through plan, append and attention for several steps,
    with lengths and the free list advanced in place; at the end every token's output equals the
    causal attention of its request over all of its tokens."""
    rp = _rp()
    H, Hkv, d, P, k, B, M = 4, 2, 64, 16, 8, 4, 24
    steps = [[40, 0, 130, 7], [1, 21, 1, 1], [1, 1, 100, 1], [1, 1, 1, 1], [0, 1, 1, 16], [1, 1, 1, 1]]
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g).to(BF16)
    N = 64
    kp = torch.full((N, Hkv, P, d), float("nan"), dtype=BF16, device=DEV)
    vp = kp.clone()
    aK, aV = rnd(Hkv, 2 * k + 1, d), rnd(Hkv, 2 * k + 1, d)
    lens, head = i32([0] * B), i32([0])
    table = i32(np.full((B, M), -1))
    free = i32(np.random.default_rng(1).permutation(N))
    tok = [[] for _ in range(B)]
    outs = [[] for _ in range(B)]
    for new in steps:
        T = sum(new)
        q, kx, vx = rnd(T, H, d), rnd(T, Hkv, d), rnd(T, Hkv, d)
        kv, qs, slots, _ = rp.relattn_paged_plan(lens, i32(new), table, free, head, P, T + 3, kv_len=lens,
                                                 free_head_out=head)
        pad = torch.full((3, Hkv, d), 7.0, dtype=BF16)      # a padded batch: slots -1
        rp.relattn_paged_append(torch.cat([kx, pad]).to(DEV), torch.cat([vx, pad]).to(DEV), slots, kp, vp)
        z = rp.relattn_paged_fwd(q.to(DEV), kp, vp, table, qs, kv, aK=aK.to(DEV), aV=aV.to(DEV), clip_k=k,
                                 max_new=max(new)).cpu()
        at = 0
        for b, n in enumerate(new):
            tok[b] += [(q[at + i], kx[at + i], vx[at + i]) for i in range(n)]
            outs[b] += [z[at + i] for i in range(n)]
            at += n
    assert rp.relattn_get_device_error() == 0
    import oracle
    rep = H // Hkv
    for b in range(B):
        st = lambda i, r: torch.stack([t[i] for t in tok[b]]).double().repeat_interleave(r, 1).transpose(0, 1)[None].numpy()
        t2 = lambda t: t.double().repeat_interleave(rep, 0).numpy()
        ref = oracle.relattn_fwd(st(0, 1), st(1, rep), st(2, rep), t2(aK), t2(aV), k, True, d ** -0.5)[0]
        got = torch.stack(outs[b]).double().numpy().transpose(1, 0, 2)
        tol = 1e-2 * np.abs(ref).max() + 1e-3
        assert np.abs(got - ref).max() <= tol


def test_a_captured_decoding_step_replays():
    """plan, append and attention of a decoding step in one CUDA graph, replayed: lengths and the
    free list advance in place, pages are taken when a row is full."""
    rp = _rp()
    H, Hkv, d, P, B, M, N = 4, 2, 64, 8, 3, 16, 40
    rnd = np.random.default_rng(5)
    mk = lambda *s: torch.from_numpy(rnd.standard_normal(s)).to(BF16).to(DEV)
    kp, vp = mk(N, Hkv, P, d), mk(N, Hkv, P, d)
    q, kx, vx = mk(B, H, d), mk(B, Hkv, d), mk(B, Hkv, d)
    lens, head, ones = i32([5, 0, 16]), i32([4]), i32([1, 1, 1])
    table = i32([[0] + [-1] * 15, [-1] * 16, [1, 2] + [-1] * 14])
    free = i32(np.arange(N))
    qs, slots = i32([0] * 4), i32([0] * 3)
    out = torch.empty((B, H, d), dtype=BF16, device=DEV)
    ws = torch.empty(rp.relattn_paged_workspace_size(H, Hkv, d), dtype=torch.uint8, device=DEV)

    def step():
        rp.relattn_paged_plan(lens, ones, table, free, head, P, B, kv_len=lens, q_start=qs, slots=slots,
                              free_head_out=head)
        rp.relattn_paged_append(kx, vx, slots, kp, vp)
        rp.relattn_paged_fwd(q, kp, vp, table, qs, lens, max_new=1, out=out, workspace=ws)

    keep = [t.clone() for t in (lens, head, table, kp, vp)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for dst, src in zip((lens, head, table, kp, vp), keep):
        dst.copy_(src)
    outs = []
    for i in range(20):
        q.copy_(mk(B, H, d))
        graph.replay()
        outs.append((q.clone(), lens.clone(), table.clone(), kp.clone(), vp.clone(), out.clone()))
    torch.cuda.synchronize()
    # pages taken: 5 + 20 tokens grow from 1 page to 4, 0 + 20 from 0 to 3, 16 + 20 from 2 to 5
    assert lens.tolist() == [25, 20, 36] and int(head) == 4 + 3 + 3 + 3
    for qv, ln, tb, kc, vc, z in outs:
        x = dict(q=qv.cpu(), k_pages=kc.cpu(), v_pages=vc.cpu(), table=tb.cpu().numpy(), q_start=np.arange(4),
                 kv_len=ln.cpu().numpy(), aK=None, aV=None)
        check(x, z, 0)


def test_two_streams_with_a_workspace_each():
    rp = _rp()
    xs = [make([1] * 6, [900, 33, 257, 128, 4000, 1], 4, 2, 64, 16, BF16, 8, True, True, seed=s) for s in (1, 2)]
    want = [call(x, 8) for x in xs]
    g = lambda t: t.to(DEV)
    args = [(g(x["q"]), g(x["k_pages"]), g(x["v_pages"]), i32(x["table"]), i32(x["q_start"]), i32(x["kv_len"]),
             g(x["aK"]), g(x["aV"])) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            got[i].append(rp.relattn_paged_fwd(*args[i], clip_k=8, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(z, want[i]) for z in got[i])


# ------------------------------------------------------------------------------------ calls in a row
@pytest.mark.parametrize("B,Hkv,d", [(19, 8, 128), (38, 8, 64), (2, 3, 64)])
def test_a_chain_of_calls_reads_finished_outputs(B, Hkv, d):
    # the first two give every block whole requests (152 or 304 equal shares): no pieces to join
    # between one call's attention and the next one's
    rp = _rp()
    x = make([1] * B, [3000] * B, Hkv, Hkv, d, 16, BF16, stale=False)
    g = lambda t: t.to(DEV)
    kp, vp, bt = g(x["k_pages"]), g(x["v_pages"]), i32(x["table"])
    qs, ln = i32(x["q_start"]), i32(x["kv_len"])
    ws = torch.empty(rp.relattn_paged_workspace_size(Hkv, Hkv, d), dtype=torch.uint8, device=DEV)

    def chain(sync):
        z = [g(x["q"])] + [torch.full((B, Hkv, d), float("nan"), dtype=BF16, device=DEV) for _ in range(12)]
        torch.cuda.synchronize()
        for i in range(12):
            rp.relattn_paged_fwd(z[i], kp, vp, bt, qs, ln, scale=4.0, max_new=1, out=z[i + 1], workspace=ws)
            if sync:
                torch.cuda.synchronize()
        z.append(z[-1] + 0)   # a kernel that is not one of these
        torch.cuda.synchronize()
        return z

    want = chain(True)
    assert all(bool(torch.isfinite(t).all()) for t in want)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))


@pytest.mark.parametrize("new,H,Hkv,d,k", [([1, 1], 16, 1, 128, 256), ([1, 1], 12, 1, 128, 140), ([9, 2], 1, 1, 128, 200),
                                           ([1, 1], 16, 1, 64, 256), ([1, 3], 4, 2, 128, 256)])
def test_generated_tokens_with_long_tables(new, H, Hkv, d, k):
    x = make(new, [700, 300], H, Hkv, d, 16, BF16, k, True, True, seed=k + d)
    got = call(x, k, max_new=max(new))
    assert _rp().relattn_get_device_error() == 0
    check(x, got, k)


def test_plan_refuses_a_length_past_31_bits():
    M = 2 ** 21 + 2
    free = np.arange(8)
    run_plan([2 ** 31 - 3], [5], 1024, M, free, 0, 8)
    run_plan([2 ** 31 - 3], [2], 1024, M, free, 0, 8, table=np.full((1, M), 7))


def test_plans_of_two_sizes_at_once():
    # both need more shared memory than a kernel has by default, and not the same amount
    import threading
    rp = _rp()
    fails = []

    def work(B, max_tokens):
        try:
            c, n = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
            bt = torch.zeros((B, 1), dtype=torch.int32, device=DEV)
            free, head = torch.arange(B, dtype=torch.int32, device=DEV), i32([0])
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            for _ in range(200):
                rp.relattn_paged_plan(c, n, bt, free, head, 8, max_tokens, stream=s)
            s.synchronize()
            assert torch.equal(bt[:, 0], free)
        except Exception as e:   # noqa: BLE001
            fails.append(e)

    for tokens in (8000, 16384):
        ts = [threading.Thread(target=work, args=(b, tokens)) for b in (4100 if tokens < 8192 else 16384, 7990)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
    assert not fails and rp.relattn_get_device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,off", [(36, 0), (12, 0), (64, 1), (128, 4), (40, 2)])
def test_joined_outputs_of_any_width_and_place(d, off, dtype):
    # long keys of few tokens, so that every item comes in pieces; outputs that start off the boundary
    # of the join's widest stores
    rp = _rp()
    new, kv, H, Hkv = [9, 1, 1], [2600, 700, 1], 4, 2
    x = make(new, kv, H, Hkv, d, 16, dtype, 5, True, True, seed=d)
    g = lambda t: t.to(DEV)
    T = sum(new)
    buf = torch.full((T * H * d + 2 * off,), float("nan"), dtype=dtype, device=DEV)
    out = buf[off:off + T * H * d].view(T, H, d)
    rp.relattn_paged_fwd(g(x["q"]), g(x["k_pages"]), g(x["v_pages"]), i32(x["table"]), i32(x["q_start"]),
                         i32(x["kv_len"]), aK=g(x["aK"]), aV=g(x["aV"]), clip_k=5, out=out)
    assert rp.relattn_get_device_error() == 0
    check(x, out, 5)
    assert bool(torch.isnan(buf[:off]).all()) and bool(torch.isnan(buf[off + T * H * d:]).all())


def test_results_dropped_early_keep_their_memory_until_written():
    # a call on a stream that is still busy; its results are dropped, and what is allocated next on
    # the current stream must not lie where that call will write
    rp = _rp()
    x = make([1] * 6, [900, 33, 257, 128, 400, 1], 4, 2, 64, 16, BF16, seed=3)
    g = lambda t: t.to(DEV)
    args = (g(x["q"]), g(x["k_pages"]), g(x["v_pages"]), i32(x["table"]), i32(x["q_start"]), i32(x["kv_len"]))
    B = 5000
    c, n = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    bt, free, head = i32(np.zeros((B, 1))), i32(np.arange(B)), i32([0])
    s = torch.cuda.Stream()
    rp.relattn_paged_fwd(*args)
    torch.cuda.synchronize()
    for call_it, shape, dtype in (
            (lambda: rp.relattn_paged_fwd(*args, stream=s), x["q"].shape, BF16),
            (lambda: rp.relattn_paged_plan(c, n, bt, free, head, 8, B, stream=s), (B,), torch.int32)):
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)   # some 50 ms
        call_it()
        kept = [torch.zeros(shape, dtype=dtype, device=DEV) for _ in range(6)]
        torch.cuda.synchronize()
        assert all(not bool(t.any()) for t in kept)


def test_memory_made_for_a_stream_is_not_in_use_elsewhere():
    # the current stream is busy and will still read temporaries that the caller has dropped; a call on
    # an idle stream must not write its results or its workspace there, nor lose them
    rp = _rp()
    x = make([1] * 6, [900, 33, 257, 128, 400, 1], 4, 2, 64, 16, BF16, seed=4)
    g = lambda t: t.to(DEV)
    args = (g(x["q"]), g(x["k_pages"]), g(x["v_pages"]), i32(x["table"]), i32(x["q_start"]), i32(x["kv_len"]))
    B = 5000
    c, n = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    bt, free, head = i32(np.zeros((B, 1))), i32(np.arange(B)), i32([0])
    s = torch.cuda.Stream()
    for call_it, sizes in (
            (lambda **kw: [rp.relattn_paged_fwd(*args, **kw)],
             [x["q"].numel() * 2, rp.relattn_paged_workspace_size(4, 2, 64)]),
            (lambda **kw: rp.relattn_paged_plan(c, n, bt, free, head, 8, B, **kw), [4 * B] * 4)):
        want = [t.clone() for t in call_it()]
        torch.cuda.synchronize()
        temporaries = [torch.full((b,), 77, dtype=torch.uint8, device=DEV) for b in sizes]
        torch.cuda._sleep(100_000_000)   # some 50 ms
        kept = [t.clone() for t in temporaries]
        del temporaries
        got = call_it(stream=s)
        torch.cuda.synchronize()
        assert all(bool((t == 77).all()) for t in kept)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------------------------ many slots
@pytest.mark.parametrize("path", ["generated", "chunks", "f32"])
@pytest.mark.parametrize("B,busy,keys", [
    (65, 0.7, 60), (129, 0.7, 60), (300, 0.5, 90), (1025, 0.3, 40),
    # a handful of long requests far apart: a block's share goes on behind a gap of idle slots
    (700, 0.004, 5000), (4100, 0.0008, 3000)])
def test_steps_over_many_slots(B, busy, keys, path):
    rng = np.random.default_rng(B)
    on = rng.random(B) < busy
    on[[0, B - 1]] = True
    new = np.where(on, rng.integers(1, 3, B), 0)
    if path != "generated":
        new[np.flatnonzero(on)[::7]] = 20          # more than one tile of rows in the f32 kernel
    kv = np.where(on, np.maximum(new, rng.integers(1, keys, B)), rng.integers(0, 9, B))
    kv[np.flatnonzero(on)[:3]] = keys
    x = make(new, kv, 4, 2, 64, 16, F32 if path == "f32" else BF16, 3, True, True, seed=B)
    got = call(x, 3, max_new=2 if path == "generated" else 0)
    assert _rp().relattn_get_device_error() == 0
    check(x, got, 3)


@pytest.mark.parametrize("path", ["generated", "chunks", "f32"])
def test_offsets_that_do_not_ascend_are_kept_in_bounds(path):
    # every other request is given all the rows: any of their outputs may stay, within the array
    rp = _rp()
    T, B, H, Hkv, d, P = 23, 40, 4, 2, 64, 16
    dtype = F32 if path == "f32" else BF16
    x = make([T], [3000], H, Hkv, d, P, dtype, stale=False)
    g = lambda t: t.to(DEV)
    buf = torch.full((T + 16, H, d), float("nan"), dtype=dtype, device=DEV)
    table = i32(np.repeat(x["table"], B, 0))
    rp.relattn_paged_fwd(g(x["q"]), g(x["k_pages"]), g(x["v_pages"]), table, i32([0, T] * (B // 2) + [0]), i32([3000] * B),
                         max_new=2 if path == "generated" else 0, out=buf[8:8 + T])
    # (the last request's rows end at 0: it has none, as have those that begin at T)
    assert bool(torch.isnan(buf[:8]).all()) and bool(torch.isnan(buf[8 + T:]).all())
    one = buf[8:8 + T].cpu()
    want = call(dict(x, kv_len=np.array([3000])), 0, max_new=2 if path == "generated" else 0).cpu()
    # the keys may be cut differently. sum p |v| < 1 (3000 keys): bf16 weights and outputs are each off
    # by 2^-8 of it on both sides; sums of 3000 fp32 terms and of the weights by 3000 x 2^-24 each
    tol = 4 * 2.0 ** -8 if dtype == BF16 else 4 * 3000 * 2.0 ** -24
    assert float((one.float() - want.float()).abs().max()) <= tol


# ------------------------------------------------------------------------------------ weights
def cancelling(H, d, keys, clip_k, terms, seed):
    """One token whose outputs nearly cancel: queries of one non-zero column, so that scores carry next
    to no error, and first values that take back what the other keys add up to. What is left are the
    errors of the weights."""
    x = make([1], [keys], H, H, d, 16, BF16, clip_k, terms, terms, seed=seed, stale=False)
    x["q"].zero_()
    x["q"][..., 0] = 4.0
    x["k_pages"].clamp_(-2.0, 2.0)
    x["k_pages"][x["table"][0, 0], :, 0, 0] = 2.5
    f = lambda t: None if t is None else t.double().numpy()
    v0 = x["v_pages"][x["table"][0, 0], :, 0]
    run = lambda: op.attend(f(x["q"]), f(x["k_pages"]), f(x["v_pages"]), x["table"], x["q_start"], x["kv_len"],
                            f(x["aK"]), f(x["aV"]), clip_k, 0, 0, 0.25)
    v0.zero_()
    rest = run()[0][0]
    v0.fill_(1.0)
    v0.copy_(torch.from_numpy(-rest / (run()[0][0] - rest)))
    return x, run()


@pytest.mark.parametrize("hint", [1, 16], ids=["8_rows", "16_rows"])
@pytest.mark.parametrize("terms", [False, True], ids=["plain", "terms"])
@pytest.mark.parametrize("d", [64, 128])
def test_generated_tokens_keep_their_weights(d, terms, hint):
    """The weights of generated tokens take part with 16 bits (two bf16 numbers), as do the table's
    bins; relattn_decode_fwd's are fp32."""
    keys, k = 40, 4
    x, (z, mass, size) = cancelling(8, d, keys, k, terms, d + hint)
    got = call(x, k, scale=0.25, max_new=hint)
    # a weight in two parts is off by 2^-8 x 2^-8; one product to a score; the tensor cores' sums may
    # drop bits where the unit rounds: twice the keys' share
    tol = op.tolerance(z, mass, size, 2 * (keys + k + 1), 1, 2.0 ** -8, 2.0 ** -16)
    bad = np.abs(got.double().cpu().numpy() - z) - tol
    assert bad.max() <= 0, (bad.max(), tol.max())


# ------------------------------------------------------------------------------------ one slot twice
@pytest.mark.parametrize("T,d", [(4, 64), (2000, 128)])
def test_two_tokens_of_one_slot(T, d):
    """Such a row is left with a mixture of the tokens' numbers, and every other row is right."""
    rp = _rp()
    rnd = torch.Generator().manual_seed(T)
    k, v = (torch.randn((T, 2, d), generator=rnd).to(BF16) for _ in range(2))
    N, P = T // 8 + 1, 8
    slots = np.random.default_rng(T).permutation(N * P)[:T]
    slots[-1] = slots[0]
    kp, vp = (torch.zeros((N, 2, P, d), dtype=BF16, device=DEV) for _ in range(2))
    rp.relattn_paged_append(k.to(DEV), v.to(DEV), i32(slots), kp, vp)
    for x, pages in ((k, kp.cpu()), (v, vp.cpu())):
        rows = pages.transpose(1, 2).reshape(-1, 2, d)
        assert torch.equal(rows[slots[1:-1]], x[1:-1])
        twice = rows[slots[0]]
        assert bool(((twice == x[0]) | (twice == x[-1])).all())
        left = np.setdiff1d(np.arange(N * P), slots)
        assert not bool(rows[left].any())


# ------------------------------------------------------------------------------------ long tables
@pytest.mark.parametrize("new,kv,H,Hkv,k,key,value,kw", [
    # at d = 128 the R rows of clip_k >= 98 leave room for one query tile per item, not two
    ([70, 3], [400, 900], 6, 2, 97, True, True, {}),
    ([70, 3], [400, 900], 6, 2, 98, True, True, {}),
    ([70, 3], [400, 900], 6, 2, 127, True, True, {}),
    ([300, 1], [300, 700], 2, 2, 98, True, False, {}),
    ([300, 1], [300, 700], 2, 2, 127, False, True, {}),
    ([131], [3300], 8, 8, 127, True, True, {}),
    ([131], [3300], 8, 8, 98, True, True, dict(window=2000, sinks=200)),
    ([20, 37], [6100, 4000], 32, 8, 127, True, True, {}),
    ([200], [260], 2, 1, 127, True, True, dict(window=60, sinks=3))])
def test_chunks_with_long_tables(new, kv, H, Hkv, k, key, value, kw):
    x = make(new, kv, H, Hkv, 128, 16, BF16, k, key, value, seed=sum(kv) + k, extra_rows=1)
    got = call(x, k, max_new=max(new), **kw)
    assert _rp().relattn_get_device_error() == 0
    check(x, got, k, **kw)


# ------------------------------------------------------------------------------------ long prompts
@pytest.mark.parametrize("new,kv,H,Hkv,d,k,key,value,dtype,kw", [
    ([2100], [2100], 2, 1, 128, 64, True, False, BF16, {}),
    ([1900, 1], [2500, 1000], 2, 2, 64, 16, True, True, BF16, dict(window=700, sinks=20)),
    ([1200], [1300], 2, 1, 64, 16, True, True, F32, {}),
    ([1], [40000], 16, 4, 128, 16, True, True, BF16, {}),
    ([40], [33000], 2, 1, 64, 0, False, False, BF16, {}),
    ([1], [40000], 4, 2, 64, 16, True, True, F32, {})])
def test_long_requests(new, kv, H, Hkv, d, k, key, value, dtype, kw):
    x = make(new, kv, H, Hkv, d, 64, dtype, k, key, value, seed=sum(kv) + k)
    got = call(x, k, max_new=max(new), **kw)
    assert _rp().relattn_get_device_error() == 0
    check(x, got, k, **kw)


# ------------------------------------------------------------------------------------ which kernel
def ran_on_tensor_cores(x, k, max_new, **kw):
    """The tensor-core kernels heed the hook that withholds the first queries, the SIMT kernel does
    not: its call is right and reports nothing."""
    rp = _rp()
    rp.relattn_set_wait_limit(1000000)
    rp.relattn_debug_withhold_first_load(True)
    try:
        call(x, k, max_new=max_new, **kw)
        torch.cuda.synchronize()
    finally:
        rp.relattn_debug_withhold_first_load(False)
        rp.relattn_set_wait_limit(2000000000)
    return rp.relattn_get_device_error() == 4


@pytest.mark.parametrize("key,value", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,H,Hkv", [(1, 4, 4), (1, 16, 1), (60, 4, 2)])
def test_bf16_runs_on_the_tensor_cores(new, H, Hkv, d, key, value):
    # (a variant compiled to another register count would move to the SIMT kernel)
    x = make([new], [200], H, Hkv, d, 16, BF16, 16, key, value)
    assert ran_on_tensor_cores(x, 16, new)


@pytest.mark.parametrize("new,d,P,k,tensor", [
    (60, 128, 16, 127, True), (60, 128, 16, 128, False), (60, 80, 16, 16, False), (60, 64, 4, 16, False),
    (60, 64, 8, 16, True), (1, 128, 16, 256, True), (1, 96, 16, 16, False)])
def test_the_documented_shapes_run_on_the_tensor_cores(new, d, P, k, tensor):
    x = make([new], [200], 4, 2, d, P, BF16, k, True, True)
    assert ran_on_tensor_cores(x, k, new) == tensor


@pytest.mark.parametrize("path", ["generated", "chunks", "f32"])
def test_a_table_for_very_long_requests(path):
    """A table whose rows could hold 2^31 keys: the measure of the work may pass 31 bits, so every path
    takes the SIMT kernel's 64-bit one, whatever the lengths are."""
    rp = _rp()
    B, H, P, M, d = 40, 4, 1024, 1 << 21, 64
    rng = np.random.default_rng(5)
    new = rng.integers(1, 3 if path == "generated" else 30, B)
    kv = new + rng.integers(0, 2000, B)
    x = make(new, kv, H, H, d, P, F32 if path == "f32" else BF16, 8, True, True, seed=2)
    wide = torch.full((B, M), -7, dtype=torch.int32, device=DEV)
    wide[:, :x["table"].shape[1]] = i32(x["table"])
    g = lambda t: t.to(DEV)
    args = (g(x["q"]), g(x["k_pages"]), g(x["v_pages"]), wide, i32(x["q_start"]), i32(x["kv_len"]))
    kw = dict(aK=g(x["aK"]), aV=g(x["aV"]), clip_k=8, max_new=2 if path == "generated" else 0)
    rp.relattn_set_wait_limit(1000000)
    rp.relattn_debug_withhold_first_load(True)
    try:
        got = rp.relattn_paged_fwd(*args, **kw)
        torch.cuda.synchronize()
    finally:
        rp.relattn_debug_withhold_first_load(False)
        rp.relattn_set_wait_limit(2000000000)
    assert rp.relattn_get_device_error() == 0
    check(x, got, 8)


def test_a_step_in_which_a_request_is_left_out():
    """The status says so, and the others' outputs are right."""
    rp = _rp()
    H, Hkv, d, P = 4, 2, 64, 16
    new, cached = np.array([5, 40, 3]), np.array([20, 0, 31])
    x = make(new, cached + new, H, Hkv, d, P, BF16, 8, True, True, stale=False)
    table = x["table"].copy()
    g = lambda t: t.to(DEV)
    bt, lens, head = i32(table), i32(cached), i32([0])
    # the first request's page has room (20 + 5 of 32), the others want three pages and one: none is free
    kv, qs, slots, _ = rp.relattn_paged_plan(lens, i32(new), bt, i32([]), head, P, int(new.sum()))
    assert rp.relattn_get_device_error() == 1
    assert kv.tolist() == [25, 0, 31] and qs.tolist() == [0, 5, 45, 48]
    assert (slots[5:] == -1).all() and (slots[:5] >= 0).all()
    z = rp.relattn_paged_fwd(g(x["q"]), g(x["k_pages"]), g(x["v_pages"]), bt, qs, kv, aK=g(x["aK"]), aV=g(x["aV"]),
                             clip_k=8)
    assert rp.relattn_get_device_error() == 0
    one = dict(x, q=x["q"][:5], table=table[:1], q_start=np.array([0, 5]), kv_len=np.array([25]))
    check(one, z[:5], 8)
