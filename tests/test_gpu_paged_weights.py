"""The attention weights of cached keys on the GPU, and the log-sum-exp that they need, against
oracle/paged.py in 64 bits and within the bound that it derives from fp32 arithmetic."""
import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.test_gpu_paged import make

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


def args_of(x):
    return dict(q=f64(x["q"]), k_pages=f64(x["k_pages"]), table=x["table"], q_start=x["q_start"], kv_len=x["kv_len"],
                aK=f64(x["aK"]))


def on_gpu(x):
    d = {k: x[k].to(DEV) if x[k] is not None else None for k in ("q", "k_pages", "v_pages", "aK", "aV")}
    return dict(d, table=i32(x["table"]), q_start=i32(x["q_start"]), kv_len=i32(x["kv_len"]))


def check(x, clip_k=0, window=0, sinks=0, scale=None, accumulate=True, max_new=0, spaced=False, seed=0, stream=None):
    rp = _rp()
    N, Hkv, P, d = x["k_pages"].shape
    scale = d ** -0.5 if scale is None else scale
    a = args_of(x)
    lse = op.log_sum(**a, clip_k=clip_k, window=window, sinks=sinks, scale=scale)[0].astype(np.float32)
    rng = np.random.default_rng(seed)
    mass = rng.random((N, Hkv, P)).astype(np.float32) * 3
    want, bound = op.weights(**a, clip_k=clip_k, window=window, sinks=sinks, scale=scale, lse=lse.astype(np.float64),
                             mass=mass.astype(np.float64), accumulate=accumulate)
    g = on_gpu(x)
    q = g["q"]
    T, H, _ = q.shape
    if spaced:   # slices of a joint projection; masses with room between the pages
        wide = torch.zeros((T, H + 2, d), dtype=q.dtype, device=DEV)
        wide[:, 1:H + 1] = q
        q = wide[:, 1:H + 1]
        room = torch.full((N, Hkv + 1, P), 7.0, device=DEV)
        m = room[:, :Hkv]
        m.copy_(torch.from_numpy(mass))
    else:
        m = torch.from_numpy(mass).to(DEV)
    run = lambda m: rp.relattn_paged_weights(
        q, g["k_pages"], g["table"], g["q_start"], g["kv_len"], torch.from_numpy(lse).to(DEV), m, aK=g["aK"],
        clip_k=clip_k, window=window, sinks=sinks, scale=scale, accumulate=accumulate, max_new=max_new)
    again = m.clone()
    assert run(m) is m
    assert rp.relattn_get_device_error() == 0
    got = f64(m)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.abs(got - want)[bad].max(), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
    if spaced:
        assert (room[:, Hkv] == 7.0).all()
    assert torch.equal(run(again), m)    # the same bits
    return want


# ------------------------------------------------------------------------------------ generated tokens
@pytest.mark.parametrize("H,Hkv,d,P", [(4, 4, 64, 16), (8, 2, 128, 8), (16, 2, 64, 128), (16, 1, 128, 64), (3, 1, 64, 256),
                                       (10, 2, 128, 32)])
@pytest.mark.parametrize("clip_k,key,window,sinks", [(0, False, 0, 0), (16, True, 0, 0), (200, True, 0, 0), (0, True, 0, 0),
                                                     (5, True, 100, 3), (0, False, 64, 130), (1, True, 1, 0)])
def test_one_token_each(H, Hkv, d, P, clip_k, key, window, sinks):
    kv = [1, 2, 127, 128, 129, 500, 0, 777, 40]
    new = [1] * 6 + [0] + [1] * 2
    x = make(new, kv, H, Hkv, d, P, BF16, clip_k, key=key, seed=H + P)
    check(x, clip_k, window, sinks, max_new=1)
    check(x, clip_k, window, sinks, max_new=1, accumulate=False, spaced=True)


@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_a_few_tokens_each(g):
    new, kv = [3, 2, 0, 1, 4], [300, 2, 50, 90, 4]
    for d in (64, 128):
        check(make(new, kv, 2 * g, 2, d, 16, BF16, 7, key=True, seed=g), 7, max_new=4)
        check(make(new, kv, 2 * g, 2, d, 16, BF16, 7, key=True, seed=g), 7, window=20, sinks=2, max_new=4)


@pytest.mark.parametrize("max_new", [1, 2, 16])
def test_any_max_new_is_right(max_new):
    """More rows than the kernel for generated tokens takes at once: the rows come in groups."""
    new, kv = [40, 1, 17], [300, 260, 17]
    x = make(new, kv, 3, 3, 64, 16, BF16, 20, key=True, seed=max_new)
    check(x, 20, max_new=max_new)
    check(x, 20, window=33, sinks=5, max_new=max_new)
    check(make(new, kv, 6, 3, 128, 8, BF16, seed=1), max_new=max_new)


# ------------------------------------------------------------------------------------ chunks and prompts
@pytest.mark.parametrize("H,Hkv,d,P", [(4, 4, 64, 16), (8, 2, 128, 8), (3, 1, 64, 64), (10, 2, 64, 32), (48, 1, 128, 16),
                                       (2, 2, 128, 256)])
@pytest.mark.parametrize("clip_k,key,window,sinks", [(0, False, 0, 0), (16, True, 0, 0), (127, True, 0, 0), (0, True, 0, 0),
                                                     (5, True, 100, 3), (64, True, 40, 200), (0, False, 1, 0)])
def test_chunks(H, Hkv, d, P, clip_k, key, window, sinks):
    new = [17, 130, 1, 0, 64] if H < 48 else [5, 30, 1, 0, 12]
    kv = [17, 400, 300, 9, 257]
    x = make(new, kv, H, Hkv, d, P, BF16, clip_k, key=key, seed=H + P)
    check(x, clip_k, window, sinks)
    check(x, clip_k, window, sinks, accumulate=False, spaced=True)


@pytest.mark.parametrize("g", [1, 5, 128])
def test_long_prompts(g):
    n = {1: 700, 5: 150, 128: 9}[g]
    x = make([n, 3], [n, 600], g, 1, 128, 32, BF16, 30, key=True, seed=g)
    check(x, 30)
    check(x, 30, window=256, sinks=4)


def test_rows_of_the_next_request_and_behind_the_last_may_hold_anything():
    x = make([20, 3], [200, 150], 4, 2, 64, 16, BF16, 4, key=True, extra_rows=90)
    x["q"][23:] = float("nan")
    check(x, 4)
    x = make([130, 40], [200, 150], 1, 1, 64, 16, BF16, 4, key=True)
    x["q"][130:] = float("inf")
    x["kv_len"] = np.array([200, 0])      # the second request's rows see no key
    check(x, 4)


# ------------------------------------------------------------------------------------ the SIMT units
@pytest.mark.parametrize("dtype,H,Hkv,d,P", [(F32, 4, 2, 64, 16), (F32, 3, 3, 33, 1), (F32, 40, 1, 128, 8), (BF16, 4, 2, 80, 16),
                                             (BF16, 4, 4, 64, 4), (BF16, 2, 1, 7, 2), (F32, 2, 2, 1, 32)])
@pytest.mark.parametrize("clip_k,key,window,sinks", [(0, False, 0, 0), (16, True, 0, 0), (150, True, 50, 3), (33, True, 7, 0)])
def test_simt(dtype, H, Hkv, d, P, clip_k, key, window, sinks):
    new, kv = [1, 40, 0, 7], [300, 40, 9, 131]
    x = make(new, kv, H, Hkv, d, P, dtype, clip_k, key=key, seed=H + P)
    check(x, clip_k, window, sinks)
    check(x, clip_k, window, sinks, accumulate=False, spaced=True, max_new=1)


def test_wide_clips_of_chunks():
    x = make([60, 2], [200, 300], 2, 2, 64, 16, BF16, 200, key=True)
    check(x, 200)


# ------------------------------------------------------------------------------------ odd requests
@pytest.mark.parametrize("d,dtype,max_new", [(64, BF16, 3), (64, BF16, 0), (48, F32, 0)])
def test_tokens_without_a_position_and_long_lengths(d, dtype, max_new):
    x = make([3, 3, 2], [2, 0, 40], 2, 1, d, 16, dtype, 2, key=True)
    check(x, 2, max_new=max_new)
    x["kv_len"] = np.array([2, 0, 1000])     # past the table row: the tokens are its last
    M = x["table"].shape[1]
    x["table"] = np.concatenate([x["table"][:2], np.arange(M)[None]])
    x["k_pages"][x["k_pages"] != x["k_pages"]] = 0.5
    keep = slice(2, 3)   # (its pages are shared with the others': look at it alone)
    y = dict(x, table=x["table"][keep], kv_len=x["kv_len"][keep], q_start=np.array([0, 2]))
    check(y, 2, max_new=max_new)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    for max_new, new in ((1, 1), (0, 30)):
        check(make([new] * 2, [100, 45], 4, 2, 64, 16, BF16, 4, key=True), 4, scale=scale, max_new=max_new)


@pytest.mark.parametrize("max_new,dtype", [(1, BF16), (0, BF16), (0, F32)])
def test_pages_outside_the_cache(max_new, dtype):
    rp = _rp()
    x = make([1], [60], 2, 2, 64, 16, dtype)
    x["table"][0, 1] = 10 ** 6
    g = on_gpu(x)
    N = x["k_pages"].shape[0]
    m = torch.ones((N, 2, 16), device=DEV)
    rp.relattn_paged_weights(g["q"], g["k_pages"], g["table"], g["q_start"], g["kv_len"], torch.zeros((1, 2), device=DEV),
                             m, max_new=max_new)
    assert rp.relattn_get_device_error() == 1
    touched = {int(p) for p in x["table"][0] if 0 <= p < N}
    for p in range(N):
        assert (p in touched) or bool((m[p] == 1).all())


@pytest.mark.parametrize("max_new,dtype", [(1, BF16), (0, BF16), (0, F32)])
@pytest.mark.parametrize("q_start", [[0, 12, 3, 9, -4, 12], [12, 0, 12, 0, 12, 0], [5, 4, 3, 2, 1, 0], [0, 1, 0, 1, 0, 1],
                                     [-9, 99, -9, 99, -9, 99]])
def test_offsets_that_are_not_ascending_end_and_stay_within_the_arrays(max_new, dtype, q_start):
    rp = _rp()
    x = make([3, 2, 2, 4, 1], [30, 90, 40, 12, 70], 4, 2, 64, 16, dtype, 3, key=True)
    g = on_gpu(x)
    N = x["k_pages"].shape[0]
    for T in (12, 2):
        room = torch.full((N + 4, 2, 16), 3.0, device=DEV)
        rp.relattn_paged_weights(g["q"][:T], g["k_pages"].nan_to_num(), g["table"].clamp(0, N - 1), i32(q_start), g["kv_len"],
                                 torch.zeros((T, 4), device=DEV), room[2:-2], aK=g["aK"], clip_k=3, max_new=max_new)
        assert rp.relattn_get_device_error() == 0
        assert bool((room[:2] == 3).all()) and bool((room[-2:] == 3).all())


def test_no_tokens():
    rp = _rp()
    x = make([1], [60], 2, 2, 64, 16, BF16)
    g = on_gpu(x)
    m = torch.ones((x["k_pages"].shape[0], 2, 16), device=DEV)
    rp.relattn_paged_weights(g["q"][:0], g["k_pages"], g["table"], i32([0, 0]), g["kv_len"], torch.zeros((0, 2), device=DEV), m)
    assert bool((m == 1).all())


# ------------------------------------------------------------------------------------ log-sum-exp
@pytest.mark.parametrize("dtype,d,P,max_new", [(BF16, 64, 16, 1), (BF16, 128, 16, 1), (BF16, 64, 16, 0), (BF16, 128, 16, 0),
                                               (F32, 64, 16, 0), (BF16, 80, 4, 0)])
@pytest.mark.parametrize("terms,window,sinks", [((False, False), 0, 0), ((True, True), 0, 0), ((True, False), 50, 3)])
def test_lse_of_the_forward(dtype, d, P, max_new, terms, window, sinks):
    rp = _rp()
    new = [1] * 5 if max_new else [1, 200, 3, 40, 0]
    kv = [1, 3000, 0, 45, 700]
    clip_k = 9 if any(terms) else 0
    x = make(new, kv, 4, 2, d, P, dtype, clip_k, key=terms[0], value=terms[1], extra_rows=2)
    a = args_of(x)
    lse, size = op.log_sum(**a, clip_k=clip_k, window=window, sinks=sinks, scale=d ** -0.5)
    g = on_gpu(x)
    kw = dict(aK=g["aK"], aV=g["aV"], clip_k=clip_k, window=window, sinks=sinks, max_new=max_new)
    call = (g["q"], g["k_pages"], g["v_pages"], g["table"], g["q_start"], g["kv_len"])
    got = torch.full(lse.shape, 5.0, device=DEV)
    T = sum(new)
    plain = rp.relattn_paged_fwd(*call, **kw)
    out = rp.relattn_paged_fwd(*call, **kw, lse=got)
    assert torch.equal(plain[:T], out[:T])
    got = f64(got)
    assert (got[T:] == 5.0).all()
    u = 2.0 ** -24
    tol = 4.0 * (d + 6) * u * size + 2.0 ** -20 + 2.0 * max(kv) * u + 8.0 * u * np.abs(np.where(np.isinf(lse), 0, lse))
    with np.errstate(invalid="ignore"):
        same = (got[:T] == lse[:T]) | (np.abs(got - lse)[:T] <= tol[:T])
    assert same.all()
    out2, lse2 = rp.relattn_paged_fwd_lse(*call, **kw)
    assert torch.equal(out2[:T], out[:T]) and np.array_equal(f64(lse2)[:T], got[:T])


@pytest.mark.parametrize("offset,stride", [(1, 0), (0, 1), (2, 3)])
@pytest.mark.parametrize("max_new,new", [(1, [1, 1, 1]), (0, [40, 1, 130])])
def test_masses_on_any_boundary(offset, stride, max_new, new):
    """Masses that no 16-byte copy may take."""
    rp = _rp()
    kv, d, k = [300, 129, 200], 64, 5
    x = make(new, kv, 4, 2, d, 16, BF16, k, key=True)
    N = x["k_pages"].shape[0]
    a = args_of(x)
    lse = op.log_sum(**a, clip_k=k, window=0, sinks=0, scale=0.125)[0].astype(np.float32)
    mass = np.random.default_rng(1).random((N, 2, 16)).astype(np.float32)
    want, bound = op.weights(**a, clip_k=k, window=0, sinks=0, scale=0.125, lse=lse.astype(np.float64),
                             mass=mass.astype(np.float64), accumulate=True)
    room = torch.full((offset + N * (32 + stride) + 8,), 7.0, device=DEV)
    m = room[offset:offset + N * (32 + stride)].view(N, 32 + stride)[:, :32].unflatten(1, (2, 16))
    m.copy_(torch.from_numpy(mass))
    g = on_gpu(x)
    rp.relattn_paged_weights(g["q"], g["k_pages"], g["table"], g["q_start"], g["kv_len"], torch.from_numpy(lse).to(DEV), m,
                             aK=g["aK"], clip_k=k, scale=0.125, max_new=max_new)
    assert rp.relattn_get_device_error() == 0
    assert (np.abs(f64(m) - want) <= bound).all()
    rest = room.clone()
    rest[offset:offset + N * (32 + stride)].view(N, 32 + stride)[:, :32] = 7.0
    assert bool((rest == 7.0).all())


@pytest.mark.parametrize("max_new,new", [(1, 1), (0, 40)])
@pytest.mark.parametrize("key", [False, True])
def test_a_wait_that_runs_out(max_new, new, key):
    """Loads that never come: the kernel gives up, says so, and the next call is right."""
    rp = _rp()
    x = make([new] * 3, [900, 500, 100], 4, 2, 64, 16, BF16, 4, key=key)
    g = on_gpu(x)
    m = torch.zeros(x["k_pages"].shape[:3], device=DEV)
    lse = torch.zeros((3 * new, 4), device=DEV)
    try:
        rp.relattn_set_wait_limit(2_000_000)
        rp.relattn_debug_withhold_first_load(1)
        rp.relattn_paged_weights(g["q"], g["k_pages"], g["table"], g["q_start"], g["kv_len"], lse, m, aK=g["aK"], clip_k=4 * key,
                                 max_new=max_new)
        assert rp.relattn_get_device_error() == 4
    finally:
        rp.relattn_debug_withhold_first_load(0)
        rp.relattn_set_wait_limit(2_000_000_000)
    check(x, 4 * key, max_new=max_new)


# ------------------------------------------------------------------------------------ together
def test_a_chat_that_is_cut_again_and_again():
    """plan, append, attend, weights and evict as a server runs them, a captured decoding step replayed; the
    cache afterwards against the oracle's, its masses within what their sums leave open."""
    rp = _rp()
    P, M, H, Hkv, d, k = 8, 24, 8, 2, 64, 6
    g = torch.Generator(device=DEV).manual_seed(4)
    rnd = lambda *s: torch.randn(s, device=DEV, generator=g)
    N, B = 90, 3
    free, head = i32(np.arange(N)), i32([0])
    kv, table = i32([0] * B), torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    kp, vp = rnd(N, Hkv, P, d).to(BF16), rnd(N, Hkv, P, d).to(BF16)
    mass = torch.full((N, Hkv, P), float("nan"), device=DEV)
    aK, aV = rnd(Hkv, 2 * k + 1, d).to(BF16), rnd(Hkv, 2 * k + 1, d).to(BF16)
    budget, limit, sinks, recent = 64, 70, 2, 10
    ref = dict(kv=np.zeros(B, dtype=int), table=np.full((B, M), -1), free=np.arange(N), head=0, k=f64(kp), v=f64(vp),
               mass=np.zeros((N, Hkv, P)), slack=np.zeros((N, Hkv, P)))

    def step(new_len, T, q, kn, vn, max_new):
        lens, starts, slots, _ = rp.relattn_paged_plan(kv, new_len, table, free, head, P, T, kv_len=kv, free_head_out=head)
        rp.relattn_paged_append(kn, vn, slots, kp, vp)
        out, lse = rp.relattn_paged_fwd_lse(q, kp, vp, table, starts, kv, aK=aK, aV=aV, clip_k=k, max_new=max_new)
        rp.relattn_paged_weights(q, kp, table, starts, kv, lse, mass, aK=aK, clip_k=k, max_new=max_new)
        rp.relattn_paged_evict(kv, table, kp, vp, mass, budget, limit=limit, sinks=sinks, recent=recent, free_pages=free,
                               free_head=head, kv_len_out=kv, free_head_out=head)
        return out

    def ref_step(new, q, kn, vn):
        r = ref
        r["table"], r["kv"], starts, slots, r["head"], ok = op.plan(r["kv"], new, r["table"], r["free"], r["head"], P, sum(new))
        assert ok
        r["k"], r["v"] = op.append(f64(kn), f64(vn), slots, r["k"], r["v"])
        a = (f64(q), r["k"], r["table"], starts, r["kv"], f64(aK), k, 0, 0, d ** -0.5)
        lse, size = op.log_sum(*a)
        fresh = np.zeros_like(r["mass"])
        sums, bound = op.weights(*a, lse, fresh, True)
        r["mass"], _ = op.weights(*a, lse, r["mass"], True)
        # a weight is off by its own bound and by what the log-sum-exp may be
        off = 4.0 * (d + 6) * 2.0 ** -24 * size.max() + 2.0 ** -18
        new_slots = np.zeros(r["mass"].shape, dtype=bool)
        for s in slots:
            new_slots[s // P, :, s % P] = True
        r["slack"] = np.where(new_slots, 0, r["slack"]) + bound + 2 * off * sums + 2.0 ** -22 * np.abs(r["mass"])
        z, spread, size = op.attend(f64(q), r["k"], r["v"], r["table"], starts, r["kv"], f64(aK), f64(aV), k, 0, 0, d ** -0.5)
        return z, op.tolerance(z, spread, size, int(r["kv"].max()), d, 2.0 ** -8, 2.0 ** -8)

    def ref_cut():
        """The GPU's choice has to be one that the masses allow: its kept keys, checked against the bounds."""
        r = ref
        before = r["kv"].copy()
        out = op.evict(before, r["table"], r["k"], r["v"], r["mass"], budget, limit, sinks, recent, r["free"], r["head"])
        slack = op.evict(before, r["table"], r["k"], r["v"], r["mass"], budget, limit, sinks, recent)
        # the order of two masses is certain only where their bounds do not meet
        at = lambda m, b, h, n: np.array([m[r["table"][b, j // P], h, j % P] for j in range(n)])
        for b, n in enumerate(before):
            for h in range(Hkv if n > limit else 0):
                m, s = at(r["mass"], b, h, n), at(r["slack"], b, h, n)
                order = np.argsort(-m[sinks:n - recent], kind="stable") + sinks
                c = budget - sinks - recent
                assert m[order[c - 1]] - s[order[c - 1]] > m[order[c]] + s[order[c]], "the inputs leave it open"
        moved = op.evict(before, r["table"], r["k"], r["v"], r["slack"] * 0 + r["mass"], budget, limit, sinks, recent)
        # the slack moves with its key: rows of the masses are told apart by their place
        tag = np.arange(r["mass"].size, dtype=float).reshape(r["mass"].shape)
        places = op.evict(before, r["table"], r["k"], np.broadcast_to(tag[..., None], r["k"].shape).copy(), r["mass"], budget,
                          limit, sinks, recent)[2][..., 0].astype(int)
        r["slack"] = r["slack"].reshape(-1)[places]
        r["kv"], r["k"], r["v"], r["mass"], r["free"], r["head"] = out
        assert moved is not None and slack is not None

    def agree(out, z, tol):
        assert rp.relattn_get_device_error() == 0
        assert (np.abs(f64(out) - z) <= tol).all()
        assert kv.tolist() == ref["kv"].tolist() and int(head) == ref["head"]
        assert np.array_equal(table.cpu().numpy(), ref["table"]) and np.array_equal(free.cpu().numpy(), ref["free"])
        for b in range(B):
            for j in range(ref["kv"][b]):
                page = ref["table"][b, j // P]
                assert np.array_equal(f64(kp[page, :, j % P]), ref["k"][page, :, j % P])
                assert np.array_equal(f64(vp[page, :, j % P]), ref["v"][page, :, j % P])
                d_ = np.abs(f64(mass[page, :, j % P]) - ref["mass"][page, :, j % P])
                assert (d_ <= ref["slack"][page, :, j % P] + 1e-30).all()

    new = [50, 61, 3]
    T = sum(new)
    mk = lambda T: (rnd(T, H, d).to(BF16), rnd(T, Hkv, d).to(BF16), rnd(T, Hkv, d).to(BF16))
    q, kn, vn = mk(T)
    out = step(i32(new), T, q, kn, vn, 0)
    z, tol = ref_step(new, q, kn, vn)
    ref_cut()
    agree(out, z, tol)
    q, kn, vn = mk(B)
    ones = i32([1] * B)
    step(ones, B, q, kn, vn, 1)     # the capture must not be the first call
    z, tol = ref_step([1] * B, q, kn, vn)
    ref_cut()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ones, B, q, kn, vn, 1)
    for _ in range(14):
        for t, s in zip((q, kn, vn), mk(B)):
            t.copy_(s)
        graph.replay()
        z, tol = ref_step([1] * B, q, kn, vn)
        ref_cut()
        agree(out, z, tol)


def test_two_streams_at_once():
    rp = _rp()
    xs = [make([200, 30], [900, 700], 4, 2, 128, 16, BF16, 8, key=True, seed=s) for s in range(2)]
    gs = [on_gpu(x) for x in xs]
    lses = [torch.from_numpy(op.log_sum(**args_of(x), clip_k=8, window=0, sinks=0, scale=128 ** -0.5)[0]).float().to(DEV)
            for x in xs]
    run = lambda g, l, m, s: rp.relattn_paged_weights(g["q"], g["k_pages"], g["table"], g["q_start"], g["kv_len"], l, m,
                                                      aK=g["aK"], clip_k=8, accumulate=False, stream=s)
    ms = [torch.zeros(x["k_pages"].shape[:3], device=DEV) for x in xs]
    want = [run(g, l, m.clone(), None) for g, l, m in zip(gs, lses, ms)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for g, l, m, s in zip(gs, lses, ms, streams):
        run(g, l, m, s)
    torch.cuda.synchronize()
    for m, w in zip(ms, want):
        assert torch.equal(m, w)


@pytest.mark.parametrize("max_new,new,dtype", [(1, 1, BF16), (1, 30, BF16), (0, 40, BF16), (0, 40, F32)])
@pytest.mark.parametrize("key", [False, True])
def test_rows_marked_as_without_keys_add_nothing(max_new, new, dtype, key):
    """A log-sum-exp of -infinity is that of a row without keys, whatever the row sees."""
    rp = _rp()
    k = 5 * key
    x = make([new, new, 1], [300, 129, 200], 4, 2, 64, 16, dtype, k, key=key)
    N = x["k_pages"].shape[0]
    a = args_of(x)
    lse = op.log_sum(**a, clip_k=k, window=0, sinks=0, scale=0.125)[0].astype(np.float32)
    none = np.random.default_rng(2).random(lse.shape) < 0.5
    none[0], none[-1] = True, False
    mass = np.random.default_rng(1).random((N, 2, 16)).astype(np.float32)
    # (1e6: a weight of 0 in 64 bits as well)
    want, bound = op.weights(**a, clip_k=k, window=0, sinks=0, scale=0.125, lse=np.where(none, 1e6, lse).astype(np.float64),
                             mass=mass.astype(np.float64), accumulate=True)
    m = torch.from_numpy(mass).to(DEV)
    g = on_gpu(x)
    marked = torch.from_numpy(np.where(none, np.float32(-np.inf), lse)).to(DEV)
    rp.relattn_paged_weights(g["q"], g["k_pages"], g["table"], g["q_start"], g["kv_len"], marked, m, aK=g["aK"], clip_k=k,
                             scale=0.125, max_new=max_new)
    assert rp.relattn_get_device_error() == 0
    assert (np.abs(f64(m) - want) <= bound).all()


@pytest.mark.parametrize("new,max_new,dtype,d", [(1, 1, BF16, 64), (3, 3, BF16, 128), (40, 0, BF16, 64), (150, 0, BF16, 128),
                                                 (20, 0, F32, 64)])
@pytest.mark.parametrize("key", [False, True])
def test_pages_that_requests_share(new, max_new, dtype, d, key):
    """Prefixes of relattn_paged_shared_fwd: their keys get the weights of every request of the group."""
    from tests.test_gpu_paged_shared import make as behind_prefixes
    rp = _rp()
    k, scale = 6 * key, d ** -0.5
    x = behind_prefixes([(272, [(5, new), (60, new), (0, 1), (31, new)]), (512, [(1, new), (200, new)])], 4, 2, d, 16, dtype, k,
                        key=key, before=[(90, 1)], after=[(33, 2)])
    N = x["k_pages"].shape[0]
    a = args_of(x)
    lse = op.log_sum(**a, clip_k=k, window=0, sinks=0, scale=scale)[0].astype(np.float32)
    mass = np.random.default_rng(1).random((N, 2, 16)).astype(np.float32)
    g = on_gpu(x)
    m = torch.from_numpy(mass).to(DEV)
    run = lambda m, add: rp.relattn_paged_weights(g["q"], g["k_pages"], g["table"], g["q_start"], g["kv_len"],
                                                  torch.from_numpy(lse).to(DEV), m, aK=g["aK"], clip_k=k, accumulate=add,
                                                  max_new=max_new)
    for _ in range(3):                   # one step after the other
        want, bound = op.weights(**a, clip_k=k, window=0, sinks=0, scale=scale, lse=lse.astype(np.float64), mass=f64(m),
                                 accumulate=True)
        run(m, True)
        assert rp.relattn_get_device_error() == 0
        bad = ~(np.abs(f64(m) - want) <= bound)
        assert not bad.any(), (np.argwhere(bad)[:5], f64(m)[bad][:5], want[bad][:5])
    # set: one of the requests' sums
    run(m, False)
    at, fits = 0, np.zeros(m.shape, dtype=bool)
    written = np.zeros(m.shape, dtype=bool)
    for b, n in enumerate(np.diff(x["q_start"])):
        y = dict(a, q=a["q"][at:at + n], table=x["table"][b:b + 1], q_start=np.array([0, n]), kv_len=x["kv_len"][b:b + 1])
        want, bound = op.weights(**y, clip_k=k, window=0, sinks=0, scale=scale, lse=lse[at:at + n].astype(np.float64),
                                 mass=np.full(m.shape, np.nan), accumulate=False)
        written |= ~np.isnan(want)
        with np.errstate(invalid="ignore"):
            fits |= np.abs(f64(m) - want) <= bound
        at += n
    assert np.array_equal(written, written & fits)
