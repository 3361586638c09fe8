"""The attention weights of cached keys where every CTA has several units of work: the kernels' rings wrap, tickets are
taken and the summing groups go on from one unit to the next. Against the definition in 64 bits, head by head on the
GPU, within the bound of oracle.paged.weights."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
BF16, F32 = torch.bfloat16, torch.float32


def _rp():
    import relative_position_representations_gb300 as rp
    return rp


@pytest.fixture(autouse=True)
def _status_is_clear():
    assert _rp().relattn_get_device_error() == 0
    yield
    torch.cuda.synchronize()


def make(new, kv, H, Hkv, d, P, dtype, clip_k, key, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device=DEV, generator=g).to(dtype)
    used = [-(-n // P) for n in kv]
    N = sum(used) + 3
    perm = torch.randperm(N, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(kv), max(used)), 2 ** 30, dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    return dict(q=rnd(starts[-1], H, d), k_pages=rnd(N, Hkv, P, d), table=table, starts=starts, q_start=i32(starts), kv=kv,
                kv_len=i32(kv), aK=rnd(Hkv, 2 * clip_k + 1, d) if key else None,
                mass=torch.rand((N, Hkv, P), device=DEV, generator=g))


def definition(x, clip_k, window, sinks, scale):
    """lse [tokens, H] as fp32, the masses after the call (accumulated) and how far fp32 may be from them."""
    N, Hkv, P, d = x["k_pages"].shape
    T, H, _ = x["q"].shape
    gs, u = H // Hkv, 2.0 ** -24
    lse = torch.empty((T, H), device=DEV)
    want, bound = x["mass"].double(), torch.zeros((N, Hkv, P), dtype=torch.float64, device=DEV)
    for b, kv in enumerate(x["kv"]):
        t0, t1 = x["starts"][b], x["starts"][b + 1]
        n = t1 - t0
        j = torch.arange(kv, device=DEV)
        page, row = x["table"][b, j // P].long(), j % P
        pos = torch.arange(kv - n, kv, device=DEV)
        seen = j[None] <= pos[:, None]
        if window:
            seen &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
        lab = (j[None] - pos[:, None]).clamp(-clip_k, clip_k) + clip_k
        for h in range(Hkv):
            K = x["k_pages"][page, h, row].double()
            q = x["q"][t0:t1, h * gs:(h + 1) * gs].double().transpose(0, 1)       # [gs, n, d]
            e, a = q @ K.T, q.abs() @ K.abs().T
            if x["aK"] is not None:
                A = x["aK"][h].double()
                at = lab.expand(gs, -1, -1)
                e, a = e + (q @ A.T).gather(2, at), a + (q.abs() @ A.abs().T).gather(2, at)
            e = torch.where(seen, scale * e, -torch.inf)
            own = torch.logsumexp(e, 2).float()                                   # [gs, n]
            lse[t0:t1, h * gs:(h + 1) * gs] = own.T
            own = own.double()[..., None]
            a = scale * a
            w = torch.exp(e - own)
            slack = w * (4.0 * (d + 6) * u * a + 8.0 * u * (a + own.abs()) + 2.0 ** -21)
            s, off, some = w.sum((0, 1)), slack.sum((0, 1)), seen.any(0)
            old = torch.where(j < kv - n, want[page, h, row], 0.0)
            want[page, h, row] = torch.where(some, old + s, want[page, h, row])
            bound[page, h, row] = torch.where(some, off + 2.0 * n * gs * u * s + 2.0 * u * (old + s).abs() + 1e-36, 0.0)
    return lse, want, bound


def check(new, kv, H, Hkv, d, P, dtype=BF16, clip_k=0, key=False, window=0, sinks=0, max_new=0, seed=0):
    rp = _rp()
    x = make(new, kv, H, Hkv, d, P, dtype, clip_k, key, seed)
    scale = d ** -0.5
    lse, want, bound = definition(x, clip_k, window, sinks, scale)
    run = lambda: rp.relattn_paged_weights(x["q"], x["k_pages"], x["table"], x["q_start"], x["kv_len"], lse, x["mass"].clone(),
                                           aK=x["aK"], clip_k=clip_k, window=window, sinks=sinks, scale=scale, max_new=max_new)
    got = run()
    assert rp.relattn_get_device_error() == 0
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), got[bad][:5].tolist(), want[bad][:5].tolist())
    for _ in range(2):
        assert torch.equal(run(), got)   # the same bits, whichever CTA has which unit


def lengths(count, lo, hi, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, (count,), generator=g).tolist()


@pytest.mark.parametrize("d,new", [(64, 1), (64, 4), (128, 1), (128, 3)])
@pytest.mark.parametrize("clip_k,key,window,sinks", [(0, False, 0, 0), (16, True, 0, 0), (9, True, 700, 3)])
def test_generated_tokens_with_many_tiles_a_cta(d, new, clip_k, key, window, sinks):
    """About 3200 tiles for at most 456 CTAs: the ring of four stages comes round twice and more."""
    check([new] * 64, lengths(64, 1000, 2300, d + new), 16, 4, d, 16, clip_k=clip_k, key=key, window=window, sinks=sinks,
          max_new=new, seed=d)


@pytest.mark.parametrize("d,clip_k,key", [(64, 5, True), (128, 0, False)])
def test_generated_tokens_with_many_requests_a_cta(d, clip_k, key):
    """Over 3000 pieces of one or two tiles: the ring of four pieces comes round several times."""
    check([1] * 800, lengths(800, 1, 200, d), 8, 4, d, 8, clip_k=clip_k, key=key, max_new=1, seed=d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("clip_k,key,window,sinks", [(0, False, 0, 0), (30, True, 0, 0), (100, True, 500, 5)])
def test_prompts_with_many_units_a_cta(d, clip_k, key, window, sinks):
    """Several hundred pairs of key tiles, a dozen query tiles to most of them, for one CTA to an SM."""
    kv = lengths(7, 1200, 1700, d)
    check(kv, kv, 8, 8, d, 16, clip_k=clip_k, key=key, window=window, sinks=sinks, seed=d)


@pytest.mark.parametrize("g,d", [(3, 64), (4, 128)])
@pytest.mark.parametrize("clip_k,key", [(0, False), (12, True)])
def test_chunks_behind_long_caches(g, d, clip_k, key):
    """Chunks of two query tiles and more over caches of thousands of keys: the keys go through TMEM in unit after unit."""
    check(lengths(6, 70, 150, g), lengths(6, 5000, 9000, d), 4 * g, 4, d, 32, clip_k=clip_k, key=key, seed=g)


@pytest.mark.parametrize("d,new", [(64, 32), (128, 20)])
@pytest.mark.parametrize("clip_k,key", [(0, False), (12, True)])
def test_one_query_tile_over_many_long_units(d, new, clip_k, key):
    """At most one query tile to a request: units of eight key tiles, about a thousand of them."""
    check([new] * 20, lengths(20, 4000, 16000, d), 16, 4, d, 64, clip_k=clip_k, key=key, max_new=new, seed=d)


@pytest.mark.parametrize("dtype,d,P,clip_k,key", [(F32, 64, 16, 0, False), (F32, 64, 8, 16, True), (BF16, 80, 4, 10, True)])
def test_simt_with_many_units_a_cta(dtype, d, P, clip_k, key):
    """About 2000 runs of 32 keys for two CTAs to an SM."""
    check(lengths(8, 3, 60, d), lengths(8, 700, 1300, P), 16, 8, d, P, dtype=dtype, clip_k=clip_k, key=key, seed=d)
