"""Caches whose pages lie further apart than 32 bits count, in elements and in bytes: the same bits as of a
cache whose pages follow each other."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
BF16, F32 = torch.bfloat16, torch.float32
N, P = 6, 256
FAR = 2 ** 30 + 64      # elements from page to page


def _rp():
    import relative_position_representations_gb300 as rp
    return rp


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def _room():
    rp = _rp()
    assert rp.relattn_get_device_error() == 0
    if torch.cuda.get_device_properties(0).total_memory < 2 ** 37:
        pytest.skip("needs 128 GB")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def apart(t):
    """The same pages, FAR elements from one to the next."""
    room = torch.empty((t.shape[0] - 1) * FAR + t[0].numel(), dtype=t.dtype, device=DEV)
    out = room.as_strided(t.shape, (FAR,) + tuple(t.stride()[1:]))
    out.copy_(t)
    return out


def case(dtype, d, new, seed):
    """Five requests behind a page that they share."""
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype).to(DEV)
    table = np.array([[5, b] for b in range(5)])
    q_start = np.arange(6) * new
    return dict(q=t(5 * new, 4, d), k=t(N, 2, P, d), v=t(N, 2, P, d), aK=t(2, 9, d), aV=t(2, 9, d), table=i32(table),
                q_start=i32(q_start), kv_len=i32([512, 300, 411, 290, 477]))


@pytest.mark.parametrize("dtype,d,new", [(BF16, 64, 1), (BF16, 128, 1), (BF16, 64, 20), (BF16, 128, 20), (F32, 40, 1)])
def test_shared_prefixes_and_weights(dtype, d, new):
    rp = _rp()
    x = case(dtype, d, new, d + new)
    lists = i32([0, 5]), i32([256])

    def run(k, v, mass):
        lse = torch.empty((5 * new, 4), dtype=F32, device=DEV)
        out = rp.relattn_paged_shared_fwd(x["q"], k, v, x["table"], x["q_start"], x["kv_len"], *lists, aK=x["aK"], aV=x["aV"],
                                          clip_k=4, lse=lse, max_new=new)
        # (a page of several requests has no defined mass: their own pages alone are looked at)
        rp.relattn_paged_weights(x["q"], k, x["table"], x["q_start"], x["kv_len"], lse, mass, aK=x["aK"], clip_k=4, max_new=new)
        assert rp.relattn_get_device_error() == 0
        return out, lse, mass[:5].clone()

    mass = torch.rand((N, 2, P), device=DEV)
    want = run(x["k"], x["v"], mass.clone())
    got = run(apart(x["k"]), apart(x["v"]), apart(mass))
    assert bool(torch.isfinite(want[0]).all()) and bool((want[2] != mass[:5]).any())
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 33), (F32, 128)])
def test_eviction(dtype, d):
    rp = _rp()
    rng = np.random.default_rng(d)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype).to(DEV)
    k, v, mass = t(N, 2, P, d), t(N, 2, P, d), torch.rand((N, 2, P), device=DEV)
    table, lens = i32([[5, 0, 3], [1, 4, 2]]), i32([700, 520])

    def run(k, v, mass):
        n, _ = rp.relattn_paged_evict(lens, table, k, v, mass, 400, limit=500, sinks=4, recent=30)
        assert rp.relattn_get_device_error() == 0 and n.tolist() == [400, 400]
        return k, v, mass

    far = run(apart(k), apart(v), apart(mass))
    before = k.clone()
    near = run(k, v, mass)
    assert not torch.equal(before, k)
    for a, b in zip(far, near):
        assert torch.equal(a, b)
