"""The paged cache without a GPU: pins of the oracle (oracle/paged.py) and the refusals of the
entry points, which check their arguments before any CUDA call."""
import numpy as np
import pytest
import torch

import oracle
from oracle import paged as op


@pytest.fixture(scope="module")
def lib():
    from relative_position_representations_gb300 import build
    build.build()
    from relative_position_representations_gb300 import _lib
    return _lib


# ------------------------------------------------------------------------------------ oracle
def _case(rng, new, kv, H, Hkv, d, P, k):
    M = max(-(-c // P) for c in kv) + 1
    N = sum(-(-c // P) for c in kv) + 2
    perm = rng.permutation(N)
    table, at = np.full((len(kv), M), -1), 0
    for b, c in enumerate(kv):
        u = -(-c // P)
        table[b, :u] = perm[at:at + u]
        at += u
    r = rng.standard_normal
    return dict(q=r((sum(new), H, d)), k_pages=r((N, Hkv, P, d)), v_pages=r((N, Hkv, P, d)), table=table,
                q_start=np.concatenate([[0], np.cumsum(new)]), kv_len=np.array(kv), aK=r((Hkv, 2 * k + 1, d)),
                aV=r((Hkv, 2 * k + 1, d)), clip_k=k)


@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 2), (3, 1)])
def test_attend_is_the_dense_causal_forward(H, Hkv):
    """Whole prompts and chunks: the last rows of the dense forward over the gathered cache."""
    rng = np.random.default_rng(H)
    new, kv, d, P, k = [7, 12, 1], [7, 30, 21], 6, 4, 3
    x = _case(rng, new, kv, H, Hkv, d, P, k)
    z, mass, _ = op.attend(**x, window=0, sinks=0, scale=0.4)
    g = H // Hkv
    for b, (n, c) in enumerate(zip(new, kv)):
        j = np.arange(c)
        K = x["k_pages"][x["table"][b, j // P], :, j % P].transpose(1, 0, 2).repeat(g, 0)[None]
        V = x["v_pages"][x["table"][b, j // P], :, j % P].transpose(1, 0, 2).repeat(g, 0)[None]
        q = np.zeros((1, H, c, d))
        rows = slice(x["q_start"][b], x["q_start"][b + 1])
        q[0, :, c - n:] = x["q"][rows].transpose(1, 0, 2)
        ref = oracle.relattn_fwd(q, K, V, x["aK"].repeat(g, 0), x["aV"].repeat(g, 0), k, True, 0.4)
        assert np.allclose(ref[0, :, c - n:].transpose(1, 0, 2), z[rows], rtol=1e-12, atol=1e-12)
    assert (np.abs(z) <= mass + 1e-12).all()


def test_window_and_sinks_of_the_oracle():
    rng = np.random.default_rng(0)
    x = _case(rng, [1], [20], 1, 1, 4, 8, 2)
    x["aK"] = x["aV"] = None
    x["q"][:] = 0.0                                   # equal weights: the mean of what is seen
    V = lambda j: x["v_pages"][x["table"][0, j // 8], 0, j % 8]
    mean = lambda js: np.mean([V(j) for j in js], 0)
    run = lambda w, s: op.attend(**x, window=w, sinks=s, scale=1.0)[0][0, 0]
    assert np.allclose(run(0, 3), mean(range(20)))
    assert np.allclose(run(1, 0), V(19))
    assert np.allclose(run(5, 0), mean(range(15, 20)))
    assert np.allclose(run(5, 2), mean([0, 1, 15, 16, 17, 18, 19]))
    assert np.allclose(run(5, 17), mean(range(20)))
    assert np.allclose(run(50, 2), mean(range(20)))


def test_attend_without_keys_and_past_the_table():
    rng = np.random.default_rng(1)
    x = _case(rng, [3], [8], 1, 1, 4, 4, 1)
    x["kv_len"] = np.array([2])                       # the first of three tokens has no position
    z, _, _ = op.attend(**x, window=0, sinks=0, scale=1.0)
    assert not z[0].any() and z[1:].all()


def test_plan_of_the_oracle_is_an_allocator():
    """Every placed token has a slot of its own, in pages of its own request, taken in order."""
    rng = np.random.default_rng(2)
    for P in (1, 4, 16):
        B = 9
        table, head, cached = np.full((B, 200), -1), 0, np.zeros(B, dtype=int)
        free = rng.permutation(700)
        seen = {}
        for _ in range(6):
            new = rng.integers(0, 17, B)
            table, cached, qs, slots, head, ok = op.plan(cached, new, table, free, head, P, int(new.sum()) + 2)
            assert ok and list(slots[qs[-1]:]) == [-1, -1]
            for b in range(B):
                for i, s in enumerate(slots[qs[b]:qs[b + 1]]):
                    assert s not in seen
                    seen[s] = (b, cached[b] - new[b] + i)
        pages = {}
        for s, (b, pos) in seen.items():
            assert pages.setdefault(s // P, (b, pos // P)) == (b, pos // P) and s % P == pos % P
        assert head == len(pages) and set(pages) == set(free[:head])


# ------------------------------------------------------------------------------------ refusals
A = 4096   # a pointer value that the host checks never follow

PLAN = dict(cached_len=A, new_len=A, B=2, page_size=16, block_table=A, table_stride=8, max_pages=8, free_pages=A,
            num_free=4, free_head=A, max_tokens=10, kv_len=A, q_start=A, slots=A, free_head_out=A, stream=None)
APPEND = dict(k=A, v=A, k_stride=128, v_stride=128, slots=A, tokens=3, k_pages=A, v_pages=2 * A, page_stride=2048,
              num_pages=4, Hkv=2, page_size=16, d=64, dtype=0, stream=None)
FWD = dict(q=A, q_stride=256, k_pages=2 * A, v_pages=3 * A, page_stride=2048, num_pages=4, page_size=16,
           block_table=A, table_stride=8, max_pages=8, q_start=A, kv_len=A, aK=4 * A, aV=5 * A, ths=7 * 64, clip_k=3,
           window=0, sinks=0, scale=0.125, B=2, tokens=5, max_new=0, H=4, Hkv=2, d=64, dtype=0, workspace=A,
           workspace_bytes=1 << 40, out=6 * A, stream=None)


def refused(lib, name, base, status, **change):
    assert set(change) <= set(base)
    args = dict(base, **change)
    assert lib.raw_call(name, *args.values()) == status, change


@pytest.mark.parametrize("status,change", [
    (1, dict(cached_len=None)), (1, dict(new_len=None)), (1, dict(block_table=None)), (1, dict(free_head=None)),
    (1, dict(kv_len=None)), (1, dict(q_start=None)), (1, dict(slots=None)), (1, dict(free_head_out=None)),
    (1, dict(free_pages=None)), (1, dict(B=0)), (1, dict(max_pages=0)), (1, dict(num_free=-1)),
    (1, dict(max_tokens=-1)), (1, dict(page_size=0)), (1, dict(page_size=12)), (1, dict(page_size=2048)),
    (1, dict(table_stride=7)), (1, dict(slots=A + 2)), (2, dict(B=16385)), (2, dict(max_tokens=(1 << 23) + 1))])
def test_plan_refuses(lib, status, change):
    refused(lib, "relattn_paged_plan", PLAN, status, **change)


@pytest.mark.parametrize("status,change", [
    (1, dict(k=None)), (1, dict(v=None)), (1, dict(slots=None)), (1, dict(k_pages=None)), (1, dict(v_pages=None)),
    (1, dict(v_pages=A)), (1, dict(tokens=-1)), (1, dict(num_pages=0)), (1, dict(Hkv=0)), (1, dict(d=0)),
    (1, dict(page_size=24)), (1, dict(page_stride=2047)), (1, dict(dtype=2)), (1, dict(k_stride=127)),
    (1, dict(v_stride=127)), (1, dict(k=A + 1)), (1, dict(dtype=1, v_pages=2 * A + 2)),
    (1, dict(num_pages=1 << 27)), (0, dict(tokens=0, k=None, v=None, slots=None))])
def test_append_refuses(lib, status, change):
    refused(lib, "relattn_paged_append", APPEND, status, **change)


@pytest.mark.parametrize("status,change", [
    (1, dict(q=None)), (1, dict(out=None)), (1, dict(workspace=None)), (1, dict(k_pages=None)),
    (1, dict(block_table=None)), (1, dict(q_start=None)), (1, dict(kv_len=None)), (1, dict(B=0)),
    (1, dict(tokens=-1)), (1, dict(max_new=-1)), (1, dict(max_pages=0)), (1, dict(out=A)), (1, dict(out=2 * A)),
    (1, dict(out=4 * A)), (1, dict(H=3)), (1, dict(Hkv=0)), (1, dict(dtype=3)), (1, dict(page_size=20)),
    (1, dict(page_stride=2047)), (1, dict(q_stride=255)), (1, dict(table_stride=7)), (1, dict(clip_k=-1)),
    (1, dict(window=-1)), (1, dict(window=(1 << 30) + 1)), (1, dict(sinks=-1)), (1, dict(ths=447)),
    (1, dict(q=A + 1)), (1, dict(block_table=A + 2)), (1, dict(workspace=A + 8)), (1, dict(workspace_bytes=1000)),
    (1, dict(tokens=1 << 30)), (2, dict(d=129, page_stride=1 << 20, q_stride=1 << 12, ths=0)),
    (2, dict(H=258, q_stride=1 << 20)), (2, dict(clip_k=257, ths=0)),
    (0, dict(tokens=0, q=None, out=None, workspace=None))])
def test_attention_refuses(lib, status, change):
    refused(lib, "relattn_paged_fwd", FWD, status, **change)


def test_workspace_size(lib):
    assert lib.relattn_paged_workspace_size(16, 4, 64) < lib.relattn_paged_workspace_size(16, 4, 128) < 1 << 27
    for bad, status in (((3, 2, 64), 1), ((4, 0, 64), 1), ((4, 2, 0), 1), ((4, 2, 129), 2), ((129, 1, 64), 2)):
        with pytest.raises(lib.RelattnError) as e:
            lib.relattn_paged_workspace_size(*bad)
        assert e.value.status == status


def test_binding_wants_cuda_tensors(lib):
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        lib.relattn_paged_plan(z, z, z.reshape(2, 1), z, z[:1], 16, 4)
    p = torch.zeros((2, 1, 8, 64))
    with pytest.raises(TypeError):
        lib.relattn_paged_append(p[:, :, 0], p[:, :, 0], z, p, p.clone())
    with pytest.raises(TypeError):
        lib.relattn_paged_fwd(p[:, :, 0], p, p.clone(), z.reshape(2, 1), torch.zeros(3, dtype=torch.int32), z)


@pytest.mark.parametrize("B,status", [((1 << 24) + 1, 2), ((1 << 31) - 1, 2), (1 << 24, 0)])
def test_attention_refuses_more_requests_than_its_scan_counts(lib, B, status):
    # (with no tokens, so that what is accepted ends on the host)
    refused(lib, "relattn_paged_fwd", FWD, status, B=B, tokens=0)
