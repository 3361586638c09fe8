"""Attention weights and shared prefixes without a GPU: pins of the oracle and the refusals of the entry points and
the binding."""
import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.test_paged_binding import I32, Binding, gpu
from tests.test_paged_host import FWD, A, _case, lib, refused  # noqa: F401 (a fixture)

F32 = torch.float32
LSE = dict(list(FWD.items())[:-1] + [("lse", 7 * A), ("stream", None)])
SHARED = dict(list(FWD.items())[:12] + [("group_start", A), ("prefix_len", A), ("groups", 3)] + list(FWD.items())[12:-1] +
              [("lse", 7 * A), ("stream", None)])
WEIGHTS = dict(q=A, q_stride=256, k_pages=2 * A, page_stride=2048, num_pages=4, page_size=16, block_table=A, table_stride=8,
               max_pages=8, q_start=A, kv_len=A, aK=4 * A, ths=7 * 64, clip_k=3, window=0, sinks=0, scale=0.125, lse=7 * A,
               accumulate=1, B=2, tokens=5, max_new=0, H=4, Hkv=2, d=64, dtype=0, workspace=A, workspace_bytes=1 << 40,
               mass=8 * A, mass_stride=32, stream=None)
COMMON = [(1, dict(q=None)), (1, dict(workspace=None)), (1, dict(k_pages=None)), (1, dict(block_table=None)),
          (1, dict(q_start=None)), (1, dict(kv_len=None)), (1, dict(B=0)), (1, dict(tokens=-1)), (1, dict(max_new=-1)),
          (1, dict(max_pages=0)), (1, dict(H=3)), (1, dict(Hkv=0)), (1, dict(dtype=3)), (1, dict(page_size=20)),
          (1, dict(page_stride=2047)), (1, dict(q_stride=255)), (1, dict(table_stride=7)), (1, dict(clip_k=-1)),
          (1, dict(window=-1)), (1, dict(window=(1 << 30) + 1)), (1, dict(sinks=-1)), (1, dict(ths=447)), (1, dict(q=A + 1)),
          (1, dict(block_table=A + 2)), (1, dict(lse=7 * A + 2)), (1, dict(workspace=A + 8)), (1, dict(workspace_bytes=60)),
          (1, dict(tokens=1 << 30)), (2, dict(d=129, page_stride=1 << 20, q_stride=1 << 12, ths=0)),
          (2, dict(H=258, q_stride=1 << 20)), (2, dict(clip_k=257, ths=0)), (2, dict(B=(1 << 24) + 1))]


@pytest.mark.parametrize("status,change", COMMON + [
    (1, dict(out=None)), (1, dict(out=A)), (1, dict(out=4 * A)), (1, dict(lse=6 * A)), (1, dict(lse=A)), (1, dict(lse=2 * A)),
    (0, dict(tokens=0, q=None, out=None, workspace=None, lse=None))])
def test_lse_refuses(lib, status, change):  # noqa: F811
    refused(lib, "relattn_paged_fwd_lse", LSE, status, **change)


@pytest.mark.parametrize("status,change", COMMON + [
    (1, dict(out=None)), (1, dict(lse=6 * A)), (1, dict(groups=-1)), (1, dict(group_start=None)), (1, dict(prefix_len=None)),
    (1, dict(group_start=A + 1)), (1, dict(prefix_len=A + 3)), (2, dict(groups=(1 << 24) + 1)),
    (1, dict(workspace_bytes=4 * 5 * 4 * 64)),
    (0, dict(tokens=0, q=None, out=None, workspace=None, lse=None)),
    (0, dict(tokens=0, groups=0, group_start=None, prefix_len=None))])
def test_shared_refuses(lib, status, change):  # noqa: F811
    refused(lib, "relattn_paged_shared_fwd", SHARED, status, **change)


@pytest.mark.parametrize("status,change", COMMON + [
    (1, dict(lse=None)), (1, dict(mass=None)), (1, dict(mass=8 * A + 2)), (1, dict(mass=A)), (1, dict(mass=2 * A)),
    (1, dict(mass=7 * A)), (1, dict(mass=4 * A)), (1, dict(mass_stride=31)), (1, dict(accumulate=2)), (1, dict(accumulate=-1)),
    (0, dict(tokens=0, q=None, lse=None, workspace=None))])
def test_weights_refuses(lib, status, change):  # noqa: F811
    refused(lib, "relattn_paged_weights", WEIGHTS, status, **change)


def test_workspace_sizes(lib):  # noqa: F811
    assert 0 < lib.relattn_paged_weights_workspace_size(0, 4) < lib.relattn_paged_weights_workspace_size(100, 16) < 20000
    fwd, shared = lib.relattn_paged_workspace_size, lib.relattn_paged_shared_workspace_size
    assert fwd(16, 4, 64) < shared(0, 16, 4, 64) < shared(100, 16, 4, 64)
    for bad, status in (((-1, 4), 1), ((4, 0), 1), ((1 << 30, 4), 1)):
        with pytest.raises(lib.RelattnError) as e:
            lib.relattn_paged_weights_workspace_size(*bad)
        assert e.value.status == status
    for bad, status in (((-1, 4, 2, 64), 1), ((4, 3, 2, 64), 1), ((4, 4, 2, 129), 2), ((1 << 30, 4, 2, 64), 1), ((4, 129, 1, 64), 2)):
        with pytest.raises(lib.RelattnError) as e:
            shared(*bad)
        assert e.value.status == status


# ------------------------------------------------------------------------------------ the oracle
def test_weights_of_the_oracle_sum_to_the_rows():
    """Every row's weights add up to one, wherever they go; the log-sum-exp is the one that the output goes by."""
    rng = np.random.default_rng(0)
    new, kv, H, Hkv, d, P, k = [3, 1, 5], [9, 20, 5], 4, 2, 6, 4, 3
    x = _case(rng, new, kv, H, Hkv, d, P, k)
    x.pop("aV")
    v = x.pop("v_pages")
    for window, sinks in ((0, 0), (4, 1)):
        lse, size = op.log_sum(**x, window=window, sinks=sinks, scale=0.3)
        mass, bound = op.weights(**x, window=window, sinks=sinks, scale=0.3, lse=lse, mass=np.zeros(v.shape[:3]), accumulate=True)
        assert np.isclose(mass.sum(), sum(new) * H) and (bound[mass > 0] > 0).all() and (bound < 1e-4).all()
        assert (size > 0).all()
        # with values that are 1 in one place, the output is that key's weight
        b, j, h = 1, 17, 1
        v1 = np.zeros_like(v)
        v1[x["table"][b, j // P], h, j % P] = 1
        z, _, _ = op.attend(**x, v_pages=v1, aV=None, window=window, sinks=sinks, scale=0.3)
        assert np.isclose(z[3, 2:, 0].sum(), mass[x["table"][b, j // P], h, j % P])
    once, _ = op.weights(**x, window=0, sinks=0, scale=0.3, lse=op.log_sum(**x, window=0, sinks=0, scale=0.3)[0],
                         mass=np.full(v.shape[:3], 7.0), accumulate=True)
    t = x["table"]
    assert once[t[1, 4], 0, 3] < 5 and once[t[1, 4], 0, 2] > 7        # position 19 is new, 18 is not


# ------------------------------------------------------------------------------------ the binding
@pytest.fixture
def paged(monkeypatch):
    b = Binding(monkeypatch)
    real = b.lib._lib
    for n in ("relattn_paged_fwd_lse", "relattn_paged_shared_fwd", "relattn_paged_weights"):
        setattr(real, n, (lambda n: lambda *a: b.calls.append((n, a)) or 0)(n))
    import ctypes
    from relative_position_representations_gb300 import _lib as m

    def size(*a):
        ctypes.cast(a[-1], ctypes.POINTER(ctypes.c_ulonglong))[0] = 4096
        return 0
    real.relattn_paged_shared_workspace_size = real.relattn_paged_weights_workspace_size = size
    assert m is b.lib
    return b


def base():
    return dict(q=gpu(5, 4, 64), k_pages=gpu(9, 2, 16, 64), block_table=gpu(2, 4, dtype=I32), q_start=gpu(3, dtype=I32),
                kv_len=gpu(2, dtype=I32))


def weights(b, **change):
    return b.lib.relattn_paged_weights(**dict(base(), lse=gpu(5, 4, dtype=F32), mass=gpu(9, 2, 16, dtype=F32), **change))


def shared(b, **change):
    args = dict(base(), v_pages=gpu(9, 2, 16, 64), group_start=gpu(3, dtype=I32), prefix_len=gpu(2, dtype=I32))
    args.update(change)
    return b.lib.relattn_paged_shared_fwd(**args)


@pytest.mark.parametrize("change,error", [
    (dict(aK=gpu(2, 7, 64), clip_k=4), ValueError), (dict(aK=gpu(2, 7, 64, dtype=F32), clip_k=3), TypeError),
    (dict(window=1 << 32), ValueError), (dict(max_new=1 << 31), ValueError), (dict(clip_k=(1 << 32) + 1), ValueError),
    (dict(workspace=torch.zeros(9, dtype=torch.uint8)), TypeError),
    (dict(aK=gpu(2, 7, 64), clip_k=3, table_head_stride=9999), ValueError)])
@pytest.mark.parametrize("call", [weights, shared])
def test_the_binding_refuses(paged, call, change, error):
    with pytest.raises(error):
        call(paged, **change)
    assert not paged.calls


@pytest.mark.parametrize("change,error", [
    (dict(group_start=gpu(2, dtype=I32)), ValueError), (dict(prefix_len=gpu(2, dtype=torch.int64)), TypeError),
    (dict(group_start=torch.zeros(3, dtype=I32)), TypeError), (dict(lse=gpu(5, 5, dtype=F32)), ValueError),
    (dict(lse=gpu(5, 4)), TypeError), (dict(lse=gpu(4, 5, dtype=F32).t()), ValueError), (dict(out=gpu(5, 4, 32)), ValueError)])
def test_shared_binding_refuses(paged, change, error):
    with pytest.raises(error):
        shared(paged, **change)
    assert not paged.calls


def test_weights_binding(paged):
    for change, error in ((dict(mass=gpu(9, 2, 16)), TypeError), (dict(mass=gpu(8, 2, 16, dtype=F32)), ValueError),
                          (dict(lse=gpu(4, 4, dtype=F32)), ValueError), (dict(q=gpu(5, 4, 32)), ValueError),
                          (dict(q_start=gpu(2, dtype=I32)), ValueError)):
        with pytest.raises(error):
            args = dict(base(), lse=gpu(5, 4, dtype=F32), mass=gpu(9, 2, 16, dtype=F32))
            paged.lib.relattn_paged_weights(**dict(args, **change))
    assert not paged.calls
    room = gpu(9, 3, 16, dtype=F32)
    mass = room[:, :2]
    args = dict(base(), lse=gpu(5, 4, dtype=F32))
    assert paged.lib.relattn_paged_weights(**args, mass=mass, accumulate=False) is mass
    name, a = paged.calls[-1]
    assert name == "relattn_paged_weights" and a[-2] == 48 and a[18] == 0


def test_what_is_made_comes_out_of_the_calls_stream(paged):
    s = type("S", (), {"cuda_stream": 7})()
    out = shared(paged, stream=s)
    assert paged.calls[-1][0] == "relattn_paged_shared_fwd" and paged.calls[-1][1][-1] is s
    assert all(on is s for _, on in paged.made) and out.used_on == ["current"]
    paged.made.clear()
    args = dict(base(), v_pages=gpu(9, 2, 16, 64))
    out, lse = paged.lib.relattn_paged_fwd_lse(**args, stream=s)
    assert paged.calls[-1][0] == "relattn_paged_fwd_lse" and lse.shape == (5, 4) and lse.dtype == F32
    assert all(on is s for _, on in paged.made) and lse.used_on == ["current"]
