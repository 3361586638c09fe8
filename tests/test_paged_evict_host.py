"""Eviction without a GPU: pins of the oracle and the refusals of the entry point and the binding."""
import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.test_paged_binding import BF16, I32, Binding, gpu
from tests.test_paged_host import A, lib, refused  # noqa: F401 (a fixture)

EVICT = dict(kv_len=A, block_table=A, table_stride=8, max_pages=8, k_pages=2 * A, v_pages=3 * A, page_stride=2048,
             mass=4 * A, mass_stride=32, num_pages=4, page_size=16, budget=64, limit=80, sinks=4, recent=16,
             free_pages=A, num_free=9, free_head=A, B=2, Hkv=2, d=64, dtype=0, workspace=A, workspace_bytes=1 << 40,
             kv_len_out=A, free_head_out=A, stream=None)


@pytest.mark.parametrize("status,change", [
    (1, dict(kv_len=None)), (1, dict(block_table=None)), (1, dict(k_pages=None)), (1, dict(v_pages=None)),
    (1, dict(mass=None)), (1, dict(workspace=None)), (1, dict(kv_len_out=None)), (1, dict(v_pages=2 * A)),
    (1, dict(mass=2 * A)), (1, dict(B=0)), (1, dict(max_pages=0)), (1, dict(num_free=-1)), (1, dict(free_head=None)),
    (1, dict(free_head_out=None)), (1, dict(free_pages=None)), (1, dict(budget=0)), (1, dict(limit=63)),
    (1, dict(sinks=-1)), (1, dict(recent=-1)), (1, dict(recent=61)), (1, dict(sinks=1 << 30, recent=1 << 30)),
    (1, dict(page_size=20)), (1, dict(page_stride=2047)), (1, dict(mass_stride=31)), (1, dict(dtype=2)),
    (1, dict(table_stride=7)), (1, dict(k_pages=2 * A + 1)), (1, dict(mass=4 * A + 2)), (1, dict(workspace=A + 8)),
    (1, dict(workspace_bytes=100)), (2, dict(d=129, page_stride=1 << 20)), (2, dict(B=16385)),
    (2, dict(max_pages=1 << 27, table_stride=1 << 27)), (2, dict(B=16384, max_pages=1 << 17, table_stride=1 << 17))])
def test_evict_refuses(lib, status, change):  # noqa: F811
    refused(lib, "relattn_paged_evict", EVICT, status, **change)


def test_workspace_size(lib):  # noqa: F811
    size = lib.relattn_paged_evict_workspace_size
    assert size(1, 1, 1) < size(2, 1, 1) < size(2, 4, 1 << 17) < 1 << 21
    for bad, status in (((0, 1, 1), 1), ((1, 0, 1), 1), ((1, 1, 0), 1), ((16385, 1, 1), 2), ((1, 1, (1 << 31) - 1), 2),
                        ((16384, 128, 1 << 20), 2)):
        with pytest.raises(lib.RelattnError) as e:
            size(*bad)
        assert e.value.status == status
    with pytest.raises(ValueError):
        size(1, 1, 1 << 31)


def test_the_oracle_keeps_what_the_definition_says():
    """Eight keys in pages of four: the first, the last two, and the two heaviest between, the earlier
    of two equal ones."""
    k = np.arange(16.0).reshape(4, 1, 4, 1)
    table = np.array([[2, 0]])
    mass = np.zeros((4, 1, 4))
    mass[2, 0], mass[0, 0] = [0, 5, 1, 7], [5, 9, 0, 0]     # positions 0 .. 7
    kv, kp, vp, m, free, head = op.evict([8], table, k, -k, mass, 4, 4, 1, 2, [2, 0, 1], 2)
    # position 5 (9) is the heaviest of 1 .. 5; budget 4 leaves one place
    assert kv.tolist() == [4] and kp[2, 0, :, 0].tolist() == [8, 1, 2, 3] and m[2, 0].tolist() == [0, 9, 0, 0]
    assert np.array_equal(vp, -kp) and head == 1 and free.tolist() == [2, 0, 1]
    kv, kp, *_ = op.evict([8], table, k, -k, mass, 5, 5, 1, 1)
    # three of 1 .. 6: positions 5 (9), 3 (7), and of the two fives the earlier, position 1
    assert kp[2, 0, :, 0].tolist() == [8, 9, 11, 1] and kp[0, 0, 0, 0] == 3
    assert op.evict([8], table, k, -k, mass, 5, 8, 1, 1)[0].tolist() == [8]


def _call(b, **change):
    args = dict(kv_len=gpu(2, dtype=I32), block_table=gpu(2, 4, dtype=I32), k_pages=gpu(9, 2, 16, 64),
                v_pages=gpu(9, 2, 16, 64), mass=gpu(9, 2, 16, dtype=torch.float32), budget=32)
    args.update(change)
    return b.lib.relattn_paged_evict(**args)


@pytest.fixture
def evict(monkeypatch):
    b = Binding(monkeypatch)
    real = b.lib._lib
    import relative_position_representations_gb300._lib as m
    import ctypes
    real.relattn_paged_evict = lambda *a: b.calls.append(("relattn_paged_evict", a)) or 0

    def size(B, Hkv, keys, out):
        ctypes.cast(out, ctypes.POINTER(ctypes.c_ulonglong))[0] = 4096
        return 0
    real.relattn_paged_evict_workspace_size = size
    assert m is b.lib
    return b


@pytest.mark.parametrize("change,error", [
    (dict(mass=gpu(9, 2, 16)), TypeError), (dict(mass=gpu(9, 2, 8, dtype=torch.float32)), ValueError),
    (dict(mass=gpu(9, 16, 2, dtype=torch.float32).transpose(1, 2)), ValueError),
    (dict(mass=gpu(1, 2, 16, dtype=torch.float32).expand(9, 2, 16)), ValueError),
    (dict(mass=torch.zeros(9, 2, 16)), TypeError), (dict(free_pages=gpu(3, dtype=I32)), ValueError),
    (dict(free_head_out=gpu(1, dtype=I32)), ValueError), (dict(budget=(1 << 32) + 32), ValueError),
    (dict(limit=1 << 32), ValueError), (dict(sinks=1 << 33), ValueError), (dict(kv_len_out=gpu(3, dtype=I32)), ValueError),
    (dict(v_pages=gpu(9, 2, 16, 64, dtype=torch.float32)), TypeError),
    (dict(k_pages=gpu(9, 2, 16, 64, dtype=torch.float16), v_pages=gpu(9, 2, 16, 64, dtype=torch.float16)), TypeError),
    (dict(workspace=torch.zeros(99, dtype=torch.uint8)), TypeError),
    (dict(block_table=gpu(3, 4, dtype=I32)), ValueError)])
def test_the_binding_refuses(evict, change, error):
    with pytest.raises(error):
        _call(evict, **change)
    assert not evict.calls


def test_the_binding_makes_what_is_not_given(evict):
    out, head = _call(evict)
    assert out.shape == (2,) and head is None and len(evict.calls) == 1
    out, head = _call(evict, free_pages=gpu(5, dtype=I32), free_head=gpu(1, dtype=I32))
    assert head.shape == (1,)
    evict.made.clear()
    out, _ = _call(evict, stream=type("S", (), {"cuda_stream": 7})())
    assert evict.calls[-1][1][-1].cuda_stream == 7
    assert all(s is not None and s != "current" for _, s in evict.made) and out.used_on == ["current"]
