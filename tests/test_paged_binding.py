"""The binding of the paged calls without a GPU: tensors that only claim to lie on one, and a library
that only records. What the binding refuses, it refuses before the library is called."""
import contextlib
import types

import pytest
import torch

I32, BF16 = torch.int32, torch.bfloat16


class OnGpu(torch.Tensor):
    """A host tensor that says it is on cuda:0."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))
    used_on = property(lambda self: self.__dict__.setdefault("_used_on", []))

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.used_on.append(stream)


def gpu(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Binding:
    """The binding with `calls` in place of the library's and `made`: (tensor, its stream) of each
    allocation."""

    def __init__(self, monkeypatch):
        from relative_position_representations_gb300 import build
        build.build()
        from relative_position_representations_gb300 import _lib
        self.lib, self.calls, self.made, self.current = _lib, [], [], "current"

        def entry(name):
            def call(*args):
                self.calls.append((name, args))
                return 0
            return call

        names = ("relattn_paged_plan", "relattn_paged_append", "relattn_paged_fwd")
        fake = types.SimpleNamespace(**{n: entry(n) for n in names})
        fake.relattn_paged_workspace_size = _lib._lib.relattn_paged_workspace_size
        monkeypatch.setattr(_lib, "_lib", fake)
        monkeypatch.setattr(_lib, "_call_on", lambda dev, stream, fn, *args: fn(*args, stream))
        empty = torch.empty

        def record(shape, dtype=None, device=None):
            t = empty(shape, dtype=dtype).as_subclass(OnGpu)
            self.made.append((t, self.current))
            return t

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            yield
            self.current = before

        monkeypatch.setattr(torch, "empty", record)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)


@pytest.fixture
def binding(monkeypatch):
    return Binding(monkeypatch)


def plan_args(B=3, M=4):
    return dict(cached_len=gpu(B, dtype=I32), new_len=gpu(B, dtype=I32), block_table=gpu(B, M, dtype=I32),
                free_pages=gpu(9, dtype=I32), free_head=gpu(1, dtype=I32), page_size=16, max_tokens=5)


def fwd_args(T=5, H=4, Hkv=2, d=64, N=6, P=16, B=3, M=4):
    return dict(q=gpu(T, H, d), k_pages=gpu(N, Hkv, P, d), v_pages=gpu(N, Hkv, P, d),
                block_table=gpu(B, M, dtype=I32), q_start=gpu(B + 1, dtype=I32), kv_len=gpu(B, dtype=I32))


@pytest.mark.parametrize("op,count", [("plan", 4), ("fwd", 2)])
def test_memory_made_for_a_stream_is_that_streams(binding, op, count):
    # taken from the current stream, a block may still be in use by work queued there
    lib = binding.lib
    call = lambda **kw: (lib.relattn_paged_plan(**plan_args(), **kw) if op == "plan"
                         else lib.relattn_paged_fwd(**fwd_args(), **kw))
    call()
    assert [s for _, s in binding.made] == ["current"] * count
    del binding.made[:]
    call(stream="side")
    assert [s for _, s in binding.made] == ["side"] * count
    # what is returned is used on the current stream next, the workspace never is
    assert [t.used_on for t, _ in binding.made] == [["current"]] * (4 if op == "plan" else 1) + \
        [[]] * (op == "fwd")
    assert len(binding.calls) == 2 and binding.current == "current"


@pytest.mark.parametrize("heads,stride,fine", [
    (2, None, True), (2, 7 * 64, True), (2, 0, True), (1, None, True), (1, 0, True),
    (1, 7 * 64, False), (2, 7 * 64 + 1, False), (2, 1 << 40, False), (2, -7 * 64, False)])
def test_a_table_stride_stays_within_the_tables(binding, heads, stride, fine):
    # the kernels read rows of head h from h * stride on
    tables = dict(aK=gpu(heads, 7, 64), aV=gpu(heads, 7, 64), clip_k=3, table_head_stride=stride)
    if fine:
        binding.lib.relattn_paged_fwd(**fwd_args(), **tables)
        assert binding.calls[0][1][14] == (7 * 64 if heads == 2 and stride is None else stride or 0)
    else:
        with pytest.raises(ValueError, match="table_head_stride"):
            binding.lib.relattn_paged_fwd(**fwd_args(), **tables)
        assert not binding.calls


@pytest.mark.parametrize("big", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1])
@pytest.mark.parametrize("name", ["window", "sinks", "max_new", "clip_k", "page_size", "max_tokens"])
def test_integers_past_32_bits_are_refused(binding, name, big):
    # (a window of 2^32 + 5 keys would have been one of 5)
    lib = binding.lib
    with pytest.raises(ValueError, match="32 bits"):
        if name in ("page_size", "max_tokens"):
            lib.relattn_paged_plan(**dict(plan_args(), **{name: big}))
        else:
            lib.relattn_paged_fwd(**fwd_args(), **{name: big})
    assert not binding.calls


def test_shapes_past_32_bits_are_refused(binding):
    lib = binding.lib
    pages = lambda: torch.empty_strided(((1 << 32) + 2, 1, 1, 1), (1, 1, 1, 1), dtype=BF16, device="meta").as_subclass(OnGpu)
    with pytest.raises(ValueError, match="32 bits"):
        lib.relattn_paged_append(gpu(3, 1, 1), gpu(3, 1, 1), gpu(3, dtype=I32), pages(), pages())
    with pytest.raises(ValueError, match="32 bits"):
        lib.relattn_paged_fwd(**dict(fwd_args(H=1, Hkv=1, d=1, P=1), k_pages=pages(), v_pages=pages()))
    assert not binding.calls
