"""The Python binding's own checks, with the library replaced by one that records what it is given."""

import builtins

import pytest
import torch

from bit_kv_cache_write_gb300 import oscar as O


class Calls:
    """A library whose calls all succeed and are recorded."""

    def __init__(self):
        self.got = []

    def __getattr__(self, name):
        def call(*args):
            self.got.append((name, args))
            if name == "oscar_create":
                args[1]._obj.value = 4096
            return 0
        return call

    def named(self, name):
        return [args for n, args in self.got if n == name]


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(O, "lib", lambda: c)
    monkeypatch.setattr(O, "_configs", {})
    return c


def create():
    return O.oscar_create(n_layers=1, n_q_heads=4, n_kv_heads=2, head_dim=64, group=32)


@pytest.mark.parametrize("error", [RuntimeError, AssertionError])
def test_create_needs_no_device_of_torch_s(calls, monkeypatch, error):
    """The library has made the context: a torch that sees no device neither loses it nor fails the call."""
    def current_device():
        raise error("no device")
    monkeypatch.setattr(torch.cuda, "current_device", current_device)
    ctx = create()
    assert ctx == 4096 and not calls.named("oscar_destroy")
    with pytest.raises(ValueError, match="torch"):
        O.oscar_decode_bf16(ctx, None, None, None, None, 1, None, None)
    O.oscar_destroy(ctx)
    assert calls.named("oscar_destroy") == [(4096,)]


def test_create_works_without_torch(calls, monkeypatch):
    real = builtins.__import__

    def without(name, *args, **kw):
        if name == "torch":
            raise ImportError(name)
        return real(name, *args, **kw)
    monkeypatch.setattr(builtins, "__import__", without)
    assert create() == 4096


def test_create_registers_the_device(calls, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    ctx = create()
    assert O._configs[ctx][:4] == (4, 2, 64, 3)
    O.oscar_destroy(ctx)
    assert ctx not in O._configs


BIG = (1 << 32) + 5                       # 5 to a C int


@pytest.fixture
def meta(calls, monkeypatch):
    """A context on the device that tensors without memory count as theirs."""
    O._configs[4096] = (4, 2, 64, -1, 21)
    monkeypatch.setattr(O, "_stream_on", lambda stream, device: 0)
    return lambda *s, dt=torch.int32: torch.empty(*s, dtype=dt, device="meta")


@pytest.mark.parametrize("size", [BIG, 1 << 31, -(1 << 31) - 1])
def test_sizes_past_32_bits_are_refused(calls, size):
    """A cut size would be that of another, smaller call."""
    for call, args in ((O.oscar_decode_bf16_workspace_size, (4096, size, 5)), (O.oscar_decode_bf16_workspace_size, (4096, 5, size)),
                       (O.oscar_decode_bf16_sparse_workspace_size, (4096, size, 5, 5)),
                       (O.oscar_decode_bf16_sparse_workspace_size, (4096, 5, size, 5)),
                       (O.oscar_decode_bf16_sparse_workspace_size, (4096, 5, 5, size)), (O.oscar_sparse_capacity, (4096, size))):
        with pytest.raises(ValueError, match="32 bits"):
            call(*args)
    assert not calls.got


def test_tensors_past_32_bits_are_refused(calls, meta):
    i = meta
    plan = lambda free, slots: O.oscar_plan_append(4096, i(1), i(1), free, i(1), i(1, 3), slots, i(2), i(1), i(4))
    plan(i(7), i(9, dt=torch.int64))
    assert [(a[3], a[5], a[8], a[10]) for a in calls.named("oscar_plan_append")] == [(1, 7, 3, 9)]
    for free, slots in ((i(BIG), i(9, dt=torch.int64)), (i(7), i(BIG, dt=torch.int64))):
        with pytest.raises(ValueError, match="32 bits"):
            plan(free, slots)
    rows = lambda n: meta(1, 2, 64, dt=torch.bfloat16).expand(n, 2, 64)
    pool = meta(4, 2, 2, 16, 64, dt=torch.bfloat16)
    with pytest.raises(ValueError, match="32 bits"):
        O.oscar_append_bf16(4096, rows(BIG), rows(BIG), meta(BIG, dt=torch.int64), pool)
    q = meta(1, 4, 64, dt=torch.bfloat16).expand(BIG, 4, 64)
    out = meta(BIG, 4, 64, dt=torch.float32)
    with pytest.raises(ValueError, match="32 bits"):
        O.oscar_decode_bf16(4096, q, pool, meta(BIG, 1), meta(BIG), 16, out, None)
    with pytest.raises(ValueError, match="32 bits"):
        O.oscar_decode_bf16_sparse(4096, q, pool, meta(2, 64, dt=torch.int8), meta(4, 2, 2, 64, dt=torch.int8), meta(BIG, 1),
                                   meta(BIG), 16, 3, meta(BIG * 2 * 24), meta(BIG * 2), out, None)
    with pytest.raises(ValueError, match="32 bits"):
        O.oscar_plan_append(4096, meta(1), meta(1), meta(7), meta(1), meta(1, BIG), meta(9, dt=torch.int64), meta(2), meta(1), meta(4))
    assert len(calls.got) == 1
