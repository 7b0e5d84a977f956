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
