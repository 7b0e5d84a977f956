"""The Python binding's checks of the calls on chunks of new tokens, with the library replaced by one that records."""

import pytest
import torch

from bit_kv_cache_write_gb300 import oscar as O

BF, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


class Calls:
    def __init__(self):
        self.got = []

    def __getattr__(self, name):
        def call(*args):
            self.got.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(O, "lib", lambda: c)
    monkeypatch.setattr(O, "_configs", {4096: (4, 2, 64, -1, 21)})
    monkeypatch.setattr(O, "_stream_on", lambda stream, device: 0)
    return c


def meta(*shape, dt=BF):
    return torch.empty(*shape, dtype=dt, device="meta")


def rope(**over):
    a = dict(q=meta(3, 4, 64), k=meta(3, 2, 64), q_out=meta(3, 4, 64), k_out=meta(3, 2, 64), turns=meta(32, dt=I64),
             positions=meta(3, dt=I32))
    a.update(over)
    O.oscar_norm_rope(4096, a.pop("q"), a.pop("k"), a.pop("q_out"), a.pop("k_out"), a.pop("turns"), **a)


def test_norm_rope_marshals(calls):
    qkv = meta(3, 8, 64)
    rope(q=qkv[:, :4], k=qkv[:, 4:6], q_weight=meta(64, dt=F32), layout=O.OSCAR_ROPE_INTERLEAVED, scale=1.5, eps=1e-5)
    rope(positions=None, row_start=meta(6, dt=I32), total_len=meta(5, dt=I32), turns=None)
    rope(k=None, k_out=None, q_out=meta(3, 5, 64)[:, :4])
    (_, a), (_, b), (_, c) = calls.got
    assert (a[2], a[4], a[6], a[8]) == (512, 256, 512, 128) and a[11] == 1e-5 and a[13:16] == (64, 1, 1.5) and a[19:21] == (0, 3)
    assert b[12] is None and b[13] == 0 and b[19:21] == (5, 3) and b[16] is None
    assert c[5] is None and c[7] is None and c[4] == 320


@pytest.mark.parametrize("over", [
    dict(q=meta(3, 4, 64, dt=F32)), dict(q=meta(3, 3, 64)), dict(q=meta(3, 4, 32)), dict(k=meta(4, 2, 64)), dict(q_out=meta(2, 4, 64)),
    dict(k_out=meta(3, 3, 64)[:, :2].transpose(0, 1)), dict(q_out=None), dict(k=None), dict(turns=meta(32, dt=I32)),
    dict(positions=meta(2, dt=I32)), dict(positions=meta(3, dt=I64)), dict(positions=None), dict(positions=None, row_start=meta(3, dt=I32)),
    dict(positions=None, row_start=meta(3, dt=I32), total_len=meta(3, dt=I32)), dict(q_weight=meta(64)), dict(k_weight=meta(63, dt=F32)),
    dict(q=meta(3, 64, 4).transpose(1, 2)), dict(layout=1 << 40)])
def test_norm_rope_refuses(calls, over):
    with pytest.raises(ValueError):
        rope(**over)
    assert not calls.got


def extend(**over):
    a = dict(q=meta(5, 4, 64), pool=meta(9, 2, 2, 16, 64), tables=meta(3, 4, dt=I32), row_start=meta(4, dt=I32),
             total_len=meta(3, dt=I32), out=meta(5, 4, 64), ws=meta(100, dt=torch.uint8))
    a.update(over)
    O.oscar_extend_bf16(4096, a["q"], a["pool"], a["tables"], a["row_start"], a["total_len"], a["out"], a["ws"])


def test_extend_marshals(calls):
    extend()
    extend(q=meta(5, 8, 64)[:, :4], ws=None)
    (_, a), (_, b) = calls.got
    assert (a[2], a[4], a[6], a[9], a[10], a[13]) == (256, 9, 4, 3, 5, 100) and b[2] == 512 and b[12:14] == (None, 0)


@pytest.mark.parametrize("over", [
    dict(q=meta(5, 3, 64)), dict(q=meta(5, 4, 64, dt=F32)), dict(out=meta(4, 4, 64)), dict(out=meta(5, 4, 64, dt=F32)),
    dict(tables=meta(2, 4, dt=I32)), dict(tables=meta(3, 4, dt=I64)), dict(row_start=meta(3, dt=I32)), dict(total_len=meta(3, dt=I64)),
    dict(pool=meta(9, 2, 2, 16, 64, dt=F32)), dict(total_len=meta(2, dt=I32))])
def test_extend_refuses(calls, over):
    with pytest.raises(ValueError):
        extend(**over)
    assert not calls.got


def test_sizes_past_32_bits(calls):
    for args in ((1 << 32, 5), (5, 1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            O.oscar_extend_bf16_workspace_size(4096, *args)
    big = (1 << 32) + 5
    with pytest.raises(ValueError, match="32 bits"):
        extend(q=meta(1, 4, 64).expand(big, 4, 64), out=meta(big, 4, 64))
    with pytest.raises(ValueError, match="32 bits"):
        rope(q=meta(1, 4, 64).expand(big, 4, 64), k=None, k_out=None, q_out=meta(big, 4, 64), positions=meta(big, dt=I32))
    assert not calls.got
