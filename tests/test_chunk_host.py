"""What the calls on chunks of new tokens refuse on the host, tested without a GPU: chunk_api.cu built with its launches
replaced by counters. No pointer is ever followed; a call that would launch shows as a launch."""

import ctypes
import math
import os
import subprocess

import pytest

from bit_kv_cache_write_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
BASE = 1 << 30                               # a pointer aligned to everything
H_Q, H_KV, D = 4, 2, 64
Q, K = H_Q * D, H_KV * D                     # elements of a row


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("chunk_host") / "chunk_host.so")
    r = subprocess.run([build.nvcc()] + build.ARCH + build.FLAGS + ["-shared", "-cudart", "static", "-I", build.CSRC, "-o", out,
                                                                     os.path.join(build.CSRC, "chunk_api.cu"),
                                                                     os.path.join(HERE, "chunk_host.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    lib = ctypes.CDLL(out)
    lib.chunk_host_context.restype = ctypes.c_void_p
    lib.chunk_host_message.restype = ctypes.c_char_p
    lib.chunk_host_free.argtypes = [ctypes.c_void_p]
    lib.oscar_extend_bf16_workspace_size.restype = ctypes.c_size_t
    return lib


@pytest.fixture
def ctx(host):
    c = host.chunk_host_context(H_Q, H_KV, D)
    yield c
    host.chunk_host_free(c)


def mib(x):
    return BASE + (x << 20)


def rope(host, ctx, **over):
    """(status, launches) of a norm and rotation of three tokens; every buffer a MiB of its own."""
    a = dict(q=mib(0), q_stride=Q, q_out=mib(1), q_out_stride=Q, k=mib(2), k_stride=K, k_out=mib(3), k_out_stride=K,
             q_weight=mib(4), k_weight=mib(5), eps=1e-6, turns=mib(6), rot=D, layout=0, scale=1.0, positions=mib(7),
             row_start=None, total_len=None, batch=0, n=3)
    a.update(over)
    p, i64, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
    before = host.chunk_host_launches()
    st = host.oscar_norm_rope(p(ctx), p(a["q"]), i64(a["q_stride"]), p(a["q_out"]), i64(a["q_out_stride"]), p(a["k"]),
                              i64(a["k_stride"]), p(a["k_out"]), i64(a["k_out_stride"]), p(a["q_weight"]), p(a["k_weight"]),
                              f(a["eps"]), p(a["turns"]), a["rot"], a["layout"], f(a["scale"]), p(a["positions"]),
                              p(a["row_start"]), p(a["total_len"]), a["batch"], a["n"], p(None))
    return st, host.chunk_host_launches() - before


@pytest.mark.parametrize("over", [
    {}, dict(q=None, q_out=None), dict(k=None, k_out=None), dict(q_weight=None, k_weight=None), dict(rot=0, turns=None),
    dict(rot=8), dict(layout=1), dict(eps=0.0), dict(scale=-2.0), dict(positions=None, row_start=mib(8), total_len=mib(9), batch=2),
    dict(positions=None, row_start=mib(8), batch=0), dict(q_out=mib(0)), dict(q_out=mib(0), k_out=mib(2)),
    # slices of one row: queries, keys and room for both outputs
    dict(q=mib(0), k=mib(0) + 2 * Q, q_out=mib(0) + 2 * (Q + K), k_out=mib(0) + 2 * (2 * Q + K), q_stride=1024, k_stride=1024,
         q_out_stride=1024, k_out_stride=1024),
    dict(n=1, q_stride=0, k_stride=0), dict(n=1, q=mib(0), q_out=mib(0), q_stride=8)])
def test_norm_rope_as_documented(host, ctx, over):
    assert rope(host, ctx, **over) == (0, 1), host.chunk_host_message()


@pytest.mark.parametrize("over", [dict(n=0), dict(q=None, q_out=None, k=None, k_out=None)])
def test_norm_rope_of_nothing(host, ctx, over):
    assert rope(host, ctx, **over) == (0, 0)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), -1), (dict(batch=-1), -1), (dict(batch=65536), -2), (dict(layout=2), -2), (dict(layout=-1), -2), (dict(rot=12), -2),
    (dict(rot=72), -2), (dict(rot=-8), -2), (dict(eps=-1e-6), -1), (dict(eps=math.nan), -1), (dict(eps=math.inf), -1),
    (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(turns=None), -1), (dict(positions=None), -1),
    (dict(positions=None, row_start=mib(8), batch=1), -1), (dict(q_out=None), -1), (dict(q=None), -1), (dict(k=None), -1),
    (dict(q_stride=Q + 4), -1), (dict(k_out_stride=K + 4), -1), (dict(q_stride=-8), -1), (dict(q_stride=(1 << 31) + 8), -1),
    (dict(q_out_stride=Q - 8), -1), (dict(k_out_stride=0), -1), (dict(turns=mib(6) + 4), -1), (dict(q_weight=mib(4) + 4), -1),
    # overlaps
    (dict(q_out=mib(0) + 16), -1), (dict(q_out=mib(0), q_out_stride=Q + 8), -1), (dict(k_out=mib(0)), -1), (dict(q_out=mib(2)), -1),
    (dict(k_out=mib(1) + 2 * Q), -1), (dict(q=mib(0), k=mib(0) + 2 * Q, q_stride=1024, k_stride=1024, q_out=mib(0) + 2 * K, q_out_stride=1024), -1),
    (dict(q=mib(0), q_stride=1024, q_out=mib(0) + 2 * (1024 - 8), q_out_stride=1024), -1)])
def test_norm_rope_refuses(host, ctx, over, status):
    assert rope(host, ctx, **over) == (status, 0)


@pytest.mark.parametrize("name", ["q", "q_out", "k", "k_out"])
def test_norm_rope_refuses_rows_off_16_bytes(host, ctx, name):
    for off in (2, 4, 8):
        assert rope(host, ctx, **{name: mib(10) + off}) == (-1, 0)
    assert rope(host, ctx, **{name: mib(10) + 16}) == (0, 1)


def extend(host, ctx, **over):
    """(status, launches) of an attention of five rows of two requests."""
    a = dict(q=mib(0), q_stride=Q, pool=mib(1), pages=9, tables=mib(2), stride=4, row_start=mib(3), total_len=mib(4), batch=2,
             n=5, out=mib(5), ws=mib(6), ws_bytes=1024 + 7)
    a.update(over)
    p, i64 = ctypes.c_void_p, ctypes.c_int64
    before = host.chunk_host_launches()
    st = host.oscar_extend_bf16(p(ctx), p(a["q"]), i64(a["q_stride"]), p(a["pool"]), i64(a["pages"]), p(a["tables"]), a["stride"],
                                p(a["row_start"]), p(a["total_len"]), a["batch"], a["n"], p(a["out"]), p(a["ws"]),
                                ctypes.c_size_t(a["ws_bytes"]), p(None))
    return st, host.chunk_host_launches() - before


@pytest.mark.parametrize("over", [{}, dict(q_stride=0), dict(q=mib(0) + 16), dict(stride=0, tables=None), dict(out=mib(0) + 2 * 5 * Q),
                                  dict(n=1, ws_bytes=1027), dict(stride=1 << 26), dict(n=1 << 24, out=mib(1 << 16), ws_bytes=1 << 40)])
def test_extend_as_documented(host, ctx, over):
    assert extend(host, ctx, **over) == (0, 1), host.chunk_host_message()


@pytest.mark.parametrize("over", [dict(n=0), dict(batch=0), dict(n=0, q=None, ws=None)])
def test_extend_of_nothing(host, ctx, over):
    assert extend(host, ctx, **over) == (0, 0)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), -1), (dict(batch=-1), -1), (dict(stride=-1), -1), (dict(batch=65536), -2), (dict(n=(1 << 24) + 1), -2),
    (dict(stride=(1 << 26) + 1), -2), (dict(pages=1 << 31), -2), (dict(q=None), -1), (dict(out=None), -1), (dict(row_start=None), -1),
    (dict(total_len=None), -1), (dict(pool=None), -1), (dict(pages=0), -1), (dict(tables=None), -1), (dict(q_stride=Q + 4), -1),
    (dict(q_stride=-8), -1), (dict(q=mib(0) + 8), -1), (dict(pool=mib(1) + 16), -1), (dict(out=mib(5) + 16), -1), (dict(ws=None), -7),
    (dict(ws_bytes=1030), -7), (dict(ws=mib(6) + 128), -1), (dict(out=mib(0)), -1), (dict(out=mib(0) + 2 * 4 * Q), -1),
    (dict(out=mib(0) + 32, q_stride=1024), -1)])
def test_extend_refuses(host, ctx, over, status):
    assert extend(host, ctx, **over) == (status, 0)


def test_extend_workspace_of_bad_sizes(host, ctx):
    size = lambda b, n: host.oscar_extend_bf16_workspace_size(ctypes.c_void_p(ctx), b, n)
    assert size(2, 5) == 1024 + 7
    for b, n in ((-1, 5), (2, -1), (65536, 5), (2, (1 << 24) + 1), (0, 5), (2, 0)):
        assert size(b, n) == 0
    assert host.oscar_extend_bf16_workspace_size(None, 2, 5) == 0
    assert host.oscar_extend_bf16(None, None, ctypes.c_int64(0), None, ctypes.c_int64(0), None, 0, None, None, 0, 0, None, None,
                                  ctypes.c_size_t(0), None) == -1
