"""What the BF16 paged-cache calls refuse on the host, tested without a GPU: paged_api.cu built with its launches
replaced by counters. No pointer is ever followed; a call that would launch on a pointer that the kernel cannot read
shows as a launch."""

import ctypes
import os
import subprocess

import pytest

from bit_kv_cache_write_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
BASE = 1 << 20                               # a pointer aligned to everything


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("paged_host") / "paged_host.so")
    r = subprocess.run([build.nvcc()] + build.ARCH + build.FLAGS + ["-shared", "-cudart", "static", "-I", build.CSRC, "-o", out,
                                                                     os.path.join(build.CSRC, "paged_api.cu"),
                                                                     os.path.join(HERE, "paged_host.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    lib = ctypes.CDLL(out)
    lib.paged_host_context.restype = ctypes.c_void_p
    lib.paged_host_message.restype = ctypes.c_char_p
    lib.paged_host_free.argtypes = [ctypes.c_void_p]
    return lib


@pytest.fixture
def ctx(host):
    c = host.paged_host_context(4, 2, 64)
    yield c
    host.paged_host_free(c)


def append(host, ctx, **over):
    """(status, launches) of an append of two rows with bounds."""
    a = dict(k=BASE, k_stride=256, v=BASE + 256, v_stride=256, slots=BASE, n=2, pool=BASE, pages=4, steps=BASE, bounds=BASE)
    a.update(over)
    p, i64 = ctypes.c_void_p, ctypes.c_int64
    before = host.paged_host_launches()
    st = host.oscar_append_bf16(p(ctx), p(a["k"]), i64(a["k_stride"]), p(a["v"]), i64(a["v_stride"]), p(a["slots"]), a["n"],
                                p(a["pool"]), i64(a["pages"]), p(a["steps"]), p(a["bounds"]), p(None))
    return st, host.paged_host_launches() - before


def test_append_as_documented(host, ctx):
    assert append(host, ctx) == (0, 1)
    assert append(host, ctx, steps=None, bounds=None) == (0, 1)
    assert append(host, ctx, n=0) == (0, 0)


@pytest.mark.parametrize("name,unit", [("k", 16), ("v", 16), ("pool", 16), ("bounds", 16), ("steps", 8)])
def test_append_refuses_pointers_that_the_kernel_cannot_read(host, ctx, name, unit):
    """Rows, pages and bounds move 16 bytes a lane; a lane reads the steps of its eight channels as one word."""
    for off in range(1, unit):
        assert append(host, ctx, **{name: BASE + off}) == (-1, 0), (name, off)
        assert b"aligned" in host.paged_host_message()
    assert append(host, ctx, **{name: BASE + unit}) == (0, 1)
