"""Host-only checks of AdamW's bookkeeping on the host: lists longer than its memory
are an error of the call, not the process's end."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, ALLOC = -1, -6


def child(code, *args):
    """A child's output; an abort shows as a negative return code."""
    r = subprocess.run([sys.executable, "-c", code, *args], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    return r.stdout.split()


@pytest.fixture(scope="module")
def lib():
    from verifiable_repops_gemm_gb300 import build
    return build.build()


def test_a_list_that_no_host_could_hold_is_an_error(lib):
    """2^31 - 1 tensors of 1024 contributors, the first of a size that is refused: the
    bookkeeping for all of them is not asked for before the sizes are looked at, and
    no C++ exception leaves the call."""
    out = child("""
import ctypes, sys
L = ctypes.CDLL(sys.argv[1])
order = (ctypes.c_int * 1024)(*range(1024))
sizes = (ctypes.c_int64 * 1)(-1)
one = (ctypes.c_uint64 * 1)(0x10000000)
words, hyper = (ctypes.c_uint32 * 4)(), (ctypes.c_double * 3)(0.9, 0.99, 1e-8)
p = lambda a: ctypes.c_void_p(ctypes.addressof(a))
print(L.repops_adamw(2**31 - 1, p(sizes), p(one), 1024, p(one), 0, p(order), p(one), p(one), None, None, None, p(hyper),
                     p(words), 0, None, None))
""", lib)
    assert out == [str(INVALID)]


def test_out_of_host_memory_is_an_error(lib):
    """A million tensors under a limit of address space that leaves no room for their
    ranges: the error of an allocation, with nothing launched."""
    out = child("""
import ctypes, resource, sys
L = ctypes.CDLL(sys.argv[1])
n = 1 << 20
def column(first, step):
    a = (ctypes.c_uint64 * n)()
    for i in range(n):
        a[i] = first + step * i
    return a
sizes = (ctypes.c_int64 * n)(*([1] * n))
theta, g, m, v = (column(i << 40, 16) for i in (1, 2, 3, 4))
order = (ctypes.c_int * 1)(0)
words, hyper = (ctypes.c_uint32 * 4)(), (ctypes.c_double * 3)(0.9, 0.99, 1e-8)
p = lambda a: ctypes.c_void_p(ctypes.addressof(a))
held = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (held + (48 << 20), resource.RLIM_INFINITY))
rc = L.repops_adamw(n, p(sizes), p(theta), 1, p(g), 0, p(order), p(m), p(v), None, None, None, p(hyper), p(words), 0, None,
                    None)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
print(rc)
""", lib)
    assert out == [str(ALLOC)]
