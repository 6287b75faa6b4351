"""A C entry that runs out of host memory returns a status: no C++ exception leaves the library (it would end the process).

Each case runs in a process of its own, whose address space is limited to what it holds already and a few megabytes.
"""

import subprocess
import sys

import pytest

PROGRAM = r"""
import resource, sys
import numpy as np
import radixattention_prefix_shared_radix_gb300 as sgl

def room(megabytes):
    pages = int(open("/proc/self/statm").read().split()[0])
    limit = pages * resource.getpagesize() + (megabytes << 20)
    resource.setrlimit(resource.RLIMIT_AS, (limit, resource.RLIM_INFINITY))

def everything():
    resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))

def status(f, *args):
    try:
        f(*args)
    except sgl.SglError as e:
        return e.status
    return 0

what = sys.argv[1]
B = 600000
table = np.arange(2 * B, dtype=np.int32).reshape(B, 2)
lens = np.full(B, 2, dtype=np.int32)
g = sgl.sgl_groups_create()
if what == "groups":
    room(8)
    st = status(sgl.sgl_groups_from_table, table, lens, g)
    everything()
    assert st == -1, st
    view = sgl.groups_as_numpy(sgl.sgl_groups_view(g))
    assert len(view["seg_begin"]) == 0          # (emptied, not half filled)
    sgl.sgl_groups_from_table(table, lens, g)   # and of use again
    assert len(sgl.groups_as_numpy(sgl.sgl_groups_view(g))["seg_begin"]) == B
else:
    sgl.sgl_groups_from_table(table, lens, g)
    if what == "mla":
        plan, p = sgl.sgl_mla_decode_plan, sgl.make_mla_params(B, 16, 2 * B)
    else:
        plan, p = sgl.sgl_decode_plan, sgl.make_params(int(what), B, 1, 1, 64, 2 * B)
    room(8)
    st = status(plan, p, lens, sgl.sgl_groups_view(g))
    everything()
    assert st == -1, st
    print("refused")
print("ok")
"""


@pytest.mark.parametrize("what", ["groups", "mla", "1", "3"])
def test_status_instead_of_an_exception(what):
    pytest.importorskip("resource")
    r = subprocess.run([sys.executable, "-c", PROGRAM, what], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.returncode, r.stdout, r.stderr[-2000:])
