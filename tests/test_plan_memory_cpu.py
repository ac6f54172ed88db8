"""Plans that the host has no memory for are refused, on CPU: no exception crosses the C boundary."""
import subprocess
import sys

CODE = """
import resource
import numpy as np
from paged_sliding_window_qkv_gb300 import pg

T = 1 << 28  # the token table alone takes 1 GiB
one = np.ones(1, np.int32)
pages = np.arange(2, dtype=np.int32)

def plan(segment):
    if segment:
        return pg.pg_plan_paged_segment(None, 1, np.array([0, T], np.int64), np.array([0, 2], np.int64), pages,
                                        np.array([1 << 27], np.int32), np.array([0], np.int64),
                                        np.array([0], np.int64), 16, 8, 256, 1 << 27, stream=0)
    return pg.pg_plan_paged_prefill(None, 1, np.array([0, T], np.int64), np.array([0, 2], np.int64), pages,
                                    np.array([1 << 27], np.int32), np.array([0], np.int64), 16, 8, 256, 1 << 27,
                                    stream=0)

used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (700 << 20),) * 2)
for segment in (False, True):
    rc, p = plan(segment)
    assert rc == pg.PG_ERR_ARG and p is None, rc
print("refused")
"""


def test_a_plan_without_memory_is_refused():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "refused" in r.stdout, (r.returncode, r.stdout[-500:], r.stderr[-2000:])
