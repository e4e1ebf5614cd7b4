"""What a synchronous call sends to the device has arrived when the call returns, on the CPU.

A device memset, and a copy from pageable memory that has only been staged, may still be under way on the legacy
default stream when they return to the host, and streams made with cudaStreamNonBlocking are not ordered behind
that stream.  The library runs here, in a process of its own, on a fake of the CUDA runtime that counts the uploads
which no synchronisation has covered.
"""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = r"""
#include <stdlib.h>
#include <string.h>
static int uploads, pending;
int fake_uploads(void) { return uploads; }
int fake_pending(void) { return pending; }
static int upload(void) { ++uploads; ++pending; return 0; }
int cudaGetDevice(int *d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int *v, int attr, int d) { *v = 152; return 0; }
static void *last;
void fake_set_last(int v) { *(int *)last = v; } /* the last device word that was allocated */
int cudaMalloc(void **p, size_t n) { *p = malloc(n ? n : 1); if (n == sizeof(int)) last = *p; return 0; }
int cudaFree(void *p) { free(p); return 0; }
int cudaHostAlloc(void **p, size_t n, unsigned flags) { *p = malloc(n ? n : 1); return 0; }
int cudaFreeHost(void *p) { free(p); return 0; }
int cudaMemset(void *p, int v, size_t n) { memset(p, v, n); return upload(); }
int cudaMemcpy(void *to, const void *from, size_t n, int kind) { memcpy(to, from, n); return kind == 2 ? 0 : upload(); } /* 2: to the host */
int cudaEventCreateWithFlags(void **e, unsigned flags) { *e = malloc(1); return 0; }
int cudaEventSynchronize(void *e) { return 0; }
int cudaEventDestroy(void *e) { free(e); return 0; }
int cudaStreamSynchronize(void *s) { if ((size_t)s <= 1) pending = 0; return 0; } /* NULL and cudaStreamLegacy */
int cudaDeviceSynchronize(void) { pending = 0; return 0; }
"""

CHILD = """
import ctypes, sys
sys.path.insert(0, {root!r})
fake = ctypes.CDLL({fake!r}, ctypes.RTLD_GLOBAL)  # found before the runtime that the library is linked to
import all_gather_tide_gb300 as tide
handle = {create}
{then}
print(fake.fake_uploads(), fake.fake_pending())
{destroy}(handle)
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from all_gather_tide_gb300 import build

    build.build()
    path = tmp_path_factory.mktemp("fake")
    (path / "fake.c").write_text(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(path / "fake.so"), str(path / "fake.c")], check=True)
    return str(path / "fake.so")


def created(fake, create, destroy, then=""):
    """Uploads that the creation and what follows it made, and those of them that were not waited for."""
    child = textwrap.dedent(CHILD).format(root=ROOT, fake=fake, create=create, destroy=destroy, then=then)
    out = subprocess.run([sys.executable, "-c", child], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    return tuple(int(v) for v in out.stdout.split())


@pytest.mark.parametrize("elems", [[0], [100], [5000, 0, 7]], ids=str)
def test_a_list_waits_for_its_uploads(fake, elems):
    uploads, pending = created(fake, f"tide.tide_tensors_create({elems})", "tide.tide_tensors_destroy")
    assert uploads > 0 and pending == 0


@pytest.mark.parametrize("params", [[(3, 1)], [(50, 16), (7, 24)], [(300, 8192)]], ids=str)
def test_a_group_waits_for_its_uploads(fake, params):
    rows, length = [r for r, _ in params], [n for _, n in params]
    uploads, pending = created(fake, f"tide.tide_group_create(3, {rows}, {length})", "tide.tide_group_destroy")
    assert uploads > 1 and pending == 0


def test_clearing_a_status_is_waited_for(fake):
    """A kernel of a later call may record its own, which a clearing that comes late would lose."""
    read = "fake.fake_set_last(64); assert tide.tide_group_device_status(handle) == 64; assert tide.tide_group_device_status(handle) == 0"
    uploads, pending = created(fake, "tide.tide_group_create(3, [50], [16])", "tide.tide_group_destroy", read)
    assert uploads > 1 and pending == 0
