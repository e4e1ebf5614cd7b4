"""How long the thread that issued a CTA's copies stays for their end, on the CPU.

`wait_for_last_uses` (all_gather_tide_gb300/csrc/copies_end.h) runs here on a clock that goes by 50 ns with each look at it, with products and copies that end when the
test says so, or never.
"""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MS = 1_000_000
NEVER = 2 ** 64 - 1
LANDING = 20 * MS
SLACK = 10_000  # some looks at the clock

HARNESS = r"""
#include "copies_end.h"
struct At {
    mutable uint64_t time;
    uint64_t stop_at;
    const uint64_t *ended_at, *landed_at;  // of each stage; the parities are checked apart
    mutable uint64_t looked;               // stages asked about, one bit each
    mutable int bad;                       // a wrong parity
    const uint32_t *parities;
    uint64_t now() const { return time += 50; }
    bool stopped() const { return now() >= stop_at; }
    bool ended(int s, uint32_t parity) const { looked |= 1ull << s; bad |= parity != parities[s]; return now() >= ended_at[s]; }
    bool landed(int s, uint32_t parity) const { looked |= 1ull << s; bad |= parity != parities[s]; return now() >= landed_at[s]; }
};
extern "C" uint64_t run(int64_t uses, int stages, int stopped, uint64_t limit, uint64_t stop_at, const uint64_t *ended_at, const uint64_t *landed_at,
                        const uint32_t *parities, uint64_t *looked, int *bad) {
    At at{0, stop_at, ended_at, landed_at, 0, 0, parities};
    tide::wait_for_last_uses(uses, stages, stopped != 0, limit, at);
    *looked = at.looked, *bad = at.bad;
    return at.time;
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    path = tmp_path_factory.mktemp("copies_end")
    (path / "harness.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "all_gather_tide_gb300", "csrc"), "-o", str(path / "h.so"),
                    str(path / "harness.cpp")], check=True)
    lib = ctypes.CDLL(str(path / "h.so"))
    lib.run.restype = ctypes.c_uint64
    u64, i64 = ctypes.c_uint64, ctypes.c_int64

    def go(uses, stages, ended, landed, stop_at=NEVER, stopped=False, limit=2000 * MS):
        """Returns when it came back, and the stages that it asked about."""
        parity = [((max(u for u in range(s, uses, stages)) // stages) & 1) if s < uses else 0 for s in range(stages)]
        looked, bad = u64(), ctypes.c_int()
        t = lib.run(i64(uses), stages, int(stopped), u64(limit), u64(stop_at), (u64 * stages)(*ended), (u64 * stages)(*landed), (ctypes.c_uint32 * stages)(*parity),
                    ctypes.byref(looked), ctypes.byref(bad))
        assert not bad.value, "the phase of another use"
        return t, [s for s in range(stages) if looked.value >> s & 1]

    return go


@pytest.mark.parametrize("uses", [0, 1, 5, 11, 12, 40])
@pytest.mark.parametrize("stages", [3, 6, 11])
def test_it_stays_until_the_products_have_ended(run, uses, stages):
    ended = [MS * (s + 1) for s in range(stages)]
    t, looked = run(uses, stages, ended, [NEVER] * stages)
    used = list(range(min(uses, stages)))
    assert looked == used
    last = max([ended[s] for s in used], default=0)
    assert last <= t <= last + SLACK


@pytest.mark.parametrize("stages", [1, 3, 11])
@pytest.mark.parametrize("stop_at", [100, MS, 300 * MS])
@pytest.mark.parametrize("limit", [2000 * MS, 2 ** 63 - 1])
def test_a_cta_that_is_stopped_meanwhile_does_not_wait_for_its_products(run, stages, stop_at, limit):
    """Another thread's wait ran out: no product of this CTA will end. Its copies have landed, land a little later, or never do."""
    for landed in (0, stop_at + 5 * MS, NEVER):
        t, _ = run(4 * stages, stages, [NEVER] * stages, [landed] * stages, stop_at=stop_at, limit=limit)
        assert max(stop_at, landed if landed != NEVER else stop_at + LANDING) <= t <= stop_at + LANDING + SLACK
        if landed != NEVER:
            assert t <= max(stop_at, landed) + SLACK


@pytest.mark.parametrize("stages", [1, 3, 11])
def test_one_limit_for_all_stages(run, stages):
    t, _ = run(40, stages, [NEVER] * stages, [0] * stages, limit=100 * MS)
    assert 100 * MS <= t <= 100 * MS + SLACK
    t, _ = run(40, stages, [NEVER] * stages, [NEVER] * stages, limit=100 * MS)
    assert t <= 100 * MS + LANDING + SLACK


@pytest.mark.parametrize("stages", [1, 3, 11])
def test_a_cta_that_was_stopped_before_waits_for_its_copies_alone(run, stages):
    t, _ = run(40, stages, [NEVER] * stages, [3 * MS] * stages, stopped=True)
    assert 3 * MS <= t <= 3 * MS + SLACK
    t, _ = run(40, stages, [NEVER] * stages, [NEVER] * stages, stopped=True)
    assert LANDING <= t <= LANDING + SLACK
