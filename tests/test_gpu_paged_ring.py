"""The ring of free pages at its limits: what a step may take and hand back."""
import pytest

import test_gpu_paged as paged
from test_gpu_paged_window import Server

pytestmark = pytest.mark.gpu
pkg = paged.pkg


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 4)])
@pytest.mark.parametrize("cap,free,at", [(3, 3, 1), (4, 3, 2), (3, 2, 2), (2, 2, 0), (5, 4, 4), (4, 4, 3)])
def test_room_for_free_and_returned_pages(pkg, cap, free, at, window, sinks):
    """One sequence ends (a page), another takes a page: done if the pages free before and the one that comes back fit the ring together,
    whatever the step takes."""
    s = Server(pkg, 2, pages=8, width=6, window=window, sinks=sinks)
    s.step([16, 16])
    numbers = s.ring.tolist()
    ring = s.i32([-9] * cap)
    for i in range(free):
        ring[(at + i) % cap] = numbers[(s.books.state[0] + i) % 8]
    state, before = s.i32([at, free]), (s.table.clone(), s.lens.clone(), ring.clone())
    pkg.attn_paged_assign(s.kv, s.i32([-1, 1]), ring, state, window=window, sinks=sinks)
    if free + 1 <= cap:
        assert pkg.sync_status() == 0
        assert s.lens.tolist() == [0, 17] and state.tolist() == [(at + 1) % cap, free]
        assert s.table[1, 1] == before[2][at] and ring[(at + free) % cap] == before[0][0, 0]
    else:
        assert pkg.status_string(pkg.sync_status()) == "device-side check failed"
        assert s.lens.tolist() == [16, 16] and state.tolist() == [at, free]
        assert (s.table == before[0]).all() and (ring == before[2]).all()


def test_a_ring_of_all_pages_is_never_too_small(pkg):
    """All sequences end at once, with every page in use or free."""
    s = Server(pkg, 6, pages=12, width=2, at=7)
    s.step([32] * 6)
    s.step([-1] * 6)
    assert s.books.state[1] == 12
    s.step([32, 0, 32, 0, 1, 17])
    s.step([-1, 32, -1, 16, -1, -1])
    s.step([0, -1, 0, -1, 0, 0])
    assert s.books.state[1] == 12 and sorted(s.books.ring) == list(range(12))
