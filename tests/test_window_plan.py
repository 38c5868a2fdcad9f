"""How the windowed backward cuts tiles of keys into runs, seen by the workspace that it
asks for: by the number of query tiles that see a tile, counted here pair by pair.  No
GPU is needed."""
import pytest

from io_aware_exact_12_gb300 import build as build_mod


@pytest.fixture(scope="module")
def pkg():
    build_mod.build()
    import io_aware_exact_12_gb300 as p
    p.lib()
    return p


def _visits(nq, nk, window):
    """The most query tiles that see a key tile."""
    off, seen = nk - nq, {}
    for i in range(nq):
        for t in range(max(0, i + off - window + 1) // 128, (i + off) // 128 + 1):
            seen.setdefault(t, set()).add(i // 128)
    return max(len(s) for s in seen.values())


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 200, 255, 256, 300, 1000])
@pytest.mark.parametrize("off", [0, 1, 64, 127, 128, 130, 255])
def test_runs_follow_the_visits(pkg, window, off):
    nq, d = 2048, 64
    nk, tiles = nq + off, -(-(nq + off) // 128)
    for G, hk in ((1, 1), (2, 3), (3, 2), (8, 1), (8, 5)):
        visits, w_tiles = G * _visits(nq, nk, window), hk * tiles
        cut = w_tiles % 152
        runs = min(152 // cut, (visits + 1) // 2, 16) if cut else 1
        if visits - -(-visits // runs) < 8:
            cut = runs = 0
        need = pkg.lib().attn_bwd_window_workspace(1, G * hk, hk, nq, nk, d, window, 0)
        partial = need - 2 * G * hk * nq * 4
        tile = 2 * 128 * d * 4
        assert partial // tile == cut * runs, (G, hk)  # (less than a tile beside them: the rows' norms)
