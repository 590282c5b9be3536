"""The paged 4-bit cache at the limits of what its calls may meet.  References and tolerances are test_kv4's."""
import pytest
import torch

from test_kv4 import BF, DEV, G, L, case, gpu   # noqa: F401 (fixtures)


def test_selftest_warp_wait_rejects_bad_arguments_without_device(L):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    lib, P = L.lib(), 4096   # a fake, never-dereferenced address
    assert lib.lcs_selftest_warp_wait(1000, None, 256, P, None) == L.LCS_ERR_INVALID
    assert lib.lcs_selftest_warp_wait(1000, P, 255, P, None) == L.LCS_ERR_INVALID
    assert lib.lcs_selftest_warp_wait(1000, P, 256, None, None) == L.LCS_ERR_INVALID
    assert lib.lcs_selftest_warp_wait(0, P, 256, P, None) == L.LCS_ERR_INVALID
    assert lib.lcs_selftest_warp_wait(1000001, P, 256, P, None) == L.LCS_ERR_INVALID
    assert lib.lcs_selftest_warp_wait(1000, P, 256, P, None) == L.LCS_ERR_CUDA


@gpu
@pytest.mark.parametrize("code,gave_up,held", [(0, 0, True), (-5, 0, True), (-4, 0, False), (-5, -4, False)])
def test_waits_outlast_another_requests_error(G, code, gave_up, held):
    """The attention's waits, on a barrier that completes after 50 ms, under a status word that is set already: one
    request's bad block ends no other request's wait; a wait of the grid that ran out ends them all."""
    ws, out = G.workspace(256), torch.full((2,), -1, dtype=torch.int64, device=DEV)
    ws[:12].view(torch.int32).copy_(torch.tensor([code, 602 if code else 0, gave_up], dtype=torch.int32))
    G.lcs_selftest_warp_wait(50000, ws, out)
    torch.cuda.synchronize()
    ok, ns = out.tolist()
    assert ok == held
    assert 40_000_000 <= ns < 1_000_000_000 if held else ns < 40_000_000
    assert ws[:4].view(torch.int32).item() == code           # what was recorded stays
    assert G.lcs_status(ws) == code and G.lcs_status(ws) == 0
    assert (ws == 0).all()


@gpu
@pytest.mark.parametrize("d_c,d_r,dt", [(512, 64, BF), (64, 16, torch.float32)])
@pytest.mark.parametrize("op", ["csa", "hca"])
def test_window_positions_of_any_size(G, op, d_c, d_r, dt):
    """A query before the window's first row sees none of it and one far past it none either, also where the
    difference of the two positions passes 64 bits (it must not wrap to a small one)."""
    top, low = (1 << 63) - 1, -(1 << 63)
    win0 = [top, low, top - 1, 0]
    pos = [[low, low + 1, top, -1], [top, top - 1, low, low + 3], [low, low + 20, top, 5], [low, top, 7, -1]]
    case(G, op, 4, 30, 4, 8, d_c, d_r, dt, Tw=20, k=9, Q=4, q_pos=pos, win_pos0=win0, m=3, W=6, seed=1)
    case(G, op, 4, 0, 4, 8, d_c, d_r, dt, Tw=1, k=9, Q=4, q_pos=pos, win_pos0=win0, m=3, W=1, seed=2)
