"""The paged 4-bit cache at the limits of what its calls may meet.  References and tolerances are test_kv4's."""
import math

import pytest
import torch

from test_kv4 import BF, DEV, G, L, case, gen, gpu, make_pool   # noqa: F401 (fixtures)


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


@gpu
def test_page_plan_of_long_requests(G):
    """Tables of large blocks hold more than 2^40 tokens: block and slot of the entry that completes are those of
    the length itself; lengths that no table holds are refused, whatever their size."""
    P, wide = 1 << 20, (1 << 21) + 3
    lens = torch.tensor([1 << 41, 5, (1 << 40) + P, 1 << 60], device=DEV)
    new = torch.tensor([P, P, 3 * P, 0], device=DEV)
    free = torch.arange(90, 100, dtype=torch.int32, device=DEV)
    table = torch.full((4, wide), -9, dtype=torch.int32, device=DEV)
    table[1, 0] = 7
    ws = G.workspace(256)
    slots, off, slots2, off2, taken = G.lcs_page_plan(lens, new, free, table, block_tokens=P, m=P // 2, max_slots=20, m2=P,
                                                      max_slots2=9, ws=ws)
    assert G.lcs_status(ws) == 0
    want = torch.full((4, wide), -9, dtype=torch.int32)
    want[0, 1 << 21] = 90
    want[1, 0], want[1, 1] = 7, 91
    want[2, (1 << 20) + 1:(1 << 20) + 4] = torch.tensor([92, 93, 94], dtype=torch.int32)
    assert torch.equal(table.cpu(), want) and taken.item() == 5
    assert off.tolist() == [0, 2, 4, 10, 10] and off2.tolist() == [0, 1, 2, 5, 5]
    # request 1 completes half-block entries 0, 1 of block 7; the others fill whole new blocks
    assert slots.tolist() == [180, 181, 14, 15, 184, 185, 186, 187, 188, 189] + [-1] * 10
    assert slots2.tolist() == [90, 7, 92, 93, 94] + [-1] * 4
    for n, a in (((1 << 41) + 3 * P, 1), (1 << 62, 1), ((1 << 63) - 1, (1 << 63) - 1), (0, (1 << 63) - 1), (0, 1 << 52), (1 << 45, 1 << 41)):
        t = want.to(DEV)
        out = G.lcs_page_plan(torch.tensor([0, n] * 20, device=DEV), torch.tensor([0, a] * 20, device=DEV), free,
                              t[:1].repeat(40, 1), block_tokens=P, m=1, max_slots=20, ws=ws)
        assert G.lcs_status(ws) == -5 and out[4].item() == 0 and (out[0] == -1).all() and (out[1] == 0).all(), (n, a)


@gpu
@pytest.mark.parametrize("N,Tw", [(20, 20), (300, 0), (2000, 20), (8000, 128)])
@pytest.mark.parametrize("d_c,d_r,dt", [(512, 64, BF), (64, 16, torch.float32), (512, 64, torch.float32)])
def test_a_head_that_is_no_number(G, N, Tw, d_c, d_r, dt):
    """One split, splits merged in their cluster and by a second kernel, CUDA cores: a NaN in a head's query gives that
    head NaN outputs and a NaN log-sum, not the -inf of a query without rows, and the other heads what they had."""
    B, H, D, be = 2, 9, d_c + d_r, 16
    width = -(-N // be)
    pool = make_pool(G, B * width, be, d_c, d_r, 1)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    n = torch.full((B,), N, device=DEV)
    q = torch.randn((B, 1, H, D), generator=gen(2), device=DEV).to(dt)
    win = torch.randn((B, Tw, D), generator=gen(3), device=DEV).to(dt) if Tw else None
    idx = torch.arange(min(N, 1000), dtype=torch.int32, device=DEV).repeat(B, 1, 1).contiguous()
    bad = q.clone()
    bad[0, 0, 4, 7] = math.nan          # a content dim
    bad[1, 0, 0, D - 1] = math.nan      # a RoPE dim
    hit = torch.zeros((B, 1, H), dtype=torch.bool, device=DEV)
    hit[0, 0, 4] = hit[1, 0, 0] = True
    for call in (lambda q: G.hca_attend_kv4(q, pool, table, n, win, D ** -0.5, d_c=d_c, want_lse=True, out_dtype=torch.float32),
                 lambda q: G.csa_attend_kv4(q, pool, table, n, win, idx, D ** -0.5, d_c=d_c, want_lse=True)):
        want, wl = call(q)
        o, lse = call(bad)
        assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
        assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit])


@gpu
def test_errors_of_calls_without_a_workspace(G):
    """Without a workspace there is no status word to read later: the call itself raises what its kernels recorded."""
    i32 = torch.int32
    z = lambda v, dt=torch.int64: torch.tensor(v, dtype=dt, device=DEV)
    pool = make_pool(G, 8, 16, 512, 64, 0)
    table = torch.arange(8, dtype=i32, device=DEV).view(2, 4)
    n = z([60, 60])
    q = torch.randn((2, 1, 8, 576), generator=gen(1), device=DEV).to(BF)
    win = torch.randn((2, 20, 576), generator=gen(2), device=DEV).to(BF)
    big, bad = win.clone(), table.clone()
    big[1, 3, 5] = 2.0 ** 17
    bad[0, 1] = 8
    idx = torch.full((2, 1, 4), 60, dtype=i32, device=DEV)
    x = torch.randn((2, 576), generator=gen(3), device=DEV)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for kw in ({}, {"stream": st}):
        for call in (lambda: G.lcs_page_plan(z([0]), z([300]), z([1, 2, 3], i32), z([[0, 0, 0]], i32), max_slots=74, **kw),
                     lambda: G.lcs_page_plan(z([3]), z([1]), z([1], i32), z([[0]], i32), **kw),
                     lambda: G.lcs_kv4_store(x, z([0, 128]), pool.clone(), **kw),
                     lambda: G.lcs_kv4_load(pool, z([128, 3]), **kw),
                     lambda: G.hca_attend_kv4(q, pool, bad, n, win, 0.1, **kw),
                     lambda: G.hca_attend_kv4(q, pool, table, z([60, 65]), win, 0.1, **kw),
                     lambda: G.hca_attend_kv4(q, pool, table, n, big, 0.1, **kw),
                     lambda: G.hca_attend_kv4(q.float(), pool, bad, n, win.float(), 0.1, **kw),
                     lambda: G.csa_attend_kv4(q, pool, table, n, win, idx, 0.1, **kw)):
            torch.cuda.synchronize()
            with pytest.raises(G.LcsError) as e:
                call()
            assert e.value.code == -5
    # the calls that are right, and those with a workspace, raise nothing
    slots, off, _, _, taken = G.lcs_page_plan(z([0]), z([300]), z([1, 2, 3], i32), z([[0, 0, 0]], i32), max_slots=75)
    assert taken.item() == 3 and off.tolist() == [0, 75]
    want = G.hca_attend_kv4(q, pool, table, n, win, 0.1)
    ws = G.workspace(G.lcs_workspace_size(G.OP_ATTEND_KV4, 2, 1, 64, 20, 0, 8))
    G.hca_attend_kv4(q, pool, bad, n, win, 0.1, ws=ws)
    assert G.lcs_status(ws) == -5
    # a captured call cannot wait for its kernels
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = G.hca_attend_kv4(q, pool, table, n, win, 0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


@gpu
def test_page_plan_with_the_most_slots(G):
    """max_slots up to 2^31 - 1: the last turn's slot indexes end there; every slot behind the last entry is -1."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    z = lambda v, dt=torch.int64: torch.tensor(v, dtype=dt, device=DEV)
    for most in ((1 << 31) - 1, (1 << 31) - 98):
        table, ws = torch.full((2, 5), -1, dtype=torch.int32, device=DEV), G.workspace(256)
        slots, off, _, _, taken = G.lcs_page_plan(z([0, 7]), z([300, 90]), z([4, 1, 3, 9], torch.int32), table, max_slots=most, ws=ws)
        assert G.lcs_status(ws) == 0 and taken.item() == 3 and off.tolist() == [0, 75, 98]
        # request 1 holds its first block's first entry: that block is its own table's entry 0, which is -1 here
        assert slots[:75].tolist() == [b * 32 + j for b in (4, 1, 3) for j in range(32)][:75]
        assert all((part == -1).all() for part in slots[75:].split(1 << 28))
        del slots, off, taken


@gpu
def test_values_on_a_second_device(G):
    """After the same calls on device 0, device 1 gives the same bytes: a plan, stored and loaded rows, attention with one
    split, splits in clusters, splits merged by a kernel, and on CUDA cores with opted-in shared memory."""
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two devices")

    def all_calls(dev):
        g = torch.Generator("cpu").manual_seed(1)
        r = lambda *s: torch.randn(s, generator=g).to(dev)
        i = lambda v, dt=torch.int64: torch.tensor(v, dtype=dt, device=dev)
        ws = G.workspace(1 << 26, dev)
        table = i([[-1] * 700], torch.int32)
        out = list(G.lcs_page_plan(i([0]), i([700 * 16]), torch.arange(700, dtype=torch.int32, device=dev), table, block_tokens=16, m=1,
                                   max_slots=700 * 16, ws=ws)[:2]) + [table]
        slots = out[0]
        pool = torch.zeros((700, 16, 400), dtype=torch.uint8, device=dev)
        G.lcs_kv4_store(r(700 * 16, 576), slots, pool, ws=ws)
        out += [pool, G.lcs_kv4_load(pool, slots, ws=ws)]
        q, win, idx = r(1, 1, 64, 576).to(BF), r(1, 128, 576).to(BF), torch.arange(0, 900, 3, dtype=torch.int32, device=dev).view(1, 1, 300)
        for n, width in ((20, 2), (300, 20), (11200, 700)):
            t = table[:, :width].contiguous()
            out += G.hca_attend_kv4(q, pool, t, i([n]), win, 1 / 24, want_lse=True, ws=ws)
            out += G.hca_attend_kv4(q.float(), pool, t, i([n]), win.float(), 1 / 24, want_lse=True, ws=ws)
        out += G.csa_attend_kv4(q, pool, table, i([11200]), win, idx, 1 / 24, want_lse=True, ws=ws)
        st = int(ws[:4].view(torch.int32))
        return [o.cpu() for o in out] + [torch.tensor(st)]

    first, second = all_calls(torch.device("cuda", 0)), all_calls(torch.device("cuda", 1))
    assert first[-1] == 0 and second[-1] == 0
    for a, b in zip(first, second):
        assert torch.equal(a, b)


@gpu
def test_small_window_values(G):
    """One window row alone is the output: content is exact from 2^-17 up and off by at most 2^-25 below."""
    v = torch.arange(128, 256, device=DEV) * 2.0 ** -24                                  # every bf16 value of [2^-17, 2^-16)
    small = torch.randint(-255, 256, (256,), generator=gen(1), device=DEV) * 2.0 ** -27
    win = torch.cat((v, -4 * v, small, torch.zeros(64, device=DEV))).to(BF).view(1, 1, 576)
    q = torch.randn((1, 1, 64, 576), generator=gen(2), device=DEV).to(BF)
    z = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    o = G.hca_attend_kv4(q, make_pool(G, 1, 1, 512, 64, 3), z, z[0].long(), win, 1 / 24, out_dtype=torch.float32)[0, 0]
    want = win[0, 0, :512].double()
    assert torch.equal(o[:, :256].double(), want[:256].expand(64, 256))
    assert ((o.double() - want).abs() <= 2.0 ** -25).all() and (o[:, 256:] != 0).any()


@gpu
def test_small_weights(G):
    """Two window rows whose scores lie (h + 1) / 2 apart, content 0 and 1: the output is the second's weight, off by at
    most 2^-11 of itself or 2^-31 of the first's, and by the 2^-17 of exp2 and its argument; the log-sum has all of it."""
    win = torch.zeros((1, 2, 576), device=DEV)
    win[0, 1, :512], win[0, 1, 512] = 1, 1
    q = torch.zeros((1, 1, 64, 576), device=DEV)
    q[0, 0, :, 512] = -(torch.arange(64, device=DEV) + 1) / 2
    z = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    o, lse = G.hca_attend_kv4(q.to(BF), make_pool(G, 1, 1, 512, 64, 3), z, z[0].long(), win.to(BF), 1.0, want_lse=True, out_dtype=torch.float32)
    e = torch.exp(q[0, 0, :, 512].double())
    p = (e / (1 + e))[:, None]
    tol = torch.clamp(p * 2.0 ** -11, min=2.0 ** -31) + p * 2.0 ** -17
    assert ((o[0, 0].double() - p).abs() <= tol).all()
    assert ((lse[0, 0].double() - torch.log1p(e)).abs() <= 2.0 ** -18).all()
