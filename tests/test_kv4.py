"""The paged compressed cache in 4 bits: block tables and slots (lcs_page_plan), stored rows
(lcs_kv4_store, lcs_kv4_load) and the attention over them (csa_attend_kv4, hca_attend_kv4).

References are plain Python / float64 torch written from the formulas in include/lcs.h.

Tolerances (derived, per element, from the data of the test):
  * plans and stored rows: equal;
  * a score differs from the exact one by at most delta = |scale| * (D/16 + 2) * 2^-23 * sum|q||k|
    (the tensor cores' fp32 partial sums, 16 products each, with one truncation per step; the CUDA-core
    path sums D terms with a rounding of 2^-24 each: D * 2^-24 in place of (D/16 + 2) * 2^-23);
  * a weight p_r / l then has the relative error 2 delta (its own and the sum's) + 2^-21 (exp2 and
    the scaling of its argument: arguments up to 2^5 lose 2^-24 * 2^5 = 2^-19: counted as 2^-18),
    plus its own rounding, 2^-11 (fp16; none on the CUDA cores); window content below 2^-14 is off by
    2^-25 on the tensor cores (fp16's subnormals), in the scores and in the values; weights below the
    smallest fp16 step 2^-24 / 2^6 of the largest lose that much absolutely; the sum over R rows in fp32
    adds (R/16 + 2) * 2^-23 of sum p|v|;
  * a bf16 output is off by half a step, 2^-8 |o|; fp32 by 2^-24 |o|.
"""
import math

import numpy as np
import pytest
import torch

DEV = "cuda"
LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from long_context_sparse_06_b200 import build
    build.build()
    import long_context_sparse_06_b200 as lcs
    lcs.lib()
    return lcs


@pytest.fixture(scope="module")
def G(L):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    return L


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


# ------------------------------------------------------------------ plain references
def plan_ref(lens, new, free, table, P, m, max_slots):
    """Python loops over the definition; table is a list of lists (changed), -> (slots, offsets, taken)."""
    taken = 0
    for b, (n, a) in enumerate(zip(lens, new)):
        if n < 0 or a <= 0:
            continue
        for i in range(-(-n // P), -(-(n + a) // P)):
            table[b][i] = free[taken]
            taken += 1
    slots, off = [], [0]
    for b, (n, a) in enumerate(zip(lens, new)):
        if n >= 0 and a > 0:
            for j in range(n // m, (n + a) // m):
                slots.append(table[b][j * m // P] * (P // m) + j % (P // m))
        off.append(len(slots))
    return slots + [-1] * (max_slots - len(slots)), off, taken


def decode_rows(rows, d_c, d_r):
    """Stored rows [n, bytes] uint8 -> float64 [n, d_c + d_r]."""
    packed = rows[:, :d_c // 2].long()
    codes = torch.stack((packed & 15, packed >> 4), -1).reshape(rows.shape[0], d_c)
    val = torch.tensor(LUT + tuple(-v for v in LUT), dtype=torch.float64, device=rows.device)[codes]
    sc = rows[:, d_c // 2 + 2 * d_r:d_c // 2 + 2 * d_r + d_c // 32].contiguous().view(torch.float8_e4m3fn).double()
    rope = rows[:, d_c // 2:d_c // 2 + 2 * d_r].contiguous().view(torch.bfloat16).double()
    return torch.cat((val * sc.repeat_interleave(32, 1), rope), 1)


def attend_ref(q, K, n_comp, d_c, scale, tc):
    """Float64 attention of q [H, D] over rows K [R, D], the first n_comp of them compressed:
    (o, bound on an fp32 o, lse, bound on lse)."""
    q, K = q.double(), K.double()
    H, D = q.shape
    R = K.shape[0]
    if R == 0:
        z = torch.zeros((H, d_c), dtype=torch.float64, device=q.device)
        return z, z, torch.full((H,), -math.inf, dtype=torch.float64, device=q.device), z[:, 0]
    s = (q @ K.T) * scale
    mags = (q.abs() @ K.abs().T) * abs(scale)
    delta = mags * ((D / 16 + 2) * 2.0 ** -23 if tc else D * 2.0 ** -24) + s.abs() * 2.0 ** -22
    if tc:
        delta[:, n_comp:] += abs(scale) * q.abs().sum(-1, keepdim=True) * 2.0 ** -25
    p = torch.softmax(s, -1)
    V = K[:, :d_c]
    o = p @ V
    off = p[:, n_comp:].sum(-1, keepdim=True) * 2.0 ** -25 if tc else 0.0
    dmax = delta.amax(-1, keepdim=True)
    rel = 2 * dmax + 2.0 ** -18 + torch.zeros_like(s)
    if tc:
        rel += 2.0 ** -11
    rel = rel + (R / 16 + 2 if tc else R) * 2.0 ** -23
    pa = p * rel + ((2.0 ** -31) * p.amax(-1, keepdim=True) if tc else 0.0)
    bound = pa @ V.abs() + off + 1e-30
    return o, bound, torch.logsumexp(s, -1), dmax[:, 0] + 2.0 ** -18 + torch.logsumexp(s, -1).abs() * 2.0 ** -22


def make_pool(L, n_blocks, be, d_c, d_r, seed, heavy=False):
    """A pool of stored random rows, written by the library (its bytes are tested below)."""
    g = gen(seed)
    x = torch.randn((n_blocks * be, d_c + d_r), generator=g, device=DEV)
    if heavy:
        x = torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.01, x * 20, x)
    pool = torch.full((n_blocks, be, L.kv_fp4_row_bytes(d_c, d_r)), 0xFF, dtype=torch.uint8, device=DEV)
    if x.shape[0]:
        L.lcs_kv4_store(x, torch.arange(n_blocks * be, device=DEV), pool, d_c=d_c)
    return pool


# ------------------------------------------------------------------ refusals (no device)
def test_refusals_without_device(L):
    lib = L.lib()
    P = 4096   # a fake, aligned, never-dereferenced address
    big = 1 << 20
    plan = lambda **k: lib.lcs_page_plan(*[{**dict(B=2, len=P, n=P, bt=128, fb=P, nf=8, t=P, mb=4, m=4, s=P, ms=8, o=P, m2=0,
                                                   s2=None, ms2=0, o2=None, tk=P, ws=P, wb=256, st=None), **k}[i] for i in
                                           ("B", "len", "n", "bt", "fb", "nf", "t", "mb", "m", "s", "ms", "o", "m2", "s2", "ms2",
                                            "o2", "tk", "ws", "wb", "st")])
    for bad in (dict(B=-1), dict(len=None), dict(n=None), dict(bt=0), dict(bt=130), dict(fb=None), dict(t=None), dict(m=0),
                dict(s=None), dict(o=None), dict(tk=None), dict(m2=3, s2=P, ms2=4, o2=P), dict(m2=128, ms2=4, o2=P),
                dict(m2=128, s2=P, ms2=4), dict(ms=-1), dict(mb=-1), dict(nf=-1)):
        assert plan(**bad) == -1, bad
    assert plan(B=8193) == -2
    assert plan(ws=None) == -6 and plan(wb=128) == -6 and plan(ws=P + 8) == -6
    for bad in ((None, 0, 4, 512, 64, P, P, 8), (P, 0, 4, 512, 64, None, P, 8), (P, 0, 4, 512, 64, P, None, 8),
                (P, 0, -1, 512, 64, P, P, 8), (P, 0, 4, 48, 64, P, P, 8), (P, 0, 4, 544, 64, P, P, 8), (P, 0, 4, 512, 4, P, P, 8),
                (P, 0, 4, 512, 136, P, P, 8), (P + 4, 0, 4, 512, 64, P, P, 8), (P, 0, 4, 512, 64, P, P + 8, 8),
                (P, 0, 4, 512, 64, P, P, -1)):
        assert lib.lcs_kv4_store(*bad, P, 256, None) == -1, bad
    assert lib.lcs_kv4_store(P, 2, 4, 512, 64, P, P, 8, P, 256, None) == -2
    assert lib.lcs_kv4_store(P, 0, 4, 512, 64, P, P, 8, None, 256, None) == -6
    assert lib.lcs_kv4_load(None, 8, P, 4, 512, 64, P, 1, P, 256, None) == -1
    assert lib.lcs_kv4_load(P, 8, P, 4, 512, 64, None, 1, P, 256, None) == -1
    assert lib.lcs_kv4_load(P, 8, P, 4, 512, 64, P + 2, 1, P, 256, None) == -1
    assert lib.lcs_kv4_load(P, 8, P, 4, 512, 64, P, 3, P, 256, None) == -2
    assert lib.lcs_kv4_load(P, 8, P, 4, 512, 64, P, 1, P, 255, None) == -6
    base = dict(q=P, qd=1, pool=P, nb=9, be=32, t=P, mb=4, ne=P, win=P, nw=None, B=2, Q=1, Tw=128, idx=P, k=8, qp=None, wp=None,
                W=128, H=64, dc=512, dr=64, sc=0.1, out=P, od=1, lse=None, ws=P, wb=1 << 30, st=None)

    def csa(**k):
        a = {**base, **k}
        return lib.csa_attend_kv4(*[a[i] for i in ("q", "qd", "pool", "nb", "be", "t", "mb", "ne", "win", "nw", "B", "Q", "Tw", "idx",
                                                   "k", "qp", "wp", "W", "H", "dc", "dr", "sc", "out", "od", "lse", "ws", "wb", "st")])

    def hca(**k):
        a = {**base, **dict(m=128), **k}
        return lib.hca_attend_kv4(*[a[i] for i in ("q", "qd", "pool", "nb", "be", "t", "mb", "ne", "win", "nw", "B", "Q", "Tw", "qp",
                                                   "wp", "m", "W", "H", "dc", "dr", "sc", "out", "od", "lse", "ws", "wb", "st")])

    for f in (csa, hca):
        for bad in (dict(q=None), dict(out=None), dict(ne=None), dict(t=None), dict(pool=None), dict(win=None), dict(B=-1),
                    dict(Q=-1), dict(be=0), dict(W=0), dict(H=0), dict(dc=500), dict(dc=1024), dict(dr=7), dict(Q=2),
                    dict(qp=P), dict(wp=P), dict(qp=P, wp=P, nw=P), dict(q=P + 2), dict(pool=P + 8), dict(win=P + 8),
                    dict(out=P + 4), dict(Tw=-1), dict(mb=-1), dict(nb=-1)):
            assert f(**bad) == -1, (f.__name__, bad)
        for bad in (dict(H=129), dict(qd=2), dict(qd=4), dict(od=2), dict(mb=1 << 27), dict(B=1 << 24), dict(nb=1 << 31),
                    dict(be=1, mb=(1 << 31) - (1 << 16) - 128), dict(Tw=(1 << 31) - (1 << 16))):
            assert f(**bad) == -2, (f.__name__, bad)
        for bad in (dict(ws=None), dict(wb=16), dict(ws=P + 64)):
            assert f(**bad) == -6, (f.__name__, bad)
    assert csa(idx=None) == -1 and csa(k=-1) == -1 and csa(k=4097) == -1
    assert hca(m=0) == -1
    assert lib.lcs_workspace_size(L.OP_ATTEND_KV4, 2, 1, 128, 128, 8, 0, 512, 0) == -1
    assert lib.lcs_workspace_size(L.OP_ATTEND_KV4, 2, 1, 128, 128, 8, 64, 512, 0) >= 256
    if not torch.cuda.is_available():
        assert plan() == -3 and csa() == -3 and hca() == -3
        assert plan(B=0) == -3 and csa(B=0) == -3 and hca(B=0) == -3 and hca(Q=0, qp=P, wp=P) == -3
        assert lib.lcs_kv4_store(P, 0, 4, 512, 64, P, P, 8, P, 256, None) == -3
        assert lib.lcs_kv4_load(P, 8, P, 4, 512, 64, P, 1, P, 256, None) == -3


def test_the_workspace_size_covers_every_window(L):
    """Fewer window rows can mean more splits: lcs_workspace_size holds for any W up to Tw."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only where nothing can be launched")
    lib, P = L.lib(), 4096
    for B, Q, N, Tw, k, H in ((1, 1, 200, 384, 64, 64), (1, 1, 1500, 300, 500, 128), (4, 1, 900, 128, 300, 64), (3, 1, 4000, 5000, 100, 64),
                              (2, 3, 700, 240, 333, 64), (9, 1, 640, 200, 512, 64), (1, 1, 0, 600, 0, 64)):
        size = L.lcs_workspace_size(L.OP_ATTEND_KV4, B, Q, N, Tw, k, H, 512)
        for W in range(1, Tw + 30, 7):
            args = (P, 1, P, 9, 1, P, N, P, P, None, B, Q, Tw)
            dims = (H, 512, 64, 0.1, P, 1, None, P, size, None)
            assert lib.csa_attend_kv4(*args, P, k, P, P, W, *dims) == -3, (B, Q, N, Tw, W)
            assert lib.hca_attend_kv4(*args, P, P, 4, W, *dims) == -3, (B, Q, N, Tw, W)


def test_binding_refuses_cpu_and_mismatched_tensors(L):
    z = torch.zeros
    i64 = torch.int64
    with pytest.raises(ValueError):
        L.lcs_kv4_store(z(2, 576), z(2, dtype=torch.int32), z((4, 400), dtype=torch.uint8))
    with pytest.raises(ValueError):
        L.lcs_kv4_store(z(2, 576), z(2, dtype=i64), z((4, 401), dtype=torch.uint8))
    with pytest.raises(ValueError):
        L.lcs_kv4_store(z(2, 576), z(3, dtype=i64), z((4, 400), dtype=torch.uint8))
    with pytest.raises(ValueError):
        L.hca_attend_kv4(z(1, 1, 64, 576), z((2, 4, 400), dtype=torch.uint8), z((1, 2), dtype=i64), z(1, dtype=i64), None, 0.1)
    with pytest.raises(ValueError):
        L.hca_attend_kv4(z(1, 1, 64, 576), z((2, 4, 400), dtype=torch.uint8), z((1, 2), dtype=torch.int32), z(1, dtype=i64),
                         z((1, 8, 576), dtype=torch.bfloat16), 0.1)
    with pytest.raises(ValueError):
        L.lcs_page_plan(z(2, dtype=i64), z(3, dtype=i64), z(4, dtype=torch.int32), z((2, 2), dtype=torch.int32))


# ------------------------------------------------------------------ page plan
def run_plan(L, lens, new, free, table, P, m, ms, m2=0, ms2=0, ws=None):
    t = lambda v, d: torch.tensor(v, dtype=d, device=DEV)
    tab = t(table, torch.int32).reshape(len(lens), -1)
    ws = ws if ws is not None else L.workspace(256)
    out = L.lcs_page_plan(t(lens, torch.int64), t(new, torch.int64), t(free, torch.int32), tab, block_tokens=P, m=m, max_slots=ms,
                          m2=m2, max_slots2=ms2, ws=ws)
    return tab, out, L.lcs_status(ws)


@gpu
@pytest.mark.parametrize("B,P,m,m2,most", [(1, 128, 4, 128, 1), (1, 128, 4, 128, 1000), (3, 128, 4, 128, 300), (33, 128, 4, 0, 700),
                                           (7, 4, 4, 2, 9), (5, 1, 1, 0, 6), (511, 128, 4, 128, 200), (512, 16, 4, 8, 40),
                                           (513, 128, 128, 4, 260), (8192, 128, 4, 128, 12), (4094, 128, 4, 128, 9), (4095, 128, 4, 128, 9)])
def test_page_plan(G, B, P, m, m2, most):
    rng = np.random.RandomState(B + most)
    lens = rng.randint(0, 3 * P + 5, B).tolist()
    new = rng.randint(0, most + 1, B).tolist()
    if B > 4:
        new[1], new[2], lens[3] = 0, -7, -5
    width = max((max(n, 0) + max(a, 0) + P - 1) // P for n, a in zip(lens, new)) + 2
    ids = rng.permutation(B * width + 9).tolist()
    table = [[ids.pop() if i * P < n else -9 for i in range(width)] for n in lens]
    tot = lambda mm: sum((n + a) // mm - n // mm for n, a in zip(lens, new) if n >= 0 and a > 0)
    ms, ms2 = tot(m) + 5, (tot(m2) + 3 if m2 else 0)
    tab, (s, off, s2, off2, taken), st = run_plan(G, lens, new, ids, table, P, m, ms, m2, ms2)
    want = [list(r) for r in table]
    ws, woff, wt = plan_ref(lens, new, ids, want, P, m, ms)
    assert st == 0
    assert tab.cpu().tolist() == want
    assert s.cpu().tolist() == ws and off.cpu().tolist() == woff and taken.item() == wt
    if m2:
        w2, woff2, _ = plan_ref(lens, new, ids, [list(r) for r in table], P, m2, ms2)
        assert s2.cpu().tolist() == w2 and off2.cpu().tolist() == woff2
    else:
        assert s2 is None and off2 is None


@gpu
def test_page_plan_empty_and_exact_fit(G):
    ws = G.workspace(256)
    z = lambda *sh, dt=torch.int64: torch.zeros(sh, dtype=dt, device=DEV)
    s, off, s2, off2, taken = G.lcs_page_plan(z(0), z(0), z(2, dt=torch.int32), z(0, 4, dt=torch.int32), max_slots=3, m2=128,
                                              max_slots2=0, ws=ws)
    assert s.cpu().tolist() == [-1] * 3 and off.cpu().tolist() == [0] and off2.cpu().tolist() == [0] and taken.item() == 0
    assert G.lcs_status(ws) == 0
    # every free block, table entry and slot used
    tab, (s, off, _, _, taken), st = run_plan(G, [0], [512], [7, 3, 5, 1], [[-1] * 4], 128, 4, 128)
    assert st == 0 and taken.item() == 4 and tab.cpu().tolist() == [[7, 3, 5, 1]]
    assert s.cpu().tolist() == [b * 32 + j for b in (7, 3, 5, 1) for j in range(32)]


@gpu
@pytest.mark.parametrize("what", ["free", "table", "slots", "slots2", "huge"])
def test_page_plan_that_does_not_fit_takes_nothing(G, what):
    lens, new = [100, 0, 640], [300, 40, 10]
    free, width, ms, ms2 = [4, 9, 2, 8, 6], 6, 100, 10
    if what == "free":
        free = free[:3]
    elif what == "table":
        width = 5     # request 2 needs a sixth block
    elif what == "slots":
        ms = 85
    elif what == "slots2":
        ms2 = 2
    else:
        new[1] = 1 << 50
    table = [[70 + b * 10 + i for i in range(width)] for b in range(3)]
    tab, (s, off, s2, off2, taken), st = run_plan(G, lens, new, free, table, 128, 4, ms, 128, ms2)
    assert st == -5
    assert tab.cpu().tolist() == table and taken.item() == 0
    assert s.cpu().tolist() == [-1] * ms and s2.cpu().tolist() == [-1] * ms2
    assert off.cpu().tolist() == [0] * 4 and off2.cpu().tolist() == [0] * 4
    # the same call with room
    if what != "huge":
        _, out, st = run_plan(G, lens, new, [4, 9, 2, 8, 6], [[0] * 6 for _ in range(3)], 128, 4, 100, 128, 10)
        assert st == 0 and out[4].item() == 5


# ------------------------------------------------------------------ stored rows
def store_values(kind, n, d, seed):
    g = gen(seed)
    x = torch.randn((n, d), generator=g, device=DEV)
    if kind == "heavy":
        x = torch.where(torch.rand((n, d), generator=g, device=DEV) < 0.02, x * 50, x)
    elif kind == "tiny":
        x = x * 2.0 ** -12        # scales among E4M3's subnormals, and zero scales
    elif kind == "huge":
        x = x * 4000.0            # scales saturate at 448
    elif kind == "ties":          # exact midpoints of the code grid, signed zeros, empty blocks
        x = torch.randint(-28, 29, (n, d), generator=g, device=DEV) / 4.0
        x[:, ::32] = 6.0
        x[::3] = -0.0
    return x


@gpu
@pytest.mark.parametrize("d_c,d_r", [(512, 64), (32, 0), (32, 8), (96, 16), (480, 128), (64, 16)])
@pytest.mark.parametrize("kind", ["normal", "heavy", "tiny", "huge", "ties"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_equal_the_fp4_quantiser(G, orc, d_c, d_r, kind, dt):
    """The stored bytes are lcs_quant_fp4's codes and scales (pinned to the oracle elsewhere) and the
    bf16 RoPE dims; what is loaded is exactly their values."""
    n = 37
    x = store_values(kind, n, d_c + d_r, d_c + d_r).to(dt)
    slots = torch.randperm(50, generator=gen(3), device=DEV)[:n].contiguous()
    slots[5] = -1
    slots[36] = -(1 << 40)
    pool = torch.full((10, 5, G.kv_fp4_row_bytes(d_c, d_r)), 0xA5, dtype=torch.uint8, device=DEV)
    ws = G.workspace(256)
    G.lcs_kv4_store(x, slots, pool, d_c=d_c, ws=ws)
    assert G.lcs_status(ws) == 0
    planes = G.lcs_quant_fp4(x[:, :d_c].float().contiguous())
    codes, scales = planes[:n * d_c // 2].view(n, -1), planes[n * d_c // 2:].view(n, -1)
    rows = torch.full_like(pool.view(50, -1), 0xA5)
    keep = slots >= 0
    want = torch.zeros((n, pool.shape[-1]), dtype=torch.uint8, device=DEV)
    want[:, :d_c // 2] = codes
    if d_r:
        want[:, d_c // 2:d_c // 2 + 2 * d_r] = x[:, d_c:].to(torch.bfloat16).contiguous().view(torch.uint8)
    want[:, d_c // 2 + 2 * d_r:d_c // 2 + 2 * d_r + d_c // 32] = scales
    rows[slots[keep]] = want[keep]
    assert torch.equal(pool.view(50, -1), rows)
    vals = decode_rows(want, d_c, d_r)
    vals[~keep] = 0
    for od in (torch.float32, torch.bfloat16):
        got = G.lcs_kv4_load(pool, slots, d_c=d_c, d_r=d_r, out_dtype=od, ws=ws)
        assert torch.equal(got.double(), vals)
    assert G.lcs_status(ws) == 0


@gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_at_the_code_grids_midpoints(G, dt):
    """Every scale with every midpoint times it and the values one step of the type beside it, signed zeros and
    infinities: the quotient's codes (zeros keep their sign, infinities saturate with theirs)."""
    scales = torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(1, 127)])
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    at = scales[:, None] * mids                                        # exact in either type
    ints = torch.int32 if dt == torch.float32 else torch.int16
    step = lambda d: (at.to(dt).view(ints) + d).view(dt).float()
    x = torch.cat((step(-1), at, step(1), -at, 6 * scales[:, None], 0 * at[:, :2], -0.0 * at[:, :1]), 1)
    x = torch.cat((x, 0 * x[:, :32 - x.shape[1]] if x.shape[1] < 32 else x[:, :0]), 1)[:, :32].contiguous()
    x[:, 28] = 6 * scales                                              # the block's largest: its scale is the one meant
    x = torch.cat((x, x[:1].clone()))
    x[-1, ::2], x[-1, 1::2] = math.inf, -math.inf
    assert torch.equal(x, x.to(dt).float())
    pool = torch.zeros((127, G.kv_fp4_row_bytes(32, 0)), dtype=torch.uint8, device=DEV)
    G.lcs_kv4_store(x.to(dt).to(DEV), torch.arange(127, device=DEV), pool, d_c=32)
    got = pool.cpu()
    want_scale = torch.arange(1, 127, dtype=torch.uint8)
    assert torch.equal(got[:126, 16], want_scale)
    q = (x[:126].double() / scales[:, None].double())
    grid = torch.tensor(LUT, dtype=torch.float64)
    a = q.abs()
    lo = (torch.bucketize(a, grid, right=True) - 1).clamp(0, 7)
    hi = (lo + 1).clamp(max=7)
    mid = (grid[lo] + grid[hi]) / 2
    code = torch.where((a > mid) | ((a == mid) & (lo % 2 == 1)), hi, lo) + 8 * torch.signbit(q).long()
    codes = torch.stack((got[:, :16] & 15, got[:, :16] >> 4), -1).view(127, 32)
    assert torch.equal(codes[:126].long(), code)
    assert codes[126].tolist() == [7, 15] * 16 and got[126, 16] == 126


@gpu
@pytest.mark.parametrize("n", [0, 1, 2, 9, 1000, 20011])
def test_rows_any_count_and_bad_slots(G, n):
    x = torch.randn((n, 576), generator=gen(n), device=DEV)
    pool = torch.full((n + 3, 400), 0x11, dtype=torch.uint8, device=DEV)
    slots = torch.randperm(n + 3, generator=gen(n + 1), device=DEV)[:n].contiguous()
    ws = G.workspace(256)
    G.lcs_kv4_store(x, slots, pool, ws=ws)
    assert G.lcs_status(ws) == 0
    left = torch.ones(n + 3, dtype=torch.bool, device=DEV)
    left[slots] = False
    assert (pool[left] == 0x11).all()
    got = G.lcs_kv4_load(pool, slots, out_dtype=torch.float32, ws=ws)
    assert torch.equal(got.double(), decode_rows(pool[slots], 512, 64))
    if n:
        before = pool.clone()
        bad = slots.clone()
        bad[n // 2] = n + 3
        G.lcs_kv4_store(x * 2, bad, pool, ws=ws)
        assert G.lcs_status(ws) == -5
        assert torch.equal(pool[slots[n // 2]], before[slots[n // 2]])   # the bad slot's row stayed
        got = G.lcs_kv4_load(pool, bad, ws=ws)
        assert G.lcs_status(ws) == -5 and (got[n // 2] == 0).all()


# ------------------------------------------------------------------ attention
def check(o, lse, ref, out_bf16, what):
    want, bound, wl, lb = ref
    step = 2.0 ** -8 if out_bf16 else 2.0 ** -24
    tol = bound + want.abs() * step * (1 + 2.0 ** -7) + bound * step
    err = (o.double() - want).abs()
    assert torch.isfinite(o.float()).all(), what
    worst = (err / tol.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert (err <= tol).all(), f"{what}: error {err.max().item():.3e}, {worst:.2f} of its bound"
    if lse is not None:
        inf = torch.isinf(wl)
        assert torch.equal(torch.isinf(lse), inf) and (lse[inf] < 0).all(), what
        assert ((lse.double() - wl).abs()[~inf] <= lb[~inf]).all(), what


def case(L, op, B, N, be, H, d_c, d_r, dt, Tw=128, k=0, ragged=None, n_win=None, Q=1, q_pos=None, win_pos0=None, m=4, W=128,
         out_dtype=None, heavy=False, seed=0, scale=None, spare=3, ws=None):
    """Runs one call on random data and checks every query against the float64 reference."""
    g = gen(seed)
    D = d_c + d_r
    width = max(1, -(-N // be)) + 1                     # one unused table entry per request
    n_blocks = B * width + spare
    pool = make_pool(L, n_blocks, be, d_c, d_r, seed + 1, heavy)
    perm = torch.randperm(n_blocks, generator=g, device=DEV, dtype=torch.int32)[:B * width].view(B, width).contiguous()
    lens = torch.tensor(ragged if ragged is not None else [N] * B, device=DEV)
    flat = pool.view(n_blocks * be, -1)
    table = perm.clone()
    used = (lens + be - 1) // be
    col = torch.arange(width, device=DEV)[None]
    table[col >= used[:, None]] = 1 << 30               # entries behind the last block are not looked up
    # rows that no query may read hold NaN scales and NaN RoPE dims
    live = torch.zeros(n_blocks * be, dtype=torch.bool, device=DEV)
    for b in range(B):
        j = torch.arange(int(lens[b]), device=DEV)
        live[perm[b, j // be].long() * be + j % be] = True
    flat[~live] = 0xFF
    q = torch.randn((B, Q, H, D), generator=g, device=DEV).to(dt)
    win = torch.randn((B, Tw, D), generator=g, device=DEV).to(dt)
    scale = D ** -0.5 if scale is None else scale
    qp = torch.tensor(q_pos, device=DEV) if q_pos is not None else None
    wp = torch.tensor(win_pos0, device=DEV) if win_pos0 is not None else None
    nw = torch.tensor(n_win, device=DEV) if n_win is not None else None
    seen = lens[:, None].expand(B, Q) if qp is None else torch.minimum(lens[:, None].expand(B, Q), (qp // m + (qp % m == m - 1)).clamp(min=0))
    idx = None
    if op == "csa":
        idx = torch.full((B, Q, k), -1, dtype=torch.int32, device=DEV)
        for b in range(B):
            for t in range(Q):
                n = min(k, int(seen[b, t]))
                pick = torch.randperm(int(seen[b, t]), generator=g, device=DEV)[:n].sort()[0]
                idx[b, t, :n] = pick.int()
    kw = dict(d_c=d_c, n_win=nw, q_pos=qp, win_pos0=wp, W=W, want_lse=True, out_dtype=out_dtype, ws=ws)
    ws = ws if ws is not None else L.workspace(L.lcs_workspace_size(L.OP_ATTEND_KV4, B, Q, width * be, Tw, k, H, d_c))
    kw["ws"] = ws
    if op == "csa":
        o, lse = L.csa_attend_kv4(q, pool, table, lens, win if Tw else None, idx, scale, **kw)
    else:
        o, lse = L.hca_attend_kv4(q, pool, table, lens, win if Tw else None, scale, m=m, **kw)
    assert L.lcs_status(ws) == 0
    assert o.dtype == (out_dtype or dt) and o.shape == (B, Q, H, d_c)
    tc = d_c == 512 and d_r == 64 and dt == torch.bfloat16
    for b in range(B):
        for t in range(Q):
            if op == "csa":
                j = idx[b, t][idx[b, t] >= 0].long()
            else:
                j = torch.arange(int(seen[b, t]), device=DEV)
            rows = decode_rows(flat[perm[b, j // be].long() * be + j % be], d_c, d_r)
            lo, hi = 0, Tw if nw is None else min(max(int(nw[b]), 0), Tw)
            if qp is not None:
                p, p0 = int(qp[b, t]), int(wp[b])
                lo, hi = max(0, p - W + 1 - p0), min(Tw, p - p0 + 1)
            K = torch.cat((rows, win[b, lo:max(lo, hi)].double()))
            check(o[b, t], lse[b, t], attend_ref(q[b, t], K, j.numel(), d_c, scale, tc), o.dtype == torch.bfloat16,
                  f"{op} request {b} query {t}")
    return o, lse


SMALL = [(8, 64, 16, torch.float32), (1, 32, 0, torch.float32), (3, 96, 32, torch.bfloat16), (13, 32, 8, torch.bfloat16),
         (128, 64, 16, torch.float32), (9, 512, 64, torch.float32), (5, 480, 128, torch.bfloat16), (16, 128, 32, torch.float32),
         (8, 256, 64, torch.bfloat16), (17, 160, 0, torch.float32)]


@gpu
@pytest.mark.parametrize("H,d_c,d_r,dt", SMALL)
@pytest.mark.parametrize("op", ["csa", "hca"])
def test_small_shapes(G, op, H, d_c, d_r, dt):
    """The CUDA-core shapes: ragged requests (one empty, one with a window alone), odd pages."""
    case(G, op, 4, 70, 7, H, d_c, d_r, dt, Tw=19, k=33, ragged=[70, 0, 31, 1], n_win=[19, 5, 0, 1], seed=H)
    case(G, op, 2, 40, 1, H, d_c, d_r, dt, Tw=0, k=40, ragged=[0, 40], seed=H + 1, out_dtype=torch.float32)


@gpu
@pytest.mark.parametrize("H,d_c,d_r,dt", SMALL)
def test_small_shapes_over_many_rows(G, H, d_c, d_r, dt):
    """Few queries and long row lists: their rows are split; many queries: they are not."""
    case(G, "hca", 1, 1500, 16, H, d_c, d_r, dt, Tw=100, seed=H)
    case(G, "csa", 3, 900, 16, H, d_c, d_r, dt, Tw=40, k=300, ragged=[900, 17, 280], n_win=[40, 0, 3], seed=H + 1)
    case(G, "hca", 170, 20, 4, H, d_c, d_r, dt, Tw=9, ragged=[b % 21 for b in range(170)], n_win=[b % 10 for b in range(170)], seed=H + 2)


@gpu
@pytest.mark.parametrize("op", ["csa", "hca"])
@pytest.mark.parametrize("H,d_c,d_r,dt", SMALL[:2])
def test_small_causal(G, op, H, d_c, d_r, dt):
    pos = [[-1, 0, 2, 3, 4, 11, 100, 163], [5, 6, 7, 8, 9, 10, 11, 12]]
    case(G, op, 2, 41, 4, H, d_c, d_r, dt, Tw=70, k=20, Q=8, q_pos=pos, win_pos0=[94, -3], m=4, W=33, seed=5)


BF = torch.bfloat16


@gpu
@pytest.mark.parametrize("N", [0, 1, 37, 63, 64, 65, 127, 128, 129, 500, 2100])
@pytest.mark.parametrize("be", [1, 32, 48])
def test_hca_decode_lengths(G, N, be):
    case(G, "hca", 2, N, be, 64, 512, 64, BF, Tw=128, ragged=[N, max(0, N - 5)], seed=N)


@gpu
@pytest.mark.parametrize("H", [1, 15, 16, 40, 63, 65, 128])
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_decode_head_counts(G, H, out_dtype):
    case(G, "hca", 3, 150, 16, H, 512, 64, BF, Tw=128, ragged=[150, 0, 66], n_win=[128, 3, 0], seed=H, out_dtype=out_dtype)
    case(G, "csa", 3, 150, 16, H, 512, 64, BF, Tw=33, k=70, ragged=[150, 0, 66], n_win=[33, 0, 0], seed=H, out_dtype=out_dtype)


@gpu
@pytest.mark.parametrize("Tw,n_win", [(0, None), (1, None), (50, [50, 0]), (64, None), (128, [1, 127]), (200, [200, 65]), (300, None)])
@pytest.mark.parametrize("op", ["csa", "hca"])
def test_decode_windows(G, op, Tw, n_win):
    case(G, op, 2, 90, 8, 64, 512, 64, BF, Tw=Tw, k=64, n_win=n_win, seed=Tw)
    case(G, op, 2, 0, 8, 64, 512, 64, BF, Tw=Tw, k=5, ragged=[0, 0], n_win=n_win, seed=Tw + 1)   # the window alone, or nothing


@gpu
@pytest.mark.parametrize("k", [0, 1, 63, 64, 65, 511, 512, 1024, 4096])
def test_csa_decode_selections(G, k):
    case(G, "csa", 3, 5000, 32, 64, 512, 64, BF, k=k, ragged=[5000, 700, 40], seed=k)


@gpu
@pytest.mark.parametrize("op", ["csa", "hca"])
@pytest.mark.parametrize("B,Q", [(1, 7), (2, 33), (1, 200)])
def test_causal_chunks(G, op, B, Q):
    pos = [[(b + 1) * 150 + t for t in range(Q)] for b in range(B)]
    m = 4 if op == "csa" else 2
    case(G, op, B, (B + 1) * 200 // m + 60, 32, 64, 512, 64, BF, Tw=Q + 90, k=48, Q=Q, q_pos=pos, win_pos0=[(b + 1) * 150 - 90 for b in range(B)],
         m=m, W=128, seed=Q)


@gpu
def test_causal_edges(G):
    """Queries before any entry, windows that end before the chunk, positions past every entry."""
    pos = [[-1, 0, 1, 2, 127, 128, 5000, 1 << 40]]
    case(G, "hca", 1, 30, 4, 64, 512, 64, BF, Tw=140, Q=8, q_pos=pos, win_pos0=[-2], m=4, seed=1)
    case(G, "csa", 1, 30, 4, 64, 512, 64, BF, Tw=140, k=12, Q=8, q_pos=pos, win_pos0=[-2], m=4, seed=2)


@gpu
@pytest.mark.parametrize("op", ["csa", "hca"])
@pytest.mark.parametrize("scale,heavy", [(1.0, True), (-0.3, False), (0.0, False), (2.0 ** -30, True), (4.0, False)])
def test_scores_of_any_size(G, op, scale, heavy):
    """Weights on one row, on all alike, and outliers in the rows."""
    case(G, op, 2, 300, 32, 64, 512, 64, BF, k=200, seed=9, heavy=heavy, scale=scale)


@gpu
@pytest.mark.parametrize("mag", [2.0 ** -100, 2.0 ** -20, 2.0 ** 12, 2.0 ** 100, 0.0])
def test_queries_of_any_size(G, mag):
    """The query's size and the scale cancel: the same attention as with N(0, 1) queries."""
    B, N, H, D = 1, 100, 64, 576
    g = gen(4)
    pool = make_pool(G, 8, 16, 512, 64, 11)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(1, 8)
    n = torch.tensor([N], device=DEV)
    q0 = torch.randn((B, 1, H, D), generator=g, device=DEV).to(BF)
    q0[..., 1::7] *= 2.0 ** -9
    win = torch.randn((B, 20, D), generator=g, device=DEV).to(BF)
    q = (q0.double() * mag).to(BF)
    scale = 1 / 24 if mag in (0.0, 2.0 ** 12, 2.0 ** -20) else 1 / 24 / mag
    o, lse = G.hca_attend_kv4(q, pool, table, n, win, scale, want_lse=True)
    rows = torch.cat((decode_rows(pool.view(128, -1)[:N], 512, 64), win[0].double()))
    check(o[0, 0], lse[0, 0], attend_ref(q[0, 0], rows, N, 512, scale, True), True, f"queries of {mag}")


@gpu
def test_few_rows_long_axis(G):
    """One request over many splits; the largest batch of short ones."""
    case(G, "hca", 1, 8192, 1, 64, 512, 64, BF, seed=1)
    case(G, "hca", 1, 20000, 64, 64, 512, 64, BF, seed=2)
    case(G, "hca", 1, 4500, 64, 128, 512, 64, BF, seed=3)
    case(G, "hca", 5, 3000, 32, 64, 512, 64, BF, ragged=[3000, 0, 1, 1500, 64], n_win=[128, 0, 1, 128, 64], seed=4)
    case(G, "csa", 160, 40, 32, 64, 512, 64, BF, k=16, ragged=[(7 * b) % 41 for b in range(160)], seed=5)


@gpu
@pytest.mark.parametrize("op", ["csa", "hca"])
@pytest.mark.parametrize("d_c,d_r,dt", [(512, 64, BF), (64, 16, torch.float32)])
def test_errors_are_reported(G, op, d_c, d_r, dt):
    B, H, N = 2, 8, 60
    pool = make_pool(G, 8, 16, d_c, d_r, 0)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    n = torch.tensor([N, N], device=DEV)
    q = torch.randn((B, 1, H, d_c + d_r), generator=gen(1), device=DEV).to(dt)
    win = torch.randn((B, 20, d_c + d_r), generator=gen(2), device=DEV).to(dt)
    idx = torch.arange(40, dtype=torch.int32, device=DEV).repeat(B, 1, 1).contiguous()
    ws = G.workspace(G.lcs_workspace_size(G.OP_ATTEND_KV4, B, 1, 64, 20, 40, H, d_c))

    def go(table=table, n=n, idx=idx):
        o = (G.csa_attend_kv4(q, pool, table, n, win, idx, 0.1, d_c=d_c, ws=ws) if op == "csa" else
             G.hca_attend_kv4(q, pool, table, n, win, 0.1, d_c=d_c, ws=ws))
        return o, G.lcs_status(ws)

    good, st = go()
    assert st == 0
    for bad in (-1, 8, 1 << 30, -(1 << 31)):
        t = table.clone()
        t[1, 1] = bad
        o, st = go(table=t)
        assert st == -5 and torch.equal(o[0], good[0])   # the other request's output stands
    o, st = go(n=torch.tensor([N, 65], device=DEV))
    assert st == -5 and torch.equal(o[0], good[0])
    full, st = go(n=torch.tensor([N, 64], device=DEV))
    assert st == 0 and (op == "csa" or torch.equal(full[1], o[1]))
    if op == "csa":
        i = idx.clone()
        i[1, 0, 30:] = N                                   # ends the selection
        o, st = go(idx=i)
        assert st == -5
        i[1, 0, 30:] = -1
        want, st = go(idx=i)
        assert st == 0 and torch.equal(o, want)
        i[1, 0, 35:] = 3                                   # behind the first -1: not read as rows
        o, st = go(idx=i)
        assert st == 0 and torch.equal(o, want)
    o, st = go(n=torch.tensor([N, -4], device=DEV), idx=torch.full_like(idx, -1))
    assert st == 0


@gpu
def test_the_same_entry_twice(G):
    """A selection that repeats an entry gives it two weights, as two rows would."""
    pool = make_pool(G, 2, 32, 512, 64, 5)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    q = torch.randn((1, 1, 64, 576), generator=gen(1), device=DEV).to(BF)
    idx = torch.tensor([[[4, 4, 4, 40]]], dtype=torch.int32, device=DEV)
    o, lse = G.csa_attend_kv4(q, pool, table, torch.tensor([64], device=DEV), None, idx, 0.05, want_lse=True)
    flat = pool.view(64, -1)
    K = decode_rows(flat[torch.tensor([36, 36, 36, 8], device=DEV)], 512, 64)
    check(o[0, 0], lse[0, 0], attend_ref(q[0, 0], K, 4, 512, 0.05, True), True, "repeated entry")


@gpu
def test_batch_invariance_and_determinism(G):
    B, N = 6, 400
    pool = make_pool(G, B * 13, 32, 512, 64, 8)
    table = torch.randperm(B * 13, generator=gen(1), device=DEV, dtype=torch.int32).view(B, 13).contiguous()
    lens = torch.tensor([400, 10, 0, 399, 64, 200], device=DEV)
    q = torch.randn((B, 1, 64, 576), generator=gen(2), device=DEV).to(BF)
    win = torch.randn((B, 128, 576), generator=gen(3), device=DEV).to(BF)
    a = G.hca_attend_kv4(q, pool, table, lens, win, 1 / 24, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(a, G.hca_attend_kv4(q, pool, table, lens, win, 1 / 24, out_dtype=torch.float32))
    p = torch.tensor([3, 1, 5, 0, 2, 4], device=DEV)
    b = G.hca_attend_kv4(q[p].contiguous(), pool, table[p].contiguous(), lens[p], win[p].contiguous(), 1 / 24, out_dtype=torch.float32)
    assert torch.equal(a[p], b)
    # where the rows lie in the pool does not matter
    move = torch.randperm(B * 13, generator=gen(4), device=DEV)
    pool2 = torch.empty_like(pool)
    pool2[move] = pool
    c = G.hca_attend_kv4(q, pool2, move[table.long()].int(), lens, win, 1 / 24, out_dtype=torch.float32)
    assert torch.equal(a, c)


@gpu
def test_offsets_past_32_bits(G):
    """A pool of more than 4 GB: rows near its end."""
    be, n_blocks = 64, 172000                                # 4.4 GB
    pool = torch.zeros((n_blocks, be, 400), dtype=torch.uint8, device=DEV)
    N = 200
    x = torch.randn((N, 576), generator=gen(1), device=DEV)
    table = torch.tensor([[n_blocks - 1, n_blocks - 170, n_blocks - 3, 170000]], dtype=torch.int32, device=DEV)
    e = torch.arange(N, device=DEV)
    slots = table[0, e // be].long() * be + e % be
    G.lcs_kv4_store(x, slots, pool)
    assert torch.equal(G.lcs_kv4_load(pool, slots, out_dtype=torch.float32).double(), decode_rows(pool.view(-1, 400)[slots], 512, 64))
    q = torch.randn((1, 1, 64, 576), generator=gen(2), device=DEV).to(BF)
    o, lse = G.hca_attend_kv4(q, pool, table, torch.tensor([N], device=DEV), None, 1 / 24, want_lse=True)
    check(o[0, 0], lse[0, 0], attend_ref(q[0, 0], decode_rows(pool.view(-1, 400)[slots], 512, 64), N, 512, 1 / 24, True), True, "4.4 GB")
    idx = torch.tensor([[[0, 63, 64, 130, 199]]], dtype=torch.int32, device=DEV)
    o = G.csa_attend_kv4(q, pool, table, torch.tensor([N], device=DEV), None, idx, 1 / 24)
    K = decode_rows(pool.view(-1, 400)[slots[idx[0, 0].long()]], 512, 64)
    check(o[0, 0], None, attend_ref(q[0, 0], K, 5, 512, 1 / 24, True), True, "4.4 GB, selected")


# ------------------------------------------------------------------ together
class Serving:
    """B requests that grow token by token over one pool of blocks of 128 tokens: the plan, the
    compressors, the stores, and CSA and HCA attention, as a serving loop runs them."""

    def __init__(self, L, B, most, seed=0):
        self.L, self.B, g = L, B, gen(seed)
        self.x = torch.randn((B, most, 576), generator=g, device=DEV)
        self.z = torch.randn((B, most), generator=g, device=DEV)
        self.bias_c, self.bias_h = torch.randn(6, generator=g, device=DEV), torch.randn(128, generator=g, device=DEV)
        self.csa = L.csa_compress(self.x, self.z, self.bias_c, d_rope=64)
        self.hca = L.hca_compress(self.x, self.z, self.bias_h, d_rope=64)
        self.win = L.lcs_rope(self.x.clone(), torch.arange(most, device=DEV).repeat(B), 64).to(BF)
        width = most // 128 + 1
        n_blocks = B * width
        self.free = torch.randperm(n_blocks, generator=g, device=DEV, dtype=torch.int32)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.pool_c = torch.full((n_blocks, 32, 400), 0xFF, dtype=torch.uint8, device=DEV)
        self.pool_h = torch.full((n_blocks, 1, 400), 0xFF, dtype=torch.uint8, device=DEV)
        self.ws = L.workspace(L.lcs_workspace_size(L.OP_ATTEND_KV4, B, 1, width * 32, 128, 64))
        self.lens = torch.zeros(B, dtype=torch.int64, device=DEV)

    def append(self, new):
        L, new = self.L, torch.tensor(new, device=DEV)
        n = int(new.clamp(min=0).sum())
        sc, oc, sh, oh, taken = L.lcs_page_plan(self.lens, new, self.free, self.table, m=4, max_slots=n // 4 + self.B, m2=128,
                                                max_slots2=n // 128 + self.B, ws=self.ws)
        self.free = self.free[int(taken):].contiguous()
        for rows, m, slots, off, pool in ((self.csa, 4, sc, oc, self.pool_c), (self.hca, 128, sh, oh, self.pool_h)):
            some = torch.zeros((slots.numel(), 576), device=DEV)
            off = off.tolist()
            for b in range(self.B):
                e0 = int(self.lens[b]) // m
                some[off[b]:off[b + 1]] = rows[b, e0:e0 + off[b + 1] - off[b]]
            L.lcs_kv4_store(some, slots, pool, ws=self.ws)
        self.lens = self.lens + new.clamp(min=0)

    def check(self, what):
        L = self.L
        q = torch.randn((self.B, 1, 64, 576), generator=gen(int(self.lens.sum())), device=DEV).to(BF)
        win = torch.zeros((self.B, 128, 576), dtype=BF, device=DEV)
        lens = self.lens.tolist()
        for b, n in enumerate(lens):
            win[b, :min(n, 128)] = self.win[b, max(0, n - 128):n]
        nw = self.lens.clamp(max=128)
        scores = torch.randn((self.B, 1, max(1, max(lens) // 4)), generator=gen(5), device=DEV)
        pos = (self.lens - 1).view(-1, 1).contiguous()
        idx = L.lcs_topk(scores, 64, q_pos=pos, m=4)
        oc = L.csa_attend_kv4(q, self.pool_c, self.table, self.lens // 4, win, idx, 1 / 24, n_win=nw, ws=self.ws)
        oh = L.hca_attend_kv4(q, self.pool_h, self.table, self.lens // 128, win, 1 / 24, n_win=nw, ws=self.ws)
        assert L.lcs_status(self.ws) == 0
        for b, n in enumerate(lens):
            w = win[b, :min(n, 128)].double()
            for o, rows in ((oc, self.csa[b][idx[b, 0][idx[b, 0] >= 0].long()]), (oh, self.hca[b, :n // 128])):
                flat = torch.zeros((rows.shape[0], 400), dtype=torch.uint8, device=DEV)
                L.lcs_kv4_store(rows.contiguous(), torch.arange(rows.shape[0], device=DEV), flat)
                K = torch.cat((decode_rows(flat, 512, 64), w))
                check(o[b, 0], None, attend_ref(q[b, 0], K, rows.shape[0], 512, 1 / 24, True), True, f"{what}, request {b}")


@gpu
def test_serving_run(G):
    s = Serving(G, 3, 1024)
    s.append([300, 0, 130])          # prompts
    s.check("prompts")
    for _ in range(9):               # decode steps
        s.append([1, 1, 1])
    s.check("decode")
    s.append([0, 500, -1])           # one prompt joins, a request pauses
    s.append([130, 1, 2])
    s.check("joined")


@gpu
def test_other_stream_and_graph(G):
    """The calls on a stream of their own, and captured into a graph that is replayed on changed inputs."""
    B, N, be = 3, 200, 8
    pool = make_pool(G, 80, be, 512, 64, 2)
    table = torch.randperm(80, generator=gen(1), device=DEV, dtype=torch.int32)[:75].view(3, 25).contiguous()
    lens = torch.tensor([200, 77, 0], device=DEV)
    q = torch.randn((B, 1, 64, 576), generator=gen(2), device=DEV).to(BF)
    win = torch.randn((B, 128, 576), generator=gen(3), device=DEV).to(BF)
    x = torch.randn((4, 576), generator=gen(4), device=DEV)
    slots = torch.tensor([3, -1, 500, 9], device=DEV)
    size = G.lcs_workspace_size(G.OP_ATTEND_KV4, B, 1, N, 128, 0)
    ws = G.workspace(size)
    want = G.hca_attend_kv4(q, pool, table, lens, win, 1 / 24, ws=ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        a = G.hca_attend_kv4(q, pool, table, lens, win, 1 / 24, ws=ws)
    b = G.hca_attend_kv4(q, pool, table, lens, win, 1 / 24, ws=G.workspace(size), stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    held, new, free = torch.tensor([0, 5, 9], device=DEV), torch.tensor([300, 1, 4], device=DEV), torch.arange(40, dtype=torch.int32, device=DEV)
    tab = torch.full((3, 4), 7, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    ws2, ws3 = G.workspace(256), G.workspace(size)
    with torch.cuda.graph(graph):
        G.lcs_kv4_store(x, slots, pool, ws=ws2)
        back = G.lcs_kv4_load(pool, slots, ws=ws2)
        plan = G.lcs_page_plan(held, new, free, tab, max_slots=100, m2=128, max_slots2=5, ws=ws2)
        o = G.hca_attend_kv4(q, pool, table, lens, win, 1 / 24, ws=ws3)
    for seed in (7, 8):
        q.copy_(torch.randn(q.shape, generator=gen(seed), device=DEV))
        x.copy_(torch.randn(x.shape, generator=gen(seed), device=DEV))
        lens.copy_(torch.tensor([seed * 20, 3, 199], device=DEV))
        new[0] = seed * 10
        tab.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back, G.lcs_kv4_load(pool, slots)) and (back[1] == 0).all()
        assert torch.equal(o, G.hca_attend_kv4(q, pool, table, lens, win, 1 / 24))
        t2 = torch.full((3, 4), 7, dtype=torch.int32, device=DEV)
        for u, v in zip(plan, G.lcs_page_plan(held, new, free, t2, max_slots=100, m2=128, max_slots2=5)):
            assert torch.equal(u, v)
        assert torch.equal(tab, t2)
    assert G.lcs_status(ws2) == 0 and G.lcs_status(ws3) == 0


@gpu
@pytest.mark.parametrize("d_c,d_r,dt", [(512, 64, BF), (64, 16, torch.float32)])
def test_positions_of_any_size(G, d_c, d_r, dt):
    """Positions up to the type's ends: every entry, no window row; before everything: nothing."""
    top, low = (1 << 63) - 1, -(1 << 63)
    case(G, "hca", 1, 50, 4, 8, d_c, d_r, dt, Tw=30, Q=5, q_pos=[[top, top - 1, 1 << 62, low, -5]], win_pos0=[0], m=3, seed=1)
    case(G, "csa", 1, 50, 4, 8, d_c, d_r, dt, Tw=30, k=20, Q=3, q_pos=[[top, 1 << 62, -5]], win_pos0=[0], m=3, seed=2)


@gpu
def test_window_values_past_fp16(G):
    """Window content of up to 65280 (bf16's last below 2^16) is exact in fp16; from 2^16 on it is an error."""
    pool = make_pool(G, 4, 16, 512, 64, 3)
    table, n = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4), torch.tensor([20], device=DEV)
    q = torch.randn((1, 1, 64, 576), generator=gen(1), device=DEV).to(BF)
    win = torch.randn((1, 60, 576), generator=gen(2), device=DEV).to(BF)
    win[0, 50, 7], win[0, 3, 511], win[0, 9, 530] = 65280.0, -65280.0, 2.0 ** 20    # (RoPE dims stay bf16)
    ws = G.workspace(G.lcs_workspace_size(G.OP_ATTEND_KV4, 1, 1, 64, 60, 0))
    o, lse = G.hca_attend_kv4(q, pool, table, n, win, 1e-5, want_lse=True, ws=ws)
    assert G.lcs_status(ws) == 0
    K = torch.cat((decode_rows(pool.view(64, -1)[:20], 512, 64), win[0].double()))
    check(o[0, 0], lse[0, 0], attend_ref(q[0, 0], K, 20, 512, 1e-5, True), True, "large window values")
    for v in (65536.0, -3e38, math.inf):
        w = win.clone()
        w[0, 59, 0] = v
        G.hca_attend_kv4(q, pool, table, n, w, 1e-5, ws=ws)
        assert G.lcs_status(ws) == -5
        G.hca_attend_kv4(q, pool, table, n, w, 1e-5, n_win=torch.tensor([59], device=DEV), ws=ws)   # not attended
        assert G.lcs_status(ws) == 0


@gpu
def test_selections_made_just_before(G):
    """Top-k and the attention over its selection, step after step on the same buffers without a pause."""
    B, N, k = 8, 3000, 128
    pool = make_pool(G, B * 94, 32, 512, 64, 6)
    table = torch.randperm(B * 94, generator=gen(1), device=DEV, dtype=torch.int32).view(B, 94).contiguous()
    n = torch.full((B,), N, device=DEV)
    q = torch.randn((B, 1, 64, 576), generator=gen(2), device=DEV).to(BF)
    win = torch.randn((B, 128, 576), generator=gen(3), device=DEV).to(BF)
    steps = [torch.randn((B, 1, N), generator=gen(10 + i), device=DEV) for i in range(12)]
    ws = G.workspace(G.lcs_workspace_size(G.OP_ATTEND_KV4, B, 1, 94 * 32, 128, k))
    idx = torch.full((B, 1, k), -1, dtype=torch.int32, device=DEV)
    tws = G.workspace(max(256, G.lcs_workspace_size(G.OP_TOPK, B, 1, N, k=k)))
    pos = torch.full((B, 1), 4 * N - 1, device=DEV)

    def step(s):
        G._call("lcs_topk", s.data_ptr(), G.F32, B, 1, N, pos.data_ptr(), 4, k, idx.data_ptr(), tws.data_ptr(), tws.numel(),
                torch.cuda.current_stream().cuda_stream)
        return G.csa_attend_kv4(q, pool, table, n, win, idx, 1 / 24, ws=ws)

    want = []
    for s in steps:
        want.append(step(s))
        torch.cuda.synchronize()
    got = [step(s) for s in steps]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [step(s) for s in steps]
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, held):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert G.lcs_status(ws) == 0


@gpu
def test_one_workspace_for_calls_in_turn(G):
    """Calls of different sizes and split counts, one after the other on one workspace."""
    pool = make_pool(G, 300, 32, 512, 64, 7)
    mk = lambda B, seed: (torch.randn((B, 1, 64, 576), generator=gen(seed), device=DEV).to(BF),
                          torch.randint(0, 300, (B, 280), generator=gen(seed), device=DEV, dtype=torch.int32),
                          torch.randint(0, 280 * 32, (B,), generator=gen(seed), device=DEV),
                          torch.randn((B, 128, 576), generator=gen(seed), device=DEV).to(BF))
    sets = [mk(B, B) for B in (1, 16, 3, 150, 2, 40)]
    ws = G.workspace(max(G.lcs_workspace_size(G.OP_ATTEND_KV4, B, 1, 280 * 32, 128, 0) for B in (1, 16, 3, 150, 2, 40)))
    alone = [G.hca_attend_kv4(q, pool, t, n, w, 1 / 24, out_dtype=torch.float32) for q, t, n, w in sets]
    torch.cuda.synchronize()
    turn = [G.hca_attend_kv4(q, pool, t, n, w, 1 / 24, out_dtype=torch.float32, ws=ws) for q, t, n, w in sets * 3]
    for i, o in enumerate(turn):
        assert torch.equal(o, alone[i % len(sets)])
    assert G.lcs_status(ws) == 0


@gpu
def test_two_graphs_at_once(G):
    """Two captured decode steps with a workspace each, replayed on two streams at the same time."""
    pool = make_pool(G, 200, 32, 512, 64, 9)
    steps = []
    for i, B in enumerate((4, 9)):
        q = torch.randn((B, 1, 64, 576), generator=gen(20 + i), device=DEV).to(BF)
        table = torch.randint(0, 200, (B, 60), generator=gen(30 + i), device=DEV, dtype=torch.int32)
        n = torch.randint(0, 60 * 32, (B,), generator=gen(40 + i), device=DEV)
        want = G.hca_attend_kv4(q, pool, table, n, None, 1 / 24)
        ws = G.workspace(G.lcs_workspace_size(G.OP_ATTEND_KV4, B, 1, 60 * 32, 0, 0))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [G.hca_attend_kv4(q, pool, table, n, None, 1 / 24, ws=ws) for _ in range(20)]
        steps.append((graph, outs, want, torch.cuda.Stream(), ws, (q, table, n)))   # (a graph keeps no inputs alive)
    for _ in range(3):
        for graph, _, _, st, _, _ in steps:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, outs, want, _, ws, _ in steps:
        assert all(torch.equal(o, want) for o in outs) and G.lcs_status(ws) == 0


@gpu
def test_stream_argument_without_a_workspace(G):
    """What the call allocates belongs to the given stream: work on the current one does not touch it."""
    pool = make_pool(G, 64, 32, 512, 64, 8)
    table, n = torch.arange(64, dtype=torch.int32, device=DEV).view(1, 64), torch.tensor([2000], device=DEV)
    q = torch.randn((1, 1, 64, 576), generator=gen(2), device=DEV).to(BF)
    x, slots = torch.randn((40, 576), generator=gen(3), device=DEV), torch.arange(40, device=DEV)
    want, rows = G.hca_attend_kv4(q, pool, table, n, None, 1 / 24), G.lcs_kv4_load(pool, slots)
    big = torch.randn((4096, 4096), device=DEV)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        big @ big                                   # the current stream is busy when the calls are made
        a, b = G.hca_attend_kv4(q, pool, table, n, None, 1 / 24, stream=st), G.lcs_kv4_load(pool, slots, stream=st)
        st.synchronize()
        assert torch.equal(a, want) and torch.equal(b, rows)
    own = torch.zeros((64, 400), dtype=torch.uint8, device=DEV)
    tab = torch.full((1, 4), -1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    G.lcs_kv4_store(x, slots, own, stream=st)
    plan = G.lcs_page_plan(torch.tensor([0], device=DEV), torch.tensor([300], device=DEV), torch.tensor([5, 2, 9], dtype=torch.int32, device=DEV),
                           tab, max_slots=75, stream=None)
    st.synchronize()
    assert torch.equal(G.lcs_kv4_load(own, slots, out_dtype=torch.float32).double(), decode_rows(own[:40], 512, 64))
    assert tab.tolist() == [[5, 2, 9, -1]] and plan[4].item() == 3


@gpu
def test_nothing_to_do(G):
    """No requests, no queries, no rows, no blocks: empty results, and no row seen gives zeros."""
    z = lambda *s, dt=torch.int64: torch.zeros(s, dtype=dt, device=DEV)
    i32, u8 = torch.int32, torch.uint8
    pool = make_pool(G, 4, 16, 512, 64, 3)
    for H, dc, dr, dt in ((64, 512, 64, BF), (3, 64, 8, torch.float32)):
        p = pool if dc == 512 else make_pool(G, 4, 16, dc, dr, 4)
        o = G.hca_attend_kv4(z(0, 1, H, dc + dr, dt=dt), p, z(0, 3, dt=i32), z(0), None, 0.1, d_c=dc)
        assert o.shape == (0, 1, H, dc)
        o = G.csa_attend_kv4(z(2, 0, H, dc + dr, dt=dt), p, z(2, 3, dt=i32), z(2), None, z(2, 0, 5, dt=i32), 0.1, d_c=dc, q_pos=z(2, 0), win_pos0=z(2))
        assert o.shape == (2, 0, H, dc)
        q = torch.ones((2, 1, H, dc + dr), device=DEV).to(dt)
        for table, win in ((z(2, 0, dt=i32), None), (z(2, 3, dt=i32), torch.ones((2, 4, dc + dr), device=DEV).to(dt))):
            o, lse = G.hca_attend_kv4(q, p, table, z(2), win, 0.1, d_c=dc, n_win=z(2), want_lse=True)
            assert (o == 0).all() and (lse == -math.inf).all()
            o, lse = G.csa_attend_kv4(q, p, table, z(2), win, z(2, 1, 0, dt=i32), 0.1, d_c=dc, n_win=z(2), want_lse=True)
            assert (o == 0).all() and (lse == -math.inf).all()
    G.lcs_kv4_store(z(0, 576, dt=BF), z(0), pool)
    assert G.lcs_kv4_load(pool, z(0)).shape == (0, 576)
    ws = G.workspace(256)
    none = z(0, 16, 400, dt=u8)
    G.lcs_kv4_store(torch.ones((2, 576), device=DEV), torch.tensor([-1, -1], device=DEV), none, ws=ws)
    assert (G.lcs_kv4_load(none, torch.tensor([-1], device=DEV), ws=ws) == 0).all() and G.lcs_status(ws) == 0


@gpu
def test_views_that_do_not_fit_are_refused(G):
    pool = make_pool(G, 4, 16, 512, 64, 3)
    table, n = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4), torch.tensor([20], device=DEV)
    q = torch.randn((1, 1, 64, 576), device=DEV).to(BF)
    with pytest.raises(ValueError):
        G.hca_attend_kv4(q.transpose(2, 3).contiguous().transpose(2, 3), pool, table, n, None, 0.1)
    with pytest.raises(ValueError):
        G.hca_attend_kv4(q, pool[:, ::2], table, n, None, 0.1)
    with pytest.raises(ValueError):
        G.hca_attend_kv4(q, pool, table.view(4, 1).expand(4, 2)[:1], n.float(), None, 0.1)
    with pytest.raises(ValueError):
        G.lcs_kv4_store(torch.randn((4, 600), device=DEV)[:, :576], torch.arange(4, device=DEV), pool)
    off = torch.empty(64 * 576 + 4, dtype=BF, device=DEV)[4:].view(1, 1, 64, 576)     # 8 bytes off
    with pytest.raises(G.LcsError):
        G.hca_attend_kv4(off, pool, table, n, None, 0.1)
    with pytest.raises(G.LcsError):
        G.hca_attend_kv4(q, pool, table, n, None, 0.1, ws=G.workspace(512)[8:264])
    with pytest.raises(G.LcsError):
        G.hca_attend_kv4(q.half().to(BF), pool, table, n, None, 0.1, q_pos=torch.tensor([[4]], device=DEV))   # win_pos0 missing


@gpu
def test_first_call_inside_a_capture(G):
    """A process whose first calls are captured ones."""
    import subprocess
    import sys
    code = """
import torch, long_context_sparse_06_b200 as L
L.lib()
g = torch.Generator('cuda').manual_seed(1)
pool = torch.zeros((64, 32, 400), dtype=torch.uint8, device='cuda')
x = torch.randn((2048, 576), generator=g, device='cuda')
slots = torch.arange(2048, device='cuda')
table = torch.arange(64, dtype=torch.int32, device='cuda').view(1, 64)
n = torch.tensor([2000], device='cuda')
q = torch.randn((1, 1, 64, 576), generator=g, device='cuda').bfloat16()
short, m = table[:, :10].contiguous(), torch.tensor([300], device='cuda')
idx = torch.arange(0, 1500, 5, dtype=torch.int32, device='cuda').view(1, 1, 300)
ws = L.workspace(max(L.lcs_workspace_size(L.OP_ATTEND_KV4, 1, 1, N, 0, k) for N, k in ((2048, 0), (320, 0), (2048, 300))))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    L.lcs_kv4_store(x, slots, pool, ws=ws)
    o = L.hca_attend_kv4(q, pool, table, n, None, 1 / 24, ws=ws)
    p = L.hca_attend_kv4(q.float(), pool, table, n, None, 1 / 24, ws=ws)
    few = L.hca_attend_kv4(q, pool, short, m, None, 1 / 24, ws=ws)      # seven splits, one cluster
    sel = L.csa_attend_kv4(q, pool, table, n, None, idx, 1 / 24, ws=ws)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(o, L.hca_attend_kv4(q, pool, table, n, None, 1 / 24))
assert torch.equal(few, L.hca_attend_kv4(q, pool, short, m, None, 1 / 24))
assert torch.equal(sel, L.csa_attend_kv4(q, pool, table, n, None, idx, 1 / 24))
assert (o.float() - p).abs().max() < 0.05 and p.abs().max() > 0.01
assert L.lcs_status(ws) == 0
print('captured')
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert "captured" in r.stdout, r.stdout + r.stderr


@gpu
def test_on_another_device(G):
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two devices")
    dev = torch.device("cuda", 1)
    x = torch.randn((4, 576), device=dev)
    pool = torch.zeros((2, 4, 400), dtype=torch.uint8, device=dev)
    G.lcs_kv4_store(x, torch.arange(4, device=dev), pool)
    o = G.hca_attend_kv4(x.to(BF)[:1].repeat(64, 1).view(1, 1, 64, 576), pool, torch.zeros((1, 1), dtype=torch.int32, device=dev),
                         torch.tensor([4], device=dev), None, 0.1)
    assert torch.isfinite(o.float()).all()
