"""Measured cases of the paged 4-bit KV cache operators.

A serving step of the compressed-attention path over a paged cache runs them in this order:

* ``page_plan``  -- from the requests' lengths and their new tokens: the block tables extended
  from a list of free blocks, and the slot of every compressed entry that the new tokens
  complete (CSA entries, one per m = 4 tokens; HCA entries, one per 128);
* ``rows``       -- compressed rows quantised to 4 bits (E2M1 codes, an E4M3 scale per 32 content
  dims, RoPE dims in bf16) and stored at their slots, and rows read back from slots;
* ``hca``        -- dense shared-KV attention over a request's paged entries and its window;
* ``csa``        -- the same over the entries that the indexer selected.

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits; with ``own``
true it calls the library.
"""
import torch

own = False

BLOCK_TOKENS = 128   # raw tokens of one cache block: 32 CSA entries, one HCA entry
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # block tables and slots of one decode step: each of 32 requests gets one token
        dict(name="plan_decode_32", op="page_plan", B=32, held=131072, new=1, ragged=True),
        # block tables and slots of a batch of 64 prompts, the longest 131072 tokens
        dict(name="plan_prompts_64", op="page_plan", B=64, held=0, new=131072, ragged=True),
        # the entries that one decode step of 32 requests completes, from fp32 rows
        dict(name="rows_decode_32", op="rows", n=32, d_c=512, d_r=64, bf16=False, skip=4, heavy=False),
        # the CSA entries of one million-token prompt, bf16 rows
        dict(name="rows_prompt_1m", op="rows", n=262144, d_c=512, d_r=64, bf16=True, skip=0, heavy=True),
        # HCA decode of one short request: 37 entries (4.7K tokens), latency
        dict(name="hca_decode_1_short", op="hca", B=1, Q=1, N=37, H=64, d_c=512, d_r=64, be=1, bf16=True, Tw=128,
             W=128, m=128, causal=False, ragged=False, heavy=False, lse=False),
        # HCA decode of one million-token request: few rows of queries, a long axis
        dict(name="hca_decode_1_1m", op="hca", B=1, Q=1, N=8192, H=64, d_c=512, d_r=64, be=1, bf16=True, Tw=128,
             W=128, m=128, causal=False, ragged=False, heavy=False, lse=True),
        # HCA decode, 16 requests of a million tokens each
        dict(name="hca_decode_16_1m", op="hca", B=16, Q=1, N=8192, H=64, d_c=512, d_r=64, be=32, bf16=True, Tw=128,
             W=128, m=128, causal=False, ragged=False, heavy=False, lse=False),
        # HCA prefill of a chunk of 1000 queries after a 128K prefix, causal over the entries
        dict(name="hca_prefill_1000", op="hca", B=1, Q=1000, N=1031, H=64, d_c=512, d_r=64, be=1, bf16=True, Tw=1127,
             W=128, m=128, causal=True, ragged=False, heavy=False, lse=False),
        # CSA decode: 32 requests of 128K tokens, top-512 of 32768 entries
        dict(name="csa_decode_32_128k", op="csa", B=32, Q=1, N=32768, k=512, H=64, d_c=512, d_r=64, be=32, bf16=True,
             Tw=128, W=128, m=4, causal=False, ragged=False, heavy=False, lse=False),
        # CSA decode: 4 requests of a million tokens, top-1024 of 262144 entries, outliers in the rows
        dict(name="csa_decode_4_1m", op="csa", B=4, Q=1, N=262144, k=1024, H=64, d_c=512, d_r=64, be=32, bf16=True,
             Tw=128, W=128, m=4, causal=False, ragged=False, heavy=True, lse=True),
        # CSA prefill of a chunk of 1500 queries after a 128K prefix, top-1024
        dict(name="csa_prefill_1500", op="csa", B=1, Q=1500, N=33143, k=1024, H=64, d_c=512, d_r=64, be=32, bf16=True,
             Tw=1627, W=128, m=4, causal=True, ragged=False, heavy=False, lse=False),
        # the tiny fp32 configuration: 8 heads, top-64 of 256 entries, 1024 causal queries
        dict(name="csa_small_f32", op="csa", B=1, Q=1024, N=256, k=64, H=8, d_c=64, d_r=16, be=32, bf16=False, Tw=1024,
             W=128, m=4, causal=True, ragged=False, heavy=False, lse=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(("plan", "rows", "hca_decode", "hca_decode", "hca_prefill", "csa_decode", "csa_decode",
                       "csa_prefill", "small"))
    if kind == "plan":
        B = _log(rng, 1, 512)
        if rng.random() < 0.5:
            return dict(op="page_plan", B=B, held=_log(rng, 100, 200000), new=_log(rng, 1, 9), ragged=True)
        return dict(op="page_plan", B=B, held=rng.choice((0, _log(rng, 1, 5000))), new=_log(rng, 50, 4000000 // B),
                    ragged=rng.random() < 0.8)
    if kind == "rows":
        n = _log(rng, 1, 250000)
        return dict(op="rows", n=n, d_c=512, d_r=64, bf16=rng.random() < 0.7, skip=rng.choice((0, 2, 7)),
                    heavy=rng.random() < 0.5)
    c = dict(op="hca", B=1, Q=1, N=1, H=64, d_c=512, d_r=64, be=rng.choice((1, 1, 2, 16, 32, 48, 64)), bf16=True,
             Tw=128, W=128, m=128, causal=False, ragged=rng.random() < 0.5, heavy=rng.random() < 0.3,
             lse=rng.random() < 0.5)
    if kind == "hca_decode":
        c["B"] = _log(rng, 1, 48)
        c["N"] = _log(rng, 1, min(16000, 120000 // c["B"]))
        c["Tw"] = rng.choice((128, 128, 1, 50, 100))
        c["H"] = rng.choice((64, 64, 64, 16, 40, 128)) if c["N"] * c["B"] < 40000 else 64
    elif kind == "hca_prefill":
        c.update(causal=True, ragged=False, B=rng.choice((1, 1, 2, 3)))
        c["Q"] = _log(rng, 2, 900 // c["B"])
        c["N"] = _log(rng, 10, 1000)
        c["Tw"] = c["Q"] + rng.choice((127, 127, 60, 0))
    elif kind == "csa_decode":
        c.update(op="csa", m=4, be=rng.choice((32, 32, 8, 24, 64)), B=_log(rng, 1, 64))
        c["N"] = _log(rng, 20, min(262144, 2000000 // c["B"]))
        c["k"] = _log(rng, 1, 1024)
        c["Tw"] = rng.choice((128, 128, 1, 77))
        c["H"] = rng.choice((64, 64, 64, 8, 128))
    elif kind == "csa_prefill":
        c.update(op="csa", m=4, causal=True, ragged=False, be=rng.choice((32, 32, 8, 64)), B=rng.choice((1, 1, 2)))
        c["Q"] = _log(rng, 2, 1200 // c["B"])
        c["N"] = _log(rng, 100, 33000)
        c["k"] = _log(rng, 16, 1024)
        c["Tw"] = c["Q"] + rng.choice((127, 127, 31))
    else:
        c.update(op=rng.choice(("csa", "hca")), bf16=rng.random() < 0.3, H=rng.choice((1, 4, 8, 13)),
                 d_c=rng.choice((32, 64, 96)), d_r=rng.choice((16, 32)), m=4, heavy=False, be=rng.choice((1, 8, 32)),
                 B=rng.choice((1, 2, 3)))
        c["N"] = _log(rng, 5, 300)
        if rng.random() < 0.5:
            c.update(causal=True, ragged=False)
            c["Q"] = _log(rng, 2, 600)
            c["Tw"] = c["Q"] + 127
        if c["op"] == "csa":
            c["k"] = _log(rng, 1, 96)
    return c


def _spread(B, most, ragged):
    """Lengths of B requests: all `most`, or between 0 and `most`, one of them `most`."""
    if not ragged:
        return [most] * B
    return [most - (most * ((b * 5) % B)) // B for b in range(B)]


# --------------------------------------------------------------------------- the row format
def _row_bytes(d_c, d_r):
    return (d_c // 2 + 2 * d_r + d_c // 32 + 15) // 16 * 16


def _quantise(x, d_c, d_r):
    """Rows [n, d_c + d_r] -> codes [n, d_c] (0..15) and scales [n, d_c / 32] (E4M3).  Per block of 32
    content dims: scale = E4M3(amax / 6), 1 where that is 0; code = E2M1(x / scale), ties to even."""
    n = x.shape[0]
    c = x[:, :d_c].float().view(n, d_c // 32, 32)
    s = (c.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = torch.where(s.float() == 0, torch.ones_like(s.float()), s.float()).to(torch.float8_e4m3fn)
    v = c / s.float()[:, :, None]
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + (v < 0).to(torch.uint8) * 8
    return code.view(n, d_c), s


def _values(code, s, d_c):
    """The values of codes [..., d_c] with scales [..., d_c / 32]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    return lut[code.int()] * s.float().repeat_interleave(32, -1)


def _pack(x, d_c, d_r):
    """Rows as stored: packed codes (element 2j in the low nibble of byte j), RoPE dims in bf16, scales."""
    code, s = _quantise(x, d_c, d_r)
    row = torch.zeros((x.shape[0], _row_bytes(d_c, d_r)), dtype=torch.uint8, device=x.device)
    row[:, :d_c // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    if d_r:
        row[:, d_c // 2:d_c // 2 + 2 * d_r] = x[:, d_c:].to(torch.bfloat16).contiguous().view(torch.uint8)
    row[:, d_c // 2 + 2 * d_r:d_c // 2 + 2 * d_r + d_c // 32] = s.view(torch.uint8)
    return row


def _unpack(row, d_c, d_r):
    """Stored rows [..., bytes] -> fp32 rows [..., d_c + d_r]."""
    packed = row[..., :d_c // 2]
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    s = row[..., d_c // 2 + 2 * d_r:d_c // 2 + 2 * d_r + d_c // 32].contiguous().view(torch.float8_e4m3fn)
    r = row[..., d_c // 2:d_c // 2 + 2 * d_r].contiguous().view(torch.bfloat16).float()
    return torch.cat((_values(code, s, d_c), r), -1)


# ------------------------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rows(g, n, d, heavy):
    """N(0, 1) rows; heavy: one element in a hundred is 20 times as large."""
    x = _normal(g, n, d)
    if heavy:
        x = torch.where(torch.rand((n, d), generator=g, device="cuda") < 0.01, x * 20, x)
    return x


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    c, s = case, {"case": case, "ws": {}}
    if c["op"] == "page_plan":
        B = c["B"]
        held = torch.tensor(_spread(B, c["held"], c["ragged"]), device="cuda")
        if c["new"] < 16:   # a decode step: requests at any phase of their block
            held = held + torch.randint(0, 256, (B,), generator=g, device="cuda")
            new = torch.full((B,), c["new"], device="cuda")
        else:
            new = torch.tensor(_spread(B, c["new"], c["ragged"]), device="cuda")
        width = (c["held"] + 256 + c["new"]) // BLOCK_TOKENS + 2
        need = int(((held + new + BLOCK_TOKENS - 1) // BLOCK_TOKENS).sum())
        ids = torch.randperm(need + 64, generator=g, device="cuda", dtype=torch.int32)
        col = torch.arange(width, device="cuda")
        nb = (held + BLOCK_TOKENS - 1) // BLOCK_TOKENS
        used = int(nb.sum())
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        table[col[None] < nb[:, None]] = ids[:used]
        s.update(held=held, new=new, free=ids[used:].contiguous(), table=table,
                 most_csa=sum(_spread(B, c["new"], c["ragged"])) // 4 + B,
                 most_hca=sum(_spread(B, c["new"], c["ragged"])) // 128 + B)
        return s
    d_c, d_r = c["d_c"], c["d_r"]
    D = d_c + d_r
    if c["op"] == "rows":
        n = c["n"]
        blocks = (n + 31) // 32 + 3
        x = _rows(g, n, D, c["heavy"])
        slots = torch.randperm(blocks * 32, generator=g, device="cuda")[:n].contiguous()
        if c["skip"]:   # rows of requests that completed no entry
            slots[::c["skip"]] = -1
        s.update(x=x.to(torch.bfloat16) if c["bf16"] else x, slots=slots,
                 pool=torch.zeros((blocks, 32, _row_bytes(d_c, d_r)), dtype=torch.uint8, device="cuda"))
        return s
    B, Q, N, H, be = c["B"], c["Q"], c["N"], c["H"], c["be"]
    dt = torch.bfloat16 if c["bf16"] else torch.float32
    width = (N + be - 1) // be
    n_blocks = B * width + 5
    table = torch.randperm(n_blocks, generator=g, device="cuda", dtype=torch.int32)[:B * width].view(B, width)
    lens = torch.tensor(_spread(B, N, c["ragged"]), device="cuda")
    pool = torch.zeros((n_blocks * be, _row_bytes(d_c, d_r)), dtype=torch.uint8, device="cuda")
    for at in range(0, n_blocks * be, 1 << 18):   # a quarter of a million rows at a time
        some = min(1 << 18, n_blocks * be - at)
        pool[at:at + some] = _pack(_rows(g, some, D, c["heavy"]), d_c, d_r)
    s.update(pool=pool.view(n_blocks, be, -1), table=table.contiguous(), lens=lens,
             q=_normal(g, B, Q, H, D).to(dt), win=_rows(g, B * c["Tw"], D, c["heavy"]).to(dt).view(B, c["Tw"], D),
             scale=D ** -0.5, n_win=None, q_pos=None, win_pos0=None)
    if c["causal"]:   # the chunk's last query sees every entry
        first = N * c["m"] - Q
        s["q_pos"] = (first + torch.arange(Q, device="cuda"))[None].repeat(B, 1).contiguous()
        s["win_pos0"] = torch.full((B,), first - (c["Tw"] - Q), device="cuda")
    elif c["ragged"]:
        s["n_win"] = torch.clamp(lens * c["m"], max=c["Tw"])
    if c["op"] == "csa":   # ascending entries without repeats, among those that the query may see; then -1
        k = c["k"]
        seen = lens[:, None].expand(B, Q) if s["q_pos"] is None else torch.clamp((s["q_pos"] + 1) // c["m"], min=0)
        step = torch.clamp((seen[..., None] - torch.rand((B, Q, 1), generator=g, device="cuda")) / k, min=1.0)
        at = (torch.arange(k, device="cuda") * step.double()).floor().long()
        s["idx"] = torch.where(at < seen[..., None], at, -1).int()
    return s


# ------------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    if op == "page_plan":
        return _plan(state)
    if op == "rows":
        c = state["case"]
        code, s = _quantise(state["x"], c["d_c"], c["d_r"])
        v = torch.cat((_values(code, s, c["d_c"]), state["x"][:, c["d_c"]:].to(torch.bfloat16).float()), -1)
        return torch.where(state["slots"][:, None] >= 0, v, 0.0).to(torch.bfloat16)
    return _attend(state)


def _workspace(state, lib, *args, **kw):
    if "ws" not in state["ws"]:
        state["ws"]["ws"] = lib.workspace(lib.lcs_workspace_size(*args, **kw) if args else 256)
    return state["ws"]["ws"]


def _own(state):
    import long_context_sparse_06_b200 as lcs
    c, s = state["case"], state
    if c["op"] == "page_plan":
        csa, csa_off, hca, hca_off, taken = lcs.lcs_page_plan(
            s["held"], s["new"], s["free"], s["table"], block_tokens=BLOCK_TOKENS, m=4, max_slots=s["most_csa"], m2=128,
            max_slots2=s["most_hca"], ws=_workspace(s, lcs))
        return s["table"], csa, csa_off, hca, hca_off, taken
    d_c, d_r = c["d_c"], c["d_r"]
    if c["op"] == "rows":
        ws = _workspace(s, lcs)
        lcs.lcs_kv4_store(s["x"], s["slots"], s["pool"], d_c=d_c, ws=ws)
        return lcs.lcs_kv4_load(s["pool"], s["slots"], d_c=d_c, d_r=d_r, out_dtype=torch.bfloat16, ws=ws)
    ws = _workspace(s, lcs, lcs.OP_ATTEND_KV4, c["B"], c["Q"], s["table"].shape[1] * c["be"], c["Tw"], c.get("k", 0),
                    c["H"], d_c)
    kw = dict(d_c=d_c, n_win=s["n_win"], q_pos=s["q_pos"], win_pos0=s["win_pos0"], W=c["W"], want_lse=c["lse"], ws=ws)
    if c["op"] == "csa":
        return lcs.csa_attend_kv4(s["q"], s["pool"], s["table"], s["lens"], s["win"], s["idx"], s["scale"], **kw)
    return lcs.hca_attend_kv4(s["q"], s["pool"], s["table"], s["lens"], s["win"], s["scale"], m=c["m"], **kw)


def _plan(s):
    """Request b holds ceil(held / 128) blocks and needs ceil((held + new) / 128): the missing ones come
    from the free list, request by request.  Entry j of m tokens is complete once (j + 1) m tokens are
    there; its slot is block_table[b, j m / 128] * (128 / m) + j mod (128 / m)."""
    held, new, free, table = s["held"], s["new"], s["free"], s["table"]
    b0 = (held + BLOCK_TOKENS - 1) // BLOCK_TOKENS
    b1 = (held + new + BLOCK_TOKENS - 1) // BLOCK_TOKENS
    start = torch.cumsum(b1 - b0, 0) - (b1 - b0)
    col = torch.arange(table.shape[1], device=table.device)[None]
    at = torch.clamp(start[:, None] + col - b0[:, None], 0, max(0, free.numel() - 1))
    table = torch.where((col >= b0[:, None]) & (col < b1[:, None]), free[at], table)

    def slots(m, most):
        e0, e1 = held // m, (held + new) // m
        ends = torch.cumsum(e1 - e0, 0)
        i = torch.arange(most, device=table.device)
        b = torch.clamp(torch.searchsorted(ends, i, right=True), max=held.numel() - 1)
        j = e0[b] + i - (ends - (e1 - e0))[b]
        per = BLOCK_TOKENS // m
        blk = torch.clamp(j // per, 0, table.shape[1] - 1)
        slot = table[b, blk].long() * per + j % per
        return torch.where(i < ends[-1], slot, -1), torch.cat((ends.new_zeros(1), ends))

    csa, csa_off = slots(4, s["most_csa"])
    hca, hca_off = slots(128, s["most_hca"])
    return table, csa, csa_off, hca, hca_off, (b1 - b0).sum().view(1)


def _attend(s):
    """softmax over the entries and the window rows that a query sees, scale * q . K, and the sum of
    V = the first d_c dims of K; a query that sees nothing gives 0 and a log-sum of -inf."""
    c, table, be = s["case"], s["table"], s["case"]["be"]
    d_c, d_r = c["d_c"], c["d_r"]
    B, Q, H, D = s["q"].shape
    dev = table.device
    flat = s["pool"].view(-1, s["pool"].shape[-1])
    q = s["q"].float()
    if c["op"] == "csa":
        idx = s["idx"].long()
        at = torch.clamp(idx, min=0)
        blk = torch.gather(table, 1, (at // be).view(B, -1)).view(at.shape).long()
        rows = _unpack(flat[blk * be + at % be], d_c, d_r)                    # [B, Q, k, D]
        sc = torch.einsum("bqhd,bqkd->bqhk", q, rows)
        sees = (idx >= 0)[:, :, None]
    else:
        j = torch.arange(table.shape[1] * be, device=dev)
        rows = _unpack(flat[table[:, j // be].long() * be + j % be], d_c, d_r)   # [B, N, D]
        sc = torch.einsum("bqhd,bkd->bqhk", q, rows)
        some = s["lens"][:, None].expand(B, Q)
        if s["q_pos"] is not None:
            some = torch.minimum(some, torch.clamp((s["q_pos"] + 1) // c["m"], min=0))
        sees = (j < some[..., None])[:, :, None]
    win = s["win"].float()
    r = torch.arange(c["Tw"], device=dev)
    if s["q_pos"] is not None:
        at = s["win_pos0"][:, None, None] + r
        there = (at <= s["q_pos"][..., None]) & (at > s["q_pos"][..., None] - c["W"])
    elif s["n_win"] is not None:
        there = (r < s["n_win"][:, None])[:, None]
    else:
        there = torch.ones((B, 1, c["Tw"]), dtype=torch.bool, device=dev)
    sw = torch.einsum("bqhd,brd->bqhr", q, win)
    low = torch.tensor(float("-inf"), device=dev)
    sc = torch.where(sees, sc * s["scale"], low)
    sw = torch.where(there[:, :, None], sw * s["scale"], low)
    most = torch.maximum(sc.amax(-1), sw.amax(-1))
    m = torch.where(most == low, 0.0, most)[..., None]
    pc, pw = torch.exp(sc - m), torch.exp(sw - m)
    total = pc.sum(-1) + pw.sum(-1)
    o = torch.einsum("bqhk,bqkd->bqhd" if c["op"] == "csa" else "bqhk,bkd->bqhd", pc, rows[..., :d_c])
    o = (o + torch.einsum("bqhr,brd->bqhd", pw, win[..., :d_c])) / torch.where(total == 0, 1.0, total)[..., None]
    o = o.to(s["q"].dtype)
    return (o, torch.where(total == 0, low, m[..., 0] + torch.log(total))) if c["lse"] else o


# ------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "page_plan":
        new = _spread(c["B"], c["new"], c["ragged"]) if c["new"] >= 16 else [c["new"]] * c["B"]
        entries = sum(n // 4 + n // 128 for n in new)
        blocks = sum(n // BLOCK_TOKENS for n in new)
        return {"bytes": 16 * c["B"] + 8 * entries + 8 * blocks + 16 * c["B"], "flops": 0}
    d_c, d_r = c["d_c"], c["d_r"]
    D, row = d_c + d_r, _row_bytes(d_c, d_r)
    if c["op"] == "rows":
        n = c["n"] - (-(-c["n"] // c["skip"]) if c["skip"] else 0)
        return {"bytes": n * (D * (2 if c["bf16"] else 4) + 2 * row) + c["n"] * (16 + 2 * D), "flops": 3 * n * d_c}
    e = 2 if c["bf16"] else 4
    B, Q, H = c["B"], c["Q"], c["H"]
    lens = _spread(B, c["N"], c["ragged"])
    wins = [min(c["Tw"], n * c["m"]) if c["ragged"] else c["Tw"] for n in lens]
    if c["causal"]:
        first = c["N"] * c["m"] - Q
        ends = [max(0, (first + t + 1) // c["m"]) for t in range(Q)]
        per = [min(n, c["k"]) if c["op"] == "csa" else min(n, c["N"]) for n in ends]
        pos0 = first - (c["Tw"] - Q)
        seen = [min(c["W"], first + t - pos0 + 1) for t in range(Q)]
        pairs = B * (sum(per) + sum(seen))
        entries = B * (min(sum(per), c["N"]) if c["op"] == "csa" else max(per))
        window = B * c["Tw"]
    else:
        entries = sum(min(n, c["k"]) for n in lens) if c["op"] == "csa" else sum(lens)
        window = sum(wins)
        pairs = entries + window
    more = 4 * B * Q * c["k"] if c["op"] == "csa" else 0
    return {"bytes": entries * row + window * D * e + B * Q * H * (D + d_c) * e + more,
            "flops": 2 * pairs * H * (D + d_c)}


# ------------------------------------------------------------------------------- in 64 bits
def _round(v, mantissa, low, top):
    """v (float64) to the nearest value of `mantissa` bits after the point, exponents from `low`, at most `top`."""
    e = torch.clamp(torch.frexp(v)[1] - 1, min=low)
    step = torch.ldexp(torch.ones_like(v), e - mantissa)
    return torch.clamp(torch.round(v / step) * step, -top, top)


def _as_stored(x, d_c):
    """The values that rows x (float64) have once they are stored."""
    out = torch.empty_like(x)
    for at in range(0, d_c, 32):
        part = x[:, at:at + 32]
        scale = _round(part.abs().amax(1, keepdim=True) / 6, 3, -6, 448.0)
        scale[scale == 0] = 1
        out[:, at:at + 32] = _round(part / scale, 1, 0, 6.0) * scale
    out[:, d_c:] = x[:, d_c:].to(torch.bfloat16).double()
    return out


def _stored_values(row, d_c, d_r):
    """The float64 values of stored rows [n, bytes]."""
    n = row.shape[0]
    out = torch.empty((n, d_c + d_r), dtype=torch.float64, device=row.device)
    byte = row[:, :d_c // 2].int()
    for half, code in enumerate((byte % 16, byte // 16)):
        e, f = (code % 8) // 2, (code % 2).double()
        mag = torch.where(e == 0, f / 2, (1 + f / 2) * torch.pow(2.0, (e - 1).double()))
        out[:, half:d_c:2] = torch.where(code >= 8, -mag, mag)
    sb = row[:, d_c // 2 + 2 * d_r:][:, :d_c // 32].int()
    e, f = sb // 8, (sb % 8).double()
    scale = torch.where(e == 0, f / 512, (1 + f / 8) * torch.pow(2.0, (e - 7).double()))
    for i in range(d_c // 32):
        out[:, 32 * i:32 * i + 32] *= scale[:, i:i + 1]
    out[:, d_c:] = row[:, d_c // 2:d_c // 2 + 2 * d_r].contiguous().view(torch.bfloat16).double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "page_plan":
        held, new, free = s["held"].tolist(), s["new"].tolist(), s["free"].tolist()
        table, taken = s["table"].tolist(), 0
        for b in range(c["B"]):
            for i in range(-(-held[b] // BLOCK_TOKENS), -(-(held[b] + new[b]) // BLOCK_TOKENS)):
                table[b][i] = free[taken]
                taken += 1
        outs = [torch.tensor(table, dtype=torch.int32)]
        for m, most in ((4, s["most_csa"]), (128, s["most_hca"])):
            got, off = [], [0]
            for b in range(c["B"]):
                got += [table[b][j * m // BLOCK_TOKENS] * (BLOCK_TOKENS // m) + j % (BLOCK_TOKENS // m)
                        for j in range(held[b] // m, (held[b] + new[b]) // m)]
                off.append(len(got))
            outs += [torch.tensor(got + [-1] * (most - len(got))), torch.tensor(off)]
        return tuple(o.cuda() for o in outs) + (torch.tensor([taken]).cuda(),)
    d_c, d_r = c["d_c"], c["d_r"]
    if c["op"] == "rows":
        v = torch.cat([_as_stored(p.double(), d_c) for p in s["x"].split(1 << 16)])
        v[s["slots"] < 0] = 0
        return v
    B, Q, H, be = c["B"], c["Q"], c["H"], c["be"]
    flat = s["pool"].view(-1, s["pool"].shape[-1])
    o = torch.zeros((B, Q, H, d_c), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), float("-inf"), dtype=torch.float64, device="cuda")
    lens, wins = s["lens"].tolist(), s["n_win"].tolist() if s["n_win"] is not None else [c["Tw"]] * B
    for b in range(B):
        if c["op"] == "hca":
            j = torch.arange(lens[b], device="cuda")
            entries = _stored_values(flat[s["table"][b, j // be].long() * be + j % be], d_c, d_r)
        for t in range(Q):
            if c["op"] == "csa":
                j = s["idx"][b, t]
                j = j[j >= 0].long()
                k = _stored_values(flat[s["table"][b, j // be].long() * be + j % be], d_c, d_r)
            else:
                k = entries
            lo, hi = 0, wins[b]
            if c["causal"]:
                first = c["N"] * c["m"] - Q
                p, p0 = first + t, first - (c["Tw"] - Q)
                lo, hi = max(0, p - c["W"] + 1 - p0), min(c["Tw"], p - p0 + 1)
                if c["op"] == "hca":
                    k = entries[:max(0, (p + 1) // c["m"])]
            k = torch.cat((k, s["win"][b, lo:hi].double()))
            if k.shape[0]:
                z = (s["q"][b, t].double() @ k.T) * s["scale"]
                lse[b, t] = torch.logsumexp(z, -1)
                o[b, t] = torch.softmax(z, -1) @ k[:, :d_c]
    return (o, lse) if c["lse"] else o
