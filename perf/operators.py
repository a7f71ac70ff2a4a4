"""The paged key/value cache's operators as measured workloads: the page tables
built from request lengths, the write of new entries into pages, and the decode
step that attends over them.

`own = False` computes each operator in elementary torch operations, in fp32
(angles of positions in fp64) and rounded once at the end; `own = True` calls the
library. listed() are the fixed cases, draw() makes further ones of the same
ranges, exact() is the definition in fp64, written apart from the plain form.

Head counts, head dims, window and batch are the d20 model's (10 heads of 128,
windows of 512, 64 decoding sequences, prompts of up to 2048) or generic
grouped-query shapes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROPE_BASE = 10000.0
EPS = 1e-6


def listed():
    return [
        # one decode step of the 64 sequences: a token each, most of them inside their last page
        dict(name="tables_step_64", op="tables", B=64, page=16, columns=256, pad=1, kind="step", scarce=False),
        # prompts admitted together with sequences that finish, packed token rows
        dict(name="tables_prompts_96", op="tables", B=96, page=64, columns=64, pad=0, kind="prompts", scarce=False),
        # a large continuous batch: single tokens, prompt chunks and ends, more asked for than the pool holds
        dict(name="tables_mixed_2048", op="tables", B=2048, page=16, columns=320, pad=0, kind="mixed", scarce=True),
        # one token of each of the 64 sequences, with the memory mixed in
        dict(name="write_step_64", op="write", n=64, H_kv=10, hd=128, page=16, dtype="bf16", mode="mix"),
        # four prompts of 2048 of an injected layer
        dict(name="write_mix_8192", op="write", n=8192, H_kv=10, hd=128, page=64, dtype="bf16", mode="mix"),
        # entries a forward pass has already mixed, copied as they are, fp32, few key/value heads
        dict(name="write_copy_5003", op="write", n=5003, H_kv=4, hd=64, page=32, dtype="f32", mode="copy"),
        # prompts of a layer without memory: rotation and write
        dict(name="write_rope_65536", op="write", n=65536, H_kv=10, hd=128, page=64, dtype="bf16", mode="rope"),
        # the first tokens of a single conversation: latency
        dict(name="decode_one_short", op="decode", B=1, H=10, H_kv=10, hd=128, page=16, longest=190, window=0,
             inject=False, dtype="bf16"),
        # the prefiller's full-causal layer over 64 ragged sequences
        dict(name="decode_full_64", op="decode", B=64, H=10, H_kv=10, hd=128, page=64, longest=4096, window=0,
             inject=False, dtype="bf16"),
        # the decoder's injected layer: the last 512 keys of sequences of any age, small pages
        dict(name="decode_window_64", op="decode", B=64, H=10, H_kv=10, hd=128, page=16, longest=8192, window=512,
             inject=True, dtype="bf16"),
        # few sequences with long caches, eight query heads to a key/value head
        dict(name="decode_grouped_long", op="decode", B=8, H=32, H_kv=4, hd=128, page=64, longest=65536, window=0,
             inject=False, dtype="bf16"),
        # two long fp32 caches, odd lengths
        dict(name="decode_f32_long", op="decode", B=2, H=8, H_kv=4, hd=64, page=32, longest=30011, window=0,
             inject=True, dtype="f32"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "write", "decode", "decode"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        kind = rng.choice(["step", "prompts", "mixed"])
        return dict(op=op, B=_log_uniform(rng, 1, 2048 if kind != "prompts" else 128), page=page,
                    columns=rng.randint(max(1, 512 // page), 5120 // page), pad=1 if kind == "step" else 0, kind=kind,
                    scarce=rng.random() < 0.4)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    hd = rng.choice([64, 128])
    if op == "write":
        H_kv = rng.choice([1, 2, 4, 8, 10])
        return dict(op=op, n=_log_uniform(rng, 1, 32768), H_kv=H_kv, hd=hd, page=page, dtype=dtype,
                    mode=rng.choice(["mix", "rope", "copy"]))
    H_kv, group = rng.choice([(10, 1), (10, 1), (8, 1), (5, 2), (4, 4), (2, 5), (4, 8), (1, 10), (2, 16), (1, 24)])
    inject = rng.random() < 0.5
    window = rng.choice([0, 0, rng.randint(1, 2048)])
    longest = _log_uniform(rng, 1, 65536)
    per_token = H_kv * hd * 2 * (4 if dtype == "f32" else 2)
    room = max(1, (300 << 20) // (per_token * min(longest, window or longest)))
    return dict(op=op, B=min(room, _log_uniform(rng, 1, 256)), H=H_kv * group, H_kv=H_kv, hd=hd, page=page,
                longest=longest, window=window, inject=inject, dtype=dtype)


# ---------------------------------------------------------------------------
# what a case holds: counts that do not depend on the seed, dealt out by it
# ---------------------------------------------------------------------------
def _request(kind, i, f, cap):
    """(cached, new) of request i, f of the way through the lengths; new = -1: finished."""
    if kind == "step":
        return int(f * (cap - 1)), 1
    if kind == "prompts":
        return (int(f * cap), -1) if i % 6 == 5 else (0, max(1, int(f * min(cap, 2048))))
    if i % 20 == 7:
        return int(f * cap), -1
    if i % 20 == 13:
        return int(f * cap / 2), min(512, cap - int(f * cap / 2))
    if i % 20 == 17:
        return int(f * cap), 0
    return int(f * (cap - 1)), 1


def _request_counts(case):
    """_request() of every request, before the seed's shuffle."""
    return [_request(case["kind"], i, (i + 0.5) / case["B"], case["columns"] * case["page"]) for i in range(case["B"])]


def _table_sizes(case):
    page, counts = case["page"], _request_counts(case)
    held = sum(-(-c // page) for c, _ in counts)
    need = sum(-(-(c + n) // page) + (-c // page) for c, n in counts if n >= 0)
    freed = sum(-(-c // page) for c, n in counts if n < 0)
    free = max(0, need - freed) + 7 if not case["scarce"] else max(0, (need - freed) * 3 // 4)
    tokens = sum(max(0, n) for _, n in counts)
    n_tokens = case["B"] * case["pad"] if case["pad"] else tokens + 5
    return held, need, freed, free, max(1, n_tokens)


def _lengths(case):
    """Positions of the decode step's new tokens, before the seed's shuffle."""
    return [int((case["longest"] - 1) * (i + 1) / case["B"]) for i in range(case["B"])]


def _pages_of(case):
    """Pages in use by the decode case's sequences: those a window still reaches."""
    page, w = case["page"], case["window"]
    return sum(p // page - (max(0, p - w + 1) // page if w else 0) + 1 for p in _lengths(case))


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)


def _gates(g, H_kv):
    return torch.rand(4, H_kv, generator=g, device="cuda") * 4 - 2


def _scratch(n):
    return torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "tables":
        B, page, columns = case["B"], case["page"], case["columns"]
        held, _, _, free, n_tokens = _table_sizes(case)
        counts = torch.tensor(_request_counts(case), dtype=torch.int64, device="cuda")
        counts = counts[torch.randperm(B, generator=g, device="cuda")]
        s["ctx_len"], s["new_len"] = counts[:, 0].contiguous(), counts[:, 1].contiguous()
        s["num_pages"] = held + free + 3
        order = torch.randperm(s["num_pages"], generator=g, device="cuda").to(torch.int32)
        # pages held by the requests, in any order, then the free ones
        cols = torch.arange(columns, device="cuda")
        used = cols[None, :] < ((s["ctx_len"] + page - 1) // page)[:, None]
        s["block_table"] = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
        s["block_table"][used] = order[:held]
        s["free_pages"] = torch.zeros(s["num_pages"], dtype=torch.int32, device="cuda")
        s["free_pages"][:free] = order[held:held + free]
        s["n_free"] = torch.tensor([free], dtype=torch.int32, device="cuda")
        s["n_tokens"] = n_tokens
        s["seq_len"] = torch.zeros(B, dtype=torch.int64, device="cuda")
        s["n_free_out"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["cu_tokens"] = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
        s["pos"] = torch.zeros(n_tokens, dtype=torch.int64, device="cuda")
        s["slots"] = torch.zeros(n_tokens, dtype=torch.int64, device="cuda")
        if own:
            s["desc"] = _desc(B=B, page_size=page, max_pages=columns, num_pages=s["num_pages"])
            s["workspace"] = _scratch(_mg().maglev_page_tables_workspace_bytes(s["desc"]))
        return s
    dt, hd, H_kv, page = DTYPES[case["dtype"]], case["hd"], case["H_kv"], case["page"]
    if case["op"] == "write":
        n = case["n"]
        s["num_pages"] = -(-n // page) + max(4, n // page // 4)
        # sequences of up to 2048 tokens, each over its own scattered pages; one row in 50 is padding
        cols = torch.randperm(s["num_pages"], generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        s["slots"] = cols[t // page] * page + t % page
        s["slots"][t % 50 == 49] = -1
        starts = torch.randint(0, 4096, (n // 2048 + 1,), generator=g, device="cuda")
        s["pos"] = starts[t // 2048] + t % 2048
        s["k"], s["v"] = _normal(g, (n, H_kv, hd), dt), _normal(g, (n, H_kv, hd), dt)
        s["R_k"] = s["R_v"] = s["gates"] = None
        if case["mode"] == "mix":
            s["R_k"], s["R_v"] = _normal(g, (n, H_kv, hd), dt), _normal(g, (n, H_kv, hd), dt)
            s["gates"] = _gates(g, H_kv)
        s["k_pages"] = _normal(g, (s["num_pages"], H_kv, page, hd), dt)
        s["v_pages"] = _normal(g, (s["num_pages"], H_kv, page, hd), dt)
        if case["mode"] == "copy":
            s["pos"] = None
        if own:
            s["desc"] = _desc(B=1, H=H_kv, H_kv=H_kv, hd=hd, page_size=page, max_pages=s["num_pages"],
                              num_pages=s["num_pages"], inject=int(case["mode"] == "mix"),
                              dtype=int(case["dtype"] == "bf16"))
        return s
    B, H, window = case["B"], case["H"], case["window"]
    pos = torch.tensor(_lengths(case), dtype=torch.int64, device="cuda")
    s["pos"] = pos[torch.randperm(B, generator=g, device="cuda")]
    s["columns"] = max(_lengths(case)) // page + 1
    used = _pages_of(case)
    s["num_pages"] = used + 3
    first = (s["pos"] - window + 1).clamp_min(0) // page if window else torch.zeros_like(s["pos"])
    cols = torch.arange(s["columns"], device="cuda")
    live = (cols[None, :] >= first[:, None]) & (cols[None, :] <= (s["pos"] // page)[:, None])
    s["block_table"] = torch.full((B, s["columns"]), -1, dtype=torch.int32, device="cuda")
    s["block_table"][live] = torch.randperm(s["num_pages"], generator=g, device="cuda")[:used].to(torch.int32)
    s["q"] = _normal(g, (B, H, hd), dt)
    s["k"], s["v"] = _normal(g, (B, H_kv, hd), dt), _normal(g, (B, H_kv, hd), dt)
    s["krec"] = s["vrec"] = s["gates"] = None
    if case["inject"]:
        x = torch.randn((B, H_kv, hd), generator=g, device="cuda")
        s["krec"] = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)).to(dt)
        s["vrec"] = _normal(g, (B, H_kv, hd), dt)
        s["gates"] = _gates(g, H_kv)
    s["k_pages"] = _normal(g, (s["num_pages"], H_kv, page, hd), dt)
    s["v_pages"] = _normal(g, (s["num_pages"], H_kv, page, hd), dt)
    s["out"] = torch.empty(B, H, hd, dtype=dt, device="cuda")
    if own:
        s["desc"] = _desc(B=B, H=H, H_kv=H_kv, hd=hd, page_size=page, max_pages=s["columns"],
                          num_pages=s["num_pages"], window=window, inject=int(case["inject"]),
                          dtype=int(case["dtype"] == "bf16"))
        s["workspace"] = _scratch(_mg().maglev_paged_decode_workspace_bytes(s["desc"]))
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _mg():
    import sliding_window_recurrent_b200 as mg
    return mg


def _desc(**kw):
    base = dict(B=1, H=1, H_kv=1, hd=128, page_size=16, max_pages=1, num_pages=1, window=0, rope_base=ROPE_BASE,
                rms_eps=EPS, inject=0, dtype=1, shared_kv_gates=0)
    base.update(kw)
    return _mg().PagedDesc(**base)


def _run_own(s):
    mg = _mg()
    if s["op"] == "tables":
        mg.maglev_page_tables(s["desc"], s["ctx_len"], s["new_len"], s["n_tokens"], s["pad"], s["free_pages"],
                              s["n_free"], s["block_table"], s["seq_len"], s["n_free_out"], s["cu_tokens"], s["pos"],
                              s["slots"], s["workspace"])
        return {k: s[k] for k in ("block_table", "free_pages", "n_free_out", "seq_len", "cu_tokens", "pos", "slots")}
    if s["op"] == "write":
        mg.maglev_paged_write(s["desc"], s["n"], s["slots"], s["pos"], s["k"], s["v"], s["R_k"], s["R_v"], s["gates"],
                              s["k_pages"], s["v_pages"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    mg.maglev_paged_decode_step(s["desc"], s["pos"], s["q"], s["k"], s["v"], s["krec"], s["vrec"], s["gates"],
                                s["block_table"], s["k_pages"], s["v_pages"], s["out"], s["workspace"])
    return {"out": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def run(state):
    if own:
        return _run_own(state)
    return {"tables": _plain_tables, "write": _plain_write, "decode": _plain_decode}[state["op"]](state)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_tables(s):
    page, columns, pad, n_tokens = s["page"], s["columns"], s["pad"], s["n_tokens"]
    ctx, new = s["ctx_len"], s["new_len"]
    dev, cap = ctx.device, columns * page
    done, held = new < 0, (ctx + page - 1) // page
    rel = torch.where(done, held, torch.zeros_like(held))
    rel_end = rel.cumsum(0)
    rows = new.clamp(0, n_tokens + 1)
    row_end = rows.cumsum(0)
    cu = torch.cat([row_end.new_zeros(1), row_end]).clamp_max(n_tokens)
    fits = ~done & (ctx + rows <= cap) & (rows <= pad if pad else row_end <= n_tokens)
    need = torch.where(fits, (ctx + rows + page - 1) // page - held, torch.zeros_like(held))
    need_end = need.cumsum(0)
    n_free = s["n_free"].to(torch.int64)
    avail = n_free + rel_end[-1:]
    served = fits & ((need == 0) | (need_end <= avail))
    take = torch.where(served, need, torch.zeros_like(need))
    taken = take.sum()
    # the free stack with the pages that finished requests give back on top
    j = torch.arange(s["num_pages"], device=dev)
    back = (j - n_free).clamp_min(0)
    r = torch.searchsorted(rel_end, back, right=True).clamp_max(ctx.numel() - 1)
    col = (back - (rel_end - rel)[r]).clamp(0, columns - 1)
    stack = torch.where(j < n_free, s["free_pages"], s["block_table"][r, col])
    left = avail - taken
    c = torch.arange(columns, device=dev)
    mine = served[:, None] & (c >= held[:, None]) & (c < (held + take)[:, None])
    top = (avail - 1 - ((need_end - need)[:, None] + c - held[:, None])).clamp(0, s["num_pages"] - 1)
    table = torch.where(mine, stack[top], s["block_table"])
    free = torch.where((j >= n_free) & (j < left), stack, s["free_pages"])
    t = torch.arange(n_tokens, device=dev)
    if pad:
        b = t // pad
        i = t - b * pad
    else:
        b = torch.searchsorted(cu[1:], t, right=True).clamp_max(ctx.numel() - 1)
        i = t - cu[b]
    p = ctx[b] + i
    live = served[b] & (i < rows[b])
    pc = (p // page).clamp_max(columns - 1)
    slot = table[b, pc].to(torch.int64) * page + p % page
    none = torch.full_like(p, -1)
    return {"block_table": table, "free_pages": free, "n_free_out": left.to(torch.int32),
            "seq_len": torch.where(done, torch.zeros_like(ctx), torch.where(served, ctx + rows, ctx)),
            "cu_tokens": cu, "pos": torch.where(live, p, none), "slots": torch.where(live, slot, none)}


def _cos_sin(pos, hd):
    freq = ROPE_BASE ** (-torch.arange(0, hd, 2, device=pos.device, dtype=torch.float64) / hd)
    a = pos.to(torch.float64)[:, None] * freq
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _rotate(x, cos, sin):
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)


def _gate(gates):
    return (2.0 / (1.0 + torch.exp(-gates)))[:, None, :, None]


def _plain_write(s):
    k, v = s["k"].float(), s["v"].float()
    if s["pos"] is not None:
        cos, sin = _cos_sin(s["pos"], s["hd"])
        k = _rotate(k, cos, sin)
        if s["R_k"] is not None:
            r = s["R_k"].float()
            r = _rotate(r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS), cos, sin)
            g = _gate(s["gates"])
            k = g[0] * k + g[1] * r
            v = g[2] * v + g[3] * s["R_v"].float()
    page = s["page"]
    row = s["slots"].argsort()[s["n"] // 50:]  # the padding rows come first
    at = s["slots"][row]
    s["k_pages"][at // page, :, at % page] = k[row].to(s["k_pages"].dtype)
    s["v_pages"][at // page, :, at % page] = v[row].to(s["v_pages"].dtype)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_decode(s):
    B, H, H_kv, hd, page, window = s["B"], s["H"], s["H_kv"], s["hd"], s["page"], s["window"]
    pos, dt = s["pos"], s["k_pages"].dtype
    cos, sin = _cos_sin(pos, hd)
    q = _rotate(s["q"].float(), cos, sin)
    k, v = _rotate(s["k"].float(), cos, sin), s["v"].float()
    if s["gates"] is not None:
        g = _gate(s["gates"])
        k = g[0] * k + g[1] * s["krec"].float()
        v = g[2] * v + g[3] * s["vrec"].float()
    rows = torch.arange(B, device=pos.device)
    own_page = s["block_table"][rows, pos // page].long()
    s["k_pages"][own_page, :, pos % page] = k.to(dt)
    s["v_pages"][own_page, :, pos % page] = v.to(dt)
    # the columns the longest window or sequence covers, counted from each row's first
    first = (pos - window + 1).clamp_min(0) // page if window else torch.zeros_like(pos)
    span = min(s["columns"], (window - 1) // page + 2) if window else s["columns"]
    cols = first[:, None] + torch.arange(span, device=pos.device)
    ids = s["block_table"].gather(1, cols.clamp_max(s["columns"] - 1)).long().clamp_min(0)
    at = (cols[:, :, None] * page + torch.arange(page, device=pos.device)).reshape(B, 1, 1, span * page)
    keep = at <= pos[:, None, None, None]
    if window:
        keep = keep & (at > pos[:, None, None, None] - window)
    keys = s["k_pages"][ids].transpose(1, 2).reshape(B, H_kv, span * page, hd).float()
    score = q.view(B, H_kv, H // H_kv, hd) @ keys.transpose(-1, -2) / math.sqrt(hd)
    score = torch.where(keep, score, torch.full_like(score, float("-inf")))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    vals = s["v_pages"][ids].transpose(1, 2).reshape(B, H_kv, span * page, hd).float()
    out = (p @ vals).reshape(B, H, hd).to(dt)
    return {"out": out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ---------------------------------------------------------------------------
# work and definition
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "tables":
        B = case["B"]
        _, need, _, free, n_tokens = _table_sizes(case)
        # lengths in and out, offsets, the pages handed out (read and written), position and slot of every token
        return {"bytes": B * (8 * 3) + 8 * (B + 1) + 8 * need + 16 * n_tokens, "flops": 0}
    size = 4 if case["dtype"] == "f32" else 2
    row = case["H_kv"] * case["hd"]
    if case["op"] == "write":
        per = {"copy": 4, "rope": 4, "mix": 6}[case["mode"]]
        n = case["n"] - case["n"] // 50
        return {"bytes": n * per * row * size + case["n"] * (8 if case["mode"] == "copy" else 16),
                "flops": n * row * {"copy": 0, "rope": 3, "mix": 12}[case["mode"]]}
    w = case["window"]
    keys = sum(min(p, w - 1) if w else p for p in _lengths(case))  # cached ones; the new entry is written
    B, H = case["B"], case["H"]
    new = B * (2 + 2 + (2 if case["inject"] else 0)) * row * size + 2 * B * H * case["hd"] * size
    return {"bytes": 2 * keys * row * size + new + 4 * _pages_of(case), "flops": 4 * (keys + B) * H * case["hd"]}


def _turn(x, pos):
    """x [n, heads, hd] fp64 turned by its position, as complex numbers."""
    half = x.shape[-1] // 2
    theta = torch.exp(-math.log(ROPE_BASE) * torch.arange(half, device=x.device, dtype=torch.float64) / half)
    w = torch.polar(torch.ones((), device=x.device, dtype=torch.float64), pos.double()[:, None] * theta)[:, None]
    y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * w
    return torch.cat([y.real, y.imag], -1)


def _entry64(s, krec, vrec, k, v, pos):
    k, v = _turn(k.double(), pos), v.double()
    if krec is None:
        return k, v
    a, b, c, d = (2 * torch.sigmoid(s["gates"].double()))[:, None, :, None]
    return a * k + b * krec, c * v + d * vrec.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":  # request by request, on the host
        page, columns, pad, n_tokens = s["page"], s["columns"], s["pad"], s["n_tokens"]
        ctx, new = s["ctx_len"].tolist(), s["new_len"].tolist()
        table, n_free = s["block_table"].cpu(), int(s["n_free"].item())
        free = s["free_pages"].cpu()
        stack = free[:n_free].tolist()
        lens, cu, row = list(ctx), [0], 0
        pos, slots = torch.full((n_tokens,), -1), torch.full((n_tokens,), -1)
        for b, (c, n) in enumerate(zip(ctx, new)):
            if n < 0:
                stack += table[b, :-(-c // page)].tolist()
                lens[b] = 0
        budget, asked = len(stack), 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            start, n = (b * pad if pad else row), max(n, 0)
            row += n
            cu.append(min(row, n_tokens))
            if new[b] < 0 or c + n > columns * page or (n > pad if pad else row > n_tokens):
                continue
            lo, hi = -(-c // page), -(-(c + n) // page)
            asked += hi - lo
            if hi > lo and asked > budget:
                continue
            for col in range(lo, hi):
                table[b, col] = stack.pop()
            at = torch.arange(c, c + n)
            pos[start:start + n] = at
            slots[start:start + n] = table[b, at // page].long() * page + at % page
            lens[b] = c + n
        if len(stack) > n_free:
            free[n_free:len(stack)] = torch.tensor(stack[n_free:], dtype=free.dtype)
        return {"block_table": table, "free_pages": free, "n_free_out": torch.tensor([len(stack)], dtype=torch.int32),
                "seq_len": torch.tensor(lens), "cu_tokens": torch.tensor(cu), "pos": pos, "slots": slots}
    page, kp, vp = case["page"], s["k_pages"].double(), s["v_pages"].double()
    if case["op"] == "write":
        k, v = s["k"].double(), s["v"].double()
        if case["mode"] != "copy":
            r = None
            if case["mode"] == "mix":
                r = s["R_k"].double()
                r = _turn(r / (r.square().mean(-1, keepdim=True) + EPS).sqrt(), s["pos"])
            k, v = _entry64(s, r, s["R_v"], k, v, s["pos"])
        t = (s["slots"] >= 0).nonzero()[:, 0]
        a, o = s["slots"][t] // page, s["slots"][t] % page
        kp[a, :, o], vp[a, :, o] = k[t], v[t]
        return {"k_pages": kp, "v_pages": vp}
    k, v = _entry64(s, None if s["krec"] is None else s["krec"].double(), s["vrec"], s["k"], s["v"], s["pos"])
    q = _turn(s["q"].double(), s["pos"])
    dt, group = s["k_pages"].dtype, case["H"] // case["H_kv"]
    out = torch.empty(s["q"].shape, device="cuda", dtype=torch.float64)
    for b, p in enumerate(s["pos"].tolist()):
        lo = max(0, p - case["window"] + 1) if case["window"] else 0
        ids = s["block_table"][b, lo // page:p // page + 1].long()
        skip = lo - lo // page * page
        n = p - lo  # cached keys, then the new entry as the cache stores it
        key = s["k_pages"][ids].transpose(0, 1).reshape(case["H_kv"], -1, case["hd"])[:, skip:skip + n].double()
        val = s["v_pages"][ids].transpose(0, 1).reshape(case["H_kv"], -1, case["hd"])[:, skip:skip + n].double()
        key = torch.cat([key, k[b].to(dt).double()[:, None]], 1).repeat_interleave(group, 0)
        val = torch.cat([val, v[b].to(dt).double()[:, None]], 1).repeat_interleave(group, 0)
        w = torch.softmax((key * q[b][:, None]).sum(-1) * case["hd"] ** -0.5, -1)
        out[b] = (w[..., None] * val).sum(1)
        a = int(s["block_table"][b, p // page])
        kp[a, :, p % page], vp[a, :, p % page] = k[b], v[b]
    return {"out": out, "k_pages": kp, "v_pages": vp}
