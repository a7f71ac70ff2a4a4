"""The paged cache on the GPU, through the C ABI, against the fp64 oracle.

Bounds. A stored value is rounded once: at most eps/2 of itself (bf16 2^-8, fp32
2^-24), beside fp32 arithmetic errors that are bounded term by term below (U =
2^-24 per fp32 operation).
  entries: each is a sum of at most four products of an input, a cosine or sine
    (its angle rounded to fp32 in [-pi, pi]: pi U, its value 2 U), a gate (8 U) and
    a norm factor (hd/16 + 8 additions and roundings U): 64 U times the sum of
    the magnitudes covers it for hd <= 128.
  attention: scores are dot products of hd terms. With q rotated in fp32 (16 U) and
    carried in two bf16 parts (2^-16) the error of a score is at most e = (2^-16 +
    (hd + 32) U) |q| |k| / sqrt(hd). Weights then err by a factor 1 + 2 e + 2^-16 (the
    weights' own two parts) + 8 U, their sums over n keys by n U, all relative to the
    largest |v|.
The attention is checked against the pages as the call left them, so that the
new entry's own rounding is not counted twice.
"""
import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sliding_window_recurrent_b200 import build as _build
    _build.build(quiet=True)
    import sliding_window_recurrent_b200 as mg
    from sliding_window_recurrent_b200.layer import PagedLayerState, PageTables

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(x):
    return x.detach().to(torch.float64).cpu().numpy()


def normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(TD[dtype])


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def desc(dtype="bf16", **kw):
    base = dict(B=1, H=2, H_kv=2, hd=128, page_size=16, max_pages=4, num_pages=8, window=0, rope_base=10000.0,
                rms_eps=1e-6, inject=0, dtype=int(dtype == "bf16"), shared_kv_gates=0)
    base.update(kw)
    return mg.PagedDesc(**base)


def within(got, ref, tol, name):
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{name}: non-finite values"
    bad = err > tol
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} beyond the bound, worst {np.max(err / tol):.3g} of it"


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------
class Tables:
    """Device copies of one step's inputs, and the call."""

    def __init__(self, lens, new, n_tokens, pad, ps, free, table, pool):
        i64 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int64, device="cuda")
        self.B, self.columns = table.shape
        self.lens, self.new = i64(lens), i64(new)
        self.free = torch.full((pool,), -7, dtype=torch.int32, device="cuda")
        self.free[:len(free)] = torch.tensor(free, dtype=torch.int32)
        self.n_free = torch.tensor([len(free)], dtype=torch.int32, device="cuda")
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda")
        self.seq_len, self.cu = torch.empty_like(self.lens), i64(np.zeros(self.B + 1))
        self.n_out = torch.empty_like(self.n_free)
        self.pos, self.slots = (torch.full((max(n_tokens, 1),), -9, dtype=torch.int64, device="cuda") for _ in range(2))
        self.args = (n_tokens, pad)
        self.desc = desc(B=self.B, page_size=ps, max_pages=self.columns, num_pages=pool)
        self.ws = torch.empty(mg.maglev_page_tables_workspace_bytes(self.desc), dtype=torch.uint8, device="cuda")

    def run(self, stream=None, in_place=False):
        mg.maglev_page_tables(self.desc, self.lens, self.new, *self.args, self.free, self.n_free, self.table,
                              self.lens if in_place else self.seq_len, self.n_free if in_place else self.n_out, self.cu,
                              self.pos, self.slots, self.ws, stream)

    def check(self, want, in_place=False):
        torch.cuda.synchronize()
        n = self.args[0]
        eq = np.testing.assert_array_equal
        eq(self.table.cpu().numpy(), want["block_table"])
        eq((self.lens if in_place else self.seq_len).cpu().numpy(), want["seq_len"])
        eq(self.cu.cpu().numpy(), want["cu_tokens"])
        eq(self.pos[:n].cpu().numpy(), want["pos"])
        eq(self.slots[:n].cpu().numpy(), want["slots"])
        left = int((self.n_free if in_place else self.n_out).item())
        assert left == len(want["free"])
        eq(self.free[:left].cpu().numpy(), want["free"])
        assert mg.maglev_device_status() == mg.MAGLEV_OK


def draw_tables(seed, B, ps, columns, pad, mix, spare):
    """lens, new, n_tokens, free list, table, pool of one step; spare: free pages per page asked for."""
    r = np.random.Generator(np.random.Philox(seed))
    cap = columns * ps
    lens = r.integers(0, cap + 1, B)
    new = np.ones(B, dtype=np.int64)
    if mix:
        new = np.where(r.random(B) < 0.5, new, r.integers(0, cap + 2, B))
        new[r.random(B) < 0.2] = -1
        new[r.random(B) < 0.1] = 0
    held = -(-lens // ps)
    asked = int(np.maximum(-(-(lens + np.maximum(new, 0)) // ps) - held, 0).sum())
    pool = int(held.sum()) + int(asked * spare) + 3
    order = r.permutation(pool).astype(np.int32)
    table = np.full((B, columns), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    n_tokens = B * pad if pad else int(np.maximum(new, 0).sum())
    return lens, new, n_tokens, [int(x) for x in order[at:pool - 3]], table, pool


@pytest.mark.parametrize("B,ps,columns,pad,mix,spare,extra", [
    (1, 16, 1, 0, False, 1.0, 0), (1, 16, 3, 1, False, 1.0, 0), (64, 16, 20, 1, False, 1.0, 0), (64, 16, 20, 1, False, 0.3, 0),
    (7, 16, 9, 0, True, 1.0, 0), (7, 64, 9, 0, True, 0.4, 13), (33, 32, 5, 50, True, 0.7, 0), (33, 256, 3, 300, True, 0.7, 0),
    (1023, 16, 4, 0, True, 1.0, 5), (1024, 16, 4, 0, True, 0.5, 0), (1025, 16, 4, 1, True, 0.5, 0),
    (2500, 128, 2, 0, True, 0.6, -3000), (3, 16, 700, 0, True, 1.0, 0), (5000, 16, 2, 1, False, 0.9, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_tables(B, ps, columns, pad, mix, spare, extra, in_place):
    """Every output equals the oracle's, for packed and padded rows, few and many requests, pages that run out,
    rows behind the last token (extra > 0) and too few token rows (extra < 0)."""
    lens, new, n_tokens, free, table, pool = draw_tables(B + columns, B, ps, columns, pad, mix, spare)
    n_tokens = max(0, n_tokens + extra)
    t = Tables(lens, new, n_tokens, pad, ps, free, table, pool)
    t.run(in_place=in_place)
    t.check(oracle.page_tables(lens, new, n_tokens, pad, ps, free, table), in_place)


def test_page_tables_many_returned_pages():
    """Finished requests give back more pages than are taken, over one and over two launches."""
    for n_tokens in (6, 9000):
        B, ps, columns = 40, 16, 600
        r = np.random.Generator(np.random.Philox(n_tokens))
        lens = r.integers(0, columns * ps // 2, B)
        new = np.full(B, -1, dtype=np.int64)
        new[::9] = [n_tokens // 6] * len(new[::9])
        held = -(-lens // ps)
        pool = int(held.sum()) + 4
        order = r.permutation(pool).astype(np.int32)
        table = np.full((B, columns), -1, dtype=np.int32)
        for b in range(B):
            table[b, :held[b]] = order[held[:b].sum():held[:b + 1].sum()]
        free = [int(x) for x in order[pool - 4:]]
        t = Tables(lens, new, n_tokens, 0, ps, free, table, pool)
        t.run()
        t.check(oracle.page_tables(lens, new, n_tokens, 0, ps, free, table))


@pytest.mark.parametrize("B,ps,columns,take", [(5, 16, 4, 0.5), (9, 16, 40, 0.9), (40, 16, 600, 0.3), (96, 64, 64, 0.8),
                                               (2048, 16, 20, 0.7), (2500, 16, 9, 1.0), (1, 16, 5000, 0.6)])
@pytest.mark.parametrize("many_rows", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_tables_of_rows_that_gave_pages_back_before(B, ps, columns, take, many_rows, in_place):
    """Finished requests whose first columns hold no page any more (negative) give back the others, in order, over one and
    over two launches; `take` of what is there then is handed out again."""
    r = np.random.Generator(np.random.Philox(B + columns + many_rows))
    cap = columns * ps
    lens = r.integers(1, cap + 1, B)
    new = np.full(B, -1, dtype=np.int64)
    new[B // 3::3] = 0
    held = -(-lens // ps)
    pool = int(held.sum()) + 4
    order = r.permutation(pool).astype(np.int32)
    table = np.full((B, columns), -1, dtype=np.int32)
    for b in range(B):
        table[b, :held[b]] = order[held[:b].sum():held[:b + 1].sum()]
    for b in np.flatnonzero(new < 0):
        if b % 3 != 1:
            table[b, :r.integers(0, held[b] + 1)] = -1 - 4 * (b % 2)  # what a window has passed
    back = int((table[new < 0] >= 0).sum())
    idle = np.flatnonzero(new == 0)
    lens[idle] = 0  # empty rows that ask for `take` of the pages between them
    for i, b in enumerate(idle):
        new[b] = min(cap, int((back + 4) * take) // len(idle) * ps - (0 if many_rows else ps - 1))
        new[b] = max(new[b], 0)
    n_tokens = int(new[new > 0].sum()) if many_rows else min(500, int(new[new > 0].sum()))
    free = [int(x) for x in order[pool - 4:]]
    t = Tables(lens, new, n_tokens, 0, ps, free, table, pool)
    t.run(in_place=in_place)
    t.check(oracle.page_tables(lens, new, n_tokens, 0, ps, free, table, pool), in_place)


@pytest.mark.parametrize("B", [3, 2050])
@pytest.mark.parametrize("new", [-1, 0, 1])
@pytest.mark.parametrize("length", [-5, 33, 1 << 40])
def test_page_tables_record_a_bad_length_alone(B, new, length):
    """A length outside its row, with nothing else wrong: recorded; a running request is not served, a finished one gives
    nothing back (its row would name pages that it does not hold)."""
    table = np.full((B, 2), -1, dtype=np.int32)
    table[1] = [3, 4]
    lens, news = np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64)
    lens[1], news[1] = length, new
    t = Tables(lens, news, 4, 0, 16, [2], table, 6)
    t.run()
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == mg.MAGLEV_ERR_BOUNDS
    assert t.n_out.tolist() == [1] and t.free.tolist() == [2] + [-7] * 5
    assert t.seq_len[1].item() == (0 if new < 0 else length) and (t.pos == -1).all() and (t.slots == -1).all()
    np.testing.assert_array_equal(t.table.cpu().numpy(), table)


@pytest.mark.parametrize("B", [3, 2050])
@pytest.mark.parametrize("bad", [-1, 6, 1 << 30])
def test_page_tables_keep_numbers_outside_the_pool_off_the_stack(B, bad):
    """A finished row that names no page behind its first one: recorded, its place on the stack holds -1; handed out
    again it gives no slot."""
    table = np.full((B, 3), -1, dtype=np.int32)
    table[1] = [3, bad, 4]
    lens, news = np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64)
    lens[1], news[1] = 48, -1
    t = Tables(lens, news, 0, 0, 16, [2], table, 6)
    t.run(in_place=True)
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == mg.MAGLEV_ERR_BOUNDS
    assert t.n_free.tolist() == [4] and t.free.tolist() == [2, 3, -1, 4, -7, -7] and (t.lens == 0).all()
    t.new.zero_()
    t.new[2] = 17
    t.args = (17, 0)
    t.pos, t.slots = (torch.full((17,), -9, dtype=torch.int64, device="cuda") for _ in range(2))
    t.run(in_place=True)
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == mg.MAGLEV_ERR_BOUNDS
    assert t.slots.tolist() == list(range(64, 80)) + [-1] and t.pos.tolist() == list(range(16)) + [-1]
    assert t.n_free.tolist() == [2] and t.free[:2].tolist() == [2, 3]


def test_page_tables_without_token_rows():
    """Only ends and idle requests: no rows, pos and slots NULL; requests with tokens find no room and stay."""
    table = np.array([[4, 2], [3, -1], [0, -1]], dtype=np.int32)
    t = Tables([20, 7, 16], [-1, 0, 3], 0, 0, 16, [1], table, 6)
    t.pos = t.slots = None
    t.run()
    torch.cuda.synchronize()
    assert t.seq_len.tolist() == [0, 7, 16] and t.cu.tolist() == [0, 0, 0, 0] and t.n_out.tolist() == [3]
    assert t.free[:3].tolist() == [1, 4, 2] and mg.maglev_device_status() == 0


def test_index_arrays_may_be_slices():
    """Lengths, positions, slots and tables at odd places of larger arrays (their type's alignment only)."""
    B, ps, columns = 5, 16, 3
    lens, new, n_tokens, free, table, pool = draw_tables(3, B, ps, columns, 0, True, 1.0)
    t = Tables(lens, new, n_tokens, 0, ps, free, table, pool)

    def odd(x):
        big = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        big[1:] = x.flatten()
        return big[1:].view(x.shape)

    for name in ("lens", "new", "free", "n_free", "table", "seq_len", "n_out", "cu", "pos", "slots"):
        setattr(t, name, odd(getattr(t, name)))
    t.run()
    t.check(oracle.page_tables(lens, new, n_tokens, 0, ps, free, table))
    s = Step(3, [40, 3, -1], 4, 2, 64, 16)
    s.pos, s.table = odd(s.pos), odd(s.table)
    run_checked(s)
    k = normal(generator(3), (3, 2, 64), "bf16")
    kp, vp = torch.zeros(2, 2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    mg.maglev_paged_write(desc(hd=64, num_pages=2), 3, odd(torch.tensor([3, 31, 16], device="cuda")),
                          odd(torch.tensor([0, 0, 0], device="cuda")), k, k, None, None, None, kp, vp)
    torch.cuda.synchronize()
    assert torch.equal(vp[1, :, 15], k[1]) and torch.equal(kp[1, :, 0], k[2])


def test_page_tables_bad_lengths_and_pages():
    """Lengths outside a row are refused; a page number outside the pool gives no slot and is recorded; a free count
    above the pool's size is cut and recorded. (All are bounds checks of the kernel; nothing is followed.)"""
    table = np.array([[3, -1], [1 << 30, -1], [0, 1]], dtype=np.int32)
    t = Tables([-5, 3, 32], [1, 1, 1], 3, 0, 16, [2], table, 5)
    t.run()
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == mg.MAGLEV_ERR_BOUNDS
    assert t.slots.tolist() == [-1, -1, -1] and t.pos.tolist() == [-1, -1, -1]
    assert t.seq_len.tolist() == [-5, 4, 32] and t.n_out.tolist() == [1]
    t = Tables([0], [1 << 62], 3, 0, 16, [2], table[:1], 5)
    t.run()
    torch.cuda.synchronize()
    assert t.seq_len.tolist() == [0] and t.cu.tolist() == [0, 3] and t.slots.tolist() == [-1] * 3
    assert mg.maglev_device_status() == mg.MAGLEV_OK
    t = Tables([0], [1], 1, 0, 16, [2], table[:1], 5)
    t.n_free.fill_(1 << 30)
    t.run()
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == mg.MAGLEV_ERR_BOUNDS and t.n_out.tolist() == [4]


# ---------------------------------------------------------------------------
# writes
# ---------------------------------------------------------------------------
def entry_bound(pos, k, v, R_k, R_v, gates, ref_k, ref_v, dtype, eps=1e-6):
    """Bounds on the stored entries' errors (see the file's head)."""
    spread = lambda x: np.abs(x) + np.abs(np.roll(x, x.shape[-1] // 2, -1))  # both channels of a pair
    mk, mv = spread(k), np.abs(v)
    if R_k is not None:
        g = oracle.gate(oracle.gate_rows(gates))[:, None, :, None]
        mk = g[0] * mk + g[1] * spread(oracle.rmsnorm(R_k, eps))
        mv = g[2] * mv + g[3] * np.abs(R_v)
    h = HALF[dtype]
    return h * np.abs(ref_k) + 64 * U * mk, h * np.abs(ref_v) + 64 * U * mv


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,H_kv,ps,n", [(128, 10, 16, 1), (64, 1, 32, 5), (128, 3, 64, 333), (64, 7, 256, 1000),
                                          (128, 2, 128, 5000), (64, 10, 16, 2369), (128, 40, 32, 70), (64, 130, 16, 9)])
@pytest.mark.parametrize("mode", ["copy", "rope", "mix", "mix_shared"])
def test_paged_write(dtype, hd, H_kv, ps, n, mode):
    """Entries against the oracle within the bounds, every other slot as it was (NaN bytes included), rows with a
    negative slot or position skipped; positions up to 2^30."""
    gen = generator(n + hd)
    pool = -(-n // ps) + 3
    order = torch.randperm(pool * ps, generator=gen, device="cuda")[:n]
    slots = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.1, torch.full_like(order, -1), order)
    if n == 1:
        slots = order
    pos = torch.randint(0, 1 << 30, (n,), generator=gen, device="cuda")
    pos[::3] %= 4096
    inject = mode.startswith("mix")
    k, v, R_k, R_v = (normal(gen, (n, H_kv, hd), dtype) for _ in range(4))
    gates = torch.rand(2 if mode == "mix_shared" else 4, H_kv, generator=gen, device="cuda") * 4 - 2
    gates[1, 0] = float("-inf")
    if n > 1 and mode != "copy":
        pos[1] = -1
    kp, vp = (torch.full((pool, H_kv, ps, hd), float("nan"), dtype=TD[dtype], device="cuda") for _ in range(2))
    d = desc(dtype, H=H_kv, H_kv=H_kv, hd=hd, page_size=ps, num_pages=pool, inject=int(inject),
             shared_kv_gates=int(mode == "mix_shared"))
    mg.maglev_paged_write(d, n, slots, None if mode == "copy" else pos, k, v, R_k if inject else None,
                          R_v if inject else None, gates if inject else None, kp, vp)
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == mg.MAGLEV_OK
    sl = slots.cpu().numpy()
    if mode != "copy":
        sl = np.where(pos.cpu().numpy() < 0, -1, sl)
    rows = np.flatnonzero(sl >= 0)
    got_k, got_v = (host(x)[sl[rows] // ps, :, sl[rows] % ps] for x in (kp, vp))
    if mode == "copy":
        np.testing.assert_array_equal(got_k, host(k)[rows])
        np.testing.assert_array_equal(got_v, host(v)[rows])
    else:
        p = pos.cpu().numpy()[rows]
        rk, rv, g = (host(R_k)[rows], host(R_v)[rows], host(gates)) if inject else (None, None, None)
        ref_k, ref_v = oracle.paged_entries(p, host(k)[rows], host(v)[rows], rk, rv, g)
        tk, tv = entry_bound(p, host(k)[rows], host(v)[rows], rk, rv, g, ref_k, ref_v, dtype)
        within(got_k, ref_k, tk, "k")
        within(got_v, ref_v, tv, "v")
    rest = np.ones((pool, ps), dtype=bool)
    rest[sl[rows] // ps, sl[rows] % ps] = False
    for x in (kp, vp):
        assert torch.isnan(x.transpose(1, 2)[torch.from_numpy(rest).cuda()].float()).all()


def test_paged_write_refuses_slots_outside_the_pool():
    k = torch.randn(3, 2, 64, device="cuda")
    kp, vp = torch.zeros(2, 2, 2, 16, 64, device="cuda")
    slots = torch.tensor([32, 5, 1 << 40], device="cuda")
    mg.maglev_paged_write(desc("f32", hd=64, num_pages=2), 3, slots, None, k, k, None, None, None, kp, vp)
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == mg.MAGLEV_ERR_BOUNDS
    assert torch.equal(kp[0, :, 5], k[1]) and int((kp != 0).sum()) == k[1].numel()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
class Step:
    """A decode step's inputs over scattered pages; everything the step may not read is NaN or -1."""

    def __init__(self, seed, pos, H, H_kv, hd, ps, window=0, inject=False, shared=False, dtype="bf16", spare=2,
                 scale=1.0):
        gen = generator(seed)
        self.pos_h = np.asarray(pos, dtype=np.int64)
        B = len(pos)
        self.B, self.H, self.H_kv, self.hd, self.ps, self.window, self.dtype = B, H, H_kv, hd, ps, window, dtype
        columns = int(self.pos_h.max()) // ps + 1 if B and self.pos_h.max() >= 0 else 1
        lo = np.maximum(0, self.pos_h - window + 1) if window else np.zeros_like(self.pos_h)
        first, count = lo // ps, np.where(self.pos_h >= 0, self.pos_h // ps - lo // ps + 1, 0)
        pool = int(count.sum()) + spare
        order = np.random.Generator(np.random.Philox(seed)).permutation(pool)
        table = np.full((B, columns), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            table[b, first[b]:first[b] + count[b]] = order[at:at + count[b]]
            at += count[b]
        self.kp, self.vp = (torch.full((pool, H_kv, ps, hd), float("nan"), dtype=TD[dtype], device="cuda")
                            for _ in range(2))
        for b in range(B):
            if self.pos_h[b] > lo[b]:
                j = torch.arange(int(lo[b]), int(self.pos_h[b]))
                page = torch.from_numpy(table[b]).long()[j // ps].cuda()
                self.kp[page, :, (j % ps).cuda()] = normal(gen, (len(j), H_kv, hd), dtype) * scale
                self.vp[page, :, (j % ps).cuda()] = normal(gen, (len(j), H_kv, hd), dtype)
        self.table_h, self.table = table, torch.from_numpy(table).cuda()
        self.pos = torch.from_numpy(self.pos_h).cuda()
        self.q = normal(gen, (B, H, hd), dtype) * scale
        self.k, self.v = (normal(gen, (B, H_kv, hd), dtype) for _ in range(2))
        self.krec = self.vrec = self.gates = None
        if inject:
            self.krec, self.vrec = (normal(gen, (B, H_kv, hd), dtype) for _ in range(2))
            self.gates = torch.rand(2 if shared else 4, H_kv, generator=gen, device="cuda") * 4 - 2
        self.out = torch.full((B, H, hd), float("nan"), dtype=TD[dtype], device="cuda")
        self.desc = desc(dtype, B=B, H=H, H_kv=H_kv, hd=hd, page_size=ps, max_pages=columns, num_pages=pool,
                         window=window, inject=int(inject), shared_kv_gates=int(shared))
        self.ws = torch.zeros(max(16, mg.maglev_paged_decode_workspace_bytes(self.desc)), dtype=torch.uint8,
                              device="cuda")

    def run(self, stream=None):
        mg.maglev_paged_decode_step(self.desc, self.pos, self.q, self.k, self.v, self.krec, self.vrec, self.gates,
                                    self.table, self.kp, self.vp, self.out, self.ws, stream)
        return self.out

    def check(self, before, status=0):
        """Output, the written entries and every untouched byte of the pools."""
        torch.cuda.synchronize()
        assert mg.maglev_device_status() == status
        bits = torch.int16 if self.dtype == "bf16" else torch.int32
        live = np.flatnonzero(self.pos_h >= 0)
        page = self.table_h[live, self.pos_h[live] // self.ps]
        row = self.pos_h[live] % self.ps
        same = torch.ones(self.kp.shape[0], self.ps, dtype=torch.bool, device="cuda")
        same[torch.from_numpy(page).long().cuda(), torch.from_numpy(row).cuda()] = False
        for new, old in zip((self.kp, self.vp), before):
            assert torch.equal(new.view(bits).transpose(1, 2)[same], old.view(bits).transpose(1, 2)[same])
        rec = (None, None, None) if self.krec is None else tuple(host(x)[live] for x in (self.krec, self.vrec)) + (
            host(self.gates),)
        k, v = host(self.k)[live], host(self.v)[live]
        posb = np.broadcast_to(self.pos_h[live][:, None], k.shape[:2])
        ref_k, ref_v = oracle.rope(k, posb, 10000.0), v
        tk, tv = entry_bound(None, k, v, None, None, None, ref_k, ref_v, self.dtype)
        if rec[0] is not None:
            g = oracle.gate(oracle.gate_rows(rec[2]))[:, None, :, None]
            mag = np.abs(k) + np.abs(np.roll(k, self.hd // 2, -1))
            ref_k, ref_v = g[0] * ref_k + g[1] * rec[0], g[2] * v + g[3] * rec[1]
            tk = HALF[self.dtype] * np.abs(ref_k) + 64 * U * (g[0] * mag + g[1] * np.abs(rec[0]))
            tv = HALF[self.dtype] * np.abs(ref_v) + 64 * U * (g[2] * np.abs(v) + g[3] * np.abs(rec[1]))
        pg, rw = torch.from_numpy(page).long().cuda(), torch.from_numpy(row).cuda()
        if len(live):
            within(host(self.kp[pg, :, rw]), ref_k, tk, "new k")
            within(host(self.vp[pg, :, rw]), ref_v, tv, "new v")
        self.check_out(live)

    def check_out(self, live):
        got = host(self.out)
        for b in range(self.B):
            p = int(self.pos_h[b])
            if p < 0:
                assert (got[b] == 0).all()
                continue
            lo = max(0, p - self.window + 1) if self.window else 0
            cols = np.arange(lo // self.ps, p // self.ps + 1)
            pages = torch.from_numpy(self.table_h[b, cols]).long().cuda()
            kb, vb = host(self.kp[pages]), host(self.vp[pages])
            table = np.full((1, p // self.ps + 1), -1)
            table[0, cols] = np.arange(len(cols))
            q = host(self.q[b:b + 1])
            ref = oracle.paged_attention([p], q, table, kb, vb, self.window)[0]
            j = np.arange(lo, p + 1)
            keys, vals = kb[table[0, j // self.ps], :, j % self.ps], vb[table[0, j // self.ps], :, j % self.ps]
            kn = np.linalg.norm(keys, axis=-1).max()
            e = (2.0 ** -16 + (self.hd + 32) * U) * np.linalg.norm(q, axis=-1).max() * kn / np.sqrt(self.hd)
            slack = (2 * e + 2.0 ** -16 + (8 + len(j)) * U) * np.abs(vals).max()
            within(got[b], ref, HALF[self.dtype] * np.abs(ref) + slack, f"out of sequence {b} at {p}")


def run_checked(s, status=0):
    before = s.kp.clone(), s.vp.clone()
    s.run()
    s.check(before, status)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,H_kv,hd", [(10, 10, 128), (2, 2, 64), (8, 4, 128), (15, 3, 64), (7, 1, 128), (8, 1, 64),
                                       (9, 1, 128), (32, 2, 64), (17, 1, 128), (40, 1, 128)])
@pytest.mark.parametrize("ps", [16, 64])
def test_decode_heads(dtype, H, H_kv, hd, ps):
    """Every grouping of heads, sequences of one token to a few pages around every boundary, one not running."""
    run_checked(Step(H + hd, [0, 1, ps - 1, -1, ps, 2 * ps + 7, 200, 333], H, H_kv, hd, ps, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 512, 5000])
@pytest.mark.parametrize("ps", [16, 128])
def test_decode_windows(dtype, window, ps):
    """Windows that begin and end anywhere in a page; pages before them are gone from the table (-1)."""
    run_checked(Step(window, [0, 14, 15, 16, 31, 99, 100, 511, 512, 1023, 3000], 4, 2, 128, ps, window=window,
                     dtype=dtype))


def in_two_parts(x):
    """x as two bf16 numbers carry it: what a path on bf16 tensor cores would compute with."""
    upper = torch.from_numpy(x).to(torch.bfloat16).double()
    return (upper + (torch.from_numpy(x) - upper).to(torch.bfloat16).double()).numpy()


@pytest.mark.parametrize("H,H_kv,hd", [(2, 2, 128), (4, 1, 64), (8, 1, 128), (12, 1, 64), (32, 2, 128)])
def test_decode_keeps_fp32(H, H_kv, hd):
    """fp32 to fp32's accuracy, with a bound that two bf16 parts (2^-16) do not keep to. Queries and keys live in the channel
    that turns slowest, so that a score is one product and its error small: the turned query errs by 4 U (cosine and sine
    of an angle below 2^-7, one rounding each), product, scale and the difference to the maximum by another 4 U, so the
    score by e = 8 U of the largest one. A weight errs by e and 8 U of its power, two sums over n keys by n U each,
    three parts' rescaling and joining by at most 8 factors of 5 U in each of the two sums: 2 e + (2 n + 96) U of the sum
    of the terms' magnitudes, and the output by its rounding. The same sums with queries and keys in two parts lie outside."""
    pos = np.array([0, 1, 15, 16, 31, 40, 39, 7])
    s = Step(91, pos, H, H_kv, hd, 16, dtype="f32")
    r = np.random.Generator(np.random.Philox(hd))
    c = hd // 2 - 1
    s.q.zero_()
    s.q[:, :, c] = torch.from_numpy(r.standard_normal((len(pos), H)) * 30).float()
    s.k.zero_()
    s.k[:, :, c] = torch.from_numpy(r.standard_normal((len(pos), H_kv)) * 3).float()
    s.kp[:] = s.kp * (torch.arange(hd, device="cuda") == c) * 3  # (NaN stays where nothing is read)
    s.run()
    torch.cuda.synchronize()
    got, kp, vp = host(s.out), host(s.kp), host(s.vp)
    rejected = False
    for b, p in enumerate(pos):
        q = oracle.rope(host(s.q)[b:b + 1], np.full((1, H), p), 10000.0)[0]
        j = np.arange(p + 1)
        keys, vals = (np.repeat(x[s.table_h[b, j // 16], :, j % 16], H // H_kv, 1) for x in (kp, vp))

        def attend(q, keys):
            x = np.einsum("hd,jhd->hj", q, keys) / np.sqrt(hd)
            w = np.exp(x - x.max(1, keepdims=True))
            return x, w / w.sum(1, keepdims=True)

        x, w = attend(q, keys)
        ref, mass = np.einsum("hj,jhd->hd", w, vals), np.einsum("hj,jhd->hd", w, np.abs(vals))
        delta = 2 * 8 * U * np.abs(x).max(1, keepdims=True) + (2 * len(j) + 96) * U
        tol = U * np.abs(ref) + delta * mass
        within(got[b], ref, tol, f"sequence {b}")
        worse = np.einsum("hj,jhd->hd", attend(in_two_parts(q), in_two_parts(keys))[1], vals)
        rejected |= bool((np.abs(worse - ref) > tol).any())
    assert rejected


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [2**31 - 17, 2**31 - 16, 2**31 - 1])
def test_decode_window_without_a_limit(dtype, window):
    """The largest windows an int holds attend to every position, as window 0 does."""
    s = Step(13, [0, 16, 1000, 4097], 4, 2, 128, 16, dtype=dtype)
    want = s.run().clone()
    s.desc.window = s.window = window
    s.out.zero_()
    run_checked(s)
    assert torch.equal(s.out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("ps,hd", [(16, 128), (32, 64), (256, 128)])
def test_decode_injected(dtype, shared, ps, hd):
    """The memory mixed into the new entry, four or two gate logits per key/value head."""
    run_checked(Step(ps, [5, 0, 700, 511, 512, -3, 64], 6, 3, hd, ps, window=512, inject=True, shared=shared,
                     dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pos", [[20011], [9000, 3, 0, 12345], [4095] * 9, list(range(0, 2600, 13))])
def test_decode_lengths_split_and_joined(dtype, pos):
    """One long sequence (its keys split over many blocks), very uneven ones, many short ones."""
    run_checked(Step(len(pos), pos, 4, 2, 128, 64, dtype=dtype))


def test_decode_many_short_and_one_long_sequence():
    """More sequences than a block has threads (several to a thread in the plan, several rounds of the join), some not
    running, and a long one among them whose parts a whole block joins."""
    r = np.random.Generator(np.random.Philox(77))
    pos = r.integers(-1, 40, 700)
    pos[300] = 30000
    run_checked(Step(77, list(pos), 6, 2, 64, 32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_long_sequences_of_many_heads(dtype):
    """Units of many parts and more heads than the join has blocks."""
    run_checked(Step(78, [4000, 3900, 100], 256, 16, 64, 64, dtype=dtype))


def test_decode_shared_prefix_pages_and_layers_side_by_side():
    """Two sequences whose first pages are the same ones, and two layers (each its own pages and workspace) at once on
    two streams."""
    s = Step(81, [200, 150], 4, 2, 64, 16)
    s.table_h[1, :8] = s.table_h[0, :8]
    s.table.copy_(torch.from_numpy(s.table_h))
    run_checked(s)
    steps = [Step(82, [3000, 70, 512], 4, 2, 128, 32), Step(83, [2500, 9], 8, 1, 128, 16)]
    want = [x.run().clone() for x in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(25):
        for x, st in zip(steps, streams):
            x.out.zero_()
            st.wait_stream(torch.cuda.current_stream())
            x.run(st)
        torch.cuda.synchronize()
        for x, w in zip(steps, want):
            assert torch.equal(x.out, w)


def test_decode_nothing_running():
    """No sequence runs: zeros, nothing written."""
    run_checked(Step(79, [-1] * 5, 4, 2, 128, 16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,H_kv", [(4, 2), (12, 2), (32, 2)])
def test_decode_masked_garbage_and_infinities(dtype, H, H_kv):
    """Infinite and NaN entries outside the attended positions (before the window, behind the last position, other heads'
    and other sequences' rows) change nothing; infinite attended values and keys come through as the formula has it:
    a value times a positive weight is infinite, a key with a score of minus infinity has no weight."""
    s = Step(80, [333, 40], H, H_kv, 128, 16, window=100, dtype=dtype)
    G = H // H_kv
    first = s.run().clone()
    torch.cuda.synchronize()
    lo = 333 - 100 + 1
    page = int(s.table_h[0, lo // 16])
    for bad in (float("inf"), float("-inf"), float("nan"), torch.finfo(TD[dtype]).min):
        s.kp[page, :, : lo % 16] = bad
        s.vp[page, :, : lo % 16] = bad
        last = int(s.table_h[0, 333 // 16])
        s.kp[last, :, 333 % 16 + 1:] = bad
        s.vp[last, :, 333 % 16 + 1:] = bad
        assert torch.equal(s.run(), first), bad
    j = 300
    row = int(s.table_h[0, j // 16]), 0, j % 16
    kept = s.vp[row].clone()
    s.vp[row][5] = float("inf")
    s.vp[row][6] = float("-inf")
    out = s.run()
    torch.cuda.synchronize()
    assert (out[0, :G, 5] == float("inf")).all() and (out[0, :G, 6] == float("-inf")).all()
    keep = torch.arange(128, device="cuda") % 128
    keep = (keep != 5) & (keep != 6)
    assert torch.equal(out[0, :G][:, keep], first[0, :G][:, keep])
    assert torch.equal(out[0, G:], first[0, G:]) and torch.equal(out[1], first[1])
    # a key against which every query of its group scores minus infinity is as good as absent
    s.vp[row].copy_(kept)
    q = oracle.rope(host(s.q)[:1], np.full((1, H), 333), 10000.0)[0]
    c = int(np.argmax(np.abs(q[:G]).min(0)))
    for h in range(G):
        s.q[0, h] = s.q[0, 0]  # one sign for the group
    s.kp[row][c] = float("-inf") if q[0, c] > 0 else float("inf")
    without = s.run().clone()
    s.vp[row].fill_(0)
    torch.cuda.synchronize()
    assert torch.isfinite(without).all()
    assert torch.equal(s.run(), without)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (12, 1), (32, 1)])
@pytest.mark.parametrize("window", [1, 40, 3000])
def test_decode_without_any_weight_is_not_a_number(dtype, H, H_kv, window):
    """Scores that are all minus infinity have no softmax: NaN, as in the formula, from one part or from several; zeros are
    for sequences that do not run."""
    pos = [2999, -1, 50]
    s = Step(84, pos, H, H_kv, 128, 16, window=window, dtype=dtype)
    s.q[:] = s.q[:, :1]
    good = s.run().clone()
    q = oracle.rope(host(s.q)[:1, :1], np.full((1, 1), 2999), 10000.0)[0, 0]
    c = 5
    lo = max(0, 2999 - window + 1)
    j = np.arange(lo, 2999)
    pages = s.table_h[0, j // 16]
    s.kp[pages, :, j % 16, c] = float("-inf") if q[c] > 0 else float("inf")
    # the new key is turned, which makes both channels of the pair infinite: of four ways one points away from q in both
    turn = oracle.rope(np.eye(128)[None, [c, c + 64]], np.full((1, 2), 2999), 10000.0)[0][:, [c, c + 64]]
    i, sign = next((i, z) for i in (0, 1) for z in (1, -1) if (z * turn[i] * q[[c, c + 64]] < 0).all())
    s.k[0, :, c + 64 * i] = float("inf") * sign
    out = s.run()
    torch.cuda.synchronize()
    new = host(s.kp)[s.table_h[0, 2999 // 16], 0, 2999 % 16][[c, c + 64]]
    assert np.isinf(new).all() and (new * q[[c, c + 64]] < 0).all()
    assert out[0].isnan().all() and (out[1] == 0).all() and torch.equal(out[2], good[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (4, 1), (8, 1), (16, 1)])
@pytest.mark.parametrize("gap", [20, 60, 80, 85, 200, 1000])
def test_decode_huge_values_behind_small_weights(dtype, H, H_kv, gap):
    """A value near the type's largest with a weight of e^-gap contributes what the formula says, and nothing (the same
    bits as a zero) where the weight lies below fp32's range. Every query is the same, and one key points against it.
    The weight errs by a factor of at most 1 + 2 e + 2^-16 + (8 + n) U (see the file's head), the sum relative to the sum
    of the terms' magnitudes, and the output by its rounding."""
    s = Step(83, [60], H, H_kv, 128, 16, dtype=dtype)
    s.q[:] = s.q[:, :1]
    rot = oracle.rope(host(s.q)[:, :1], np.full((1, 1), 60), 10000.0)[0, 0]
    page, row = int(s.table_h[0, 33 // 16]), 33 % 16
    s.run()  # stores the new entry
    torch.cuda.synchronize()

    def rows(pool):
        return host(pool)[s.table_h[0, np.arange(61) // 16], 0, np.arange(61) % 16]

    scores = rows(s.kp) @ rot / np.sqrt(128)
    top = np.max(np.delete(scores, 33))
    s.kp[page, 0, row] = torch.from_numpy(rot * ((top - gap) * np.sqrt(128) / (rot @ rot))).to(TD[dtype])
    s.vp[page, 0, row] = 0
    without = s.run().clone()
    s.vp[page, 0, row] = 3e38
    got = s.run()
    torch.cuda.synchronize()
    if gap >= 200:
        assert torch.equal(got, without)
        return
    keys, vals = rows(s.kp), rows(s.vp)
    w = keys @ rot / np.sqrt(128)
    w = np.exp(w - w.max())
    w /= w.sum()
    e = (2.0 ** -16 + 160 * U) * np.linalg.norm(rot) * np.linalg.norm(keys, axis=-1).max() / np.sqrt(128)
    tol = HALF[dtype] * np.abs(w @ vals) + (2 * e + 2.0 ** -16 + (8 + 61) * U) * (w @ np.abs(vals))
    within(host(got)[0], np.broadcast_to(w @ vals, (H, 128)), np.broadcast_to(tol, (H, 128)), f"gap {gap}")


def test_decode_far_positions_and_large_scores():
    """Angles at positions near 2^24 (fp32 cannot hold them), and scores of some hundreds: the running maximum has
    to move, and most weights underflow."""
    run_checked(Step(3, [(1 << 24) + 5, (1 << 24) - 16, 7], 2, 1, 64, 256, window=300))
    for dtype in ("bf16", "f32"):
        run_checked(Step(4, [900, 2000], 4, 2, 128, 16, dtype=dtype, scale=8.0))


def test_decode_rising_scores():
    """Keys whose scores grow along the sequence by some units a page: every tile raises the maximum."""
    s = Step(11, [1999], 2, 1, 128, 16)
    dirn = host(s.q)[0, 0]
    rot = oracle.rope(dirn[None, None], np.array([[1999]]), 10000.0)[0, 0]
    j = torch.arange(1999)
    page = s.table[0].long().cpu()[j // 16].cuda()
    unit = torch.from_numpy(rot / np.linalg.norm(rot)).cuda()
    s.kp[page, 0, (j % 16).cuda()] = (unit * (j.cuda().double() / 10)[:, None]).to(torch.bfloat16)
    run_checked(s)


def test_decode_offsets_beyond_32_bits():
    """Pages at the end of a pool of more than 2^31 elements."""
    s = Step(5, [100, 31], 2, 2, 128, 256)
    big = (1 << 31) // (2 * 256 * 128) + 40
    kp, vp = (torch.empty(big, 2, 256, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = s.kp.shape[0]
    kp[-n:], vp[-n:] = s.kp, s.vp
    s.table_h = np.where(s.table_h >= 0, s.table_h + big - n, -1).astype(np.int32)
    s.table = torch.from_numpy(s.table_h).cuda()
    s.kp, s.vp, s.desc.num_pages = kp, vp, big
    s.run()
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == 0
    s.check_out([0, 1])
    d = desc(H=2, page_size=256, num_pages=big)
    slots = torch.tensor([big * 256 - 1], device="cuda")
    k = normal(generator(1), (1, 2, 128), "bf16")
    mg.maglev_paged_write(d, 1, slots, None, k, k, None, None, None, kp, vp)
    torch.cuda.synchronize()
    assert torch.equal(kp[-1, :, 255], k[0]) and torch.equal(vp[-1, :, 255], k[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_pages_outside_the_pool(dtype):
    """Entries on pages that are not in the pool take no part and are recorded; a position beyond the table is like a
    negative one; a new entry without a page is attended but not stored."""
    s = Step(9, [100, 70, 40], 4, 2, 64, 16, dtype=dtype, spare=0)
    columns = s.table_h.shape[1]
    s.table[0, 2] = 1 << 29
    s.table[0, 3] = -1
    s.table[1, 70 // 16] = -1
    s.pos[2] = columns * 16
    before = s.kp.clone()
    s.run()
    torch.cuda.synchronize()
    assert mg.maglev_device_status() == mg.MAGLEV_ERR_BOUNDS
    got = host(s.out)
    assert (got[2] == 0).all() and np.isfinite(got).all()
    j = np.r_[0:32, 64:101]
    kb, vb = host(s.kp), host(s.vp)
    q = oracle.rope(host(s.q)[:1], np.full((1, 4), 100), 10000.0)[0]
    for h in range(4):
        page = s.table_h[0, j // 16]
        x = kb[page, h // 2, j % 16] @ q[h] / 8.0
        w = np.exp(x - x.max())
        ref = w / w.sum() @ vb[page, h // 2, j % 16]
        within(got[0, h], ref, HALF[dtype] * np.abs(ref) + 2e-3, f"head {h}")
    own = int(s.table_h[0, 100 // 16])
    changed = (s.kp != before) & ~(s.kp.isnan() & before.isnan())
    assert int(changed.any(-1).any(1).sum()) == 1 and bool(changed[own, :, 100 % 16].any())


def test_decode_repeats_bit_for_bit_on_any_stream_and_in_a_graph():
    """Twenty repeats on two streams and replays of a graph all give the first result's bits: the parts are joined in
    the order of the keys."""
    s = Step(21, [5000, 17, 0, 333, -1, 2048], 8, 4, 128, 16, inject=True)
    first = s.run().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i in range(20):
        s.out.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
            s.run()
        torch.cuda.synchronize()
        assert torch.equal(s.out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for _ in range(3):
        s.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out, first)
    # the graph follows positions that change under it (within the entries each sequence has)
    s.pos_h = np.array([100, 16, 0, 0, -1, 900])
    s.pos.copy_(torch.from_numpy(s.pos_h))
    before = s.kp.clone(), s.vp.clone()
    g.replay()
    s.check(before)


def test_calls_follow_their_producers_and_precede_their_consumers():
    """The calls' blocks may be scheduled before the stream's last kernel has ended, but read and write nothing before:
    inputs made by slow kernels just before, outputs read and inputs overwritten just behind, many times over."""
    s = Step(31, [900, 5, 333, 64], 4, 2, 128, 16)
    want = s.run().clone()
    torch.cuda.synchronize()
    slow = torch.randn(3000, 2999, device="cuda")
    q, pos, table = s.q.clone(), s.pos.clone(), s.table.clone()
    kept = []
    for i in range(40):
        zero = (slow @ slow.T)[:1, :1] * 0  # a kernel of some 100 us before each input is there
        s.q.copy_(q + zero.to(q.dtype))
        s.pos.copy_(pos + zero.to(pos.dtype).view(1))
        s.table.copy_(table + zero.to(table.dtype))
        kept.append(s.run().clone())
        s.q.fill_(float("nan"))
        s.pos.fill_(-1)
        s.table.fill_(-1)
        s.out.fill_(0)
    torch.cuda.synchronize()
    for i, o in enumerate(kept):
        assert torch.equal(o, want), i
    # tables, write and step one behind the other, on a stream that waits for another one's work
    T = PageTables(2, 16, 8, 16, 64)
    L = PagedLayerState(T, 2, 64)
    k, q = normal(generator(5), (64, 2, 64), "bf16"), normal(generator(6), (2, 2, 64), "bf16")
    side, outs = torch.cuda.Stream(), []
    for i in range(20):
        T.lengths.zero_()
        T.n_free.fill_(16)
        new = (slow @ slow.T)[:1, :2].to(torch.int64) * 0 + torch.tensor([33, 31], device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            pos, slots = T.step(new.view(2), 64)
            L.write(slots, pos, k, k)
            pos, _ = T.step(torch.ones_like(new.view(2)), 2, 1)
            outs.append(L.step(pos, q, k[:2], k[:2]).clone())
        torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.isfinite(outs[0]).all() and all(torch.equal(o, outs[0]) for o in outs)
    assert mg.maglev_device_status() == 0


def test_chained_calls_read_what_the_call_before_wrote():
    """Tables, write and step one behind the other on a side stream, with nothing between them and with different lengths,
    rows and pages every time: a write that read its slots, positions or rows too early would leave the poison that
    they and the pools held. Outputs and pools equal those of the same calls with a synchronisation after each."""
    B, ps, rows, H, H_kv, hd = 3, 16, 64, 4, 2, 64
    r = np.random.Generator(np.random.Philox(12))
    gen = generator(12)
    rounds = []
    for _ in range(30):
        new = r.multinomial(rows, [0.3, 0.5, 0.2])
        rounds.append((torch.from_numpy(new).cuda(), torch.randperm(20, generator=gen, device="cuda").int(),
                       [normal(gen, (rows, H_kv, hd), "bf16") for _ in range(2)], normal(gen, (B, H, hd), "bf16")))
    ones = torch.ones(B, dtype=torch.int64, device="cuda")
    slow = torch.randn(3000, 2999, device="cuda")
    side = torch.cuda.Stream()

    def run_all(apart):
        T = PageTables(B, ps, 8, 20, rows)
        L = PagedLayerState(T, H, hd, H_kv)
        k, v, q = (torch.empty_like(x) for x in (*rounds[0][2], rounds[0][3]))
        results = []

        def then():
            if apart:
                torch.cuda.synchronize()

        for new, order, (kn, vn), qn in rounds:
            with torch.cuda.stream(side):
                for x in (L.k_pages, L.v_pages, k, v, q):
                    x.fill_(float("nan"))
                T.pos.fill_(-1)
                T.slots.fill_(-1)
                T.lengths.zero_()
                T.n_free.fill_(20)
                T.free_pages.copy_(order)
                T.block_table.fill_(-1)
                zero = (slow @ slow.T)[:1, :1].to(torch.bfloat16) * 0  # some 100 us, so that the calls queue up behind it
                q.copy_(qn + zero)
                v.copy_(vn + zero)
                k.copy_(kn + zero)  # the last kernel before the calls
                then()
                pos, slots = T.step(new, rows)
                then()
                L.write(slots, pos, k, v)
                then()
                prompt = slots.clone(), L.k_pages.clone()
                then()
                # a token each, its rows written over before the step writes them again
                T.step(ones, B, 1)
                then()
                L.write(T.slots[:B], T.pos[:B], v[:B], k[:B])
                then()
                prompt += (L.v_pages.clone(),)
                then()
                out = L.step(T.pos[:B], q, k[:B], v[:B]).clone()
                then()
                results.append((*prompt, out, L.k_pages.clone(), L.v_pages.clone(), T.slots.clone(), T.block_table.clone()))
        torch.cuda.synchronize()
        return results

    for i, (got, want) in enumerate(zip(run_all(False), run_all(True))):
        assert bool((want[0] >= 0).all()) and torch.isfinite(want[3]).all()
        for a, b in zip(got, want):
            assert torch.equal(a.nan_to_num(nan=7.0) if a.is_floating_point() else a,
                               b.nan_to_num(nan=7.0) if b.is_floating_point() else b), i
    assert mg.maglev_device_status() == 0


def test_captured_behind_copies_fills_and_other_streams():
    """In a graph the calls follow memory copies, fills and kernels of a stream that was forked off and joined again;
    replays with changed sources give what separate calls give."""
    s = Step(41, [700, 33, 0, 128], 4, 2, 128, 16)
    s.run()
    torch.cuda.synchronize()
    sources = [(normal(generator(50 + i), s.q.shape, "bf16"), normal(generator(60 + i), s.k.shape, "bf16")) for i in range(3)]
    want = []
    for q, k in sources:
        s.q.copy_(q)
        s.k.copy_(k)
        want.append(s.run().clone())
    torch.cuda.synchronize()
    src_q, src_k, result = sources[0][0].clone(), sources[0][1].clone(), torch.empty_like(s.out)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        s.out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.k.copy_((src_k.float() * 1).to(s.k.dtype))
        s.q.copy_(src_q)
        torch.cuda.current_stream().wait_stream(side)
        s.run()
        result.copy_(s.out)
        s.q.zero_()
    for i in (0, 1, 2, 1):
        src_q.copy_(sources[i][0])
        src_k.copy_(sources[i][1])
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(result, want[i]), i


def test_workspace_may_serve_layers_of_other_shapes():
    """One workspace, sized for the largest and with any content, for layers of different head counts and types in
    turn."""
    steps = [Step(1, [700, 5], 8, 8, 128, 16), Step(2, [9000], 4, 1, 64, 32), Step(3, [64, 65, 2], 6, 2, 128, 16, dtype="f32")]
    ws = max((s.ws for s in steps), key=torch.numel)
    for _ in range(2):
        for s in steps:
            s.ws = ws.fill_(0xff)
            run_checked(s)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,H,H_kv,window,inject", [("bf16", 10, 10, 512, True), ("bf16", 8, 2, 0, False),
                                                        ("f32", 4, 2, 100, True)])
def test_serving_run(dtype, H, H_kv, window, inject):
    """Prompts, decode steps, sequences that end and new ones that take their pages, in two layers over one table:
    every output against the oracle over its own copy of the whole history of each sequence."""
    B, hd, ps, d_mem = 6, 128, 16, 64
    r = np.random.Generator(np.random.Philox(H))
    gen = generator(H)
    T = PageTables(B, ps, 64, 120, 2048)
    L = [PagedLayerState(T, H, hd, H_kv, window, d_mem, dtype, inject) for _ in range(2)]
    gates = [torch.rand(4, H_kv, generator=gen, device="cuda") * 4 - 2 for _ in L] if inject else [None] * 2
    w_mk, w_mv = (normal(gen, (H_kv * hd, d_mem), dtype) / 8 for _ in range(2))
    lens, hist = np.zeros(B, dtype=np.int64), [[[] for _ in range(B)] for _ in L]  # stored entries
    refused = 0
    for it in range(14):
        new = np.where(lens > 0, 1, r.integers(1, 400, B))
        new[(r.random(B) < 0.2) & (lens > 0)] = -1
        new_d = torch.from_numpy(new).cuda()
        decode = (new == 1) & (lens > 0)
        prompts = np.where(decode, 0, new)
        # prompts and ends first, packed rows
        n = int(np.maximum(prompts, 0).sum())
        pos, slots = T.step(torch.from_numpy(prompts).cuda(), n + 3)
        torch.cuda.synchronize()
        seq = T.lengths.cpu().numpy()
        cu = T.cu_tokens.cpu().numpy()
        x = [normal(gen, (n + 3, H_kv, hd), dtype) for _ in range(4)]
        for l, layer in enumerate(L):
            layer.write(slots, pos, x[0], x[1], x[2] if inject else None, x[3] if inject else None, gates[l])
        torch.cuda.synchronize()
        for b in range(B):
            if prompts[b] < 0:
                for l in range(2):
                    hist[l][b] = []
            elif prompts[b] > 0:
                if seq[b] != prompts[b]:
                    refused += 1
                    continue
                rows = slice(int(cu[b]), int(cu[b + 1]))
                np.testing.assert_array_equal(pos[rows].cpu().numpy(), np.arange(prompts[b]))
                h = [host(y[rows]) for y in x]
                for l in range(2):
                    kb, vb = oracle.paged_entries(np.arange(prompts[b]), h[0], h[1], h[2] if inject else None,
                                                  h[3] if inject else None, host(gates[l]) if inject else None)
                    hist[l][b] = [(kb[i], vb[i]) for i in range(len(kb))]
        lens = seq
        # then one token of every running sequence
        pos, slots = T.step(torch.from_numpy((lens > 0).astype(np.int64)).cuda(), B, 1)
        q, k, v = normal(gen, (B, H, hd), dtype), normal(gen, (B, H_kv, hd), dtype), normal(gen, (B, H_kv, hd), dtype)
        m = normal(gen, (B, d_mem), dtype)
        for l, layer in enumerate(L):
            if inject:
                layer.mem_project(pos, m, w_mk, w_mv)
            layer.step(pos, q, k, v, gates[l])
        torch.cuda.synchronize()
        assert mg.maglev_device_status() == 0
        p_h, lens2 = pos.cpu().numpy(), T.lengths.cpu().numpy()
        krec, vrec = (oracle.decode_mem_project(np.maximum(p_h, 0), host(m), host(w_mk), host(w_mv), H_kv)
                      if inject else (None, None))
        for l, layer in enumerate(L):
            out = host(layer.out)
            for b in range(B):
                if p_h[b] < 0:
                    assert (out[b] == 0).all() and lens2[b] == lens[b]
                    continue
                assert p_h[b] == lens[b] == len(hist[l][b]) and lens2[b] == lens[b] + 1
                rec = (krec[b:b + 1], vrec[b:b + 1]) if inject else (None, None)
                kb, vb = oracle.rope(host(k)[b:b + 1], np.full((1, H_kv), p_h[b]), 10000.0), host(v)[b:b + 1]
                if inject:
                    g = oracle.gate(host(gates[l]))[:, None, :, None]
                    kb, vb = g[0] * kb + g[1] * rec[0], g[2] * vb + g[3] * rec[1]
                hist[l][b].append((kb[0], vb[0]))
                ks, vs = (np.stack([e[i] for e in hist[l][b]], 1)[None] for i in range(2))  # one page of all entries
                ref = oracle.paged_attention([p_h[b]], host(q)[b:b + 1], np.zeros((1, 1), dtype=int), ks, vs, window)[0]
                # stored entries, krec and vrec are off by a rounding each (2^-8 or 2^-24 of a value below ~6 gates):
                # scores move by at most that of |q| |k| / sqrt(hd), of which a quarter is far beyond what signs leave
                h = HALF[dtype]
                e = 0.25 * 2 * h * np.linalg.norm(host(q)[b], axis=-1).max() * np.linalg.norm(ks, axis=-1).max() / np.sqrt(hd)
                tol = h * np.abs(ref) + (2 * min(e, 0.5) + 2 * h + 1e-5) * np.abs(vs).max()
                within(out[b], ref, tol, f"step {it} layer {l} sequence {b}")
        lens = lens2
    assert refused < 14 * B


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inject", [False, True])
@pytest.mark.parametrize("B,T,H,hd,W", [(1, 77, 1, 64, 32), (2, 45, 3, 128, 20), (3, 128, 10, 128, 512)])
def test_a_prompts_entries_move_from_the_forward_to_pages(dtype, inject, B, T, H, hd, W):
    """The forward of the dense layer, its entries (also where a third of `saved` is padded to 256 bytes) as they are into
    pages, and a step behind them: the entries against the oracle's, the pages bit for bit, the step against the oracle
    over the pages as they are."""
    from sliding_window_recurrent_b200.layer import InjectedSWALayer
    d_mem, ps, gen = 64, 16, generator(T)
    F = InjectedSWALayer(B, T, H, hd, d_mem, W, dtype, inject)
    q, k, v = (normal(gen, (B, T, H, hd), dtype) for _ in range(3))
    gates = torch.rand(4, H, generator=gen, device="cuda") * 4 - 2 if inject else None
    m = normal(gen, (B, T, d_mem), dtype)
    w_mk, w_mv = (normal(gen, (H * hd, d_mem), dtype) / 8 for _ in range(2))
    F.forward(q, k, v, gates, m if inject else None, w_mk, w_mv)
    kb, vb = F.entries()
    assert kb.shape == vb.shape == (B, T, H, hd) and kb.data_ptr() % 256 == vb.data_ptr() % 256 == F.saved.data_ptr() % 256
    torch.cuda.synchronize()
    for b in range(B):
        Rk, Rv = (host(x)[b].reshape(T, H, hd) if inject else None for x in (F.R_k, F.R_v))
        g = host(gates) if inject else None
        ref_k, ref_v = oracle.paged_entries(np.arange(T), host(k)[b], host(v)[b], Rk, Rv, g)
        tk, tv = entry_bound(None, host(k)[b], host(v)[b], Rk, Rv, g, ref_k, ref_v, dtype)
        within(host(kb)[b], ref_k, tk, "k_bar")
        within(host(vb)[b], ref_v, tv, "v_bar")
    tabs = PageTables(B, ps, -(-T // ps) + 1, B * (-(-T // ps) + 1), B * T)
    L = PagedLayerState(tabs, H, hd, H, W, d_mem, dtype, inject)
    pos, slots = tabs.step(torch.full((B,), T, device="cuda"), B * T, T)
    L.write(slots, None, kb.reshape(B * T, H, hd), vb.reshape(B * T, H, hd))
    page, row = slots // ps, slots % ps
    assert torch.equal(L.k_pages[page, :, row], kb.reshape(B * T, H, hd))
    assert torch.equal(L.v_pages[page, :, row], vb.reshape(B * T, H, hd))
    pos, _ = tabs.step(torch.ones(B, dtype=torch.int64, device="cuda"), B, 1)
    if inject:
        L.mem_project(pos, m[:, 0].contiguous(), w_mk, w_mv)
    L.step(pos, q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), gates)
    torch.cuda.synchronize()
    kp, vp, table = host(L.k_pages), host(L.v_pages), tabs.block_table.cpu().numpy()
    ref = oracle.paged_attention([T] * B, host(q)[:, 0], table, kp, vp, W)
    j = np.arange(max(0, T - W + 1), T + 1)
    keys, vals = (np.stack([x[table[b, j // ps], :, j % ps] for b in range(B)]) for x in (kp, vp))
    e = (2.0 ** -16 + (hd + 32) * U) * np.linalg.norm(host(q)[:, 0], axis=-1).max() * np.linalg.norm(keys, axis=-1).max() / np.sqrt(hd)
    within(host(L.out), ref, HALF[dtype] * np.abs(ref) + (2 * e + 2.0 ** -16 + (8 + len(j)) * U) * np.abs(vals).max(), "out")
    assert mg.maglev_device_status() == 0


def test_pages_behind_a_window_and_shared_ones_are_given_back_once():
    """What the tables leave to the caller: pages that a window has passed go on the stack and their columns to -1, and a
    row that shares its first pages finishes with those columns at -1. Outputs are those of a cache that keeps every page,
    each page is on the stack or in one row's columns at any time, and at the end all are back."""
    B, H, hd, ps, W, pool = 3, 2, 64, 16, 20, 30
    gen = generator(95)
    one = torch.ones(B, dtype=torch.int64, device="cuda")
    caches = []
    for _ in range(2):
        T = PageTables(B, ps, 16, pool, 128)
        L = PagedLayerState(T, H, hd, window=W)
        caches.append((T, L))
    k0, v0 = normal(gen, (128, H, hd), "bf16"), normal(gen, (128, H, hd), "bf16")
    for T, L in caches:
        pos, slots = T.step(torch.tensor([40, 5, 0], device="cuda"), 45)
        L.write(slots, pos, k0[:45], v0[:45])
    # the third sequence continues the first one's first 32 tokens: two pages of its own column go back for the shared ones
    for T, L in caches:
        pos, slots = T.step(torch.tensor([0, 0, 33], device="cuda"), 33)
        own = T.block_table[2, :2].clone()
        n = int(T.n_free)
        T.free_pages[n:n + 2] = own
        T.n_free += 2
        T.block_table[2, :2] = T.block_table[0, :2]
        L.write(slots[32:], pos[32:], k0[32:33], v0[32:33])
    for step in range(60):
        q, k, v = (normal(gen, (B, H, hd), "bf16") for _ in range(3))
        outs = []
        for i, (T, L) in enumerate(caches):
            pos, _ = T.step(one, B, 1)
            outs.append(L.step(pos, q, k, v).clone())
            if i == 0:  # give back what every later query is past; shared pages with their last holder
                table, n = T.block_table.cpu().numpy(), int(T.n_free)
                for b, p in enumerate(pos.tolist()):
                    for c in range(max(0, p + 1 - W + 1) // ps):
                        page = int(table[b, c])
                        if page >= 0:
                            T.block_table[b, c] = table[b, c] = -1
                            if not (table[:, :16] == page).any():
                                T.free_pages[n] = page
                                n += 1
                T.n_free.fill_(n)
                held = [int(x) for b in range(B) for x in table[b, :-(-int(T.lengths[b]) // ps)] if x >= 0]
                assert sorted(set(held) | set(T.free_pages[:n].tolist())) == list(range(pool))
                assert len(set(held)) + n == pool
        assert torch.isfinite(outs[0]).all() and torch.equal(*outs), step
    T, L = caches[0]
    T.step(-one, 0)
    torch.cuda.synchronize()
    assert int(T.n_free) == pool and sorted(T.free_pages.tolist()) == list(range(pool))
    T, L = caches[1]  # keeps every page: the shared columns are taken out by hand before the end
    T.block_table[2, :2] = -1
    T.step(-one, 0)
    torch.cuda.synchronize()
    assert int(T.n_free) == pool and sorted(T.free_pages.tolist()) == list(range(pool))
    assert mg.maglev_device_status() == 0


def test_step_captured_in_a_graph_runs_on():
    """A whole serving step (tables in place, two layers) in one graph: replays continue the sequences by a token each,
    as separate calls do."""
    def build():
        T = PageTables(3, 16, 8, 20, 64)
        L = [PagedLayerState(T, 4, 64, 2) for _ in range(2)]
        for x in L:
            x.k_pages.zero_()
            x.v_pages.zero_()
        return T, L

    gen = generator(91)
    q, k, v = normal(gen, (3, 4, 64), "bf16"), normal(gen, (3, 2, 64), "bf16"), normal(gen, (3, 2, 64), "bf16")
    new = torch.tensor([1, 0, 1], device="cuda")
    results = []
    for captured in (False, True):
        T, L = build()
        T.step(torch.tensor([20, 5, 0], device="cuda"), 64)
        for x in L:
            x.write(T.slots, T.pos, k.repeat(22, 1, 1)[:64], v.repeat(22, 1, 1)[:64])

        def step():
            pos, _ = T.step(new, 3, 1)
            for x in L:
                x.step(pos, q, k, v)

        if captured:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            for _ in range(30):
                g.replay()
        else:
            for _ in range(30):
                step()
        torch.cuda.synchronize()
        assert T.lengths.tolist() == [50, 5, 30] and int(T.n_free) == 20 - 4 - 1 - 2
        results.append([x.out.clone() for x in L] + [T.block_table.clone(), L[1].k_pages.clone()])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert mg.maglev_device_status() == 0
    with pytest.raises(ValueError):
        T.step(new, 65)


def test_owners_refuse_tensors_the_library_would_misread():
    """The classes check what the library, which sees addresses, cannot: shapes, types, strides and the device."""
    T = PageTables(2, 16, 4, 8, 32)
    L = PagedLayerState(T, 4, 64, 2)
    new = torch.ones(2, dtype=torch.int64, device="cuda")
    for bad in (new.int(), new.cpu(), torch.ones(3, dtype=torch.int64, device="cuda"), torch.ones(4, dtype=torch.int64, device="cuda")[::2]):
        with pytest.raises(ValueError, match="new_len"):
            T.step(bad, 2)
    pos, slots = T.step(new, 2)
    k = normal(generator(1), (2, 2, 64), "bf16")
    with pytest.raises(ValueError, match="k must"):
        L.write(slots, pos, k[:1], k)
    with pytest.raises(ValueError, match="v must"):
        L.write(slots, pos, k, k.float())
    with pytest.raises(ValueError, match="pos must"):
        L.write(slots, pos[:1], k, k)
    q = normal(generator(1), (2, 4, 64), "bf16")
    with pytest.raises(ValueError, match="q must"):
        L.step(pos, q[:, :2], k, k)
    with pytest.raises(ValueError, match="k must"):
        L.step(pos, q, q[:, ::2], k)
    J = PagedLayerState(T, 4, 64, 2, inject=True, d_mem=16)
    with pytest.raises(ValueError, match="gates"):
        J.step(pos, q, k, k)
    with pytest.raises(ValueError, match="R_k"):
        J.write(slots, pos, k, k, gates=torch.zeros(4, 2, device="cuda"))
