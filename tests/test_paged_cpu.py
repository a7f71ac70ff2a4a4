"""The paged cache without a GPU: what its oracle is pinned to, and what the
library refuses before any launch."""
import numpy as np
import pytest

import oracle
from sliding_window_recurrent_b200 import build as _build

_build.build(quiet=True)

import sliding_window_recurrent_b200 as mg  # noqa: E402

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first


def rng(seed):
    return np.random.Generator(np.random.Philox(seed))


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("seed", range(4))
def test_page_tables_conserve_pages(seed):
    """Random serving steps: no page is ever lost, shared or handed out twice, every live position has a slot of its
    own, lengths grow only for requests that were served, and refusals happen only for want of pages or columns."""
    r = rng(seed)
    B, ps, columns, pool = 7, 4, 6, 20
    table, free = np.full((B, columns), -1, dtype=np.int32), list(range(pool))
    lens = np.zeros(B, dtype=np.int64)
    for _ in range(60):
        new = r.integers(0, 9, B)
        new[r.random(B) < 0.2] = -1
        pad = 8 if r.random() < 0.5 else 0
        n_tokens = B * 8 if pad else int(np.maximum(new, 0).sum())
        got = oracle.page_tables(lens, new, n_tokens, pad, ps, free, table)
        held = [list(got["block_table"][b, :-(-int(got["seq_len"][b]) // ps)]) for b in range(B)]
        flat = [int(x) for h in held for x in h] + got["free"]
        assert sorted(flat) == list(range(pool))
        s = got["slots"][got["slots"] >= 0]
        assert len(set(s.tolist())) == len(s)
        assert ((got["pos"] >= 0) == (got["slots"] >= 0)).all()
        for b in range(B):
            at = b * pad if pad else got["cu_tokens"][b]
            n = max(int(new[b]), 0)
            served = got["seq_len"][b] == lens[b] + n
            if new[b] < 0:
                assert got["seq_len"][b] == 0
            elif n and served:
                np.testing.assert_array_equal(got["pos"][at:at + n], np.arange(lens[b], lens[b] + n))
            elif n:
                assert got["seq_len"][b] == lens[b] and (got["slots"][at:at + n] == -1).all()
        table, free, lens = got["block_table"], got["free"], got["seq_len"]


def test_page_tables_order_and_refusals():
    """Hand-worked: finished pages are reused first (last returned first), a request that does not fit is passed
    over together with later ones that need pages, one that stays inside its page is served all the same."""
    table = np.array([[5, 6, -1], [7, -1, -1], [8, 9, 10], [4, -1, -1]], dtype=np.int32)
    got = oracle.page_tables([8, 3, 9, 2], [9, 1, -1, 5], 15, 0, 4, [0], table)
    # stack after the return: 0, 8, 9, 10; request 0 is over its row, 1 stays inside its page, 3 takes one page
    np.testing.assert_array_equal(got["block_table"], [[5, 6, -1], [7, -1, -1], [8, 9, 10], [4, 10, -1]])
    assert got["free"] == [0, 8, 9] and got["seq_len"].tolist() == [8, 4, 0, 7]
    assert got["cu_tokens"].tolist() == [0, 9, 10, 10, 15]
    assert got["slots"].tolist() == [-1] * 9 + [7 * 4 + 3] + [4 * 4 + 2, 4 * 4 + 3, 40, 41, 42]
    got = oracle.page_tables([0, 4, 4], [8, 1, 0], 9, 0, 4, [3], np.full((3, 2), 1, dtype=np.int32))
    assert got["seq_len"].tolist() == [0, 4, 4] and got["free"] == [3]


def test_page_tables_take_nothing_from_a_row_of_a_bad_length():
    """Hand-worked: a finished row whose length lies outside it puts nothing on the stack."""
    table = np.array([[2, 3, 4, -1], [0, 10, 11, 12], [5, 6, 7, 8]])
    got = oracle.page_tables([65, -1, 64], [-1] * 3, 0, 0, 16, [13], table)
    assert got["free"] == [13, 5, 6, 7, 8] and got["seq_len"].tolist() == [0] * 3


def test_page_tables_give_back_only_pages():
    """Hand-worked: first columns without a page (negative: given back before) and rows whose length lies outside them put
    nothing on the stack, another number outside the pool puts -1 there."""
    table = np.array([[-1, -1, 5, 6], [-5, -1, -1, -1], [1, 30, -1, -1], [2, 3, 4, -1], [0, 10, 11, 12]])
    got = oracle.page_tables([60, 64, 30, 65, -1], [-1] * 5, 0, 0, 16, [13], table, num_pages=30)
    assert got["free"] == [13, 5, 6, 1, -1] and got["seq_len"].tolist() == [0] * 5
    np.testing.assert_array_equal(got["block_table"], table)


def _paged_from_forward(seed, T, H, hd, W, ps, inject):
    """A forward pass's entries of one sequence in scattered pages, and what went into it."""
    r = rng(seed)
    q, k, v = (r.standard_normal((1, T, H, hd)) for _ in range(3))
    R_k, R_v = (r.standard_normal((1, T, H * hd)) if inject else None for _ in range(2))
    gates = r.uniform(-2, 2, (4, H)) if inject else None
    f = oracle.inject_swa_forward(q, k, v, R_k, R_v, gates, W, inject=inject)
    return q, k, v, R_k, R_v, gates, f


@pytest.mark.parametrize("inject", [False, True])
@pytest.mark.parametrize("T,W", [(1, 4), (9, 4), (16, 16), (21, 100), (21, 1)])
def test_oracle_write_and_attention_equal_the_forward(T, W, inject):
    """Entries written through slots are the forward's, and the query of each row attending over the pages gives
    the forward's row, whatever lies in the rest of the pages."""
    H, hd, ps = 2, 8, 4
    q, k, v, R_k, R_v, gates, f = _paged_from_forward(3, T, H, hd, W, ps, inject)
    npages = -(-T // ps) + 2
    table = rng(4).permutation(npages)[None, :-(-T // ps)].astype(np.int32)
    j = np.arange(T)
    slots = table[0, j // ps] * ps + j % ps
    rk = None if R_k is None else R_k.reshape(T, H, hd)
    rv = None if R_v is None else R_v.reshape(T, H, hd)
    kb, vb = oracle.paged_entries(j, k[0], v[0], rk, rv, gates)
    np.testing.assert_allclose(kb, f["k_bar"][0], rtol=0, atol=1e-12)
    np.testing.assert_allclose(vb, f["v_bar"][0], rtol=0, atol=1e-12)
    kp, vp = oracle.paged_write(slots, kb, vb, np.full((npages, H, ps, hd), np.nan), np.full((npages, H, ps, hd), np.nan))
    for t in range(T):
        out = oracle.paged_attention([t], q[:, t], table, kp, vp, W)
        np.testing.assert_allclose(out[0], f["out"][0, t], rtol=0, atol=1e-12)


def test_oracle_decode_equals_the_ring_step():
    """The same entries in a ring and in pages: the two steps agree, first lap and later ones."""
    r = rng(5)
    B, H, hd, W, ps = 3, 2, 8, 8, 4
    pos = np.array([3, 7, 29])
    columns = 8
    kr, vr = r.standard_normal((2, B, H, W, hd))
    table = r.permutation(B * columns).reshape(B, columns).astype(np.int32)
    kp, vp = np.full((2, B * columns, H, ps, hd), np.nan)
    for b in range(B):
        for j in range(max(0, pos[b] - W + 1), pos[b]):
            kp[table[b, j // ps], :, j % ps] = kr[b, :, j % W]
            vp[table[b, j // ps], :, j % ps] = vr[b, :, j % W]
    x = [r.standard_normal((B, H, hd)) for _ in range(5)]
    gates = r.uniform(-2, 2, (4, H))
    ring, _, _ = oracle.decode_step(pos, *x, gates, kr, vr)
    paged, kp2, _ = oracle.paged_decode_step(pos, *x, gates, table, kp, vp, W)
    np.testing.assert_allclose(paged, ring, rtol=0, atol=1e-12)
    assert np.isfinite(kp2[table[2, 29 // ps], :, 29 % ps]).all()


def test_oracle_grouped_heads_equal_repeated_ones():
    r = rng(6)
    kp, vp = r.standard_normal((2, 5, 2, 4, 8))
    q = r.standard_normal((1, 6, 8))
    table = np.array([[4, 1, 0]], dtype=np.int32)
    a = oracle.paged_attention([10], q, table, kp, vp)
    b = oracle.paged_attention([10], q, table, np.repeat(kp, 3, 1), np.repeat(vp, 3, 1))
    np.testing.assert_array_equal(a, b)
    assert (oracle.paged_attention([-1], q, table, kp, vp) == 0).all()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def desc(**kw):
    base = dict(B=2, H=4, H_kv=2, hd=64, page_size=16, max_pages=8, num_pages=32, window=0, rope_base=10000.0,
                rms_eps=1e-6, inject=0, dtype=mg.MAGLEV_BF16, shared_kv_gates=0)
    base.update(kw)
    return mg.PagedDesc(**base)


def tables(d, n_tokens=4, pad=0, **kw):
    a = dict(ctx_len=FAKE, new_len=FAKE, free_pages=FAKE, n_free=FAKE, block_table=FAKE, seq_len=FAKE, n_free_out=FAKE,
             cu_tokens=FAKE, pos=FAKE, slots=FAKE, workspace=FAKE)
    a.update(kw)
    mg.maglev_page_tables(d, a["ctx_len"], a["new_len"], n_tokens, pad, a["free_pages"], a["n_free"], a["block_table"],
                          a["seq_len"], a["n_free_out"], a["cu_tokens"], a["pos"], a["slots"], a["workspace"], stream=0)


def write(d, n=4, **kw):
    a = dict(slots=FAKE, pos=FAKE, k=FAKE, v=FAKE, R_k=FAKE, R_v=FAKE, gates=FAKE, k_pages=FAKE, v_pages=FAKE)
    a.update(kw)
    mg.maglev_paged_write(d, n, *a.values(), stream=0)


def step(d, **kw):
    a = dict(pos=FAKE, q=FAKE, k=FAKE, v=FAKE, krec=FAKE, vrec=FAKE, gates=FAKE, block_table=FAKE, k_pages=FAKE,
             v_pages=FAKE, out=FAKE, workspace=FAKE)
    a.update(kw)
    mg.maglev_paged_decode_step(d, *a.values(), stream=0)


def refused(call, status, text, *args, **kw):
    with pytest.raises(mg.MaglevError) as e:
        call(*args, **kw)
    assert e.value.status == status and text in str(e.value), str(e.value)


INV, UNS = mg.MAGLEV_ERR_INVALID_ARG, mg.MAGLEV_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [tables, write, step])
@pytest.mark.parametrize("bad,status,text", [
    (dict(B=-1), INV, "B must"), (dict(page_size=24), UNS, "page_size"), (dict(page_size=8), UNS, "page_size"),
    (dict(page_size=512), UNS, "page_size"), (dict(page_size=0), UNS, "page_size"), (dict(max_pages=0), INV, "max_pages"),
    (dict(num_pages=0), INV, "num_pages"), (dict(B=1 << 16, max_pages=1 << 15), UNS, "2^31")])
def test_every_call_refuses_bad_page_sizes(call, bad, status, text):
    refused(call, status, text, desc(**bad))


@pytest.mark.parametrize("call", [write, step])
@pytest.mark.parametrize("bad,status,text", [
    (dict(H=0), INV, "H"), (dict(H_kv=0), INV, "H_kv"), (dict(H_kv=3), INV, "multiple"), (dict(hd=96), UNS, "head dim"),
    (dict(window=-1), INV, "window"), (dict(dtype=7), INV, "dtype"), (dict(rope_base=1.0), INV, "rope_base"),
    (dict(rms_eps=float("nan")), INV, "rms_eps"), (dict(H=1 << 17, H_kv=1), UNS, "H must")])
def test_write_and_step_refuse_bad_layers(call, bad, status, text):
    refused(call, status, text, desc(**bad))


def test_pointers_are_checked():
    """NULL and misaligned pointers are refused by name: 16 bytes for data, the type's size for index arrays."""
    for name, size in (("ctx_len", 8), ("new_len", 8), ("free_pages", 4), ("n_free", 4), ("block_table", 4),
                       ("seq_len", 8), ("n_free_out", 4), ("cu_tokens", 8), ("pos", 8), ("slots", 8), ("workspace", 16)):
        refused(tables, INV, name, desc(), **{name: None})
        refused(tables, INV, f"{name} must be {size}-byte aligned", desc(), **{name: FAKE + size // 2})
        if size < 16:  # the type's alignment will do: the next refusal is another one
            refused(tables, INV, "workspace", desc(), **{name: FAKE + size, "workspace": None})
    for name, size in (("slots", 8), ("pos", 8), ("k", 16), ("v", 16), ("k_pages", 16), ("v_pages", 16)):
        if name != "pos":
            refused(write, INV, name, desc(), **{name: None})
        refused(write, INV, f"{name} must be {size}-byte aligned", desc(), **{name: FAKE + size // 2})
    for name, size in (("pos", 8), ("q", 16), ("k", 16), ("v", 16), ("block_table", 4), ("k_pages", 16), ("v_pages", 16),
                       ("out", 16), ("workspace", 16)):
        refused(step, INV, name, desc(), **{name: None})
        refused(step, INV, f"{name} must be {size}-byte aligned", desc(), **{name: FAKE + size // 2})
    for name, arg in (("R_k", "R_k"), ("R_v", "R_v"), ("gate_logits", "gates")):
        refused(write, INV, name, desc(inject=1), **{arg: None})
    for name, arg in (("krec_rot", "krec"), ("vrec", "vrec"), ("gate_logits", "gates")):
        refused(step, INV, name, desc(inject=1), **{arg: None})


def test_counts_are_checked():
    refused(tables, INV, "n_tokens", desc(), n_tokens=-1)
    refused(tables, INV, "pad", desc(), pad=-1)
    refused(tables, INV, "B * pad", desc(), n_tokens=5, pad=2)
    refused(tables, UNS, "n_tokens", desc(), n_tokens=(1 << 31) + 1)
    refused(write, INV, "n must", desc(), n=-1)
    refused(write, UNS, "n must", desc(), n=(1 << 31) + 1)
    refused(write, INV, "injection", desc(inject=1), pos=None)


def test_empty_problems_enqueue_nothing():
    tables(desc(B=0), n_tokens=0)
    write(desc(), n=0)
    step(desc(B=0))


def test_workspace_sizes():
    assert mg.maglev_page_tables_workspace_bytes(desc()) > 0
    assert mg.maglev_page_tables_workspace_bytes(desc(page_size=20)) == 0
    assert mg.maglev_paged_decode_workspace_bytes(desc(hd=96)) == 0


@pytest.mark.parametrize("call", [tables, write, step])
@pytest.mark.parametrize("B", [(1 << 30) + 1, 2**31 - 1])
def test_more_sequences_than_32_bit_loops_can_step_over_are_refused(call, B):
    """The kernels step over the sequences in strides of up to 2048 in int: near 2^31 the last step would wrap."""
    refused(call, UNS, "2^30", desc(B=B, max_pages=1))
    assert mg.maglev_page_tables_workspace_bytes(desc(B=B, max_pages=1)) == 0
    assert mg.maglev_paged_decode_workspace_bytes(desc(B=B, max_pages=1)) == 0
    assert mg.maglev_page_tables_workspace_bytes(desc(B=1 << 30, max_pages=1)) > 0


def test_dependent_kernels_promise_nothing_about_their_inputs():
    """A kernel that may be scheduled while its inputs are still being written must not declare them __restrict__:
    const __restrict__ says that nothing writes them while it runs, and lets the compiler read them through the
    read-only path and before the wait."""
    import os
    import re
    seen = 0
    for path in _build.sources():
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        if "launch_dependent(" in text:
            seen += 1
            assert "__restrict__" not in text and "__ldg(" not in text, os.path.basename(path)
    assert seen == 2


def test_the_join_reads_positions_past_l1():
    """What the join reads before it has waited for the first kernel is visible in L2 only (that kernel has waited for
    whatever wrote it): every position it reads has to come from there."""
    import os
    import re
    with open(os.path.join(_build.CSRC, "paged_decode.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.index("paged_join_kernel(PagedShape"):text.index("int units_of(")]
    assert "wait_for_last()" in body and "a.pos[" not in body
    reads = re.findall(r"\b(?:form_plan|sequence|position)\b(<\w+>)?\(", body)
    assert len(reads) == 4 and set(reads) == {"<true>"}


# ---------------------------------------------------------------------------
# the owner classes, with stand-ins for device tensors
# ---------------------------------------------------------------------------
class Placed:
    """What the owners look at of a dense tensor on a GPU; it has no memory."""

    def __init__(self, shape, dtype, index=0):
        import torch
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, torch.device("cuda", index), True

    def numel(self):
        return int(np.prod(self.shape))

    def stride(self):
        return ()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("passed to the library")


@pytest.fixture
def owners(monkeypatch):
    """A table and a layer whose (host) buffers are taken for ones on cuda:0, the current device."""
    torch = pytest.importorskip("torch")
    from sliding_window_recurrent_b200.layer import PagedLayerState, PageTables
    T = PageTables(2, 16, 4, 8, 32, device="cpu")
    L = PagedLayerState(T, 4, 64, 2, d_mem=16, inject=True, device="cpu")
    T.device = L.device = torch.device("cuda", 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return torch, T, L


def paged_arguments(torch):
    i64, bf = torch.int64, torch.bfloat16
    return (dict(new_len=((2,), i64)),
            dict(slots=((2,), i64), pos=((2,), i64), k=((2, 2, 64), bf), v=((2, 2, 64), bf), R_k=((2, 2, 64), bf),
                 R_v=((2, 2, 64), bf), gates=((4, 2), torch.float32)),
            dict(pos=((2,), i64), q=((2, 4, 64), bf), k=((2, 2, 64), bf), v=((2, 2, 64), bf), gates=((4, 2), torch.float32)))


@pytest.mark.parametrize("call", [0, 1, 2])
def test_owners_refuse_tensors_on_another_device(owners, call):
    """Each argument in turn on a second GPU: its address means nothing to a kernel on the first."""
    torch, T, L = owners
    fn = (T.step, L.write, L.step)[call]
    spec = paged_arguments(torch)[call]
    for name in spec:
        with pytest.raises(ValueError, match=f"{name} must.*cuda:0"):
            fn(**{n: Placed(*x, index=int(n == name)) for n, x in spec.items()})


def test_owners_refuse_another_current_device(owners, monkeypatch):
    """The library launches on the current device: its owners' buffers have to lie there."""
    torch, T, L = owners
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for fn, spec in zip((T.step, L.write, L.step), paged_arguments(torch)):
        with pytest.raises(ValueError, match="not the current device"):
            fn(**{n: Placed(*x) for n, x in spec.items()})


def test_a_layer_lies_where_its_tables_do(owners):
    torch, T, _ = owners
    from sliding_window_recurrent_b200.layer import PagedLayerState
    with pytest.raises(ValueError, match="its tables lie on cuda:0"):
        PagedLayerState(T, 4, 64, 2, device="cpu")


def test_mem_project_refuses_what_the_library_would_misread(owners):
    """Each argument too small, of another type and on another device: the library would read past its end."""
    torch, T, L = owners
    bf = torch.bfloat16
    good = dict(pos=((2,), torch.int64), m_prev=((2, 16), bf), w_mk=((128, 16), bf), w_mv=((128, 16), bf))
    for name, (shape, dtype) in good.items():
        for bad in (Placed((shape[0] - 1,) + shape[1:], dtype), Placed(shape, torch.float32), Placed(shape, dtype, 1), None):
            with pytest.raises(ValueError, match=f"{name} must"):
                L.mem_project(**{**{n: Placed(*x) for n, x in good.items()}, name: bad})
