"""Torch-allocated buffers around the C ABI (device memory and streams only).

InjectedSWALayer owns the outputs, saved activations, gradients and scratch
of one layer and calls the library entry points; it performs no arithmetic.
"""
from __future__ import annotations

import torch

from . import (DecodeDesc, MAGLEV_BF16, MAGLEV_BWD_PREPARED, MAGLEV_DR_WRITE, MAGLEV_F32, PagedDesc, SwaDesc,
               maglev_consistency_loss, maglev_consistency_loss_prepare_bwd, maglev_consistency_workspace_bytes, maglev_decode_mem_project, maglev_decode_step,
               maglev_decode_workspace_bytes,
               maglev_inject_swa_bwd, maglev_inject_swa_fwd, maglev_page_tables, maglev_page_tables_workspace_bytes,
               maglev_paged_decode_step, maglev_paged_decode_workspace_bytes, maglev_paged_write,
               maglev_swa_bwd_workspace_bytes, maglev_swa_saved_bytes)

TORCH_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": MAGLEV_BF16, "f32": MAGLEV_F32}


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)


def saved_entries(desc, saved):
    """The mixed keys and values k_bar, v_bar [B, T, H, hd] in a forward's `saved` buffer, as views of it."""
    shape, third = (desc.B, desc.T, desc.H, desc.hd), maglev_swa_saved_bytes(desc) // 3
    td = torch.bfloat16 if desc.dtype == MAGLEV_BF16 else torch.float32
    size = desc.B * desc.T * desc.H * desc.hd * td.itemsize
    return tuple(saved[i * third:i * third + size].view(td).view(shape) for i in (1, 2))


class InjectedSWALayer:
    def __init__(self, B, T, H, hd, d_mem, window, dtype="bf16", inject=True, pos0=0,
                 rope_base=10000.0, eps=1e-6, device="cuda", spin_limit=0, shared_kv_gates=False):
        self.shape = (B, T, H, hd)
        self.d_mem, self.dtype, self.device = d_mem, dtype, device
        self.inject = bool(inject)
        self.desc = SwaDesc(B=B, T=T, H=H, hd=hd, d_mem=d_mem, window=window, rope_base=rope_base,
                            rms_eps=eps, inject=int(inject), pos0=pos0, dtype=CODE[dtype],
                            spin_limit=spin_limit, shared_kv_gates=int(shared_kv_gates))
        td = TORCH_DTYPE[dtype]
        D = H * hd
        self.out = torch.empty(B, T, H, hd, dtype=td, device=device)
        self.lse = torch.empty(B, H, T, dtype=torch.float32, device=device)
        self.saved = _bytes(maglev_swa_saved_bytes(self.desc), device)
        self.workspace = _bytes(maglev_swa_bwd_workspace_bytes(self.desc), device)
        self.R_k = torch.empty(B, T, D, dtype=td, device=device) if inject else None
        self.R_v = torch.empty(B, T, D, dtype=td, device=device) if inject else None
        self.dq = torch.empty(B, T, H, hd, dtype=td, device=device)
        self.dk = torch.empty_like(self.dq)
        self.dv = torch.empty_like(self.dq)
        self.dR_k = torch.empty(B, T, D, dtype=td, device=device) if inject else None
        self.dR_v = torch.empty(B, T, D, dtype=td, device=device) if inject else None
        self.dgate = torch.empty(2 if shared_kv_gates else 4, H, dtype=torch.float32,
                                 device=device) if inject else None
        self.dm_shift = torch.empty(B, T, d_mem, dtype=td, device=device) if inject else None
        self.dw_mk = torch.empty(D, d_mem, dtype=td, device=device) if inject else None
        self.dw_mv = torch.empty(D, d_mem, dtype=td, device=device) if inject else None
        self.loss = torch.zeros((), dtype=torch.float32, device=device)
        self.loss_ws = _bytes(maglev_consistency_workspace_bytes(B * T, D), device)

    def forward(self, q, k, v, gates=None, m_shift=None, w_mk=None, w_mv=None, stream=None):
        """m_shift given: project it here; m_shift None: R_k/R_v already hold the projection."""
        maglev_inject_swa_fwd(self.desc, q, k, v, m_shift if self.inject else None, w_mk, w_mv,
                              self.R_k, self.R_v, gates, self.out, self.lse, self.saved, stream)
        return self.out

    def entries(self):
        """The last forward's mixed keys and values [B, T, H, hd], views of `saved`: what a paged cache stores of a prompt
        (PagedLayerState.write without positions, rows b * T + t)."""
        return saved_entries(self.desc, self.saved)

    def consistency(self, m, target, lam, dm=None, accumulate_dm=False, inv_count=0.0, stream=None):
        rows = m.numel() // m.shape[-1]
        maglev_consistency_loss(m, target, rows, m.shape[-1], CODE[self.dtype], lam, inv_count,
                                self.loss, dm, None, accumulate_dm, self.loss_ws, stream)
        return self.loss

    def consistency_prepare_bwd(self, target, lam, dout, inv_count=0.0, stream=None):
        """The consistency loss of this layer's own output against target,
        added into dout, together with the backward's first pass (the next
        backward call is given prepared=True)."""
        maglev_consistency_loss_prepare_bwd(self.desc, self.out, target, lam, inv_count, self.loss, dout,
                                            self.workspace, self.loss_ws, stream)
        return self.loss

    def backward(self, k, v, dout, gates=None, m_shift=None, w_mk=None, w_mv=None,
                 dR_mode=MAGLEV_DR_WRITE, dR_acc=(None, None), stream=None, prepared=False):
        """dR_mode / dR_acc: how dL/dR is stored (maglev_dr_mode) and the fp32
        running sums it reads or writes when several layers share W^rec;
        prepared: consistency_prepare_bwd ran on this out and dout."""
        maglev_inject_swa_bwd(self.desc, k, v, self.R_k, self.R_v, gates, self.out, self.lse,
                              self.saved, dout, self.dq, self.dk, self.dv, self.dR_k, self.dR_v,
                              dR_acc[0], dR_acc[1], dR_mode | (MAGLEV_BWD_PREPARED if prepared else 0), self.dgate,
                              m_shift if self.inject else None, w_mk, w_mv,
                              self.dm_shift, self.dw_mk, self.dw_mv, self.workspace, stream)


class DecodeLayerState:
    """Buffers of one decode step of one layer (rings are caller tensors)."""

    def __init__(self, B, H, hd, d_mem, window, dtype="bf16", inject=True, rope_base=10000.0,
                 eps=1e-6, device="cuda", shared_kv_gates=False):
        self.desc = DecodeDesc(B=B, H=H, hd=hd, d_mem=d_mem, window=window, rope_base=rope_base,
                               rms_eps=eps, inject=int(inject), dtype=CODE[dtype], spin_limit=0,
                               shared_kv_gates=int(shared_kv_gates))
        td = TORCH_DTYPE[dtype]
        self.krec = torch.empty(B, H, hd, dtype=td, device=device)
        self.vrec = torch.empty(B, H, hd, dtype=td, device=device)
        self.out = torch.empty(B, H, hd, dtype=td, device=device)
        # zero-filled once; every completed step leaves it zero-filled
        self.workspace = torch.zeros(max(16, maglev_decode_workspace_bytes(self.desc)), dtype=torch.uint8,
                                     device=device)

    def mem_project(self, pos, m_prev, w_mk, w_mv, stream=None):
        maglev_decode_mem_project(self.desc, pos, m_prev, w_mk, w_mv, self.krec, self.vrec, stream)

    def step(self, pos, q, k, v, gates, k_ring, v_ring, stream=None):
        maglev_decode_step(self.desc, pos, q, k, v, self.krec, self.vrec, gates, k_ring, v_ring,
                           self.out, self.workspace, stream)
        return self.out


def _paged_desc(tables, H, H_kv, hd, window, dtype, inject, rope_base, eps, shared_kv_gates):
    return PagedDesc(B=tables.B, H=H, H_kv=H_kv, hd=hd, page_size=tables.page_size, max_pages=tables.max_pages,
                     num_pages=tables.num_pages, window=window, rope_base=rope_base, rms_eps=eps, inject=int(inject),
                     dtype=CODE[dtype], shared_kv_gates=int(shared_kv_gates))


def _need(name, t, shape, dtype, device):
    """A dense tensor of this shape and type on the owner's GPU: the library sees its address only."""
    if (t is None or tuple(t.shape) != shape or t.dtype != dtype or not t.is_cuda or t.device != device
            or not t.is_contiguous()):
        have = "None" if t is None else f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}"
        raise ValueError(f"{name} must be a dense {shape} {dtype} tensor on {device}, not {have}")


def _need_current(device):
    """The library launches on the current device, whatever its pointers belong to."""
    if device.type == "cuda" and torch.cuda.current_device() != device.index:
        raise ValueError(f"the buffers lie on {device}, which is not the current device")


class PageTables:
    """Block table, free pages and lengths of B sequences in a paged cache, shared by its layers.

    step() takes the new token counts of one serving step and returns the
    positions and slots of its token rows; all state stays on the device, so
    that a step can be captured in a CUDA graph.
    """

    def __init__(self, B, page_size, max_pages, num_pages, max_tokens, device="cuda"):
        self.B, self.page_size, self.max_pages, self.num_pages = B, page_size, max_pages, num_pages
        self.max_tokens = max_tokens
        i32, i64 = dict(dtype=torch.int32, device=device), dict(dtype=torch.int64, device=device)
        self.block_table = torch.full((B, max_pages), -1, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)  # page 0 is handed out first
        self.n_free = torch.full((1,), num_pages, **i32)
        self.lengths = torch.zeros(B, **i64)
        self.device = self.block_table.device
        self.cu_tokens = torch.zeros(B + 1, **i64)
        self.pos = torch.full((max_tokens,), -1, **i64)
        self.slots = torch.full((max_tokens,), -1, **i64)
        # the library call reads the sizes only
        self.desc = _paged_desc(self, 1, 1, 64, 0, "bf16", False, 10000.0, 1e-6, False)
        self.workspace = _bytes(maglev_page_tables_workspace_bytes(self.desc), device)

    def step(self, new_len, n_tokens=None, pad=0, stream=None):
        """new_len [B] int64 on the device: tokens each sequence brings, -1 where it is finished.
        Returns (pos, slots) of the first n_tokens rows (packed; pad > 0: row b * pad + i), views that the next step
        writes over."""
        n = self.max_tokens if n_tokens is None else n_tokens
        if n > self.max_tokens:
            raise ValueError(f"n_tokens {n} exceeds the {self.max_tokens} rows this table was made for")
        _need_current(self.device)
        _need("new_len", new_len, (self.B,), torch.int64, self.device)
        maglev_page_tables(self.desc, self.lengths, new_len, n, pad, self.free_pages, self.n_free, self.block_table,
                           self.lengths, self.n_free, self.cu_tokens, self.pos, self.slots, self.workspace, stream)
        return self.pos[:n], self.slots[:n]


class PagedLayerState:
    """One layer's pages over a PageTables, and the buffers of its decode step."""

    def __init__(self, tables, H, hd, H_kv=None, window=0, d_mem=0, dtype="bf16", inject=False, rope_base=10000.0,
                 eps=1e-6, device="cuda", shared_kv_gates=False):
        self.tables = tables
        H_kv = H if H_kv is None else H_kv
        self.desc = _paged_desc(tables, H, H_kv, hd, window, dtype, inject, rope_base, eps, shared_kv_gates)
        self.copy_desc = _paged_desc(tables, H, H_kv, hd, window, dtype, False, rope_base, eps, shared_kv_gates)
        td = TORCH_DTYPE[dtype]
        B = tables.B
        self.dtype, self.inject = td, bool(inject)
        self.k_pages = torch.empty(tables.num_pages, H_kv, tables.page_size, hd, dtype=td, device=device)
        self.v_pages = torch.empty_like(self.k_pages)
        self.out = torch.empty(B, H, hd, dtype=td, device=device)
        self.device = self.out.device
        if self.device != tables.device:
            raise ValueError(f"the layer's pages would lie on {self.device}, its tables lie on {tables.device}")
        self.krec = torch.empty(B, H_kv, hd, dtype=td, device=device) if inject else None
        self.vrec = torch.empty(B, H_kv, hd, dtype=td, device=device) if inject else None
        self.mem_desc = DecodeDesc(B=B, H=H_kv, hd=hd, d_mem=d_mem, window=1, rope_base=rope_base, rms_eps=eps,
                                   inject=int(inject), dtype=CODE[dtype], spin_limit=0,
                                   shared_kv_gates=int(shared_kv_gates))
        self.workspace = _bytes(maglev_paged_decode_workspace_bytes(self.desc), device)

    def write(self, slots, pos, k, v, R_k=None, R_v=None, gates=None, stream=None):
        """Entries of the token rows k, v [n, H_kv, hd] into their slots. pos None: k and v are entries that a forward has
        mixed and are stored as they are, in an injected layer too (R_k, R_v and gates then are not used)."""
        n, rows = slots.numel(), (slots.numel(), self.desc.H_kv, self.desc.hd)
        desc, inject = (self.copy_desc, False) if pos is None else (self.desc, self.inject)
        _need_current(self.device)
        _need("slots", slots, (n,), torch.int64, self.device)
        if pos is not None:
            _need("pos", pos, (n,), torch.int64, self.device)
        for name, t in (("k", k), ("v", v)) + ((("R_k", R_k), ("R_v", R_v)) if inject else ()):
            _need(name, t, rows, self.dtype, self.device)
        if inject:
            self._need_gates(gates)
        maglev_paged_write(desc, n, slots, pos, k, v, R_k, R_v, gates, self.k_pages, self.v_pages, stream)

    def mem_project(self, pos, m_prev, w_mk, w_mv, stream=None):
        """The step's memory entries (inject): m_prev [B, d_mem], w_mk, w_mv [H_kv * hd, d_mem]."""
        d, weights = self.mem_desc, (self.desc.H_kv * self.desc.hd, self.mem_desc.d_mem)
        _need_current(self.device)
        _need("pos", pos, (d.B,), torch.int64, self.device)
        _need("m_prev", m_prev, (d.B, d.d_mem), self.dtype, self.device)
        _need("w_mk", w_mk, weights, self.dtype, self.device)
        _need("w_mv", w_mv, weights, self.dtype, self.device)
        maglev_decode_mem_project(self.mem_desc, pos, m_prev, w_mk, w_mv, self.krec, self.vrec, stream)

    def _need_gates(self, gates):
        _need("gates", gates, (2 if self.desc.shared_kv_gates else 4, self.desc.H_kv), torch.float32, self.device)

    def step(self, pos, q, k, v, gates=None, stream=None):
        """Attention of one token per sequence, q [B, H, hd], k, v [B, H_kv, hd] at pos [B] (-1: not running)."""
        d = self.desc
        _need_current(self.device)
        _need("pos", pos, (d.B,), torch.int64, self.device)
        _need("q", q, (d.B, d.H, d.hd), self.dtype, self.device)
        _need("k", k, (d.B, d.H_kv, d.hd), self.dtype, self.device)
        _need("v", v, (d.B, d.H_kv, d.hd), self.dtype, self.device)
        if self.inject:
            self._need_gates(gates)
        maglev_paged_decode_step(self.desc, pos, q, k, v, self.krec, self.vrec, gates, self.tables.block_table,
                                 self.k_pages, self.v_pages, self.out, self.workspace, stream)
        return self.out
