"""Device-resident decode state on top of the C ABI.

A ``GqaSession`` does the same for the GQA route (qkn_gqa_append,
qkn_gqa_decode): the per-group expanded cache, the group weights, the raw
queries and a workspace.

A ``DecodeSession`` owns a paged cache, the key up-projection and norm
weights, the value up-projection (optional), the absorbed queries and a
decode workspace, and forwards to ``qkn_append``, ``qkn_absorb_query``,
``qkn_decode`` and ``qkn_decode_up``.  It moves host
arrays to the device and nothing else: all arithmetic runs in libqkn.

With ``load_projections`` the session starts from hidden states and ends in
them: the layer's projections around the attention run in 8 bits
(``qkn_norm_quant``, ``qkn_fp8_linear``; weights quantised on the device at
load time, ``qkn_quant_weight``).

A session's calls share its buffers: they run on one stream, or one after the
other.
"""
from __future__ import annotations

import weakref
from typing import Optional

import numpy as np
import torch

from . import (AK_CACHE, KERNEL_AUTO, OK, WORKSPACE_BYTES, Cache, Dims, Fp8Rows, Fp8Weight, GqaCache, absorb_query,
               append, append_absorb, decode, decode_up, decode_workspace_size, fp8_linear, gqa_append, gqa_decode,
               gqa_workspace_size, key_gram, norm_quant, quant_weight, read_device_status, workspace_init)


def to_device(x, dtype: torch.dtype, device) -> torch.Tensor:
    if isinstance(x, torch.Tensor):
        return x.to(device=device, dtype=dtype).contiguous()
    return torch.from_numpy(np.ascontiguousarray(x)).to(device=device, dtype=dtype).contiguous()


class DecodeSession:
    def __init__(self, dims: Dims, num_blocks: int, device="cuda"):
        self.dims = dims
        self.device = torch.device(device)
        self.cache = Cache(dims, num_blocks, device=self.device)
        self.w_k = self.key_gram = self.gamma_q = self.gamma_k = self.gamma_qr = self.gamma_kr = None
        self.w_uv: Optional[torch.Tensor] = None
        self.q_tilde = self.a_q = self.q_rope_hat = None
        self.workspace: Optional[torch.Tensor] = None
        self._workspaces = []                          # weak references to the ones before, which steps may hold
        self._kept = {}                                # what captured calls use, by id
        self.w_in: Optional[Fp8Weight] = None
        self.w_out: Optional[Fp8Weight] = None
        self.gamma_x: Optional[torch.Tensor] = None
        self.x8 = self.o8 = None                       # the projections' inputs in 8 bits
        self.q = self.q_rope = self.c_new = self.k_rope_new = None
        self.proj_workspace: Optional[torch.Tensor] = None

    def _keep(self, *used) -> None:
        """Buffers and weights that a call is about to use.  If a graph captures the call it holds their addresses, so
        they stay when other sizes or other weights take their place here."""
        if torch.cuda.is_current_stream_capturing():
            self._kept.update((id(t), t) for t in used)

    # ------------------------------------------------------------ weights
    def load_weights(self, w_k, gamma_q, gamma_k, gamma_qr, gamma_kr) -> None:
        f32, dev = torch.float32, self.device
        self.w_k = to_device(w_k, f32, dev)
        d = self.dims
        self.key_gram = torch.empty((d.num_groups, d.r_kv, d.r_kv), dtype=f32, device=dev)
        key_gram(d, self.w_k, self.key_gram)
        self.gamma_q = to_device(gamma_q, f32, dev)
        self.gamma_k = to_device(gamma_k, f32, dev)
        self.gamma_qr = to_device(gamma_qr, f32, dev)
        self.gamma_kr = to_device(gamma_kr, f32, dev)

    def load_value_weights(self, w_uv) -> None:
        """W^UV [H, r_kv, d_v], kept in the storage dtype (the fused merge reads it every step)."""
        self.w_uv = to_device(w_uv, self.dims.torch_dtype, self.device)

    def load_projections(self, gamma_x, w_in, w_out=None) -> None:
        """The layer's projections, quantised to 8 bits here (in the storage dtype until then): ``gamma_x`` [D] the
        norm in front of them, ``w_in`` [H d_h + H d_R + r + d_R, D] with the rows of q, q^R, c and k^R in this order,
        ``w_out`` [D, H d_v] the output projection of the up-projected values (needs load_value_weights)."""
        d, dev = self.dims, self.device
        gamma_x = to_device(gamma_x, torch.float32, dev)
        if tuple(w_in.shape) != (sum(self.projection_widths()), gamma_x.shape[0]):
            raise ValueError("w_in is [H d_h + H d_R + r + d_R, D], gamma_x [D]")
        if w_out is not None and (self.w_uv is None or w_out.shape[1] != d.num_heads * self.w_uv.shape[-1]):
            raise ValueError("w_out is [D, H d_v] for the value weights loaded before")
        w_in, w_out = self._quantised(w_in), None if w_out is None else self._quantised(w_out)
        self.gamma_x, self.w_in, self.w_out = gamma_x, w_in, w_out
        self.q = self.x8 = self.o8 = None              # sized by the weights
        if self.proj_workspace is None:                # kept: steps record into it, and an error stays until cleared
            self.proj_workspace = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
            workspace_init(self.proj_workspace)

    def check_out_width(self) -> None:
        """load_value_weights may have replaced the weights that load_projections was given w_out for."""
        if self.w_out.cols != self.dims.num_heads * self.w_uv.shape[-1]:
            raise ValueError("w_out was loaded for value weights of another width")

    def _quantised(self, w) -> Fp8Weight:
        w = to_device(w, self.dims.torch_dtype, self.device)
        q = Fp8Weight.empty(int(w.shape[0]), int(w.shape[1]), self.device)
        quant_weight(w, q)
        return q

    def projection_widths(self):
        """Columns of q, q^R, c and k^R in the input projection."""
        d = self.dims
        return d.num_heads * d.d_h, d.num_heads * d.d_rope, d.r_kv, d.d_rope

    # ------------------------------------------------------------ hidden states
    def project(self, x, residual=None):
        """Hidden states [n, D] -> q [n, H, d_h], q^R [n, H, d_R], c [n, r], k^R [n, d_R] (raw, as append and absorb
        take them).  ``residual`` (a device tensor [n, D]) is added first and takes the sum.  The output buffers are
        reused while n stays the same."""
        d, dt, dev = self.dims, self.dims.torch_dtype, self.device
        if self.w_in is None:
            raise RuntimeError("project needs load_projections first")
        x = to_device(x, dt, dev)
        n = int(x.shape[0])
        if self.q is None or self.q.shape[0] != n:
            self.x8 = Fp8Rows.empty(n, self.w_in.cols, dev)
            self.q, self.q_rope, self.c_new, self.k_rope_new = (
                torch.empty((n, w), dtype=dt, device=dev) for w in self.projection_widths())
        self._keep(self.x8, self.q, self.q_rope, self.c_new, self.k_rope_new, self.gamma_x, self.w_in)
        norm_quant(x, self.x8, gamma=self.gamma_x, eps=d.eps, residual=residual, residual_out=residual)
        fp8_linear(self.x8, self.w_in, (self.q, self.q_rope, self.c_new, self.k_rope_new), self.proj_workspace)
        return (self.q.view(n, d.num_heads, d.d_h), self.q_rope.view(n, d.num_heads, d.d_rope), self.c_new,
                self.k_rope_new)

    def prepare_hidden(self, x, slot, pos, residual=None) -> None:
        """A decode step's preparation from hidden states: every row of ``x`` is a new token and a query at its
        position (append, query absorption)."""
        q, q_rope, c, k_rope = self.project(x, residual)
        pos = to_device(pos, torch.int32, self.device)
        self.prepare(c, k_rope, slot, pos, q, q_rope, pos)

    def project_out(self, o_v, out=None):
        """The output projection: o_v [..., H, d_v] -> hidden states [n, D]."""
        if self.w_out is None:
            raise RuntimeError("project_out needs load_projections with w_out first")
        self.check_out_width()
        if o_v.shape[-1] != self.w_out.cols and o_v.shape[-2:] != (self.dims.num_heads, self.w_uv.shape[-1]):
            raise ValueError("o_v is [..., H, d_v] or [..., H d_v]")
        rows = o_v.reshape(-1, self.w_out.cols)
        n = int(rows.shape[0])
        if self.o8 is None or self.o8.rows != n:
            self.o8 = Fp8Rows.empty(n, self.w_out.cols, self.device)
        if out is None:
            out = torch.empty((n, self.w_out.rows), dtype=self.dims.torch_dtype, device=self.device)
        self._keep(self.o8, self.w_out)
        norm_quant(rows, self.o8)
        fp8_linear(self.o8, self.w_out, (out,), self.proj_workspace)
        return out

    # ------------------------------------------------------------ cache
    def append(self, c, k_rope_raw, slot, pos, chunk: int = 1 << 16) -> None:
        """Append tokens (host or device arrays) in chunks of ``chunk`` tokens."""
        dt, dev = self.dims.torch_dtype, self.device
        n = int(c.shape[0])
        self._keep(self.w_k, self.key_gram, self.gamma_kr)
        for t0 in range(0, n, chunk):
            sl = slice(t0, min(n, t0 + chunk))
            append(self.dims, self.cache, to_device(c[sl], dt, dev), to_device(k_rope_raw[sl], dt, dev),
                   to_device(slot[sl], torch.int32, dev), to_device(pos[sl], torch.int32, dev),
                   self.w_k, self.key_gram, self.gamma_kr)

    # ------------------------------------------------------------ queries
    def absorb(self, q, q_rope, pos) -> None:
        """q [n_q, H, d_h], q_rope [n_q, H, d_R], pos [n_q] -> q~, a_q, q^R^ on the device.
        The output buffers are reused while the query count stays the same."""
        d, dt, dev = self.dims, self.dims.torch_dtype, self.device
        q = to_device(q, dt, dev)
        q_rope = to_device(q_rope, dt, dev)
        self.ensure_query_buffers(q.shape[0])
        self._keep(self.w_k, self.gamma_q, self.gamma_k, self.gamma_qr)
        absorb_query(d, q, q_rope, to_device(pos, torch.int32, dev), self.w_k, self.gamma_q, self.gamma_k,
                     self.gamma_qr, self.q_tilde, self.a_q, self.q_rope_hat)

    def prepare(self, c, k_rope_raw, slot, pos, q, q_rope, qpos) -> None:
        """A decode step's append and query absorption, in one launch where possible."""
        d, dt, dev = self.dims, self.dims.torch_dtype, self.device
        q = to_device(q, dt, dev)
        self.ensure_query_buffers(q.shape[0])
        self._keep(self.w_k, self.key_gram, self.gamma_q, self.gamma_k, self.gamma_qr, self.gamma_kr)
        append_absorb(d, self.cache, to_device(c, dt, dev), to_device(k_rope_raw, dt, dev),
                      to_device(slot, torch.int32, dev), to_device(pos, torch.int32, dev), q,
                      to_device(q_rope, dt, dev), to_device(qpos, torch.int32, dev), self.w_k, self.key_gram,
                      self.gamma_q,
                      self.gamma_k, self.gamma_qr, self.gamma_kr, self.q_tilde, self.a_q, self.q_rope_hat)

    def ensure_query_buffers(self, n_q: int) -> None:
        """Device buffers for q~, a_q and q^R^ of n_q query rows (kept while n_q stays the same)."""
        d, dt, dev = self.dims, self.dims.torch_dtype, self.device
        if self.q_tilde is None or self.q_tilde.shape[0] != n_q:
            self.q_tilde = torch.empty((n_q, d.num_heads, d.r_kv), dtype=dt, device=dev)
            self.a_q = torch.empty((n_q, d.num_heads), dtype=torch.float32, device=dev)
            self.q_rope_hat = torch.empty((n_q, d.num_heads, d.d_rope), dtype=dt, device=dev)
        self._keep(self.q_tilde, self.a_q, self.q_rope_hat)

    # ------------------------------------------------------------ decode
    def ensure_workspace(self, batch: int, s_q: int) -> torch.Tensor:
        need = decode_workspace_size(self.dims, batch, s_q)
        if self.workspace is None or self.workspace.numel() < need:
            old, self.workspace = self.workspace, torch.empty(need, dtype=torch.uint8, device=self.device)
            workspace_init(self.workspace)
            if old is not None:                        # an error that is recorded there stays until it is cleared
                if torch.cuda.is_current_stream_capturing():
                    self._keep(old)                    # (a copy would run again with every replay)
                else:
                    self.workspace[:4].copy_(old[:4])
                self._workspaces = [r for r in self._workspaces if r() is not None] + [weakref.ref(old)]
        self._keep(self.workspace)
        return self.workspace

    def decode(self, block_table, seq_lens, s_q: int, out=None, lse=None, ak_mode: int = AK_CACHE,
               kernel: int = KERNEL_AUTO, max_ctas: int = 0, head_tile: int = 0, wait_limit: int = 0,
               split_event=None, step_writes_only: bool = False, test_withhold_ak: bool = False, vis_end=None):
        d, dev = self.dims, self.device
        bt = to_device(block_table, torch.int32, dev)
        sl = to_device(seq_lens, torch.int32, dev)
        batch = bt.shape[0]
        ws = self.ensure_workspace(batch, s_q)
        if out is None:
            out = torch.empty((batch, s_q, d.num_heads, d.r_kv), dtype=d.torch_dtype, device=dev)
        if lse is None:
            lse = torch.empty((batch, s_q, d.num_heads), dtype=torch.float32, device=dev)
        self._keep(self.q_tilde, self.a_q, self.q_rope_hat)
        decode(d, self.cache, self.q_tilde, self.a_q, self.q_rope_hat, bt, sl, s_q, ws, out, lse,
               ak_mode=ak_mode, kernel=kernel, max_ctas=max_ctas, head_tile=head_tile, wait_limit=wait_limit,
               split_event=split_event, step_writes_only=step_writes_only, test_withhold_ak=test_withhold_ak,
               vis_end=None if vis_end is None else to_device(vis_end, torch.int32, dev))
        return out, lse

    def decode_up(self, block_table, seq_lens, s_q: int, out_v=None, lse=None, ak_mode: int = AK_CACHE,
                  kernel: int = KERNEL_AUTO, max_ctas: int = 0, head_tile: int = 0, wait_limit: int = 0,
                  split_event=None, step_writes_only: bool = False):
        """The decode step with the value up-projection fused into the merge: o_v [batch, s_q, H, d_v]."""
        d, dev = self.dims, self.device
        if self.w_uv is None:
            raise RuntimeError("decode_up needs load_value_weights first")
        bt = to_device(block_table, torch.int32, dev)
        sl = to_device(seq_lens, torch.int32, dev)
        batch = bt.shape[0]
        ws = self.ensure_workspace(batch, s_q)
        if out_v is None:
            out_v = torch.empty((batch, s_q, d.num_heads, self.w_uv.shape[-1]), dtype=d.torch_dtype, device=dev)
        if lse is None:
            lse = torch.empty((batch, s_q, d.num_heads), dtype=torch.float32, device=dev)
        self._keep(self.w_uv, self.q_tilde, self.a_q, self.q_rope_hat)
        decode_up(d, self.cache, self.q_tilde, self.a_q, self.q_rope_hat, bt, sl, s_q, self.w_uv, ws, out_v, lse,
                  ak_mode=ak_mode, kernel=kernel, max_ctas=max_ctas, head_tile=head_tile, wait_limit=wait_limit,
                  split_event=split_event, step_writes_only=step_writes_only)
        return out_v, lse

    def _status_words(self):
        """The workspaces whose status words a kernel of the session's or of a step's may write: the decode's, those
        that it has outgrown but a step still holds, the projections'."""
        outgrown = [w for w in (r() for r in self._workspaces) if w is not None]
        return [w for w in (self.workspace, *outgrown, self.proj_workspace) if w is not None] or [None]

    def device_status(self) -> int:
        """The first error that a kernel recorded: the decode's, then the projections'.  The steps of the session
        record here too."""
        return next((st for st in map(read_device_status, self._status_words()) if st != OK), OK)

    def clear_status(self) -> None:
        for w in self._status_words():
            workspace_init(w)


def session_from_inputs(inp, device="cuda", dtype=None) -> DecodeSession:
    """Build a session from a seeded problem (an object with the fields of qkn_inputs.Inputs):
    weights loaded, every context token appended, queries absorbed."""
    wl = inp.wl
    dt = dtype if dtype is not None else (1 if wl.dtype == "bf16" else 0)
    dims = Dims(num_heads=wl.heads, num_groups=wl.groups, r_kv=wl.r_kv, d_h=wl.d_h, d_rope=wl.d_rope,
                eps=wl.eps, softmax_scale=wl.softmax_scale, rope_theta=wl.rope_theta, dtype=dt,
                block_size=wl.block_size)
    s = DecodeSession(dims, inp.num_blocks, device=device)
    s.load_weights(inp.w_k, inp.gamma_q, inp.gamma_k, inp.gamma_qr, inp.gamma_kr)
    s.load_value_weights(inp.w_uv)
    s.append(inp.c, inp.k_rope, inp.token_slots(), inp.token_positions())
    B, s_q = wl.batch, wl.s_q
    s.absorb(inp.q.reshape(B * s_q, wl.heads, wl.d_h), inp.q_rope.reshape(B * s_q, wl.heads, wl.d_rope),
             inp.query_positions().reshape(-1))
    return s


class GqaSession:
    """Device state of the GQA route: per-group keys and values expanded from the latent, the group weights
    W^UK_g, gamma_k[g], W^UV_g, the norm weights of the queries and RoPE key, the step's raw queries and a
    workspace."""

    def __init__(self, dims: Dims, num_blocks: int, d_v: int, device="cuda"):
        self.dims = dims
        self.device = torch.device(device)
        self.cache = GqaCache(dims, num_blocks, d_v, device=self.device)
        self.w_uk = self.gamma_k = self.w_uv = self.gamma_q = self.gamma_qr = self.gamma_kr = None
        self.q = self.q_rope = None
        self.workspace: Optional[torch.Tensor] = None

    def load_weights(self, w_uk, gamma_k, w_uv, gamma_q, gamma_qr, gamma_kr) -> None:
        """W^UK [g, r, d_h] and the gammas in fp32, W^UV [g, r, d_v] in the storage dtype."""
        f32, dev = torch.float32, self.device
        self.w_uk = to_device(w_uk, f32, dev)
        self.gamma_k = to_device(gamma_k, f32, dev)
        self.w_uv = to_device(w_uv, self.dims.torch_dtype, dev)
        self.gamma_q = to_device(gamma_q, f32, dev)
        self.gamma_qr = to_device(gamma_qr, f32, dev)
        self.gamma_kr = to_device(gamma_kr, f32, dev)

    def append(self, c, k_rope_raw, slot, pos, chunk: int = 1 << 16) -> None:
        dt, dev = self.dims.torch_dtype, self.device
        n = int(c.shape[0])
        for t0 in range(0, n, chunk):
            sl = slice(t0, min(n, t0 + chunk))
            gqa_append(self.dims, self.cache, to_device(c[sl], dt, dev), to_device(k_rope_raw[sl], dt, dev),
                       to_device(slot[sl], torch.int32, dev), to_device(pos[sl], torch.int32, dev), self.w_uk,
                       self.gamma_k, self.w_uv, self.gamma_kr)

    def set_queries(self, q, q_rope) -> None:
        """The step's raw queries: q [batch, s_q, H, d_h], q_rope [batch, s_q, H, d_R]."""
        dt, dev = self.dims.torch_dtype, self.device
        self.q = to_device(q, dt, dev)
        self.q_rope = to_device(q_rope, dt, dev)

    def ensure_workspace(self, batch: int, s_q: int) -> torch.Tensor:
        need = gqa_workspace_size(self.dims, self.cache.d_v, batch, s_q)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            workspace_init(self.workspace)
        return self.workspace

    def decode(self, block_table, seq_lens, s_q: int, selection=None, max_ctas: int = 0, out_v=None, lse=None):
        """o_v [batch, s_q, H, d_v] and lse [batch, s_q, H]; ``selection`` [batch, s_q, g, k] for sparse."""
        d, dev = self.dims, self.device
        bt = to_device(block_table, torch.int32, dev)
        sl = to_device(seq_lens, torch.int32, dev)
        batch = bt.shape[0]
        ws = self.ensure_workspace(batch, s_q)
        if out_v is None:
            out_v = torch.empty((batch, s_q, d.num_heads, self.cache.d_v), dtype=d.torch_dtype, device=dev)
        if lse is None:
            lse = torch.empty((batch, s_q, d.num_heads), dtype=torch.float32, device=dev)
        sel = None if selection is None else to_device(selection, torch.int32, dev)
        gqa_decode(d, self.cache, self.q, self.q_rope, self.gamma_q, self.gamma_qr, bt, sl, s_q, ws, out_v, lse,
                   selection=sel, max_ctas=max_ctas)
        return out_v, lse

    def device_status(self) -> int:
        return read_device_status(self.workspace)

    def clear_status(self) -> None:
        workspace_init(self.workspace)


def gqa_session_from_inputs(inp, device="cuda") -> GqaSession:
    """A GQA-route session from a seeded problem of a tied-groups workload: group weights loaded, every
    context token expanded into the cache, the step's queries set."""
    wl = inp.wl
    dims = Dims(num_heads=wl.heads, num_groups=wl.groups, r_kv=wl.r_kv, d_h=wl.d_h, d_rope=wl.d_rope,
                eps=wl.eps, softmax_scale=wl.softmax_scale, rope_theta=wl.rope_theta,
                dtype=1 if wl.dtype == "bf16" else 0, block_size=wl.block_size)
    s = GqaSession(dims, inp.num_blocks, wl.d_v, device=device)
    w_uk, gamma_k, w_uv = inp.group_weights()
    s.load_weights(w_uk, gamma_k, w_uv, inp.gamma_q, inp.gamma_qr, inp.gamma_kr)
    s.append(inp.c, inp.k_rope, inp.token_slots(), inp.token_positions())
    s.set_queries(inp.q, inp.q_rope)
    return s

