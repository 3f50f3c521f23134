"""A whole decode step replayed as one CUDA graph.

Serving loops run the same step shape over and over: copy the step's new
tokens and queries in, append the tokens to the cache, absorb the queries,
decode, copy the result out.  ``DecodeStep`` captures that sequence once over
fixed buffers (pinned host buffers for the inputs and outputs, device buffers
for everything else) and replays it, so a step costs one graph launch instead
of a dozen API calls and copies.  Append and query absorption run as one
launch (qkn_append_absorb); the split-KV decode and its merge follow on the
same stream.  All arithmetic runs in libqkn.

Usage::

    step = DecodeStep(session, batch=B, s_q=1, max_blocks=M, n_tok=B)
    step.host_in["c"][:] = ...        # fill the pinned inputs (see NAMES)
    out, lse = step.run()             # pinned host outputs, valid after run() returns

``LayerStep`` is the same for a whole attention layer, hidden states in and
out: norm with the residual's addition, input projections, append + absorb,
decode with the value up-projection, output projection (the projections in 8
bits, see DecodeSession.load_projections).
"""
from __future__ import annotations

import torch

from . import AK_CACHE, KERNEL_AUTO, Fp8Rows, append_absorb, decode, decode_up, fp8_linear, norm_quant


class DecodeStep:
    # pinned host inputs of one step
    NAMES = ("c", "k_rope", "slot", "pos", "q", "q_rope", "qpos", "block_table", "seq_lens")

    def __init__(self, session, batch: int, s_q: int, max_blocks: int, n_tok: int, kernel: int = KERNEL_AUTO,
                 ak_mode: int = AK_CACHE, head_tile: int = 0):
        d = session.dims
        dt, dev, i32 = d.torch_dtype, session.device, torch.int32
        n_q = batch * s_q
        self.session, self.batch, self.s_q, self.kernel, self.ak_mode = session, batch, s_q, kernel, ak_mode
        self.head_tile = head_tile
        shapes = {
            "c": ((n_tok, d.r_kv), dt), "k_rope": ((n_tok, d.d_rope), dt),
            "slot": ((n_tok,), i32), "pos": ((n_tok,), i32),
            "q": ((n_q, d.num_heads, d.d_h), dt), "q_rope": ((n_q, d.num_heads, d.d_rope), dt),
            "qpos": ((n_q,), i32),
            "block_table": ((batch, max_blocks), i32), "seq_lens": ((batch,), i32),
        }
        # inputs and outputs are views of one byte buffer each (256-byte aligned fields), so that a
        # step moves them with one copy each way
        in_off, in_bytes = self._layout([shapes[k] for k in self.NAMES])
        self._host_in_buf = torch.zeros(in_bytes, dtype=torch.uint8, pin_memory=True)
        self._dev_in_buf = torch.zeros(in_bytes, dtype=torch.uint8, device=dev)
        self.host_in = self._views(self._host_in_buf, self.NAMES, shapes, in_off)
        self.dev_in = self._views(self._dev_in_buf, self.NAMES, shapes, in_off)
        oshapes = {"out": ((batch, s_q, d.num_heads, d.r_kv), dt), "lse": ((batch, s_q, d.num_heads), torch.float32)}
        out_off, out_bytes = self._layout([oshapes["out"], oshapes["lse"]])
        self._host_out_buf = torch.zeros(out_bytes, dtype=torch.uint8, pin_memory=True)
        self._dev_out_buf = torch.zeros(out_bytes, dtype=torch.uint8, device=dev)
        dv = self._views(self._dev_out_buf, ("out", "lse"), oshapes, out_off)
        hv = self._views(self._host_out_buf, ("out", "lse"), oshapes, out_off)
        self.out, self.lse = dv["out"], dv["lse"]
        self.host_out = (hv["out"], hv["lse"])
        session.ensure_query_buffers(n_q)
        self.workspace = session.ensure_workspace(batch, s_q)
        self.graph = None
        self.h2d_bytes = in_bytes
        self.d2h_bytes = out_bytes

    @staticmethod
    def _layout(fields):
        offs, pos = [], 0
        for shape, dtype in fields:
            offs.append(pos)
            n = int(torch.Size(shape).numel()) * torch.empty((), dtype=dtype).element_size()
            pos += (n + 255) // 256 * 256
        return offs, pos

    @staticmethod
    def _views(buf, names, shapes, offs):
        out = {}
        for name, off in zip(names, offs):
            shape, dtype = shapes[name]
            n = int(torch.Size(shape).numel()) * torch.empty((), dtype=dtype).element_size()
            out[name] = buf[off:off + n].view(dtype).view(shape)
        return out

    def _body(self) -> None:
        s, d, di = self.session, self.session.dims, self.dev_in
        self._dev_in_buf.copy_(self._host_in_buf, non_blocking=True)
        append_absorb(d, s.cache, di["c"], di["k_rope"], di["slot"], di["pos"], di["q"], di["q_rope"], di["qpos"],
                      s.w_k, s.key_gram, s.gamma_q, s.gamma_k, s.gamma_qr, s.gamma_kr, s.q_tilde, s.a_q,
                      s.q_rope_hat)
        decode(d, s.cache, s.q_tilde, s.a_q, s.q_rope_hat, di["block_table"], di["seq_lens"], self.s_q,
               self.workspace, self.out, self.lse, ak_mode=self.ak_mode, kernel=self.kernel, head_tile=self.head_tile,
               step_writes_only=True)
        self._host_out_buf.copy_(self._dev_out_buf, non_blocking=True)

    def _read(self) -> tuple:
        """What the graph reads or writes of the session's."""
        s = self.session
        s.ensure_query_buffers(self.batch * self.s_q)    # (other sizes may have come since __init__)
        return s.q_tilde, s.a_q, s.q_rope_hat

    def capture(self) -> None:
        """Run the step once eagerly (first-call setup in the library), then capture it.  The graph keeps the session's
        weights and buffers of this moment: they live as long as it does, and weights that are loaded later are for
        steps that are captured later."""
        s, c = self.session, self.session.cache
        kept = (c.latent, c.k_rope, c.a_k, c.ak_scratch, s.w_k, s.key_gram, s.gamma_q, s.gamma_k, s.gamma_qr,
                s.gamma_kr, *self._read())
        stream = torch.cuda.Stream(device=self.session.device)
        stream.wait_stream(torch.cuda.current_stream(self.session.device))
        with torch.cuda.stream(stream):
            self._body()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream, capture_error_mode="relaxed"):
            self._body()
        self.graph, self.kept = graph, kept
        torch.cuda.current_stream(self.session.device).wait_stream(stream)

    def run(self):
        """Replay the step on the current stream and wait for it; returns the pinned (out, lse)."""
        if self.graph is None:
            self.capture()
        self.graph.replay()
        torch.cuda.current_stream(self.session.device).synchronize()
        return self.host_out


class LayerStep(DecodeStep):
    """One attention layer's decode step: row b s_q + j of ``x`` and ``residual`` is the j-th new token of sequence b.
    ``run`` returns pinned (hidden, residual): the layer's output [n, D] and x + residual, which the next layer takes
    as its ``x`` and ``residual`` (a stack of steps passes both through these host buffers)."""

    NAMES = ("x", "residual", "slot", "pos", "block_table", "seq_lens")

    def __init__(self, session, batch: int, s_q: int, max_blocks: int, kernel: int = KERNEL_AUTO,
                 ak_mode: int = AK_CACHE, head_tile: int = 0):
        if session.w_in is None or session.w_out is None:
            raise RuntimeError("LayerStep needs a session with load_projections (w_out included)")
        session.check_out_width()
        d = session.dims
        dt, dev, i32 = d.torch_dtype, session.device, torch.int32
        n, width = batch * s_q, session.w_in.cols
        self.session, self.batch, self.s_q, self.kernel, self.ak_mode = session, batch, s_q, kernel, ak_mode
        self.head_tile = head_tile
        shapes = {
            "x": ((n, width), dt), "residual": ((n, width), dt), "slot": ((n,), i32), "pos": ((n,), i32),
            "block_table": ((batch, max_blocks), i32), "seq_lens": ((batch,), i32),
        }
        in_off, in_bytes = self._layout([shapes[k] for k in self.NAMES])
        self._host_in_buf = torch.zeros(in_bytes, dtype=torch.uint8, pin_memory=True)
        self._dev_in_buf = torch.zeros(in_bytes, dtype=torch.uint8, device=dev)
        self.host_in = self._views(self._host_in_buf, self.NAMES, shapes, in_off)
        self.dev_in = self._views(self._dev_in_buf, self.NAMES, shapes, in_off)
        oshapes = {"hidden": ((n, session.w_out.rows), dt), "residual": ((n, width), dt)}
        out_off, out_bytes = self._layout([oshapes["hidden"], oshapes["residual"]])
        self._host_out_buf = torch.zeros(out_bytes, dtype=torch.uint8, pin_memory=True)
        self._dev_out_buf = torch.zeros(out_bytes, dtype=torch.uint8, device=dev)
        dv = self._views(self._dev_out_buf, ("hidden", "residual"), oshapes, out_off)
        hv = self._views(self._host_out_buf, ("hidden", "residual"), oshapes, out_off)
        self.hidden, self.residual = dv["hidden"], dv["residual"]
        self.host_out = (hv["hidden"], hv["residual"])
        # buffers of its own, so that other sizes on the same session leave the captured ones alone, and the
        # projections that the graph will read (capture keeps the attention's weights)
        self.gamma_x, self.w_in, self.w_out, self.w_uv = session.gamma_x, session.w_in, session.w_out, session.w_uv
        self.proj_workspace = session.proj_workspace
        self.x8 = Fp8Rows.empty(n, width, dev)
        self.o8 = Fp8Rows.empty(n, session.w_out.cols, dev)
        self.q, self.q_rope, self.c, self.k_rope = (torch.empty((n, w), dtype=dt, device=dev)
                                                    for w in session.projection_widths())
        self.q_tilde = torch.empty((n, d.num_heads, d.r_kv), dtype=dt, device=dev)
        self.a_q = torch.empty((n, d.num_heads), dtype=torch.float32, device=dev)
        self.q_rope_hat = torch.empty((n, d.num_heads, d.d_rope), dtype=dt, device=dev)
        self.o_v = torch.empty((n, session.w_out.cols), dtype=dt, device=dev)
        self.lse = torch.empty((n, d.num_heads), dtype=torch.float32, device=dev)
        self.workspace = session.ensure_workspace(batch, s_q)
        # the decode may start beside the preparation only where that is one launch
        self.step_writes_only = 0 < n <= 256 and session.cache.ak_scratch is not None
        self.graph = None
        self.h2d_bytes = in_bytes
        self.d2h_bytes = out_bytes

    def _read(self) -> tuple:
        return ()                                        # buffers of its own, projections held by __init__

    def _body(self) -> None:
        s, d, di = self.session, self.session.dims, self.dev_in
        self._dev_in_buf.copy_(self._host_in_buf, non_blocking=True)
        norm_quant(di["x"], self.x8, gamma=self.gamma_x, eps=d.eps, residual=di["residual"], residual_out=self.residual)
        fp8_linear(self.x8, self.w_in, (self.q, self.q_rope, self.c, self.k_rope), self.proj_workspace)
        append_absorb(d, s.cache, self.c, self.k_rope, di["slot"], di["pos"], self.q, self.q_rope, di["pos"], s.w_k,
                      s.key_gram, s.gamma_q, s.gamma_k, s.gamma_qr, s.gamma_kr, self.q_tilde, self.a_q,
                      self.q_rope_hat)
        decode_up(d, s.cache, self.q_tilde, self.a_q, self.q_rope_hat, di["block_table"], di["seq_lens"], self.s_q,
                  self.w_uv, self.workspace, self.o_v, self.lse, ak_mode=self.ak_mode, kernel=self.kernel,
                  head_tile=self.head_tile, step_writes_only=self.step_writes_only)
        norm_quant(self.o_v, self.o8)
        fp8_linear(self.o8, self.w_out, (self.hidden,), self.proj_workspace)
        self._host_out_buf.copy_(self._dev_out_buf, non_blocking=True)
