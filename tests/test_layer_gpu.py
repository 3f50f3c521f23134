"""An attention layer from hidden states to hidden states, its projections in 8 bits (GPU): the session's calls
one after the other, and LayerStep's captured graph.  Every stage is compared with its definition in 64 bits on
the values that the stage before it left on the device, under that stage's own tolerances."""
import copy

import numpy as np
import pytest
import torch

import oracle
import qk_normed_latent_qkn_b200 as qkn
from gpu_common import REL_TOL
from qk_normed_latent_qkn_b200.session import session_from_inputs
from qk_normed_latent_qkn_b200.step import LayerStep
from qkn_inputs import WORKLOADS, make_inputs
from test_projection_gpu import check_codes, check_product, host

pytestmark = pytest.mark.gpu

CASES = {
    # fp32 storage, a hidden width that no block of 128 divides
    "tiny_f32": (WORKLOADS["tiny_f32"].with_(batch=3, context=(100, 300), seed=81), 200),
    "small_mla_bf16": (WORKLOADS["small_mla_bf16"].with_(batch=4, context=(300, 700), seed=82), 1024),
    # two new tokens per sequence, four groups
    "grouped_mtp_bf16": (WORKLOADS["grouped_mtp_bf16"].with_(batch=5, context=(130, 900), seed=83), 1536),
    # a chunk of a prompt: more rows than the single-launch preparation takes
    "prefill_mla_bf16": (WORKLOADS["prefill_mla_bf16"].with_(batch=2, s_q=150, context=(150, 400), seed=84), 512),
}


def build(name):
    wl, width = CASES[name]
    inp = make_inputs(wl)
    s = session_from_inputs(inp)
    n, heads = wl.batch * wl.s_q, wl.heads
    g = torch.Generator().manual_seed(wl.seed)
    dt = s.dims.torch_dtype
    rows = sum(s.projection_widths())
    x = torch.randn((n, width), generator=g).to(dt).cuda()
    res = (2 * torch.randn((n, width), generator=g)).to(dt).cuda()
    gamma = 1 + 0.1 * torch.randn(width, generator=g)
    w_in = torch.randn((rows, width), generator=g) / width ** 0.5
    w_out = torch.randn((width, heads * wl.d_v), generator=g) / (heads * wl.d_v) ** 0.5
    s.load_projections(gamma, w_in, w_out)
    last = np.concatenate([np.arange(inp.tok_off[b + 1] - wl.s_q, inp.tok_off[b + 1]) for b in range(wl.batch)])
    return inp, s, x, res, host(gamma), last


def check_linear(rows, weight, outs, dtype):
    av = oracle.row_values(host(rows.codes[:, :rows.cols]), host(rows.scale[:, :rows.rows]))
    wv = oracle.weight_values(host(weight.codes[:, :weight.cols]), host(weight.scale))
    got = np.concatenate([host(o).reshape(rows.rows, -1) for o in outs], axis=1)
    check_product(got, av @ wv.T, np.abs(av) @ np.abs(wv).T, rows.cols, dtype)


def check_stages(inp, s, last, x8, h, gamma, parts, o_v, o8, hidden):
    """x8 from h, the four parts from x8, o_v from the parts over the cache, o8 from o_v, hidden from o8."""
    wl, dt = inp.wl, s.dims.torch_dtype
    n = x8.rows
    check_codes(host(x8.codes[:, :x8.cols]), host(x8.scale[:, :n]), oracle.rms_norm(h, gamma, wl.eps), x8.cols)
    check_linear(x8, s.w_in, parts, dt)
    q, q_rope, c, k_rope = (host(t) for t in parts)
    inp2 = copy.copy(inp)
    inp2.c, inp2.k_rope = inp.c.copy(), inp.k_rope.copy()
    inp2.c[last], inp2.k_rope[last] = c, k_rope
    inp2.q = q.reshape(wl.batch, wl.s_q, wl.heads, wl.d_h)
    inp2.q_rope = q_rope.reshape(wl.batch, wl.s_q, wl.heads, wl.d_rope)
    ref = oracle.up_project(oracle.decode(inp2)[0], inp.w_uv).reshape(n, -1)
    o = host(o_v).reshape(n, -1)
    assert np.abs(o - ref).max() <= REL_TOL[wl.dtype] * np.abs(ref).max()
    check_codes(host(o8.codes[:, :o8.cols]), host(o8.scale[:, :n]), o, 0)
    check_linear(o8, s.w_out, [hidden], dt)


@pytest.mark.parametrize("name", sorted(CASES))
def test_session_runs_a_layer_from_hidden_states(name):
    inp, s, x, res, gamma, last = build(name)
    total = host(x) + host(res)
    s.prepare_hidden(x, inp.token_slots()[last], inp.token_positions()[last], residual=res)
    h = host(res)                                     # the residual took the sum
    assert np.all(np.abs(h - total) <= np.abs(total) * 2.0 ** -8 + 1e-30)
    o_v, _ = s.decode_up(inp.block_table, inp.seq_lens, inp.wl.s_q)
    hidden = s.project_out(o_v)
    torch.cuda.synchronize()
    assert s.device_status() == qkn.OK
    check_stages(inp, s, last, s.x8, h, gamma, (s.q, s.q_rope, s.c_new, s.k_rope_new), o_v, s.o8, hidden)


@pytest.mark.parametrize("name", sorted(CASES))
def test_layer_step_replays_on_new_inputs(name):
    inp, s, x, res, gamma, last = build(name)
    wl = inp.wl
    step = LayerStep(s, wl.batch, wl.s_q, inp.block_table.shape[1])
    fixed = {"slot": inp.token_slots()[last], "pos": inp.token_positions()[last], "block_table": inp.block_table,
             "seq_lens": inp.seq_lens}
    for k, v in fixed.items():
        step.host_in[k].copy_(torch.from_numpy(np.ascontiguousarray(v)))
    for a, r in ((res, x), (x, res)):                 # the second replay must not see the first one's values
        step.host_in["x"].copy_(a)
        step.host_in["residual"].copy_(r)
        hidden, total = step.run()
    assert s.device_status() == qkn.OK
    check_stages(inp, s, last, step.x8, host(total), gamma, (step.q, step.q_rope, step.c, step.k_rope), step.o_v,
                 step.o8, hidden)
    assert torch.equal(total, step.residual.cpu())
    # other sizes on the same session leave the captured buffers alone
    first = hidden.clone()
    s.project(x[:1])
    step.host_in["x"].copy_(x)
    again, _ = step.run()
    # (the key statistics of re-appended tokens are summed with atomics: equal up to rounding and the codes it moves)
    assert (again.float() - first.float()).abs().max() <= 2 ** -4 * first.float().abs().max()


def test_layer_calls_need_their_weights():
    inp = make_inputs(WORKLOADS["tiny_f32"])
    s = session_from_inputs(inp)
    with pytest.raises(RuntimeError):
        s.project(torch.zeros((1, 64)))
    with pytest.raises(RuntimeError):
        LayerStep(s, 1, 1, 4)
    rows = sum(s.projection_widths())
    with pytest.raises(ValueError):
        s.load_projections(torch.ones(64), torch.zeros((rows + 1, 64)))
    with pytest.raises(ValueError):
        s.load_projections(torch.ones(63), torch.zeros((rows, 64)))
    with pytest.raises(ValueError):
        s.load_projections(torch.ones(64), torch.zeros((rows, 64)), torch.zeros((64, 100)))
    s.load_projections(torch.ones(64), torch.zeros((rows, 64)))
    with pytest.raises(RuntimeError):
        s.project_out(torch.zeros((1, 4, 32), device="cuda"))
    with pytest.raises(RuntimeError):
        LayerStep(s, 1, 1, 4)
    s.project(torch.ones((2, 64)))
    assert (s.q == 0).all() and s.device_status() == qkn.OK


def test_projections_loaded_again_with_another_width():
    """The buffers follow the weights, not the number of rows alone; and an output projection whose value weights were
    replaced by others of another width is refused."""
    s = session_from_inputs(make_inputs(WORKLOADS["tiny_f32"]))
    rows, g = sum(s.projection_widths()), torch.Generator().manual_seed(5)
    heads, d_v = s.dims.num_heads, s.w_uv.shape[-1]
    for width in (64, 200, 136):
        s.load_projections(torch.ones(width), torch.randn((rows, width), generator=g),
                           torch.randn((width, heads * d_v), generator=g))
        s.project(torch.randn((2, width), generator=g))
        check_linear(s.x8, s.w_in, (s.q, s.q_rope, s.c_new, s.k_rope_new), torch.float32)
        o_v = torch.randn((2, heads, d_v), generator=g).cuda()
        hidden = s.project_out(o_v)
        assert hidden.shape == (2, width)
        check_linear(s.o8, s.w_out, [hidden], torch.float32)
    s.load_value_weights(torch.randn((heads, s.dims.r_kv, 2 * d_v), generator=g))
    with pytest.raises(ValueError):
        s.project_out(torch.randn((1, heads, 2 * d_v), generator=g).cuda())
    with pytest.raises(ValueError):
        LayerStep(s, 1, 1, 4)


def test_a_captured_layer_keeps_the_weights_of_its_capture():
    """Every weight of the session loaded again, the attention's and the projections': the graph replays with its own."""
    import weakref
    inp, s, x, res, gamma, last = build("small_mla_bf16")
    wl = inp.wl
    step = LayerStep(s, wl.batch, wl.s_q, inp.block_table.shape[1])
    fixed = {"slot": inp.token_slots()[last], "pos": inp.token_positions()[last], "block_table": inp.block_table,
             "seq_lens": inp.seq_lens}
    for k, v in fixed.items():
        step.host_in[k].copy_(torch.from_numpy(np.ascontiguousarray(v)))
    step.host_in["x"].copy_(x)
    step.host_in["residual"].copy_(res)
    first = [t.clone() for t in step.run()]
    names = ("w_k", "key_gram", "gamma_q", "gamma_k", "gamma_qr", "gamma_kr", "w_uv", "gamma_x")
    held = {k: weakref.ref(getattr(s, k)) for k in names}
    held.update({w + part: weakref.ref(getattr(getattr(s, w), part)) for w in ("w_in", "w_out")
                 for part in ("codes", "scale")})
    width, rows = s.w_in.cols, s.w_in.rows
    s.load_weights(inp.w_k * 3.0, inp.gamma_q * 0.5, inp.gamma_k + 1.0, inp.gamma_qr * 2.0, inp.gamma_kr * 2.0)
    s.load_value_weights(inp.w_uv * 2.0)
    s.load_projections(torch.ones(width), torch.zeros((rows, width)), torch.zeros((width, wl.heads * wl.d_v)))
    assert [k for k, r in held.items() if r() is None] == []
    junk = [torch.full_like(r(), 7.0) for r in held.values() for _ in range(2)]
    hidden, total = step.run()
    del junk
    assert s.device_status() == qkn.OK
    assert torch.equal(total, first[1])
    # (the key statistics are summed with atomics: equal up to rounding and the codes it moves)
    assert (hidden.float() - first[0].float()).abs().max() <= 2 ** -4 * first[0].float().abs().max()


def test_errors_that_a_step_recorded_are_the_session_s():
    """A step's status words stay visible when the session loads its projections again or grows its workspace, an
    error that nobody has read yet too, and clear_status clears them all.  (The words are written by hand.)"""
    inp, s, x, res, gamma, last = build("tiny_f32")
    step = LayerStep(s, inp.wl.batch, inp.wl.s_q, inp.block_table.shape[1])
    record = lambda w, code: w[:4].view(torch.int32).fill_(code)
    rows, width = sum(s.projection_widths()), s.w_in.cols
    w_out = torch.zeros((width, s.w_out.cols))
    record(step.proj_workspace, qkn.ERR_TIMEOUT)                 # not read yet
    s.load_projections(torch.ones(width), torch.zeros((rows, width)), w_out)
    assert s.device_status() == qkn.ERR_TIMEOUT
    s.clear_status()
    assert s.device_status() == qkn.OK
    record(step.proj_workspace, qkn.ERR_TIMEOUT)                 # recorded by the older step
    assert s.device_status() == qkn.ERR_TIMEOUT
    s.clear_status()
    before = step.workspace
    record(before, qkn.ERR_BOUNDS)
    assert s.ensure_workspace(512, 4) is not before
    assert s.device_status() == qkn.ERR_BOUNDS
    s.clear_status()
    assert s.device_status() == qkn.OK and qkn.read_device_status(before) == qkn.OK
    record(step.workspace, qkn.ERR_TIMEOUT)
    assert s.device_status() == qkn.ERR_TIMEOUT
    s.clear_status()
    del step, before
    assert s.device_status() == qkn.OK


def test_a_workspace_outgrown_inside_a_capture_is_not_read_by_the_replays():
    s = session_from_inputs(make_inputs(WORKLOADS["tiny_f32"]))
    s.ensure_workspace(1, 1)
    size = s.workspace.numel()
    s.workspace[:4].view(torch.int32).fill_(qkn.ERR_BOUNDS)      # recorded, and not read yet
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.ensure_workspace(512, 4)
    assert s.workspace.numel() > size
    junk = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    graph.replay()
    torch.cuda.synchronize()
    del junk
    assert s.device_status() == qkn.ERR_BOUNDS
    s.clear_status()
    assert s.device_status() == qkn.OK
    graph.replay()
    assert s.device_status() == qkn.OK


def test_session_calls_in_a_graph_of_the_caller_s():
    """The session's calls captured by the caller, then other sizes, other weights and a larger workspace on the
    session: the graph replays with what it captured, and none of that went back to the allocator."""
    import weakref
    inp, s, x, res, gamma, last = build("small_mla_bf16")
    wl = inp.wl
    slot, pos = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in
                 (inp.token_slots()[last].astype(np.int32), inp.token_positions()[last].astype(np.int32)))
    bt, sl = torch.from_numpy(inp.block_table).cuda(), torch.from_numpy(inp.seq_lens).cuda()

    def layer():
        s.prepare_hidden(x, slot, pos)
        return s.project_out(s.decode_up(bt, sl, wl.s_q)[0])

    want = layer().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hidden = layer()
    names = ("w_k", "key_gram", "gamma_q", "gamma_k", "gamma_qr", "gamma_kr", "w_uv", "gamma_x", "q", "q_rope", "c_new",
             "k_rope_new", "q_tilde", "a_q", "q_rope_hat", "workspace")
    held = {k: weakref.ref(getattr(s, k)) for k in names}
    held.update({w + part: weakref.ref(getattr(getattr(s, w), part)) for w in ("w_in", "w_out", "x8", "o8")
                 for part in ("codes", "scale")})
    width, rows = s.w_in.cols, s.w_in.rows
    s.load_weights(inp.w_k * 3.0, inp.gamma_q * 0.5, inp.gamma_k + 1.0, inp.gamma_qr * 2.0, inp.gamma_kr * 2.0)
    s.load_value_weights(inp.w_uv * 2.0)
    s.load_projections(torch.ones(width), torch.zeros((rows, width)), torch.zeros((width, wl.heads * wl.d_v)))
    s.ensure_query_buffers(1)
    s.project(x[:1])
    s.ensure_workspace(512, 4)
    assert [k for k, r in held.items() if r() is None] == []
    hidden.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert s.device_status() == qkn.OK
    # (the key statistics are summed with atomics: equal up to rounding and the codes it moves)
    assert (hidden.float() - want.float()).abs().max() <= 2 ** -4 * want.float().abs().max()


class _Broken:
    """Weights whose shape is right and whose values cannot be had."""

    def __init__(self, shape):
        self.shape = shape

    def __array__(self, *args, **kwargs):
        raise OSError("unreadable")


def test_projections_that_fail_to_load_leave_the_old_ones():
    inp, s, x, res, gamma, last = build("tiny_f32")
    want = [t.clone() for t in s.project(x)]
    rows, width = sum(s.projection_widths()), 64
    before = (s.gamma_x, s.w_in, s.w_out)
    with pytest.raises(OSError):
        s.load_projections(torch.ones(width), torch.zeros((rows, width)), _Broken((width, s.w_out.cols)))
    assert all(a is b for a, b in zip(before, (s.gamma_x, s.w_in, s.w_out)))
    for a, b in zip(s.project(x), want):
        assert torch.equal(a, b)
