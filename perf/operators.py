"""Workloads and plain forms of the 8-bit projections around the latent decode.

A decode step starts from hidden states and ends in them.  Three operators carry it between the two
and the attention: the norm in front of a projection, with the residual's addition and an output in
8 bits (``norm``), the projection itself, an fp8 product with a scale for every block of 128
(``linear``), and the quantisation of its weights when a model is loaded (``weight``).

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits; with ``own``
true it calls the library.  The numbers are the same in both:

* rows in 8 bits: codes e4m3 [n, ld], ld a multiple of 16, and scales fp32 [ceil(d / 128), lds], lds
  a multiple of 4: the value of element (i, j) is codes[i, j] * scale[j // 128, i];
* weights in 8 bits: codes e4m3 [n, ld] and scales fp32 [ceil(n / 128), ceil(k / 128)], one for each
  block of 128 x 128;
* a scale is max(largest magnitude / 448, 2^-100), a code its value over the scale, rounded to e4m3.
"""
import math

import torch

own = False

GROUP = 128           # columns (and, for weights, rows) that share a scale
TOP = 448.0           # the largest e4m3 value
LEAST = 2.0 ** -100   # the least scale
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# hidden -> queries of 128 heads (128 + 64 wide), the latent and the RoPE key
STEP_128 = "16384,8192,512,64"


def listed():
    return [
        # the norm in front of the projections: one sequence's new token, a batch's, a long prompt's
        {"name": "norm_one_token", "op": "norm", "n": 1, "d": 2048, "type": "bf16", "residual": True, "gamma": True, "y": False},
        {"name": "norm_step_32", "op": "norm", "n": 32, "d": 4096, "type": "bf16", "residual": True, "gamma": True, "y": False},
        {"name": "norm_prompt_16k", "op": "norm", "n": 16384, "d": 4096, "type": "bf16", "residual": True, "gamma": True, "y": False},
        # the attention's output in front of the output projection: 128 heads of 128, no norm
        {"name": "quant_heads_out", "op": "norm", "n": 1021, "d": 16384, "type": "bf16", "residual": False, "gamma": False, "y": False},
        # fp32 activations, a width that no group of 128 divides, the normalised row wanted too
        {"name": "norm_f32_ragged", "op": "norm", "n": 777, "d": 5000, "type": "f32", "residual": True, "gamma": True, "y": True},
        # weights at load time: the latent's and RoPE key's down-projection, and a whole step's
        {"name": "weight_latent", "op": "weight", "n": 576, "k": 2048, "type": "f32"},
        {"name": "weight_step_128h", "op": "weight", "n": 25152, "k": 4096, "type": "bf16"},
        # the latent and RoPE key of one new token: a few microseconds, latency counts
        {"name": "linear_latent_one", "op": "linear", "m": 1, "k": 2048, "segs": "512,64"},
        # a decode step of 32 sequences at 128 heads: the weights' bytes count
        {"name": "linear_step_32", "op": "linear", "m": 32, "k": 4096, "segs": STEP_128},
        # a chunk of a prompt with sizes that no tile divides
        {"name": "linear_ragged", "op": "linear", "m": 333, "k": 1960, "segs": "904,96"},
        # the output projection of a chunk, and a prompt's projections: the tensor cores count
        {"name": "linear_out_4k", "op": "linear", "m": 4096, "k": 16384, "segs": "4096"},
        {"name": "linear_prompt_8k", "op": "linear", "m": 8192, "k": 4096, "segs": STEP_128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "weight", "linear", "linear", "linear"])
    if op == "norm":
        d = _log(rng, 64, 16384)
        d -= d % rng.choice([1, 8, 64])
        n = _log(rng, 1, min(16384, (1 << 26) // d))
        gamma = rng.random() < 0.8
        return {"op": op, "n": n, "d": d, "type": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.random() < 0.7, "gamma": gamma, "y": gamma and rng.random() < 0.3}
    if op == "weight":
        k = _log(rng, 64, 16384)
        k -= k % rng.choice([1, 8, 64])
        return {"op": op, "n": _log(rng, 64, min(25152, (25152 << 12) // k)), "k": k, "type": rng.choice(["bf16", "f32"])}
    m = _log(rng, 1, 8192)
    k = _log(rng, 128, 16384)
    k -= k % rng.choice([1, 16, 128])
    n = _log(rng, 64, min(25152, (8192 * 25152 * 4096) // (m * k), (25152 << 13) // m, (25152 << 12) // k))
    n -= n % rng.choice([1, 8, 64])
    cuts = sorted(rng.sample(range(1, n), rng.choice([0, 0, 1, 3])))
    if rng.random() < 0.7:  # segments of whole 16-byte pieces, as heads and latents are
        cuts = sorted({max(8, c - c % 8) for c in cuts if c >= 8 and c - c % 8 < n})
    return {"op": op, "m": m, "k": k, "segs": ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [n]))}


def _pad(v, to):
    return -(-v // to) * to


def _widths(case):
    return list(map(int, case["segs"].split(",")))


def _quant_rows(y):
    """fp32 [n, d] -> codes [n, ceil(d / 128) * 128] and scales [n, ceil(d / 128)]."""
    n, d = y.shape
    g = torch.nn.functional.pad(y, (0, _pad(d, GROUP) - d)).view(n, -1, GROUP)
    scale = (g.abs().amax(-1) / TOP).clamp_min(LEAST)
    return (g / scale[..., None]).to(torch.float8_e4m3fn).view(n, -1), scale


def _blocks(w):
    """[n, k] -> [ceil(n / 128), 128, ceil(k / 128), 128], zeros behind the edges."""
    n, k = w.shape
    p = torch.nn.functional.pad(w, (0, _pad(k, GROUP) - k, 0, _pad(n, GROUP) - n))
    return p.view(_pad(n, GROUP) // GROUP, GROUP, -1, GROUP)


def _quant_weight(w):
    """fp32 [n, k] -> codes [n, k] and scales of the blocks."""
    n, k = w.shape
    b = _blocks(w)
    scale = (b.abs().amax((1, 3)) / TOP).clamp_min(LEAST)
    codes = (b / scale[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.reshape(_pad(n, GROUP), -1)[:n, :k], scale


def _padded(codes, ld):
    out = torch.zeros((codes.shape[0], ld), dtype=torch.float8_e4m3fn, device=codes.device)
    out.view(torch.uint8)[:, :codes.shape[1]] = codes.view(torch.uint8)
    return out


def _activations(gen, n, d):
    """Hidden states: a magnitude of its own for each token, and one channel in 64 far larger."""
    x = torch.randn((n, d), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((n, 1), generator=gen, device="cuda"))
    return x * torch.where(torch.rand((1, d), generator=gen, device="cuda") < 1 / 64, 12.0, 1.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    state = dict(case)
    if case["op"] == "norm":
        dt = TYPES[case["type"]]
        state["x"] = _activations(gen, case["n"], case["d"]).to(dt)
        state["res"] = (2 * _activations(gen, case["n"], case["d"])).to(dt) if case["residual"] else None
        state["g"] = 1 + 0.1 * torch.randn(case["d"], generator=gen, device="cuda") if case["gamma"] else None
    elif case["op"] == "weight":
        w = torch.randn((case["n"], case["k"]), generator=gen, device="cuda") / math.sqrt(case["k"])
        state["w"] = w.to(TYPES[case["type"]])
    else:
        m, k, n = case["m"], case["k"], sum(_widths(case))
        codes, scale = _quant_rows(_activations(gen, m, k))
        state["a"] = _padded(codes[:, :k], _pad(k, 16))
        state["a_scale"] = torch.zeros((scale.shape[1], _pad(m, 4)), device="cuda")
        state["a_scale"][:, :m] = scale.t()
        codes, state["w_scale"] = _quant_weight(torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k))
        state["w"] = _padded(codes, _pad(k, 16))
        state["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return state


def _run_own(s):
    import qk_normed_latent_qkn_b200 as qkn
    if s["op"] == "norm":
        n, d, x = s["n"], s["d"], s["x"]
        q = qkn.Fp8Rows.empty(n, d, x.device)
        h = torch.empty_like(x) if s["residual"] else None
        y = torch.empty_like(x) if s["y"] else None
        qkn.norm_quant(x, q, gamma=s["g"], eps=EPS, residual=s["res"], residual_out=h, y=y)
        return {"codes": q.codes[:, :d], "scale": q.scale[:, :n], "residual": h, "y": y}
    if s["op"] == "weight":
        q = qkn.Fp8Weight.empty(s["n"], s["k"], s["w"].device)
        qkn.quant_weight(s["w"], q)
        return {"codes": q.codes[:, :s["k"]], "scale": q.scale}
    a = qkn.Fp8Rows(s["a"], s["a_scale"], s["k"])
    w = qkn.Fp8Weight(s["w"], s["w_scale"], s["k"])
    outs = [torch.empty((s["m"], c), dtype=torch.bfloat16, device=s["a"].device) for c in _widths(s)]
    qkn.fp8_linear(a, w, outs, s["workspace"])
    return outs


def _values(s, to):
    """The values of a product's operands, [m, k] and [n, k]."""
    k = s["k"]
    a = s["a"][:, :k].to(to) * s["a_scale"][:, :s["m"]].t().to(to).repeat_interleave(GROUP, 1)[:, :k]
    n = s["w"].shape[0]
    per = s["w_scale"].to(to).repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)[:, :k]
    return a, s["w"][:, :k].to(to) * per


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm":
        d, dt = s["d"], s["x"].dtype
        h = s["x"].float()
        if s["residual"]:
            h = (h + s["res"].float()).to(dt).float()
        y = h
        if s["gamma"]:
            y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["g"]
        codes, scale = _quant_rows(y)
        return {"codes": codes[:, :d], "scale": scale.t(), "residual": h.to(dt) if s["residual"] else None,
                "y": y.to(dt) if s["y"] else None}
    if s["op"] == "weight":
        codes, scale = _quant_weight(s["w"].float())
        return {"codes": codes, "scale": scale}
    a, w = _values(s, torch.float32)
    return list(torch.split((a @ w.t()).to(torch.bfloat16), _widths(s), dim=1))


def work(case):
    if case["op"] == "norm":
        n, d, e = case["n"], case["d"], 2 if case["type"] == "bf16" else 4
        arrays = 1 + 2 * case["residual"] + case["y"]
        return {"bytes": n * d * (e * arrays + 1) + n * -(-d // GROUP) * 4 + 4 * d * case["gamma"], "flops": 8 * n * d}
    if case["op"] == "weight":
        n, k, e = case["n"], case["k"], 2 if case["type"] == "bf16" else 4
        return {"bytes": n * k * (e + 1) + -(-n // GROUP) * -(-k // GROUP) * 4, "flops": 3 * n * k}
    m, k, n = case["m"], case["k"], sum(_widths(case))
    groups = -(-k // GROUP)
    return {"bytes": m * k + n * k + 4 * groups * (m + -(-n // GROUP)) + 2 * m * n, "flops": 2 * m * n * k}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits and unrounded (the residual's sum, which the
    norm reads as it is stored, is rounded where it is read)."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        k = case["k"]
        of = torch.arange(k, device="cuda") // GROUP
        a = s["a"][:, :k].double() * s["a_scale"].double()[of, :case["m"]].t()
        w = s["w"][:, :k].double()
        w *= s["w_scale"].double()[torch.arange(w.shape[0], device="cuda") // GROUP][:, of]
        out, at = [], 0
        for c in _widths(case):
            out.append(a @ w[at:at + c].t())
            at += c
        return out
    if case["op"] == "norm":
        h = s["x"].double()
        total = None
        if case["residual"]:
            total = h + s["res"].double()
            h = total.to(s["x"].dtype).double()
        y = h
        if case["gamma"]:
            y = h / (h.pow(2).sum(1, keepdim=True) / case["d"] + EPS).sqrt() * s["g"].double()
        d, groups = case["d"], -(-case["d"] // GROUP)
        scale = torch.stack([y[:, g * GROUP:(g + 1) * GROUP].abs().max(1).values for g in range(groups)]) / TOP
        scale = torch.maximum(scale, torch.full_like(scale, LEAST))
        codes = y / scale[torch.arange(d, device="cuda") // GROUP].t()
        return {"codes": codes, "scale": scale, "residual": total, "y": y if case["y"] else None}
    w = s["w"].double()
    n, k = w.shape
    rows = torch.arange(n, device="cuda") // GROUP
    cols = torch.arange(k, device="cuda") // GROUP
    tall = torch.zeros((-(-n // GROUP), k), dtype=torch.float64, device="cuda")
    tall.scatter_reduce_(0, rows[:, None].expand(n, k), w.abs(), "amax")
    scale = torch.zeros((tall.shape[0], -(-k // GROUP)), dtype=torch.float64, device="cuda")
    scale.scatter_reduce_(1, cols[None].expand(tall.shape[0], k), tall, "amax")
    scale = torch.maximum(scale / TOP, torch.full_like(scale, LEAST))
    return {"codes": w / scale[rows][:, cols], "scale": scale}
