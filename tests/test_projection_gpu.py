"""The 8-bit projections on the GPU against their definitions in 64 bits.

Tolerances, from the roundings alone (u = 2^-24, half a step of fp32):
  * h: the fp32 sum and its rounding to the storage type: |h64| (2^-8 + u) in bf16, |h64| u in fp32;
  * scale: a sum of d squares in a tree of at most d / 256 + 32 additions in a row (half of its relative
    error after the square root), the root, the divisions and the products: (d / 256 + 40) u;
  * a code: half a step of e4m3 (2^-4 of the value, 2^-10 below the normal range) around y / scale, whose
    own error is at most the scale's and the reciprocal's (another d / 256 + 48 units);
  * a product: every addition within a block may lose up to one unit of fp32 (2 u) of the block's sum of
    magnitudes, every block's entry into the total u: (2 * 128 + blocks + 4) u sum|a||w|, and half a step
    of bf16 (2^-8) of the result.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import qk_normed_latent_qkn_b200 as qkn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DTYPES = [torch.bfloat16, torch.float32]


def host(t):
    return t.detach().double().cpu().numpy()


def hidden(n, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g) * torch.exp(0.5 * torch.randn((n, 1), generator=g))
    return (x * torch.where(torch.rand((1, d), generator=g) < 1 / 64, 12.0, 1.0)).to(dtype).cuda()


def check_codes(codes, scale, y, d_chain):
    """codes [n, d] and scale [g, n] on the host against y [n, d] in 64 bits."""
    ratio, want = oracle.quant_rows(y)
    tol = (d_chain // 256 + 40) * U
    assert np.abs(scale / want - 1).max() <= tol
    slack = (2 * tol + 8 * U) * np.abs(ratio)
    assert np.all(np.abs(codes - ratio) <= np.maximum(np.abs(ratio) * 2.0 ** -4, 2.0 ** -10) + slack)


def run_norm(x, gamma=None, residual=None, want_y=False, eps=1e-6, inplace=False):
    n, d = x.shape
    q = qkn.Fp8Rows.empty(n, d)
    q.codes.view(torch.uint8).fill_(0x35)
    q.scale.fill_(-7.0)
    h = None if residual is None else (residual if inplace else torch.empty_like(residual))
    y = torch.empty((n, d), dtype=x.dtype, device="cuda") if want_y else None
    qkn.norm_quant(x, q, gamma=gamma, eps=eps, residual=residual, residual_out=h, y=y)
    torch.cuda.synchronize()
    # nothing behind a row's codes or a block's scales is written
    assert (q.codes.view(torch.uint8)[:, d:] == 0x35).all() and (q.scale[:, n:] == -7.0).all()
    return q, h, y


SHAPES = [(1, 1), (1, 2048), (3, 64), (2, 127), (5, 128), (4, 129), (7, 136), (33, 4096), (9, 5000), (130, 1000),
          (2, 16384), (3, 32768), (2, 32776), (2, 40001), (257, 576)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("form", ["norm", "residual", "plain", "sum"])
def test_norm_quant(n, d, dtype, form):
    x = hidden(n, d, dtype, seed=n * 7 + d)
    res = hidden(n, d, dtype, seed=n + d * 3 + 1) * 2 if form in ("residual", "sum") else None
    gamma = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(d))).cuda() if form in (
        "norm", "residual") else None
    q, h, y = run_norm(x, gamma, res, want_y=gamma is not None)
    h64 = host(x)
    if res is not None:
        total = host(x) + host(res)
        h64 = host(h)
        assert np.all(np.abs(h64 - total) <= np.abs(total) * (HALF_STEP[dtype] + U) + 1e-40)
    y64 = h64 if gamma is None else oracle.rms_norm(h64, host(gamma), 1e-6)
    check_codes(host(q.codes[:, :d]), host(q.scale[:, :n]), y64, d if gamma is not None else 0)
    if y is not None:
        assert np.all(np.abs(host(y) - y64) <= np.abs(y64) * (HALF_STEP[dtype] + (d // 256 + 40) * U))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [512, 500, 40001])
def test_norm_quant_in_place_and_strided_rows(dtype, d):
    """The sum may be written over the residual or over x, and x may be a slice of wider rows; unaligned rows
    take the same values."""
    n = 6
    x, res = hidden(n, d, dtype, 1), hidden(n, d, dtype, 2)
    gamma = torch.ones(d, device="cuda")
    ref, h, _ = run_norm(x, gamma, res.clone())
    q, h2, _ = run_norm(x, gamma, res.clone(), inplace=True)
    assert torch.equal(h, h2) and torch.equal(ref.codes.view(torch.uint8)[:, :d], q.codes.view(torch.uint8)[:, :d])
    xx = x.clone()
    q = qkn.Fp8Rows.empty(n, d)
    qkn.norm_quant(xx, q, gamma=gamma, residual=res, residual_out=xx)
    assert torch.equal(xx, h) and torch.equal(ref.scale[:, :n], q.scale[:, :n])
    xx = x.clone()
    q1, q2 = qkn.Fp8Rows.empty(n, d), qkn.Fp8Rows.empty(n, d)
    qkn.norm_quant(x, q1, gamma=gamma)
    qkn.norm_quant(xx, q2, gamma=gamma, y=xx)
    assert torch.equal(q1.scale[:, :n], q2.scale[:, :n])
    assert torch.equal(q1.codes.view(torch.uint8)[:, :d], q2.codes.view(torch.uint8)[:, :d])
    for off in (1, 8):          # a slice of wider rows, off the 16-byte grid and on it
        wide = torch.full((n, d + 24), 9.0, dtype=dtype, device="cuda")
        wide[:, off:off + d] = x
        q3, _, _ = run_norm(wide[:, off:off + d], gamma)
        y64 = oracle.rms_norm(host(x), host(gamma), 1e-6)
        check_codes(host(q3.codes[:, :d]), host(q3.scale[:, :n]), y64, d)


def shifted(t, by):
    """A dense copy of t that starts ``by`` elements behind an aligned address."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    flat[by:] = t.reshape(-1)
    return flat[by:].view(t.shape)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("by", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("n,d", [(3, 264), (600, 1000), (2, 20000)])
def test_unaligned_bases(n, d, by, dtype):
    """Every array of a call starts off the 16-byte grid, by amounts of their own."""
    x, res = hidden(n, d, dtype, by), hidden(n, d, dtype, by + 1)
    gamma = shifted((1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(by))).cuda(), by)
    q = qkn.Fp8Rows.empty(n, d)
    h, y = shifted(torch.zeros_like(x), by), shifted(torch.zeros_like(x), by + 2)
    qkn.norm_quant(shifted(x, by + 1), q, gamma=gamma, residual=shifted(res, by + 3), residual_out=h, y=y)
    total = host(x) + host(res)
    assert np.all(np.abs(host(h) - total) <= np.abs(total) * (HALF_STEP[dtype] + U) + 1e-40)
    y64 = oracle.rms_norm(host(h), host(gamma), 1e-6)
    check_codes(host(q.codes[:, :d]), host(q.scale[:, :n]), y64, d)
    assert np.all(np.abs(host(y) - y64) <= np.abs(y64) * (HALF_STEP[dtype] + (d // 256 + 40) * U))
    w, w1 = qkn.Fp8Weight.empty(n, d), qkn.Fp8Weight.empty(n, d)
    qkn.quant_weight(x, w)
    qkn.quant_weight(shifted(x, by), w1)
    assert torch.equal(w.scale, w1.scale) and torch.equal(w.codes.view(torch.uint8)[:, :d], w1.codes.view(torch.uint8)[:, :d])


@pytest.mark.parametrize("d", [256, 250])
def test_norm_quant_of_zeros_infinities_and_nan(d):
    """A zero row has zero codes and the least scale; a NaN or an infinity spoils its block (with gamma, its row)
    and no other row."""
    x = hidden(5, d, torch.float32, 5)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 1e-36
    q, _, _ = run_norm(x)
    v = oracle.row_values(host(q.codes[:, :d]), host(q.scale[:, :5]))
    assert (v[1] == 0).all() and (host(q.scale)[:, 1] == 2.0 ** -100).all()
    assert np.isnan(v[2, :128]).all() and np.isfinite(v[2, 128:]).all()
    assert np.isnan(v[3, 128:]).all() and np.isfinite(v[3, :128]).all()
    ratio, _ = oracle.quant_rows(host(x[4:]))
    assert np.abs(host(q.codes)[4, :d] - oracle.e4m3_round(ratio)[0]).max() == 0
    assert np.isfinite(v[0]).all()
    q, _, _ = run_norm(x, torch.ones(d, device="cuda"))
    v = oracle.row_values(host(q.codes[:, :d]), host(q.scale[:, :5]))
    assert (v[1] == 0).all() and np.isnan(v[2]).all() and np.isnan(v[3, 128:]).all()
    assert np.isfinite(v[[0, 4]]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(1, 1), (64, 512), (128, 128), (129, 130), (576, 2048), (200, 1000), (300, 77), (7, 4104)])
def test_quant_weight(n, k, dtype):
    w = (torch.randn((n, k), generator=torch.Generator().manual_seed(n + k)) / k ** 0.5).to(dtype).cuda()
    q = qkn.Fp8Weight.empty(n, k)
    q.codes.view(torch.uint8).fill_(0x35)
    qkn.quant_weight(w, q)
    ratio, want = oracle.quant_weight(host(w))
    assert np.abs(host(q.scale) / want - 1).max() <= 2 * U
    slack = 8 * U * np.abs(ratio)
    assert np.all(np.abs(host(q.codes[:, :k]) - ratio) <= np.maximum(np.abs(ratio) * 2.0 ** -4, 2.0 ** -10) + slack)
    assert (q.codes.view(torch.uint8)[:, k:] == 0x35).all()


def test_quant_weight_keeps_nan_in_its_block():
    w = torch.randn((256, 256), device="cuda")
    w[130, 5] = float("nan")
    w[3, 250] = float("inf")
    q = qkn.Fp8Weight.empty(256, 256)
    qkn.quant_weight(w, q)
    v = oracle.weight_values(host(q.codes), host(q.scale))
    assert np.isnan(v[128:, :128]).all() and np.isnan(v[:128, 128:]).all()
    assert np.isfinite(v[:128, :128]).all() and np.isfinite(v[128:, 128:]).all()


# ---------------------------------------------------------------- the product
def operands(m, n, k, seed=0, pad=0):
    """Codes and scales of rows and a weight; what lies behind the edges is poisoned with NaN codes."""
    x = hidden(m, k, torch.float32, seed)
    a = qkn.Fp8Rows.empty(m, k)
    if pad:
        a = qkn.Fp8Rows(torch.empty((m, a.codes.shape[1] + pad), dtype=torch.float8_e4m3fn, device="cuda"), a.scale, k)
    a.codes.view(torch.uint8).fill_(0x7F)
    a.scale.fill_(float("nan"))
    qkn.norm_quant(x, a)
    w32 = (torch.randn((n, k), generator=torch.Generator().manual_seed(seed + 1)) / k ** 0.5).cuda()
    w = qkn.Fp8Weight.empty(n, k)
    w.codes.view(torch.uint8).fill_(0x7F)
    qkn.quant_weight(w32, w)
    return a, w


def product(a, w):
    m, n, k = a.rows, w.rows, a.cols
    av = oracle.row_values(host(a.codes[:, :k]), host(a.scale[:, :m]))
    wv = oracle.weight_values(host(w.codes[:, :k]), host(w.scale))
    return av @ wv.T, np.abs(av) @ np.abs(wv).T


def check_product(out, ref, mag, k, dtype):
    tol = (2 * 128 + (k + 127) // 128 + 4) * U * mag
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    err = np.abs(out - ref)
    assert np.isfinite(out).all()
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3f} of the tolerance"


def workspace():
    ws = torch.empty(qkn.WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    qkn.workspace_init(ws)
    return ws


LINEAR = [  # m, n, k, widths
    (1, 1, 1, [1]), (1, 576, 2048, [512, 64]), (2, 64, 128, [64]), (16, 130, 256, [130]), (17, 128, 384, [1, 127]),
    (5, 7, 77, [3, 4]), (31, 1000, 1960, [904, 96]), (33, 257, 144, [257]), (64, 640, 4096, [512, 64, 64]),
    (65, 384, 1000, [384]), (100, 2000, 130, [1000, 1000]), (128, 512, 512, [512]), (129, 264, 640, [8, 256]),
    (200, 1029, 900, [5, 1024]), (256, 256, 128, [256]), (300, 700, 3000, [700]), (333, 1000, 1960, [904, 96]),
    (513, 1536, 512, [1024, 8, 504]), (1000, 3333, 260, [1111, 1111, 1111]), (2049, 520, 256, [520]),
    (4, 4096, 16384, [4096]), (48, 12288, 512, [8192, 4096]), (1, 25152, 640, [16384, 8192, 512, 64]),
    (700, 2560, 128, [320] * 8),
    # several tiles for every pair of CTAs, of 256 columns (three waves) and of 128 (two)
    (2049, 5000, 300, [4000, 1000]), (700, 6200, 300, [6200]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k,widths", LINEAR)
def test_fp8_linear(m, n, k, widths, dtype):
    a, w = operands(m, n, k, seed=m + n + k)
    outs = [torch.full((m, c), float("nan"), dtype=dtype, device="cuda") for c in widths]
    ws = workspace()
    qkn.fp8_linear(a, w, outs, ws)
    torch.cuda.synchronize()
    assert qkn.read_device_status(ws) == qkn.OK
    ref, mag = product(a, w)
    check_product(np.concatenate([host(o) for o in outs], axis=1), ref, mag, k, dtype)


@pytest.mark.parametrize("m", [3, 40, 300])
def test_fp8_linear_strides_and_alignment(m):
    """Outputs as slices of wider buffers at odd places, codes with a longer row: what lies around stays."""
    n, k = 520, 400
    a, w = operands(m, n, k, seed=9, pad=48)
    ref, mag = product(a, w)
    for dtype in DTYPES:
        for off, widths in ((0, [520]), (1, [260, 260]), (3, [8, 509, 3]), (8, [512, 8])):
            bufs = [torch.full((m, c + 16), 5.0, dtype=dtype, device="cuda") for c in widths]
            qkn.fp8_linear(a, w, [b[:, off:off + c] for b, c in zip(bufs, widths)], workspace())
            got = np.concatenate([host(b[:, off:off + c]) for b, c in zip(bufs, widths)], axis=1)
            check_product(got, ref, mag, k, dtype)
            for b, c in zip(bufs, widths):
                assert (b[:, :off] == 5.0).all() and (b[:, off + c:] == 5.0).all()


@pytest.mark.parametrize("m,n,k", [(3, 700, 4096), (300, 520, 640), (700, 2560, 384)])
def test_fp8_linear_repeats_bit_for_bit_and_keeps_nan_in_its_row(m, n, k):
    a, w = operands(m, n, k, seed=2)
    a.scale[1, 1] = float("nan")
    outs = [torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    ws = workspace()
    for o in outs:
        qkn.fp8_linear(a, w, [o], ws)
    bits = [o.view(torch.int16) for o in outs]
    assert torch.equal(bits[0], bits[1]) and torch.equal(bits[0], bits[2])
    assert torch.isnan(outs[0][1]).all() and torch.isfinite(outs[0][0]).all() and torch.isfinite(outs[0][2:]).all()


@pytest.mark.parametrize("m,n,k", [(1, 576, 2048), (32, 2000, 1024), (333, 1000, 1960), (1024, 2560, 512)])
def test_norm_and_product_captured_replayed_and_on_two_streams(m, n, k):
    """The pair in a CUDA graph over fixed buffers, replayed on new inputs, and two at once on two streams that
    share a workspace: the same bits as one after the other."""
    gamma = torch.ones(k, device="cuda")
    w = operands(1, n, k, seed=3)[1]
    ws = workspace()

    def buffers():
        return (hidden(m, k, torch.bfloat16, 0), qkn.Fp8Rows.empty(m, k),
                torch.empty((m, n), dtype=torch.bfloat16, device="cuda"))

    def run(b):
        qkn.norm_quant(b[0], b[1], gamma=gamma)
        qkn.fp8_linear(b[1], w, [b[2]], ws)

    xs = [hidden(m, k, torch.bfloat16, s) for s in range(3)]
    want = []
    b = buffers()
    for x in xs:
        b[0].copy_(x)
        run(b)
        want.append(b[2].clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b)
    for x, o in zip(xs, want):
        b[0].copy_(x)
        b[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b[2], o)
    pairs = [(torch.cuda.Stream(), buffers()) for _ in range(3)]
    for (st, p), x in zip(pairs, xs):
        p[0].copy_(x)
    torch.cuda.synchronize()
    for _ in range(5):
        for st, p in pairs:
            with torch.cuda.stream(st):
                run(p)
    torch.cuda.synchronize()
    for (st, p), o in zip(pairs, want):
        assert torch.equal(p[2], o)
    assert qkn.read_device_status(ws) == qkn.OK


@pytest.mark.parametrize("m,n,k", [(1, 576, 2048), (40, 9472, 512), (100, 2000, 1024), (333, 1000, 1960),
                                   (600, 9472, 1024), (4096, 1024, 512)])
def test_one_buffer_rewritten_between_back_to_back_products(m, n, k):
    """Norm and product in a chain with nothing else on the stream, the rows in 8 bits (and the weight) in one
    buffer that every pair rewrites: each kernel starts while the one before it runs, and must see its values."""
    rounds = 12
    xs = [hidden(m, k, torch.bfloat16, s) * 2.0 ** (s % 5) for s in range(rounds)]
    ws_ = [(torch.randn((n, k), generator=torch.Generator().manual_seed(s)) * 2.0 ** (s % 3)).cuda() for s in range(3)]
    gamma = torch.ones(k, device="cuda")
    ws = workspace()

    def chain(sync):
        q, w = qkn.Fp8Rows.empty(m, k), qkn.Fp8Weight.empty(n, k)
        outs = [torch.empty((m, n), dtype=torch.float32, device="cuda") for _ in range(rounds)]
        torch.cuda.synchronize()
        for i in range(rounds):
            if i % 4 == 0:
                qkn.quant_weight(ws_[i // 4], w)
            qkn.norm_quant(xs[i], q, gamma=gamma if i % 2 else None)
            if sync:
                torch.cuda.synchronize()
            qkn.fp8_linear(q, w, [outs[i]], ws)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    want = chain(True)
    for _ in range(4):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)
    assert qkn.read_device_status(ws) == qkn.OK


def test_first_calls_of_a_process_may_be_captured():
    """What the library sets up once per kernel and device happens inside a capture too."""
    code = """
import torch
import qk_normed_latent_qkn_b200 as qkn
torch.manual_seed(0)
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
w = qkn.Fp8Weight(torch.randn((576, 1024), device="cuda").to(torch.float8_e4m3fn), torch.rand((5, 8), device="cuda"), 1024)
jobs = []
for m in (1, 20, 50, 100, 600, 9000):
    x, q = torch.randn((m, 1024), device="cuda"), qkn.Fp8Rows.empty(m, 1024)
    jobs.append((x, q, torch.zeros((m, 576), device="cuda")))
def run():
    for x, q, out in jobs:
        qkn.norm_quant(x, q)
        qkn.fp8_linear(q, w, [out], ws)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
first = [o.clone() for _, _, o in jobs]
run()
torch.cuda.synchronize()
assert all(torch.equal(a, o) and a.abs().sum() > 0 for a, (_, _, o) in zip(first, jobs))
assert qkn.read_device_status(ws) == qkn.OK
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)


def test_calls_on_a_given_stream():
    """``stream`` names the stream; the work waits for what is enqueued there and for nothing else."""
    m, n, k = 40, 300, 512
    a, w = operands(m, n, k, seed=6)
    want = torch.empty((m, n), dtype=torch.float32, device="cuda")
    ws = workspace()
    qkn.fp8_linear(a, w, [want], ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    x = hidden(m, k, torch.float32, 6)
    late = torch.zeros_like(x)
    q, out = qkn.Fp8Rows.empty(m, k), torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    qkn.norm_quant(late, q, stream=st)
    qkn.fp8_linear(q, w, [out], ws, stream=st)
    st.synchronize()
    assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """Rows so far apart that element and byte offsets pass 2^31 and 2^32."""
    m, k, n, ld = 70000, 128, 64, 65536
    w = operands(1, n, k, seed=7)[1]
    wide = torch.empty((m, ld), dtype=torch.float8_e4m3fn, device="cuda")        # 4.6e9 codes
    x = hidden(m, k, torch.bfloat16, 7)
    buf = torch.empty((m, ld // 2), dtype=torch.bfloat16, device="cuda")         # 2.3e9 elements
    far, out = buf[:, 1000:1000 + k], buf[:, 2000:2000 + n]
    far.copy_(x)
    q = qkn.Fp8Rows(wide, torch.empty((1, m), dtype=torch.float32, device="cuda"), k)
    qkn.norm_quant(far, q)
    qkn.fp8_linear(q, w, [out], workspace())
    torch.cuda.synchronize()
    for rows in (slice(0, 300), slice(m - 300, m)):
        codes, scale = host(wide[rows, :k]), host(q.scale[:, rows])
        check_codes(codes, scale, host(x[rows]), 0)
        av, wv = oracle.row_values(codes, scale), oracle.weight_values(host(w.codes[:, :k]), host(w.scale))
        check_product(host(out[rows]), av @ wv.T, np.abs(av) @ np.abs(wv).T, k, torch.bfloat16)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_on_another_device_than_the_current_one():
    a, w = operands(40, 300, 512, seed=8)
    want = torch.empty((40, 300), device="cuda")
    qkn.fp8_linear(a, w, [want], workspace())
    other = torch.device("cuda", 1)
    a1 = qkn.Fp8Rows(a.codes.to(other), a.scale.to(other), a.cols)
    w1 = qkn.Fp8Weight(w.codes.to(other), w.scale.to(other), w.cols)
    out = torch.empty((40, 300), device=other)
    qkn.fp8_linear(a1, w1, [out], torch.zeros(256, dtype=torch.uint8, device=other))
    torch.cuda.synchronize(other)
    assert torch.equal(out.cpu(), want.cpu())
    with pytest.raises(ValueError):
        qkn.fp8_linear(a1, w, [out], workspace())


# ---------------------------------------------------------------- codes to the bit
def quotient_codes(y, scale):
    """The codes of fp32 values on the host, by their definition: the fp32 quotient, rounded to the nearest e4m3."""
    return (y.float() / scale).to(torch.float8_e4m3fn).float()


def quotient_scale(amax):
    """A block's scale by its definition in fp32, on the host: the largest magnitude times the rounded 1 / 448."""
    return torch.clamp(torch.as_tensor(amax, dtype=torch.float32).cpu() * torch.tensor(1 / 448, dtype=torch.float32),
                       min=2.0 ** -100)


def assert_codes(codes, y, scale):
    got, want = codes.float().cpu(), quotient_codes(y.cpu(), scale.cpu())
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0)), f"{(got != want).sum().item()} codes differ"


def beside_midpoints(n, d, dtype, seed):
    """Rows whose blocks hold, next to a random largest value, values in the middle between two codes and the
    numbers of the type next to these, some zeros and tiny values, and ordinary ones."""
    g = torch.Generator().manual_seed(seed)
    grid = torch.from_numpy(oracle.e4m3_values())
    mid = ((grid[1:] + grid[:-1]) / 2).float()
    x = torch.randn((n, d), generator=g)
    for i in range(n):
        for j in range(0, d, 128):
            row = x[i, j:j + 128]
            top = (torch.rand((), generator=g) + 1) * 2.0 ** int(torch.randint(-40, 40, (), generator=g))
            top = top.to(dtype).float()
            v = mid[torch.randint(0, len(mid), (len(row),), generator=g)] * (top / 448)
            step = torch.randint(-1, 2, (len(row),), generator=g, dtype=torch.int32)
            bits = v.to(dtype).view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
            v = (bits + step.to(bits.dtype)).view(dtype).float()
            pick = torch.rand(len(row), generator=g)
            row.copy_(torch.where(pick < 0.8, v, torch.where(pick < 0.9, row * top / 4, torch.zeros(()))))
            row.clamp_(-top, top)
            row.mul_(torch.where(torch.rand(len(row), generator=g) < 0.5, -1.0, 1.0))
            row[int(torch.randint(0, len(row), (), generator=g))] = top
    return x.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(2, 8), (70, 512), (300, 333), (513, 1000)])
def test_weight_codes_are_the_rounded_quotients(n, k, dtype):
    for w in (torch.randn((n, k), generator=torch.Generator().manual_seed(n)).to(dtype),
              beside_midpoints(n, k, dtype, n + k)):
        q = qkn.Fp8Weight.empty(n, k)
        qkn.quant_weight(w.cuda(), q)
        per = np.array([[w[i:i + 128, j:j + 128].float().abs().max() for j in range(0, k, 128)] for i in range(0, n, 128)])
        scale = quotient_scale(per)
        assert torch.equal(q.scale.cpu(), scale)
        of = scale.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        assert_codes(q.codes[:, :k], w, of)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 8), (40, 512), (9, 5000), (33, 333), (1030, 264), (2, 20001), (2, 33000)])
def test_row_codes_are_the_rounded_quotients(n, d, dtype):
    """Without a norm from the values as they come; with one, in fp32, from the normalised rows that the call wrote."""
    for x in (hidden(n, d, dtype, d), beside_midpoints(min(n, 40), d, dtype, n + d).cuda()):
        m = x.shape[0]
        q, _, _ = run_norm(x)
        of = lambda q: q.scale[:, :m].t().repeat_interleave(128, 1)[:, :d]
        assert_codes(q.codes[:, :d], x, of(q))
        per = torch.stack([x[:, j:j + 128].float().abs().amax(1) for j in range(0, d, 128)])
        assert torch.equal(q.scale[:, :m].cpu(), quotient_scale(per))
        if dtype == torch.float32:
            q, _, y = run_norm(x, torch.ones(d, device="cuda"), want_y=True)
            assert_codes(q.codes[:, :d], y, of(q))


def test_finite_values_beside_an_infinity_have_zero_codes():
    x = hidden(2, 256, torch.float32, 3)
    x[0, 5], x[1, 200] = float("inf"), float("-inf")
    q, _, _ = run_norm(x)
    assert_codes(q.codes, x, q.scale[:, :2].t().repeat_interleave(128, 1))
    assert torch.isnan(q.codes.float()).sum() == 2 and (q.codes.float()[0, :5] == 0).all()


# ---------------------------------------------------------------- waits that run out
SHORT_WAIT = 1_000_000      # about half a millisecond


@pytest.mark.parametrize("stop", [1, 2, 3, 4])
@pytest.mark.parametrize("kernel,m,n,k,ats", [
    (qkn.LINEAR_SPLIT, 3, 700, 4096, (0, 1, 3)), (qkn.LINEAR_SPLIT, 30, 300, 2500, (0, 1)),
    (qkn.LINEAR_SPLIT, 64, 9000, 1500, (0, 1)), (qkn.LINEAR_SPLIT, 333, 1000, 5000, (0, 7)),
    (qkn.LINEAR_PAIR_128, 300, 500, 2000, (0, 3, 15)), (qkn.LINEAR_PAIR_128, 2049, 5000, 300, (0, 4)),
    (qkn.LINEAR_PAIR_256, 300, 500, 2000, (0, 3, 15)), (qkn.LINEAR_PAIR_256, 2049, 5000, 300, (0, 4)),
])
def test_wait_that_runs_out_is_reported_and_the_next_product_is_correct(kernel, m, n, k, ats, stop):
    """A role of every CTA gives up; the call records it and winds down, and the next one is right."""
    a, w = operands(m, n, k, seed=11)
    ws = workspace()
    want = torch.empty((m, n), dtype=torch.float32, device="cuda")
    qkn.fp8_linear(a, w, [want], ws, kernel=kernel)
    torch.cuda.synchronize()
    assert qkn.read_device_status(ws) == qkn.OK
    out = torch.empty_like(want)
    for at in ats if stop < 4 else ats[:1]:
        qkn.fp8_linear(a, w, [out], ws, kernel=kernel, wait_limit=SHORT_WAIT, test_stop=stop, test_at=at)
        assert qkn.read_device_status(ws) == qkn.ERR_TIMEOUT
        qkn.workspace_init(ws)
        out.fill_(float("nan"))
        qkn.fp8_linear(a, w, [out], ws, kernel=kernel)
        torch.cuda.synchronize()
        assert qkn.read_device_status(ws) == qkn.OK
        assert torch.equal(out, want)


# ---------------------------------------------------------------- every kernel by name
KERNELS = [qkn.LINEAR_SPLIT, qkn.LINEAR_PAIR_128, qkn.LINEAR_PAIR_256]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (5, 130, 300), (70, 1029, 128), (257, 520, 400), (300, 1400, 1100),
                                   (1030, 2600, 260)])
def test_every_kernel_writes_odd_places_and_nothing_else(m, n, k, kernel, dtype):
    """Slices of wider buffers at odd places, widths that end inside a tile or a box, in every kernel: right values,
    and what lies around stays."""
    a, w = operands(m, n, k, seed=m + n, pad=48)
    ref, mag = product(a, w)
    for off, cuts in ((0, []), (1, []), (3, [8, n - 3]), (8, [n // 2]), (5, [n // 3, n // 2 + 1]), (2, [n - 1])):
        cuts = sorted({0, n, *(c for c in cuts if 0 < c < n)})
        widths = [q - p for p, q in zip(cuts, cuts[1:])]
        bufs = [torch.full((m, c + 16), 5.0, dtype=dtype, device="cuda") for c in widths]
        ws = workspace()
        qkn.fp8_linear(a, w, [b[:, off:off + c] for b, c in zip(bufs, widths)], ws, kernel=kernel)
        assert qkn.read_device_status(ws) == qkn.OK
        got = np.concatenate([host(b[:, off:off + c]) for b, c in zip(bufs, widths)], axis=1)
        check_product(got, ref, mag, k, dtype)
        for b, c in zip(bufs, widths):
            assert (b[:, :off] == 5.0).all() and (b[:, off + c:] == 5.0).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m,n,k", [(3, 700, 1000), (300, 520, 640), (1500, 2560, 384)])
def test_every_kernel_repeats_bit_for_bit_and_keeps_nan_in_its_row(m, n, k, kernel):
    a, w = operands(m, n, k, seed=2)
    a.scale[1, 1] = float("nan")
    a.codes.view(torch.uint8)[2, 7] = 0x7F              # a code that is NaN
    outs = [torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    ws = workspace()
    for o in outs:
        qkn.fp8_linear(a, w, [o], ws, kernel=kernel)
    bits = [o.view(torch.int16) for o in outs]
    assert torch.equal(bits[0], bits[1]) and torch.equal(bits[0], bits[2])
    assert torch.isnan(outs[0][1:3]).all() and torch.isfinite(outs[0][0]).all() and torch.isfinite(outs[0][3:]).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m", [40, 600])
def test_every_kernel_in_a_chain_through_rewritten_buffers(m, kernel):
    """As test_one_buffer_rewritten_between_back_to_back_products, with the kernel given and the weight rewritten by
    every pair: its scales and codes come from the kernel before the last, the rows' from the last."""
    n, k, rounds = 1300, 900, 12
    xs = [hidden(m, k, torch.bfloat16, s) * 2.0 ** (s % 5) for s in range(rounds)]
    ww = [(torch.randn((n, k), generator=torch.Generator().manual_seed(s)) * 2.0 ** (s % 3)).cuda() for s in range(3)]
    ws = workspace()

    def chain(sync):
        q, w = qkn.Fp8Rows.empty(m, k), qkn.Fp8Weight.empty(n, k)
        outs = [torch.empty((m, n), dtype=torch.float32, device="cuda") for _ in range(rounds)]
        torch.cuda.synchronize()
        for i in range(rounds):
            qkn.norm_quant(xs[i], q)
            qkn.quant_weight(ww[i % 3], w)
            if sync:
                torch.cuda.synchronize()
            qkn.fp8_linear(q, w, [outs[i]], ws, kernel=kernel)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    want = chain(True)
    for _ in range(4):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)
    assert qkn.read_device_status(ws) == qkn.OK


@pytest.mark.parametrize("dtype", DTYPES)
def test_codes_and_scales_are_those_of_torch_on_the_gpu(dtype):
    """Weights and rows quantised with elementary torch operations on the GPU, to the bit."""
    for x in (hidden(300, 900, dtype, 1), beside_midpoints(140, 640, dtype, 2).cuda()):
        n, d = x.shape
        q, _, _ = run_norm(x)
        blocks = torch.nn.functional.pad(x.float(), (0, -d % 128)).view(n, -1, 128)
        scale = (blocks.abs().amax(-1) / 448.0).clamp_min(2.0 ** -100)
        codes = (blocks / scale[..., None]).to(torch.float8_e4m3fn).view(n, -1)[:, :d]
        assert torch.equal(q.scale[:, :n], scale.t()) and torch.equal(q.codes[:, :d].float(), codes.float())
        w = qkn.Fp8Weight.empty(n, d)
        qkn.quant_weight(x, w)
        scale = torch.stack([blocks[i:i + 128].abs().amax((0, 2)) / 448.0 for i in range(0, n, 128)])
        codes = (blocks / scale.repeat_interleave(128, 0)[:n][..., None]).to(torch.float8_e4m3fn).view(n, -1)[:, :d]
        assert torch.equal(w.scale, scale) and torch.equal(w.codes[:, :d].float(), codes.float())
