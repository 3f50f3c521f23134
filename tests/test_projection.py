"""The 8-bit projections without a GPU: the oracle's pins, the argument checks of the C ABI and of the
binding (nothing is launched)."""
import ctypes
import os
import subprocess
import sys
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import qk_normed_latent_qkn_b200 as qkn

P = 0x1000   # a well-aligned address that no call may touch


# ---------------------------------------------------------------- oracle pins
def test_e4m3_rounding_matches_torch_at_values_and_midpoints():
    grid = oracle.e4m3_values()
    assert grid[0] == 0 and grid[-1] == 448 and len(grid) == 127
    mid = (grid[1:] + grid[:-1]) / 2
    x = np.concatenate([grid, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), [1e-12, 447.99, 450.0]])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float32)
    keep = want.double().numpy() == x            # what fp32 holds exactly (the grid and the midpoints)
    got = oracle.e4m3_round(x)
    assert np.array_equal(got[keep], want.to(torch.float8_e4m3fn).double().numpy()[keep])
    # the neighbours of a midpoint go to the nearer side
    assert np.all(np.abs(got - x) <= np.abs(grid[None] - np.abs(x)[:, None]).min(axis=1) + 2)
    for v in np.concatenate([np.nextafter(mid, 0), np.nextafter(mid, 1e9)]):
        assert abs(oracle.e4m3_round(v) - v) == np.abs(grid - v).min()
    assert np.isnan(oracle.e4m3_round(np.nan)) and oracle.e4m3_round(1e9) == 448


def test_quantised_values_are_within_half_a_step():
    rng = np.random.default_rng(3)
    y = rng.standard_normal((5, 300)) * np.exp(rng.standard_normal((5, 1)) * 3)
    y[2, 128:256] = 0
    ratio, scale = oracle.quant_rows(y)
    assert scale.shape == (3, 5) and scale[1, 2] == oracle.FP8_LEAST
    assert np.abs(ratio).max() == pytest.approx(448, rel=1e-15)
    back = oracle.row_values(oracle.e4m3_round(ratio), scale)
    per = scale[np.arange(300) // 128].T
    assert np.all(np.abs(back - y) <= np.maximum(np.abs(y) * 2.0 ** -4, per * 2.0 ** -10) * (1 + 1e-12))
    w = rng.standard_normal((200, 130))
    ratio, scale = oracle.quant_weight(w)
    assert scale.shape == (2, 2)
    assert scale[1, 1] == np.abs(w[128:, 128:]).max() / 448
    back = oracle.weight_values(oracle.e4m3_round(ratio), scale)
    assert np.abs(back - w).max() <= np.abs(w).max() * 2.0 ** -4


def test_product_is_exact_on_a_small_case():
    rng = np.random.default_rng(4)
    a = oracle.e4m3_round(rng.standard_normal((2, 140)) * 20)
    w = oracle.e4m3_round(rng.standard_normal((130, 140)) * 20)
    sa, sw = 2.0 ** rng.integers(-3, 3, (2, 4)), 2.0 ** rng.integers(-3, 3, (2, 2))
    got = oracle.fp8_linear(a, sa, w, sw)
    for i, n in ((0, 0), (1, 127), (0, 128), (1, 129)):
        want = sum(Fraction(float(a[i, k])) * Fraction(float(sa[k // 128, i])) * Fraction(float(w[n, k]))
                   * Fraction(float(sw[n // 128, k // 128])) for k in range(140))
        assert got[i, n] == pytest.approx(float(want), rel=1e-13)


# ---------------------------------------------------------------- C ABI
def _rows(codes=P, scale=P, rows=4, cols=256, ld=256, ld_scale=4):
    return qkn._Fp8Rows(codes, scale, rows, cols, ld, ld_scale)


def _weight(codes=P, scale=P, rows=64, cols=256, ld=256):
    return qkn._Fp8Weight(codes, scale, rows, cols, ld)


def _norm(q, dtype=qkn.BF16, x=P, ld_x=256, residual=None, gamma=None, eps=1e-6, residual_out=None, y=None):
    return qkn.raw_library().qkn_norm_quant(dtype, x, ld_x, residual, gamma, eps, residual_out, y, ctypes.byref(q),
                                            None)


@pytest.mark.parametrize("q", [
    dict(codes=None), dict(codes=P + 8), dict(scale=None), dict(scale=P + 4), dict(rows=-1), dict(cols=0),
    dict(ld=240), dict(ld=264), dict(ld_scale=2), dict(ld_scale=3), dict(ld_scale=6), dict(rows=5), dict(ld_scale=0),
])
def test_norm_quant_refuses_bad_rows(q):
    assert _norm(_rows(**q)) == qkn.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(x=None), dict(x=P + 1), dict(ld_x=255), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(residual=P), dict(residual_out=P), dict(gamma=P + 2), dict(y=P + 1),
    dict(residual=2 * P, residual_out=P, ld_x=320),      # x overwritten in place needs its rows dense
    dict(y=P, ld_x=320),
    dict(residual=2 * P, residual_out=3 * P, y=2 * P),   # y over the residual, its sum, or an x still needed
    dict(residual=2 * P, residual_out=3 * P, y=3 * P),
    dict(residual=2 * P, residual_out=3 * P, y=P),
])
def test_norm_quant_refuses_bad_arguments(kw):
    assert _norm(_rows(), **kw) == qkn.ERR_INVALID_ARG


def test_empty_calls_are_no_ops():
    assert _norm(_rows(codes=None, scale=None, rows=0), x=None) == qkn.OK
    lib = qkn.raw_library()
    assert lib.qkn_quant_weight(qkn.F32, None, ctypes.byref(_weight(rows=0)), None) == qkn.OK
    assert _linear(a=_rows(codes=None, scale=None, rows=0), outs=[(None, 64, 64)]) == qkn.OK
    x = torch.empty((0, 256), dtype=torch.bfloat16)
    qkn.norm_quant(x, qkn.Fp8Rows.empty(0, 256, "cpu"))


def test_quant_weight_refuses_bad_arguments():
    f = qkn.raw_library().qkn_quant_weight
    for q in (dict(codes=None), dict(codes=P + 8), dict(scale=None), dict(scale=P + 2), dict(rows=-1), dict(cols=0),
              dict(ld=128), dict(ld=257)):
        assert f(qkn.BF16, P, ctypes.byref(_weight(**q)), None) == qkn.ERR_INVALID_ARG, q
    assert f(3, P, ctypes.byref(_weight()), None) == qkn.ERR_INVALID_ARG
    assert f(qkn.BF16, None, ctypes.byref(_weight()), None) == qkn.ERR_INVALID_ARG
    assert f(qkn.F32, P + 2, ctypes.byref(_weight()), None) == qkn.ERR_INVALID_ARG
    assert f(qkn.F32, P, None, None) == qkn.ERR_INVALID_ARG


def _linear(a=None, w=None, outs=((P, 64, 64),), dtype=qkn.BF16, ws=P, ws_bytes=256, n_outs=None):
    arr = (qkn._OutCols * max(1, len(outs)))(*[qkn._OutCols(*o) for o in outs])
    return qkn.raw_library().qkn_fp8_linear(ctypes.byref(a or _rows()), ctypes.byref(w or _weight()), dtype,
                                            len(outs) if n_outs is None else n_outs, arr, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(a=_rows(codes=None)), dict(a=_rows(scale=P + 8)), dict(a=_rows(ld_scale=0)), dict(a=_rows(rows=-2)),
    dict(a=_rows(cols=255)), dict(w=_weight(codes=P + 1)), dict(w=_weight(scale=None)), dict(w=_weight(rows=0)),
    dict(w=_weight(cols=128)), dict(w=_weight(ld=250)), dict(dtype=5),
    dict(outs=()), dict(n_outs=9), dict(n_outs=-1),
    dict(outs=[(None, 64, 64)]), dict(outs=[(P + 1, 64, 64)]), dict(outs=[(P + 2, 64, 64)], dtype=qkn.F32),
    dict(outs=[(P, 63, 64)]), dict(outs=[(P, 65, 65)]), dict(outs=[(P, 64, 63)]), dict(outs=[(P, 64, 64), (P, 0, 4)]),
    dict(outs=[(P, 40, 64), (P, 25, 64)]), dict(outs=[(P, 2 ** 31 - 1, 2 ** 31), (P, 2 ** 31 - 1, 2 ** 31)]),
    dict(ws=None), dict(ws=P + 128), dict(ws_bytes=255),
])
def test_fp8_linear_refuses_bad_arguments(kw):
    assert _linear(**kw) == qkn.ERR_INVALID_ARG


# ---------------------------------------------------------------- binding
def test_binding_refuses_tensors_that_do_not_fit():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q = qkn.Fp8Rows.empty(4, 256, "cpu")
    w = qkn.Fp8Weight.empty(64, 256, "cpu")
    ws = torch.zeros(256, dtype=torch.uint8)
    out = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (
            lambda: qkn.norm_quant(x[0], q),
            lambda: qkn.norm_quant(x.t().contiguous().t(), q),
            lambda: qkn.norm_quant(x[:3], q),
            lambda: qkn.norm_quant(x[:, :128], q),
            lambda: qkn.norm_quant(x.half(), q),
            lambda: qkn.norm_quant(x, q, gamma=torch.ones(256, dtype=torch.bfloat16)),
            lambda: qkn.norm_quant(x, q, gamma=torch.ones(255)),
            lambda: qkn.norm_quant(x, q, residual=x.float(), residual_out=x.clone()),
            lambda: qkn.norm_quant(x, q, y=torch.zeros((4, 512), dtype=torch.bfloat16)[:, ::2]),
            lambda: qkn.quant_weight(torch.zeros((256, 64)).t(), w),
            lambda: qkn.quant_weight(torch.zeros((64, 255)), w),
            lambda: qkn.fp8_linear(q, w, [], ws),
            lambda: qkn.fp8_linear(q, w, [out[:, :8]] * 9, ws),
            lambda: qkn.fp8_linear(q, w, [out[:3]], ws),
            lambda: qkn.fp8_linear(q, w, [out.half()], ws),
            lambda: qkn.fp8_linear(q, w, [out[:, :32], out[:, 32:].float()], ws),
            lambda: qkn.Fp8Rows(q.codes.view(torch.uint8), q.scale, 256),
            lambda: qkn.Fp8Rows(q.codes, q.scale[:1], 256),
            lambda: qkn.Fp8Rows(q.codes, q.scale, 257),
            lambda: qkn.Fp8Weight(w.codes, w.scale, 100),
            lambda: qkn.Fp8Weight(w.codes, w.scale.double(), 256)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(qkn.QknError):               # one without the other
        qkn.norm_quant(x, q, residual=x.clone())


def test_binding_refuses_cpu_tensors():
    """A kernel must not be handed host memory: refused before anything is launched."""
    x = torch.zeros((4, 256))
    q, w = qkn.Fp8Rows.empty(4, 256, "cpu"), qkn.Fp8Weight.empty(64, 256, "cpu")
    for call in (lambda: qkn.norm_quant(x, q),
                 lambda: qkn.quant_weight(torch.zeros((64, 256)), w),
                 lambda: qkn.fp8_linear(q, w, [torch.zeros((4, 64))], torch.zeros(512, dtype=torch.uint8))):
        with pytest.raises(qkn.QknError) as e:
            call()
        assert e.value.status == qkn.ERR_INVALID_ARG


def test_holders_allocate_what_the_calls_need():
    q = qkn.Fp8Rows.empty(5, 300, "cpu")
    assert q.codes.shape == (5, 304) and q.scale.shape == (3, 8)
    w = qkn.Fp8Weight.empty(130, 300, "cpu")
    assert w.codes.shape == (130, 304) and w.scale.shape == (2, 3)


# ---------------------------------------------------------------- the kernels' quotient
def _fp32(x):
    """An exact number rounded to 24 significant bits, ties to even (any exponent)."""
    if x == 0:
        return x
    sign, x, e = (-1 if x < 0 else 1), abs(x), 0
    while x >= 2:
        x, e = x / 2, e + 1
    while x < 1:
        x, e = x * 2, e - 1
    y = x * 2 ** 23
    f = y.numerator // y.denominator
    if y - f > Fraction(1, 2) or (y - f == Fraction(1, 2) and f % 2):
        f += 1
    return sign * Fraction(f) * Fraction(2) ** (e - 23)


def test_corrected_quotient_gives_the_code_of_the_rounded_one():
    """The kernels take v / s as q = v r with r = 1 / s, corrected by (v - q s) r.  q differs from v / s by at most
    1.5 units of the last place, so the corrected value before its rounding by at most 2^-22 units, and its code is
    that of the rounded quotient unless v / s lies that close to a border M -+ 2^-24 (M in [1, 2): the middle of two
    codes, 5 significant bits) between the numbers that round to M and their neighbours.  With s = S 2^-23 and v on
    its grid that is |S u - r| = 0 modulo 2^24 for u = M 2^24 -+ 1 and a small r: a few S for each u and r, all of
    which are tried here, in exact arithmetic (64 times the bound's share of r)."""
    cases = 0
    for m in range(16, 32):
        for side in (1, -1):
            u = m * 2 ** 20 + side
            inv = pow(u, -1, 2 ** 24)
            for r in range(-64, 65):
                S = r * inv % 2 ** 24
                if S < 2 ** 23:
                    continue
                s = Fraction(S, 2 ** 23)
                for bits in (23, 22):
                    near = round(s * Fraction(u, 2 ** 24) * 2 ** bits)
                    for v in (Fraction(near + i, 2 ** bits) for i in (-1, 0, 1)):
                        if _fp32(v) != v:
                            continue
                        inverse = _fp32(1 / s)
                        q = _fp32(v * inverse)
                        q = _fp32(q + _fp32(v - q * s) * inverse)
                        mid, want = Fraction(m, 16), _fp32(v / s)
                        assert (q > mid) - (q < mid) == (want > mid) - (want < mid), (S, v, m)
                        cases += 1
    assert cases > 5000


# ---------------------------------------------------------------- what a chained kernel may read how
def test_no_read_only_loads_of_what_the_kernel_before_writes():
    """The product and the quantisation start while the kernel before them still runs and take their inputs from it.
    The read-only path (ld.global.nc, __ldg, __restrict__ on const pointers) is for data that nothing writes while
    the kernel runs, the wait for its predecessor included; whether a stale line is hit cannot be tested on a GPU."""
    csrc = os.path.join(os.path.dirname(qkn.__file__), "csrc")
    for name in ("fp8_linear.cu", "quant.cu"):
        with open(os.path.join(csrc, name)) as f:
            code = "\n".join(line.split("//")[0] for line in f)
        for form in ("global.nc", "__ldg", "__restrict__", "__ldcs", "__ldca"):
            assert form not in code, (name, form)


# ---------------------------------------------------------------- options of the product
@pytest.mark.parametrize("opts", [dict(kernel=-1), dict(kernel=4), dict(wait_limit=-1), dict(test_stop=-1),
                                  dict(test_stop=5), dict(test_stop=1, test_at=-1)])
def test_fp8_linear_refuses_bad_options(opts):
    arr = (qkn._OutCols * 1)(qkn._OutCols(P, 64, 64))
    call = lambda o: qkn.raw_library().qkn_fp8_linear_ex(ctypes.byref(_rows()), ctypes.byref(_weight()), qkn.BF16, 1,
                                                         arr, P, 256, ctypes.byref(o), None)
    assert call(qkn._LinearOpts(**opts)) == qkn.ERR_INVALID_ARG
    rows = _rows(rows=0, codes=None, scale=None)
    assert qkn.raw_library().qkn_fp8_linear_ex(ctypes.byref(rows), ctypes.byref(_weight()), qkn.BF16, 1, arr, P, 256,
                                               ctypes.byref(qkn._LinearOpts(kernel=3)), None) == qkn.OK


def test_package_imports_where_torch_lacks_its_private_shortcuts():
    """As in a torch without CUDA: the package imports, and calls on CPU tensors are refused as ever."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import qk_normed_latent_qkn_b200 as qkn
try:
    qkn.norm_quant(torch.zeros((4, 256)), qkn.Fp8Rows.empty(4, 256, "cpu"))
except qkn.QknError as e:
    assert e.status == qkn.ERR_INVALID_ARG
else:
    raise SystemExit("not refused")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(qkn.__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)
