"""The 8-bit format and its entry points on the CPU: the oracle against torch's conversions and
closed forms, and every refusal of the C calls and of the binding, before any device work."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F

tp = pytest.importorskip("tensor_sharded_linear_tp_gb300",
                         reason="libtp.so not built (python tensor_sharded_linear_tp_gb300/build.py)")

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below is refused first
FAKE_SCALE = 0x10001


# ----------------------------------------------------------------------------- the oracle

def test_code_values_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(F.VALUES, codes.view(torch.float8_e4m3fn).double().numpy())


def test_encoding_matches_torch_to_nearest_even():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 20000), rng.normal(0, 0.01, 20000), F.VALUES[~np.isnan(F.VALUES)],
                        (F.VALUES[1:127] + F.VALUES[:126]) / 2, [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11]])
    v = v.astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(F.f64_to_e4m3(v.astype(np.float64)), want)


def test_scale_is_the_least_power_of_two_that_fits():
    rng = np.random.default_rng(1)
    amax = np.concatenate([2.0 ** rng.uniform(-100, 120, 5000), 448.0 * 2.0 ** np.arange(-100, 100),
                           np.nextafter(448.0 * 2.0 ** np.arange(-100, 100), np.inf)])
    s = F.scale_value(F.scale_byte(amax))
    assert np.all(amax <= 448 * s) and np.all(amax > 448 * s / 2)
    assert F.scale_byte(0.0) == 127 and F.scale_byte(np.inf) == 255 and F.scale_byte(np.nan) == 255
    assert F.scale_byte(2.0 ** -140) == 0


def test_quantized_group_keeps_half_a_step():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(70, 300)) * 10.0 ** rng.uniform(-4, 4, (70, 300))
    for rows in (1, 128):
        codes, byte = F.quantize(x, rows)
        s = F.spread(F.scale_value(byte), x.shape, rows)
        err = np.abs(F.dequantize(codes, byte, rows) - x)
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))


def test_residual_norm_closed_forms():
    x = np.array([[3.0, -3.0, 3.0, -3.0]])
    h, u = F.residual_norm(x, norm="rms", eps=0.0)
    np.testing.assert_allclose(u, [[1, -1, 1, -1]])
    h, u = F.residual_norm(x, x + 5, post_norm="layer", gate=np.full((1, 4), 2.0), alpha=0.5, eps=0.0, norm="none")
    np.testing.assert_allclose(h, [[3.5, -3.5, 3.5, -3.5]])
    np.testing.assert_allclose(u, h)


# ----------------------------------------------------------------------------- refusals of the C calls

def _ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def _name(status):
    return tp.STATUS_NAMES[status]


def _quant(x=FAKE, ldx=0, rows=4, cols=256, block=1, q=FAKE, ldq=0, s=FAKE_SCALE, lds=0):
    return _name(tp.lib.tp_quantize_fp8(x, ldx, rows, cols, block, q, ldq, s, lds, None))


@pytest.mark.parametrize("kw, want", [
    (dict(rows=-1), "TP_ERR_INVALID_ARG"), (dict(cols=-16), "TP_ERR_INVALID_ARG"), (dict(block=64), "TP_ERR_INVALID_ARG"),
    (dict(block=0), "TP_ERR_INVALID_ARG"), (dict(x=None), "TP_ERR_INVALID_ARG"), (dict(q=None), "TP_ERR_INVALID_ARG"),
    (dict(s=None), "TP_ERR_INVALID_ARG"), (dict(ldx=128), "TP_ERR_INVALID_ARG"), (dict(ldq=128), "TP_ERR_INVALID_ARG"),
    (dict(lds=1), "TP_ERR_INVALID_ARG"), (dict(cols=264), "TP_ERR_ALIGNMENT"), (dict(ldx=260), "TP_ERR_ALIGNMENT"),
    (dict(ldq=264), "TP_ERR_ALIGNMENT"), (dict(x=FAKE + 8), "TP_ERR_ALIGNMENT"), (dict(q=FAKE + 8), "TP_ERR_ALIGNMENT"),
    (dict(cols=1 << 32), "TP_ERR_UNSUPPORTED"), (dict(rows=1 << 40, cols=1 << 20), "TP_ERR_UNSUPPORTED"),
    (dict(rows=0), "TP_OK"), (dict(cols=0), "TP_OK"),
])
def test_quantize_refusals(kw, want):
    assert _quant(**kw) == want


def _col(x=FAKE, ldx=0, xs=FAKE_SCALE, ld_xs=0, w=FAKE, ws=FAKE_SCALE, act=0, p=2, T=4, K=256, N=256, y=FAKE, ldy=0,
         ys=None, ld_ys=0, w_arr=True, y_arr=True):
    n = max(1, min(p, 16))
    return _name(tp.lib.tp_linear_colwise_fp8(
        x, ldx, xs, ld_xs, _ptrs(*[w] * n) if w_arr else None, _ptrs(*[ws] * n), None, act, p, T, K, N,
        _ptrs(*[y] * n) if y_arr else None, ldy, _ptrs(*[ys] * n) if ys != None else None, ld_ys, None))  # noqa: E711


SIZES = [
    (dict(p=0), "TP_ERR_INVALID_ARG"), (dict(p=17), "TP_ERR_UNSUPPORTED"), (dict(T=-1), "TP_ERR_INVALID_ARG"),
    (dict(K=-16), "TP_ERR_INVALID_ARG"), (dict(N=-8), "TP_ERR_INVALID_ARG"), (dict(K=0), "TP_ERR_INVALID_ARG"),
    (dict(T=1 << 31), "TP_ERR_UNSUPPORTED"), (dict(K=1 << 31), "TP_ERR_UNSUPPORTED"), (dict(K=264), "TP_ERR_ALIGNMENT"),
    (dict(N=260), "TP_ERR_ALIGNMENT"), (dict(ldx=128), "TP_ERR_INVALID_ARG"), (dict(ldx=264), "TP_ERR_ALIGNMENT"),
    (dict(ld_xs=1), "TP_ERR_INVALID_ARG"), (dict(x=None), "TP_ERR_INVALID_ARG"), (dict(xs=None), "TP_ERR_INVALID_ARG"),
    (dict(w=None), "TP_ERR_INVALID_ARG"), (dict(ws=None), "TP_ERR_INVALID_ARG"), (dict(x=FAKE + 8), "TP_ERR_ALIGNMENT"),
    (dict(w=FAKE + 8), "TP_ERR_ALIGNMENT"), (dict(w_arr=False), "TP_ERR_INVALID_ARG"), (dict(T=0), "TP_OK"),
    (dict(N=0), "TP_OK"),
]


@pytest.mark.parametrize("kw, want", SIZES + [
    (dict(act=3), "TP_ERR_INVALID_ARG"), (dict(act=0x100), "TP_ERR_INVALID_ARG"), (dict(act=2, N=257), "TP_ERR_INVALID_ARG"),
    (dict(act=2, N=264), "TP_ERR_ALIGNMENT"), (dict(ldy=128), "TP_ERR_INVALID_ARG"), (dict(ldy=260), "TP_ERR_ALIGNMENT"),
    (dict(ys=FAKE_SCALE, N=264), "TP_ERR_ALIGNMENT"), (dict(ys=FAKE_SCALE, ldy=264), "TP_ERR_ALIGNMENT"),
    (dict(ys=FAKE_SCALE, ld_ys=1), "TP_ERR_INVALID_ARG"), (dict(y=None), "TP_ERR_INVALID_ARG"),
    (dict(ys=0), "TP_ERR_INVALID_ARG"), (dict(y=FAKE + 8), "TP_ERR_ALIGNMENT"), (dict(y_arr=False), "TP_ERR_INVALID_ARG"),
])
def test_colwise_refusals(kw, want):
    assert _col(**kw) == want


def _row(x=FAKE, ldx=0, xs=FAKE_SCALE, ld_xs=0, w=FAKE, ws=FAKE_SCALE, p=2, T=4, K=256, N=256, out=FAKE, ldo=0,
         w_arr=True):
    n = max(1, min(p, 16))
    return _name(tp.lib.tp_linear_rowwise_fp8(_ptrs(*[x] * n), ldx, _ptrs(*[xs] * n), ld_xs,
                                              _ptrs(*[w] * n) if w_arr else None, _ptrs(*[ws] * n), None, p, T, K, N,
                                              out, ldo, None))


@pytest.mark.parametrize("kw, want", SIZES + [
    (dict(out=None), "TP_ERR_INVALID_ARG"), (dict(ldo=128), "TP_ERR_INVALID_ARG"), (dict(ldo=260), "TP_ERR_ALIGNMENT"),
    (dict(out=FAKE + 8), "TP_ERR_ALIGNMENT"),
])
def test_rowwise_refusals(kw, want):
    assert _row(**kw) == want


def test_bias_inside_an_element_is_refused():
    lib, F16, S = tp.lib, FAKE, FAKE_SCALE
    two = lambda v: _ptrs(v, v)  # noqa: E731
    for bias in (_ptrs(FAKE + 1, 0), _ptrs(None, FAKE + 3)):
        assert _name(lib.tp_linear_colwise_fp8(F16, 0, S, 0, two(F16), two(S), bias, 0, 2, 4, 256, 256, two(F16), 0, None,
                                               0, None)) == "TP_ERR_ALIGNMENT"
    assert _name(lib.tp_linear_rowwise_fp8(two(F16), 0, two(S), 0, two(F16), two(S), FAKE + 1, 2, 4, 256, 256, F16, 0,
                                           None)) == "TP_ERR_ALIGNMENT"


def _norm(**kw):
    a = tp.ResidualNormArgs()
    base = dict(T=4, D=256, x=FAKE, y=FAKE, h=FAKE, u=FAKE, norm=1, alpha=1.0, eps=1e-6)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return _name(tp.lib.tp_residual_norm(ctypes.byref(a), None))


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), "TP_ERR_INVALID_ARG"), (dict(D=-8), "TP_ERR_INVALID_ARG"), (dict(x=None), "TP_ERR_INVALID_ARG"),
    (dict(h=None, u=None, norm=0), "TP_ERR_INVALID_ARG"), (dict(y=None), "TP_ERR_INVALID_ARG"),
    (dict(y=None, h=None, gate=FAKE, mod_rows=1, rows_per_mod=4), "TP_ERR_INVALID_ARG"),
    (dict(y=None, h=None, post_norm=1), "TP_ERR_INVALID_ARG"), (dict(norm=3), "TP_ERR_INVALID_ARG"),
    (dict(post_norm=-1), "TP_ERR_INVALID_ARG"), (dict(post_weight=FAKE), "TP_ERR_INVALID_ARG"),
    (dict(norm=0, weight=FAKE), "TP_ERR_INVALID_ARG"), (dict(u=None), "TP_ERR_INVALID_ARG"),
    (dict(u=None, norm=0, u_scales=FAKE_SCALE), "TP_ERR_INVALID_ARG"), (dict(eps=-1.0), "TP_ERR_INVALID_ARG"),
    (dict(eps=float("nan")), "TP_ERR_INVALID_ARG"), (dict(eps=float("inf")), "TP_ERR_INVALID_ARG"),
    (dict(gate=FAKE), "TP_ERR_INVALID_ARG"), (dict(gate=FAKE, mod_rows=1, rows_per_mod=3), "TP_ERR_INVALID_ARG"),
    (dict(scale=FAKE, mod_rows=1, rows_per_mod=0), "TP_ERR_INVALID_ARG"), (dict(ldx=128), "TP_ERR_INVALID_ARG"),
    (dict(ld_mod=128), "TP_ERR_INVALID_ARG"), (dict(ld_u_scales=1), "TP_ERR_INVALID_ARG"),
    (dict(D=260), "TP_ERR_ALIGNMENT"), (dict(D=264, u_scales=FAKE_SCALE), "TP_ERR_ALIGNMENT"),
    (dict(ldx=260), "TP_ERR_ALIGNMENT"), (dict(ldu=264, u_scales=FAKE_SCALE), "TP_ERR_ALIGNMENT"),
    (dict(x=FAKE + 2), "TP_ERR_ALIGNMENT"), (dict(shift=FAKE + 8, mod_rows=1, rows_per_mod=4), "TP_ERR_ALIGNMENT"),
    (dict(D=32776), "TP_ERR_UNSUPPORTED"), (dict(T=0), "TP_OK"), (dict(D=0), "TP_OK"),
])
def test_residual_norm_refusals(kw, want):
    assert _norm(**kw) == want


def test_residual_norm_args_null():
    assert _name(tp.lib.tp_residual_norm(None, None)) == "TP_ERR_INVALID_ARG"


# ----------------------------------------------------------------------------- the binding

def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    x8, sx = x.to(torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8)
    w, sw = torch.zeros(128, 256).to(torch.float8_e4m3fn), torch.zeros(1, 2, dtype=torch.uint8)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        tp.tp_quantize_fp8(x)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        tp.tp_linear_colwise_fp8(x8, sx, [w], [sw])
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        tp.tp_linear_rowwise_fp8([x8], [sx], [w], [sw])
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        tp.tp_residual_norm(x, x)


class _NoCalls:
    """In the library's place where every call has to be refused before it."""

    def __getattr__(self, name):
        pytest.fail(f"{name} was called")


@pytest.mark.parametrize("tables", [dict(gate=2), dict(scale=2), dict(scale=3, shift=3)], ids=str)
def test_tables_of_several_rows_need_rows_per_mod(monkeypatch, tables):
    """Without it every row of x would silently be modulated as the first sample's."""
    monkeypatch.setattr(tp, "_device_of", lambda name, t: t.get_device())
    monkeypatch.setattr(tp, "lib", _NoCalls())
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rows_per_mod"):
        tp.tp_residual_norm(x, x, **{k: torch.zeros(n, 256, dtype=torch.bfloat16) for k, n in tables.items()})


def test_struct_mirrors_header():
    """The field order of the binding's structure is the header's."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "tp.h")).read()
    body = text[:text.index("} tp_residual_norm_args;")]
    body = re.sub(r"/\*.*?\*/", "", body[body.rindex("typedef struct {"):], flags=re.S)
    names = re.findall(r"[\*\s,](\w+)\s*(?=[;,])", body)
    assert names == [n for n, _ in tp.ResidualNormArgs._fields_]
    values = [float(i + 1) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(tp.ResidualNormArgs._fields_)]
    packed = tp._residual_norm_args(*values)
    assert len(packed) == ctypes.sizeof(tp.ResidualNormArgs)
    a = tp.ResidualNormArgs.from_buffer_copy(packed)
    assert [getattr(a, n) for n in names] == values
