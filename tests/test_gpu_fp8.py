"""The 8-bit projections, their quantiser and the residual norm against float64 numpy.

Quantised bf16 inputs are compared bit for bit (scaling by a power of two is exact, so a code has
one right value).  Products of small integer codes with power-of-two scales have exact fp32 sums
and are compared bit for bit too: they pin every index, tail and scale.  The rest is held to
bounds made of the steps that round:

* a stored bf16 value: 2^-8 relative; a stored code: 2^-4 relative, or half the subnormal spacing,
  2^-10 times its scale;
* the tensor core's sum over K: its products are exact in fp32, each step of 32 adds into an fp32
  accumulator without rounding to nearest, so at most 2^-22 of the sum of magnitudes a step, and
  one fp32 rounding (2^-24) for each of up to 8 partial sums and the bias;
* GELU and SiLU: at most 1.13 times the error of their argument, and the exponential's error,
  (2 + |argument|) 2^-22 relative, with 4 more roundings;
* the norm: a sum of D squares in any order is within D 2^-24 relative of exact; its values pass
  at most 16 more fp32 roundings, each relative to the largest term it meets.
"""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F

pytestmark = pytest.mark.gpu

tp = pytest.importorskip("tensor_sharded_linear_tp_gb300")

DEV = "cuda"
E4M3, E8M0, BF16 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    tp.tp_device_status()   # raises if any kernel gave up on a bounded wait


def f64(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def codes(t):
    torch.cuda.synchronize()
    return t.detach().view(torch.uint8).cpu().numpy()


def to_bf16(a, **kw):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(BF16).to(DEV, **kw)


def to_codes(c):
    return torch.from_numpy(np.ascontiguousarray(c, dtype=np.uint8)).to(DEV).view(E4M3)


def to_scales(b):
    return torch.from_numpy(np.ascontiguousarray(b, dtype=np.uint8)).to(DEV).view(E8M0)


def quantized(rng, rows, cols, block_rows, std=1.0):
    """(codes tensor, scales tensor, float64 values) of a random matrix."""
    c, b = F.quantize(rng.normal(0, std, (rows, cols)), block_rows)
    return to_codes(c), to_scales(b), F.dequantize(c, b, block_rows)


def integers(rng, rows, cols, block_rows):
    """Codes that stand for integers up to 4, scales of 2^-2 .. 2^2 at random."""
    c = F.f64_to_e4m3(rng.integers(-4, 5, (rows, cols)).astype(np.float64))
    b = rng.integers(125, 130, (-(-rows // block_rows), -(-cols // 128))).astype(np.uint8)
    return to_codes(c), to_scales(b), F.dequantize(c, b, block_rows)


def bf16_round(v):
    return torch.from_numpy(v.astype(np.float32)).to(BF16).float().numpy().astype(np.float64)


def accumulated(mag, K):
    """Bound on the fp32 sum's error from the sum of magnitudes."""
    return mag * ((-(-K // 32)) * 2.0 ** -22 + 9 * 2.0 ** -24)


def act_bound(pre, err, act, up=None, up_err=None):
    """(value, error bound) of an activation of `pre`, known to within `err`."""
    if act == "none":
        return pre, err
    y = F.apply_act(pre, act)
    arg = np.abs(1.5957691216 * (pre + 0.044715 * pre ** 3))
    return y, 1.13 * err + np.abs(y) * ((2 + arg) * 2.0 ** -22 + 8 * 2.0 ** -24) + 1e-35


def swiglu_bound(g, u, ge, ue):
    s = g / (1 + np.exp(-g))
    err = np.abs(u) * (1.1 * ge + np.abs(s) * ((2 + np.abs(g)) * 2.0 ** -22 + 8 * 2.0 ** -24)) + (np.abs(s) + 1.1 * ge) * ue
    return s * u, err + 2.0 ** -23 * np.abs(s * u) + 1e-35


def check_bf16(got, want, err, what=""):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bound = 2.0 ** -8 * (np.abs(want) + err) + err
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


def check_fp8(q, s, want, err, what=""):
    """Codes and scales that stand for `want`, known to within `err` (groups of 1 x 128)."""
    byte, c = codes(s), codes(q)
    assert byte.shape == F.group_amax(want, 1).shape, what
    lo, hi = np.maximum(np.abs(want) - err, 0), np.abs(want) + err
    b_lo, b_hi = F.scale_byte(F.group_amax(lo, 1)), F.scale_byte(F.group_amax(hi, 1))
    zero = (b_lo == 127) & (F.group_amax(lo, 1) == 0)
    assert np.all(((byte >= b_lo) | zero) & ((byte <= b_hi) | (byte == 127) & zero)), what
    scale = F.spread(F.scale_value(byte), want.shape, 1)
    bound = np.maximum(2.0 ** -4 * hi, 2.0 ** -10 * scale) + err
    got = F.dequantize(c, byte, 1)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


# ----------------------------------------------------------------------------- quantiser

@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 16), (1, 128), (3, 144), (127, 256), (128, 128), (129, 1040), (300, 640)], ids=str)
def test_quantize_bit_exact(shape, block_rows):
    rng = np.random.default_rng(shape[0] * 10000 + shape[1])
    # every magnitude bf16 has, normal values, exact limits (448 * 2^k) and their neighbours
    v = rng.normal(size=shape) * 2.0 ** rng.integers(-30, 30, (shape[0], 1))
    v[rng.random(shape) < 0.1] = 0
    v[rng.random(shape) < 0.02] *= 2.0 ** -12
    edge = rng.random(shape) < 0.02
    v[edge] = (448.0 * 2.0 ** rng.integers(-20, 20, shape))[edge]
    x = to_bf16(v)
    want_c, want_b = F.quantize(f64(x), block_rows)
    q, s = tp.tp_quantize_fp8(x, block_rows)
    assert q.dtype is E4M3 and s.dtype is E8M0
    np.testing.assert_array_equal(codes(s), want_b)
    np.testing.assert_array_equal(codes(q), want_c)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_any_bits(block_rows):
    """Every bf16 pattern: subnormals, infinities and NaN (which take their whole group)."""
    bits = np.random.default_rng(5).permutation(1 << 16).astype(np.uint16).reshape(256, 256)
    bits[:, 128:] &= 0xFF7F                     # right half: exponents below the top, so no infinity or NaN
    x = tp.bf16_from_bits(bits, DEV)
    q, s = tp.tp_quantize_fp8(x, block_rows)
    want_c, want_b = F.quantize(f64(x), block_rows)
    byte, c = codes(s), codes(q)
    np.testing.assert_array_equal(byte, want_b)
    nan = np.isnan(F.e4m3_to_f64(c))
    np.testing.assert_array_equal(nan, F.spread(want_b, c.shape, block_rows) == 255)
    np.testing.assert_array_equal(c[~nan], want_c[~nan])


def test_quantize_special_groups():
    v = np.ones((6, 256))
    v[0] = 0
    v[1, 5], v[2, 5], v[3, 5] = np.inf, np.nan, -np.inf
    v[4] = 2.0 ** -133                          # a bf16 subnormal: the least scale, 2^-127
    v[5] = -0.0
    q, s = tp.tp_quantize_fp8(to_bf16(v))
    byte, c = codes(s), codes(q)
    assert list(byte[:, 0]) == [127, 255, 255, 255, 0, 127] and list(byte[1:4, 1]) == [119] * 3
    assert np.isnan(F.e4m3_to_f64(c[1:4, :128])).all() and np.all(F.e4m3_to_f64(c[1:4, 128:]) == 256)
    assert np.all(c[0] == 0) and np.all(c[5] == 0x80) and np.all(F.e4m3_to_f64(c[4]) == 2.0 ** -6)


def test_quantize_strides_and_neighbours():
    """Strided input and outputs; nothing is written past the rows and columns asked for."""
    rng = np.random.default_rng(7)
    for block_rows in (1, 128):
        big = to_bf16(rng.normal(size=(131, 400)))
        x = big[:, 8:8 + 272]
        if x.data_ptr() % 16:
            pytest.fail("the view should be 16-byte aligned")
        qb = torch.full((135, 320), 0x55, dtype=torch.uint8, device=DEV)
        sb = torch.full((135, 7), 0x55, dtype=torch.uint8, device=DEV)
        n = -(-131 // block_rows)
        tp.tp_quantize_fp8(x, block_rows, q=qb[:131, 16:288].view(E4M3), scales=sb[:n, 2:5])
        want_c, want_b = F.quantize(f64(x), block_rows)
        q, s = qb.cpu().numpy(), sb.cpu().numpy()
        np.testing.assert_array_equal(q[:131, 16:288], want_c)
        np.testing.assert_array_equal(s[:n, 2:5], want_b)
        q[:131, 16:288] = 0x55
        s[:n, 2:5] = 0x55
        assert np.all(q == 0x55) and np.all(s == 0x55)


def test_empty_calls_write_nothing():
    x = torch.empty((0, 256), dtype=BF16, device=DEV)
    q, s = tp.tp_quantize_fp8(x)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    w, sw, _ = quantized(np.random.default_rng(0), 128, 256, 128)
    assert tp.tp_linear_colwise_fp8(q, s, [w], [sw])[0].shape == (0, 128)
    y, ys = tp.tp_linear_colwise_fp8(q, s, [w], [sw], out="fp8")
    assert y[0].shape == (0, 128) and ys[0].shape == (0, 1)
    assert tp.tp_linear_rowwise_fp8([q], [s], [w], [sw]).shape == (0, 128)
    h, u, su = tp.tp_residual_norm(x, x, out="fp8")
    assert h.shape == u.shape == (0, 256) and su.shape == (0, 2)


# ----------------------------------------------------------------------------- projections, exact

TOKENS = [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 257, 300, 520]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("K, N, p", [(16, 8, 1), (128, 128, 2), (144, 136, 3), (640, 264, 2), (1040, 520, 1)],
                         ids=lambda v: str(v))
def test_colwise_exact_integers(T, K, N, p):
    rng = np.random.default_rng(T * 7 + K)
    x, sx, xv = integers(rng, T, K, 1)
    ws = [integers(rng, N, K, 128) for _ in range(p)]
    y = tp.tp_linear_colwise_fp8(x, sx, [w[0] for w in ws], [w[1] for w in ws])
    for r in range(p):
        np.testing.assert_array_equal(f64(y[r]), bf16_round(xv @ ws[r][2].T), err_msg=f"rank {r}")


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("K, N, p", [(16, 8, 1), (128, 128, 4), (144, 136, 3), (640, 520, 2), (272, 1032, 16)],
                         ids=lambda v: str(v))
def test_rowwise_exact_integers(T, K, N, p):
    rng = np.random.default_rng(T * 11 + K)
    xs = [integers(rng, T, K, 1) for _ in range(p)]
    ws = [integers(rng, N, K, 128) for _ in range(p)]
    z = tp.tp_linear_rowwise_fp8([x[0] for x in xs], [x[1] for x in xs], [w[0] for w in ws], [w[1] for w in ws])
    np.testing.assert_array_equal(f64(z), bf16_round(sum(x[2] @ w[2].T for x, w in zip(xs, ws))))


@pytest.mark.parametrize("T, N", [(1, 384), (70, 384), (300, 384), (1300, 2176)])
def test_one_scale_at_a_time(T, N):
    """Every scale in turn is the only one that is not 1: each group of each operand has its own."""
    rng = np.random.default_rng(T)
    K = 1152
    x, sx, _ = integers(rng, T, K, 1)
    w, sw, _ = integers(rng, N, K, 128)
    for kg in range(9):
        bx, bw = np.full((T, 9), 127, np.uint8), np.full((N // 128, 9), 127, np.uint8)
        bx[T // 2, kg], bw[kg % 3, kg] = 130, 125
        y = tp.tp_linear_colwise_fp8(x, to_scales(bx), [w], [to_scales(bw)])[0]
        want = F.dequantize(codes(x), bx, 1) @ F.dequantize(codes(w), bw, 128).T
        np.testing.assert_array_equal(f64(y), bf16_round(want), err_msg=f"group {kg}")


# Prompts: sizes that take the 256 x 256 tiles of CTA pairs -- pairs alone (odd numbers of weight
# tiles) and clusters of two pairs (even), one tile a pair and several (both accumulators), ragged
# rows and columns, chunks of K that end early.
PROMPTS = [(1300, 144, 2064, 1), (2600, 272, 2064, 1), (1300, 640, 2300, 1), (2600, 528, 1160, 2), (4500, 1040, 1032, 2)]


@pytest.mark.parametrize("T, K, N, p", PROMPTS, ids=lambda v: str(v))
def test_colwise_prompt_exact_integers(T, K, N, p):
    rng = np.random.default_rng(T * 7 + K)
    N -= N % 8
    x, sx, xv = integers(rng, T, K, 1)
    ws = [integers(rng, N, K, 128) for _ in range(p)]
    y = tp.tp_linear_colwise_fp8(x, sx, [w[0] for w in ws], [w[1] for w in ws])
    for r in range(p):
        np.testing.assert_array_equal(f64(y[r]), bf16_round(xv @ ws[r][2].T), err_msg=f"rank {r}")


@pytest.mark.parametrize("T, K, N, p", PROMPTS, ids=lambda v: str(v))
def test_rowwise_prompt_exact_integers(T, K, N, p):
    rng = np.random.default_rng(T * 11 + K)
    N = p * N - p * N % 8
    xs = [integers(rng, T, K, 1) for _ in range(p)]
    ws = [integers(rng, N, K, 128) for _ in range(p)]
    z = tp.tp_linear_rowwise_fp8([x[0] for x in xs], [x[1] for x in xs], [w[0] for w in ws], [w[1] for w in ws])
    np.testing.assert_array_equal(f64(z), bf16_round(sum(x[2] @ w[2].T for x, w in zip(xs, ws))))


@pytest.mark.parametrize("T, K, N", [(1300, 272, 2304), (2600, 144, 2320)], ids=lambda v: str(v))
@pytest.mark.parametrize("out", ["bf16", "fp8"])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("bias", [False, True])
def test_colwise_prompt(T, K, N, out, act, bias):
    rng = np.random.default_rng(T + K)
    rows = 2 * N if act == "swiglu" else N     # 2320 rows on, the up block starts inside a scale block
    x, sx, xv = quantized(rng, T, K, 1, 1.5)
    w, sw, wv = quantized(rng, rows, K, 128, 1.5 / np.sqrt(K))
    b = to_bf16(rng.normal(size=rows + 1))[1 if act == "none" else 0:][:rows] if bias else None   # also not 16-byte aligned
    y = tp.tp_linear_colwise_fp8(x, sx, [w], [sw], act=act, bias_shards=[b] if bias else None, out=out)
    pre, mag = F.linear_terms(xv, wv)
    if bias:
        pre, mag = pre + f64(b), mag + np.abs(f64(b))
    err = accumulated(mag, K)
    if act == "swiglu":
        want, err = swiglu_bound(pre[:, :N], pre[:, N:], err[:, :N], err[:, N:])
    else:
        want, err = act_bound(pre, err, act)
    check_bf16(y[0], want, err) if out == "bf16" else check_fp8(y[0][0], y[1][0], want, err)


@pytest.mark.parametrize("T", [5, 300, 1300])
def test_views_and_gathered_output(T):
    """Row strides of every tensor: a replicated input read slice by slice, one gathered output."""
    rng = np.random.default_rng(3)
    K, N, p = 256, 136 if T < 1000 else 1160, 3
    x, sx, xv = integers(rng, T, p * K + 128, 1)
    ws = [integers(rng, N, K, 128) for _ in range(p)]
    wt, st = [w[0] for w in ws], [w[1] for w in ws]
    zb = torch.full((T + 3, N + 24), -7.0, dtype=BF16, device=DEV)
    cols = [slice(r * K, (r + 1) * K) for r in range(p)]
    z = tp.tp_linear_rowwise_fp8([x[:, c] for c in cols], [sx[:, 2 * r:2 * r + 2] for r in range(p)], wt, st,
                                 out=zb[:T, 8:8 + N])
    want = sum(xv[:, c] @ w[2].T for c, w in zip(cols, ws))
    np.testing.assert_array_equal(f64(z), bf16_round(want))
    rest = f64(zb)
    rest[:T, 8:8 + N] = -7
    assert np.all(rest == -7)
    g = torch.full((T + 2, p * N + 8), -7.0, dtype=BF16, device=DEV)
    tp.tp_linear_colwise_fp8(x[:, 128:128 + K], sx[:, 1:3], wt, st, y_shards=[g[:T, r * N:(r + 1) * N] for r in range(p)])
    got = f64(g)
    np.testing.assert_array_equal(got[:T, :p * N], bf16_round(np.concatenate([xv[:, 128:128 + K] @ w[2].T for w in ws], 1)))
    assert np.all(got[T:] == -7) and np.all(got[:, p * N:] == -7)


@pytest.mark.parametrize("T", [1, 5, 70, 300, 1300])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_quantised_outputs_in_views(T, act):
    """Codes and scales written through row strides, ranks side by side: the dense call's bytes, and no others."""
    rng = np.random.default_rng(T)
    p, K, N = 2, 272, 272 if T < 1000 else 2064
    g = -(-N // 128)
    x, sx, _ = quantized(rng, T, K, 1)
    ws = [quantized(rng, 2 * N if act == "swiglu" else N, K, 128, 0.05) for _ in range(p)]
    wt, st = [w[0] for w in ws], [w[1] for w in ws]
    want, want_s = tp.tp_linear_colwise_fp8(x, sx, wt, st, act=act, out="fp8")
    qb = torch.full((T + 3, p * N + 48), 0x55, dtype=torch.uint8, device=DEV)
    sb = torch.full((T + 3, p * g + 5), 0x55, dtype=torch.uint8, device=DEV)
    at = [(slice(1, T + 1), slice(16 + r * N, 16 + (r + 1) * N)) for r in range(p)]
    at_s = [(slice(1, T + 1), slice(3 + r * g, 3 + (r + 1) * g)) for r in range(p)]
    tp.tp_linear_colwise_fp8(x, sx, wt, st, act=act, out="fp8", y_shards=[qb[a].view(E4M3) for a in at],
                             y_scales=[sb[a].view(E8M0) for a in at_s])
    for r in range(p):
        assert torch.equal(qb[at[r]], want[r].view(torch.uint8)) and torch.equal(sb[at_s[r]], want_s[r].view(torch.uint8))
        qb[at[r]], sb[at_s[r]] = 0x55, 0x55
    assert bool((qb == 0x55).all()) and bool((sb == 0x55).all())


# ----------------------------------------------------------------------------- projections, in general

@pytest.mark.parametrize("T", [1, 9, 40, 100, 200, 333])
@pytest.mark.parametrize("K, N", [(144, 272), (1040, 1296)], ids=lambda v: str(v))
@pytest.mark.parametrize("out", ["bf16", "fp8"])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("bias", [False, True])
def test_colwise(T, K, N, out, act, bias):
    rng = np.random.default_rng(T + K)
    p = 2
    rows = 2 * N if act == "swiglu" else N     # 2 * 272 and 2 * 1296: the up block starts inside a scale block
    x, sx, xv = quantized(rng, T, K, 1, 1.5)
    ws = [quantized(rng, rows, K, 128, 1.5 / np.sqrt(K)) for _ in range(p)]
    bs = [to_bf16(rng.normal(size=rows)), None] if bias else None
    y = tp.tp_linear_colwise_fp8(x, sx, [w[0] for w in ws], [w[1] for w in ws], act=act, bias_shards=bs, out=out)
    for r in range(p):
        pre, mag = F.linear_terms(xv, ws[r][2])
        if bias and bs[r] is not None:
            pre, mag = pre + f64(bs[r]), mag + np.abs(f64(bs[r]))
        err = accumulated(mag, K)
        if act == "swiglu":
            want, err = swiglu_bound(pre[:, :N], pre[:, N:], err[:, :N], err[:, N:])
        else:
            want, err = act_bound(pre, err, act)
        if out == "bf16":
            check_bf16(y[r], want, err, f"rank {r}")
        else:
            check_fp8(y[0][r], y[1][r], want, err, f"rank {r}")


@pytest.mark.parametrize("T", [1, 40, 129, 333])
@pytest.mark.parametrize("K, N, p", [(144, 136, 3), (1040, 648, 4)], ids=lambda v: str(v))
@pytest.mark.parametrize("bias", [False, True])
def test_rowwise(T, K, N, p, bias):
    rng = np.random.default_rng(T + K)
    xs = [quantized(rng, T, K, 1, 1.5) for _ in range(p)]
    ws = [quantized(rng, N, K, 128, 1.5 / np.sqrt(K)) for _ in range(p)]
    b = to_bf16(rng.normal(size=N)) if bias else None
    z = tp.tp_linear_rowwise_fp8([x[0] for x in xs], [x[1] for x in xs], [w[0] for w in ws], [w[1] for w in ws], bias=b)
    terms = [F.linear_terms(x[2], w[2]) for x, w in zip(xs, ws)]
    want, mag = sum(t[0] for t in terms), sum(t[1] for t in terms)
    if bias:
        want, mag = want + f64(b), mag + np.abs(f64(b))
    check_bf16(z, want, accumulated(mag, p * (K + 31)))


@pytest.mark.parametrize("T, N", [(3, 272), (300, 272), (1300, 2064)])
@pytest.mark.parametrize("out", ["bf16", "fp8"])
def test_nan_stays_in_its_token(T, N, out):
    """A token with a NaN group is NaN in every output it has; the other tokens are as without it."""
    rng = np.random.default_rng(1)
    x = to_bf16(rng.normal(size=(T, 384)))
    w, sw, _ = quantized(rng, N - 8 if out == "bf16" else N, 384, 128, 0.05)
    clean = tp.tp_linear_colwise_fp8(*tp.tp_quantize_fp8(x), [w], [sw], out=out)
    x[1, 200] = float("nan")
    x[2, 3] = float("inf")
    x8, sx = tp.tp_quantize_fp8(x)
    got = tp.tp_linear_colwise_fp8(x8, sx, [w], [sw], out=out)
    keep = [t for t in range(T) if t not in (1, 2)]
    pairs = zip(got, clean) if out == "bf16" else [(got[0][0], clean[0][0]), (got[1][0], clean[1][0])]
    for a, b in pairs:
        np.testing.assert_array_equal(codes(a)[keep], codes(b)[keep])
        assert np.isnan(f64(a)[1:3]).all()


def test_zero_weights_and_padding_tokens():
    x8, sx = tp.tp_quantize_fp8(torch.zeros((5, 256), dtype=BF16, device=DEV))
    w8, sw = tp.tp_quantize_fp8(torch.ones((128, 256), dtype=BF16, device=DEV), 128)
    y, ys = tp.tp_linear_colwise_fp8(x8, sx, [w8], [sw], out="fp8")
    assert np.all(codes(y[0]) == 0) and np.all(codes(ys[0]) == 127)


@pytest.mark.parametrize("T, N", [(1, 136), (48, 136), (300, 136), (1300, 2056)])
def test_extreme_scales(T, N):
    """Scales at both ends of the format: 2^-127 on one operand against 2^120 on the other."""
    rng = np.random.default_rng(2)
    x = F.f64_to_e4m3(rng.integers(-4, 5, (T, 256)).astype(float))
    w = F.f64_to_e4m3(rng.integers(-4, 5, (N, 256)).astype(float))
    bx, bw = np.zeros((T, 2), np.uint8), np.full((-(-N // 128), 2), 247, np.uint8)
    y = tp.tp_linear_colwise_fp8(to_codes(x), to_scales(bx), [to_codes(w)], [to_scales(bw)])[0]
    want = F.e4m3_to_f64(x) @ F.e4m3_to_f64(w).T * 2.0 ** -7
    np.testing.assert_array_equal(f64(y), bf16_round(want))


@pytest.mark.parametrize("T", [1, 30, 300, 2600])
def test_same_bits_every_time_and_on_another_stream(T):
    rng = np.random.default_rng(4)
    x, sx, _ = quantized(rng, T, 2064, 1)
    ws = [quantized(rng, 1056, 2064, 128, 0.03) for _ in range(2)]
    wt, st = [w[0] for w in ws], [w[1] for w in ws]
    torch.cuda.synchronize()
    first = tp.tp_linear_colwise_fp8(x, sx, wt, st, act="swiglu", out="fp8")
    z0 = tp.tp_linear_rowwise_fp8([x, x], [sx, sx], wt, st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        again = tp.tp_linear_colwise_fp8(x, sx, wt, st, act="swiglu", out="fp8", stream=stream)
        z = tp.tp_linear_rowwise_fp8([x, x], [sx, sx], wt, st, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(first[0] + first[1] + [z0], again[0] + again[1] + [z]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ----------------------------------------------------------------------------- residual norm

def norm_bounds(x, y, kw, rel):
    """(h, u) and bounds: `rel` of the magnitudes that meet in each sum."""
    h, u = F.residual_norm(x, y, **kw)
    row = np.arange(x.shape[0]) // kw["rows_per_mod"]
    mag_h = np.abs(kw["alpha"] * x)
    if y is not None:
        b = normed_mag(y, kw["post_norm"], kw["eps"], kw.get("post_weight"), kw.get("post_bias"))
        mag_h = mag_h + (b if kw.get("gate") is None else np.abs(kw["gate"][row]) * b)
    eh = rel * mag_h
    if kw["norm"] == "none":
        eu, mag_u = eh, mag_h
    else:
        centre = h.mean(1, keepdims=True) if kw["norm"] == "layer" else 0.0
        s = np.sqrt(((h - centre) ** 2).mean(1, keepdims=True) + kw["eps"])
        w = 1.0 if kw.get("weight") is None else np.abs(kw["weight"])
        # h's own error, that of the mean (at most the mean of eh) and that of s (relative: rms of eh over s)
        e_rms = np.sqrt((eh ** 2).mean(1, keepdims=True))
        eu = w * (eh + (e_rms if kw["norm"] == "layer" else 0.0)) / s + w * np.abs(h - centre) / s * (e_rms / s)
        mag_u = normed_mag(h, kw["norm"], kw["eps"], kw.get("weight"), kw.get("bias"))
    if kw.get("scale") is not None:
        eu, mag_u = eu * np.abs(1 + kw["scale"][row]), mag_u * (1 + np.abs(kw["scale"][row]))
    if kw.get("shift") is not None:
        mag_u = mag_u + np.abs(kw["shift"][row])
    return h, eh, u, eu + rel * mag_u


def normed_mag(v, kind, eps, weight, bias):
    if kind == "none":
        return np.abs(v)
    centre = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    s = np.sqrt(((v - centre) ** 2).mean(1, keepdims=True) + eps)
    m = (np.abs(v) + np.abs(centre)) / s * (1.0 if weight is None else np.abs(weight))
    return m if bias is None else m + np.abs(bias)


NORM_SHAPES = [(1, 16), (3, 128), (5, 264), (7, 512), (6, 1024), (33, 1040), (9, 2064), (5, 6144), (4, 8192), (3, 8208),
               (2, 16400), (2, 32768)]


@pytest.mark.parametrize("T, D", NORM_SHAPES, ids=lambda v: str(v))
@pytest.mark.parametrize("norm, post", [("rms", "none"), ("layer", "rms"), ("none", "layer"), ("rms", "rms")])
@pytest.mark.parametrize("out", ["bf16", "fp8"])
def test_residual_norm(T, D, norm, post, out):
    if out == "fp8" and D % 16:
        D += 8
    rng = np.random.default_rng(T * 100003 + D)
    mod_rows = min(T, 3)
    per = -(-T // mod_rows)
    x, y = to_bf16(rng.normal(0.5, 2, (T, D))), to_bf16(rng.normal(-0.2, 0.6, (T, D)))
    vec = lambda c: to_bf16(rng.normal(c, 0.2, D))  # noqa: E731
    table = to_bf16(rng.normal(0, 0.4, (mod_rows, 3 * D)))
    t = dict(weight=vec(1), bias=vec(0)) if norm != "none" else {}
    if post != "none":
        t.update(post_weight=vec(1), post_bias=vec(0))
    t.update(gate=table[:, :D], scale=table[:, D:2 * D], shift=table[:, 2 * D:])
    h, u, su = tp.tp_residual_norm(x, y, norm=norm, post_norm=post, alpha=0.75, eps=1e-5, rows_per_mod=per, out=out, **t)
    kw = dict(norm=norm, post_norm=post, alpha=0.75, eps=1e-5, rows_per_mod=per, **{k: f64(v) for k, v in t.items()})
    hv, eh, uv, eu = norm_bounds(f64(x), f64(y), kw, (D + 16) * 2.0 ** -24)
    check_bf16(h, hv, eh, "h")
    check_bf16(u, uv, eu, "u") if out == "bf16" else check_fp8(u, su, uv, eu, "u")


# More rows than SMs: the kernels that hold a row in a warp or in 256 to 1024 threads of one to four
# vectors, whose rows ask for rows ahead of them (from some 300 rows on with 256 threads, 2500 with a
# warp a row), rows that fill their last vectors and rows that do not, tables whose rows are no whole
# fraction of the tokens.
NORM_MANY = [(2600, 256), (2500, 520), (161, 1024), (400, 1536), (400, 2064), (400, 2560), (310, 6144), (313, 6160),
             (400, 8192), (200, 8208), (161, 12288), (160, 16384), (160, 16400), (200, 32768)]


def norm_case(T, D, norm, post, out, mod_rows):
    """One call with every vector and table, held to norm_bounds."""
    rng = np.random.default_rng(T * 100003 + D)
    per = -(-T // mod_rows)
    x, y = to_bf16(rng.normal(0.5, 2, (T, D))), to_bf16(rng.normal(-0.2, 0.6, (T, D)))
    vec = lambda c: to_bf16(rng.normal(c, 0.2, D))  # noqa: E731
    table = to_bf16(rng.normal(0, 0.4, (mod_rows, 3 * D)))
    t = dict(weight=vec(1), bias=vec(0)) if norm != "none" else {}
    if post != "none":
        t.update(post_weight=vec(1), post_bias=vec(0))
    t.update(gate=table[:, :D], scale=table[:, D:2 * D], shift=table[:, 2 * D:])
    h, u, su = tp.tp_residual_norm(x, y, norm=norm, post_norm=post, alpha=0.75, eps=1e-5, rows_per_mod=per, out=out, **t)
    kw = dict(norm=norm, post_norm=post, alpha=0.75, eps=1e-5, rows_per_mod=per, **{k: f64(v) for k, v in t.items()})
    hv, eh, uv, eu = norm_bounds(f64(x), f64(y), kw, (D + 16) * 2.0 ** -24)
    check_bf16(h, hv, eh, "h")
    check_bf16(u, uv, eu, "u") if out == "bf16" else check_fp8(u, su, uv, eu, "u")


@pytest.mark.parametrize("T, D", NORM_MANY, ids=lambda v: str(v))
@pytest.mark.parametrize("norm, post", [("rms", "none"), ("layer", "rms"), ("none", "layer")])
@pytest.mark.parametrize("out", ["bf16", "fp8"])
def test_residual_norm_many_rows(T, D, norm, post, out):
    norm_case(T, D + 8 if out == "fp8" and D % 16 else D, norm, post, out, 3)


def test_residual_norm_of_a_prompt():
    norm_case(4608, 6144, "layer", "rms", "fp8", 5)


@pytest.mark.parametrize("T, D", [(2600, 264), (400, 2064), (400, 6144), (200, 16384)], ids=lambda v: str(v))
def test_residual_norm_forms_many_rows(T, D):
    """Without a branch, without u, in place."""
    rng = np.random.default_rng(T + D)
    x, y = to_bf16(rng.normal(0.3, 1.5, (T, D))), to_bf16(rng.normal(-0.1, 0.8, (T, D)))
    rel = (D + 16) * 2.0 ** -24
    base = dict(alpha=1.0, eps=1e-6, rows_per_mod=T, post_norm="none", norm="none")
    for norm in ("layer", "rms"):
        h, u, su = tp.tp_residual_norm(x, norm=norm)
        assert h is None and su is None
        _, _, uv, eu = norm_bounds(f64(x), None, {**base, "norm": norm}, rel)
        check_bf16(u, uv, eu, norm)
    hv, eh, _, _ = norm_bounds(f64(x), f64(y), {**base, "post_norm": "layer"}, rel)
    h, u, su = tp.tp_residual_norm(x, y, post_norm="layer", out=None)
    assert u is None and su is None
    check_bf16(h, hv, eh, "h")
    inplace = x.clone()
    h2, u2, _ = tp.tp_residual_norm(inplace, y, post_norm="layer", norm="rms", h=inplace)
    assert h2 is inplace and torch.equal(inplace, h)
    _, _, uv, eu = norm_bounds(f64(x), f64(y), {**base, "post_norm": "layer", "norm": "rms"}, rel)
    check_bf16(u2, uv, eu, "u beside an h in place")


def test_residual_norm_forms():
    """Without a branch, without an input for the next block, in place, and vectors as tables."""
    rng = np.random.default_rng(9)
    T, D = 10, 768
    x, y = to_bf16(rng.normal(size=(T, D))), to_bf16(rng.normal(size=(T, D)))
    rel = (D + 16) * 2.0 ** -24
    base = dict(alpha=1.0, eps=1e-6, rows_per_mod=T, post_norm="none", norm="none")
    h, u, su = tp.tp_residual_norm(x, norm="layer")
    assert h is None and su is None
    _, _, uv, eu = norm_bounds(f64(x), None, {**base, "norm": "layer"}, rel)
    check_bf16(u, uv, eu)
    g = to_bf16(rng.normal(size=D))
    hv, eh, _, _ = norm_bounds(f64(x), f64(y), {**base, "post_norm": "rms", "gate": f64(g)[None]}, rel)
    h, u, su = tp.tp_residual_norm(x, y, post_norm="rms", gate=g, out=None)
    assert u is None and su is None
    check_bf16(h, hv, eh)
    inplace = x.clone()
    tp.tp_residual_norm(inplace, y, post_norm="rms", gate=g, out=None, h=inplace)
    assert torch.equal(inplace, h)
    q, s = tp.tp_residual_norm(x, norm="none", out="fp8")[1:]     # a plain quantiser
    q2, s2 = tp.tp_quantize_fp8(x)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s.view(torch.uint8), s2.view(torch.uint8))


def test_residual_norm_strides_and_neighbours():
    rng = np.random.default_rng(10)
    T, D = 6, 528
    bx, by = to_bf16(rng.normal(size=(T, D + 40))), to_bf16(rng.normal(size=(T, D + 16)))
    hb = torch.full((T + 2, D + 32), -7.0, dtype=BF16, device=DEV)
    ub = torch.full((T + 2, D + 48), 0x55, dtype=torch.uint8, device=DEV)
    sb = torch.full((T + 2, 9), 0x55, dtype=torch.uint8, device=DEV)
    kw = dict(norm="rms", post_norm="layer", alpha=-1.5)
    tp.tp_residual_norm(bx[:, 16:16 + D], by[:, 8:8 + D], out="fp8", h=hb[1:T + 1, 8:8 + D],
                        u=ub[1:T + 1, 16:16 + D].view(E4M3), u_scales=sb[1:T + 1, 3:8], **kw)
    h, u, su = tp.tp_residual_norm(bx[:, 16:16 + D].contiguous(), by[:, 8:8 + D].contiguous(), out="fp8", **kw)
    assert torch.equal(hb[1:T + 1, 8:8 + D], h)
    assert torch.equal(ub[1:T + 1, 16:16 + D], u.view(torch.uint8)) and torch.equal(sb[1:T + 1, 3:8], su.view(torch.uint8))
    hb[1:T + 1, 8:8 + D], ub[1:T + 1, 16:16 + D], sb[1:T + 1, 3:8] = -7.0, 0x55, 0x55
    assert bool((hb == -7).all()) and bool((ub == 0x55).all()) and bool((sb == 0x55).all())


def test_residual_norm_special_rows():
    """Rows of zeros, infinities and NaN keep to themselves; a large common offset keeps its spread (layer)."""
    rng = np.random.default_rng(11)
    x = to_bf16(rng.normal(size=(5, 256)))
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 7] = float("inf")
    _, u, _ = tp.tp_residual_norm(x, norm="rms")
    v = f64(u)
    assert np.all(v[1] == 0) and np.isnan(v[2]).all() and np.isnan(v[3, 7]) and np.all(v[3, :7] == 0)
    assert np.isfinite(v[[0, 4]]).all()
    q, s = tp.tp_residual_norm(x, norm="rms", out="fp8")[1:]
    b = codes(s)
    assert np.all(b[2] == 255) and b[3, 0] == 255 and b[3, 1] == 127 and np.all(b[1] == 127)
    big = to_bf16(4096 + 16 * rng.integers(-8, 8, (4, 512)))     # exact in bf16
    _, u, _ = tp.tp_residual_norm(big, norm="layer", eps=0.0)
    _, want = F.residual_norm(f64(big), norm="layer", eps=0.0)
    assert np.max(np.abs(f64(u) - want)) <= 2.0 ** -8 * np.max(np.abs(want)) + 1e-3


# ----------------------------------------------------------------------------- together

def sharded_block(T, H, FF, p, seed=0):
    """Weights of one norm -> gate/up -> down block, sharded by the library and quantised shard by shard."""
    rng = np.random.default_rng(seed)
    gu, dn = to_bf16(rng.normal(0, 0.05, (2 * FF, H))), to_bf16(rng.normal(0, 0.05, (H, FF)))
    gus = [tp.tp_quantize_fp8(w, 128) for w in tp.tp_plan_shard_ranks(gu, "colwise", p, fused_splits=[FF, FF])]
    dns = [tp.tp_quantize_fp8(w, 128) for w in tp.tp_plan_shard_ranks(dn, "rowwise", p)]
    x, gate = to_bf16(rng.normal(size=(T, H))), to_bf16(rng.normal(0, 0.5, H))
    return x, gate, [list(v) for v in zip(*gus)], [list(v) for v in zip(*dns)]


def forward(x, gate, gu, dn, stream=None):
    _, u, su = tp.tp_residual_norm(x, norm="rms", out="fp8", stream=stream)
    h, hs = tp.tp_linear_colwise_fp8(u, su, *gu, act="swiglu", out="fp8", stream=stream)
    z = tp.tp_linear_rowwise_fp8(h, hs, *dn, stream=stream)
    x2, u2, _ = tp.tp_residual_norm(x, z, norm="rms", post_norm="rms", gate=gate, stream=stream)
    return u, su, h, hs, z, x2, u2


@pytest.mark.parametrize("T", [1, 19, 300, 3000])
@pytest.mark.parametrize("p", [1, 2, 4])
def test_block_of_all_operators(T, p):
    """Each step from the stored output of the step before, against the oracle."""
    H, FF = 512, 1024
    x, gate, gu, dn = sharded_block(T, H, FF, p)
    u, su, h, hs, z, x2, u2 = forward(x, gate, gu, dn)
    rel = (H + 16) * 2.0 ** -24
    base = dict(alpha=1.0, eps=1e-6, rows_per_mod=T, post_norm="none", norm="rms")
    _, _, uv, eu = norm_bounds(f64(x), None, base, rel)
    check_fp8(u, su, uv, eu, "pre-norm")
    xin = F.dequantize(codes(u), codes(su), 1)
    n = FF // p
    for r in range(p):
        w = F.dequantize(codes(gu[0][r]), codes(gu[1][r]), 128)
        pre, mag = F.linear_terms(xin, w)
        err = accumulated(mag, H)
        want, err = swiglu_bound(pre[:, :n], pre[:, n:], err[:, :n], err[:, n:])
        check_fp8(h[r], hs[r], want, err, f"gate/up rank {r}")
    terms = [F.linear_terms(F.dequantize(codes(h[r]), codes(hs[r]), 1), F.dequantize(codes(dn[0][r]), codes(dn[1][r]), 128))
             for r in range(p)]
    check_bf16(z, sum(t[0] for t in terms), accumulated(sum(t[1] for t in terms), FF), "down")
    hv, eh, uv, eu = norm_bounds(f64(x), f64(z), {**base, "post_norm": "rms", "gate": f64(gate)[None]}, rel)
    check_bf16(x2, hv, eh, "residual")
    check_bf16(u2, uv, eu, "next input")


@pytest.mark.parametrize("T", [1, 300, 3000])
def test_block_captured_and_replayed(T):
    """The block in a CUDA graph, replayed on new inputs, gives the eager calls' bits; two graphs at once too."""
    args = [sharded_block(T, 512, 1024, 2, seed) for seed in (1, 2)]
    for a in args:
        forward(*a)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(forward(*a))
        graphs.append(g)
    rng = np.random.default_rng(20)
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(3):
        for a in args:
            a[0].copy_(to_bf16(rng.normal(size=tuple(a[0].shape))))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, got in zip(args, outs):
            want = forward(*a)
            torch.cuda.synchronize()
            for i in (0, 1, 4, 5, 6):
                assert torch.equal(got[i].view(torch.uint8), want[i].view(torch.uint8)), i


@pytest.mark.parametrize("T", [1, 24, 260])
def test_buffers_written_anew_between_launches(T):
    """Calls queued without a pause, each reading what the one before wrote into the same buffers anew.

    A launch's CTAs may be on their SMs while the launch before the last still reads the old
    contents through the same L1: codes, scales, and the tables of the residual norm."""
    rng = np.random.default_rng(31)
    K, N, steps = 512, 512, 24
    w, sw, _ = quantized(rng, N, K, 128, 0.05)
    xs = [to_bf16(rng.normal(0, 10.0 ** (i % 5 - 2), size=(T, K))) for i in range(steps)]
    q, s = tp.tp_quantize_fp8(xs[0])
    table, hold = torch.empty_like(xs[0]), [torch.empty_like(xs[0]) for _ in range(steps)]
    ys = [torch.empty((T, N), dtype=BF16, device=DEV) for _ in range(steps)]

    def step(i):
        tp.tp_residual_norm(xs[i], norm="layer", u=table)
        tp.tp_residual_norm(xs[i - 1], xs[i], out="fp8", norm="rms", gate=table, scale=table, shift=table,
                            rows_per_mod=1, h=hold[i], u=q, u_scales=s)
        tp.tp_linear_colwise_fp8(q, s, [w], [sw], y_shards=[ys[i]])

    for i in range(steps):
        step(i)
        torch.cuda.synchronize()
    want = [(h.clone(), y.clone()) for h, y in zip(hold, ys)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(steps):
            step(i)
    for _ in range(10):
        for t in hold + ys:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for i in range(steps):
            assert torch.equal(hold[i], want[i][0]) and torch.equal(ys[i], want[i][1]), i


def test_calls_on_several_streams_at_once():
    args = [sharded_block(T, 512, 1024, 2, T) for T in (1, 40, 200, 3000)]
    want = [forward(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(5):
        got = [forward(*a, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert torch.equal(w[6], g[6]) and torch.equal(w[4], g[4])


def test_calls_from_several_threads():
    import threading
    args = [sharded_block(T, 512, 1024, 2, T) for T in (3, 70, 520)]
    want = [forward(*a) for a in args]
    torch.cuda.synchronize()
    got, errors = [None] * len(args), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got[i] = forward(*args[i], stream=s)
            s.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(args))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[6], g[6]) and torch.equal(w[4], g[4])


@pytest.mark.parametrize("T", [5, 1300])
def test_one_tensor_for_several_ranks(T):
    """The same operands as every rank's: each colwise output alike, the rowwise sum p times one product."""
    rng = np.random.default_rng(32)
    x, sx, xv = integers(rng, T, 256, 1)
    w, sw, wv = integers(rng, 2064, 256, 128)
    ys = tp.tp_linear_colwise_fp8(x, sx, [w] * 3, [sw] * 3)
    for y in ys:
        np.testing.assert_array_equal(f64(y), bf16_round(xv @ wv.T))
    z = tp.tp_linear_rowwise_fp8([x] * 4, [sx] * 4, [w] * 4, [sw] * 4)
    np.testing.assert_array_equal(f64(z), bf16_round(4 * (xv @ wv.T)))


def test_offsets_past_32_bits():
    """Rows whose bytes start beyond 4 GiB: a long quantised activation, outputs and inputs with a huge row stride."""
    rng = np.random.default_rng(30)
    T, K = 70016, 32768
    x = torch.zeros((T, K), dtype=BF16, device=DEV)
    last = to_bf16(rng.normal(size=(2, K)))
    x[-2:] = last
    q, s = tp.tp_quantize_fp8(x)
    q2, s2 = tp.tp_quantize_fp8(last)
    assert torch.equal(q[-2:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-2:].view(torch.uint8),
                                                                                        s2.view(torch.uint8))
    assert int(q[:-2].view(torch.uint8).count_nonzero()) == 0
    _, u, _ = tp.tp_residual_norm(x, norm="rms")
    assert torch.equal(u[-2:], tp.tp_residual_norm(last, norm="rms")[1])
    w, sw, _ = quantized(rng, 2176, K, 128, 0.01)
    few = tp.tp_linear_colwise_fp8(q2, s2, [w], [sw])[0]
    long = tp.tp_linear_colwise_fp8(q, s, [w], [sw])[0]
    assert float((long[-2:].float() - few.float()).abs().max()) <= 2.0 ** -6 * float(few.float().abs().max())
    assert int(long[:-2].count_nonzero()) == 0
    del x, q, u, long
    for T, N in ((40, 136), (2600, 2064)):       # either kernel, rows 8 MiB apart and more
        wide = torch.full((T, (1 << 32) // T // 64 * 64), -7.0, dtype=BF16, device=DEV)
        a, sa, av = integers(rng, T, 256, 1)
        b, sb, bv = integers(rng, N, 256, 128)
        z = tp.tp_linear_rowwise_fp8([a], [sa], [b], [sb], out=wide[:, 64:64 + N])
        np.testing.assert_array_equal(f64(z), bf16_round(av @ bv.T))
        h, _, _ = tp.tp_residual_norm(z.contiguous(), z.contiguous(), out=None, h=wide[:, 8192:8192 + N])
        assert torch.equal(h, (2 * z.float()).to(BF16))
        assert int((wide[:, 64 + N:8192] != -7).count_nonzero()) == 0
        del wide, z, h


@pytest.mark.parametrize("T", [40, 2600])
def test_codes_past_four_gib(T):
    """Codes, scales and quantised outputs whose last rows start beyond 2^32 bytes, through both projection kernels."""
    rng = np.random.default_rng(T)
    K, N = 256, 2064
    step = (1 << 32) // (T - 4) // 64 * 64 + 64              # the last three rows start past 2^32
    assert (T - 3) * step > 1 << 32
    wide = [torch.full((T, step), 0x55, dtype=torch.uint8, device=DEV) for _ in range(4)]
    q, s = wide[0][:, 32:32 + K].view(E4M3), wide[1][:, 3:5]
    x = to_bf16(rng.normal(size=(T, K)))
    tp.tp_quantize_fp8(x, q=q, scales=s)
    q2, s2 = tp.tp_quantize_fp8(x)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2.view(torch.uint8))
    w, sw, _ = quantized(rng, N, K, 128, 0.05)
    y, ys = wide[2][:, 16:16 + N].view(E4M3), wide[3][:, 5:5 + 17]
    tp.tp_linear_colwise_fp8(q, s, [w], [sw], out="fp8", y_shards=[y], y_scales=[ys])
    y2, ys2 = tp.tp_linear_colwise_fp8(q2, s2, [w], [sw], out="fp8")
    assert torch.equal(y.view(torch.uint8), y2[0].view(torch.uint8)) and torch.equal(ys, ys2[0].view(torch.uint8))
    wide[0][:, 32:32 + K], wide[1][:, 3:5], wide[2][:, 16:16 + N], wide[3][:, 5:5 + 17] = 0x55, 0x55, 0x55, 0x55
    for b in wide:
        assert int(b.min()) == int(b.max()) == 0x55


def test_first_call_may_be_captured():
    """In a new process, whose first use of the library is inside a capture."""
    import subprocess
    import sys
    code = """
import sys, torch
sys.path.insert(0, %r)
import tensor_sharded_linear_tp_gb300 as tp
mode = sys.argv[1]
T = 4 if mode == "few" else 1300
x = torch.randn(T, 512, device="cuda").to(torch.bfloat16)
w8 = torch.zeros(2064, 512, device="cuda").to(torch.float8_e4m3fn)
ws = torch.full((17, 4), 127, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    _, u, su = tp.tp_residual_norm(x, norm="rms", out="fp8")
    q, s = tp.tp_quantize_fp8(x)
    y = tp.tp_linear_colwise_fp8(u, su, [w8], [ws])[0]
    z = tp.tp_linear_rowwise_fp8([q], [s], [w8], [ws])
y.fill_(1), z.fill_(1)
g.replay()
torch.cuda.synchronize()
tp.tp_device_status()
assert int(y.count_nonzero()) == 0 and int(z.count_nonzero()) == 0
print("replayed")
""" % tp.__file__.rsplit("/", 2)[0]
    for mode in ("few", "many"):
        r = subprocess.run([sys.executable, "-c", code, mode], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and "replayed" in r.stdout, (mode, r.stdout[-500:], r.stderr[-2000:])


@pytest.mark.parametrize("T", [13, 14, 16, 27, 31, 37, 61, 71, 100, 115])
@pytest.mark.parametrize("out", ["bf16", "fp8"])
def test_join_of_uneven_shares(T, out):
    """K on two CTAs (71 tiles of four chunks), whose shares of the tokens are no multiple of the
    24 that six warps join four at a time: a warp's last turn has tokens, and the last tile columns, past the share."""
    N = 8968 if out == "bf16" else 8976
    rng = np.random.default_rng(T + N)
    x, sx, xv = integers(rng, T, 2048, 1)
    w, sw, wv = integers(rng, N, 2048, 128)
    want = xv @ wv.T
    for _ in range(3):
        y = tp.tp_linear_colwise_fp8(x, sx, [w], [sw], out=out)
        if out == "bf16":
            np.testing.assert_array_equal(f64(y[0]), bf16_round(want))
        else:
            c, b = F.quantize(want, 1)
            np.testing.assert_array_equal(codes(y[1][0]), b)
            np.testing.assert_array_equal(F.e4m3_to_f64(codes(y[0][0])), F.e4m3_to_f64(c))


# ----------------------------------------------------------------------------- refusals on the GPU's side

def test_binding_refusals():
    rng = np.random.default_rng(0)
    x, sx, _ = quantized(rng, 4, 256, 1)
    w, sw, _ = quantized(rng, 128, 256, 128)
    xb = torch.zeros((4, 256), dtype=BF16, device=DEV)
    bad = [
        (TypeError, lambda: tp.tp_quantize_fp8(xb.float())),
        (ValueError, lambda: tp.tp_quantize_fp8(xb, 64)),
        (ValueError, lambda: tp.tp_quantize_fp8(xb[:, ::2])),
        (ValueError, lambda: tp.tp_quantize_fp8(xb[0])),
        (ValueError, lambda: tp.tp_quantize_fp8(xb, q=torch.empty((4, 128), dtype=torch.uint8, device=DEV).view(E4M3))),
        (ValueError, lambda: tp.tp_quantize_fp8(xb, scales=torch.empty((4, 3), dtype=torch.uint8, device=DEV))),
        (ValueError, lambda: tp.tp_quantize_fp8(xb[:1].expand(4, 256))),
        (tp.TPError, lambda: tp.tp_quantize_fp8(torch.zeros((4, 264), dtype=BF16, device=DEV))),
        (TypeError, lambda: tp.tp_linear_colwise_fp8(xb, sx, [w], [sw])),
        (ValueError, lambda: tp.tp_linear_colwise_fp8(x, sx[:, :1], [w], [sw])),
        (ValueError, lambda: tp.tp_linear_colwise_fp8(x, sx, [w], [sw, sw])),
        (ValueError, lambda: tp.tp_linear_colwise_fp8(x, sx, [], [])),
        (ValueError, lambda: tp.tp_linear_colwise_fp8(x, sx, [w, w[:64]], [sw, sw])),
        (ValueError, lambda: tp.tp_linear_colwise_fp8(x, sx, [w], [sw], out="fp4")),
        (ValueError, lambda: tp.tp_linear_colwise_fp8(x, sx, [w], [sw], y_scales=[sx])),
        (KeyError, lambda: tp.tp_linear_colwise_fp8(x, sx, [w], [sw], act="relu")),
        (ValueError, lambda: tp.tp_linear_colwise_fp8(x, sx, [w], [sw], bias_shards=[xb[0]])),
        (ValueError, lambda: tp.tp_linear_colwise_fp8(x, sx, [w.cpu()], [sw])),
        (ValueError, lambda: tp.tp_linear_rowwise_fp8([x, x[:3]], [sx, sx], [w, w], [sw, sw])),
        (ValueError, lambda: tp.tp_linear_rowwise_fp8([x], [sx], [w], [sw], bias=xb[0])),
        (TypeError, lambda: tp.tp_linear_rowwise_fp8([x], [sx], [w], [sw], out=xb.float()[:, :128])),
        (ValueError, lambda: tp.tp_residual_norm(xb, xb[:3])),
        (ValueError, lambda: tp.tp_residual_norm(xb, gate=xb[0], y=xb, scale=xb)),
        (tp.TPError, lambda: tp.tp_residual_norm(xb, xb, gate=xb[:2], rows_per_mod=1)),
        (tp.TPError, lambda: tp.tp_residual_norm(xb, gate=xb[0])),
        (ValueError, lambda: tp.tp_residual_norm(xb, out="fp4")),
        (ValueError, lambda: tp.tp_residual_norm(xb, out=None, u=xb)),
    ]
    for i, (exc, call) in enumerate(bad):
        with pytest.raises(exc):
            call()
            pytest.fail(f"call {i} was not refused")
