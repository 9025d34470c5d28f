"""The paged cache on the CPU: the oracle against closed forms, and every refusal of the C calls before any device work."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from oracle import paged_oracle as P

tp = pytest.importorskip("tensor_sharded_linear_tp_gb300",
                         reason="libtp.so not built (python tensor_sharded_linear_tp_gb300/build.py)")

FAKE = 0x10000   # 16-byte aligned, never dereferenced: every call below is refused first, or enqueues nothing


# ----------------------------------------------------------------------------- the oracle

def test_rotation_turns_pairs_by_their_angle():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 2, 32))
    angle = rng.uniform(-9, 9, (3, 8))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    for style, (a, b) in {"half": (np.arange(8), np.arange(8) + 8), "pairs": (2 * np.arange(8), 2 * np.arange(8) + 1)}.items():
        y = P.rotate(x, cs, style)
        turned = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle)[:, None]
        np.testing.assert_allclose(y[..., a] + 1j * y[..., b], turned, atol=1e-12)
        np.testing.assert_array_equal(y[..., 16:], x[..., 16:])


def test_append_in_any_portions_keeps_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(70, 2, 64)) * 2.0 ** rng.integers(-3, 4, (70, 1, 1))
    x[5] = 0
    table = np.array([[4, 0, 2, 1, 3]])
    for cuts in ([70], [1] * 70, [3, 14, 1, 20, 32]):
        codes = rng.integers(0, 256, (5, 2, 16, 64)).astype(np.uint8)
        scales = rng.integers(0, 256, (5, 2)).astype(np.uint8)
        done = 0
        for n in cuts:
            P.append(codes, scales, x[done:done + n], [(0, n, done + n)], table)
            done += n
        got = P.values(codes, scales, table[0], 70)
        size = np.repeat(F.scale_value(scales[table[0]]).T, 16, 1)[:, :70, None]
        want = x.transpose(1, 0, 2)
        # one rounding to a code, and for portions further ones only among the subnormal codes (half a step of 2^-9 each)
        turns = 1 if len(cuts) == 1 else 8
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), turns * 2.0 ** -10 * size))
        before = codes.copy(), scales.copy()
        P.append(codes, scales, x[67:], [(0, 3, 70)], table)
        np.testing.assert_array_equal(codes, before[0])
        np.testing.assert_array_equal(scales, before[1])


def test_attention_closed_forms():
    V = np.arange(12.0).reshape(1, 6, 2)
    q, K = np.zeros((3, 1, 2)), np.ones((1, 6, 2))
    out, _ = P.attention(q, K, V, 1.0, P.seen(3, 6))          # equal weights: means of what is seen
    np.testing.assert_allclose(out[:, 0, 0], [3.0, 4.0, 5.0])
    out, _ = P.attention(q, K, V, 1.0, P.seen(3, 6, window=2))
    np.testing.assert_allclose(out[:, 0, 0], [5.0, 7.0, 9.0])
    out, _ = P.attention(np.zeros((4, 1, 2)), K[:, :2], V[:, :2], 1.0, P.seen(4, 2))
    np.testing.assert_allclose(out[:, 0, 0], [0, 0, 0, 1.0])   # two rows before the first key
    q[0, 0] = 50.0
    K[0, 2] = 20.0
    out, _ = P.attention(q, K, V, 1.0, P.seen(3, 6, causal=False))
    np.testing.assert_allclose(out[0, 0], V[0, 2])


def test_a_masked_nan_stays_out():
    V = np.ones((1, 4, 2))
    V[0, 3] = np.nan
    out, _ = P.attention(np.zeros((2, 1, 2)), np.ones((1, 4, 2)), V, 1.0, P.seen(2, 4))
    assert np.all(out[0] == 1) and np.all(np.isnan(out[1]))


# ----------------------------------------------------------------------------- refusals of the C calls

class Cache(ctypes.Structure):
    _fields_ = [("n_ranks", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_size", ctypes.c_int), ("n_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("ld_page", ctypes.c_int64),
                ("ld_scales", ctypes.c_int64)]


class Batch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("max_new", ctypes.c_int), ("seq_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
                ("max_pages", ctypes.c_int64)]


class Rope(ctypes.Structure):
    _fields_ = [("style", ctypes.c_int), ("rot_dim", ctypes.c_int), ("cos_sin", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("n_positions", ctypes.c_int64), ("positions", ctypes.c_void_p)]


def _array(v, n):
    return None if v is None else (ctypes.c_void_p * 16)(*[v] * max(1, min(n, 16)))


def _parts(kw):
    """The structures of a sound call, with the fields in kw replaced (taken out of it)."""
    n = kw.get("n_ranks", 2)
    arrays = {f: _array(kw.pop(f + "_at", FAKE), n) for f in ("k", "v", "k_scales", "v_scales")}
    for f in arrays:
        if kw.pop(f + "_none", False):
            arrays[f] = None
    c = Cache(2, 4, 128, 16, 10, *[None if a is None else ctypes.addressof(a) for a in arrays.values()], 0, 0)
    b = Batch(3, 5, FAKE, FAKE, FAKE, 0, 6)
    r = Rope(0, 64, FAKE, 0, 100, None)
    for s in (c, b, r):
        for f, _ in s._fields_:
            if f in kw:
                setattr(s, f, kw.pop(f))
    return c, b, r, arrays


COMMON = [
    (dict(n_ranks=0), "TP_ERR_INVALID_ARG"), (dict(n_ranks=17), "TP_ERR_UNSUPPORTED"),
    (dict(n_kv_heads=0), "TP_ERR_INVALID_ARG"), (dict(head_dim=96), "TP_ERR_UNSUPPORTED"),
    (dict(head_dim=256), "TP_ERR_UNSUPPORTED"), (dict(page_size=8), "TP_ERR_UNSUPPORTED"),
    (dict(page_size=48), "TP_ERR_UNSUPPORTED"), (dict(n_pages=-1), "TP_ERR_INVALID_ARG"),
    (dict(n_pages=1 << 31), "TP_ERR_UNSUPPORTED"), (dict(T=-1), "TP_ERR_INVALID_ARG"),
    (dict(T=1 << 31), "TP_ERR_UNSUPPORTED"), (dict(n_seqs=-1), "TP_ERR_INVALID_ARG"),
    (dict(max_new=-1), "TP_ERR_INVALID_ARG"), (dict(max_pages=-1), "TP_ERR_INVALID_ARG"),
    (dict(max_pages=1 << 28), "TP_ERR_UNSUPPORTED"), (dict(n_seqs=1 << 25), "TP_ERR_UNSUPPORTED"),
    (dict(ld_page=4 * 16 * 128 - 16), "TP_ERR_INVALID_ARG"), (dict(ld_page=4 * 16 * 128 + 8), "TP_ERR_ALIGNMENT"),
    (dict(ld_scales=3), "TP_ERR_INVALID_ARG"), (dict(ld_table=5), "TP_ERR_INVALID_ARG"),
    (dict(k_at=None), "TP_ERR_INVALID_ARG"), (dict(v_at=FAKE + 8), "TP_ERR_ALIGNMENT"),
    (dict(k_none=True), "TP_ERR_INVALID_ARG"), (dict(v_scales_none=True), "TP_ERR_INVALID_ARG"),
    (dict(k_scales_at=None), "TP_ERR_INVALID_ARG"), (dict(seq_start=None), "TP_ERR_INVALID_ARG"),
    (dict(kv_len=None), "TP_ERR_INVALID_ARG"), (dict(page_table=None), "TP_ERR_INVALID_ARG"),
    (dict(page_table=FAKE + 2), "TP_ERR_ALIGNMENT"), (dict(n_heads=-1), "TP_ERR_INVALID_ARG"),
    (dict(T=0), "TP_OK"), (dict(n_seqs=0), "TP_OK"), (dict(max_new=0), "TP_OK"),
    (dict(T=0, k_none=True, seq_start=None), "TP_OK"), (dict(T=0, head_dim=32), "TP_ERR_UNSUPPORTED"),
]


@pytest.mark.parametrize("kw, want", COMMON + [
    (dict(ld_qkv=16 * 128 - 8), "TP_ERR_INVALID_ARG"), (dict(ld_qkv=16 * 128 + 4), "TP_ERR_ALIGNMENT"),
    (dict(ld_q=8 * 128 - 8), "TP_ERR_INVALID_ARG"), (dict(ld_q=8 * 128 + 4), "TP_ERR_ALIGNMENT"),
    (dict(qkv=None), "TP_ERR_INVALID_ARG"), (dict(qkv=FAKE + 2), "TP_ERR_ALIGNMENT"), (dict(q_out=None), "TP_ERR_INVALID_ARG"),
    (dict(q_out=FAKE + 8), "TP_ERR_ALIGNMENT"), (dict(style=2), "TP_ERR_INVALID_ARG"), (dict(rot_dim=0), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=24), "TP_ERR_INVALID_ARG"), (dict(rot_dim=144), "TP_ERR_INVALID_ARG"), (dict(ld=48), "TP_ERR_INVALID_ARG"),
    (dict(ld=66), "TP_ERR_ALIGNMENT"), (dict(cos_sin=None), "TP_ERR_INVALID_ARG"), (dict(cos_sin=FAKE + 4), "TP_ERR_ALIGNMENT"),
    (dict(n_positions=-1), "TP_ERR_INVALID_ARG"), (dict(positions=FAKE + 1), "TP_ERR_ALIGNMENT"),
    (dict(no_cache=True), "TP_ERR_INVALID_ARG"), (dict(no_batch=True), "TP_ERR_INVALID_ARG"),
])
def test_append_refusals(kw, want):
    kw = dict(kw)
    n = kw.get("n_ranks", 2)
    c, b, r, keep = _parts(kw)
    qkv, q_out = _array(kw.pop("qkv", FAKE), n), _array(kw.pop("q_out", FAKE), n)
    st = tp.lib.tp_kv_append_fp8(None if kw.pop("no_cache", False) else ctypes.byref(c),
                                 None if kw.pop("no_batch", False) else ctypes.byref(b),
                                 ctypes.addressof(qkv) if qkv is not None else None, kw.pop("ld_qkv", 0), kw.pop("T", 7),
                                 kw.pop("n_heads", 8), ctypes.byref(r),
                                 ctypes.addressof(q_out) if q_out is not None else _null16(), kw.pop("ld_q", 0), None)
    assert not kw and tp.STATUS_NAMES[st] == want, tp.tp_last_error()


_NULLS = (ctypes.c_void_p * 16)()


def _null16():
    return ctypes.addressof(_NULLS)


def _attend(kw):
    n = kw.get("n_ranks", 2)
    c, b, _, keep = _parts(kw)
    q, out = _array(kw.pop("q", FAKE), n), _array(kw.pop("out", FAKE), n)
    T, heads = kw.pop("T", 7), kw.pop("n_heads", 8)
    st = tp.lib.tp_attention_paged_fp8(None if kw.pop("no_cache", False) else ctypes.byref(c), ctypes.byref(b),
                                       ctypes.addressof(q) if q is not None else None, kw.pop("ld_q", 0), T, heads,
                                       kw.pop("scale", 0.1), kw.pop("causal", 1), kw.pop("window", 0), FAKE, 1 << 40,
                                       ctypes.addressof(out) if out is not None else None, kw.pop("ldo", 0), None)
    assert not kw
    return tp.STATUS_NAMES[st]


@pytest.mark.parametrize("kw, want", COMMON + [
    (dict(n_heads=0), "TP_ERR_INVALID_ARG"), (dict(n_heads=6), "TP_ERR_INVALID_ARG"),
    (dict(ld_q=1016), "TP_ERR_INVALID_ARG"), (dict(ld_q=1028), "TP_ERR_ALIGNMENT"), (dict(ldo=1016), "TP_ERR_INVALID_ARG"),
    (dict(ldo=1028), "TP_ERR_ALIGNMENT"), (dict(q=None), "TP_ERR_INVALID_ARG"), (dict(q=FAKE + 8), "TP_ERR_ALIGNMENT"),
    (dict(out=None), "TP_ERR_INVALID_ARG"), (dict(out=FAKE + 2), "TP_ERR_ALIGNMENT"), (dict(causal=2), "TP_ERR_INVALID_ARG"),
    (dict(window=-1), "TP_ERR_INVALID_ARG"), (dict(window=5, causal=0), "TP_ERR_INVALID_ARG"),
    (dict(scale=3e38), "TP_ERR_INVALID_ARG"),
    (dict(n_seqs=1 << 20, max_pages=1 << 16, n_kv_heads=2, n_heads=2), "TP_ERR_UNSUPPORTED"),
    (dict(scale=float("nan")), "TP_ERR_INVALID_ARG"), (dict(scale=float("inf")), "TP_ERR_INVALID_ARG"),
    (dict(no_cache=True), "TP_ERR_INVALID_ARG"), (dict(n_kv_heads=40000, n_heads=40000), "TP_ERR_UNSUPPORTED"),
])
def test_attention_refusals(kw, want):
    assert _attend(dict(kw)) == want, tp.tp_last_error()


def test_workspace_of_a_refused_or_empty_call_is_nothing():
    for kw in (dict(head_dim=80), dict(T=0), dict(n_seqs=0)):
        T = kw.pop("T", 7)
        c, b, _, keep = _parts(kw)
        assert tp.lib.tp_attention_paged_workspace_bytes(ctypes.byref(c), ctypes.byref(b), T, 8) == 0


# ----------------------------------------------------------------------------- the binding

def test_structures_match_the_packed_bytes():
    c, b, r, keep = _parts({})
    assert len(tp._paged_cache(2, 4, 128, 16, 10, 1, 2, 3, 4, 0, 0)) == ctypes.sizeof(c)
    assert len(tp._paged_batch(3, 5, 1, 2, 3, 0, 6)) == ctypes.sizeof(b)
    assert len(tp._rope(0, 64, 1, 0, 100, 0)) == ctypes.sizeof(r)
    assert bytes(Batch(3, 5, 17, 18, 19, 7, 6)) == tp._paged_batch(3, 5, 17, 18, 19, 7, 6)
    assert bytes(Rope(1, 64, 17, 4, 100, 18)) == tp._rope(1, 64, 17, 4, 100, 18)


def test_binding_wants_device_tensors():
    codes = [torch.zeros((2, 1, 16, 64), dtype=torch.float8_e4m3fn)]
    scales = [torch.zeros((2, 1), dtype=torch.uint8)]
    with pytest.raises(ValueError, match="CUDA"):
        tp.PagedCache(codes, codes, scales, scales)
    i32 = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tp.PagedBatch(i32[0], i32[0, :1], i32, 1)
    with pytest.raises(ValueError):
        tp.PagedCache([], [], [], [])


def test_a_batchs_rows_have_two_names():
    """max_new and max_q name the same argument; one of them has to be there (the tensors are checked after it)."""
    i32 = torch.zeros((1, 2), dtype=torch.int32)
    for kw in (dict(max_new=1), dict(max_q=1)):
        with pytest.raises(ValueError, match="CUDA"):
            tp.PagedBatch(i32[0], i32[0, :1], i32, **kw)
    for args, kw in (((), {}), ((1,), dict(max_q=1)), ((), dict(max_new=1, max_q=1))):
        with pytest.raises(TypeError, match="max_q"):
            tp.PagedBatch(i32[0], i32[0, :1], i32, *args, **kw)


def test_the_build_checks_the_registers_of_a_split_kernel():
    """The many-rows kernel's warpgroups share 128 registers a thread out; a build that has others is refused."""
    from tensor_sharded_linear_tp_gb300 import build

    def log(n, m):
        entry = ("ptxas info    : Compiling entry function '_ZN2tp18paged_tiles_kernelILi{}EEEv' for 'sm_103a'\n    0 bytes stack frame\n"
                 "ptxas info    : Used {} registers, used 1 barriers\n")
        return entry.format(64, n) + entry.format(128, m) + entry.replace("tiles", "join").format(64, 60)
    build.check_registers("tp_paged_tiles.cu", log(128, 128))
    build.check_registers("tp_gemm.cu", log(40, 40))
    for text in (log(128, 120), log(96, 128), ""):
        with pytest.raises(RuntimeError, match="128 registers"):
            build.check_registers("tp_paged_tiles.cu", text)
