"""The paged 8-bit cache against float64 numpy: appending with rotation, attention, and both as they are used together.

Unrotated keys, values, and rotations by quarter turns (cosines and sines of 0, 1 and -1) have one
right code and are compared bit for bit.  The rest is held to bounds made of the steps that round:

* a rotated element: two products and a sum in fp32, 3 * 2^-24 of |x1 c| + |x2 s|; stored bf16 2^-8,
  a code 2^-4 or half the subnormal spacing, 2^-10 times its scale;
* a score: products are exact in the tensor core, each step of 16 adds into an fp32 accumulator
  without rounding to nearest, at most 2^-22 of the sum of magnitudes a step, and three more
  roundings; in log2 units it passes one subtraction and the exponential, 2^-22 relative and 2^-24 of
  its argument each; a probability moves by the score's error d relative (e^d - 1 <= 1.01 d here);
* a probability in fp16: 2^-11 relative, or half its least step, 2^-25 / 2^7, times the largest value's scale;
* the sum over keys: a step of 16 adds without rounding to nearest, 2^-22 of the sum of weights times |v|;
* the join of parts and the division: 2^-20 relative.
"""
import ctypes
import threading

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu

tp = pytest.importorskip("tensor_sharded_linear_tp_gb300")

DEV = "cuda"
E4M3, E8M0, BF16 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    tp.tp_device_status()


def f64(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def raw(t):
    torch.cuda.synchronize()
    return t.detach().view(torch.uint8).cpu().numpy().copy()


def to_bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(BF16).to(DEV)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    """A batch of sequences [(cached, new)] over a cache of random pages, on the GPU and as numpy arrays."""

    def __init__(self, seqs, p=1, n_kv=2, group=1, D=128, page=16, seed=0, spare=2, front=0, behind=0, split=False,
                 fill=None, spread=0.5):
        rng = self.rng = np.random.default_rng(seed)
        self.p, self.n_kv, self.group, self.D, self.page = p, n_kv, group, D, page
        self.heads = n_kv * group
        self.seqs, row = [], front                    # (first row, new rows, length)
        for old, new in seqs:
            self.seqs.append((row, new, old + new))
            row += new
        self.T = row + behind
        need = [-(-n // page) for _, _, n in self.seqs]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.max_pages = max(need + [1])
        self.table = np.zeros((len(seqs), self.max_pages), dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.codes, self.scales = [], []              # [rank][k or v]
        for _ in range(p):
            x = rng.normal(size=(2, self.n_pages, n_kv, page, D)) * 2.0 ** rng.normal(0, spread, (2, self.n_pages, n_kv, 1, 1))
            b = P.scale_byte(np.abs(x).max(axis=(3, 4)))
            self.codes.append(F.f64_to_e4m3(x / F.scale_value(b)[..., None, None]))
            self.scales.append(b)
        if fill is not None:                          # slots that hold no token
            for s, (_, _, n) in enumerate(self.seqs):
                if n % page:
                    for c in self.codes:
                        c[:, self.table[s, n // page], :, n % page:] = fill
        self.upload(split)

    def upload(self, split=False):
        def code(c):
            return torch.from_numpy(c).to(DEV).view(E4M3)

        def byte(b):
            return torch.from_numpy(b).to(DEV).view(E8M0)
        if split:   # K and V side by side in one allocation: strides from page to page
            both = [code(np.ascontiguousarray(c.transpose(1, 0, 2, 3, 4))) for c in self.codes]
            sc = [byte(np.ascontiguousarray(b.transpose(1, 0, 2))) for b in self.scales]
            k, v = [c[:, 0] for c in both], [c[:, 1] for c in both]
            ks, vs = [b[:, 0] for b in sc], [b[:, 1] for b in sc]
        else:
            k, v = [code(c[0]) for c in self.codes], [code(c[1]) for c in self.codes]
            ks, vs = [byte(b[0]) for b in self.scales], [byte(b[1]) for b in self.scales]
        self.cache = tp.PagedCache(k, v, ks, vs)
        self.batch = self.make_batch()

    def make_batch(self, max_new=None):
        starts = [a for a, _, _ in self.seqs] + [self.seqs[-1][0] + self.seqs[-1][1]]
        return tp.PagedBatch(i32(starts), i32([n for _, _, n in self.seqs]), i32(self.table.tolist()),
                             max_new if max_new is not None else max(n for _, n, _ in self.seqs))

    def got(self):
        """The cache's codes and scales as they are on the GPU, [rank][k or v]."""
        c = self.cache
        return ([np.stack([raw(c.k[r]), raw(c.v[r])]) for r in range(self.p)],
                [np.stack([raw(c.k_scales[r]), raw(c.v_scales[r])]) for r in range(self.p)])

    def queries(self, std=1.0):
        self.q = [to_bf16(self.rng.normal(0, std, (self.T, self.heads * self.D))) for _ in range(self.p)]
        return self.q

    def check(self, outs, scale=None, causal=True, window=0, before=None, what=""):
        """Every row against the oracle; rows of no sequence as they were."""
        scale = self.D ** -0.5 if scale is None else scale
        for r in range(self.p):
            got = f64(outs[r]).reshape(self.T, self.heads, self.D)
            q = f64(self.q[r]).reshape(self.T, self.heads, self.D)
            owned = np.zeros(self.T, dtype=bool)
            for s, (a, n, length) in enumerate(self.seqs):
                owned[a:a + n] = True
                if n == 0:
                    continue
                K, V = (P.values(self.codes[r][i], self.scales[r][i], self.table[s], length) for i in (0, 1))
                see = P.seen(n, length, causal, window)
                want, w = P.attention(q[a:a + n], K, V, scale, see)
                bound = attention_bound(q[a:a + n], K, V, scale, want, w, see)
                bad = ~(np.abs(got[a:a + n] - want) <= bound)
                assert not bad.any(), (what, r, s, np.argwhere(bad)[:5], got[a:a + n][bad][:5], want[bad][:5], bound[bad][:5])
            if before is not None:
                np.testing.assert_array_equal(got[~owned], f64(before[r]).reshape(got.shape)[~owned])


def attention_bound(q, K, V, scale, want, w, see):
    n, heads, D = q.shape
    group = heads // K.shape[0]
    bound = np.zeros_like(want)
    keys = K.shape[1]
    if keys == 0:
        return bound
    top_v = 2.0 * np.abs(V).max(axis=(1, 2))
    for h in range(heads):
        g = h // group
        mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(K[g]).T)                       # [n, keys]
        d = mag * ((D // 16) * 2.0 ** -22 + 3 * 2.0 ** -24)
        x = np.where(see, (q[:, h] @ K[g].T) * scale, 0.0)
        span = np.abs(x).max(axis=1, keepdims=True) * 2
        d = d + 2.0 ** -22 + span * 2.0 ** -23
        wd = 1.01 * w[h] * d
        total = np.abs(V[g])
        err = wd @ total + (w[h] @ total) * (2.0 ** -11 + (keys // 16 + 1) * 2.0 ** -22 + 2.0 ** -20)
        err += wd.sum(axis=1, keepdims=True) * np.abs(want[:, h])
        err += keys * 2.0 ** -32 * top_v[g] * w[h].max(axis=1, keepdims=True)
        bound[:, h] = 2.0 ** -8 * (np.abs(want[:, h]) + err) + err
    return bound


def fresh(q):
    return [torch.full_like(t, 7.0) for t in q]


# ----------------------------------------------------------------------------- append

QUARTERS = np.array([[1, 0], [0, 1], [-1, 0], [0, -1]], dtype=np.float32)   # (cos, sin)


def quarter_table(rng, rows, rot):
    turn = QUARTERS[rng.integers(0, 4, (rows, rot // 2))]
    return np.concatenate([turn[..., 0], turn[..., 1]], 1).astype(np.float32)


def qkv_of(c, std=1.0):
    width = (c.heads + 2 * c.n_kv) * c.D
    out = []
    for _ in range(c.p):
        x = c.rng.normal(0, std, (c.T, width)) * 2.0 ** c.rng.integers(-4, 5, (c.T, 1))
        out.append(to_bf16(x))
    return out


def split(c, x):
    x = x.reshape(c.T, c.heads + 2 * c.n_kv, c.D)
    return x[:, :c.heads], x[:, c.heads:c.heads + c.n_kv], x[:, c.heads + c.n_kv:]


BATCHES = [
    [(0, 1)], [(15, 1)], [(16, 1)], [(0, 0), (3, 2), (7, 0)], [(0, 129)], [(5, 300)],
    [(0, 1), (31, 1), (63, 1), (127, 1), (128, 1), (1000, 1), (0, 1)], [(100, 17), (0, 40), (129, 1), (64, 64)],
]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D, rot, style", [(128, 128, "half"), (128, 48, "pairs"), (64, 64, "pairs"), (64, 16, "half"),
                                           (128, 0, None)])
@pytest.mark.parametrize("seqs", BATCHES, ids=str)
def test_append_bit_exact(seqs, D, rot, style, page):
    c = Case(seqs, p=2, n_kv=3, group=2, D=D, page=page, seed=len(seqs) + page, front=2, behind=3, split=page == 32)
    qkv = qkv_of(c)
    rows = max(n for _, _, n in c.seqs) + 1
    cs = quarter_table(c.rng, rows, rot) if rot else None
    q_out = [torch.full((c.T, c.heads * D), 7.0, dtype=BF16, device=DEV) for _ in range(c.p)]
    tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch, rope=style, cos_sin=None if cs is None else torch.from_numpy(cs).to(DEV),
                        q_out=q_out)
    got_codes, got_scales = c.got()
    pos = np.concatenate([np.arange(n - new, n) for _, new, n in c.seqs]).astype(int)
    owned = np.concatenate([np.arange(a, a + n) for a, n, _ in c.seqs]).astype(int)
    for r in range(c.p):
        q, k, v = split(c, f64(qkv[r]))
        if rot:
            table = np.zeros((c.T, rot))
            table[owned] = cs[pos]
            q, k = P.rotate(q, table, style), P.rotate(k, table, style)
        P.append(c.codes[r][0], c.scales[r][0], k, c.seqs, c.table)
        P.append(c.codes[r][1], c.scales[r][1], v, c.seqs, c.table)
        np.testing.assert_array_equal(got_scales[r], c.scales[r])
        # (a zero's sign is lost where -0 + 0 met)
        np.testing.assert_array_equal(F.e4m3_to_f64(got_codes[r]), F.e4m3_to_f64(c.codes[r]))
        want = np.full((c.T, c.heads * D), 7.0)
        want[owned] = q.reshape(c.T, -1)[owned]
        np.testing.assert_array_equal(f64(q_out[r]), want)


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("D, rot", [(128, 128), (64, 32)])
def test_append_rotates_in_fp32(D, rot, style):
    c = Case([(0, 50), (700, 33), (11, 1)], p=2, n_kv=2, group=3, D=D, page=16, seed=3, spread=3)
    angle = np.outer(np.arange(800), 10000.0 ** (-np.arange(rot // 2) * 2 / rot))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    qkv = qkv_of(c)
    q_out = tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch, rope=style, cos_sin=torch.from_numpy(cs).to(DEV))
    got_codes, got_scales = c.got()
    pos = np.concatenate([np.arange(n - new, n) for _, new, n in c.seqs])
    for r in range(c.p):
        q, k, _ = split(c, f64(qkv[r]))
        t = cs[pos].astype(np.float64)
        err = 3 * 2.0 ** -24 * 2 * np.abs(q).max(axis=2, keepdims=True)
        want = P.rotate(q, t, style)
        got = f64(q_out[r]).reshape(want.shape)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + err) + err)
        want = P.rotate(k, t, style)
        err = 3 * 2.0 ** -24 * 2 * np.abs(k).max(axis=2, keepdims=True)
        for s, (a, n, length) in enumerate(c.seqs):
            v = P.values(got_codes[r][0], got_scales[r][0], c.table[s], length)[:, length - n:].transpose(1, 0, 2)
            pages = c.table[s][np.arange(length - n, length) // c.page]
            size = F.scale_value(got_scales[r][0][pages])[:, :, None]
            w, e = want[a:a + n], err[a:a + n]
            assert np.all(np.abs(v - w) <= np.maximum(2.0 ** -4 * (np.abs(w) + e), 2.0 ** -10 * size) + e)


def test_append_positions_of_their_own():
    c = Case([(0, 9), (30, 4)], p=1, n_kv=2, group=1, D=64, page=16, seed=5)
    cs = quarter_table(c.rng, 50, 64)
    positions = c.rng.integers(0, 50, c.T)
    qkv = qkv_of(c)
    q, = tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch, rope="half", cos_sin=torch.from_numpy(cs).to(DEV),
                             positions=i32(positions.tolist()))
    want, k, v = split(c, f64(qkv[0]))
    np.testing.assert_array_equal(f64(q), P.rotate(want, cs[positions], "half").reshape(c.T, -1))
    P.append(c.codes[0][0], c.scales[0][0], P.rotate(k, cs[positions], "half"), c.seqs, c.table)
    np.testing.assert_array_equal(c.got()[1][0][0], c.scales[0][0])


def test_append_strides_and_in_place():
    c = Case([(3, 20), (0, 5)], p=2, n_kv=2, group=2, D=128, page=16, seed=6, split=True)
    wide = (c.heads + 2 * c.n_kv) * c.D
    whole = [to_bf16(c.rng.normal(size=(c.T, wide + 64))) for _ in range(2)]
    qkv = [t[:, 16:16 + wide] for t in whole]
    cs = torch.from_numpy(quarter_table(c.rng, 40, 128)).to(DEV)
    wider = torch.zeros((40, 160), device=DEV)
    wider[:, :128] = cs
    apart = tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch, rope="half", cos_sin=wider[:, :128])
    first = c.got()
    before = [t.clone() for t in whole]
    there = tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch, rope="half", cos_sin=cs,
                                q_out=[t[:, :c.heads * c.D] for t in qkv])
    for r in range(2):
        assert torch.equal(apart[r], there[r])
        np.testing.assert_array_equal(c.got()[0][r], first[0][r])           # again: the same cache
        np.testing.assert_array_equal(c.got()[1][r], first[1][r])
        keep = torch.ones(whole[r].shape[1], dtype=torch.bool, device=DEV)
        keep[16:16 + c.heads * c.D] = False
        assert torch.equal(whole[r][:, keep], before[r][:, keep])


@pytest.mark.parametrize("page", [16, 128])
def test_append_special_values(page):
    """Zeros never raise a page's scale; a NaN or an infinity makes its page and head NaN; tiny and huge values."""
    c = Case([(4, 3), (4, 3), (4, 3), (4, 3), (0, 3)], p=1, n_kv=2, group=1, D=64, page=page, seed=7)
    x = f64(qkv_of(c)[0]).reshape(c.T, 6, 64)
    x[0:3, 2:] = 0
    x[3, 2, 5], x[4, 5, 1] = np.nan, np.inf
    x[6:9, 2:] *= 2.0 ** 110
    x[9:12, 2:] *= 2.0 ** -120
    x[12:15, 2:] = 0
    qkv = [to_bf16(x.reshape(c.T, -1))]
    q, = tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch)
    np.testing.assert_array_equal(f64(q), f64(qkv[0])[:, :c.heads * 64])
    _, k, v = split(c, f64(qkv[0]))
    P.append(c.codes[0][0], c.scales[0][0], k, c.seqs, c.table)
    P.append(c.codes[0][1], c.scales[0][1], v, c.seqs, c.table)
    codes, scales = c.got()
    np.testing.assert_array_equal(scales[0], c.scales[0])
    for s, (_, _, length) in enumerate(c.seqs):      # (a NaN's payload means nothing; slots behind stay)
        np.testing.assert_array_equal(F.e4m3_to_f64(codes[0][:, c.table[s, 0], :, :length]),
                                      F.e4m3_to_f64(c.codes[0][:, c.table[s, 0], :, :length]))
        np.testing.assert_array_equal(codes[0][:, c.table[s, 0], :, length:], c.codes[0][:, c.table[s, 0], :, length:])


def test_append_token_by_token_equals_the_oracle_and_decays_gently():
    c = Case([(0, 1)], p=1, n_kv=2, group=1, D=128, page=32, seed=8, spare=4)
    c.table = np.arange(4, dtype=np.int32)[None, :]
    x = to_bf16(c.rng.normal(size=(100, 6 * 128)) * 2.0 ** c.rng.integers(-3, 4, (100, 1)))
    starts, length = i32([0, 1]), i32([0])
    batch = tp.PagedBatch(starts, length, i32(c.table.tolist()), 1)
    for t in range(100):
        length.fill_(t + 1)
        tp.tp_kv_append_fp8([x[t:t + 1]], 2, c.cache, batch)
        _, k, v = np.split(f64(x[t:t + 1]).reshape(1, 6, 128), [2, 4], axis=1)
        P.append(c.codes[0][0], c.scales[0][0], k, [(0, 1, t + 1)], c.table)
        P.append(c.codes[0][1], c.scales[0][1], v, [(0, 1, t + 1)], c.table)
    codes, scales = c.got()
    np.testing.assert_array_equal(scales[0], c.scales[0])
    np.testing.assert_array_equal(codes[0], c.codes[0])


def test_bad_places_are_left_out_and_reported():
    """A page outside the cache, a length beyond the table, rows beyond max_new and T, more rows than tokens."""
    c = Case([(10, 3), (10, 3), (10, 3), (0, 4)], p=1, n_kv=1, group=2, D=64, page=16, seed=9, spare=1)
    qkv = qkv_of(c)
    c.queries()
    table = c.table.copy()
    table[1, 0] = c.n_pages
    table[2, 0] = -1
    for lens, starts, max_new in (([13, 13, 13, 2], [0, 3, 6, 9, 13], 4), ([13, 13, 13, 40], [0, 3, 6, 9, 13], 4),
                                  ([13, 13, 13, 4], [0, 3, 6, 9, 14], 5), ([13, 13, 13, 4], [0, 3, 6, 9, 13], 3),
                                  ([13, 13, 13, -5], [0, 3, 6, 9, 13], 4), ([13, 13, 13, 4], [0, 3, 2, 9, 13], 4),
                                  ([13, 13, 13, 2 ** 31 - 1], [0, 3, 6, 9, 13], 4)):
        c.upload()
        before = c.got()
        batch = tp.PagedBatch(i32(starts), i32(lens), i32(table.tolist()), max_new)
        tp.tp_kv_append_fp8(qkv, 2, c.cache, batch, rope="half", cos_sin=torch.ones((100, 64), device=DEV))
        with pytest.raises(tp.TPError, match="TP_ERR_INVALID_ARG"):
            tp.tp_device_status()
        outs = fresh(c.q)
        tp.tp_attention_paged_fp8(c.q, c.cache, batch, outs=outs)
        with pytest.raises(tp.TPError, match="TP_ERR_INVALID_ARG"):
            tp.tp_device_status()
        tp.tp_device_status()                                                # the record is cleared
        got = c.got()
        for page in range(c.n_pages):
            if page not in table[[0, 3], 0]:
                np.testing.assert_array_equal(got[0][0][:, page], before[0][0][:, page])
        if starts[1:3] == [3, 6]:
            assert np.all(f64(outs[0])[3:9] == 0)                            # no key of these can be read


def test_rotation_outside_its_table_is_nan_and_reported():
    c = Case([(10, 3)], p=1, n_kv=1, group=1, D=64, page=16, seed=10)
    qkv = qkv_of(c)
    q, = tp.tp_kv_append_fp8(qkv, 1, c.cache, c.batch, rope="pairs", cos_sin=torch.ones((12, 32), device=DEV))
    with pytest.raises(tp.TPError, match="TP_ERR_INVALID_ARG"):
        tp.tp_device_status()
    got = f64(q)
    assert np.all(np.isfinite(got[:2])) and np.all(np.isnan(got[2, :32])) and np.all(np.isfinite(got[2, 32:]))
    assert c.got()[1][0][0, c.table[0, 0], 0] == 255


# ----------------------------------------------------------------------------- attention

@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D, group", [(128, 1), (128, 6), (64, 1), (64, 8), (128, 16), (64, 12)])
@pytest.mark.parametrize("seqs", [
    [(0, 1)], [(31, 1)], [(32, 1), (0, 1), (15, 1), (16, 1), (127, 1), (128, 1), (500, 1)], [(1000, 1), (0, 0), (7, 1)],
], ids=str)
def test_one_token(seqs, D, group, page):
    c = Case(seqs, p=2, n_kv=2, group=group, D=D, page=page, seed=group + page, front=1, behind=2, split=page == 64, fill=0x7F)
    q = c.queries()
    outs = fresh(q)
    tp.tp_attention_paged_fp8(q, c.cache, c.batch, outs=outs)
    c.check(outs, before=fresh(q))


@pytest.mark.parametrize("causal, window", [(True, 0), (False, 0), (True, 1), (True, 37), (True, 300)])
@pytest.mark.parametrize("D, group, page", [(128, 1, 16), (128, 3, 32), (64, 5, 64), (64, 2, 128), (128, 8, 128)])
@pytest.mark.parametrize("seqs", [
    [(0, 5)], [(100, 2), (3, 5), (0, 1), (40, 4)], [(0, 131)], [(77, 40), (0, 300), (5, 1), (513, 9)], [(200, 70)],
], ids=str)
def test_several_tokens(seqs, D, group, page, causal, window):
    c = Case(seqs, p=2, n_kv=2, group=group, D=D, page=page, seed=group + page, front=3, behind=1, fill=0xFF)
    q = c.queries()
    outs = fresh(q)
    tp.tp_attention_paged_fp8(q, c.cache, c.batch, causal=causal, window=window, outs=outs)
    c.check(outs, causal=causal, window=window, before=fresh(q))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group, new", [(8, 1), (3, 3), (8, 2), (17, 1), (6, 4), (5, 5), (8, 4), (11, 3)])
@pytest.mark.parametrize("olds", [[300], [700, 3, 2500, 0, 65, 4000]], ids=len)
def test_row_counts_on_either_side_of_a_variant(olds, group, new, D):
    """8, 9, 16, 17, 24, 25, 32 and 33 rows a KV head; items of one CTA and items cut between them."""
    c = Case([(old, new) for old in olds], p=2, n_kv=2, group=group, D=D, page=16, seed=group + new, behind=1)
    q = c.queries()
    outs = fresh(q)
    tp.tp_attention_paged_fp8(q, c.cache, c.batch, outs=outs)
    c.check(outs, before=fresh(q))


@pytest.mark.parametrize("D, group, n_kv", [(128, 1, 3), (128, 4, 1), (64, 16, 2), (128, 12, 1)])
@pytest.mark.parametrize("seqs", [[(9000, 1)], [(4000, 1), (2, 1), (6000, 1), (70, 1)], [(5000, 1)] + [(33, 1)] * 40,
                                  [(11, 1)] * 300, [(0, 0)] * 5 + [(3000, 1)] + [(0, 0)] * 300 + [(2, 1)]], ids=len)
def test_long_axes_and_many_sequences(seqs, D, group, n_kv):
    """Items over several warps and CTAs, several items in one, sequences without rows between them."""
    c = Case(seqs, p=2, n_kv=n_kv, group=group, D=D, page=32, seed=len(seqs))
    q = c.queries()
    outs = tp.tp_attention_paged_fp8(q, c.cache, c.batch)
    c.check(outs)


@pytest.mark.parametrize("new", [1, 3, 60, 200])
def test_rows_that_see_nothing(new):
    """More rows than tokens: the first rows come before the first key; a sequence of no tokens at all."""
    c = Case([(0, new), (20, new)], p=1, n_kv=2, group=2, D=128, page=16, seed=new)
    c.seqs = [(0, new, 0), (new, new, new // 2 + 1)]
    c.batch = c.make_batch()
    q = c.queries()
    outs = fresh(q)
    tp.tp_attention_paged_fp8(q, c.cache, c.batch, outs=outs)
    got = f64(outs[0])
    assert np.all(got[:new] == 0)
    c.check(outs)


@pytest.mark.parametrize("new", [1, 20, 200])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window", [1, 50, 333])
def test_pages_before_every_window_may_be_gone(new, page, window):
    c = Case([(1000, new), (70, new), (345, new)], p=1, n_kv=2, group=3, D=128, page=page, seed=window + new)
    q = c.queries()
    table = c.table.copy()
    for s, (_, n, length) in enumerate(c.seqs):
        table[s, :max(length - n - window + 1, 0) // page] = (-1, c.n_pages, 2 ** 31 - 1)[s]
    batch = tp.PagedBatch(c.batch.seq_start, c.batch.kv_len, i32(table.tolist()), new)
    outs = tp.tp_attention_paged_fp8(q, c.cache, batch, window=window)
    tp.tp_device_status()
    c.check(outs, window=window)


@pytest.mark.parametrize("new", [1, 4, 100])
@pytest.mark.parametrize("page", [16, 64])
def test_a_nan_page_stays_with_the_rows_that_see_it(new, page):
    seqs = [(3 * page, new), (2 * page, new)]
    c = Case(seqs, p=1, n_kv=2, group=2, D=128, page=page, seed=page + new)
    for which, head, at in ((0, 0, c.table[0, 1]), (1, 1, c.table[1, 0])):
        c.scales[0][which, at, head] = 255
        c.codes[0][which, at, head] = 0x7F
    # the last page of sequence 0: only its rows from there on see it (causal)
    last = (3 * page + new - 1) // page
    c.scales[0][1, c.table[0, last], 1] = 255
    c.codes[0][1, c.table[0, last], 1] = 0xFF
    c.upload()
    q = c.queries()
    out = f64(tp.tp_attention_paged_fp8(q, c.cache, c.batch)[0]).reshape(c.T, 4, 128)
    for s, (a, n, length) in enumerate(c.seqs):
        K, V = (P.values(c.codes[0][i], c.scales[0][i], c.table[s], length) for i in (0, 1))
        want, _ = P.attention(f64(q[0]).reshape(c.T, 4, 128)[a:a + n], K, V, 128 ** -0.5, P.seen(n, length))
        np.testing.assert_array_equal(np.isnan(out[a:a + n]), np.isnan(want))
        fine = np.isfinite(want)
        assert np.all(np.abs(out[a:a + n][fine] - want[fine]) <= 2.0 ** -6 * (np.abs(want[fine]) + 1))
    assert np.isfinite(out).any()


@pytest.mark.parametrize("new", [1, 2, 70])
def test_special_queries(new):
    """Zero, tiny and huge queries; a NaN or an infinity makes its row NaN and no other."""
    c = Case([(100, new), (40, new)], p=1, n_kv=2, group=6, D=128, page=32, seed=11)
    q = f64(c.queries()[0]).reshape(c.T, 12, 128)
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -100
    q[0, 2] *= 2.0 ** -130
    q[0, 3] *= 2.0 ** 3
    q[0, 4, 7], q[0, 5, 100], q[new, 6, 0] = np.nan, np.inf, -np.inf
    q[new, 7] = 0
    q[new, 7, 3] = 1.0
    q[new, 7, 4] = 2.0 ** -30
    c.q = [to_bf16(q.reshape(c.T, -1))]
    out = f64(tp.tp_attention_paged_fp8(c.q, c.cache, c.batch)[0]).reshape(c.T, 12, 128)
    bad = [(0, 4), (0, 5), (new, 6)]
    for t, h in bad:
        assert np.all(np.isnan(out[t, h]))
        out[t, h] = 0
    clean = f64(c.q[0]).reshape(c.T, 12, 128)
    for t, h in bad:
        clean[t, h] = 0
    c.q = [to_bf16(clean.reshape(c.T, -1))]
    again = f64(tp.tp_attention_paged_fp8(c.q, c.cache, c.batch)[0]).reshape(c.T, 12, 128)
    for t, h in bad:
        again[t, h] = 0
    np.testing.assert_array_equal(out, again)
    c.check(tp.tp_attention_paged_fp8(c.q, c.cache, c.batch))


@pytest.mark.parametrize("new", [1, 100])
def test_page_scales_far_apart(new):
    """V pages between 2^-20 and 2^20, K pages between 2^-8 and 2^2, some all zero with the least scale."""
    c = Case([(300, new), (90, new)], p=1, n_kv=2, group=4, D=128, page=16, seed=12)
    for which, lo, hi in ((0, -8, 3), (1, -20, 21)):
        c.scales[0][which] = 121 + c.rng.integers(lo, hi, c.scales[0][which].shape)
    zero = c.rng.random(c.scales[0].shape) < 0.2
    c.codes[0][zero] = 0
    c.scales[0][zero] = 0
    c.upload()
    q = c.queries()
    c.check(tp.tp_attention_paged_fp8(q, c.cache, c.batch))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales_of_the_scores(scale):
    c = Case([(200, 1), (40, 1)], p=1, n_kv=2, group=3, D=64, page=32, seed=13)
    q = c.queries()
    c.check(tp.tp_attention_paged_fp8(q, c.cache, c.batch, scale=scale), scale=scale)


def test_shared_pages_of_a_prefix():
    c = Case([(64, 3), (64, 3), (64, 3)], p=1, n_kv=2, group=2, D=128, page=16, seed=14)
    c.table[1, :4] = c.table[2, :4] = c.table[0, :4]
    c.batch = c.make_batch()
    qkv = qkv_of(c)
    c.q = tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch)
    c.codes, c.scales = c.got()
    c.check(tp.tp_attention_paged_fp8(c.q, c.cache, c.batch))


# ----------------------------------------------------------------------------- as they are used

def heads_of(w, heads, n_kv, D):
    return [heads * D, n_kv * D, n_kv * D]


@pytest.mark.parametrize("D, page, group", [(128, 16, 2), (64, 64, 4)])
def test_a_sharded_layer_serving_several_sequences(D, page, group):
    """Prompts, then tokens one by one: projection, append, attention and out-projection against the oracle, on the
    stored output of each step before; and the cached path's last token against the whole sequence's attention."""
    p, hidden, n_kv = 2, 256, 2
    heads = n_kv * group
    rng = np.random.default_rng(15)
    width = p * (heads + 2 * n_kv) * D
    w_qkv = to_bf16(rng.normal(0, 0.06, (width, hidden)))
    w_out = to_bf16(rng.normal(0, 0.05, (hidden, p * heads * D)))
    splits = [p * heads * D, p * n_kv * D, p * n_kv * D]
    shards = tp.tp_plan_shard_ranks(w_qkv, "colwise", p, fused_splits=splits, num_heads=p * n_kv, head_dim=D)
    outs = tp.tp_plan_shard_ranks(w_out, "rowwise", p)
    cache = tp.PagedCache.empty(p, 24, n_kv, page, D)
    table = rng.permutation(24).reshape(3, 8).astype(np.int32)
    angle = np.outer(np.arange(512), 10000.0 ** (-np.arange(D // 2) * 2 / D))
    cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).to(DEV)
    lengths = [0, 0, 0]
    for step, new in enumerate([(37, 5, 90), (1, 1, 1), (1, 1, 1), (6, 0, 3)]):
        starts = np.concatenate([[0], np.cumsum(new)])
        T = int(starts[-1])
        lengths = [n + m for n, m in zip(lengths, new)]
        batch = tp.PagedBatch(i32(starts.tolist()), i32(lengths), i32(table.tolist()), max(new))
        x = to_bf16(rng.normal(size=(T, hidden)))
        qkv = tp.tp_linear_colwise(x, shards)
        q = tp.tp_kv_append_fp8(qkv, heads, cache, batch, rope="half", cos_sin=cs)
        att = tp.tp_attention_paged_fp8(q, cache, batch)
        y = tp.tp_linear_rowwise(att, outs)
        assert torch.isfinite(y).all()
        total = sum(f64(a) @ f64(w).T for a, w in zip(att, outs))
        assert np.all(np.abs(f64(y) - total) <= 2.0 ** -8 * np.abs(total) + 1e-4 * np.abs(total).max())
        for r in range(p):
            codes = [raw(cache.k[r]), raw(cache.v[r])]
            scales = [raw(cache.k_scales[r]), raw(cache.v_scales[r])]
            qf = f64(q[r]).reshape(T, heads, D)
            for s, (a, n) in enumerate(zip(starts, new)):
                if n == 0:
                    continue
                K, V = (P.values(codes[i], scales[i], table[s], lengths[s]) for i in (0, 1))
                see = P.seen(n, lengths[s])
                want, w = P.attention(qf[a:a + n], K, V, D ** -0.5, see)
                bound = attention_bound(qf[a:a + n], K, V, D ** -0.5, want, w, see)
                got = f64(att[r]).reshape(T, heads, D)[a:a + n]
                assert np.all(np.abs(got - want) <= bound), (step, r, s)
                # what was appended: this step's K, rotated, to within a code's rounding
                kx = f64(qkv[r]).reshape(T, heads + 2 * n_kv, D)[a:a + n, heads:heads + n_kv]
                want_k = P.rotate(kx, f64(cs)[lengths[s] - n:lengths[s]], "half").transpose(1, 0, 2)
                pages = table[s][np.arange(lengths[s] - n, lengths[s]) // page]
                size = F.scale_value(scales[0][pages]).T[:, :, None]
                assert np.all(np.abs(K[:, lengths[s] - n:] - want_k) <= np.maximum(2.0 ** -4 * np.abs(want_k), 2.0 ** -10 * size) * 1.001)


@pytest.mark.parametrize("new", [1, 40])
def test_same_bits_every_time_and_on_another_stream(new):
    c = Case([(700, new), (3000, new), (5, new)], p=2, n_kv=2, group=4, D=128, page=16, seed=16)
    qkv = qkv_of(c)
    first = tp.tp_attention_paged_fp8(tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch), c.cache, c.batch)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    need = tp.tp_attention_paged_workspace_bytes(c.cache, c.batch, c.T, c.heads)
    for i in range(4):
        ws = torch.randint(0, 256, (max(need, 16),), dtype=torch.uint8, device=DEV)      # any content
        torch.cuda.synchronize()
        q = tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch, stream=stream)
        outs = tp.tp_attention_paged_fp8(q, c.cache, c.batch, workspace=ws, stream=stream)
        stream.synchronize()
        for a, b in zip(first, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("long", [False, True])
def test_captured_decode_follows_the_lengths(long):
    """One captured step, replayed while lengths, pages and tokens change on the device."""
    top = 4000 if long else 200
    c = Case([(top, 1)] * 3, p=2, n_kv=2, group=3, D=128, page=16, seed=17)
    lengths, table = i32([1, 1, 1]), i32(c.table.tolist())
    batch = tp.PagedBatch(i32([0, 1, 2, 3]), lengths, table, 1)
    x = [torch.zeros((3, (c.heads + 4) * 128), dtype=BF16, device=DEV) for _ in range(2)]
    need = tp.tp_attention_paged_workspace_bytes(c.cache, batch, 3, c.heads)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    tp.tp_attention_paged_fp8(tp.tp_kv_append_fp8(x, c.heads, c.cache, batch), c.cache, batch, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = tp.tp_kv_append_fp8(x, c.heads, c.cache, batch)
        outs = tp.tp_attention_paged_fp8(q, c.cache, batch, workspace=ws)
    for lens in ([1, 2, 3], [16, 17, 33], [top, 5, top // 2], [100, 199, 1], [2, 0, 1]):
        lengths.copy_(i32(lens))
        for t in x:
            t.copy_(to_bf16(c.rng.normal(size=t.shape)))
        graph.replay()
        torch.cuda.synchronize()
        c.q, (c.codes, c.scales) = q, c.got()
        c.seqs = [(s, 1, n) for s, n in enumerate(lens)]
        if 0 in lens:      # a row without a token: reported, its output 0
            assert np.all(f64(outs[0])[lens.index(0)] == 0)
            with pytest.raises(tp.TPError):
                tp.tp_device_status()
        else:
            c.check(outs, what=lens)


def test_calls_on_several_streams_and_from_several_threads():
    cases = [Case([(400 * i + 50, 1), (3000, 1 + 30 * (i % 2))], p=2, n_kv=2, group=2, D=128, page=32, seed=20 + i) for i in range(4)]
    results, errors = [None] * 4, []
    for c in cases:
        c.queries()
    torch.cuda.synchronize()

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                results[i] = tp.tp_attention_paged_fp8(cases[i].q, cases[i].cache, cases[i].batch, stream=stream)
            stream.synchronize()
        except Exception as e:   # pragma: no cover
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for c, outs in zip(cases, results):
        c.check(outs)


def test_one_cache_for_several_ranks():
    """The same tensors as several ranks' caches (read only): every rank has rank 0's answer."""
    c = Case([(1500, 1), (33, 1)], p=1, n_kv=2, group=2, D=128, page=16, seed=30)
    q = c.queries()
    k = c.cache
    many = tp.PagedCache(k.k * 3, k.v * 3, k.k_scales * 3, k.v_scales * 3)
    outs = tp.tp_attention_paged_fp8(q * 3, many, c.batch)
    c.check(outs[:1])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("new", [1, 70])
def test_offsets_past_four_gib(new):
    """Pages whose codes lie beyond 4 GiB, from a stride of 64 KiB a page."""
    n_pages, n_kv, page, D = 70000, 1, 16, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB of free device memory")
    store = torch.zeros((n_pages, 65536), dtype=torch.uint8, device=DEV)
    size = n_kv * page * D
    k = store[:, :size].view(E4M3).view(n_pages, n_kv, page, D)
    v = store[:, size:2 * size].view(E4M3).view(n_pages, n_kv, page, D)
    scales = torch.zeros((2, n_pages, n_kv), dtype=torch.uint8, device=DEV)
    cache = tp.PagedCache([k], [v], [scales[0]], [scales[1]])
    rng = np.random.default_rng(31)
    length = 100 + new
    table = (n_pages - 1 - rng.permutation(200)[:-(-length // page)])[None, :].astype(np.int32)
    qkv = to_bf16(rng.normal(size=(length, 4 * D)))
    tp.tp_kv_append_fp8([qkv], 2, cache, tp.PagedBatch(i32([0, length]), i32([length]), i32(table.tolist()), length))
    q = [qkv[length - new:, :2 * D].contiguous()]
    out, = tp.tp_attention_paged_fp8(q, cache, tp.PagedBatch(i32([0, new]), i32([length]), i32(table.tolist()), new))
    x = f64(qkv).reshape(length, 4, D)
    pages = -(-length // page)
    codes, sc = np.zeros((2, pages, 1, page, D), np.uint8), np.zeros((2, pages, 1), np.uint8)
    at = np.arange(pages)[None, :]
    for i in (0, 1):
        P.append(codes[i], sc[i], x[:, 2 + i:3 + i], [(0, length, length)], at)
        got = raw((k, v)[i][torch.from_numpy(table[0].astype(np.int64)).to(DEV)].contiguous())
        lengths = min(page, length)
        np.testing.assert_array_equal(got.reshape(-1, D)[:length], codes[i].reshape(-1, D)[:length])
    K, V = (P.values(codes[i], sc[i], at[0], length) for i in (0, 1))
    see = P.seen(new, length)
    want, w = P.attention(f64(q[0]).reshape(new, 2, D), K, V, D ** -0.5, see)
    assert np.all(np.abs(f64(out).reshape(want.shape) - want) <= attention_bound(f64(q[0]).reshape(new, 2, D), K, V, D ** -0.5, want, w, see))


def test_empty_calls_write_nothing():
    c = Case([(5, 2)], p=1, n_kv=1, group=1, D=64, page=16, seed=32)
    before = c.got()
    none = tp.PagedBatch(i32([0, 0]), i32([0]), i32([[0]]), 0)
    q, = tp.tp_kv_append_fp8([torch.zeros((0, 3 * 64), dtype=BF16, device=DEV)], 1, c.cache, c.batch)
    assert q.shape == (0, 64)
    tp.tp_kv_append_fp8([torch.zeros((2, 3 * 64), dtype=BF16, device=DEV)], 1, c.cache, none)
    out = torch.full((2, 64), 7.0, dtype=BF16, device=DEV)
    tp.tp_attention_paged_fp8([torch.zeros_like(out)], c.cache, none, outs=[out])
    assert torch.all(out == 7)
    after = c.got()
    np.testing.assert_array_equal(before[0][0], after[0][0])
    np.testing.assert_array_equal(before[1][0], after[1][0])


def test_binding_refusals():
    c = Case([(5, 2)], p=2, n_kv=2, group=1, D=64, page=16, seed=33)
    q = c.queries()
    k = c.cache
    with pytest.raises(TypeError):
        tp.PagedCache([t.view(torch.uint8) for t in k.k], k.v, k.k_scales, k.v_scales)
    with pytest.raises(ValueError):
        tp.PagedCache(k.k, k.v[:1], k.k_scales, k.v_scales)
    with pytest.raises(ValueError):
        tp.PagedCache(k.k, [t[:-1] for t in k.v], k.k_scales, k.v_scales)
    with pytest.raises(ValueError):
        tp.PagedCache([t.transpose(1, 2).contiguous().transpose(1, 2) for t in k.k], k.v, k.k_scales, k.v_scales)
    with pytest.raises(TypeError):
        tp.PagedBatch(c.batch.seq_start.long(), c.batch.kv_len, c.batch.page_table, 2)
    with pytest.raises(ValueError):
        tp.PagedBatch(c.batch.kv_len, c.batch.kv_len, c.batch.page_table, 2)
    with pytest.raises(ValueError):
        tp.tp_attention_paged_fp8(q[:1], k, c.batch)
    with pytest.raises(ValueError):
        tp.tp_attention_paged_fp8([t[:, :100] for t in q], k, c.batch)
    with pytest.raises(TypeError):
        tp.tp_attention_paged_fp8([t.float() for t in q], k, c.batch)
    with pytest.raises(ValueError):
        tp.tp_attention_paged_fp8([t.cpu() for t in q], k, c.batch)
    long = Case([(5000, 2)], p=1, n_kv=2, group=1, D=64, page=16, seed=34)
    with pytest.raises(tp.TPError, match="TP_ERR_WORKSPACE"):
        tp.tp_attention_paged_fp8(long.queries(), long.cache, long.batch, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    qkv = qkv_of(c)
    with pytest.raises(ValueError):
        tp.tp_kv_append_fp8(qkv, c.heads, k, c.batch, rope="half")
    with pytest.raises(ValueError):
        tp.tp_kv_append_fp8(qkv, c.heads, k, c.batch, cos_sin=torch.ones((9, 64), device=DEV))
    with pytest.raises(ValueError):
        tp.tp_kv_append_fp8(qkv, c.heads + 1, k, c.batch)
    with pytest.raises(tp.TPError, match="TP_ERR_INVALID_ARG"):
        tp.tp_kv_append_fp8(qkv, c.heads, k, c.batch, rope="half", cos_sin=torch.ones((9, 20), device=DEV))


def test_a_batchs_rows_by_either_name():
    c = Case([(40, 3), (7, 5)], p=1, n_kv=2, group=2, D=64, page=16, seed=35)
    q = c.queries()
    b = c.batch
    same = tp.PagedBatch(b.seq_start, b.kv_len, b.page_table, max_q=5)
    assert same.max_new == b.max_new == 5
    outs = tp.tp_attention_paged_fp8(q, c.cache, same)
    assert torch.equal(outs[0], tp.tp_attention_paged_fp8(q, c.cache, b)[0])
    c.check(outs)


STALE = {"nan codes": (127, 0x7F), "a larger scale": (167, None), "the largest scale": (254, None), "a nan page": (255, 0xFF)}


def stale_pages(c, content, window):
    """c's batch with every table entry before all of a sequence's windows naming a page that holds something else."""
    z = sorted(set(range(c.n_pages)) - {p for s, (_, _, n) in enumerate(c.seqs) for p in c.table[s, :-(-n // c.page)]})[0]
    byte, code = STALE[content]
    for r in range(c.p):
        c.scales[r][:, z] = byte
        if code is not None:
            c.codes[r][:, z] = code
    c.upload()
    table = c.table.copy()
    for s, (_, n, length) in enumerate(c.seqs):
        table[s, :max(length - n - window + 1, 0) // c.page] = z
    return tp.PagedBatch(c.batch.seq_start, c.batch.kv_len, i32(table.tolist()), c.batch.max_new)


WINDOW_STARTS = [(600 + 16 * i + 3) for i in range(8)]     # in each 16 keys of a step of 128


@pytest.mark.parametrize("content", STALE)
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("D, new", [(128, 1), (64, 1), (128, 4), (64, 10)])
def test_few_rows_pages_before_every_window_may_hold_anything(D, new, page, content):
    c = Case([(old, new) for old in WINDOW_STARTS], p=1, n_kv=2, group=3, D=D, page=page, seed=page + new)
    batch = stale_pages(c, content, 200)
    outs = tp.tp_attention_paged_fp8(c.queries(), c.cache, batch, window=200)
    tp.tp_device_status()
    c.check(outs, window=200)


@pytest.mark.parametrize("content", STALE)
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("D, new", [(128, 20), (64, 20), (128, 100), (64, 200)])
def test_many_rows_pages_before_every_window_may_hold_anything(D, new, page, content):
    """Items of up to 128 and of 256 rows; several items of a sequence, whose windows begin in different pages."""
    c = Case([(old, new) for old in WINDOW_STARTS], p=1, n_kv=2, group=3, D=D, page=page, seed=page + new)
    batch = stale_pages(c, content, 200)
    outs = tp.tp_attention_paged_fp8(c.queries(), c.cache, batch, window=200)
    tp.tp_device_status()
    c.check(outs, window=200)


@pytest.mark.parametrize("gap", [20, 24, 30, 32, 34, 38, 45, 80])
@pytest.mark.parametrize("D, group, new", [(128, 2, 40), (64, 8, 40), (128, 1, 24), (64, 1, 30)])
def test_rows_that_see_only_a_page_of_small_scale(D, group, new, gap):
    """The first page's scales 2^-gap of the next one's, which its own rows do not see.  Many rows: an element of K or V
    is off by at most 2^-32 of the largest scale of a step, half the least step of fp16 in units of 2^-7 of it, and from a
    gap of 32 on the page enters as 0.  Few rows: a probability is off by 2^-25 in units of 2^(E_v - 14), times a code
    of up to 448, so a key by 2^-30 of V's largest."""
    c = Case([(0, new)], p=1, n_kv=2, group=group, D=D, page=16, seed=gap)
    few = new * group <= 32
    big = {0: 147, 1: 137}                       # the other pages' bytes: K 2^20, V 2^10
    for which in (0, 1):
        c.scales[0][which] = big[which]
        c.scales[0][which, c.table[0, 0]] = big[which] - gap
    c.upload()
    q = np.zeros((c.T, c.heads, D))              # (one element each, so that scores of that page are about 1)
    q[np.arange(c.T)[:, None], np.arange(c.heads)[None, :], c.rng.integers(0, D, (c.T, c.heads))] = 2.0 ** min(gap - 25, 9)
    c.q = [to_bf16(q.reshape(c.T, -1))]
    out = f64(tp.tp_attention_paged_fp8(c.q, c.cache, c.batch)[0]).reshape(c.T, c.heads, D)[:16]
    q = f64(c.q[0]).reshape(c.T, c.heads, D)[:16]
    K, V = (P.values(c.codes[0][i], c.scales[0][i], c.table[0], 16) for i in (0, 1))
    see = P.seen(16, 16)
    want, w = P.attention(q, K, V, D ** -0.5, see)
    bound = attention_bound(q, K, V, D ** -0.5, want, w, see)
    off = [2.0 ** (big[i] - 127 - 32) if gap < 32 else np.abs(x).max() for i, x in ((0, K), (1, V))]
    d = 1.01 * D ** -0.5 * np.abs(q).sum(axis=2) * off[0]                                # of a score [16, heads]
    for h in range(c.heads):
        g = h // group
        if few:
            err = np.arange(1, 17)[:, None] * 2.0 ** (big[1] - 127 - 30)
        else:
            err = np.expm1(2 * d[:, h])[:, None] * (w[h] @ np.abs(V[g])) + off[1]
        bound[:, h] += (1 + 2.0 ** -8) * err
    bad = ~(np.abs(out - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], want[bad][:5], bound[bad][:5])


@pytest.mark.parametrize("rows, D, keys", [(1, 128, 2 ** 21 + 77), (12, 64, 2 ** 21 + 77), (20, 128, 2 ** 21 + 77), (32, 128, 2 ** 21 + 77),
                                           (100, 64, 2 ** 21 + 77), (300, 128, 2 ** 21 + 77), (1, 64, 2 ** 23), (256, 64, 2 ** 23)])
def test_millions_of_keys(rows, D, keys):
    """Sums over more keys than a piece has: a warp (up to 32 rows) or a CTA has whole sequences, of a few pages again
    and again, so that the oracle needs only their tokens and how often they occur.  Later pages have larger scales.

    A piece of 2^19 keys adds 2^15 times to its accumulators, each time without rounding to nearest (2^-22 of the sum); V
    is positive, so that this is 2^-7 of the output."""
    few = rows <= 32
    p, n_kv = (16, 114) if few else (4, 38)
    page, pool, pages = 128, 16, -(-keys // 128)
    rng = np.random.default_rng(rows)
    kc = F.f64_to_e4m3(rng.normal(0, 64, (pool, n_kv, page, D)))
    vc = F.f64_to_e4m3(rng.uniform(1, 448, (pool, n_kv, page, D)))
    step = np.repeat(np.arange(pool)[:, None], n_kv, 1)
    ks, vs = (118 + step // 5).astype(np.uint8), (118 + (step * 3 + np.arange(n_kv)) % 9).astype(np.uint8)
    dev = [torch.from_numpy(a).to(DEV) for a in (kc, vc, ks, vs)]
    cache = tp.PagedCache([dev[0].view(E4M3)] * p, [dev[1].view(E4M3)] * p, [dev[2]] * p, [dev[3]] * p)
    table = np.concatenate([rng.integers(0, pool // 2, pages // 2), rng.integers(0, pool, pages - pages // 2)]).astype(np.int32)
    batch = tp.PagedBatch(i32([0, 1]), i32([keys]), torch.from_numpy(table[None]).to(DEV), 1)
    q = to_bf16(rng.normal(size=(1, n_kv * rows * D)))
    outs = tp.tp_attention_paged_fp8([q] * p, cache, batch, causal=False)
    tp.tp_device_status()
    assert all(torch.equal(outs[0], o) for o in outs)

    count = np.bincount(table, minlength=pool)[:, None] * np.ones(page)
    count[table[-1], keys - (pages - 1) * page:] -= 1
    count = torch.from_numpy(count.reshape(1, -1)).to(DEV)
    qf = q.double().view(n_kv, rows, D)
    K, V = (torch.from_numpy(F.e4m3_to_f64(c) * F.scale_value(s)[:, :, None, None]).to(DEV).transpose(0, 1).reshape(n_kv, -1, D)
            for c, s in ((kc, ks), (vc, vs)))
    x = qf @ K.transpose(1, 2) * D ** -0.5                                             # [n_kv, rows, pool * page]
    d = (qf.abs() @ K.abs().transpose(1, 2) * D ** -0.5) * ((D // 16) * 2.0 ** -22 + 3 * 2.0 ** -24)
    d = d + 2.0 ** -22 + x.abs().amax(2, keepdim=True) * 2.0 ** -22
    w = torch.exp(x - x.amax(2, keepdim=True)) * count
    w = w / w.sum(2, keepdim=True)
    want = w @ V
    err = (1.01 * w * d) @ V + want * (2.0 ** -11 + 2.0 ** -7 + 2.0 ** -18) + (1.01 * w * d).sum(2, keepdim=True) * want
    got = outs[0].double().view(n_kv, rows, D)
    bad = ~((got - want).abs() <= 2.0 ** -8 * (want + err) + err)
    assert not bad.any(), (int(bad.sum()), ((got - want) / want)[bad][:5], (got / want - 1).mean())


def test_a_part_of_more_than_two_seconds():
    """A CTA's part of some two and a half seconds in one item, and short items behind it: no wait gives up."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows, pages, page, D = 256 * sms, 1_250_000, 128, 128
    k = torch.zeros((1, 1, page, D), dtype=torch.uint8, device=DEV).view(E4M3)
    v = torch.full((1, 1, page, D), 0x38, dtype=torch.uint8, device=DEV).view(E4M3)
    one = torch.full((1, 1), 127, dtype=torch.uint8, device=DEV)
    cache = tp.PagedCache([k], [v], [one], [one])
    batch = tp.PagedBatch(i32([0] + [rows + i for i in range(9)]), i32([pages * page] + [1] * 8),
                          torch.zeros((9, pages), dtype=torch.int32, device=DEV), rows)
    q = [torch.ones((rows + 8, D), dtype=BF16, device=DEV)]
    out, = tp.tp_attention_paged_fp8(q, cache, batch, causal=False)
    tp.tp_device_status()
    assert torch.all(out == 1)                   # (every key is worth 1)


@pytest.mark.parametrize("seqs, p, n_kv, group, D, page", [
    ([(0, 4608)], 2, 12, 1, 128, 16), ([(20011, 300)], 2, 2, 6, 128, 64), ([(0, 3000)], 2, 12, 1, 64, 32),
    ([(300 * i, 8) for i in range(1, 17)], 2, 2, 6, 128, 16), ([(200 * i, 1) for i in range(1, 33)], 2, 2, 6, 128, 16),
    ([(200 * i, 5) for i in range(1, 17)], 2, 2, 6, 128, 16)], ids=["prompt", "chunk", "prompt64", "rows48", "rows6", "rows30"])
def test_calls_one_after_another(seqs, p, n_kv, group, D, page):
    """Calls that follow each other without a wait, each with outputs of its own: the bits of a call by itself."""
    c = Case(seqs, p=p, n_kv=n_kv, group=group, D=D, page=page, seed=41)
    q = c.queries()
    alone = tp.tp_attention_paged_fp8(q, c.cache, c.batch)
    torch.cuda.synchronize()
    need = tp.tp_attention_paged_workspace_bytes(c.cache, c.batch, c.T, c.heads)
    spaces = [torch.empty(max(need, 16), dtype=torch.uint8, device=DEV) for _ in range(6)]
    for _ in range(10):
        outs = [fresh(q) for _ in spaces]
        torch.cuda.synchronize()
        for o, ws in zip(outs, spaces):
            tp.tp_attention_paged_fp8(q, c.cache, c.batch, outs=o, workspace=ws)
        torch.cuda.synchronize()
        for k, o in enumerate(outs):
            for r in range(p):
                assert torch.equal(o[r], alone[r]), (k, r, int((o[r] != alone[r]).sum()))


@pytest.mark.parametrize("seqs", [[(15, 1), (40, 1), (0, 1)], [(3, 20), (0, 5)]], ids=len)
def test_append_leaves_queries_alone(seqs):
    """q_out NULL: K and V are cached, Q is neither read for it nor written."""
    c = Case(seqs, p=2, n_kv=2, group=3, D=64, page=16, seed=36)
    qkv = qkv_of(c)
    before = [t.clone() for t in qkv]
    cs = torch.from_numpy(quarter_table(c.rng, 60, 32)).to(DEV)
    at = (ctypes.c_void_p * 2)(*[t.data_ptr() for t in qkv])
    rope = tp._rope(0, 32, cs.data_ptr(), 0, 60, 0)
    tp._check(tp.lib.tp_kv_append_fp8(c.cache._struct, c.batch._struct, at, 0, c.T, c.heads, rope, None, 0,
                                      torch.cuda.current_stream().cuda_stream))
    codes, scales = c.got()
    assert all(torch.equal(a, b) for a, b in zip(qkv, before))
    c.upload()
    tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch, rope="half", cos_sin=cs)
    want_codes, want_scales = c.got()
    for r in range(2):
        np.testing.assert_array_equal(codes[r], want_codes[r])
        np.testing.assert_array_equal(scales[r], want_scales[r])


@pytest.mark.parametrize("style", ["half", "pairs"])
def test_append_one_token_at_positions_of_its_own(style):
    c = Case([(15, 1), (30, 1), (0, 1), (17, 1)], p=2, n_kv=3, group=2, D=64, page=16, seed=37, front=1, behind=1)
    cs = quarter_table(c.rng, 50, 48)
    positions = c.rng.integers(0, 50, c.T)
    positions[0] = positions[-1] = -1            # (rows of no sequence)
    qkv = qkv_of(c)
    q_out = [torch.full((c.T, c.heads * c.D), 7.0, dtype=BF16, device=DEV) for _ in range(2)]
    tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch, rope=style, cos_sin=torch.from_numpy(cs).to(DEV),
                        positions=i32(positions.tolist()), q_out=q_out)
    codes, scales = c.got()
    for r in range(2):
        q, k, v = split(c, f64(qkv[r]))
        q, k = P.rotate(q, cs[positions], style), P.rotate(k, cs[positions], style)
        want = q.reshape(c.T, -1)
        want[[0, -1]] = 7.0
        np.testing.assert_array_equal(f64(q_out[r]), want)
        P.append(c.codes[r][0], c.scales[r][0], k, c.seqs, c.table)
        P.append(c.codes[r][1], c.scales[r][1], v, c.seqs, c.table)
        np.testing.assert_array_equal(scales[r], c.scales[r])
        np.testing.assert_array_equal(F.e4m3_to_f64(codes[r]), F.e4m3_to_f64(c.codes[r]))


def test_captured_chunks_follow_the_lengths():
    """One captured step of up to 40 tokens a sequence (many rows a KV head), replayed with other counts, lengths and pages."""
    c = Case([(300, 40), (500, 40), (90, 40)], p=2, n_kv=2, group=2, D=64, page=32, seed=38, behind=7)
    starts, lengths, table = i32([0, 0, 0, 0]), i32([0, 0, 0]), i32(c.table.tolist())
    batch = tp.PagedBatch(starts, lengths, table, 40)
    x = [torch.zeros((c.T, (c.heads + 4) * c.D), dtype=BF16, device=DEV) for _ in range(2)]
    q = [torch.empty((c.T, c.heads * c.D), dtype=BF16, device=DEV) for _ in range(2)]
    outs = [torch.empty_like(t) for t in q]
    ws = torch.empty(tp.tp_attention_paged_workspace_bytes(c.cache, batch, c.T, c.heads), dtype=torch.uint8, device=DEV)

    def call():
        tp.tp_kv_append_fp8(x, c.heads, c.cache, batch, q_out=q)
        tp.tp_attention_paged_fp8(q, c.cache, batch, outs=outs, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seqs in ([(0, 3), (17, 40), (80, 1)], [(300, 40), (500, 40), (90, 40)], [(5, 0), (100, 39), (0, 0)]):
        table.copy_(table[[1, 2, 0]])
        order = table.cpu().numpy()
        room = [int((row > 0).sum()) + 1 for row in order]
        at, new = 2, []
        for s, (old, n) in enumerate(seqs):
            old = min(old, 32 * 3 - n) if room[s] < 16 else old
            new.append((at, n, old + n))
            at += n
        c.seqs, c.table = new, order
        starts.copy_(i32([a for a, _, _ in new] + [at]))
        lengths.copy_(i32([n for _, _, n in new]))
        for t in x:
            t.copy_(to_bf16(c.rng.normal(size=t.shape)))
        for t in q + outs:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        tp.tp_device_status()
        c.q, (c.codes, c.scales) = q, c.got()
        for r in range(2):
            owned = np.concatenate([np.arange(a, a + n) for a, n, _ in new]).astype(int)
            want = np.full((c.T, c.heads * c.D), 7.0)
            want[owned] = f64(x[r])[owned, :c.heads * c.D]
            np.testing.assert_array_equal(f64(q[r]), want)
        c.check(outs, before=fresh(q), what=seqs)


def test_no_pages_at_all():
    """An empty page table, and a cache without pages: no row sees a key; a length that claims some is reported."""
    c = Case([(0, 3), (0, 50)], p=1, n_kv=2, group=2, D=64, page=16, seed=39)
    q = c.queries()
    none = tp.PagedBatch(c.batch.seq_start, i32([0, 0]), torch.empty((2, 0), dtype=torch.int32, device=DEV), 50)
    small = tp.PagedBatch(i32([0, 3, 3]), i32([0, 0]), torch.empty((2, 0), dtype=torch.int32, device=DEV), 3)
    for batch, rows in ((none, 53), (small, 3)):
        outs = fresh(q)
        tp.tp_attention_paged_fp8(q, c.cache, batch, outs=outs, window=5)
        tp.tp_device_status()
        assert torch.all(outs[0][:rows] == 0) and torch.all(outs[0][rows:] == 7)
    k = torch.empty((0, 2, 16, 64), dtype=E4M3, device=DEV)
    s = torch.empty((0, 2), dtype=E8M0, device=DEV)
    empty = tp.PagedCache([k], [k], [s], [s])
    for batch in (c.batch, tp.PagedBatch(i32([0, 3, 3]), i32([3, 0]), c.batch.page_table, 3)):
        outs = tp.tp_attention_paged_fp8(q, empty, batch)
        with pytest.raises(tp.TPError, match="TP_ERR_INVALID_ARG"):
            tp.tp_device_status()
        assert torch.all(outs[0][:3] == 0)
        tp.tp_kv_append_fp8(qkv_of(c), c.heads, empty, batch)
        with pytest.raises(tp.TPError, match="TP_ERR_INVALID_ARG"):
            tp.tp_device_status()


@pytest.mark.parametrize("max_new", [2, 5, 17, 200])
def test_more_rows_allowed_than_there_are(max_new):
    """max_new chooses the kernel; any bound has the same answers."""
    c = Case([(700, 1), (33, 2), (0, 1), (2000, 1)], p=2, n_kv=2, group=3, D=128, page=16, seed=40, behind=2)
    c.batch = c.make_batch(max_new)
    qkv = qkv_of(c)
    q = tp.tp_kv_append_fp8(qkv, c.heads, c.cache, c.batch)
    c.q, (codes, scales) = q, c.got()
    for r in range(2):
        _, k, v = split(c, f64(qkv[r]))
        P.append(c.codes[r][0], c.scales[r][0], k, c.seqs, c.table)
        P.append(c.codes[r][1], c.scales[r][1], v, c.seqs, c.table)
        np.testing.assert_array_equal(scales[r], c.scales[r])
        np.testing.assert_array_equal(F.e4m3_to_f64(codes[r]), F.e4m3_to_f64(c.codes[r]))
    outs = fresh(q)
    tp.tp_attention_paged_fp8(q, c.cache, c.batch, outs=outs)
    c.check(outs, before=fresh(q))


@pytest.mark.parametrize("seqs, new, p, n_kv, group, D, page", [
    ([90 + 7 * i for i in range(40)], 1, 2, 4, 3, 128, 16), ([700, 0, 33], 70, 2, 4, 2, 128, 64), ([900, 5], 40, 2, 4, 2, 64, 32)],
    ids=["tokens", "chunks", "chunks64"])
def test_steps_one_after_another(seqs, new, p, n_kv, group, D, page):
    """Appends and attentions that follow each other without a wait, tokens growing so that scales change at every step: the
    bits of the same steps with a wait after each call."""
    steps = 24
    c = Case([(old, new) for old in seqs], p=p, n_kv=n_kv, group=group, D=D, page=page, seed=42, spare=sum(-(-new * steps // page) + 1 for _ in seqs))
    used = c.table.copy()
    free = sorted(set(range(c.n_pages)) - {int(x) for s, (_, _, n) in enumerate(c.seqs) for x in used[s, :-(-n // page)]})
    need = [-(-(old + new * steps) // page) for old in seqs]
    c.table = np.zeros((len(seqs), max(need)), dtype=np.int32)
    for s, (_, _, n) in enumerate(c.seqs):
        have = -(-n // page)
        c.table[s, :have] = used[s, :have]
        for i in range(have, need[s]):
            c.table[s, i] = free.pop()
    x = [[to_bf16(c.rng.normal(size=(c.T, (c.heads + 2 * n_kv) * D)) * 1.3 ** k) for _ in range(p)] for k in range(steps)]
    cs = torch.from_numpy(quarter_table(c.rng, max(seqs) + new * steps + 1, D)).to(DEV)
    starts, table = i32([new * s for s in range(len(seqs) + 1)]), i32(c.table.tolist())
    batches = [tp.PagedBatch(starts, i32([old + new * (k + 1) for old in seqs]), table, new) for k in range(steps)]
    results = []
    for wait in (True, False, False, False):
        c.upload()
        torch.cuda.synchronize()
        outs = []
        for k in range(steps):
            q = tp.tp_kv_append_fp8(x[k], c.heads, c.cache, batches[k], rope="half", cos_sin=cs)
            if wait:
                torch.cuda.synchronize()
            outs.append(tp.tp_attention_paged_fp8(q, c.cache, batches[k]))
            if wait:
                torch.cuda.synchronize()
        codes, scales = c.got()
        results.append(([t for o in outs for t in o], codes, scales))
    for got in results[1:]:
        for i, (a, b) in enumerate(zip(results[0][0], got[0])):
            assert torch.equal(a, b), (i // p, i % p, int((a != b).sum()))
        for r in range(p):
            np.testing.assert_array_equal(results[0][1][r], got[1][r])
            np.testing.assert_array_equal(results[0][2][r], got[2][r])
