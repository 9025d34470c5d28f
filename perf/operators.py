"""The 8-bit operators' measured cases: block-scaled fp8 projections, their quantiser, and the residual norm.

Formulas (a group is 128 consecutive features of one row, or a 128 x 128 block of a weight; the last
group of a row or column may be shorter):

* quantize      e = ceil(log2(max|x| / 448)) clamped to [-127, 127] (0 for a group of zeros), the scale 2^e is
                held as the e8m0 byte e + 127, q = e4m3(x / 2^e), one rounding to nearest even
* colwise       Y_r = act(dequant(X) . dequant(W_r)^T + b_r) for every rank r, as bf16 or quantised by token group
* rowwise       Z = sum_r dequant(X_r) . dequant(W_r)^T + b, as bf16
* residual_norm h = alpha x + gate * post_norm(y), u = norm(h) * (1 + scale) + shift, h as bf16, u as bf16 or quantised

`own` selects between the plain form (elementary torch operations in 32 bits) and the framework's calls.
"""
import math

import torch

own = False

GROUP = 128
E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
DEV = "cuda"


def listed():
    return [
        # One token's activations before a projection (decode): pure latency.
        dict(name="quantize_token", op="quantize", T=1, K=6144, rows=1),
        # A prompt's MLP hidden state before the down projection.
        dict(name="quantize_prompt", op="quantize", T=4608, K=18432, rows=1),
        # One rank's shard of the gate/up weight, quantised once at load.
        dict(name="quantize_weight", op="quantize", T=9216, K=6144, rows=128),
        # The fused Q, K, V projection of one token (decode).
        dict(name="colwise_token_qkv", op="colwise", T=1, K=6144, p=4, N=4608, act="none", bias=True, out="bf16"),
        # Gate/up of a few tokens (a small decode batch) on three ranks, the hidden state quantised for the down projection.
        dict(name="colwise_few_swiglu", op="colwise", T=23, K=6144, p=3, N=12288, act="swiglu", bias=False, out="fp8"),
        # A small model's up projection over a short odd prompt: no size a multiple of its tile.
        dict(name="colwise_ragged_gelu", op="colwise", T=333, K=2000, p=2, N=1096, act="gelu_tanh", bias=True, out="bf16"),
        # Gate/up of a whole prompt, the largest product of a block.
        dict(name="colwise_prompt_swiglu", op="colwise", T=4608, K=6144, p=4, N=9216, act="swiglu", bias=False, out="fp8"),
        # The down projection of one token (decode).
        dict(name="rowwise_token_down", op="rowwise", T=1, K=4608, p=4, N=6144, bias=False),
        # The attention out-projection over a chunk of a prompt.
        dict(name="rowwise_chunk_out", op="rowwise", T=300, K=1536, p=4, N=6144, bias=True),
        # The down projection of a whole prompt.
        dict(name="rowwise_prompt_down", op="rowwise", T=4608, K=4608, p=4, N=6144, bias=False),
        # Between two sharded blocks, one token: the block's sum joins the residual and the next block's input leaves as fp8.
        dict(name="norm_token", op="residual_norm", T=1, D=6144, pre="rms", post="rms", affine=True, gate=True, mod=True,
             batch=1, out="fp8"),
        # The same for a prompt of a modulated (AdaLN) transformer, two samples with their own gate, scale and shift.
        dict(name="norm_prompt", op="residual_norm", T=4608, D=6144, pre="layer", post="rms", affine=False, gate=True,
             mod=True, batch=2, out="fp8"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["quantize", "colwise", "colwise", "rowwise", "rowwise", "residual_norm"])
    T = _log_int(rng, 1, 4608)
    if op == "quantize":
        rows = rng.choice([1, 1, 128])
        return dict(op=op, T=T if rows == 1 else _log_int(rng, 64, 9216), K=_log_int(rng, 256, 18432, 16), rows=rows)
    if op == "colwise":
        p = rng.choice([1, 2, 3, 4, 6, 8])
        act = rng.choice(["none", "gelu_tanh", "swiglu"])
        out = rng.choice(["bf16", "fp8"])
        n_out = _log_int(rng, 128, 18432 // p, 16)
        return dict(op=op, T=T, K=_log_int(rng, 256, 6144, 16), p=p, N=2 * n_out if act == "swiglu" else n_out, act=act,
                    bias=rng.random() < 0.5, out=out)
    if op == "rowwise":
        p = rng.choice([1, 2, 3, 4, 6, 8])
        return dict(op=op, T=T, K=_log_int(rng, 128, 18432 // p, 16), p=p, N=_log_int(rng, 128, 6144, 8),
                    bias=rng.random() < 0.5)
    pre = rng.choice(["none", "rms", "rms", "layer"])
    out = rng.choice(["bf16", "fp8"])
    return dict(op=op, T=T, D=_log_int(rng, 128, 12288, 16), pre=pre, post=rng.choice(["none", "rms", "layer"]),
                affine=rng.random() < 0.5, gate=rng.random() < 0.7, mod=rng.random() < 0.7,
                batch=rng.choice([1, 2, 3]), out=out)


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _activation(g, T, K):
    """Activations with a few strong features, as transformers have; where there are several tokens the last is padding."""
    x = _normal(g, (T, K), 1.0)
    x *= torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    if T > 4:
        x[-1] = 0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    bf16 = torch.bfloat16
    if op == "quantize":
        T, K = case["T"], case["K"]
        s["x"] = _activation(g, T, K) if case["rows"] == 1 else _normal(g, (T, K), 0.02).to(bf16)
        s["q"] = torch.empty((T, K), dtype=E4M3, device=DEV)
        s["scales"] = _scale_buffer(_ceil(T, case["rows"]), _ceil(K, GROUP))
    elif op == "colwise":
        T, K, p, N = case["T"], case["K"], case["p"], case["N"]
        s["x"], s["sx"] = _quantize(_activation(g, T, K).float(), 1)
        s["w"], s["sw"] = _weights(g, p, N, K)
        s["bias"] = [_normal(g, (N,), 0.1).to(bf16) for _ in range(p)] if case["bias"] else None
        n = N // 2 if case["act"] == "swiglu" else N
        fp8 = case["out"] == "fp8"
        s["y"] = [torch.empty((T, n), dtype=E4M3 if fp8 else bf16, device=DEV) for _ in range(p)]
        s["sy"] = [_scale_buffer(T, _ceil(n, GROUP)) for _ in range(p)] if fp8 else None
    elif op == "rowwise":
        T, K, p, N = case["T"], case["K"], case["p"], case["N"]
        xs = [_quantize(_activation(g, T, K).float(), 1) for _ in range(p)]
        s["x"], s["sx"] = [x for x, _ in xs], [sx for _, sx in xs]
        s["w"], s["sw"] = _weights(g, p, N, K)
        s["bias"] = _normal(g, (N,), 0.1).to(bf16) if case["bias"] else None
        s["z"] = torch.empty((T, N), dtype=bf16, device=DEV)
    else:
        T, D, B = case["T"], case["D"], case["batch"]
        s["x"], s["y"] = (_normal(g, (T, D), 2.0) + 0.3).to(bf16), (_normal(g, (T, D), 0.7) - 0.1).to(bf16)
        vec = lambda c, std: (c + _normal(g, (D,), std)).to(bf16)  # noqa: E731
        s["post_weight"] = vec(1.0, 0.1) if case["affine"] and case["post"] != "none" else None
        s["weight"] = vec(1.0, 0.1) if case["affine"] and case["pre"] != "none" else None
        # One projection of the conditioning gives every sample's gate, scale and shift side by side.
        table = _normal(g, (B, 3 * D), 0.3).to(bf16)
        s["gate"] = table[:, :D] if case["gate"] else None
        s["scale"], s["shift"] = (table[:, D:2 * D], table[:, 2 * D:]) if case["mod"] else (None, None)
        s["rows_per_mod"] = _ceil(T, B)
        s["alpha"], s["eps"] = 1.0, 1e-6
        s["h"] = torch.empty((T, D), dtype=bf16, device=DEV)
        fp8 = case["out"] == "fp8"
        s["u"] = torch.empty((T, D), dtype=E4M3 if fp8 else bf16, device=DEV)
        s["su"] = _scale_buffer(T, _ceil(D, GROUP)) if fp8 else None
    return s


def _ceil(a, b):
    return -(-a // b)


def _scale_buffer(rows, cols):
    return torch.empty((rows, cols), dtype=torch.uint8, device=DEV).view(E8M0)


def _weights(g, p, N, K):
    ws = [_quantize(_normal(g, (N, K), 0.02).to(torch.bfloat16).float(), GROUP) for _ in range(p)]
    return [w for w, _ in ws], [sw for _, sw in ws]


# ---------------------------------------------------------------------------- the plain form

def _quantize(x, rows):
    """(q, scales) of a float32 matrix by groups of rows x 128."""
    T, K = x.shape
    nr, nc = _ceil(T, rows), _ceil(K, GROUP)
    pad = torch.nn.functional.pad(x, (0, nc * GROUP - K, 0, nr * rows - T)).view(nr, rows, nc, GROUP)
    m, k = torch.frexp(pad.abs().amax((1, 3)))                         # 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, k - 8, k - 9).clamp(-127, 127)
    e = torch.where(m > 0, e, torch.zeros_like(e))
    q = torch.ldexp(pad, -e[:, None, :, None].float()).to(E4M3).view(nr * rows, nc * GROUP)
    return q[:T, :K].contiguous(), (e + 127).to(torch.uint8).view(E8M0)


def _dequantize(q, scales, rows):
    T, K = q.shape
    s = scales.float().repeat_interleave(GROUP, 1)[:, :K]
    if rows > 1:
        s = s.repeat_interleave(rows, 0)[:T]
    return q.float() * s


def _activate(y, act):
    if act == "gelu_tanh":
        return 0.5 * y * (1.0 + torch.tanh(0.7978845608028654 * (y + 0.044715 * y * y * y)))
    if act == "swiglu":
        a, b = y.chunk(2, dim=1)
        return a / (1.0 + torch.exp(-a)) * b
    return y


def _norm(v, kind, weight, eps):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    return v if weight is None else v * weight.float()


def _rows(table, T, per):
    """A modulation table's row for every token."""
    return table.float().repeat_interleave(per, 0)[:T]


def _plain(s):
    c, op = s["case"], s["op"]
    if op == "quantize":
        return _quantize(s["x"].float(), c["rows"])
    if op == "colwise":
        x = _dequantize(s["x"], s["sx"], 1)
        ys, ss = [], []
        for r in range(c["p"]):
            y = x @ _dequantize(s["w"][r], s["sw"][r], GROUP).t()
            if s["bias"] is not None:
                y = y + s["bias"][r].float()
            y = _activate(y, c["act"])
            if c["out"] == "fp8":
                y, sy = _quantize(y, 1)
                ss.append(sy)
            ys.append(y if c["out"] == "fp8" else y.to(torch.bfloat16))
        return (ys, ss) if c["out"] == "fp8" else ys
    if op == "rowwise":
        z = torch.zeros((c["T"], c["N"]), device=DEV)
        for r in range(c["p"]):
            z = z + _dequantize(s["x"][r], s["sx"][r], 1) @ _dequantize(s["w"][r], s["sw"][r], GROUP).t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        return z.to(torch.bfloat16)
    T, per = c["T"], s["rows_per_mod"]
    b = _norm(s["y"].float(), c["post"], s["post_weight"], s["eps"])
    if s["gate"] is not None:
        b = b * _rows(s["gate"], T, per)
    h = s["alpha"] * s["x"].float() + b
    u = _norm(h, c["pre"], s["weight"], s["eps"])
    if s["scale"] is not None:
        u = u * (1.0 + _rows(s["scale"], T, per)) + _rows(s["shift"], T, per)
    u, su = _quantize(u, 1) if c["out"] == "fp8" else (u.to(torch.bfloat16), None)
    return (h.to(torch.bfloat16), u) if su is None else (h.to(torch.bfloat16), u, su)


# ---------------------------------------------------------------------------- the framework's calls

def _framework(s):
    import tensor_sharded_linear_tp_gb300 as tp
    c, op = s["case"], s["op"]
    if op == "quantize":
        return tp.tp_quantize_fp8(s["x"], block_rows=c["rows"], q=s["q"], scales=s["scales"])
    if op == "colwise":
        return tp.tp_linear_colwise_fp8(s["x"], s["sx"], s["w"], s["sw"], act=c["act"], bias_shards=s["bias"], out=c["out"],
                                        y_shards=s["y"], y_scales=s["sy"])
    if op == "rowwise":
        return tp.tp_linear_rowwise_fp8(s["x"], s["sx"], s["w"], s["sw"], bias=s["bias"], out=s["z"])
    h, u, su = tp.tp_residual_norm(s["x"], s["y"], norm=c["pre"], weight=s["weight"], scale=s["scale"], shift=s["shift"],
                                   post_norm=c["post"], post_weight=s["post_weight"], gate=s["gate"], alpha=s["alpha"],
                                   eps=s["eps"], rows_per_mod=s["rows_per_mod"], out=c["out"], h=s["h"], u=s["u"],
                                   u_scales=s["su"])
    return (h, u) if su is None else (h, u, su)


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "quantize":
        T, K = case["T"], case["K"]
        groups = _ceil(T, case["rows"]) * _ceil(K, GROUP)
        return {"bytes": 3 * T * K + groups, "flops": 3 * T * K}
    if op == "residual_norm":
        T, D = case["T"], case["D"]
        out = T * D + T * _ceil(D, GROUP) if case["out"] == "fp8" else 2 * T * D
        vecs = 2 * D * case["batch"] * ((1 if case["gate"] else 0) + (2 if case["mod"] else 0))
        return {"bytes": 6 * T * D + out + vecs, "flops": 12 * T * D}
    T, K, p, N = case["T"], case["K"], case["p"], case["N"]
    kg = _ceil(K, GROUP)
    w = p * (N * K + _ceil(N, GROUP) * kg)
    x = T * K + T * kg
    if op == "rowwise":
        return {"bytes": w + p * x + 2 * T * N, "flops": 2.0 * p * T * K * N}
    n = N // 2 if case["act"] == "swiglu" else N
    out = p * (T * n + T * _ceil(n, GROUP)) if case["out"] == "fp8" else 2 * p * T * n
    return {"bytes": w + x + out, "flops": 2.0 * p * T * K * N}


# ---------------------------------------------------------------------------- the definition in 64 bits

def _value64(q, scales, rows):
    """What codes and e8m0 bytes stand for, group by group."""
    v = q.to(torch.float64)
    e = scales.view(torch.uint8).to(torch.float64) - 127.0
    row = torch.arange(v.shape[0], device=DEV) // rows
    col = torch.arange(v.shape[1], device=DEV) // GROUP
    return v * torch.exp2(e)[row][:, col]


def _codes64(v, rows, rounded=True):
    """The quantiser's definition on float64 values: the codes' values (before their rounding where `rounded` is
    false: a computed value has its own last bits, and which code a value beside a tie gets is theirs) and the scales."""
    T, K = v.shape
    row = torch.arange(T, device=DEV) // rows
    col = torch.arange(K, device=DEV) // GROUP
    flat = (row[:, None] * (int(col[-1]) + 1) + col[None, :]).reshape(-1)
    top = torch.zeros(int(flat[-1]) + 1, dtype=torch.float64, device=DEV)
    top = top.scatter_reduce(0, flat, v.abs().reshape(-1), "amax")
    # The least e with top <= 448 * 2^e: the logarithm gives it to within one, the comparison decides.
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0)) - 1
    for _ in range(2):
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top > 0, e.clamp(-127, 127), torch.zeros_like(e))
    t = v / torch.exp2(e)[flat].view(T, K)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)   # the codes' spacing there
    return torch.round(t / step) * step if rounded else t, torch.exp2(e).view(_ceil(T, rows), -1)


def _gelu64(y):
    return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _codes64(s["x"].double(), case["rows"])
    if op == "rowwise":
        z = sum(torch.matmul(_value64(s["x"][r], s["sx"][r], 1), _value64(s["w"][r], s["sw"][r], GROUP).T)
                for r in range(case["p"]))
        return z if s["bias"] is None else z + s["bias"].double()
    if op == "colwise":
        ys, ss = [], []
        x = _value64(s["x"], s["sx"], 1)
        for r in range(case["p"]):
            y = torch.matmul(x, _value64(s["w"][r], s["sw"][r], GROUP).T)
            if s["bias"] is not None:
                y += s["bias"][r].double()
            if case["act"] == "gelu_tanh":
                y = _gelu64(y)
            elif case["act"] == "swiglu":
                n = case["N"] // 2
                y = y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:]
            if case["out"] == "fp8":
                y, sy = _codes64(y, 1, rounded=False)
                ss.append(sy)
            ys.append(y)
        return (ys, ss) if case["out"] == "fp8" else ys
    T = case["T"]
    sample = torch.arange(T, device=DEV) // s["rows_per_mod"]

    def normed(v, kind, weight):
        if kind == "none":
            return v
        centre = v.mean(1, keepdim=True) if kind == "layer" else 0.0
        spread = torch.sqrt(((v - centre) ** 2).mean(1, keepdim=True) + s["eps"])
        return (v - centre) / spread * (1.0 if weight is None else weight.double())

    branch = normed(s["y"].double(), case["post"], s["post_weight"])
    if s["gate"] is not None:
        branch = branch * s["gate"].double()[sample]
    h = s["alpha"] * s["x"].double() + branch
    u = normed(h, case["pre"], s["weight"])
    if s["scale"] is not None:
        u = u * (1 + s["scale"].double()[sample]) + s["shift"].double()[sample]
    if case["out"] == "fp8":
        u, su = _codes64(u, 1, rounded=False)
        return h, u, su
    return h, u
