"""The paged 8-bit cache's measured cases: appending keys and values with their rotation, and attention over the cache.

A rank's cache holds pages of P tokens: codes k, v [pages, kv heads, P, D] as e4m3 and one power-of-two scale (e8m0)
for each page and head.  Sequence s has the new rows [seq_start[s], seq_start[s+1]) of every rank's Q, K and V, and kv_len[s]
tokens in the cache with them; its i-th of n new rows stands at position kv_len[s] - n + i, and position j is slot j % P of the
page page_table[s][j // P].

* append     Q and K are rotated (pairs (x[i], x[i + R/2]) or (x[2i], x[2i+1]); (x1 c - x2 s, x2 c + x1 s), c and s from a
             table's row for the position).  A page's exponent e is the least from -127 on with max|x| <= 448 * 2^e over its new
             values, and not less than the one it has where older tokens of the sequence are in it; these tokens' codes q
             become e4m3(q * 2^(e_old - e)), the new ones are e4m3(x / 2^e).
* attention  out = softmax(scale q K^T) V over the visible keys j: j <= position where causal, j > position - window where
             there is a window; 0 where no key is visible.  Query head h reads KV head h // (heads / kv heads).

`own` selects between the plain form (elementary torch operations in 32 bits) and the framework's calls.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
BF16 = torch.bfloat16
DEV = "cuda"


def listed():
    return [
        # One sequence's next token joins the cache (decode): pure latency.
        _append("append_token", p=4, heads=12, kv=2, D=128, page=16, S=1, ctx=(999, 999), new=(1, 1), rot=128, style="half"),
        # A decode batch, every sequence somewhere else in its last page.
        _append("append_batch", p=4, heads=12, kv=2, D=128, page=64, S=61, ctx=(17, 3000), new=(1, 1), rot=128, style="half"),
        # A prompt of a model with as many KV heads as heads: the largest append.
        _append("append_prompt", p=4, heads=12, kv=12, D=128, page=16, S=1, ctx=(0, 0), new=(4608, 4608), rot=128, style="half"),
        # Chunks of several prompts of odd lengths; a small head, half of it rotated, in neighbouring pairs.
        _append("append_ragged", p=2, heads=10, kv=5, D=64, page=32, S=7, ctx=(0, 700), new=(1, 611), rot=32, style="pairs"),
        # One token over a short cache: latency.
        _attend("attend_token_short", p=4, heads=12, kv=2, D=128, page=16, S=1, ctx=(200, 200), new=(1, 1)),
        # One token over a long document: few rows, a long axis.
        _attend("attend_token_long", p=4, heads=12, kv=2, D=128, page=64, S=1, ctx=(131000, 131000), new=(1, 1)),
        # A decode batch of ragged lengths, six query heads on a KV head.
        _attend("attend_batch", p=4, heads=12, kv=2, D=128, page=16, S=64, ctx=(50, 8000), new=(1, 1)),
        # A decode batch of a model with as many KV heads as heads.
        _attend("attend_batch_heads", p=4, heads=12, kv=12, D=128, page=32, S=24, ctx=(1000, 2900), new=(1, 1)),
        # A few drafted tokens a sequence, to be verified in one pass.
        _attend("attend_drafts", p=4, heads=12, kv=2, D=128, page=16, S=16, ctx=(500, 9000), new=(5, 5)),
        # A whole prompt over its own keys, the largest product.
        _attend("attend_prompt", p=4, heads=12, kv=12, D=128, page=16, S=1, ctx=(0, 0), new=(4608, 4608)),
        # A chunk of a prompt over a long prefix.
        _attend("attend_chunk", p=4, heads=12, kv=2, D=128, page=64, S=1, ctx=(30011, 30011), new=(300, 300)),
        # Prompts of odd lengths with a sliding window and a small head.
        _attend("attend_ragged_window", p=2, heads=10, kv=5, D=64, page=32, S=7, ctx=(0, 700), new=(1, 1111), window=400),
    ]


def _append(name, p, heads, kv, D, page, S, ctx, new, rot, style, mix=1):
    return dict(name=name, op="append", p=p, heads=heads, kv=kv, D=D, page=page, S=S, ctx_lo=ctx[0], ctx_hi=ctx[1],
                new_lo=new[0], new_hi=new[1], rot=rot, style=style, mix=mix)


def _attend(name, p, heads, kv, D, page, S, ctx, new, causal=True, window=0, mix=1):
    return dict(name=name, op="attend", p=p, heads=heads, kv=kv, D=D, page=page, S=S, ctx_lo=ctx[0], ctx_hi=ctx[1],
                new_lo=new[0], new_hi=new[1], causal=causal, window=window, mix=mix)


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend"])
    p, kv = rng.choice([(1, 8), (1, 5), (2, 4), (4, 2), (8, 1), (4, 12), (3, 3)])
    heads = kv * rng.choice([1, 2, 4, 6, 8] if p * kv <= 15 else [1])
    D, page, mix = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), rng.randrange(1 << 30)
    kind = rng.choice(["decode", "decode", "chunk", "prompt"])
    if kind == "decode":
        S, new = _log_int(rng, 1, 64), (1, rng.choice([1, 1, 1, 3, 6]))
        top = _log_int(rng, 16, min(131000, 1_000_000 // (S * p * kv) if op == "attend" else 4000))
        ctx = (max(0, top // rng.choice([1, 2, 20])), top)
    elif kind == "chunk":
        S, top = _log_int(rng, 1, 6), _log_int(rng, 30, 700)
        ctx, new = (0, _log_int(rng, 100, 20000 // S)), (max(1, top // 3), top)
    else:
        S, top = rng.choice([(1, 4608), (2, 2000), (5, 800)])
        top = _log_int(rng, 64, top)
        ctx, new = (0, 0), (max(1, top // 2), top)
    if op == "append":
        return _append(None, p, heads, kv, D, page, S, ctx, new, rng.choice([D, D, D // 2]), rng.choice(["half", "pairs"]),
                       mix) | dict(name="")
    causal = rng.random() < 0.85
    window = _log_int(rng, 16, 4096) if causal and rng.random() < 0.25 else 0
    return _attend(None, p, heads, kv, D, page, S, ctx, new, causal, window, mix) | dict(name="")


def _lengths(case):
    """(cached tokens, new tokens) of every sequence."""
    rng = random.Random(case["mix"])
    return [(rng.randint(case["ctx_lo"], case["ctx_hi"]), rng.randint(case["new_lo"], case["new_hi"])) for _ in range(case["S"])]


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _ceil(a, b):
    return -(-a // b)


def _exponent(top):
    """The least e >= -127 with top <= 448 * 2^e."""
    m, k = torch.frexp(top)                                            # 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, k - 8, k - 9).clamp(-127, 127)
    return torch.where(top > 0, e, torch.full_like(e, -127))


def _pages(g, n, kv, page, D, std):
    """Codes and scales of n pages: values with a few strong features, as keys have, and tokens of unlike size."""
    x = _normal(g, (n, kv, page, D), std)
    x *= torch.where(torch.rand((kv, 1, D), generator=g, device=DEV) < 0.02, 6.0, 1.0)
    x *= torch.exp(_normal(g, (n, 1, page, 1), 0.3))
    e = _exponent(x.abs().amax((2, 3)))
    return torch.ldexp(x, -e[:, :, None, None].float()).to(E4M3), (e + 127).to(torch.uint8).view(E8M0)


def _rotation_table(positions, R):
    """cos and sin of position * 10000^(-2 i / R), side by side; the angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(R // 2, device=DEV, dtype=torch.float64) * 2 / R)
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g = _gen(seed)
    c = case
    at = _lengths(c)
    total = [old + new for old, new in at]
    need = [_ceil(t, c["page"]) for t in total]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV)
    table = torch.zeros((c["S"], max(need)), dtype=torch.int32, device=DEV)
    first = 0
    for s, n in enumerate(need):
        table[s, :n] = order[first:first + n]
        first += n
    starts = [0]
    for _, new in at:
        starts.append(starts[-1] + new)
    T = starts[-1]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = dict(case=c, op=c["op"], starts=starts, total=total, T=T, table=table, max_q=max(new for _, new in at),
             seq_start=i32(starts), kv_len=i32(total))
    k = [_pages(g, n_pages, c["kv"], c["page"], c["D"], 1.5) for _ in range(c["p"])]
    v = [_pages(g, n_pages, c["kv"], c["page"], c["D"], 0.8) for _ in range(c["p"])]
    s["k"], s["ks"], s["v"], s["vs"] = [x for x, _ in k], [x for _, x in k], [x for x, _ in v], [x for _, x in v]
    wide = c["heads"] * c["D"]
    if c["op"] == "append":
        s["qkv"] = [_normal(g, (T, wide + 2 * c["kv"] * c["D"]), 1.3).to(BF16) for _ in range(c["p"])]
        s["table_cs"] = _rotation_table(max(total), c["rot"])
        s["q"] = [torch.empty((T, wide), dtype=BF16, device=DEV) for _ in range(c["p"])]
    else:
        s["q"] = [_normal(g, (T, wide), 1.5).to(BF16) for _ in range(c["p"])]
        s["out"] = [torch.empty((T, wide), dtype=BF16, device=DEV) for _ in range(c["p"])]
    if own:
        import tensor_sharded_linear_tp_gb300 as tp
        s["cache"] = tp.PagedCache(s["k"], s["v"], s["ks"], s["vs"])
        s["batch"] = tp.PagedBatch(s["seq_start"], s["kv_len"], table, max_q=s["max_q"])
        if c["op"] == "attend":
            need = tp.tp_attention_paged_workspace_bytes(s["cache"], s["batch"], T, c["heads"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------- the plain form

def _rotate(x, cs, R, style):
    """x [T, heads, D] in 32 bits, cs [T, R]."""
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    if style == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _plain_append(s):
    c = s["case"]
    D, P, kv, heads, T = c["D"], c["page"], c["kv"], c["heads"], s["T"]
    place, page, group, first_slot, group_page = [], [], [], [], []
    for i, total in enumerate(s["total"]):
        new = s["starts"][i + 1] - s["starts"][i]
        j = torch.arange(total - new, total, device=DEV)
        place.append(j)
        page.append(s["table"][i, j // P].long())
        lo = (total - new) // P
        group.append(j // P - lo + len(first_slot))
        pages = range(lo, (total - 1) // P + 1)
        first_slot += [(total - new) % P if n == lo else 0 for n in pages]
        group_page.append(s["table"][i, lo:(total - 1) // P + 1].long())
    place, page, group, group_page = torch.cat(place), torch.cat(page), torch.cat(group), torch.cat(group_page)
    old = torch.tensor(first_slot, device=DEV)                       # tokens of the sequence that a page held before
    slot = place % P
    cs = s["table_cs"][place]
    for r in range(c["p"]):
        x = s["qkv"][r].float()
        q = x[:, :heads * D].view(T, heads, D)
        k = x[:, heads * D:(heads + kv) * D].view(T, kv, D)
        v = x[:, (heads + kv) * D:].view(T, kv, D)
        s["q"][r].copy_(_rotate(q, cs, c["rot"], c["style"]).view(T, heads * D))
        for new, codes, scales in ((_rotate(k, cs, c["rot"], c["style"]), s["k"][r], s["ks"][r]), (v, s["v"][r], s["vs"][r])):
            top = torch.zeros((len(old), kv), device=DEV)
            top = top.scatter_reduce(0, group[:, None].expand(-1, kv), new.abs().amax(2), "amax")
            e = _exponent(top)
            e_old = scales.view(torch.uint8)[group_page].int() - 127
            e = torch.where(old[:, None] > 0, torch.maximum(e, e_old), e)
            was = codes.view(torch.uint8)[group_page].view(E4M3).float()    # [groups, kv, P, D]
            kept = torch.ldexp(was, (e_old - e).clamp(-127, 0)[:, :, None, None].float()).to(E4M3).view(torch.uint8)
            keep = torch.arange(P, device=DEV)[None, :] < old[:, None]
            all_codes = codes.view(torch.uint8)
            all_codes[group_page] = torch.where(keep[:, None, :, None], kept, all_codes[group_page])
            scales.view(torch.uint8)[group_page] = (e + 127).to(torch.uint8)
            coded = torch.ldexp(new, -e[group][:, :, None].float()).to(E4M3).view(torch.uint8)
            all_codes[page[:, None], torch.arange(kv, device=DEV)[None, :], slot[:, None]] = coded
    return s["q"], s["k"], s["ks"], s["v"], s["vs"]


def _plain_attend(s):
    c = s["case"]
    D, P, kv, heads = c["D"], c["page"], c["kv"], c["heads"]
    G, scale = heads // kv, 1.0 / math.sqrt(D)
    for i, total in enumerate(s["total"]):
        a, b = s["starts"][i], s["starts"][i + 1]
        pages = s["table"][i, :_ceil(total, P)].long()
        pos = torch.arange(total - (b - a), total, device=DEV)[:, None]
        key = torch.arange(total, device=DEV)[None, :]
        seen = torch.ones((b - a, total), dtype=torch.bool, device=DEV)
        if c["causal"]:
            seen &= key <= pos
        if c["window"]:
            seen &= key > pos - c["window"]
        for r in range(c["p"]):
            def whole(codes, scales):
                x = codes.view(torch.uint8)[pages].view(E4M3).float()
                x = x * scales.view(torch.uint8)[pages].view(E8M0).float()[:, :, None, None]
                return x.transpose(0, 1).reshape(kv, -1, D)[:, :total]
            K, V = whole(s["k"][r], s["ks"][r]), whole(s["v"][r], s["vs"][r])
            q = s["q"][r][a:b].float().view(b - a, kv, G, D)
            for h in range(kv):
                x = torch.matmul(q[:, h].transpose(0, 1), K[h].t()) * scale          # [G, new, total]
                x = x.masked_fill(~seen, float("-inf"))
                x = torch.exp(x - x.amax(2, keepdim=True))
                x = torch.matmul(x, V[h]) / x.sum(2, keepdim=True)
                s["out"][r][a:b, h * G * D:(h + 1) * G * D] = x.transpose(0, 1).reshape(b - a, G * D).to(BF16)
    return s["out"]


# ---------------------------------------------------------------------------- the framework's calls

def _framework(s):
    import tensor_sharded_linear_tp_gb300 as tp
    c = s["case"]
    if c["op"] == "append":
        tp.tp_kv_append_fp8(s["qkv"], c["heads"], s["cache"], s["batch"], rope=c["style"], cos_sin=s["table_cs"], q_out=s["q"])
        return s["q"], s["k"], s["ks"], s["v"], s["vs"]
    return tp.tp_attention_paged_fp8(s["q"], s["cache"], s["batch"], causal=c["causal"], window=c["window"], outs=s["out"],
                                     workspace=s["workspace"])


def run(state):
    if own:
        return _framework(state)
    return _plain_append(state) if state["op"] == "append" else _plain_attend(state)


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    at = _lengths(c)
    T = sum(new for _, new in at)
    p, D, kv, heads = c["p"], c["D"], c["kv"], c["heads"]
    if c["op"] == "append":
        pages = sum(_ceil(old + new, c["page"]) - old // c["page"] for old, new in at)
        rows = p * T * D * (2 * (heads + 2 * kv) + 2 * heads + 2 * kv)
        places = len({j for old, new in at for j in range(old, old + new)})
        return {"bytes": rows + p * 2 * kv * pages + 4 * places * c["rot"], "flops": p * T * D * (6 * (heads + kv) + 3 * kv)}
    keys = pairs = 0
    for old, new in at:
        lo = max(0, old + 1 - c["window"]) if c["window"] else 0
        keys += old + new - lo
        for i in range(new):
            n = old + i + 1 if c["causal"] else old + new
            pairs += min(n, c["window"]) if c["window"] else n
    return {"bytes": p * (4 * T * heads * D + 2 * keys * kv * D + 2 * kv * _ceil(keys, c["page"])), "flops": 4.0 * p * heads * D * pairs}


# ---------------------------------------------------------------------------- the definition in 64 bits

def _power(scales):
    return torch.exp2(scales.view(torch.uint8).double() - 127.0)


def _exact_append(case, seed):
    s = prepare(case, seed)
    c = case
    D, P, R, kv, heads = c["D"], c["page"], c["rot"], c["kv"], c["heads"]
    out = ([], [], [], [], [])
    first = torch.arange(R // 2, device=DEV) * (1 if c["style"] == "half" else 2)
    second = first + (R // 2 if c["style"] == "half" else 1)
    for r in range(c["p"]):
        x = s["qkv"][r].double().view(s["T"], heads + 2 * kv, D)
        place = torch.cat([torch.arange(t - (s["starts"][i + 1] - s["starts"][i]), t, device=DEV) for i, t in enumerate(s["total"])])
        cs = s["table_cs"].double()[place]
        c1, s1 = cs[:, :R // 2].unsqueeze(1), cs[:, R // 2:].unsqueeze(1)
        y = x.clone()
        turned = slice(0, heads + kv)
        y[:, turned, first] = x[:, turned, first] * c1 - x[:, turned, second] * s1
        y[:, turned, second] = x[:, turned, second] * c1 + x[:, turned, first] * s1
        out[0].append(y[:, :heads].reshape(s["T"], heads * D))
        for codes, scales, at, to, to_s in ((s["k"][r], s["ks"][r], heads, out[1], out[2]),
                                            (s["v"][r], s["vs"][r], heads + kv, out[3], out[4])):
            value, size = codes.double(), _power(scales)
            for i, total in enumerate(s["total"]):
                a, b = s["starts"][i], s["starts"][i + 1]
                j = total - (b - a)
                while j < total:                      # page by page
                    page, lo = int(s["table"][i, j // P]), j % P
                    n = min(P - lo, total - j)
                    new = y[a:a + n, at:at + kv].transpose(0, 1)                     # [kv, n, D]
                    top = new.abs().amax((1, 2))
                    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0)) - 1
                    for _ in range(2):
                        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
                    power = torch.exp2(e.clamp(-127, 127))
                    if lo:
                        power = torch.maximum(power, size[page])
                        value[page, :, :lo] *= (size[page] / power)[:, None, None]
                    size[page] = power
                    value[page, :, lo:lo + n] = new / power[:, None, None]
                    a, j = a + n, j + n
            to.append(value)
            to_s.append(size)
    return out


def _exact_attend(case, seed):
    s = prepare(case, seed)
    c = case
    D, P, kv, heads = c["D"], c["page"], c["kv"], c["heads"]
    G = heads // kv
    outs = []
    for r in range(c["p"]):
        out = torch.empty((s["T"], heads, D), dtype=torch.float64, device=DEV)
        for i, total in enumerate(s["total"]):
            a, b = s["starts"][i], s["starts"][i + 1]
            j = torch.arange(total, device=DEV)
            page, slot = s["table"][i, j // P].long(), j % P
            pos = torch.arange(total - (b - a), total, device=DEV)
            hidden = torch.zeros((b - a, total), dtype=torch.bool, device=DEV)
            if c["causal"]:
                hidden |= j[None, :] > pos[:, None]
            if c["window"]:
                hidden |= j[None, :] <= pos[:, None] - c["window"]
            for h in range(kv):
                K = s["k"][r].view(torch.uint8)[page, h, slot].view(E4M3).double() * _power(s["ks"][r])[page, h][:, None]
                V = s["v"][r].view(torch.uint8)[page, h, slot].view(E4M3).double() * _power(s["vs"][r])[page, h][:, None]
                for n in range(h * G, (h + 1) * G):
                    z = s["q"][r][a:b, n * D:(n + 1) * D].double() @ K.T / math.sqrt(D)
                    w = torch.softmax(z.masked_fill(hidden, -math.inf), 1)
                    out[a:b, n] = w @ V
        outs.append(out.view(s["T"], heads * D))
    return outs


def exact(case, seed):
    return _exact_append(case, seed) if case["op"] == "append" else _exact_attend(case, seed)
