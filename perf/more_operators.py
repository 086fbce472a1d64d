"""The 8-bit floating-point product and the routing of rows to experts, as cases that can be timed and compared.

Five operators, each in a plain form (elementary torch operations, 32-bit arithmetic) and as the library's calls:

  linear    a whole layer in 8-bit floating point: E4M3 codes with one power-of-two scale per row and 128 channels of
            the activation and per 128 x 128 block of the weight; bias, activation, gate and residual behind it
  experts   the same for rows of tokens, sorted by expert, one layer per expert
  sort      the slots of a router's choice sorted by expert: the experts' row ranges, the rows' tokens, the slots' rows
  dispatch  the tokens' rows, weighted, written in the experts' order
  grad      the gradient of the weighted combination of a token's rows, to the rows and to the weights

``own`` chooses between the two: the plain form where it is false, the library's calls where it is true.
"""
import math

import torch

own = False

BLOCK = 128
ACTS = ("none", "gelu_tanh", "gelu_erf", "silu", "relu")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _linear(b, m, n, act="none", act_begin=0, gate=0, residual=False, bias=True, out="bf16"):
    """gate: rows that share one gate row (0 = no gate)."""
    return {"op": "linear", "b": b, "m": m, "n": n, "act": act, "act_begin": act_begin, "gate": gate,
            "residual": residual, "bias": bias, "out": out}


def _experts(tokens, topk, experts, m, n, act="none", act_begin=0, bias=True, pad=0, out="bf16"):
    return {"op": "experts", "tokens": tokens, "topk": topk, "experts": experts, "m": m, "n": n, "act": act,
            "act_begin": act_begin, "bias": bias, "pad": pad, "out": out}


def _sort(tokens, topk, experts, dropped=0.0):
    """dropped: the share of tokens that are padding (their slots name no expert)."""
    return {"op": "sort", "tokens": tokens, "topk": topk, "experts": experts, "dropped": dropped}


def _dispatch(tokens, topk, n, weight=True, dropped=0.0, out="bf16"):
    return {"op": "dispatch", "tokens": tokens, "topk": topk, "n": n, "weight": weight, "dropped": dropped, "out": out}


def _grad(tokens, topk, n, weight=True, dropped=0.0, out="bf16"):
    return {"op": "grad", "tokens": tokens, "topk": topk, "n": n, "weight": weight, "dropped": dropped, "out": out}


def listed():
    named = [
        # one sample's modulation vector, or one token's step: latency of a single layer
        ("linear, one row", _linear(1, 1152, 6912, act="silu")),
        # a text encoder's prompt of odd length through widths that no block divides, results kept in 32 bits
        ("linear, odd sizes", _linear(333, 1000, 1500, gate=111, residual=True, out="f32")),
        # PixArt-shaped MLP fc1 with its GELU (1024px latent, 4096 tokens)
        ("linear, fc1 + gelu", _linear(4096, 1152, 4608, act="gelu_tanh")),
        # a fused projection of 4608 tokens: attention columns as they are, GELU on the MLP columns behind them
        ("linear, fused projection", _linear(4608, 4608, 12288, act="gelu_tanh", act_begin=4608)),
        # a decoding batch over many small experts: most experts get a row or two, some none
        ("experts, decoding", _experts(32, 4, 64, 2048, 1408, act="silu")),
        # a long ragged prompt over many experts, in a buffer with unused rows at its end
        ("experts, prompt", _experts(3001, 6, 64, 2048, 1408, act="silu", pad=58)),
        # a decoding batch's choice of experts
        ("sort, decoding", _sort(32, 4, 64)),
        # a padded batch of prompts
        ("sort, prompt", _sort(16384, 6, 64, dropped=0.05)),
        # the tokens of a decoding batch, in the experts' order
        ("dispatch, decoding", _dispatch(32, 4, 2048, weight=False)),
        # an image's tokens, weighted on their way in
        ("dispatch, image", _dispatch(4096, 6, 2048)),
        # a step over a few tokens in 32 bits, one of them padding, in a width that no vector divides
        ("grad, few tokens", _grad(7, 2, 1153, dropped=0.15, out="f32")),
        # the same for a whole image, six experts a token
        ("grad, image", _grad(4096, 6, 2048)),
    ]
    return [dict(c, name=name) for name, c in named]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "experts", "experts", "sort", "dispatch", "grad"])
    act = rng.choice(ACTS)
    out = rng.choice(["bf16", "f32"])
    dropped = rng.choice([0.0, 0.0, 0.1])
    if op == "sort":
        experts = _log_int(rng, 2, 256)
        return _sort(_log_int(rng, 1, 16384), rng.randint(1, min(experts, 6)), experts, dropped)
    if op in ("dispatch", "grad"):
        make = _dispatch if op == "dispatch" else _grad
        return make(_log_int(rng, 1, 4096), rng.randint(1, 6), _log_int(rng, 64, 2048), rng.random() < 0.7, dropped,
                    out)
    m = _log_int(rng, 200, 9216)
    n = _log_int(rng, 200, 9216)
    if rng.random() < 0.6:  # most layers' widths are whole vectors
        m, n = 64 * -(-m // 64), 64 * -(-n // 64)
    act_begin = rng.choice([0, 0, n // 3])
    bias = rng.random() < 0.7
    if op == "linear":
        b = min(_log_int(rng, 1, 4608), max(1, 4608 * 4608 * 12288 // (m * n)))
        return _linear(b, m, n, act, act_begin, rng.choice([0, 0, b, (b + 1) // 2]), rng.random() < 0.5, bias, out)
    experts = _log_int(rng, 2, 64)
    n = min(n, max(200, 64 * 2048 * 1408 // (experts * m)))  # the experts' weights stay within the listed ones' size
    topk = rng.randint(1, min(experts, 6))
    tokens = _log_int(rng, 1, max(1, min(3001, 3001 * 6 * 2048 * 1408 // (m * n * topk))))
    return _experts(tokens, topk, experts, m, n, act, min(act_begin, n), bias, rng.choice([0, 0, 17]), out)


def _layer_bytes(m, n, bias):
    return n * m + -(-n // BLOCK) * -(-m // BLOCK) + (2 * n if bias else 0)


def work(case):
    op = case["op"]
    if op == "sort":
        b = case["tokens"] * case["topk"]
        return {"bytes": 12 * b + 4 * (case["experts"] + 1), "flops": b}
    width = 2 if case["out"] == "bf16" else 4
    n = case["n"]
    if op in ("dispatch", "grad"):
        t, b = case["tokens"], case["tokens"] * case["topk"]
        scalars = 4 * b + (4 * b if case["weight"] else 0)
        if op == "dispatch":
            return {"bytes": (t + b) * n * width + scalars, "flops": b * n}
        return {"bytes": (t + 2 * b) * n * width + scalars + 4 * b, "flops": 3 * b * n}
    m = case["m"]
    if op == "linear":
        b = case["b"]
        size = 2 * b * m + _layer_bytes(m, n, case["bias"]) + b * n * width
        if case["gate"]:
            size += 2 * n * -(-b // case["gate"])
        if case["residual"]:
            size += b * n * width
        return {"bytes": size, "flops": 2 * b * n * m}
    t, k, e = case["tokens"], case["topk"], case["experts"]
    b = t * k
    used = e * (1 - (1 - k / e) ** t)  # experts that have a row, were the choice uniform
    return {"bytes": int(used * _layer_bytes(m, n, case["bias"]) + 2 * t * m + 4 * b + 4 * (e + 1) + b * n * width),
            "flops": 2 * b * m * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _weight(gen, m, n, bias, dev):
    """A layer's weight as a checkpoint holds it, bf16 [n][m]: Gaussian, with some stronger columns; and its bias."""
    w = torch.randn(n, m, generator=gen, device=dev) / math.sqrt(m)
    w *= torch.exp(0.3 * torch.randn(n, 1, generator=gen, device=dev))
    v = (0.2 * torch.randn(n, generator=gen, device=dev)).bfloat16() if bias else None
    return w.bfloat16(), v


def _choice(gen, tokens, topk, experts, dropped, dev):
    """A router's choice, int32 [tokens][topk]: some experts preferred; -1 in the slots of padding tokens."""
    logits = torch.randn(tokens, experts, generator=gen, device=dev)
    logits += 0.7 * torch.randn(experts, generator=gen, device=dev)
    ids = logits.topk(topk, -1).indices
    pad = torch.rand(tokens, 1, generator=gen, device=dev) < dropped
    return torch.where(pad, -1, ids).to(torch.int32)


def _sorted(ids, experts):
    """Slots in the order of their experts, those without one last: offsets [experts + 1], each row's token, each slot's
    row r (-1 - r where the slot names no expert)."""
    valid = (ids >= 0) & (ids < experts)
    keys, order = torch.sort(torch.where(valid, ids, experts).reshape(-1), stable=True)
    offsets = torch.searchsorted(keys, torch.arange(experts + 1, device=ids.device, dtype=ids.dtype))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    place = place.reshape(ids.shape)
    index = torch.where(valid, place, -1 - place)
    return offsets.to(torch.int32), (order // ids.shape[1]).to(torch.int32), index.to(torch.int32)


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "sort":
        s["ids"] = _choice(gen, case["tokens"], case["topk"], case["experts"], case["dropped"], dev)
        return s
    out = s["out"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    n = case["n"]
    if op in ("dispatch", "grad"):
        t, k = case["tokens"], case["topk"]
        s["x"] = torch.randn(t, n, generator=gen, device=dev).to(out)  # the tokens, or the gradient at the tokens
        s["index"] = _sorted(_choice(gen, t, k, max(16, k), case["dropped"], dev), max(16, k))[2]
        s["weight"] = torch.softmax(torch.randn(t, k, generator=gen, device=dev), -1) if case["weight"] else None
        if op == "grad":
            s["rows"] = torch.randn(t * k, n, generator=gen, device=dev).to(out)
        return s
    m = case["m"]
    if op == "linear":
        b = case["b"]
        s["w"], s["bias"] = _weight(gen, m, n, case["bias"], dev)
        s["gate"] = None
        if case["gate"]:
            s["gate"] = (0.5 * torch.randn(-(-b // case["gate"]), n, generator=gen, device=dev)).bfloat16()
        s["residual"] = torch.randn(b, n, generator=gen, device=dev).to(out) if case["residual"] else None
        rows = b
    else:
        t, k, e = case["tokens"], case["topk"], case["experts"]
        rows, b = t, t * k + case["pad"]
        layers = [_weight(gen, m, n, case["bias"], dev) for _ in range(e)]
        s["w"] = torch.stack([w for w, _ in layers])
        s["bias"] = torch.stack([v for _, v in layers]) if case["bias"] else None
        del layers
        ids = _choice(gen, t, k, e, 0.0, dev)
        s["offsets"], order, _ = _sorted(ids, e)
        s["row_index"] = torch.zeros(b, dtype=torch.int32, device=dev)
        s["row_index"][: t * k] = order
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # for the plain form's padded products
    x = torch.randn(rows, m, generator=gen, device=dev) * torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=dev))
    x[:, torch.randperm(m, generator=gen, device=dev)[: max(1, m // 100)]] *= 20.0  # an activation's strong channels
    s["x"] = x.bfloat16()
    s["y"] = torch.zeros(b, n, dtype=out, device=dev)  # rows behind the last expert's stay as they are
    return s


def _exponents(a):
    """The least e with a <= 448 2^e (448: the largest E4M3 value), at least -126."""
    f, k = torch.frexp(a)  # a = f 2^k, 1/2 <= f < 1
    e = torch.where(f <= 0.875, k - 9, k - 8)
    return torch.where(a > 0, e, -126).clamp(-126, 127)


def _power(e):
    """2^e in 32 bits, -126 <= e <= 127, by its bits (a power function may round)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantized(v, by):
    """E4M3 codes of rows [..., R, m] and the exponents of their blocks of `by` rows x 128 channels."""
    R, m = v.shape[-2:]
    p = torch.nn.functional.pad(v, (0, -m % BLOCK, 0, -R % by)).float().unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, by))
    e = _exponents(p.abs().amax((-3, -1), keepdim=True))  # [..., R / by, 1, m / 128, 1]
    q = (p * _power(-e)).to(torch.float8_e4m3fn)
    return q.flatten(-4, -3).flatten(-2)[..., :R, :m].contiguous(), e.squeeze(-1).squeeze(-2)


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    dev = next(v for v in s.values() if torch.is_tensor(v)).device
    if op == "sort":
        t, k, e = case["tokens"], case["topk"], case["experts"]
        if own:
            import w4a4_rank_corrected_amd as S
            s["offsets"] = torch.empty(e + 1, dtype=torch.int32, device=dev)
            s["row_index"] = torch.empty(t * k, dtype=torch.int32, device=dev)
            s["index"] = torch.empty(t, k, dtype=torch.int32, device=dev)
            s["workspace"] = torch.empty(max(S.svdq_sort_rows_workspace_size(t, k, e), 1), dtype=torch.uint8, device=dev)
        return s
    if op in ("dispatch", "grad"):
        if own:
            s["drows"] = torch.empty(case["tokens"] * case["topk"], case["n"], dtype=s["out"], device=dev)
            s["dweight"] = torch.empty(case["tokens"], case["topk"], device=dev)
        return s
    m, n = case["m"], case["n"]
    w = s.pop("w")
    if not own:
        s["qw"], s["ew"] = _quantized(w, BLOCK)
        return s
    import w4a4_rank_corrected_amd as S
    if op == "linear":
        s["layer"] = S.DeviceLayerFp8(w, s["bias"], transposed=True)
        size = S.svdq_fp8_linear_workspace_size(case["b"], m, n)
    else:
        s["layer"] = S.GroupedDeviceLayerFp8(w, s["bias"], transposed=True)
        size = S.svdq_fp8_grouped_linear_workspace_size(s["row_index"].numel(), s["x"].shape[0], case["experts"], m, n)
    s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _act(v, act):
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "gelu_erf":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "relu":
        return torch.where(v < 0, 0.0, v)
    return v


def _epilogue(v, case):
    if case["act"] == "none":
        return v
    c = case["act_begin"]
    return torch.cat([v[..., :c], _act(v[..., c:], case["act"])], -1)


def _values(q, e, by):
    """What codes [..., R, m] and exponents [..., R / by, m / 128] stand for, 32 bits."""
    R, m = q.shape[-2:]
    e = e.repeat_interleave(by, -2)[..., :R, :].repeat_interleave(BLOCK, -1)[..., :m]
    return q.float() * _power(e)


def _plain_linear(s):
    case = s["case"]
    v = _values(*_quantized(s["x"], 1), 1) @ _values(s["qw"], s["ew"], BLOCK).t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _epilogue(v, case)
    if s["gate"] is not None:
        v = v * s["gate"].float().repeat_interleave(case["gate"], 0)[: case["b"]]
    if s["residual"] is not None:
        v = s["residual"].float() + v
    return v.to(s["out"])


def _plain_experts(s):
    case, e, n, cap = s["case"], s["case"]["experts"], s["case"]["n"], s["most"]
    off, b = s["offsets"].long(), s["row_index"].numel()
    slot = torch.arange(b, device=off.device)
    expert = torch.searchsorted(off[1:], slot, right=True).clamp(max=e - 1)
    live = slot < off[-1]
    x = _values(*_quantized(s["x"], 1), 1)[s["row_index"].long()]
    # rows in one padded block for each expert, one batched product over them
    at = torch.where(live, expert * cap + (slot - off[expert]), e * cap)
    p = torch.zeros(e * cap + 1, x.shape[1], device=x.device)
    p[at] = x
    w = _values(s["qw"], s["ew"], BLOCK)  # [e][n][m]
    v = torch.bmm(p[: e * cap].view(e, cap, -1), w.transpose(1, 2).contiguous())
    if s["bias"] is not None:
        v = v + s["bias"].float().unsqueeze(1)
    v = _epilogue(v, case).view(e * cap, n)[at.clamp(max=e * cap - 1)]
    return torch.where(live.unsqueeze(1), v.to(s["out"]), s["y"])


def _plain_dispatch(s):
    """Row index[t, q] is weight[t, q] x[t]; a dropped slot's row is zero."""
    index = s["index"].long()
    v = s["x"].float().unsqueeze(1)
    v = v * s["weight"].unsqueeze(-1) if s["weight"] is not None else v.expand(-1, index.shape[1], -1)
    v = torch.where((index >= 0).unsqueeze(-1), v, 0.0).to(s["out"])
    rows = torch.empty(index.numel(), v.shape[-1], dtype=v.dtype, device=v.device)
    rows[torch.where(index >= 0, index, -1 - index).reshape(-1)] = v.flatten(0, 1)
    return rows


def _plain_grad(s):
    index = s["index"].long()
    d = (s["x"].float().unsqueeze(1) * s["rows"][index.clamp(min=0)].float()).sum(-1)
    return _plain_dispatch(s), torch.where(index >= 0, d, 0.0)


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "sort":
            return _sorted(s["ids"], case["experts"])
        return {"linear": _plain_linear, "experts": _plain_experts, "dispatch": _plain_dispatch, "grad": _plain_grad}[op](s)
    import w4a4_rank_corrected_amd as S
    if op == "sort":
        return S.svdq_sort_rows(s["ids"], case["experts"], offsets=s["offsets"], row_index=s["row_index"],
                                index=s["index"], workspace=s["workspace"])
    if op == "dispatch":
        return S.svdq_dispatch_rows(s["x"], s["index"], s["weight"], rows=s["drows"])
    if op == "grad":
        return S.svdq_combine_rows_grad(s["x"], s["index"], s["weight"], s["rows"], drows=s["drows"], dweight=s["dweight"])
    if op == "experts":
        return S.svdq_fp8_grouped_linear(s["x"], s["offsets"], s["layer"], row_index=s["row_index"], act=case["act"],
                                         act_begin=case["act_begin"], out_dtype=s["out"], y=s["y"], workspace=s["workspace"])
    return S.svdq_fp8_linear(s["x"], s["layer"], act=case["act"], act_begin=case["act_begin"], gate=s["gate"],
                             gate_rows=case["gate"], residual=s["residual"], out_dtype=s["out"], y=s["y"],
                             workspace=s["workspace"])


# ---------------------------------------------------------------------------
# the same from the definition, in 64 bits
# ---------------------------------------------------------------------------

def _act64(v, act):
    if act == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "gelu_erf":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2))
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "relu":
        return v.clamp_min(0)
    return v


def _below64(a):
    """The largest power of two that is not above a > 0: its bits without those of the fraction."""
    return (a.contiguous().view(torch.int64) >> 52 << 52).view(torch.float64)


def _rounded64(v, by):
    """Rows [R][m] as the values of their codes: each block's scale the least power of two that brings its largest
    magnitude to 448 or less, the quotient rounded to E4M3 (four significant bits, steps of 2^-9 at the least, ties to
    even)."""
    v = v.double()
    R, m = v.shape
    for r0 in range(0, R, by if by > 1 else R):
        for c0 in range(0, m, BLOCK):
            t = v[r0: r0 + by if by > 1 else R, c0: c0 + BLOCK]
            a = t.abs().amax() if by > 1 else t.abs().amax(1, keepdim=True)
            scale = _below64(a.clamp_min(2.0 ** -140) / 448)
            scale = torch.where(a > 448 * scale, 2 * scale, scale).clamp_min(2.0 ** -126)
            z = t / scale
            step = _below64(z.abs().clamp_min(2.0 ** -6)) / 8
            t.copy_(torch.round(z / step) * step * scale)
    return v


def _tail64(v, case):
    if case["act"] != "none":
        v[:, case["act_begin"]:] = _act64(v[:, case["act_begin"]:], case["act"])
    return v


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "sort":
        return None  # whole numbers, compared as they are
    if op in ("dispatch", "grad"):
        t, k, n = case["tokens"], case["topk"], case["n"]
        rows = torch.zeros(t * k, n, dtype=torch.float64, device=s["x"].device)
        dw = torch.zeros(t, k, dtype=torch.float64, device=s["x"].device)
        for q in range(k):
            live = s["index"][:, q] >= 0
            at = s["index"][live, q].long()
            v = s["x"][live].double()
            rows[at] = v if s["weight"] is None else v * s["weight"][live, q: q + 1].double()
            if op == "grad":
                dw[live, q] = (v * s["rows"][at].double()).sum(-1)
        return rows if op == "dispatch" else (rows, dw)
    x = _rounded64(s["x"], 1)
    if op == "linear":
        v = x @ _rounded64(s["w"], BLOCK).t()
        if s["bias"] is not None:
            v += s["bias"].double()
        v = _tail64(v, case)
        if s["gate"] is not None:
            v *= s["gate"].double()[torch.arange(case["b"], device=v.device) // case["gate"]]
        return v if s["residual"] is None else v + s["residual"].double()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=x.device)
    off = s["offsets"].tolist()
    for e in range(case["experts"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        v = x[s["row_index"][lo:hi].long()] @ _rounded64(s["w"][e], BLOCK).t()
        if s["bias"] is not None:
            v += s["bias"][e].double()
        y[lo:hi] = _tail64(v, case)
    return y
