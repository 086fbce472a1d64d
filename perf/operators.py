"""The operators around the quantized product, as cases that can be timed and compared.

Three operators, each in a plain form (elementary torch operations, 32-bit arithmetic) and as the library's calls:

  product   quantized codes times a prepared layer, with bias, activation, gate and residual in the product's epilogue
            (the INT4, 8-bit and NVFP4 settings)
  experts   rows of tokens, sorted by expert, through one INT4 layer per expert: gather, smoothing, quantization, the
            product and the low-rank branch, bias and activation
  combine   each token's rows, read back from the experts' order, weighted and added to the residual

``own`` chooses between the two: the plain form where it is false, the library's calls where it is true.
"""
import math

import numpy as np
import torch

own = False

GROUP = 64
ACTS = ("none", "gelu_tanh", "gelu_erf", "silu", "relu")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _product(fmt, b, m, n, rank, act="none", act_begin=0, gate=0, residual=False, bias=True, out="bf16"):
    """gate: rows that share one gate row (0 = no gate)."""
    return {"op": "product", "fmt": fmt, "b": b, "m": m, "n": n, "rank": rank, "act": act, "act_begin": act_begin,
            "gate": gate, "residual": residual, "bias": bias, "out": out}


def _experts(tokens, topk, experts, m, n, rank, act="none", act_begin=0, bias=True, pad=0, out="bf16"):
    return {"op": "experts", "tokens": tokens, "topk": topk, "experts": experts, "m": m, "n": n, "rank": rank,
            "act": act, "act_begin": act_begin, "bias": bias, "pad": pad, "out": out}


def _combine(tokens, topk, n, residual=True, out="bf16"):
    return {"op": "combine", "tokens": tokens, "topk": topk, "n": n, "residual": residual, "out": out}


def listed():
    named = [
        # the second linear of a PixArt-shaped MLP for one row: latency of a single small layer, gated residual
        ("int4 one row", _product("int4", 1, 4608, 1152, 32, gate=1, residual=True)),
        # a few rows of a language model's step through an odd number of output columns, results kept in 32 bits
        ("int4 few rows, odd columns", _product("int4", 13, 2048, 5001, 16, act="silu", out="f32")),
        # PixArt-shaped MLP fc1 with its GELU (1024px latent, 4096 tokens)
        ("int4 fc1 + gelu", _product("int4", 4096, 1152, 4608, 32, act="gelu_tanh")),
        # FLUX-shaped single-block fused projection: QKV columns as they are, GELU on the MLP columns behind them
        ("int4 fused projection", _product("int4", 4608, 3072, 21504, 48, act="gelu_tanh", act_begin=9216)),
        # 8-bit fc2 of two images of 500 tokens, one gate each, residual stream in 32 bits
        ("w8a8 fc2, gate, residual", _product("w8a8", 1000, 4608, 1152, 16, gate=500, residual=True, out="f32")),
        # NVFP4 fc1 with the exact GELU, a 768px-like token count
        ("fp4 fc1 + gelu", _product("fp4", 2304, 1152, 4608, 32, act="gelu_erf")),
        # one token through two of sixteen experts
        ("experts, one token", _experts(1, 2, 16, 1152, 4608, 32, act="silu")),
        # a decoding batch over many small experts: most experts get a row or two, some none
        ("experts, decoding", _experts(32, 4, 64, 2048, 1408, 16, act="silu")),
        # a whole image's tokens through the first linear of eight PixArt-sized experts
        ("experts, image", _experts(4096, 2, 8, 1152, 4608, 32, act="gelu_tanh")),
        # a long ragged prompt over many experts, in a buffer with unused rows at its end
        ("experts, prompt", _experts(3001, 6, 64, 2048, 1408, 16, pad=58)),
        # the experts' rows of a few tokens, back in token order
        ("combine, few tokens", _combine(7, 2, 1152)),
        # the same for a whole image, six experts a token
        ("combine, image", _combine(4096, 6, 2048)),
    ]
    return [dict(c, name=name) for name, c in named]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "experts", "experts", "combine"])
    act = rng.choice(ACTS)
    out = rng.choice(["bf16", "f32"])
    if op == "combine":
        return _combine(_log_int(rng, 1, 4608), rng.randint(1, 8), _log_int(rng, 64, 4608), rng.random() < 0.5, out)
    m = GROUP * _log_int(rng, 4, 72)
    n = _log_int(rng, 256, 9216)
    rank = rng.choice([0, 8, 16, 24, 32, 48, 64, 100])
    act_begin = rng.choice([0, 0, n // 3])
    bias = rng.random() < 0.7
    if op == "product":
        b = _log_int(rng, 1, 4608)
        return _product(rng.choice(["int4", "int4", "w8a8", "fp4"]), b, m, n, rank, act, act_begin,
                        rng.choice([0, 0, b, (b + 1) // 2]), rng.random() < 0.5, bias, out)
    experts = _log_int(rng, 2, 64)
    n = min(n, max(256, 64 * 2048 * 1408 // (experts * m)))  # the experts' weights stay within the listed ones' size
    topk = rng.randint(1, min(experts, 6))
    # 16 bits out: the low-rank factor is rounded to bf16 inside the layer, and 32-bit outputs would show on which
    # side of a rounding border its own sums fall
    tokens = _log_int(rng, 1, min(3000, int(300e9 / (m * n * topk))))
    return _experts(tokens, topk, experts, m, n, rank, act, min(act_begin, n), bias,
                    rng.choice([0, 0, 17]))


def work(case):
    width = 2 if case["out"] == "bf16" else 4
    n = case["n"]
    if case["op"] == "combine":
        t, k = case["tokens"], case["topk"]
        per_row = k + 1 + (1 if case["residual"] else 0)
        return {"bytes": t * (per_row * n * width + 8 * k), "flops": 2 * t * k * n}
    m, r = case["m"], case["rank"]
    g = m // GROUP
    if case["op"] == "product":
        b, fmt = case["b"], case["fmt"]
        code = {"int4": m // 2, "w8a8": m, "fp4": m // 2}[fmt]
        scale = {"int4": 2 * g, "w8a8": 2, "fp4": 4 * g}[fmt]
        size = (b + n) * (code + scale) + 4 * b * r + 2 * n * r + (2 * n if case["bias"] else 0) + b * n * width
        if case["gate"]:
            size += 2 * n * -(-b // case["gate"])
        if case["residual"]:
            size += b * n * width
        return {"bytes": size, "flops": 2 * b * n * (m + r)}
    t, k, e = case["tokens"], case["topk"], case["experts"]
    b = t * k
    used = e * (1 - (1 - k / e) ** t)  # experts that have a row, were the choice uniform
    layer = n * (m // 2 + 2 * g + 2 * r + 2) + m * (4 + 2 * r)
    return {"bytes": int(used * layer + 2 * t * m + 4 * b + 4 * (e + 1) + b * n * width),
            "flops": 2 * b * (m + r) * n + 2 * b * m * r}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _records(codes):
    """4-bit codes [R][m] -> the group-major records [m/64][R][32], the even channel in each byte's low nibble."""
    R, m = codes.shape
    c = codes.to(torch.uint8) & 15
    c = c.reshape(R, m // GROUP, GROUP // 2, 2)
    return (c[..., 0] | (c[..., 1] << 4)).permute(1, 0, 2).contiguous()


def _int4(v):
    """Codes and fp16 scales of rows [R][m] in groups of 64: records [m/64][R][32], scales [m/64][R]."""
    R, m = v.shape
    g = v.reshape(R, m // GROUP, GROUP)
    s = (g.abs().amax(-1) / 7).half()
    q = torch.round(g / s.float().clamp_min(1e-20).unsqueeze(-1)).clamp(-7, 7)
    return _records(q.reshape(R, m).to(torch.int8)), s.t().contiguous()


def _int8(v):
    """Codes [m/64][R][64] and one fp16 scale per row [R]."""
    R, m = v.shape
    s = (v.abs().amax(-1) / 127).half()
    q = torch.round(v / s.float().clamp_min(1e-20).unsqueeze(-1)).clamp(-127, 127).to(torch.int8)
    return q.reshape(R, m // GROUP, GROUP).permute(1, 0, 2).contiguous(), s


def _fp4(v, t):
    """E2M1 records [m/64][R][32] and E4M3 scale bytes [m/64][R][4] for tensor scale t."""
    R, m = v.shape
    g = v.reshape(R, m // 16, 16)
    s8 = (g.abs().amax(-1) / 6 / t).clamp(max=448.0).to(torch.float8_e4m3fn)
    S = s8.float() * t
    q = (g / S.clamp_min(1e-20).unsqueeze(-1)).clamp(-6, 6)
    grid = torch.tensor(E2M1, device=v.device)
    borders = (grid[1:] + grid[:-1]) / 2
    code = torch.bucketize(q.abs(), borders) + torch.where(q < 0, 8, 0)
    scale = s8.view(torch.uint8).reshape(R, m // GROUP, 4).permute(1, 0, 2).contiguous()
    return _records(code.reshape(R, m).to(torch.int8)), scale


def _layer(gen, fmt, m, n, rank, bias, dev):
    """One quantized layer's tensors: a Gaussian residual with a few strong columns, a low-rank branch beside it."""
    w = torch.randn(n, m, generator=gen, device=dev) / math.sqrt(m)
    w *= torch.exp(0.3 * torch.randn(n, 1, generator=gen, device=dev))
    d = {"t_w": 2.0 ** -14}
    if fmt == "int4":
        d["qw"], d["wscale"] = _int4(w)
    elif fmt == "w8a8":
        d["qw"], d["wscale"] = _int8(w)
    else:
        d["qw"], d["wscale"] = _fp4(w, d["t_w"])
    d["l1"] = (torch.randn(rank, m, generator=gen, device=dev) / math.sqrt(m)).bfloat16() if rank else None
    d["l2"] = (0.5 * torch.randn(n, rank, generator=gen, device=dev) / math.sqrt(max(rank, 1))).bfloat16() if rank else None
    d["bias"] = (0.2 * torch.randn(n, generator=gen, device=dev)).bfloat16() if bias else None
    return d


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    out = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    s = {"case": case, "out": out}
    n = case["n"]
    if case["op"] == "combine":
        t, k = case["tokens"], case["topk"]
        s["rows"] = torch.randn(t * k, n, generator=gen, device=dev).to(out)
        place = torch.randperm(t * k, generator=gen, device=dev)  # where the experts' order put each token's rows
        s["index"] = place.reshape(t, k).to(torch.int32)
        s["weight"] = torch.softmax(torch.randn(t, k, generator=gen, device=dev), -1)
        s["residual"] = torch.randn(t, n, generator=gen, device=dev).to(out) if case["residual"] else None
        s["y"] = torch.zeros(t, n, dtype=out, device=dev)
        return s
    m, rank = case["m"], case["rank"]
    if case["op"] == "product":
        b, fmt = case["b"], case["fmt"]
        s.update(_layer(gen, fmt, m, n, rank, case["bias"], dev))
        x = torch.randn(b, m, generator=gen, device=dev)
        x[:, :: 97] *= 4.0  # what smoothing leaves of the strong channels
        s["t_x"] = 2.0 ** -8
        s["qx"], s["ascale"] = _int4(x) if fmt == "int4" else _int8(x) if fmt == "w8a8" else _fp4(x, s["t_x"])
        s["z"] = torch.randn(b, rank, generator=gen, device=dev) if rank else None
        s["gate"] = None
        if case["gate"]:
            rows = -(-b // case["gate"])
            s["gate"] = (0.5 * torch.randn(rows, n, generator=gen, device=dev)).bfloat16()
        s["residual"] = torch.randn(b, n, generator=gen, device=dev).to(out) if case["residual"] else None
        s["y"] = torch.zeros(b, n, dtype=out, device=dev)
        if own:
            import w4a4_rank_corrected_amd as S
            if fmt == "int4":
                s["layer"] = S.DeviceLayer.from_tensors(m, n, rank, s["qw"], s["wscale"], s["l1"], s["l2"], None, s["bias"])
                size = S.svdq_gemm_epi_workspace_size(b, n, m)
            elif fmt == "w8a8":
                s["layer"] = S.DeviceLayer8.from_tensors(m, n, rank, s["qw"], s["wscale"], s["l1"], s["l2"], None, s["bias"])
                size = S.svdq_w8a8_gemm_workspace_size(b, n, m)
            else:
                s["layer"] = S.DeviceLayerFp4.from_tensors(m, n, rank, s["t_x"], s["t_w"], s["qw"], s["wscale"], s["l1"],
                                                           s["l2"], None, s["bias"])
                size = S.svdq_fp4_gemm_workspace_size(b, n, m)
            s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
        return s
    # experts
    t, k, e = case["tokens"], case["topk"], case["experts"]
    b = t * k + case["pad"]
    layers = [_layer(gen, "int4", m, n, rank, case["bias"], dev) for _ in range(e)]
    for key in ("qw", "wscale", "l1", "l2", "bias"):
        s[key] = None if layers[0][key] is None else torch.stack([d[key] for d in layers])
    del layers
    s["x"] = torch.randn(t, m, generator=gen, device=dev)
    strong = torch.randperm(m, generator=gen, device=dev)[: max(1, m // 100)]
    s["x"][:, strong] *= 20.0
    s["x"] = s["x"].bfloat16()
    s["smooth_inv"] = torch.exp(0.2 * torch.randn(e, m, generator=gen, device=dev))
    s["smooth_inv"][:, strong] /= 8.0
    # a router with a preference for some experts; each token goes to its topk
    logits = torch.randn(t, e, generator=gen, device=dev) + 0.7 * torch.randn(e, generator=gen, device=dev)
    chosen = logits.topk(k, -1).indices.reshape(-1)
    order = torch.sort(chosen, stable=True).indices
    count = torch.bincount(chosen, minlength=e)
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), count.cumsum(0)]).to(torch.int32)
    s["row_index"] = torch.zeros(b, dtype=torch.int32, device=dev)
    s["row_index"][: t * k] = (order // k).to(torch.int32)
    s["most"] = int(count.max())  # the rows of the fullest expert, for the plain form's padded products
    s["y"] = torch.zeros(b, n, dtype=out, device=dev)  # rows behind the last expert's stay as they are
    if own:
        import w4a4_rank_corrected_amd as S
        s["layer"] = S.GroupedDeviceLayer.from_tensors(e, m, n, rank, s["qw"], s["wscale"], s["l1"], s["l2"], s["smooth_inv"],
                                                       s["bias"])
        size = S.svdq_grouped_linear_workspace_size(b, e, m, n, rank)
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


def _unpacked(records):
    """Records [..., m/64, R, 32] -> 4-bit patterns [..., R, m]."""
    c = torch.stack([records & 15, records >> 4], -1).flatten(-2)  # [..., m/64, R, 64]
    return c.transpose(-3, -2).flatten(-2)


def _plain_values(fmt, q, scale, t):
    """The values that codes and scales stand for, 32 bits, [R][m]."""
    if fmt == "w8a8":
        return q.transpose(0, 1).flatten(1).float() * scale.float().unsqueeze(1)
    c = _unpacked(q)
    if fmt == "int4":
        v = ((c ^ 8).to(torch.int8) - 8).float()
        return (v.unflatten(1, (-1, GROUP)) * scale.float().t().unsqueeze(-1)).flatten(1)
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    s = scale.view(torch.float8_e4m3fn).float().transpose(0, 1).flatten(1) * t  # [R][m/16]
    return (grid[c.int()].unflatten(1, (-1, 16)) * s.unsqueeze(-1)).flatten(1)


def _plain_product(s):
    case = s["case"]
    x = _plain_values(case["fmt"], s["qx"], s["ascale"], s["t_x"])
    w = _plain_values(case["fmt"], s["qw"], s["wscale"], s["t_w"])
    v = x @ w.t()
    if case["rank"]:
        v = v + s["z"].bfloat16().float() @ s["l2"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _epilogue(v, case)
    if s["gate"] is not None:
        v = v * s["gate"].float().repeat_interleave(case["gate"], 0)[: case["b"]]
    if s["residual"] is not None:
        v = s["residual"].float() + v
    return v.to(s["out"])


def _plain_experts(s):
    case, e, m, n, cap = s["case"], s["case"]["experts"], s["case"]["m"], s["case"]["n"], s["most"]
    off, b = s["offsets"].long(), s["row_index"].numel()
    slot = torch.arange(b, device=off.device)
    expert = torch.searchsorted(off[1:], slot, right=True).clamp(max=e - 1)
    live = slot < off[-1]
    # smoothing and the 4-bit codes of each row
    x = (s["x"][s["row_index"].long()].float() * s["smooth_inv"][expert]).bfloat16().float()
    g = x.unflatten(1, (-1, GROUP))
    a = (g.abs().amax(-1, keepdim=True) / 7).clamp(max=65504.0).half().float()
    q = torch.where(a > 0, torch.round(g / a), 0.0).clamp(-7, 7) * a
    # rows in one padded block for each expert, one batched product over them
    at = torch.where(live, expert * cap + (slot - off[expert]), e * cap)

    def padded(rows):
        p = torch.zeros(e * cap + 1, rows.shape[1], device=rows.device)
        p[at] = rows
        return p[: e * cap].view(e, cap, -1)

    w = ((_unpacked(s["qw"]) ^ 8).to(torch.int8) - 8).float()  # [e][n][m]
    w = (w.unflatten(2, (-1, GROUP)) * s["wscale"].float().transpose(1, 2).unsqueeze(-1)).flatten(2)
    v = torch.bmm(padded(q.flatten(1)), w.transpose(1, 2).contiguous())
    if case["rank"]:
        z = torch.bmm(padded(x), s["l1"].float().transpose(1, 2).contiguous())
        v = v + torch.bmm(z.bfloat16().float(), s["l2"].float().transpose(1, 2).contiguous())
    if s["bias"] is not None:
        v = v + s["bias"].float().unsqueeze(1)
    v = _epilogue(v, case).view(e * cap, n)
    v = v[at.clamp(max=e * cap - 1)]
    return torch.where(live.unsqueeze(1), v.to(s["out"]), s["y"])


def _plain_combine(s):
    v = (s["rows"][s["index"].long()].float() * s["weight"].unsqueeze(-1)).sum(1)
    if s["residual"] is not None:
        v = s["residual"].float() + v
    return v.to(s["out"])


def run(s):
    case = s["case"]
    if not own:
        return {"product": _plain_product, "experts": _plain_experts, "combine": _plain_combine}[case["op"]](s)
    import w4a4_rank_corrected_amd as S
    if case["op"] == "combine":
        return S.svdq_combine_rows(s["rows"], s["index"], s["weight"], residual=s["residual"], y=s["y"], out_dtype=s["out"])
    if case["op"] == "experts":
        return S.svdq_grouped_linear(s["x"], s["offsets"], s["layer"], row_index=s["row_index"], act=case["act"],
                                     act_begin=case["act_begin"], out_dtype=s["out"], y=s["y"], workspace=s["workspace"])
    call = {"int4": S.svdq_gemm_w4a4_lowrank_up_epi, "w8a8": S.svdq_w8a8_gemm_lowrank_up_epi,
            "fp4": S.svdq_fp4_gemm_lowrank_up_epi}[case["fmt"]]
    return call(s["qx"], s["ascale"], s["z"], s["layer"], act=case["act"], act_begin=case["act_begin"], gate=s["gate"],
                gate_rows=case["gate"], residual=s["residual"], out_dtype=s["out"], y=s["y"], workspace=s["workspace"])


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


def _nibbles64(records, table):
    """Group-major records [G][R][32] -> table values [R][64 G]."""
    G, R, _ = records.shape
    v = torch.empty(R, G, GROUP, dtype=torch.float64, device=records.device)
    v[:, :, 0::2] = table[(records % 16).long()].transpose(0, 1)
    v[:, :, 1::2] = table[(records // 16).long()].transpose(0, 1)
    return v


def _values64(fmt, q, scale, t):
    dev = q.device
    if fmt == "w8a8":
        G, R, _ = q.shape
        return q.double().permute(1, 0, 2).reshape(R, G * GROUP) * scale.double()[:, None]
    if fmt == "int4":
        table = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device=dev)
        v = _nibbles64(q, table) * scale.double().t()[:, :, None]
        return v.reshape(v.shape[0], -1)
    table = torch.tensor(np.concatenate([np.array(E2M1), -np.array(E2M1)]), dtype=torch.float64, device=dev)
    byte = np.arange(256)
    ex, man = (byte >> 3) & 15, byte & 7
    e4m3 = np.where(ex > 0, (1 + man / 8) * 2.0 ** (ex - 7.0), man / 8 * 2.0 ** -6)
    block = torch.tensor(e4m3, device=dev)[scale.long()] * t  # [G][R][4]
    v = _nibbles64(q, table)
    v = v.reshape(v.shape[0], v.shape[1], 4, 16) * block.transpose(0, 1)[..., None]
    return v.reshape(v.shape[0], -1)


def _tail64(v, case):
    if case["act"] != "none":
        v[:, case["act_begin"]:] = _act64(v[:, case["act_begin"]:], case["act"])
    return v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "combine":
        y = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device=s["rows"].device)
        for k in range(case["topk"]):
            y += s["rows"][s["index"][:, k].long()].double() * s["weight"][:, k: k + 1].double()
        return y if s["residual"] is None else y + s["residual"].double()
    if case["op"] == "product":
        v = _values64(case["fmt"], s["qx"], s["ascale"], s["t_x"]) @ _values64(case["fmt"], s["qw"], s["wscale"], s["t_w"]).t()
        if case["rank"]:
            v += s["z"].bfloat16().double() @ s["l2"].double().t()
        if s["bias"] is not None:
            v += s["bias"].double()
        v = _tail64(v, case)
        if s["gate"] is not None:
            row = torch.arange(case["b"], device=v.device) // case["gate"]
            v *= s["gate"].double()[row]
        return v if s["residual"] is None else v + s["residual"].double()
    y = torch.zeros(s["row_index"].numel(), case["n"], dtype=torch.float64, device=s["x"].device)
    off = s["offsets"].tolist()
    for e in range(case["experts"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        # the layer's own roundings: smoothed rows to bf16, scales to fp16, codes to whole numbers, Z to bf16
        x = s["x"][s["row_index"][lo:hi].long()].double() * s["smooth_inv"][e].double()
        x = x.float().bfloat16().double().reshape(hi - lo, -1, GROUP)
        a = (x.abs().amax(-1, keepdim=True) / 7).float().half().double()
        q = torch.round((x / torch.where(a > 0, a, 1.0)).float().double()).clamp(-7, 7) * a
        v = q.reshape(hi - lo, -1) @ _values64("int4", s["qw"][e], s["wscale"][e], 1.0).t()
        if case["rank"]:
            z = x.reshape(hi - lo, -1) @ s["l1"][e].double().t()
            v += z.bfloat16().double() @ s["l2"][e].double().t()
        if s["bias"] is not None:
            v += s["bias"][e].double()
        y[lo:hi] = _tail64(v, case)
    return y
