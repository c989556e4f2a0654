"""Workloads of the operators around the experts: what each takes, its plain form and the library's calls.

* ``quant``   -- activations (or SiLU(gate)*up of a gate/up projection) to OCP e4m3 codes with one fp32 scale
  per 128 values, along the row and, for the backward products, along the column.
* ``matmul``  -- out = A . B^T of two such operands; B's scales are per 128 x 128 block (weights) or per
  row and 128 values (the weight gradient's operand).
* ``grouped`` -- the same product for every expert of an MoE layer over its routed rows.
* ``balance`` -- the router's balance loss with per-expert counts, and its gradient.
* ``norm``    -- RMS norms before and after a block with the block's gate and the residual scale: the norm
  that makes the block's (quantized) input, the norm that ends it, and their gradients.
"""
import math

import torch

own = False

DEV = "cuda"
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def listed():
    return [
        # The middle of an fp8 expert FFN at 2048 tokens, top-8: every routed row's gate/up pair becomes the
        # down projection's input.
        {"name": "quant_act_16384x768", "op": "quant", "M": 16384, "K": 768, "act": True, "cols": False, "dtype": "bf16"},
        # A training step's gradient of a projection over a ragged token count: codes along the row for the
        # input gradient and along the column for the weight gradient, in one pass over the fp32 gradient.
        {"name": "quant_train_4111x2048", "op": "quant", "M": 4111, "K": 2048, "act": False, "cols": True, "dtype": "f32"},
        # One token through a 2048-wide projection: latency.
        {"name": "matmul_1tok_2048", "op": "matmul", "M": 1, "N": 2048, "K": 2048, "b_block": True, "dtype": "bf16"},
        # A prefill's projection at hidden 4096: the matrix cores.
        {"name": "matmul_4096", "op": "matmul", "M": 4096, "N": 4096, "K": 4096, "b_block": True, "dtype": "bf16"},
        # The gradient of a 2048 -> 1500 projection's weights over 4224 (padded) tokens, both operands scaled
        # per row, in fp32.
        {"name": "matmul_wgrad_1500x2048", "op": "matmul", "M": 1500, "N": 2048, "K": 4224, "b_block": False, "dtype": "f32"},
        # Gate/up projection of the 128-expert top-8 block: a decode step of four tokens, bound by the weights.
        {"name": "grouped_4tok_e128", "op": "grouped", "T": 4, "E": 128, "k": 8, "N": 1536, "K": 2048},
        # The same block at a 2048-token prefill.
        {"name": "grouped_2048tok_e128", "op": "grouped", "T": 2048, "E": 128, "k": 8, "N": 1536, "K": 2048},
        # The tiny block's router, one small training step.
        {"name": "balance_64_e8", "op": "balance", "T": 64, "E": 8, "k": 2, "masked": False, "coef": 0.01},
        # The 512-expert top-10 router over a padded batch of 8192 tokens with a skewed router.
        {"name": "balance_8192_e512", "op": "balance", "T": 8192, "E": 512, "k": 10, "masked": True, "coef": 0.001},
        # The layer's input for one decoded token: norm and e4m3 codes with the token's scale.
        {"name": "norm_pre_1tok_4096", "op": "norm", "what": "pre", "T": 1, "H": 4096, "out": "e4m3", "dtype": "bf16"},
        # Between two blocks of a prefill: the gated norm of the block's output, the residual and the next
        # block's quantized input.
        {"name": "norm_post_next_4096x4096", "op": "norm", "what": "post_next", "T": 4096, "H": 4096, "out": "e4m3_128", "gate": "h",
         "dtype": "bf16", "alpha": 1.0},
        # The gradient of the norm after a block over a ragged token count, with a gate per token and column.
        {"name": "norm_post_bwd_4111x2048", "op": "norm", "what": "post_bwd", "T": 4111, "H": 2048, "gate": "th", "dtype": "bf16",
         "alpha": 0.5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quant", "matmul", "matmul", "grouped", "grouped", "balance", "norm", "norm"])
    if op == "quant":
        act = rng.random() < 0.5
        return {"op": op, "M": _log(rng, 1, 16384), "K": _log(rng, 64, 2048), "act": act, "cols": not act or rng.random() < 0.3,
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "matmul":
        b_block = rng.random() < 0.7
        M, N, K = _log(rng, 1 if b_block else 64, 8192), _log(rng, 16, 8192), 128 * _log(rng, 1, 48)
        while M * N * K > 4096 ** 3:
            M, N = max(1, M // 2), max(1, N - N // 4)
        return {"op": op, "M": M, "N": N, "K": K, "b_block": b_block, "dtype": "bf16" if b_block and rng.random() < 0.8 else "f32"}
    if op == "grouped":
        E = rng.choice([8, 16, 60, 128])
        return {"op": op, "T": _log(rng, 1, 2048), "E": E, "k": rng.randint(1, 8), "N": _log(rng, 64, 1600), "K": 128 * rng.randint(1, 16)}
    if op == "balance":
        E = _log(rng, 4, 512)
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(E, 10)), "masked": rng.random() < 0.5,
                "coef": rng.choice([0.001, 0.01, 1.0])}
    what = rng.choice(["pre", "pre_bwd", "post", "post_next", "post_bwd"])
    c = {"op": op, "what": what, "T": _log(rng, 1, 4200), "H": rng.choice([_log(rng, 32, 4096), 8 * _log(rng, 8, 512)]),
         "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if what in ("pre", "post_next"):
        c["out"] = rng.choice(["bf16", "f32", "e4m3", "e4m3_128"])
    if what.startswith("post"):
        c["gate"], c["alpha"] = rng.choice(["none", "h", "t", "th"]), rng.choice([1.0, 0.5, 0.25])
    return c


def _dt(name):
    return BF if name == "bf16" else F32


def _up(v, m):
    return (v + m - 1) // m * m


def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(int(seed))
    return g


def _scale_of(amax):
    # One fp32 scale per group: absmax / 448, the smallest normal number at least, 1 for a group of zeros.
    return torch.where(amax > 0, (amax / 448.0).clamp_min(2.0 ** -126), torch.ones_like(amax))


def _codes(v, s):
    return (v / s).clamp(-448.0, 448.0).to(F8)


def _rows128(v):
    """fp32 [M, K] -> codes [M, Kp], scales [Kp/128, M], Kp the next multiple of 128 (zeros behind K)."""
    M, K = v.shape
    Kp = _up(K, 128)
    if Kp != K:
        v = torch.nn.functional.pad(v, (0, Kp - K))
    v = v.view(M, Kp // 128, 128)
    s = _scale_of(v.abs().amax(2))
    return _codes(v, s[:, :, None]).view(M, Kp), s.t().contiguous()


def _blocks128(w):
    """fp32 [B, N, K] (K a multiple of 128) -> codes, scales [B, ceil(N/128), K/128]."""
    B, N, K = w.shape
    Np = _up(N, 128)
    v = torch.nn.functional.pad(w, (0, 0, 0, Np - N)).view(B, Np // 128, 128, K // 128, 128)
    s = _scale_of(v.abs().amax((2, 4)))
    return _codes(v, s[:, :, None, :, None]).reshape(B, Np, K)[:, :N].contiguous(), s


def _activations(g, M, K):
    # Hidden states: normal values with a few channels far above the rest and rows of different sizes.
    x = torch.randn(M, K, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(M, 1, generator=g, device=DEV))
    return x * torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 12.0, 1.0)


def prepare(case, seed):
    g = _gen(seed)
    c = case
    if c["op"] == "quant":
        return {"c": c, "x": _activations(g, c["M"], c["K"] * (2 if c["act"] else 1)).to(_dt(c["dtype"]))}
    if c["op"] == "matmul":
        a, a_s = _rows128(_activations(g, c["M"], c["K"]))
        w = torch.randn(1, c["N"], c["K"], generator=g, device=DEV) * c["K"] ** -0.5
        if c["b_block"]:
            b, b_s = _blocks128(w)
            b, b_s = b[0], b_s[0]
        else:
            b, b_s = _rows128(w[0])
        return {"c": c, "a": a, "a_s": a_s, "b": b, "b_s": b_s, "ws": _matmul_ws(c)}
    if c["op"] == "grouped":
        T, E, k = c["T"], c["E"], c["k"]
        a, a_s = _rows128(_activations(g, T, c["K"]))
        b = torch.empty(E, c["N"], c["K"], dtype=F8, device=DEV)
        b_s = torch.empty(E, _up(c["N"], 128) // 128, c["K"] // 128, device=DEV)
        for e in range(0, E, 16):
            n = min(16, E - e)
            b[e:e + n], b_s[e:e + n] = _blocks128(torch.randn(n, c["N"], c["K"], generator=g, device=DEV) * c["K"] ** -0.5)
        ids = torch.randn(T, E, generator=g, device=DEV).topk(k, 1).indices.to(torch.int32)
        return {"c": c, "a": a, "a_s": a_s, "b": b, "b_s": b_s, "ids": ids, **_grouping(ids, E)}
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        z = torch.randn(T, E, generator=g, device=DEV) - 1.2 * torch.log(torch.arange(1, E + 1, device=DEV).float())
        mask = None
        if c["masked"]:  # a padded batch: rows of it behind each sequence's end
            mask = (torch.rand(T, generator=g, device=DEV) < 0.85).to(torch.uint8)
        return {"c": c, "z": z, "ids": z.topk(k, 1).indices.to(torch.int32), "mask": mask, "dloss": torch.rand(1, generator=g, device=DEV) + 0.5}
    T, H, dt = c["T"], c["H"], _dt(c["dtype"])
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = {"c": c, "x": _activations(g, T, H).to(dt), "w": 1 + 0.2 * rand(H)}
    if c["what"] == "pre_bwd":
        s |= {"dn": rand(T, H).to(dt), "dres": rand(T, H).to(dt)}
    if c["what"].startswith("post"):
        s["y"] = (0.3 * rand(T, H) * torch.exp(0.5 * rand(T, 1))).to(dt)
        s["gate"] = {"none": lambda: None, "h": lambda: 0.5 + 0.3 * rand(H), "t": lambda: torch.sigmoid(rand(T, 1)),
                     "th": lambda: torch.sigmoid(rand(T, H)).to(dt)}[c["gate"]]()
        if c["what"] == "post_next":
            s["w2"] = 1 + 0.2 * rand(H)
        if c["what"] == "post_bwd":
            s["dout"] = rand(T, H).to(dt)
    return s


def _matmul_ws(c):
    # The scratch buffer that a program keeps for the product's split sums (sized for the largest split).
    return torch.empty(32 << 20, dtype=torch.uint8, device=DEV)


def _grouping(ids, E):
    """The expert-sorted, tile-padded pair slots of a routing, as the layer's grouping step hands them on."""
    T, k = ids.shape
    P = T * k
    mean = P / E
    bm = 16 if mean <= 16 else 32 if mean <= 32 else 64 if mean <= 64 else 128
    cap = _up(max(P + min(E, P) * (bm - 1), 1), bm)
    flat = ids.reshape(-1).long()
    cnt = torch.bincount(flat, minlength=E)
    padded = (cnt + bm - 1) // bm * bm
    end = torch.cumsum(padded, 0)
    order = torch.sort(flat, stable=True).indices
    e_of = flat[order]
    rank = torch.arange(P, device=DEV) - (torch.cumsum(cnt, 0) - cnt)[e_of]
    sorted_ids = torch.full((cap,), P, dtype=torch.int32, device=DEV)
    sorted_ids[(end - padded)[e_of] + rank] = order.to(torch.int32)
    tiles = torch.arange(cap // bm, device=DEV) * bm
    tile_expert = torch.searchsorted(end, tiles, right=True).to(torch.int32)
    tile_expert[tiles >= end[-1]] = -1
    al = {"sorted_pair_ids": sorted_ids, "tile_expert": tile_expert, "num_padded": end[-1:].to(torch.int32), "block_m": bm,
          "expert_offsets": torch.cat([end.new_zeros(1), end]).to(torch.int32)}
    place = torch.empty(P, dtype=torch.long, device=DEV)
    place[order] = rank
    return {"al": al, "rank": place, "most": int(cnt.max())}


# ---------------------------------------------------------------- one pass

def run(state):
    return {"quant": _quant, "matmul": _matmul, "grouped": _grouped, "balance": _balance, "norm": _norm}[state["c"]["op"]](state)


def _f8(t):
    return t.view(F8)


def _ops():
    from quantized_mixture_experts_moe_amd import ops
    return ops


def _quant(s):
    c, x = s["c"], s["x"]
    if own:
        r = _ops().fp8_quant(x, act="silu_mul" if c["act"] else None, cols=c["cols"])
        out = {"codes": _f8(r["codes"]), "scale": r["scale"]}
        return out | {"codes_t": _f8(r["codes_t"]), "scale_t": r["scale_t"]} if c["cols"] else out
    v = x.float()
    if c["act"]:
        gate, up = v.chunk(2, 1)
        v = gate / (1 + torch.exp(-gate)) * up
    codes, scale = _rows128(v)
    if not c["cols"]:
        return {"codes": codes, "scale": scale}
    codes_t, scale_t = _rows128(v.t().contiguous())
    return {"codes": codes, "scale": scale, "codes_t": codes_t, "scale_t": scale_t}


def _wide(codes, scale, b_block=False):
    """The values that [M, K] codes with scales stand for, in the scales' width."""
    M, K = codes.shape
    if b_block:
        s = scale.repeat_interleave(128, 0)[:M]
    else:
        s = scale.t()
    return (codes.to(scale.dtype).view(M, K // 128, 128) * s[:, :, None]).view(M, K)


def _matmul(s):
    c = s["c"]
    if own:
        return _ops().fp8_matmul(s["a"].view(torch.uint8), s["a_s"], s["b"].view(torch.uint8), s["b_s"], b_block=c["b_block"],
                                 out_dtype=_dt(c["dtype"]), ws=s["ws"])
    return (_wide(s["a"], s["a_s"]) @ _wide(s["b"], s["b_s"], c["b_block"]).t()).to(_dt(c["dtype"]))


def _grouped(s):
    c = s["c"]
    T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
    if own:
        return _ops().fp8_grouped_matmul(s["a"].view(torch.uint8), s["a_s"], s["b"].view(torch.uint8), s["b_s"], s["al"], k)
    x = _wide(s["a"], s["a_s"])
    flat = s["ids"].reshape(-1).long()
    token = torch.arange(T * k, device=DEV) // k
    if T * k < E:  # few pairs: the picked experts' weights, one product each
        w = s["b"][flat].float().view(T * k, N, K // 128, 128)
        w *= s["b_s"][flat].repeat_interleave(128, 1)[:, :N, :, None]
        return torch.bmm(w.view(T * k, N, K), x[token].unsqueeze(2)).squeeze(2).to(BF)
    rows = x.new_zeros(E, s["most"], K)
    rows[flat, s["rank"]] = x[token]
    w = s["b"].float().view(E, N, K // 128, 128)
    w *= s["b_s"].repeat_interleave(128, 1)[:, :N, :, None]
    y = torch.bmm(w.view(E, N, K), rows.transpose(1, 2).contiguous())
    return y[flat, :, s["rank"]].to(BF)


def _balance(s):
    c, z, ids, mask = s["c"], s["z"], s["ids"], s["mask"]
    T, E, k, coef = (c[n] for n in ("T", "E", "k", "coef"))
    if own:
        ops = _ops()
        f = ops.balance_loss(z, ids, mask=mask, coef=coef)
        dz = ops.balance_loss_backward(z, f["counts"], f["tokens"], k, s["dloss"], mask=mask, coef=coef)
        return {"loss": f["loss"], "counts": f["counts"], "probs": f["probs"], "dlogits": dz}
    keep = torch.ones(T, device=DEV) if mask is None else mask.float()
    n = keep.sum().clamp_min(1)
    p = torch.softmax(z, 1) * keep[:, None]
    probs = p.double().sum(0) / n
    hot = torch.zeros(T, E, device=DEV).scatter_add_(1, ids.long(), keep[:, None].expand(T, k))
    counts = hot.sum(0)
    frac = counts / (k * n)
    loss = (coef * E * (frac.double() * probs).sum()).float().reshape(1)
    dz = s["dloss"] * coef * E / n * p * (frac - (p * frac).sum(1, keepdim=True))
    return {"loss": loss, "counts": counts.to(torch.int32), "probs": probs.float(), "dlogits": dz}


EPS = 1e-6


def _norm32(v, w):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * w


def _form(n, out):
    if out in ("bf16", "f32"):
        return {"n": n.to(_dt(out))}
    if out == "e4m3":
        s = _scale_of(n.abs().amax(1))
        return {"n": _codes(n, s[:, None]), "scale": s}
    codes, s = _rows128(n)
    return {"n": codes, "scale": s}


def _norm(s):
    c = s["c"]
    what, dt = c["what"], _dt(c["dtype"])
    if own:
        return _norm_own(s)
    x, w = s["x"].float(), s["w"]
    if what == "pre":
        return _form(_norm32(x, w), c["out"])
    if what == "pre_bwd":
        dn, r = s["dn"].float(), torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        h = x * r
        dh = dn * w
        dx = s["dres"].float() + r * (dh - h * (dh * h).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dw": (dn * h).double().sum(0).float()}
    y, gate, alpha = s["y"].float(), s["gate"], c["alpha"]
    gate = 1.0 if gate is None else gate.float()
    if what == "post_bwd":
        dout, r = s["dout"].float(), torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
        h = y * r
        du = dout * gate
        dh = du * w
        out = {"dy": (r * (dh - h * (dh * h).mean(1, keepdim=True))).to(dt), "dres": (alpha * dout).to(dt), "dw": (du * h).double().sum(0).float()}
        dg = dout * h * w
        if c["gate"] == "h":
            out["dgate"] = dg.double().sum(0).float()
        elif c["gate"] == "t":
            out["dgate"] = dg.sum(1, keepdim=True)
        elif c["gate"] == "th":
            out["dgate"] = dg.to(dt)
        return out
    o = (alpha * x + gate * _norm32(y, w)).to(dt)
    if what == "post":
        return {"out": o}
    return {"out": o} | _form(_norm32(o.float(), s["w2"]), c["out"])


def _norm_own(s):
    ops, c = _ops(), s["c"]
    what = c["what"]

    def form(n, scale):
        return {"n": n} if c["out"] in ("bf16", "f32") else {"n": _f8(n), "scale": scale}

    if what == "pre":
        return form(*ops.pre_norm(s["x"], s["w"], eps=EPS, out=c["out"]))
    if what == "pre_bwd":
        dx, dw = ops.pre_norm_backward(s["dn"], s["x"], s["w"], eps=EPS, dres=s["dres"])
        return {"dx": dx, "dw": dw}
    if what == "post_bwd":
        r = ops.post_norm_backward(s["dout"], s["y"], s["w"], gate=s["gate"], alpha=c["alpha"], eps=EPS)
        return {n: v for n, v in r.items() if v is not None}
    if what == "post":
        return {"out": ops.post_norm(s["y"], s["w"], s["x"], gate=s["gate"], alpha=c["alpha"], eps=EPS)[0]}
    o, n, scale = ops.post_norm(s["y"], s["w"], s["x"], gate=s["gate"], alpha=c["alpha"], eps=EPS, next_weight=s["w2"], next_out=c["out"])
    return {"out": o} | form(n, scale)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "quant":
        M, K, b = c["M"], c["K"], 2 if c["dtype"] == "bf16" else 4
        out = M * K * (1 + 4 / 128)
        return {"bytes": M * K * b * (2 if c["act"] else 1) + out * (2 if c["cols"] else 1), "flops": M * K * (8 if c["act"] else 2)}
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        s = M * K / 32 + (N * K / 32 if not c["b_block"] else N * K / 4096)
        return {"bytes": M * K + N * K + s + M * N * (2 if c["dtype"] == "bf16" else 4), "flops": 2 * M * N * K}
    if c["op"] == "grouped":
        T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
        touched = E * (1 - (1 - k / E) ** T)  # expected number of experts with a row
        return {"bytes": touched * N * K * (1 + 4 / 16384) + T * K * (1 + 4 / 128) + T * k * N * 2, "flops": 2 * T * k * N * K}
    if c["op"] == "balance":  # logits are read by the forward and by the backward pass
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 3 * T * E * 4 + T * k * 4, "flops": 12 * T * E}
    T, H, b = c["T"], c["H"], 2 if c["dtype"] == "bf16" else 4
    n = {"bf16": 2, "f32": 4, "e4m3": 1, "e4m3_128": 1 + 4 / 128}.get(c.get("out"), 0)
    g = {"th": b}.get(c.get("gate"), 0)
    streams = {"pre": b + n, "pre_bwd": 4 * b, "post": 3 * b + g, "post_next": 3 * b + g + n, "post_bwd": 4 * b + 2 * g}[c["what"]]
    return {"bytes": T * H * streams + 8 * H, "flops": 12 * T * H}


# ---------------------------------------------------------------- the definitions in 64 bits

def _e4m3_64(v):
    a = v.abs().clamp(max=448.0)
    e = (torch.frexp(a).exponent - 1).clamp(min=-6).double()
    step = torch.exp2(e - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _groups64(v, dim):
    """e4m3 values and scales of groups of 128 along `dim` (the last one may be short) of a float64 matrix."""
    if dim == 0:
        q, s = _groups64(v.t(), 1)
        return q, s
    M, K = v.shape
    q, scales = v.new_zeros(M, -(-K // 128) * 128), []
    for k in range(0, K, 128):
        part = v[:, k:k + 128]
        top = part.abs().max(1).values
        s = torch.where(top > 0, torch.maximum(top / 448, torch.full_like(top, 2.0 ** -126)), torch.ones_like(top))
        q[:, k:k + part.shape[1]] = _e4m3_64(part / s[:, None])
        scales.append(s)
    return q, torch.stack(scales)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "quant":
        v = s["x"].double()
        if c["act"]:
            gate, up = v[:, :c["K"]], v[:, c["K"]:]
            v = gate * torch.sigmoid(gate) * up
        out = dict(zip(("codes", "scale"), _groups64(v, 1)))
        if c["cols"]:
            out |= dict(zip(("codes_t", "scale_t"), _groups64(v, 0)))
        return out
    if c["op"] == "matmul":
        acc = torch.zeros(c["M"], c["N"], dtype=torch.float64, device=DEV)
        for j in range(c["K"] // 128):
            at = slice(128 * j, 128 * j + 128)
            part = s["a"][:, at].double() @ s["b"][:, at].double().t()
            if c["b_block"]:
                sb = s["b_s"][:, j].double().repeat_interleave(128)[:c["N"]]
            else:
                sb = s["b_s"][j].double()
            acc += part * s["a_s"][j].double()[:, None] * sb[None, :]
        return acc
    if c["op"] == "grouped":
        T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
        y = torch.zeros(T * k, N, dtype=torch.float64, device=DEV)
        flat = s["ids"].reshape(-1)
        for e in range(E):
            pairs = (flat == e).nonzero().reshape(-1)
            if pairs.numel():
                t = pairs // k
                w = s["b"][e].double() * s["b_s"][e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
                a = s["a"][t].double() * s["a_s"][:, t].double().t().repeat_interleave(128, 1)
                y[pairs] = a @ w.t()
        return y
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        z = s["z"].double().requires_grad_(True)
        at = torch.arange(T, device=DEV) if s["mask"] is None else s["mask"].nonzero().reshape(-1)
        n = max(1, at.numel())
        probs = torch.exp(z[at] - torch.logsumexp(z[at], 1, keepdim=True)).sum(0) / n
        counts = torch.bincount(s["ids"][at].reshape(-1).long(), minlength=E)
        loss = c["coef"] * E * (counts.double() / (k * n) * probs).sum()
        (loss * s["dloss"].double()).sum().backward()
        return {"loss": loss.detach().reshape(1), "counts": None, "probs": probs.detach(), "dlogits": z.grad}
    return _norm_exact(s)


def _norm_exact(s):
    c = s["c"]
    what, dt = c["what"], _dt(c["dtype"])
    leaf = {n: s[n].double().requires_grad_(True) for n in ("x", "w", "y", "gate") if s.get(n) is not None}

    def norm(v, w):
        return v / torch.sqrt((v * v).sum(1, keepdim=True) / c["H"] + EPS) * w

    def form(n):
        if c["out"] in ("bf16", "f32"):
            return {"n": n}
        if c["out"] == "e4m3":
            top = n.abs().max(1).values
            sc = torch.where(top > 0, torch.maximum(top / 448, torch.full_like(top, 2.0 ** -126)), torch.ones_like(top))
            return {"n": _e4m3_64(n / sc[:, None]), "scale": sc}
        return dict(zip(("n", "scale"), _groups64(n, 1)))

    if what == "pre":
        return form(norm(leaf["x"], leaf["w"]).detach())
    if what == "pre_bwd":
        norm(leaf["x"], leaf["w"]).backward(s["dn"].double())
        return {"dx": leaf["x"].grad + s["dres"].double(), "dw": leaf["w"].grad}
    u = norm(leaf["y"], leaf["w"])
    if "gate" in leaf:
        u = u * leaf["gate"]
    o = c["alpha"] * leaf["x"] + u
    if what == "post_bwd":
        o.backward(s["dout"].double())
        out = {"dy": leaf["y"].grad, "dres": leaf["x"].grad, "dw": leaf["w"].grad}
        return out | {"dgate": leaf["gate"].grad} if "gate" in leaf else out
    o = o.detach()
    if what == "post":
        return {"out": o}
    return {"out": o} | form(norm(o.to(dt).double(), s["w2"].double()))  # the next norm reads the stored (rounded) stream
