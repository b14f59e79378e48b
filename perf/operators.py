"""The microscaled 4-bit (MXFP4) operators and the router's counts and balance loss, as cases to measure.

Each case is one call (or the few calls that always go together) of a user of the library:

  pack      quantise a weight or activation matrix to MXFP4 and decode it
  matmul    y = x W^T (+ bias), bf16 activations against an MXFP4 weight matrix
  mx        the same with the activations quantised to MXFP4 on the way
  experts   routing ids -> per-expert counts and lists -> the experts' products
  balance   routing ids -> per-expert counts -> balance loss and its gradient

With `own` false, run() computes them in elementary torch operations in
32 bits; with `own` true, it calls decode_matmul_amd.
"""

import torch

own = False

DEV = "cuda"
MOST_PACK = 14336 * 4096                # largest quantised matrix (the library's ternary GEMV layer)
MOST_MNK = 2048 * 8192 * 8192           # largest dense product (its Route B prefill)


def listed():
    return [
        # a small projection quantised on its own: a launch's latency
        {"name": "pack f32 256x256", "op": "pack", "rows": 256, "K": 256, "dtype": "float32", "out": "float32"},
        # the 14336 x 4096 feed-forward weight, quantised from a bf16 checkpoint
        {"name": "pack bf16 14336x4096", "op": "pack", "rows": 14336, "K": 4096, "dtype": "bfloat16",
         "out": "bfloat16"},
        # one token's decode step through that layer
        {"name": "matmul M1 14336x4096", "op": "matmul", "M": 1, "N": 14336, "K": 4096, "pad": 0, "bias": False,
         "out": "bfloat16"},
        # a decode batch of 16 through an 8192 x 8192 layer
        {"name": "matmul M16 8192x8192", "op": "matmul", "M": 16, "N": 8192, "K": 8192, "pad": 0, "bias": True,
         "out": "float32"},
        # an odd batch through odd sizes, x a column slice of a wider tensor
        {"name": "matmul M300 1001x1000", "op": "matmul", "M": 300, "N": 1001, "K": 1000, "pad": 24, "bias": True,
         "out": "float32"},
        # a prompt of 2048 tokens
        {"name": "matmul M2048 8192x8192", "op": "matmul", "M": 2048, "N": 8192, "K": 8192, "pad": 0,
         "bias": False, "out": "bfloat16"},
        # a few tokens with 4-bit activations
        {"name": "mx M4 14336x4096", "op": "mx", "M": 4, "N": 14336, "K": 4096, "bias": False, "out": "bfloat16"},
        # a prompt with 4-bit activations
        {"name": "mx M2048 8192x8192", "op": "mx", "M": 2048, "N": 8192, "K": 8192, "bias": False,
         "out": "bfloat16"},
        # the library's expert layer: 16 tokens, top 8 of 64 experts
        {"name": "experts M16 64x2048x4096", "op": "experts", "M": 16, "N": 2048, "K": 4096, "E": 64, "top_k": 8,
         "idle": 0, "bias": False, "out": "float32"},
        # a prompt through it, its last 37 tokens padding
        {"name": "experts M2048 64x2048x4096", "op": "experts", "M": 2048, "N": 2048, "K": 4096, "E": 64,
         "top_k": 8, "idle": 37, "bias": True, "out": "bfloat16"},
        # one decode batch's router
        {"name": "balance M16 E64", "op": "balance", "M": 16, "E": 64, "top_k": 8, "dtype": "float32", "idle": 0},
        # a training batch's router, its tail padded
        {"name": "balance M65536 E128", "op": "balance", "M": 65536, "E": 128, "top_k": 8, "dtype": "bfloat16",
         "idle": 1000},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def _some(rng, lo, hi, step):
    """_log, half of the time rounded to a multiple of step."""
    v = _log(rng, lo, hi)
    return max(lo, v // step * step) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(("pack", "matmul", "mx", "experts", "balance"))
    out = rng.choice(("float32", "bfloat16"))
    if op == "pack":
        K = _some(rng, 32, 8192, 32)
        return {"op": op, "rows": _log(rng, 1, min(16384, MOST_PACK // K)), "K": K,
                "dtype": rng.choice(("float32", "bfloat16")), "out": out}
    if op in ("matmul", "mx"):
        M, K = _log(rng, 1, 2048), _some(rng, 64, 8192, 64)
        c = {"op": op, "M": M, "N": _some(rng, 64, min(14336, MOST_MNK // (M * K)), 16), "K": K,
             "bias": rng.random() < 0.5, "out": out}
        if op == "matmul":
            c["pad"] = rng.choice((0, 0, 8, 13))
        return c
    E = rng.choice((4, 8, 16, 32, 60, 64, 128))
    top_k = rng.randint(1, min(8, E // 2))
    if op == "experts":
        M, N, K = _log(rng, 1, 2048), _some(rng, 64, 2048, 16), _some(rng, 64, 4096, 64)
        return {"op": op, "M": M, "N": N, "K": K, "E": min(E, 64), "top_k": top_k,
                "idle": rng.randint(0, M // 4), "bias": rng.random() < 0.5, "out": out}
    M = _log(rng, 1, 65536)
    return {"op": op, "M": M, "E": E, "top_k": top_k, "dtype": rng.choice(("float32", "bfloat16")),
            "idle": rng.randint(0, M // 4)}


# ---------------------------------------------------------------- inputs


def _weights(shape, gen):
    """Weights of a trained layer's spread, one magnitude a row."""
    w = torch.randn(shape, generator=gen, device=DEV) * 0.02
    return w * (0.5 + torch.rand(shape[:-1] + (1,), generator=gen, device=DEV))


def _acts(M, K, pad, gen):
    """bf16 activations with a few channels far above the rest, rows K + pad apart."""
    x = torch.randn((M, K + pad), generator=gen, device=DEV)
    loud = torch.rand((K + pad,), generator=gen, device=DEV) < 0.005
    return torch.where(loud, x * 12, x).to(torch.bfloat16)[:, :K]


def _router(case, gen):
    """Logits of an uneven router, the experts each token goes to, and which tokens count."""
    M, E = case["M"], case["E"]
    z = torch.randn((M, E), generator=gen, device=DEV) + 0.7 * torch.randn((E,), generator=gen, device=DEV)
    z = z.to(getattr(torch, case.get("dtype", "float32")))
    ids = z.float().topk(case["top_k"], dim=1).indices.to(torch.int32)
    keep = torch.arange(M, device=DEV) < M - case["idle"]
    return z, torch.where(keep[:, None], ids, -1), keep


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    out = getattr(torch, case.get("out", "float32"))
    if op == "pack":
        rows, K = case["rows"], case["K"]
        s["W"] = _weights((rows, K), gen).to(getattr(torch, case["dtype"]))
        s["codes"], s["scales"] = _empty_package((rows,), K)
        s["y"] = torch.empty((rows, K), dtype=out, device=DEV)
        return s
    if op == "balance":
        s["logits"], s["ids"], keep = _router(case, gen)
        s["mask"] = keep.to(torch.uint8)
        s["dloss"] = torch.rand((1,), generator=gen, device=DEV) + 0.5
        s["grad"] = torch.empty_like(s["logits"])
        s["loss"] = torch.empty((1,), dtype=torch.float32, device=DEV)
        s["weights"] = torch.empty((case["E"],), dtype=torch.float32, device=DEV)
    M, E = case["M"], case.get("E", 1)
    if op in ("balance", "experts"):
        pairs = M * case["top_k"]
        s["counts"] = torch.empty((E,), dtype=torch.int32, device=DEV)
        s["offsets"] = torch.empty((E + 1,), dtype=torch.int32, device=DEV)
        s["order"] = torch.empty((pairs,), dtype=torch.int32, device=DEV)
    if op == "balance":
        return s
    N, K = case["N"], case["K"]
    s["x"] = _acts(M, K, case.get("pad", 0), gen)
    if op == "experts":
        _, s["ids"], _ = _router(case, gen)
        s["codes"], s["scales"] = _empty_package((E, N), K)
        for e in range(E):
            s["codes"][e], s["scales"][e] = _quantise(_weights((N, K), gen))
        s["y"] = torch.empty((M, case["top_k"], N), dtype=out, device=DEV)
        shape = (E, N)
    else:
        s["codes"], s["scales"] = _quantise(_weights((N, K), gen))
        s["y"] = torch.empty((M, N), dtype=out, device=DEV)
        shape = (N,)
    if op == "mx":
        s["x_codes"], s["x_scales"] = _empty_package((M,), K)
    s["bias"] = torch.randn(shape, generator=gen, device=DEV) if case["bias"] else None
    return s


def _empty_package(lead, K):
    nb = -(-K // 32)
    return (torch.empty(lead + (nb, 16), dtype=torch.uint8, device=DEV),
            torch.empty(lead + (nb,), dtype=torch.uint8, device=DEV))


# ------------------------------------------------------- the plain forms


def _steps(w):
    """MXFP4 of the rows of w: the elements as multiples of their block's
    scale [rows, blocks, 32], and the scales' exponents [rows, blocks, 1]."""
    rows, K = w.shape
    v = torch.nn.functional.pad(w.float(), (0, -K % 32)).view(rows, -1, 32)
    amax = v.abs().amax(dim=2, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
    a = torch.ldexp(v.abs(), -e)
    a = torch.where(a < 2, (a * 2).round() / 2, torch.where(a < 4, a.round(), (a / 2).round() * 2)).clamp(max=6)
    return torch.copysign(a, v), e


def _quantise(w):
    """codes [rows, blocks, 16] and scales [rows, blocks] of the rows of w."""
    q, e = _steps(w)
    a = q.abs()
    c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = c | (torch.signbit(q).to(torch.uint8) << 3)
    return c[..., 0::2] | (c[..., 1::2] << 4), (e.squeeze(2) + 127).to(torch.uint8)


def _decode(codes, scales, K):
    """The values of a package [..., blocks, 16], fp32 [..., K]."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    a = (c & 7).float()
    a = torch.where(a < 4, a / 2, torch.where(a < 6, a - 2, 2 * a - 8))
    a = torch.ldexp(torch.where(c > 7, -a, a), (scales.int() - 127).unsqueeze(-1))
    return a.flatten(-2)[..., :K]


def _routed(ids, E):
    """counts, offsets and the slots sorted by expert, those of no expert last."""
    flat = ids.flatten().long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(dim=0)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    order = torch.sort(flat, stable=True).indices
    return flat, counts.int(), offsets, order


def _experts(s, case):
    """Each expert's rows padded to whole tiles of B slots, one product a tile."""
    M, top_k, E, K = case["M"], case["top_k"], case["E"], case["K"]
    pairs = M * top_k
    B = 16 if pairs <= 16 * E else 128
    flat, counts, offsets, order = _routed(s["ids"], E)
    tiles = -(-counts.long() // B)
    ends = tiles.cumsum(0)
    t = torch.arange(pairs // B + E, device=flat.device)
    e = torch.searchsorted(ends, t, right=True).clamp(max=E - 1)
    row = (t - (ends - tiles)[e])[:, None] * B + torch.arange(B, device=flat.device)
    there = (row < counts[e][:, None]) & (t < ends[-1])[:, None]
    slot = order[torch.where(there, offsets[e][:, None] + row, 0)]
    x = s["x"].float()[slot // top_k] * there[..., None]
    y = torch.bmm(x, _decode(s["codes"][e], s["scales"][e], K).transpose(1, 2).contiguous())
    if s["bias"] is not None:
        y = y + s["bias"][e][:, None, :]
    whole = y.new_full((pairs + 1, case["N"]), float("nan"))
    whole[torch.where(there, slot, pairs)] = y
    return {"y": whole[:pairs].view(M, top_k, -1).to(s["y"].dtype), "counts": counts, "offsets": offsets.int(),
            "order": order.int()}


def _balance(s, case):
    E = case["E"]
    _, counts, _, _ = _routed(s["ids"], E)
    keep = s["mask"].bool()[:, None]
    T, n = keep.sum(), counts.sum()
    w = torch.where((T > 0) & (n > 0), E * counts.double() / n.clamp(min=1) / T.clamp(min=1), 0.0)
    z = s["logits"].float()
    p = torch.exp(z - z.amax(dim=1, keepdim=True))
    p = p / p.sum(dim=1, keepdim=True) * keep
    w = w.float()
    mean = (p * w).sum(dim=1, keepdim=True)
    grad = s["dloss"] * p * (w - mean)
    return {"counts": counts, "loss": mean.double().sum().float().view(1), "grad": grad.to(s["logits"].dtype)}


def _plain(s, case):
    op = case["op"]
    if op == "pack":
        q, e = _steps(s["W"])
        return torch.ldexp(q, e).flatten(1)[:, :case["K"]].to(s["y"].dtype)
    if op == "experts":
        return _experts(s, case)
    if op == "balance":
        return _balance(s, case)
    x = s["x"].float()
    if op == "mx":
        q, e = _steps(s["x"])
        x = torch.ldexp(q, e).flatten(1)[:, :case["K"]]
    y = x @ _decode(s["codes"], s["scales"], case["K"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["y"].dtype)


# ---------------------------------------------------- the library's calls


def _workspace(s, key, nbytes):
    """A workspace that the program keeps from its first pass on."""
    if nbytes and key not in s:
        s[key] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return s.get(key)


def _calls(s, case):
    import decode_matmul_amd as dmm
    op = case["op"]
    if op == "pack":
        dmm.mx_pack(s["W"], s["codes"], s["scales"])
        dmm.mx_unpack(s["codes"], s["scales"], case["rows"], case["K"], s["y"])
        return s["y"]
    if op == "matmul":
        dmm.mx_matmul(s["x"], s["codes"], s["scales"], case["N"], s["y"], bias=s["bias"])
        return s["y"]
    if op == "mx":
        dmm.mx_pack(s["x"], s["x_codes"], s["x_scales"])
        dmm.mx_matmul_mx(s["x_codes"], s["x_scales"], case["M"], case["K"], s["codes"], s["scales"], case["N"],
                         s["y"], bias=s["bias"])
        return s["y"]
    M, E, top_k = case["M"], case["E"], case["top_k"]
    ws = _workspace(s, "route_ws", dmm.moe_route_workspace_bytes(M, top_k, E))
    dmm.moe_route(s["ids"], E, s["counts"], s["offsets"], s["order"], workspace=ws)
    if op == "experts":
        dmm.mx_matmul_experts(s["x"], s["codes"], s["scales"], case["N"], s["y"], E, s["offsets"], s["order"],
                              top_k, bias=s["bias"])
        return {"y": s["y"], "counts": s["counts"], "offsets": s["offsets"], "order": s["order"]}
    ws = _workspace(s, "balance_ws", dmm.moe_balance_workspace_bytes(M, E))
    dmm.moe_balance(s["logits"], s["counts"], s["loss"], s["weights"], token_mask=s["mask"], workspace=ws)
    dmm.moe_balance_grad(s["logits"], s["weights"], s["dloss"], s["grad"], token_mask=s["mask"])
    return {"counts": s["counts"], "loss": s["loss"], "grad": s["grad"]}


def run(state):
    if own:
        return _calls(state, state["case"])
    return _plain(state, state["case"])


# ------------------------------------------------------------ what it needs


def work(case):
    op = case["op"]
    size = {"float32": 4, "bfloat16": 2}
    if op == "pack":
        n = case["rows"] * case["K"]
        package = case["rows"] * -(-case["K"] // 32) * 17
        return {"bytes": n * (size[case["dtype"]] + size[case["out"]]) + 2 * package, "flops": n}
    if op == "balance":
        M, E = case["M"], case["E"]
        return {"bytes": M * E * 3 * size[case["dtype"]] + M * (8 * case["top_k"] + 2), "flops": 12 * M * E}
    M, N, K = case["M"], case["N"], case["K"]
    package = N * -(-K // 32) * 17
    rows, touched = M, 1.0
    if op == "experts":
        live = M - case["idle"]
        rows = live * case["top_k"]
        touched = case["E"] * (1 - (1 - case["top_k"] / case["E"]) ** live)
    moved = package * touched + M * K * 2 + M * case.get("top_k", 1) * N * size[case["out"]]
    return {"bytes": int(moved), "flops": 2 * rows * N * K}


# ------------------------------------------------ the definitions in 64 bits

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest64(w):
    """Each row's blocks of 32 rounded to the nearest value of their grid; a
    value midway between two goes to the one with an even index."""
    out = torch.zeros(w.shape, dtype=torch.float64, device=w.device)
    for k in range(0, w.shape[1], 32):
        b = w[:, k:k + 32].double()
        top = b.abs().max(dim=1, keepdim=True).values
        unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2)
        r = b.abs() / unit
        v = torch.zeros_like(r)
        for i in range(1, 8):
            mid = (_GRID[i - 1] + _GRID[i]) / 2
            v = torch.where((r >= mid) if i % 2 == 0 else (r > mid), _GRID[i], v)
        out[:, k:k + 32] = torch.sign(b) * v * unit
    return out


def _values64(codes, scales, K):
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float64, device=codes.device)
    out = torch.empty(codes.shape[:-2] + (codes.shape[-2] * 32,), dtype=torch.float64, device=codes.device)
    unit = torch.exp2(scales.double() - 127).repeat_interleave(16, dim=-1)
    flat = codes.flatten(-2)
    out[..., 0::2] = grid[(flat % 16).long()] * unit
    out[..., 1::2] = grid[(flat // 16).long()] * unit
    return out[..., :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "pack":
        return _nearest64(s["W"])
    if op in ("matmul", "mx"):
        x = s["x"].double() if op == "matmul" else _nearest64(s["x"])
        y = torch.matmul(x, _values64(s["codes"], s["scales"], case["K"]).t())
        return y if s["bias"] is None else y + s["bias"].double()
    E, top_k = case["E"], case["top_k"]
    ids = s["ids"].flatten().long()
    if op == "experts":
        y = torch.full((ids.numel(), case["N"]), float("nan"), dtype=torch.float64, device=ids.device)
        for e in range(E):
            at = torch.nonzero(ids == e).flatten()
            y[at] = s["x"].double()[at // top_k] @ _values64(s["codes"][e], s["scales"][e], case["K"]).t()
            if s["bias"] is not None:
                y[at] += s["bias"][e].double()
        return {"y": y.view(case["M"], top_k, -1), "counts": None, "offsets": None, "order": None}
    valid = ids[ids >= 0]
    f = torch.bincount(valid, minlength=E).double() / max(1, valid.numel())
    z = s["logits"].double()
    z.requires_grad_(True)
    p = torch.softmax(z, dim=1)[s["mask"] > 0]
    loss = E * (f * p.sum(dim=0)).sum() / max(1, p.shape[0])
    loss.backward()
    return {"counts": None, "loss": loss.detach().view(1), "grad": z.grad * s["dloss"].double()}
