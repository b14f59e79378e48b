"""The router's choice, the combination of the experts' rows, and the products in 8-bit floating point
(e4m3, a scale for each block of 128), as cases to measure.

Each case is one call (or the few calls that always go together) of a user of the library:

  gate      router logits -> the experts of each token and their weights (with grad: dlogits of given dweights)
  combine   the experts' rows and weights -> one row a token (with grad: the gradients of both)
  norm      residual addition, root-mean-square norm, and the normed rows as an 8-bit package
  matmul    y = x W^T (+ bias) of two 8-bit packages; where not packed, bf16 activations are packed on the way
  experts   routing ids -> per-expert counts and lists -> the experts' products of 8-bit packages

With `own` false, run() computes them in elementary torch operations in
32 bits (the choice of experts in 64); with `own` true, it calls decode_matmul_amd.
"""

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
MOST_SCORES = 65536 * 128               # largest router (tokens x experts)
MOST_ROWS = 2048 * 8 * 4096             # largest combination (tokens x top_k x columns)
MOST_NORM = 2048 * 8192                 # largest norm
MOST_MNK = 2048 * 8192 * 8192           # largest dense product (the library's Route B prefill)
EPS = 1e-6


def listed():
    return [
        # one decode batch through a router of 256 experts in 8 groups, its choice shifted by a learned bias
        {"name": "gate M16 E256 groups", "op": "gate", "M": 16, "E": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5,
         "dtype": "float32", "idle": 0, "grad": False},
        # a training batch's router, its tail padded, and its gradient
        {"name": "gate M65536 E128 grad", "op": "gate", "M": 65536, "E": 128, "top_k": 8, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renorm": True, "scale": 1.0,
         "dtype": "bfloat16", "idle": 1000, "grad": True},
        # a decode batch's rows of the experts, beside the token's own row
        {"name": "combine M16 N4096", "op": "combine", "M": 16, "N": 4096, "E": 64, "top_k": 8, "idle": 0,
         "add": True, "rows": "float32", "out": "bfloat16", "grad": False},
        # a training batch's rows and their gradients, its tail padded
        {"name": "combine M2048 N4096 grad", "op": "combine", "M": 2048, "N": 4096, "E": 64, "top_k": 8, "idle": 37,
         "add": False, "rows": "bfloat16", "out": "bfloat16", "grad": True},
        # one token's residual stream on its way into a layer
        {"name": "norm M1 K4096", "op": "norm", "M": 1, "K": 4096, "residual": True, "normed": False,
         "dtype": "bfloat16"},
        # a prompt's; the normed rows are wanted beside the package
        {"name": "norm M2048 K8192", "op": "norm", "M": 2048, "K": 8192, "residual": True, "normed": True,
         "dtype": "bfloat16"},
        # one token's decode step through the 14336 x 4096 feed-forward layer, its package from the norm
        {"name": "matmul M1 14336x4096", "op": "matmul", "M": 1, "N": 14336, "K": 4096, "packed": True, "pad": 0,
         "bias": False, "out": "bfloat16"},
        # an odd batch through odd sizes, x a column slice of a wider tensor
        {"name": "matmul M300 1001x1000", "op": "matmul", "M": 300, "N": 1001, "K": 1000, "packed": False, "pad": 24,
         "bias": True, "out": "float32"},
        # a decode batch of 16 through an 8192 x 8192 layer
        {"name": "matmul M16 8192x8192", "op": "matmul", "M": 16, "N": 8192, "K": 8192, "packed": False, "pad": 0,
         "bias": True, "out": "float32"},
        # a prompt of 2048 tokens
        {"name": "matmul M2048 8192x8192", "op": "matmul", "M": 2048, "N": 8192, "K": 8192, "packed": False, "pad": 0,
         "bias": False, "out": "bfloat16"},
        # the library's expert layer: 16 tokens, top 8 of 64 experts
        {"name": "experts M16 64x2048x4096", "op": "experts", "M": 16, "N": 2048, "K": 4096, "E": 64, "top_k": 8,
         "idle": 0, "bias": False, "out": "float32"},
        # a prompt through it, its last 37 tokens padding
        {"name": "experts M2048 64x2048x4096", "op": "experts", "M": 2048, "N": 2048, "K": 4096, "E": 64,
         "top_k": 8, "idle": 37, "bias": False, "out": "bfloat16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def _some(rng, lo, hi, step):
    """_log, half of the time rounded to a multiple of step."""
    v = _log(rng, lo, hi)
    return max(lo, v // step * step) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(("gate", "combine", "norm", "matmul", "experts"))
    dtype, out = rng.choice(("float32", "bfloat16")), rng.choice(("float32", "bfloat16"))
    if op == "gate":
        E = rng.choice((8, 16, 60, 64, 128, 160, 256, 512))
        groups = rng.choice((1, 1, 4, 8)) if E % 8 == 0 else rng.choice((1, 4))
        top_groups = rng.randint((groups + 1) // 2, groups)
        M = _log(rng, 1, MOST_SCORES // max(E, 128))
        top_k = rng.randint(1, min(8, top_groups * E // groups))
        return {"op": op, "M": M, "E": E, "top_k": top_k,
                "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": top_groups, "group_top": 2 if E // groups > 1 and rng.random() < 0.5 else 1,
                "renorm": top_k > 1 and rng.random() < 0.7, "scale": rng.choice((1.0, 1.0, 2.5)), "dtype": dtype,
                "idle": rng.randint(0, M // 4), "grad": rng.random() < 0.5}
    if op == "combine":
        top_k, N = rng.randint(1, 8), _some(rng, 64, 8192, 64)
        M = _log(rng, 1, min(2048, MOST_ROWS // (top_k * N * (2 if dtype == "float32" else 1))))
        return {"op": op, "M": M, "N": N, "E": 64, "top_k": top_k, "idle": rng.randint(0, M // 4),
                "add": rng.random() < 0.5, "rows": dtype, "out": out, "grad": rng.random() < 0.5}
    if op == "norm":
        K = _some(rng, 64, 8192, 64)
        most = MOST_NORM // K if dtype == "bfloat16" else MOST_NORM // (2 * K)
        return {"op": op, "M": _log(rng, 1, min(16384, most)), "K": K, "residual": rng.random() < 0.7,
                "normed": rng.random() < 0.5, "dtype": dtype}
    if op == "matmul":
        M, K = _log(rng, 1, 2048), _some(rng, 64, 8192, 64)
        return {"op": op, "M": M, "N": _some(rng, 64, min(14336, MOST_MNK // (M * K)), 16), "K": K,
                "packed": rng.random() < 0.5, "pad": rng.choice((0, 0, 8, 13)), "bias": rng.random() < 0.5, "out": out}
    E = rng.choice((4, 8, 16, 32, 60, 64))
    M, N, K = _log(rng, 1, 2048), _some(rng, 64, 2048, 16), _some(rng, 64, 4096, 64)
    return {"op": op, "M": M, "N": N, "K": K, "E": E, "top_k": rng.randint(1, min(8, E // 2)),
            "idle": rng.randint(0, M // 4), "bias": rng.random() < 0.5, "out": out}


# ---------------------------------------------------------------- inputs


def _weights(shape, gen):
    """Weights of a trained layer's spread, one magnitude a row."""
    w = torch.randn(shape, generator=gen, device=DEV) * 0.02
    return w * (0.5 + torch.rand(shape[:-1] + (1,), generator=gen, device=DEV))


def _acts(M, K, pad, gen, dtype=torch.bfloat16):
    """Activations with a few channels far above the rest, rows K + pad apart."""
    x = torch.randn((M, K + pad), generator=gen, device=DEV)
    loud = torch.rand((K + pad,), generator=gen, device=DEV) < 0.005
    return torch.where(loud, x * 12, x).to(dtype)[:, :K]


def _router(M, E, dtype, gen):
    """Logits of an uneven router."""
    z = torch.randn((M, E), generator=gen, device=DEV) + 0.7 * torch.randn((E,), generator=gen, device=DEV)
    return z.to(dtype)


def _routed_ids(case, gen):
    """The experts of each token; the last `idle` tokens are padding and have none."""
    M = case["M"]
    z = _router(M, case["E"], torch.float32, gen)
    ids = z.topk(case["top_k"], dim=1).indices.to(torch.int32)
    keep = torch.arange(M, device=DEV) < M - case["idle"]
    w = torch.softmax(torch.gather(z, 1, ids.long()), dim=1) * keep[:, None]
    return torch.where(keep[:, None], ids, -1), w


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, M = case["op"], case["M"]
    s = {"case": dict(case)}
    if op == "gate":
        E, top_k = case["E"], case["top_k"]
        s["logits"] = _router(M, E, getattr(torch, case["dtype"]), gen)
        s["bias"] = torch.randn((E,), generator=gen, device=DEV) * 0.05 if case["bias"] else None
        s["mask"] = (torch.arange(M, device=DEV) < M - case["idle"]).to(torch.uint8)
        s["ids"] = torch.empty((M, top_k), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((M, top_k), dtype=torch.float32, device=DEV)
        if case["grad"]:
            s["dweights"] = torch.randn((M, top_k), generator=gen, device=DEV)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    if op == "combine":
        N, top_k, rows, out = case["N"], case["top_k"], getattr(torch, case["rows"]), getattr(torch, case["out"])
        s["ids"], s["weights"] = _routed_ids(case, gen)
        y = torch.randn((M, top_k, N), generator=gen, device=DEV)
        s["y"] = torch.where((s["ids"] < 0)[..., None], float("nan"), y).to(rows)   # what the products leave there
        s["add"] = torch.randn((M, N), generator=gen, device=DEV).to(out) if case["add"] else None
        s["out"] = torch.empty((M, N), dtype=out, device=DEV)
        if case["grad"]:
            s["dout"] = torch.randn((M, N), generator=gen, device=DEV).to(out)
            s["dy"] = torch.empty_like(s["y"])
            s["dweights"] = torch.empty_like(s["weights"])
        return s
    K = case["K"]
    if op == "norm":
        dtype = getattr(torch, case["dtype"])
        s["x"] = _acts(M, K, 0, gen, dtype)
        s["residual"] = (_acts(M, K, 0, gen) * 3).to(dtype) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn((K,), generator=gen, device=DEV)).to(dtype)
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["normed"] = torch.empty_like(s["x"]) if case["normed"] else None
        s["codes"], s["scales"] = _empty_package(M, K)
        return s
    N, E = case["N"], case.get("E", 1)
    if op == "experts":
        pairs = M * case["top_k"]
        s["ids"], _ = _routed_ids(case, gen)
        s["counts"] = torch.empty((E,), dtype=torch.int32, device=DEV)
        s["offsets"] = torch.empty((E + 1,), dtype=torch.int32, device=DEV)
        s["order"] = torch.empty((pairs,), dtype=torch.int32, device=DEV)
        made = [_package(_weights((N, K), gen), 128) for _ in range(E)]
        s["codes"], s["scales"] = (torch.stack(p) for p in zip(*made))
        s["y"] = torch.empty((M, case["top_k"], N), dtype=getattr(torch, case["out"]), device=DEV)
        shape = (E, N)
    else:
        s["codes"], s["scales"] = _package(_weights((N, K), gen), 128)
        s["y"] = torch.empty((M, N), dtype=getattr(torch, case["out"]), device=DEV)
        shape = (N,)
    x = _acts(M, K, case.get("pad", 0), gen)
    if case.get("packed", True):
        s["x_codes"], s["x_scales"] = _package(x, 1)
    else:
        s["x"] = x
        s["x_codes"], s["x_scales"] = _empty_package(M, K)
    s["bias"] = torch.randn(shape, generator=gen, device=DEV) if case["bias"] else None
    return s


def _empty_package(rows, K):
    nb = -(-K // 128)
    return torch.empty((rows, nb, 128), dtype=F8, device=DEV), torch.empty((rows, nb), device=DEV)


# ------------------------------------------------------- the plain forms


def _package(w, block_rows):
    """e4m3 codes [rows, blocks, 128] and scales [rows / block_rows, blocks] of the rows of w."""
    rows, K = w.shape
    v = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -rows % block_rows))
    v = v.view(-1, block_rows, v.shape[1] // 128, 128)
    m, e = torch.frexp(v.abs().amax(dim=(1, 3)))
    e = torch.where(m > 0, e - 8 - (m <= 0.875).int(), -126).clamp(min=-126)   # the least 2^e >= largest / 448
    codes = torch.ldexp(v, -e[:, None, :, None]).to(F8)
    return codes.flatten(0, 1)[:rows], torch.ldexp(torch.ones_like(m), e)


def _decode(codes, scales, K, block_rows):
    """The values of a package [..., rows, blocks, 128], fp32 [..., rows, K]."""
    rows = codes.shape[-3]
    scales = scales.repeat_interleave(block_rows, dim=-2)[..., :rows, :] if block_rows > 1 else scales
    return (codes.float() * scales[..., None]).flatten(-2)[..., :K]


def _ranked(c):
    """The indices of the last dimension by falling value, equal ones by index."""
    return torch.sort(c, dim=-1, descending=True, stable=True).indices


def _gate(s, case):
    E, top_k, groups = case["E"], case["top_k"], case["groups"]
    z = s["logits"].double()
    p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.exp(z - z.amax(dim=1, keepdim=True))
    p = p if case["score"] == "sigmoid" else p / p.sum(dim=1, keepdim=True)
    c = z if s["bias"] is None else p + s["bias"].double()
    if groups > 1:
        of = p if s["bias"] is None and case["group_top"] > 1 else c
        best = of.view(-1, groups, E // groups).sort(dim=2, descending=True).values[..., :case["group_top"]].sum(dim=2)
        kept = torch.zeros_like(best, dtype=torch.bool).scatter(1, _ranked(best)[:, :case["top_groups"]], True)
        c = torch.where(kept.repeat_interleave(E // groups, dim=1), c, float("-inf"))
    ids = _ranked(c)[:, :top_k]
    keep = s["mask"].bool()[:, None]
    z = s["logits"].float()
    p = 1 / (1 + torch.exp(-z)) if case["score"] == "sigmoid" else torch.exp(z - z.amax(dim=1, keepdim=True))
    p = p if case["score"] == "sigmoid" else p / p.sum(dim=1, keepdim=True)
    chosen = torch.gather(p, 1, ids)
    total = chosen.sum(dim=1, keepdim=True)
    w = case["scale"] * (chosen / total if case["renorm"] else chosen)
    r = {"ids": torch.where(keep, ids, -1).int(), "weights": w * keep}
    if case["grad"]:
        dw = s["dweights"]
        if case["renorm"]:
            mean = (dw * chosen).sum(dim=1, keepdim=True) / total
            dp = case["scale"] * (dw - mean) / total
        else:
            dp = case["scale"] * dw
        if case["score"] == "sigmoid":
            dz = torch.zeros_like(p).scatter(1, ids, dp * chosen * (1 - chosen))
        else:
            mean = (dp * chosen).sum(dim=1, keepdim=True)
            dz = p * (torch.zeros_like(p).scatter(1, ids, dp) - mean)
            if case["renorm"]:                  # the mean is 0
                dz = torch.zeros_like(p).scatter(1, ids, chosen * dp)
        r["dlogits"] = (dz * keep).to(s["logits"].dtype)
    return r


def _combine(s, case):
    there = (s["ids"] >= 0)[..., None]
    y = torch.where(there, s["y"].float(), 0.0)
    w = torch.where(there, s["weights"][..., None], 0.0)
    out = (w * y).sum(dim=1)
    if s["add"] is not None:
        out = out + s["add"].float()
    r = {"out": out.to(s["out"].dtype)}
    if case["grad"]:
        dout = s["dout"].float()[:, None, :]
        r["dy"] = (w * dout).to(s["y"].dtype)
        r["dweights"] = (y * dout).sum(dim=2)
    return r


def _norm(s, case):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    v = h.float()
    inv = (1 / torch.sqrt(v.double().square().mean(dim=1, keepdim=True) + EPS)).float()
    y = v * inv * s["weight"].float()
    codes, scales = _package(y, 1)
    r = {"codes": codes, "scales": scales}
    if s["residual"] is not None:
        r["h"] = h
    if case["normed"]:
        r["normed"] = y.to(s["x"].dtype)
    return r


def _experts(s, case):
    """Each expert's rows padded to whole tiles of B slots, one product a tile."""
    M, top_k, E, K = case["M"], case["top_k"], case["E"], case["K"]
    pairs = M * top_k
    B = 16 if pairs <= 16 * E else 128
    flat = s["ids"].flatten().long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(dim=0)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    order = torch.sort(flat, stable=True).indices
    tiles = -(-counts // B)
    ends = tiles.cumsum(0)
    t = torch.arange(pairs // B + E, device=flat.device)
    e = torch.searchsorted(ends, t, right=True).clamp(max=E - 1)
    row = (t - (ends - tiles)[e])[:, None] * B + torch.arange(B, device=flat.device)
    there = (row < counts[e][:, None]) & (t < ends[-1])[:, None]
    slot = order[torch.where(there, offsets[e][:, None] + row, 0)]
    x = _decode(s["x_codes"], s["x_scales"], K, 1)[slot // top_k] * there[..., None]
    w = _decode(s["codes"], s["scales"], K, 128).transpose(1, 2).contiguous()
    y = torch.bmm(x, w[e])
    if s["bias"] is not None:
        y = y + s["bias"][e][:, None, :]
    whole = y.new_full((pairs + 1, case["N"]), float("nan"))
    whole[torch.where(there, slot, pairs)] = y
    return {"y": whole[:pairs].view(M, top_k, -1).to(s["y"].dtype), "counts": counts.int(), "offsets": offsets.int(),
            "order": order.int()}


def _matmul(s, case):
    K = case["K"]
    codes, scales = (s["x_codes"], s["x_scales"]) if case["packed"] else _package(s["x"], 1)
    y = _decode(codes, scales, K, 1) @ _decode(s["codes"], s["scales"], K, 128).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["y"].dtype)


_PLAIN = {"gate": _gate, "combine": _combine, "norm": _norm, "experts": _experts, "matmul": _matmul}


# ---------------------------------------------------- the library's calls


def _calls(s, case):
    import decode_matmul_amd as dmm
    op, M = case["op"], case["M"]
    if op == "gate":
        dmm.moe_gate(s["logits"], s["ids"], s["weights"], score=case["score"], bias=s["bias"],
                     n_groups=case["groups"], top_groups=case["top_groups"], group_top=case["group_top"],
                     renorm=case["renorm"], scale=case["scale"], token_mask=s["mask"])
        if not case["grad"]:
            return {"ids": s["ids"], "weights": s["weights"]}
        dmm.moe_gate_grad(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=case["score"],
                          renorm=case["renorm"], scale=case["scale"])
        return {"ids": s["ids"], "weights": s["weights"], "dlogits": s["dlogits"]}
    if op == "combine":
        dmm.moe_combine(s["y"], s["ids"], s["weights"], case["E"], s["out"], add=s["add"])
        if not case["grad"]:
            return {"out": s["out"]}
        dmm.moe_combine_grad(s["y"], s["ids"], s["weights"], case["E"], s["dout"], s["dy"], s["dweights"])
        return {"out": s["out"], "dy": s["dy"], "dweights": s["dweights"]}
    if op == "norm":
        dmm.f8_norm_pack(s["x"], s["weight"], s["codes"], s["scales"], EPS, residual=s["residual"], h_out=s["h"],
                         y_out=s["normed"])
        r = {"codes": s["codes"], "scales": s["scales"]}
        if s["h"] is not None:
            r["h"] = s["h"]
        if s["normed"] is not None:
            r["normed"] = s["normed"]
        return r
    N, K = case["N"], case["K"]
    if op == "matmul":
        if not case["packed"]:
            dmm.f8_pack(s["x"], s["x_codes"], s["x_scales"])
        dmm.f8_matmul(s["x_codes"], s["x_scales"], M, K, s["codes"], s["scales"], N, s["y"], bias=s["bias"])
        return s["y"]
    E, top_k = case["E"], case["top_k"]
    nbytes = dmm.moe_route_workspace_bytes(M, top_k, E)
    if nbytes and "route_ws" not in s:          # a workspace that the program keeps from its first pass on
        s["route_ws"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    dmm.moe_route(s["ids"], E, s["counts"], s["offsets"], s["order"], workspace=s.get("route_ws"))
    dmm.f8_matmul_experts(s["x_codes"], s["x_scales"], M, K, s["codes"], s["scales"], N, s["y"], E, s["offsets"],
                          s["order"], top_k, bias=s["bias"])
    return {"y": s["y"], "counts": s["counts"], "offsets": s["offsets"], "order": s["order"]}


def run(state):
    if own:
        return _calls(state, state["case"])
    return _PLAIN[state["case"]["op"]](state, state["case"])


# ------------------------------------------------------------ what it needs


def work(case):
    op, M = case["op"], case["M"]
    size = {"float32": 4, "bfloat16": 2}
    if op == "gate":
        E, top_k, z = case["E"], case["top_k"], size[case["dtype"]]
        moved = M * E * z + M * (8 * top_k + 1)
        if case["grad"]:
            dense = case["score"] == "softmax" and not case["renorm"]
            moved += M * E * z + M * 8 * top_k + (M * E * z if dense else M * top_k * z)
        return {"bytes": moved, "flops": 8 * M * E}
    if op == "combine":
        N, top_k, y, o = case["N"], case["top_k"], size[case["rows"]], size[case["out"]]
        live = (M - case["idle"]) * top_k * N
        moved = live * y + M * N * o * (2 if case["add"] else 1) + M * 8 * top_k
        if case["grad"]:
            moved += live * y + M * N * o + M * top_k * N * y + M * 12 * top_k
        return {"bytes": moved, "flops": live * (5 if case["grad"] else 2)}
    K = case["K"]
    nb = -(-K // 128)
    if op == "norm":
        x = size[case["dtype"]]
        each = 1 + 2 * bool(case["residual"]) + bool(case["normed"])
        return {"bytes": M * K * x * each + K * x + M * nb * 132, "flops": 8 * M * K}
    N = case["N"]
    package = N * nb * 128 + -(-N // 128) * nb * 4
    rows, touched = M, 1.0
    if op == "experts":
        live = M - case["idle"]
        rows = live * case["top_k"]
        touched = case["E"] * (1 - (1 - case["top_k"] / case["E"]) ** live)
    x = M * nb * 132 if case.get("packed", True) else M * K * 2
    moved = package * touched + x + M * case.get("top_k", 1) * N * size[case["out"]]
    return {"bytes": int(moved), "flops": 2 * rows * N * K}


# ------------------------------------------------ the definitions in 64 bits


def _nearest64(v):
    """The e4m3 values nearest to v (at most 448 in magnitude), ties to the even one."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _blocks64(y):
    """Each row's blocks of 128 as (e4m3 values [rows, blocks, 128], scales [rows, blocks])."""
    rows, K = y.shape
    nb = -(-K // 128)
    values = torch.zeros((rows, nb * 128), dtype=torch.float64, device=y.device)
    scales = torch.zeros((rows, nb), dtype=torch.float64, device=y.device)
    for b in range(nb):
        part = y[:, b * 128:min(K, b * 128 + 128)]
        most = (part.abs().max(dim=1).values / 448).clamp(min=2.0 ** -126)
        scales[:, b] = torch.exp2(torch.ceil(torch.log2(most)))
        values[:, b * 128:b * 128 + part.shape[1]] = _nearest64(part / scales[:, b:b + 1])
    return values.view(rows, nb, 128), scales


def _dense64(codes, scales, K):
    """A weight package's values: one scale for each 128 x 128."""
    v = codes.double()
    for r in range(0, v.shape[0], 128):
        v[r:r + 128] *= scales[r // 128].double()[None, :, None]
    return v.flatten(1)[:, :K]


def _gate64(s, case):
    E, groups = case["E"], case["groups"]
    size = E // groups
    z = s["logits"].double().requires_grad_(case["grad"])
    p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, dim=1)
    with torch.no_grad():
        c = z.detach() if s["bias"] is None else p + s["bias"].double()
        of = (p if s["bias"] is None and case["group_top"] == 2 else c).detach()
        open_ = torch.ones_like(c, dtype=torch.bool)
        if groups > 1:
            score = torch.stack([of[:, h * size:(h + 1) * size].topk(case["group_top"], dim=1).values.sum(dim=1)
                                 for h in range(groups)], dim=1)
            for h in range(groups):             # a group stays if fewer than top_groups come before it
                ahead = (score > score[:, h:h + 1]).sum(dim=1) + (score[:, :h] == score[:, h:h + 1]).sum(dim=1)
                open_[:, h * size:(h + 1) * size] = (ahead < case["top_groups"])[:, None]
        c = torch.where(open_, c, float("-inf"))
        ids = []
        for _ in range(case["top_k"]):          # the largest that is left, the first of equal ones
            first = (c == c.max(dim=1, keepdim=True).values).int().argmax(dim=1)
            ids.append(first)
            c = c.scatter(1, first[:, None], float("-inf"))
        ids = torch.stack(ids, dim=1)
    keep = s["mask"].bool()[:, None]
    chosen = torch.gather(p, 1, ids)
    w = case["scale"] * (chosen / chosen.sum(dim=1, keepdim=True) if case["renorm"] else chosen) * keep
    r = {"ids": None, "weights": w.detach()}
    if case["grad"]:
        (w * s["dweights"].double()).sum().backward()
        r["dlogits"] = z.grad
    return r


def exact(case, seed):
    s = prepare(case, seed)
    op, M = case["op"], case["M"]
    if op == "gate":
        return _gate64(s, case)
    if op == "combine":
        y, w = s["y"].double(), s["weights"].double().clone()
        none = s["ids"] < 0
        y[none], w[none] = 0.0, 0.0
        out = torch.zeros((M, case["N"]), dtype=torch.float64, device=DEV) if s["add"] is None else s["add"].double()
        for j in range(case["top_k"]):
            out = out + w[:, j:j + 1] * y[:, j]
        if not case["grad"]:
            return {"out": out}
        dout = s["dout"].double()
        return {"out": out, "dy": torch.stack([w[:, j:j + 1] * dout for j in range(case["top_k"])], dim=1),
                "dweights": torch.stack([(y[:, j] * dout).sum(dim=1) for j in range(case["top_k"])], dim=1)}
    K = case["K"]
    if op == "norm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        # the norm is of the sum as it is stored, and its factor and product are fp32
        v = h.to(s["x"].dtype).double()
        factor = (v.pow(2).sum(dim=1, keepdim=True) / K + EPS).pow(-0.5).float().double()
        y = (v * factor).float().double() * s["weight"].double()
        values, scales = _blocks64(y.float().double())
        r = {"codes": values, "scales": scales}
        if s["residual"] is not None:
            r["h"] = h
        if case["normed"]:
            r["normed"] = y
        return r
    if case.get("packed", True):
        x = (s["x_codes"].double() * s["x_scales"].double()[..., None]).flatten(1)[:, :K]
    else:
        values, scales = _blocks64(s["x"].double())
        x = (values * scales[..., None]).flatten(1)[:, :K]
    if op == "matmul":
        y = torch.matmul(x, _dense64(s["codes"], s["scales"], K).t())
        return y if s["bias"] is None else y + s["bias"].double()
    ids = s["ids"].flatten().long()
    y = torch.full((ids.numel(), case["N"]), float("nan"), dtype=torch.float64, device=ids.device)
    for e in range(case["E"]):
        at = torch.nonzero(ids == e).flatten()
        y[at] = x[at // case["top_k"]] @ _dense64(s["codes"][e], s["scales"][e], K).t()
        if s["bias"] is not None:
            y[at] += s["bias"][e].double()
    return {"y": y.view(M, case["top_k"], -1), "counts": None, "offsets": None, "order": None}
