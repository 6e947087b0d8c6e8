"""Expert routing and 8-bit integer expert products: the cases that are measured, their
inputs, the plain form of every operator in elementary torch operations, its definition in
64 bits, and the calls of the library.

    gate            logits [T][E] -> experts [T][topk] and their weights
    gate_backward   gradient of the weights -> gradient of the logits
    quantize        activations [M][K] -> int8 codes and one fp32 scale per row
    permute         the same for routed tokens, written into the contiguous expert layout
    dense / contiguous / masked
                    D[m][n] = sa[m] * sb[n] * sum_k A[m][k] * B[n][k], int8 operands

`own` selects what `run` does: False computes the plain form, True calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = "bf16", "fp32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step: a softmax router over 64 experts, its weights as they are
        dict(name="gate_1x64_softmax", op="gate", T=1, E=64, topk=6, dtype=BF16, score="softmax", bias=False,
             n_group=1, topk_group=1, group_top=1, renormalize=False, scale=1.0, padded=0.0),
        # a prompt's batch through a group-limited sigmoid router with a balance bias; some tokens are padding
        dict(name="gate_16384x256_groups", op="gate", T=16384, E=256, topk=8, dtype=F32, score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_top=2, renormalize=True, scale=2.5, padded=0.01),
        # a small training batch: softmax weights that are not renormalised have a dense gradient
        dict(name="gate_grad_777x60_softmax", op="gate_backward", T=777, E=60, topk=4, dtype=BF16, score="softmax",
             renormalize=False, scale=1.0, padded=0.0),
        # a large training batch of the group-limited router: zero but for the chosen experts
        dict(name="gate_grad_16384x256_sigmoid", op="gate_backward", T=16384, E=256, topk=8, dtype=F32,
             score="sigmoid", renormalize=True, scale=2.5, padded=0.01),
        # activations of a decode batch
        dict(name="quantize_64x7168", op="quantize", M=64, K=7168, dtype=BF16),
        # activations of a long prompt
        dict(name="quantize_32768x7168", op="quantize", M=32768, K=7168, dtype=BF16),
        # a decode batch spread over many experts
        dict(name="permute_64x2048_top8_of_256", op="permute", T=64, K=2048, E=256, topk=8, dtype=BF16, unrouted=0.0),
        # a prompt's batch over few experts
        dict(name="permute_16384x7168_top2_of_8", op="permute", T=16384, K=7168, E=8, topk=2, dtype=BF16,
             unrouted=0.02),
        # decode through a dense layer: bound by reading the weights
        dict(name="dense_64x7168x2048", op="dense", M=64, N=7168, K=2048, out=BF16),
        # a prompt through a dense layer, its row count not a multiple of any tile, summed further in fp32
        dict(name="dense_4097x7168x2048_fp32", op="dense", M=4097, N=7168, K=2048, out=F32),
        # a prompt through 8 experts, ragged segments padded to 128 rows and spare rows at the end
        dict(name="contiguous_8x32768x4096x7168", op="contiguous", G=8, rows=32768, N=4096, K=7168),
        # a decode batch over 16 experts with room for 256 rows each
        dict(name="masked_16x256x7168x2048", op="masked", G=16, M=256, N=7168, K=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate_backward", "quantize", "permute", "dense", "contiguous", "masked"])
    dtype = rng.choice([BF16, F32])
    if op in ("gate", "gate_backward"):
        n_group = rng.choice([1, 1, 2, 4, 8]) if op == "gate" else 1
        size = _log(rng, 2, 256 // n_group)
        E = n_group * size
        topk_group = rng.randint(1, n_group)
        renormalize = rng.random() < 0.5
        # a single renormalised weight is constant: its gradient is zero but for rounding
        least = 2 if op == "gate_backward" and renormalize else 1
        case = dict(op=op, T=_log(rng, 1, 16384), E=E, topk=rng.randint(least, min(8, topk_group * size)),
                    dtype=dtype, score=rng.choice(["softmax", "sigmoid"]), renormalize=renormalize,
                    scale=rng.choice([1.0, 2.5]), padded=rng.choice([0.0, 0.02]))
        if op == "gate":
            case.update(bias=rng.random() < 0.5, n_group=n_group, topk_group=topk_group,
                        group_top=rng.choice([1, 2]))
        return case
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 16384), K=16 * _log(rng, 1, 448), dtype=dtype)
    if op == "permute":
        E = _log(rng, 1, 256)
        return dict(op=op, T=_log(rng, 1, 8192), K=16 * _log(rng, 8, 448), E=E, topk=rng.randint(1, min(E, 4)),
                    dtype=dtype, unrouted=rng.choice([0.0, 0.1]))
    N, K = 16 * _log(rng, 1, 448), 16 * _log(rng, 1, 448)
    if op == "dense":
        return dict(op=op, M=_log(rng, 1, 8192), N=N, K=K, out=dtype)
    G = _log(rng, 1, 16)
    if op == "contiguous":
        return dict(op=op, G=G, rows=_log(rng, 1, 8192), N=N, K=K)
    return dict(op=op, G=G, M=_log(rng, 1, 512), N=N, K=K)


# ------------------------------------------------------------------ inputs

def _logits(g, c):
    """Router logits; a padded token's row is masked everywhere."""
    x = 1.5 * torch.randn(c["T"], c["E"], generator=g, device=DEV)
    x[torch.rand(c["T"], generator=g, device=DEV) < c["padded"]] = -math.inf
    return x.to(TYPES[c["dtype"]])


def _activations(g, rows, K, dtype):
    """Normal values with a spread of row magnitudes and a few channels far above the others."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    x *= torch.exp(torch.randn(rows, 1, generator=g, device=DEV))
    x *= 1 + 15 * (torch.rand(K, generator=g, device=DEV) < 0.01)
    return x.to(TYPES[dtype])


def _codes(g, *shape):
    """Normal values in 8 bits with a scale for each row, the largest value of a row at about 127."""
    top = math.sqrt(2 * math.log(max(2, shape[-1])))
    q = torch.empty(shape, dtype=torch.int8, device=DEV)
    for part in q.reshape(-1, shape[-1]).split(16384):
        x = torch.randn(part.shape, generator=g, device=DEV)
        part.copy_((x * (127 / top)).round_().clamp_(-127, 127))
    s = torch.rand(shape[:-1], generator=g, device=DEV).add_(0.5).mul_(top / 127 / math.sqrt(shape[-1]))
    return q, s


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": dict(c)}
    if c["op"] == "gate":
        st["logits"] = _logits(g, c)
        st["bias"] = 0.05 * torch.randn(c["E"], generator=g, device=DEV) if c["bias"] else None
        st["ids"] = torch.empty(c["T"], c["topk"], dtype=torch.int32, device=DEV)
        st["weights"] = torch.empty(c["T"], c["topk"], device=DEV)
    elif c["op"] == "gate_backward":
        st["logits"] = _logits(g, c)
        noisy = st["logits"].float() + 0.05 * torch.randn(c["E"], generator=g, device=DEV)
        top = torch.topk(noisy, c["topk"], dim=1)
        st["ids"] = torch.where(top.values == -math.inf, -1, top.indices).to(torch.int32)
        st["d_weights"] = torch.randn(c["T"], c["topk"], generator=g, device=DEV)
        st["d_logits"] = torch.empty_like(st["logits"])
    elif c["op"] == "quantize":
        st["x"] = _activations(g, c["M"], c["K"], c["dtype"])
        st["q"] = torch.empty(c["M"], c["K"], dtype=torch.int8, device=DEV)
        st["scale"] = torch.empty(c["M"], device=DEV)
    elif c["op"] == "permute":
        T, E, topk = c["T"], c["E"], c["topk"]
        st["x"] = _activations(g, T, c["K"], c["dtype"])
        popular = torch.arange(1, E + 1, device=DEV).float().log().neg()   # some experts are chosen more often
        noise = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-6, 1 - 1e-6)
        ids = torch.topk(popular - torch.log(-torch.log(noise)), topk, dim=1).indices.to(torch.int32)
        ids[torch.rand(T, topk, generator=g, device=DEV) < c["unrouted"]] = -1
        cap = -(-(T * topk + 127 * E) // 128) * 128
        st["topk_ids"] = ids
        st["out"] = {"a": torch.zeros(cap, c["K"], dtype=torch.int8, device=DEV),
                     "sa": torch.zeros(cap, device=DEV),
                     "m_indices": torch.zeros(cap, dtype=torch.int32, device=DEV),
                     "src_of": torch.zeros(cap, dtype=torch.int32, device=DEV),
                     "row_of": torch.zeros(T, topk, dtype=torch.int32, device=DEV)}
    elif c["op"] == "dense":
        st["a"], st["sa"] = _codes(g, c["M"], c["K"])
        st["b"], st["sb"] = _codes(g, c["N"], c["K"])
        st["d"] = torch.empty(c["M"], c["N"], dtype=TYPES[c["out"]], device=DEV)
    elif c["op"] == "contiguous":
        G, rows = c["G"], c["rows"]
        share = torch.rand(G, generator=g, device=DEV) + 0.5
        expert = torch.multinomial(share, rows, replacement=True, generator=g)
        counts = torch.bincount(expert, minlength=G).tolist()
        total = -(-(rows + 127 * G) // 128) * 128
        idx = torch.full((total,), -1, dtype=torch.int32)
        at, first = 0, []
        for e, n in enumerate(counts):
            idx[at:at + n] = e
            first.append(at)
            at += -(-n // 128) * 128
        st["a"], st["sa"] = _codes(g, total, c["K"])
        st["b"], st["sb"] = _codes(g, G, c["N"], c["K"])
        st["m_indices"] = idx.to(DEV)
        st["d"] = torch.zeros(total, c["N"], dtype=torch.bfloat16, device=DEV)
        # the plan of the plain form: every expert's rows, padded to the longest segment
        most = max(counts)
        r = torch.arange(most)
        pad = torch.tensor(first)[:, None] + r[None, :]
        ok = r[None, :] < torch.tensor(counts)[:, None]
        st["segment"] = torch.where(ok, pad, 0).to(DEV)
        st["filled"] = ok.reshape(-1).nonzero()[:, 0].to(DEV)
        st["row"] = pad[ok].to(DEV)
    elif c["op"] == "masked":
        st["a"], st["sa"] = _codes(g, c["G"], c["M"], c["K"])
        st["b"], st["sb"] = _codes(g, c["G"], c["N"], c["K"])
        st["masked_m"] = torch.randint(0, c["M"] + 1, (c["G"],), generator=g, device=DEV).to(torch.int32)
        st["masked_m"][0] = c["M"]
        st["d"] = torch.zeros(c["G"], c["M"], c["N"], dtype=torch.bfloat16, device=DEV)
    return st


# ------------------------------------------------------------------ the plain forms

def _scores64(logits, score):
    """Scores in 64 bits: the choice of experts compares values that may be next to one another."""
    l = logits.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def _gate(st):
    c, logits, bias = st["case"], st["logits"], st["bias"]
    T, E = logits.shape
    masked = logits == -math.inf
    if bias is None:
        key = logits.double()
        if c["n_group"] > 1 and c["group_top"] > 1:
            rank = _scores64(logits, c["score"])
        else:
            rank = key
    else:
        masked = masked | (bias == -math.inf)
        key = rank = _scores64(logits, c["score"]) + bias.double()
    key = torch.where(masked, -math.inf, key)
    if c["n_group"] > 1:
        rank = torch.where(masked, -math.inf, rank).view(T, c["n_group"], -1)
        best = torch.sort(rank, dim=2, descending=True).values[:, :, :c["group_top"]]
        total = torch.where(best == -math.inf, 0.0, best).sum(2)
        total = torch.where(best[:, :, 0] == -math.inf, -math.inf, total)
        order = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        kept = torch.zeros(T, c["n_group"], dtype=torch.bool, device=key.device).scatter_(1, order, True)
        key = torch.where(kept[:, :, None].expand_as(rank).reshape(T, E), key, -math.inf)
    chosen = torch.sort(key, dim=1, descending=True, stable=True)
    ids = chosen.indices[:, :c["topk"]]
    none = chosen.values[:, :c["topk"]] == -math.inf
    l = torch.where(none, -math.inf, logits.float().gather(1, ids))
    if c["renormalize"]:
        top = l.amax(1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        if c["score"] == "sigmoid":
            low = torch.clamp(top, max=0.0)
            t = torch.where(l < 0, torch.exp(l - low) / (1 + torch.exp(l)), torch.exp(-low) / (1 + torch.exp(-l)))
        else:
            t = torch.exp(l - top)
        total = t.sum(1, keepdim=True)
        w = t / torch.where(total == 0, 1.0, total)
    elif c["score"] == "sigmoid":
        w = 1 / (1 + torch.exp(-l))
    else:
        full = logits.float()
        top = full.amax(1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        total = torch.exp(full - top).sum(1, keepdim=True)
        w = torch.exp(l - top) / torch.where(total == 0, 1.0, total)
    return {"ids": torch.where(none, -1, ids).to(torch.int32), "weights": torch.where(none, 0.0, c["scale"] * w)}


def _gate_backward(st):
    c, logits = st["case"], st["logits"].float()
    ids, g = st["ids"].long(), st["d_weights"]
    none = ids < 0
    at = ids.clamp(min=0)
    l = torch.where(none, -math.inf, logits.gather(1, at))
    g = torch.where(none, 0.0, g)
    sig = 1 / (1 + torch.exp(-l))
    if c["renormalize"]:
        top = l.amax(1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        if c["score"] == "sigmoid":
            low = torch.clamp(top, max=0.0)
            t = torch.where(l < 0, torch.exp(l - low) / (1 + torch.exp(l)), torch.exp(-low) * sig)
            slope = 1 / (1 + torch.exp(l))
        else:
            t, slope = torch.exp(l - top), 1.0
        total = t.sum(1, keepdim=True)
        r = t / torch.where(total == 0, 1.0, total)
        v = c["scale"] * r * slope * (g - (r * g).sum(1, keepdim=True))
    elif c["score"] == "sigmoid":
        v = c["scale"] * sig * (1 / (1 + torch.exp(l))) * g
    else:
        top = logits.amax(1, keepdim=True)
        e = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
        total = e.sum(1, keepdim=True)
        p = e / torch.where(total == 0, 1.0, total)
        dense = torch.zeros_like(p).scatter_add_(1, at, g)
        return (c["scale"] * p * (dense - (p * dense).sum(1, keepdim=True))).to(st["logits"].dtype)
    v = torch.where(none, 0.0, v)
    return torch.zeros_like(logits).scatter_add_(1, at, v).to(st["logits"].dtype)


LEAST = 2.0 ** -126


def _quantize(x):
    """scale = fp32(amax / 127), codes = the integers nearest to x * fp32(127 / amax), the product not rounded."""
    x = x.float()
    amax = x.abs().amax(1, keepdim=True)
    tiny = amax < 127 * LEAST
    top = torch.full_like(amax, 127.0)      # as a tensor: by a number, torch multiplies with a rounded reciprocal
    scale = torch.where(amax == 0, 1.0, torch.where(tiny, LEAST, amax / top))
    inverse = torch.where(amax == 0, 1.0, torch.where(tiny, 1 / LEAST, top / torch.where(tiny, 1.0, amax)))
    return (x.double() * inverse.double()).round().to(torch.int8), scale[:, 0]


def _permute(st):
    c, ids = st["case"], st["topk_ids"].reshape(-1).long()
    T, E, topk = c["T"], c["E"], c["topk"]
    cap = st["out"]["a"].shape[0]
    q, scale = _quantize(st["x"])
    # slots by expert, in slot order; unrouted ones go behind the last expert
    expert = torch.where(ids < 0, E, ids)
    order = torch.sort(expert, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, expert, torch.ones_like(expert))
    padded = (counts[:E] + 127) // 128 * 128
    first = torch.cat([padded.cumsum(0) - padded, torch.full_like(padded[:1], cap)])
    rank = torch.empty_like(order).scatter_(0, order, torch.arange(len(order), device=ids.device))
    row = first[expert] + rank - (counts.cumsum(0) - counts)[expert]
    token = torch.arange(T * topk, device=ids.device) // topk
    to = torch.where(ids < 0, cap, row)             # one spare row takes what is not routed
    a = torch.zeros(cap + 1, c["K"], dtype=torch.int8, device=ids.device)
    a[to] = q[token]
    sa = torch.zeros(cap + 1, device=ids.device)
    sa[to] = scale[token]
    m_indices = torch.full((cap + 1,), -1, dtype=torch.int32, device=ids.device)
    m_indices[to] = ids.to(torch.int32)
    src_of = torch.full((cap + 1,), -1, dtype=torch.int32, device=ids.device)
    src_of[to] = token.to(torch.int32)
    return {"a": a[:cap], "sa": sa[:cap], "m_indices": m_indices[:cap], "src_of": src_of[:cap],
            "row_of": torch.where(ids < 0, -1, row).to(torch.int32).view(T, topk)}


def _dense(st):
    out = torch.matmul(st["a"].float(), st["b"].float().t())
    return (out * st["sa"][:, None] * st["sb"]).to(st["d"].dtype)


def _contiguous(st):
    at = st["segment"]
    out = torch.bmm(st["a"].float()[at], st["b"].float().transpose(1, 2))
    out = (out * st["sa"][at][:, :, None] * st["sb"][:, None, :]).to(torch.bfloat16)
    d = torch.zeros_like(st["d"])
    d[st["row"]] = out.reshape(-1, out.shape[2])[st["filled"]]
    return d


def _masked(st):
    out = torch.bmm(st["a"].float(), st["b"].float().transpose(1, 2))
    out = (out * st["sa"][:, :, None] * st["sb"][:, None, :]).to(torch.bfloat16)
    row = torch.arange(out.shape[1], device=out.device)
    return torch.where(row[None, :, None] < st["masked_m"][:, None, None], out, torch.zeros_like(out))


PLAIN = {"gate": _gate, "gate_backward": _gate_backward, "permute": _permute, "dense": _dense,
         "contiguous": _contiguous, "masked": _masked}


# ------------------------------------------------------------------ one pass

def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "quantize":
            q, scale = _quantize(st["x"])
            return {"q": q, "scale": scale}
        return PLAIN[op](st)
    from moe_grouped_gemm_05_b200 import binding as dg

    if op == "gate":
        ids, weights = dg.moe_gate(st["logits"], c["topk"], st["bias"], score=c["score"], n_group=c["n_group"],
                                   topk_group=c["topk_group"], group_top=c["group_top"],
                                   renormalize=c["renormalize"], scale=c["scale"], ids=st["ids"],
                                   weights=st["weights"])
        return {"ids": ids, "weights": weights}
    if op == "gate_backward":
        return dg.moe_gate_backward(st["logits"], st["ids"], st["d_weights"], score=c["score"],
                                    renormalize=c["renormalize"], scale=c["scale"], d_logits=st["d_logits"])
    if op == "quantize":
        q, scale = dg.quantize_int8_per_token(st["x"], q=st["q"], scale=st["scale"])
        return {"q": q, "scale": scale}
    if op == "permute":
        return dg.moe_quantize_permute_int8(st["topk_ids"], c["E"], st["x"], out=st["out"])
    if op == "dense":
        return dg.int8_gemm_nt(st["a"], st["sa"], st["b"], st["sb"], d=st["d"])
    if op == "contiguous":
        return dg.m_grouped_int8_gemm_nt_contiguous(st["a"], st["sa"], st["b"], st["sb"], st["m_indices"], d=st["d"])
    return dg.m_grouped_int8_gemm_nt_masked(st["a"], st["sa"], st["b"], st["sb"], st["masked_m"], d=st["d"])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    size = 2 if c.get("dtype") == BF16 else 4
    if c["op"] == "gate":
        return {"bytes": c["T"] * (c["E"] * size + 8 * c["topk"]), "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "gate_backward":
        dense = c["score"] == "softmax" and not c["renormalize"]
        read = c["E"] if dense else c["topk"]
        return {"bytes": c["T"] * ((read + c["E"]) * size + 8 * c["topk"]), "flops": 4 * c["T"] * read}
    if c["op"] == "quantize":
        return {"bytes": c["M"] * (c["K"] * (size + 1) + 4), "flops": 2 * c["M"] * c["K"]}
    if c["op"] == "permute":
        slots = round(c["T"] * c["topk"] * (1 - c["unrouted"]))
        cap = -(-(c["T"] * c["topk"] + 127 * c["E"]) // 128) * 128
        return {"bytes": c["T"] * c["K"] * size + slots * c["K"] + 12 * cap + 8 * c["T"] * c["topk"],
                "flops": 2 * c["T"] * c["K"]}
    if c["op"] == "dense":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * (K + 4) + M * N * (2 if c["out"] == BF16 else 4), "flops": 2 * M * N * K}
    G, N, K = c["G"], c["N"], c["K"]
    rows = c["rows"] if c["op"] == "contiguous" else G * c["M"] / 2     # half of the room is used on average
    return {"bytes": (rows + G * N) * (K + 4) + rows * N * 2, "flops": 2 * rows * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_ids(st):
    """Experts by counting, for each, those that come before it."""
    c = st["case"]
    l = st["logits"].double()
    T, E = l.shape
    dead = torch.isneginf(l)
    prob = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    value = l
    if st["bias"] is not None:
        b = st["bias"].double()
        dead = dead | torch.isneginf(b)
        value = prob = prob + b
    gs = E // c["n_group"]
    ids = torch.full((T, c["topk"]), -1, dtype=torch.long, device=l.device)
    e = torch.arange(E, device=l.device)
    for t0 in range(0, T, 256):
        t = slice(t0, min(T, t0 + 256))
        out = dead[t].clone()
        if c["n_group"] > 1:
            key = value if c["group_top"] == 1 and st["bias"] is None else prob
            key = key[t].masked_fill(out, -math.inf).view(-1, c["n_group"], gs)
            two = torch.topk(key, min(c["group_top"], gs), dim=2).values
            total = two.masked_fill(torch.isneginf(two), 0.0).sum(2).masked_fill(torch.isneginf(two[:, :, 0]), -math.inf)
            gi = torch.arange(c["n_group"], device=l.device)
            before = (total[:, None, :] > total[:, :, None]) | ((total[:, None, :] == total[:, :, None])
                                                               & (gi[None, None, :] < gi[None, :, None]))
            out |= (before.sum(2) >= c["topk_group"]).repeat_interleave(gs, dim=1)
        key = value[t].masked_fill(out, -math.inf)
        before = (key[:, None, :] > key[:, :, None]) | ((key[:, None, :] == key[:, :, None])
                                                       & (e[None, None, :] < e[None, :, None]))
        place = before.sum(2)
        hit = (place < c["topk"]) & ~out
        rows, cols = hit.nonzero(as_tuple=True)
        ids[t][rows, place[rows, cols]] = cols
    return ids


def _exact_weights(logits, ids, c):
    """Weights of the chosen experts from 64-bit logits, as the definition has them."""
    none = ids < 0
    if c["score"] == "softmax":
        log_s = logits - torch.logsumexp(logits, 1, keepdim=True)
    else:
        log_s = torch.nn.functional.logsigmoid(logits)
    s = log_s.gather(1, ids.clamp(min=0)).masked_fill(none, -math.inf)
    w = torch.softmax(s, 1) if c["renormalize"] else torch.exp(s)
    return (c["scale"] * w).masked_fill(none, 0.0)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "gate":
        ids = _exact_ids(st)
        w = torch.zeros(ids.shape, dtype=torch.float64, device=ids.device)
        live = (ids >= 0).any(1)
        w[live] = _exact_weights(st["logits"].double()[live], ids[live], c)
        return {"ids": ids.to(torch.int32), "weights": w}
    if c["op"] == "gate_backward":
        ids = st["ids"].long()
        live = (ids >= 0).any(1)
        l = st["logits"].double()[live].requires_grad_(True)
        d = torch.zeros(st["logits"].shape, dtype=torch.float64, device=l.device)
        if live.any():
            w = _exact_weights(l, ids[live], c)
            d[live] = torch.autograd.grad((w * st["d_weights"].double()[live]).sum(), l)[0]
        return d
    if c["op"] in ("quantize", "permute"):
        scale = st["x"].double().abs().amax(1) / 127
        scale = torch.where(scale == 0, 1.0, scale.clamp(min=LEAST))
        if c["op"] == "quantize":
            return {"q": None, "scale": scale}
        sa = torch.zeros(st["out"]["sa"].shape, dtype=torch.float64, device=scale.device)
        ids = st["topk_ids"].long()
        at = 0
        for e in range(c["E"]):
            token = (ids == e).any(1).nonzero()[:, 0]
            sa[at:at + len(token)] = scale[token]
            at += -(-len(token) // 128) * 128
        return {"a": None, "sa": sa, "m_indices": None, "src_of": None, "row_of": None}
    a, b, sa, sb = st["a"].double(), st["b"], st["sa"].double(), st["sb"].double()
    if c["op"] == "dense":
        return (a * sa[:, None]) @ (b.double() * sb[:, None]).t()
    d = torch.zeros(st["d"].shape, dtype=torch.float64, device=a.device)
    for e in range(c["G"]):
        w = (b[e].double() * sb[e][:, None]).t()
        if c["op"] == "masked":
            n = int(st["masked_m"][e])
            d[e, :n] = (a[e, :n] * sa[e, :n, None]) @ w
        else:
            rows = (st["m_indices"] == e).nonzero()[:, 0]
            d[rows] = (a[rows] * sa[rows][:, None]) @ w
    return d
