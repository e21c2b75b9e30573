"""Timed cases of the training and 4-bit expert operators.

Four operators of one MoE layer around the token path:

- ``balance``  moe_balance_loss: balance and z loss of a router, per-expert counts;
- ``route``    moe_route_backward: gradient of the routing weights and of both losses in the logits;
- ``combine``  moe_combine_backward: gradient of the weighted combine in the expert rows and weights;
- ``experts``  moe_expert_product_w4: the experts' products with 4-bit weights and group scales, plain
  or gated (silu(gate) * up).

``run`` computes them in elementary torch operations in 32 bits, or with ``own`` through the
framework's calls.  ``exact`` holds the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_E2M1_MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def listed():
    return [
        # the smallest training batch of the repository's configurations: latency
        {"name": "balance_tiny", "op": "balance", "S": 1, "T": 128, "E": 16, "k": 2,
         "dtype": "f32", "mask": False},
        # eight sources of a prefill batch with skewed popularity and padded tails
        {"name": "balance_skewed", "op": "balance", "S": 8, "T": 4096, "E": 384, "k": 6,
         "dtype": "f32", "mask": True},
        # one source of the prefill batch
        {"name": "route_prefill", "op": "route", "S": 1, "T": 4096, "E": 384, "k": 6,
         "dtype": "f32", "mask": False},
        # the large batch in four padded sources, a router that computes in bf16
        {"name": "route_large_bf16", "op": "route", "S": 4, "T": 4096, "E": 64, "k": 8,
         "dtype": "bf16", "mask": True},
        {"name": "combine_tiny", "op": "combine", "T": 128, "H": 256, "k": 2, "share": 1.0,
         "spare": 0},
        # the prefill batch with every expert's rows in one memory
        {"name": "combine_prefill", "op": "combine", "T": 4096, "H": 5120, "k": 6, "share": 1.0,
         "spare": 0},
        # the large batch seen by one of eight partitions, run padding among its rows
        {"name": "combine_part", "op": "combine", "T": 16384, "H": 2048, "k": 8, "share": 0.125,
         "spare": 500},
        # one token's six experts: a single-stream decode step
        {"name": "experts_token", "op": "experts", "E": 48, "rows": 6, "skew": 0.0, "K": 5120,
         "N": 2048, "gated": True, "layout": "runs", "align": 1},
        # one partition of the 64-token decode batch, receive blocks of 64 rows
        {"name": "experts_decode", "op": "experts", "E": 48, "rows": 48, "skew": 0.0, "K": 5120,
         "N": 2048, "gated": True, "layout": "blocks", "align": 64},
        # the second product of a decode step that eight ranks feed
        {"name": "experts_down", "op": "experts", "E": 48, "rows": 384, "skew": 0.5, "K": 2048,
         "N": 5120, "gated": False, "layout": "runs", "align": 1},
        # sizes off every tile, runs padded to 8 rows
        {"name": "experts_odd", "op": "experts", "E": 5, "rows": 37, "skew": 1.0, "K": 1040,
         "N": 328, "gated": True, "layout": "runs", "align": 8},
        # one partition of the large batch: thousands of rows an expert
        {"name": "experts_large", "op": "experts", "E": 8, "rows": 16384, "skew": 0.2, "K": 2048,
         "N": 1408, "gated": True, "layout": "runs", "align": 1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng: random.Random):
    op = rng.choice(["balance", "route", "combine", "experts", "experts"])
    if op in ("balance", "route"):
        S, E = rng.randint(1, 8), _log_int(rng, 2, 1024)
        T = min(_log_int(rng, 1, 16384), max(1, 12_000_000 // (S * E)))
        return {"op": op, "S": S, "T": T, "E": E, "k": rng.randint(1, min(E, 10)),
                "dtype": rng.choice(["f32", "f32", "bf16"]), "mask": rng.random() < 0.5}
    if op == "combine":
        H = 8 * _log_int(rng, 4, 900)
        k = rng.randint(1, 10)
        T = min(_log_int(rng, 1, 16384), max(1, 120_000_000 // (H * k)))
        return {"op": op, "T": T, "H": H, "k": k, "share": rng.choice([1.0, 1.0, 0.5, 0.125]),
                "spare": rng.randint(0, 300)}
    gated = rng.random() < 0.5
    K, N = 16 * _log_int(rng, 4, 448), 8 * _log_int(rng, 4, 512)
    E = min(_log_int(rng, 1, 64), max(1, 600_000_000 // (K * N * (2 if gated else 1))))
    flops_a_row = 2 * K * N * (2 if gated else 1)
    rows = min(_log_int(rng, 1, 12000), max(1, int(1.2e11) // flops_a_row))
    layout = rng.choice(["runs", "runs", "blocks"])
    case = {"op": op, "E": E, "rows": rows, "skew": round(rng.uniform(0, 0.8), 2), "K": K, "N": N,
            "gated": gated, "layout": layout, "align": rng.choice([1, 1, 8, 16])}
    if layout == "blocks":
        case["align"] = max(_counts(case)) + rng.randint(0, 9)
    return case


def _counts(case):
    """Rows of each expert: `rows` picks, expert popularity (rank + 1)^-skew in shuffled order."""
    E, rows = case["E"], case["rows"]
    rng = random.Random(f"{E} {rows} {case['skew']} {case['K']} {case['N']}")
    weight = [(i + 1.0) ** -case["skew"] for i in range(E)]
    rng.shuffle(weight)
    counts = [0] * E
    for e in rng.choices(range(E), weights=weight, k=rows):
        counts[e] += 1
    return counts


def _starts(case):
    """First row of each expert and the row count of the whole receive buffer."""
    counts, align = _counts(case), case["align"]
    if case["layout"] == "blocks":
        return [e * align for e in range(case["E"])], case["E"] * align
    starts, at = [], 0
    for c in counts:
        starts.append(at)
        at += -(-c // align) * align
    return starts, at


def work(case):
    if case["op"] in ("balance", "route"):
        N, E, k = case["S"] * case["T"], case["E"], case["k"]
        b = 4 if case["dtype"] == "f32" else 2
        mask = N if case["mask"] else 0
        if case["op"] == "balance":   # logits, ids, mask -> counts, mean probabilities, lse
            return {"bytes": N * E * b + N * k * 4 + mask + case["S"] * E * 8 + N * 4,
                    "flops": 5 * N * E}
        # logits, ids, weights, their gradients, lse, counts, mask -> gradient of the logits
        return {"bytes": 2 * N * E * b + N * k * 12 + N * 4 + case["S"] * E * 4 + mask,
                "flops": 8 * N * E}
    if case["op"] == "combine":
        N, H, k = case["T"], case["H"], case["k"]
        R = round(case["share"] * N * k)
        tokens = N * (1 - (1 - case["share"]) ** k)
        # rows and their gradients, d_out, pair rows, weights and their gradients, recv_pair
        return {"bytes": 4 * R * H + 2 * case["spare"] * H + 2 * tokens * H + 12 * N * k
                + 4 * (R + case["spare"]), "flops": 4 * R * H}
    counts = _counts(case)
    active, rows = sum(c > 0 for c in counts), sum(counts)
    n = case["N"] * (2 if case["gated"] else 1)
    # codes and scales of the experts in use, rows in, rows out
    return {"bytes": active * n * case["K"] * 9 / 16 + 2 * rows * (case["K"] + case["N"])
            + 4 * active, "flops": 2 * rows * n * case["K"]}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _prepare_router(case, seed):
    g = _generator(seed)
    S, T, E, k = case["S"], case["T"], case["E"], case["k"]
    # router logits: noise of unit size over a popularity that a few experts lead
    bias = 1.5 * torch.rand(S, 1, E, generator=g, device="cuda").pow(4)
    logits = (torch.randn(S, T, E, generator=g, device="cuda") + bias).to(_DTYPES[case["dtype"]])
    top, ids = torch.topk(logits.float(), k, dim=-1)
    st = {"case": case, "logits": logits.contiguous(), "ids": ids.int().contiguous(),
          "w": torch.softmax(top, -1).contiguous(), "mask": None}
    if case["mask"]:                      # every source padded from some token on
        ends = (torch.rand(S, 1, generator=g, device="cuda") * T).ceil()
        st["mask"] = (torch.arange(T, device="cuda") < ends).to(torch.uint8).contiguous()
    if case["op"] == "balance":
        if own:
            import combine_moe_route_06_gb300 as moe
            f32, i32 = (dict(dtype=d, device="cuda") for d in (torch.float32, torch.int32))
            st.update(moe=moe, counts=torch.empty(S, E, **i32), prob=torch.empty(S, E, **f32),
                      lse=torch.empty(S, T, **f32), n_valid=torch.empty(S, **i32),
                      losses=torch.empty(2, **f32),
                      ws=torch.empty(moe.moe_balance_loss_workspace_bytes(S, T, E),
                                     dtype=torch.uint8, device="cuda"))
        return st
    out = _balance(st)                    # a training step keeps these from its forward pass
    st.update(lse=out["lse"], counts=out["counts"], n_valid=out["n_valid"],
              dw=torch.randn(S, T, k, generator=g, device="cuda") / 16,
              d_losses=torch.rand(2, generator=g, device="cuda") * 0.02)
    if own:
        import combine_moe_route_06_gb300 as moe
        st.update(moe=moe, d_logits=torch.empty_like(st["logits"]))
    return st


def _prepare_combine(case, seed):
    g = _generator(seed)
    N, H, k = case["T"], case["H"], case["k"]
    R = round(case["share"] * N * k)
    rows = R + case["spare"]
    y = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
    d_out = (torch.randn(N, H, generator=g, device="cuda") / 64).bfloat16()
    w = torch.softmax(torch.randn(N, k, generator=g, device="cuda"), -1)
    pairs = torch.randperm(N * k, generator=g, device="cuda")[:R]
    places = torch.randperm(rows, generator=g, device="cuda")[:R].int()
    pair_row = torch.full((N * k,), -1, dtype=torch.int32, device="cuda")
    recv_pair = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    pair_row[pairs] = places
    recv_pair[places.long()] = pairs.int()
    st = {"case": case, "y": y, "d_out": d_out.view(1, N, H), "w": w.view(1, N, k).contiguous(),
          "pair_row": pair_row.view(1, N, k), "recv_pair": recv_pair}
    if own:
        import combine_moe_route_06_gb300 as moe
        st.update(moe=moe, d_y=torch.empty_like(y), dw=torch.empty_like(st["w"]))
    return st


def _quantize(w, factor):
    """Rows of normal weights as E2M1 codes (first value in the low nibble) and E4M3 group scales."""
    n, K = w.shape
    groups = w.view(n, K // 16, 16)
    s8 = (groups.abs().amax(-1) / (6 * factor)).to(torch.float8_e4m3fn)
    q = groups / (s8.float() * factor).clamp(min=1e-30).unsqueeze(-1)
    code = torch.bucketize(q.abs(), torch.tensor(_E2M1_MIDS, device="cuda"), out_int32=True)
    code = (code + 8 * (q < 0)).to(torch.uint8).view(n, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), s8.view(torch.uint8)


def _prepare_experts(case, seed):
    g = _generator(seed)
    E, K, N = case["E"], case["K"], case["N"]
    n = N * (2 if case["gated"] else 1)
    codes = torch.empty(E, n, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, n, K // 16, dtype=torch.uint8, device="cuda")
    factor = (0.8 + 0.4 * torch.rand(E, generator=g, device="cuda")) * 0.01 / math.sqrt(K)
    for e in range(E):
        w = torch.randn(n, K, generator=g, device="cuda") / math.sqrt(K)
        codes[e], scales[e] = _quantize(w, factor[e])
    counts = _counts(case)
    starts, rows = _starts(case)
    M = max(counts)
    counts_t = torch.tensor(counts, dtype=torch.int32, device="cuda")
    index = (torch.tensor(starts, device="cuda")[:, None] + torch.arange(M, device="cuda"))
    used = torch.arange(M, device="cuda") < counts_t[:, None]
    # hidden states of unit size with a few channels that stand out, zero rows as run padding
    a = torch.randn(rows, K, generator=g, device="cuda")
    a[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")] *= 12
    live = torch.zeros(rows, 1, device="cuda").index_fill_(0, index[used], 1.0)
    st = {"case": case, "a": (a * live).bfloat16(), "codes": codes, "scales": scales,
          "factor": factor, "index": index.clamp(max=rows - 1), "used": used, "rows": rows}
    if own:
        import combine_moe_route_06_gb300 as moe
        w4 = torch.empty(moe.moe_w4_bytes(E, N, K, case["gated"]), dtype=torch.uint8,
                         device="cuda")
        moe.moe_w4_pack(codes, scales, w4, gated=case["gated"])
        st.update(moe=moe, w4=w4, y=torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"),
                  ws=torch.empty(moe.moe_expert_product_w4_workspace_bytes(rows, E, N, K),
                                 dtype=torch.uint8, device="cuda"))
        if case["layout"] == "blocks":
            st["rows_by"] = {"masked_counts": counts_t, "block_rows": case["align"]}
        else:
            st["rows_by"] = {"expert_offsets": torch.tensor(starts + [rows], dtype=torch.int32,
                                                            device="cuda")}
    return st


def prepare(case, seed):
    if case["op"] == "combine":
        return _prepare_combine(case, seed)
    return _prepare_experts(case, seed) if case["op"] == "experts" else _prepare_router(case, seed)


# ---------------------------------------------------------------- plain forms

def _balance(st):
    E, k = st["case"]["E"], st["case"]["k"]
    logits, ids = st["logits"].float(), st["ids"].long()
    m = torch.ones_like(logits[..., 0]) if st["mask"] is None else st["mask"].float()
    n = m.sum(1)
    top = logits.max(-1, keepdim=True).values
    ex = (logits - top).exp()
    lse = ((top + ex.sum(-1, keepdim=True).log()).squeeze(-1)) * m
    prob = (ex / ex.sum(-1, keepdim=True) * m.unsqueeze(-1)).sum(1) / n.clamp(min=1).unsqueeze(-1)
    picks = m.unsqueeze(-1).expand(ids.shape).reshape(ids.shape[0], -1).int()
    counts = torch.zeros(prob.shape, dtype=torch.int32, device="cuda")
    counts = counts.scatter_add(1, ids.reshape(ids.shape[0], -1), picks)
    per = 1 / n.clamp(min=1)
    balance = (E / k * per * (counts.float() * prob).sum(-1)).mean()
    z = (per * lse.square().sum(1)).mean()
    return {"losses": torch.stack((balance, z)), "counts": counts, "prob_mean": prob, "lse": lse,
            "n_valid": n.int()}


def _route(st):
    S, E, k = st["case"]["S"], st["case"]["E"], st["case"]["k"]
    logits, ids = st["logits"].float(), st["ids"].long()
    m = torch.ones_like(logits[..., 0]) if st["mask"] is None else st["mask"].float()
    per = 1 / (S * st["n_valid"].clamp(min=1).float())
    p = (logits - st["lse"].unsqueeze(-1)).exp()
    lead = st["d_losses"][0] * E / k * (per / st["n_valid"].clamp(min=1))[:, None] * st["counts"]
    lead = lead.unsqueeze(1)
    grad = p * (lead - (lead * p).sum(-1, keepdim=True))
    grad = grad + p * (2 * st["d_losses"][1] * per[:, None] * st["lse"]).unsqueeze(-1)
    chosen = st["w"] * (st["dw"] - (st["w"] * st["dw"]).sum(-1, keepdim=True))
    return (grad.scatter_add(-1, ids, chosen) * m.unsqueeze(-1)).to(st["logits"].dtype)


def _combine(st):
    y, d_out = st["y"].float(), st["d_out"][0].float()
    N, k = st["w"].shape[1:]
    rows, have = st["pair_row"].view(-1).clamp(min=0).long(), st["pair_row"].view(-1) >= 0
    token = torch.arange(N * k, device="cuda") // k
    dw = torch.where(have, (y[rows] * d_out[token]).sum(-1), 0.0).view(1, N, k)
    pair, live = st["recv_pair"].clamp(min=0).long(), (st["recv_pair"] >= 0).unsqueeze(-1)
    d_y = torch.where(live, st["w"].view(-1)[pair].unsqueeze(-1) * d_out[pair // k], 0.0)
    return {"d_y": d_y.bfloat16(), "d_topk_w": dw}


def _experts(st):
    case = st["case"]
    E, K, N = case["E"], case["K"], case["N"]
    values = torch.tensor(_E2M1, device="cuda")
    nibbles = torch.stack((st["codes"] & 15, st["codes"] >> 4), -1).int()
    w = values[nibbles].view(E, -1, K // 16, 16)
    w = w * (st["scales"].view(torch.float8_e4m3fn).float() * st["factor"][:, None, None])[..., None]
    x = st["a"].float()[st["index"]] * st["used"].unsqueeze(-1)
    out = torch.bmm(x, w.view(E, -1, K).transpose(1, 2))
    if case["gated"]:
        gate, up = out[..., :N], out[..., N:]
        out = gate / (1 + (-gate).exp()) * up
    y = torch.zeros(st["rows"], N, device="cuda")
    return y.index_copy(0, st["index"][st["used"]], out[st["used"]]).bfloat16()


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"balance": _balance, "route": _route, "combine": _combine, "experts": _experts}[op](st)
    moe = st["moe"]
    if op == "balance":
        moe.moe_balance_loss(st["logits"], st["ids"], st["counts"], st["prob"], st["lse"],
                             st["n_valid"], st["losses"], st["ws"], token_mask=st["mask"])
        return {"losses": st["losses"], "counts": st["counts"], "prob_mean": st["prob"],
                "lse": st["lse"], "n_valid": st["n_valid"]}
    if op == "route":
        moe.moe_route_backward(st["logits"], st["ids"], st["w"], st["dw"], st["lse"],
                               st["counts"], st["n_valid"], st["d_losses"], st["d_logits"],
                               token_mask=st["mask"])
        return st["d_logits"]
    if op == "combine":
        moe.moe_combine_backward(st["d_out"], st["y"], st["pair_row"], st["w"], st["d_y"],
                                 st["dw"], recv_pair=st["recv_pair"])
        return {"d_y": st["d_y"], "d_topk_w": st["dw"]}
    moe.moe_expert_product_w4(st["a"], st["w4"], st["factor"], st["y"], st["ws"],
                              gated=st["case"]["gated"], **st["rows_by"])
    return st["y"]


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_router(case, st):
    S, T, E, k = case["S"], case["T"], case["E"], case["k"]
    logits, ids = st["logits"].double(), st["ids"].long()
    valid = (torch.ones(S, T, dtype=torch.bool, device="cuda") if st["mask"] is None
             else st["mask"].bool())
    counts = torch.zeros(S, E, dtype=torch.int32, device="cuda")
    prob = torch.zeros(S, E, dtype=torch.float64, device="cuda")
    lse = torch.zeros(S, T, dtype=torch.float64, device="cuda")
    losses = torch.zeros(2, dtype=torch.float64, device="cuda")
    grad = torch.zeros(S, T, E, dtype=torch.float64, device="cuda")
    for s in range(S):
        rows = logits[s, valid[s]]
        n = rows.shape[0]
        if n == 0:
            continue
        counts[s] = torch.bincount(ids[s, valid[s]].view(-1), minlength=E).int()
        z = torch.logsumexp(rows, -1)
        lse[s, valid[s]] = z
        p = torch.softmax(rows, -1)
        prob[s] = p.mean(0)
        share = counts[s].double() / (n * k)                 # of the picks that each expert has
        losses[0] += E * (share * prob[s]).sum() / S
        losses[1] += z.square().mean() / S
        if case["op"] == "route":
            d0, d1 = st["d_losses"].double()
            d = p * (E * share - (p * (E * share)).sum(-1, keepdim=True)) * (d0 / (S * n))
            d += 2 * z[:, None] * p * (d1 / (S * n))
            w, dw = st["w"][s, valid[s]].double(), st["dw"][s, valid[s]].double()
            d.scatter_add_(-1, ids[s, valid[s]], w * dw - w * (w * dw).sum(-1, keepdim=True))
            grad[s, valid[s]] = d
    if case["op"] == "route":
        return grad
    return {"losses": losses, "counts": counts, "prob_mean": prob, "lse": lse,
            "n_valid": valid.sum(1).int()}


def _exact_combine(case, st):
    N, k = case["T"], case["k"]
    d_y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(1, N, k, dtype=torch.float64, device="cuda")
    d_out = st["d_out"][0].double()
    for j in range(k):
        rows = st["pair_row"][0, :, j].long()
        have = torch.nonzero(rows >= 0).view(-1)
        d_y[rows[have]] = st["w"][0, have, j].double()[:, None] * d_out[have]
        dw[0, have, j] = torch.einsum("nh,nh->n", st["y"][rows[have]].double(), d_out[have])
    return {"d_y": d_y, "d_topk_w": dw}


def _exact_experts(case, st):
    K, N = case["K"], case["N"]
    y = torch.zeros(st["rows"], N, dtype=torch.float64, device="cuda")
    starts, _ = _starts(case)
    for e, c in enumerate(_counts(case)):
        if c == 0:
            continue
        code = st["codes"][e].int()
        w = torch.empty(code.shape[0], K, dtype=torch.float64, device="cuda")
        for half in range(2):
            q = (code >> (4 * half)) & 15
            exponent, mantissa = (q >> 1) & 3, (q & 1).double()
            size = torch.where(exponent > 0, torch.exp2(exponent.double() - 1) * (1 + mantissa / 2),
                               mantissa / 2)
            w[:, half::2] = torch.where(q >= 8, -size, size)
        s = st["scales"][e].view(torch.float8_e4m3fn).double() * st["factor"][e].double()
        w *= torch.repeat_interleave(s, 16, dim=1)
        at = slice(starts[e], starts[e] + c)
        out = st["a"][at].double() @ w.t()
        y[at] = torch.nn.functional.silu(out[:, :N]) * out[:, N:] if case["gated"] else out
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "combine":
        return _exact_combine(case, st)
    return _exact_experts(case, st) if case["op"] == "experts" else _exact_router(case, st)
