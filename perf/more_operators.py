"""Timed cases of the norm around the token path and of the experts' bf16 products.

Four operators of one MoE layer:

- ``norm``           moe_rms_norm: residual addition and RMS norm, rows out in bf16 and as MXFP8 records;
- ``norm_backward``  moe_rms_norm_backward: its gradient in the rows and in the weight;
- ``product``        moe_expert_product: the experts' products with bf16 weights, plain or gated
  (silu(gate) * up);
- ``backward``       moe_expert_product_backward: the gradient of a product in its rows (or, where the
  rows were silu(gate) * up, in gate and up) and in the experts' weights.

``run`` computes them in elementary torch operations in 32 bits, or with ``own`` through the
framework's calls.  ``exact`` holds the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_EPS = 1e-6


def listed():
    return [
        # one decode token between two layers: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "H": 5120, "residual": "bf16",
         "weight": "bf16", "y": True, "record": True},
        # the prefill batch, rows for the router in bf16 and for the dispatch as records
        {"name": "norm_prefill", "op": "norm", "rows": 4096, "H": 5120, "residual": "bf16",
         "weight": "bf16", "y": True, "record": True},
        # the large training batch with a residual stream in 32 bits
        {"name": "norm_train", "op": "norm", "rows": 16384, "H": 2048, "residual": "f32",
         "weight": "f32", "y": True, "record": False},
        # a short batch of odd length
        {"name": "norm_backward_odd", "op": "norm_backward", "rows": 333, "H": 1040, "h": "f32",
         "weight": "f32", "residual": True},
        # four prefill batches of one training step
        {"name": "norm_backward_train", "op": "norm_backward", "rows": 16384, "H": 5120, "h": "bf16",
         "weight": "bf16", "residual": True},
        # one token's six experts: a single-stream decode step
        {"name": "product_token", "op": "product", "E": 48, "rows": 6, "skew": 0.0, "K": 5120,
         "N": 2048, "gated": True, "keep": False, "layout": "runs", "align": 1},
        # one partition of the 64-token decode batch, receive blocks of 64 rows
        {"name": "product_decode", "op": "product", "E": 48, "rows": 48, "skew": 0.0, "K": 2048,
         "N": 5120, "gated": False, "keep": False, "layout": "blocks", "align": 64},
        # sizes off every tile, runs padded to 8 rows
        {"name": "product_odd", "op": "product", "E": 5, "rows": 37, "skew": 1.0, "K": 1048,
         "N": 328, "gated": True, "keep": True, "layout": "runs", "align": 8},
        # the large training batch: thousands of rows an expert, gate and up kept for the way back
        {"name": "product_train", "op": "product", "E": 8, "rows": 16384, "skew": 0.2, "K": 2048,
         "N": 1408, "gated": True, "keep": True, "layout": "runs", "align": 1},
        {"name": "backward_odd", "op": "backward", "E": 5, "rows": 300, "skew": 1.0, "N": 328,
         "K": 648, "gate": True, "d_w": "f32", "layout": "blocks", "align": 200},
        # the way back through the second product of the large batch, weight gradients in 32 bits
        {"name": "backward_down", "op": "backward", "E": 8, "rows": 16384, "skew": 0.2, "N": 2048,
         "K": 1408, "gate": True, "d_w": "f32", "layout": "runs", "align": 1},
        # and through its first one
        {"name": "backward_up", "op": "backward", "E": 8, "rows": 16384, "skew": 0.2, "N": 2816,
         "K": 2048, "gate": False, "d_w": "bf16", "layout": "runs", "align": 1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng: random.Random):
    op = rng.choice(["norm", "norm_backward", "product", "product", "backward"])
    if op in ("norm", "norm_backward"):
        record = op == "norm" and rng.random() < 0.5
        H = 32 * _log_int(rng, 2, 256) if record else 8 * _log_int(rng, 8, 1024)
        rows = min(_log_int(rng, 1, 16384), 16384 * 5120 // H)
        case = {"op": op, "rows": rows, "H": H, "weight": rng.choice(["bf16", "f32"])}
        if op == "norm":
            return {**case, "residual": rng.choice(["none", "bf16", "f32"]), "record": record,
                    "y": not record or rng.random() < 0.5}
        return {**case, "h": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.7}
    K, N = 8 * _log_int(rng, 8, 640), 8 * _log_int(rng, 4, 640)
    n = 2 * N if op == "product" else N
    E = min(_log_int(rng, 1, 64), max(1, 400_000_000 // (K * n)))
    rows = min(_log_int(rng, 1, 16384), max(1, int(1.5e11) // (2 * K * n)))
    case = {"op": op, "E": E, "rows": rows, "skew": round(rng.uniform(0, 0.8), 2), "K": K, "N": N,
            "layout": rng.choice(["runs", "runs", "blocks"]), "align": rng.choice([1, 1, 8, 16])}
    if op == "product":
        case["gated"] = rng.random() < 0.6
        case["keep"] = case["gated"] and rng.random() < 0.5
    else:
        case["gate"], case["d_w"] = rng.random() < 0.5, rng.choice(["f32", "bf16"])
    if case["layout"] == "blocks":
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


def _size(name):
    return 4 if name == "f32" else 2 if name == "bf16" else 0


def work(case):
    if case["op"] == "norm":
        R, H = case["rows"], case["H"]
        record = H + H // 32 if case["record"] else 0
        # rows, residual in and out, rows out, records out, weight
        return {"bytes": R * (2 * H + 2 * H * _size(case["residual"]) + 2 * H * case["y"] + record)
                + H * _size(case["weight"]), "flops": 4 * R * H}
    if case["op"] == "norm_backward":
        R, H, h = case["rows"], case["H"], _size(case["h"])
        # d_y, h, d_residual in, d_h (and for 32 bits its bf16 copy) out, weight and its gradient
        return {"bytes": R * H * (2 + h + h * case["residual"] + h + 2 * (h == 4))
                + H * (_size(case["weight"]) + 4), "flops": 9 * R * H}
    counts = _counts(case)
    active, rows, K, N = sum(c > 0 for c in counts), sum(counts), case["K"], case["N"]
    if case["op"] == "product":
        n = N * (2 if case["gated"] else 1)
        # weights of the experts in use, rows in, rows (and gate and up) out
        return {"bytes": 2 * active * n * K + 2 * rows * (K + N + 2 * N * case["keep"]),
                "flops": 2 * rows * n * K}
    # weights in use, d_y, rows, (gate and up,) their gradient, the weights' gradient
    return {"bytes": 2 * active * N * K + 2 * rows * (N + K + K * (4 if case["gate"] else 1))
            + case["E"] * N * K * _size(case["d_w"]), "flops": 4 * rows * N * K}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _states(rows, width, g):
    """Hidden states of unit size with a few channels that stand out."""
    a = torch.randn(rows, width, generator=g, device="cuda")
    a[:, torch.randint(0, width, (max(1, width // 256),), generator=g, device="cuda")] *= 12
    return a


def _prepare_norm(case, seed):
    g = _generator(seed)
    R, H = case["rows"], case["H"]
    weight = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(_DTYPES[case["weight"]])
    st = {"case": case, "weight": weight}
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if case["op"] == "norm":
        st["x"] = (0.5 * _states(R, H, g)).bfloat16()
        st["residual"] = (None if case["residual"] == "none"
                          else (3 * _states(R, H, g)).to(_DTYPES[case["residual"]]))
        if own:
            import combine_moe_route_06_gb300 as moe
            st.update(moe=moe, y=torch.empty(R, H, **bf16) if case["y"] else None,
                      residual_out=None if st["residual"] is None else torch.empty_like(st["residual"]),
                      record=torch.empty(R, moe.mxfp8_record_bytes(H), dtype=torch.uint8,
                                         device="cuda") if case["record"] else None)
        return st
    dtype = _DTYPES[case["h"]]
    st["h"] = (3 * _states(R, H, g)).to(dtype)
    st["d_y"] = (torch.randn(R, H, generator=g, device="cuda") / 64).bfloat16()
    st["d_residual"] = ((torch.randn(R, H, generator=g, device="cuda") / 64).to(dtype)
                        if case["residual"] else None)
    if own:
        import combine_moe_route_06_gb300 as moe
        st.update(moe=moe, d_h=torch.empty_like(st["h"]),
                  d_x=torch.empty(R, H, **bf16) if case["h"] == "f32" else None,
                  d_weight=torch.empty(H, dtype=torch.float32, device="cuda"),
                  ws=torch.empty(moe.moe_rms_norm_backward_workspace_bytes(R, H), dtype=torch.uint8,
                                 device="cuda"))
    return st


def _prepare_experts(case, seed):
    g = _generator(seed)
    E, K, N = case["E"], case["K"], case["N"]
    forward = case["op"] == "product"
    n = 2 * N if forward and case["gated"] else N
    w = torch.empty(E, n, K, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = torch.randn(n, K, generator=g, device="cuda") / math.sqrt(K)
    counts = _counts(case)
    starts, rows = _starts(case)
    M = max(counts)
    counts_t = torch.tensor(counts, dtype=torch.int32, device="cuda")
    index = (torch.tensor(starts, device="cuda")[:, None] + torch.arange(M, device="cuda"))
    used = torch.arange(M, device="cuda") < counts_t[:, None]
    live = torch.zeros(rows, 1, device="cuda").index_fill_(0, index[used], 1.0)   # zero run padding
    st = {"case": case, "w": w, "index": index.clamp(max=rows - 1), "used": used, "rows": rows,
          "a": (_states(rows, K, g) * live).bfloat16(), "pre": None}
    if not forward:
        st["d_y"] = (torch.randn(rows, N, generator=g, device="cuda") / 64 * live).bfloat16()
        if case["gate"]:      # rows that came from gate and up
            pre = (torch.randn(rows, 2 * K, generator=g, device="cuda") * live).bfloat16()
            gate, up = pre.float().chunk(2, 1)
            st["pre"], st["a"] = pre, (gate / (1 + (-gate).exp()) * up).bfloat16()
    if own:
        import combine_moe_route_06_gb300 as moe
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        if case["layout"] == "blocks":
            st["rows_by"] = {"masked_counts": counts_t, "block_rows": case["align"]}
        else:
            st["rows_by"] = {"expert_offsets": torch.tensor(starts + [rows], dtype=torch.int32,
                                                            device="cuda")}
        if forward:
            need = moe.moe_expert_product_workspace_bytes(rows, E, N, K, case["gated"])
            st.update(y=torch.zeros(rows, N, **bf16),
                      keep=torch.zeros(rows, 2 * N, **bf16) if case["keep"] else None)
        else:
            need = moe.moe_expert_product_backward_workspace_bytes(rows, E, N, K)
            st.update(d_a=torch.zeros(rows, 2 * K if case["gate"] else K, **bf16),
                      d_w=torch.empty(E, N, K, dtype=_DTYPES[case["d_w"]], device="cuda"))
        st.update(moe=moe, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    return st


def prepare(case, seed):
    return _prepare_norm(case, seed) if case["op"].startswith("norm") else _prepare_experts(case, seed)


# ---------------------------------------------------------------- plain forms

def _norm(st):
    case = st["case"]
    h = st["x"].float()
    out = {}
    if st["residual"] is not None:
        h = h + st["residual"].float()
        out["residual"] = h.to(st["residual"].dtype)
    y = (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + _EPS) * st["weight"].float()).bfloat16()
    if case["y"]:
        out["y"] = y
    if case["record"]:      # blocks of 32: a power of two for each, and values in E4M3
        blocks = y.float().view(case["rows"], -1, 32)
        top = blocks.abs().amax(-1)
        shift = torch.where(top > 0, torch.frexp(top).exponent - 9, -127)
        by = ((127 - shift).int() << 23).view(torch.float32)
        out["codes"] = (blocks * by.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(1)
        out["scales"] = (shift + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _norm_backward(st):
    h, d_y = st["h"].float(), st["d_y"].float()
    inv = torch.rsqrt(h.square().mean(-1, keepdim=True) + _EPS)
    q = d_y * st["weight"].float()
    d_h = q * inv - h * (inv * inv * inv * (q * h).mean(-1, keepdim=True))
    if st["d_residual"] is not None:
        d_h = d_h + st["d_residual"].float()
    out = {"d_h": d_h.to(st["h"].dtype), "d_weight": (d_y * h * inv).sum(0)}
    if st["case"]["h"] == "f32":
        out["d_x"] = d_h.bfloat16()
    return out


def _padded(st, t):
    """An expert's rows after another, [E, M, width], zero where it has none left."""
    return torch.where(st["used"].unsqueeze(-1), t.float()[st["index"]], 0.0)


def _back(st, t):
    out = torch.zeros(st["rows"], t.shape[-1], device="cuda")
    return out.index_copy(0, st["index"][st["used"]], t[st["used"]]).bfloat16()


def _product(st):
    case, N = st["case"], st["case"]["N"]
    out = torch.bmm(_padded(st, st["a"]), st["w"].float().transpose(1, 2))
    if not case["gated"]:
        return {"y": _back(st, out)}
    gate, up = out[..., :N], out[..., N:]
    got = {"y": _back(st, gate / (1 + (-gate).exp()) * up)}
    if case["keep"]:
        got["pre"] = _back(st, out)
    return got


def _backward(st):
    case, K = st["case"], st["case"]["K"]
    d_y = _padded(st, st["d_y"])
    d_a = torch.bmm(d_y, st["w"].float())
    if case["gate"]:
        pre = _padded(st, st["pre"])
        gate, up = pre[..., :K], pre[..., K:]
        s = 1 / (1 + (-gate).exp())
        d_a = torch.cat((d_a * up * (s * (1 + gate * (1 - s))), d_a * (gate * s)), -1)
    d_w = torch.bmm(d_y.transpose(1, 2), _padded(st, st["a"]))
    return {"d_a": _back(st, d_a), "d_w": d_w.to(_DTYPES[case["d_w"]])}


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        return {"norm": _norm, "norm_backward": _norm_backward, "product": _product,
                "backward": _backward}[op](st)
    moe = st["moe"]
    if op == "norm":
        moe.moe_rms_norm(st["x"], st["weight"], y=st["y"], record=st["record"],
                         residual=st["residual"], residual_out=st["residual_out"], eps=_EPS)
        out = {"y": st["y"], "residual": st["residual_out"]}
        if case["record"]:      # the bytes as what they are: E4M3 values, then powers of two
            out["codes"] = st["record"][:, :case["H"]].view(torch.float8_e4m3fn)
            out["scales"] = st["record"][:, case["H"]:].view(torch.float8_e8m0fnu)
        return out
    if op == "norm_backward":
        moe.moe_rms_norm_backward(st["d_y"], st["h"], st["weight"], st["d_h"], st["ws"],
                                  d_weight=st["d_weight"], d_residual=st["d_residual"],
                                  d_x=st["d_x"], eps=_EPS)
        return {"d_h": st["d_h"], "d_weight": st["d_weight"], "d_x": st["d_x"]}
    if op == "product":
        moe.moe_expert_product(st["a"], st["w"], st["y"], st["ws"], gated=case["gated"],
                               pre=st["keep"], **st["rows_by"])
        return {"y": st["y"], "pre": st["keep"]}
    moe.moe_expert_product_backward(st["d_y"], st["a"], st["w"], st["ws"], d_a=st["d_a"],
                                    d_w=st["d_w"], pre=st["pre"], **st["rows_by"])
    return {"d_a": st["d_a"], "d_w": st["d_w"]}


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_norm(case, st):
    x = st["x"].double()
    out = {}
    if case["residual"] != "none":
        x = x + st["residual"].double()
        out["residual"] = x
    size = (torch.linalg.vector_norm(x, dim=1) ** 2 / case["H"] + _EPS).sqrt()
    y = x / size[:, None] * st["weight"].double()
    if case["y"]:
        out["y"] = y
    if case["record"]:
        # values as stored in bf16, so that the records are those of the rows in bf16
        blocks = y.float().bfloat16().double().view(-1, case["H"] // 32, 32)
        top = blocks.abs().amax(-1)
        power = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 8, -127.0)
        q = blocks / torch.exp2(power)[..., None]
        size = q.abs()
        # E4M3: three bits after the leading one down to 2^-6, below it steps of 2^-9
        step = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
        size = (torch.round(size / step) * step).clamp(max=448.0)
        out["codes"] = torch.where(q < 0, -size, size).flatten(1)
        out["scales"] = torch.exp2(power)
    return out


def _exact_norm_backward(case, st):
    h, d_y, w = st["h"].double(), st["d_y"].double(), st["weight"].double()
    size = (torch.linalg.vector_norm(h, dim=1) ** 2 / case["H"] + _EPS).sqrt()[:, None]
    unit = h / size                                   # y = unit * w
    d_unit = d_y * w
    along = (d_unit * unit).sum(1, keepdim=True) / case["H"]
    d_h = (d_unit - along * unit) / size
    if case["residual"]:
        d_h = d_h + st["d_residual"].double()
    out = {"d_h": d_h, "d_weight": torch.einsum("rh,rh->h", d_y, unit)}
    if case["h"] == "f32":
        out["d_x"] = d_h
    return out


def _exact_experts(case, st):
    N, K, rows = case["N"], case["K"], st["rows"]
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    forward = case["op"] == "product"
    if forward:
        out = {"y": zeros(rows, N)}
        if case["keep"]:
            out["pre"] = zeros(rows, 2 * N)
    else:
        out = {"d_a": zeros(rows, 2 * K if case["gate"] else K), "d_w": zeros(case["E"], N, K)}
    starts, _ = _starts(case)
    for e, c in enumerate(_counts(case)):
        if c == 0:
            continue
        at = slice(starts[e], starts[e] + c)
        a, w = st["a"][at].double(), st["w"][e].double()
        if forward:
            both = a @ w.t()
            out["y"][at] = (torch.nn.functional.silu(both[:, :N]) * both[:, N:] if case["gated"]
                            else both)
            if case["keep"]:
                out["pre"][at] = both
            continue
        d_y = st["d_y"][at].double()
        out["d_w"][e] = d_y.t() @ a
        d_a = d_y @ w
        if case["gate"]:
            gate, up = st["pre"][at].double().split(K, 1)
            s = torch.sigmoid(gate)
            d_a = torch.cat((d_a * up * (s + gate * s * (1 - s)), d_a * gate * s), 1)
        out["d_a"][at] = d_a
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "product": _exact_experts,
            "backward": _exact_experts}[case["op"]](case, st)
