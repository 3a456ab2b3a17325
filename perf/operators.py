"""Measured cases of the operators that read a model's stored weights for a few
tokens, or make a table's gradient: products with 4-bit weights (q4), rows of
an embedding table with scaling (lookup, from the entropy-coded scope or a bf16
table), and the table's gradient by sorted tokens (grad).

``run`` computes a case in its plain form (elementary torch operations in fp32,
rounded once) or, with ``own``, through the library.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "fp32": F32}
SIZES = {"bf16": 2, "fp32": 4, "int32": 4, "int64": 8}


def listed():
    return [
        # 4-bit products.  One token through a k or v projection of the 8B-shaped model: latency.
        {"name": "q4_kv_1", "op": "q4", "rows": 1024, "cols": 4096, "group": 128, "zeros": False, "tokens": 1, "out": "fp32"},
        # one token through q, k and v held as one matrix
        {"name": "q4_qkv_1", "op": "q4", "rows": 6144, "cols": 4096, "group": 64, "zeros": True, "tokens": 1, "out": "bf16"},
        # sixteen sequences decoding together, the block's down projection
        {"name": "q4_down_16", "op": "q4", "rows": 4096, "cols": 14336, "group": 128, "zeros": False, "tokens": 16, "out": "bf16"},
        # the 7B-shaped block's width, an odd number of rows and of tokens, fine groups
        {"name": "q4_ragged_5", "op": "q4", "rows": 4091, "cols": 11008, "group": 32, "zeros": True, "tokens": 5, "out": "fp32"},
        # lm_head of the 8B-shaped model, four sequences: the largest weights
        {"name": "q4_head_4", "op": "q4", "rows": 128256, "cols": 4096, "group": 128, "zeros": False, "tokens": 4, "out": "fp32"},
        # Rows of the 8B-shaped model's coded embedding: one decoding step, and a prompt batch.
        {"name": "lookup_coded_1", "op": "lookup", "coded": True, "rows": 128256, "dim": 4096, "tokens": 1, "scale": 1.0, "ids": "int64"},
        {"name": "lookup_coded_8192", "op": "lookup", "coded": True, "rows": 128256, "dim": 4096, "tokens": 8192, "scale": 64.0, "ids": "int64"},
        # a small table whose rows start anywhere in a chunk of the code, with padding ids
        {"name": "lookup_coded_ragged", "op": "lookup", "coded": True, "rows": 5003, "dim": 1000, "tokens": 777, "scale": 31.625, "ids": "int32"},
        # the decoded table of a model in training
        {"name": "lookup_table_16384", "op": "lookup", "coded": False, "rows": 32000, "dim": 2048, "tokens": 16384, "scale": 45.25, "ids": "int64"},
        # The table's gradient.  A small table and a few tokens: latency.
        {"name": "grad_small", "op": "grad", "rows": 1000, "dim": 129, "tokens": 33, "scale": 1.0, "dy": "fp32", "out": "fp32", "ids": "int32"},
        # a step on 8192 tokens of a 32000-row table
        {"name": "grad_8192", "op": "grad", "rows": 32000, "dim": 4096, "tokens": 8192, "scale": 64.0, "dy": "bf16", "out": "bf16", "ids": "int64"},
        # byte-level vocabulary: every row has hundreds of tokens
        {"name": "grad_bytes", "op": "grad", "rows": 259, "dim": 1024, "tokens": 65536, "scale": 32.0, "dy": "bf16", "out": "fp32", "ids": "int64"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["q4", "lookup", "grad"])
    if op == "q4":
        cols = 32 * _log_int(rng, 2, 512)
        group = rng.choice([g for g in (32, 64, 128) if cols % g == 0])
        rows = _log_int(rng, 16, min(131072, 100000 * 4096 // cols))
        return {"op": op, "rows": rows, "cols": cols, "group": group, "zeros": rng.random() < 0.5,
                "tokens": _log_int(rng, 1, 16), "out": rng.choice(["fp32", "bf16"])}
    dim = _log_int(rng, 32, 8192)
    if rng.random() < 0.6:
        dim = max(64, dim // 64 * 64)
    if op == "lookup":
        rows = _log_int(rng, 64, min(131072, 128256 * 4096 // dim))
        return {"op": op, "coded": rng.random() < 0.7, "rows": rows, "dim": dim,
                "tokens": _log_int(rng, 1, min(16384, 8192 * 4096 // dim)),
                "scale": rng.choice([1.0, 64.0, 45.25, 0.5]), "ids": rng.choice(["int32", "int64"])}
    dy, out = rng.choice(["bf16", "fp32"]), rng.choice(["bf16", "fp32"])
    return {"op": op, "rows": _log_int(rng, 64, min(65536, 32000 * 4096 // (dim * SIZES[out] // 2))), "dim": dim,
            "tokens": _log_int(rng, 1, min(65536, 8192 * 4096 // (dim * SIZES[dy] // 2))),
            "scale": rng.choice([1.0, 64.0, 45.25]), "dy": dy, "out": out, "ids": rng.choice(["int32", "int64"])}


# ------------------------------------------------------------------- inputs

def _token_ids(g, case):
    """Log-uniform ranks (frequencies fall as 1 / rank, as words' do) on a
    random numbering of the rows; one token in twenty is padding (-1)."""
    t, v = case["tokens"], case["rows"]
    rank = (torch.rand(t, generator=g, device="cuda", dtype=torch.float64) * math.log(v + 1)).exp().long() - 1
    ids = torch.randperm(v, generator=g, device="cuda")[rank.clamp_(0, v - 1)]
    if t > 1:
        ids[torch.rand(t, generator=g, device="cuda") < 0.05] = -1
    return ids.to(getattr(torch, case["ids"])).contiguous()


def _q4_weights(g, case):
    """Gaussian weights rounded to 4 bits: codes two to a byte (even column in
    the low half), bf16 scales, and whole zero points or None (then 8)."""
    n, k, grp = case["rows"], case["cols"], case["group"]
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, k // grp, dtype=BF16, device="cuda")
    zeros = torch.empty(n, k // grp, dtype=torch.uint8, device="cuda") if case["zeros"] else None
    step = max(1, (1 << 26) // k)
    for r in range(0, n, step):
        w = (torch.randn(min(step, n - r), k // grp, grp, generator=g, device="cuda") * 0.02).to(BF16).float()
        if zeros is None:
            s = (w.abs().amax(-1) / 7).to(BF16)
            z = torch.full_like(s, 8.0, dtype=F32)
            q = (w / s.float()[..., None]).round().clamp(-8, 7) + 8
        else:
            lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
            s = (hi / 15 - lo / 15).to(BF16)
            z = (-lo / s.float()).round().clamp(0, 15)
            q = ((w / s.float()[..., None]).round() + z[..., None]).clamp(0, 15)
            zeros[r: r + step] = z.to(torch.uint8)
        q = q.to(torch.uint8).reshape(-1, k)
        scales[r: r + step] = s
        codes[r: r + step] = q[:, 0::2] | (q[:, 1::2] << 4)
    return codes, scales, zeros


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "q4":
        codes, scales, zeros = _q4_weights(g, case)
        x = torch.randn(case["tokens"], case["cols"], generator=g, device="cuda").to(BF16)
        state.update(x=x)
        if own:  # a serving program lays its weights out once, when it loads them
            import lossless_entropy_coded_canonical_b200 as dfw
            state.update(weights=dfw.q4_pack(codes, scales, zeros, group=case["group"]))
        else:
            state.update(codes=codes, scales=scales, zeros=zeros)
    elif case["op"] == "lookup":
        table = torch.randn(case["rows"], case["dim"], generator=g, device="cuda", dtype=BF16).mul_(0.02)
        state.update(ids=_token_ids(g, case))
        if own and case["coded"]:  # the model's embedding is held coded
            import lossless_entropy_coded_canonical_b200 as dfw
            state.update(scope=dfw.encode_device(table))
        else:
            state.update(table=table)
    else:
        dy = torch.randn(case["tokens"], case["dim"], generator=g, device="cuda").to(DTYPES[case["dy"]])
        state.update(ids=_token_ids(g, case), dy=dy)
    return state


# -------------------------------------------------------------------- passes

def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case, state)


def _run_own(case, state):
    import lossless_entropy_coded_canonical_b200 as dfw
    if case["op"] == "q4":
        return dfw.q4_gemv(state["weights"], state["x"], out_dtype=DTYPES[case["out"]])
    if case["op"] == "lookup":
        if case["coded"]:
            return dfw.embed_lanes(state["scope"], state["ids"], case["dim"], scale=case["scale"])
        return dfw.embed_rows(state["table"], state["ids"], scale=case["scale"])
    return dfw.embed_grad(state["ids"], state["dy"], case["rows"], scale=case["scale"], out_dtype=DTYPES[case["out"]])


def _run_plain(case, state):
    if case["op"] == "q4":
        codes, scales, zeros = state["codes"], state["scales"], state["zeros"]
        q = torch.stack([codes & 15, codes >> 4], -1).view(case["rows"], -1, case["group"]).float()
        q -= 8.0 if zeros is None else zeros[..., None].float()
        w = q.mul_(scales[..., None].float()).view(case["rows"], case["cols"])
        return (state["x"].float() @ w.t()).to(DTYPES[case["out"]])
    ids = state["ids"].long()
    keep = (ids >= 0)[:, None]
    if case["op"] == "lookup":
        rows = state["table"][ids.clamp(min=0)].float()
        return torch.where(keep, rows * case["scale"], 0.0).to(BF16)
    dy = torch.where(keep, state["dy"].float(), 0.0)
    grad = torch.zeros(case["rows"], case["dim"], device=dy.device).index_add_(0, ids.clamp(min=0), dy)
    return (grad * case["scale"]).to(DTYPES[case["out"]])


def exact(case, seed):
    """The definition in 64 bits."""
    g = torch.Generator("cuda").manual_seed(seed)
    if case["op"] == "q4":
        codes, scales, zeros = _q4_weights(g, case)
        x = torch.randn(case["tokens"], case["cols"], generator=g, device="cuda").to(BF16).double()
        y = torch.empty(case["tokens"], case["rows"], dtype=torch.float64, device="cuda")
        step = max(1, (1 << 25) // case["cols"])
        for r in range(0, case["rows"], step):
            c = codes[r: r + step]
            w = torch.empty(c.shape[0], case["cols"], dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = (c % 16).double(), (c // 16).double()
            z = 8.0 if zeros is None else zeros[r: r + step].double().repeat_interleave(case["group"], 1)
            s = scales[r: r + step].double().repeat_interleave(case["group"], 1)
            y[:, r: r + step] = x @ ((w - z) * s).t()
        return y
    if case["op"] == "lookup":
        table = torch.randn(case["rows"], case["dim"], generator=g, device="cuda", dtype=BF16).mul_(0.02)
        ids = _token_ids(g, case).long()
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        out[ids >= 0] = table[ids[ids >= 0]].double() * case["scale"]
        return out
    dy = torch.randn(case["tokens"], case["dim"], generator=g, device="cuda").to(DTYPES[case["dy"]]).double()
    ids = _token_ids(g, case).long()
    grad = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
    return grad.index_put_((ids[ids >= 0],), dy[ids >= 0] * case["scale"], accumulate=True)


def work(case):
    if case["op"] == "q4":
        n, k, m = case["rows"], case["cols"], case["tokens"]
        groups = n * k // case["group"]
        return {"bytes": n * k // 2 + groups * (3 if case["zeros"] else 2) + 2 * m * k + SIZES[case["out"]] * m * n,
                "flops": 2 * m * n * k}
    t, d = case["tokens"], case["dim"]
    if case["op"] == "lookup":
        # a coded weight: its raw byte, its share of the stream (2.6 bits for Gaussian weights) and of the plan
        row = 1 + 2.6 / 8 + 2 / 64 + 8 / 2048 if case["coded"] else 2
        return {"bytes": int(t * d * (row + 2)) + t * SIZES[case["ids"]], "flops": t * d}
    return {"bytes": t * d * SIZES[case["dy"]] + t * SIZES[case["ids"]] + case["rows"] * d * SIZES[case["out"]],
            "flops": t * d + case["rows"] * d}
