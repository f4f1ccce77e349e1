"""Attention operators, as they are measured: cross attention (forward, forward and
backward, and one token against long states) and attention of a batch over one shared
prefix.

A case is a dict of sizes; `prepare` draws its inputs, `run` takes one pass through the
operator: in elementary torch operations in 32 bits where `own` is false, through
linear_memory_attention_b200.attention where it is true.  `exact` is the definition in
64 bits, one head of keys at a time.

Fields of a case: op ("cross": the forward pass; "train": forward and backward;
"prefix": a batch over one shared prefix), dtype, B sequences, Hq query heads over Hkv
key heads, n query rows a sequence, d the head size, layout ("bhnd": heads before rows,
"bnhd": rows before heads, as a projection leaves them); cross and train: m key rows a
sequence and ragged (keys of different lengths, one of them empty from four sequences
on); prefix: P shared rows and room for S rows of each sequence's own.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # One token of one decoder against a short encoded input: the call's latency.
        {"name": "cross token short", "op": "cross", "dtype": "bf16", "B": 1, "Hq": 32, "Hkv": 8, "n": 1, "m": 300,
         "d": 64, "ragged": False, "layout": "bhnd"},
        # A serving batch, one token each, over encoded documents of different lengths.
        {"name": "cross token batch", "op": "cross", "dtype": "bf16", "B": 16, "Hq": 32, "Hkv": 8, "n": 1, "m": 8000,
         "d": 128, "ragged": True, "layout": "bnhd"},
        # Evaluating a small model on a padded batch: odd sizes, one input empty.
        {"name": "cross forward ragged", "op": "cross", "dtype": "bf16", "B": 4, "Hq": 32, "Hkv": 32, "n": 1000,
         "m": 1500, "d": 64, "ragged": True, "layout": "bnhd"},
        # A decoder's context of 4096 rows over 16384 encoded ones.
        {"name": "cross forward long", "op": "cross", "dtype": "bf16", "B": 1, "Hq": 32, "Hkv": 8, "n": 4096,
         "m": 16384, "d": 128, "ragged": False, "layout": "bhnd"},
        # The full-precision path at the size it is checked with.
        {"name": "cross train fp32 small", "op": "train", "dtype": "fp32", "B": 1, "Hq": 2, "Hkv": 2, "n": 256,
         "m": 517, "d": 64, "ragged": False, "layout": "bhnd"},
        # The same path on a layer's worth of heads.
        {"name": "cross train fp32", "op": "train", "dtype": "fp32", "B": 1, "Hq": 8, "Hkv": 8, "n": 1000, "m": 2000,
         "d": 128, "ragged": False, "layout": "bhnd"},
        # A training step of a grouped-query model on a padded batch.
        {"name": "cross train grouped", "op": "train", "dtype": "bf16", "B": 2, "Hq": 32, "Hkv": 8, "n": 1000,
         "m": 4096, "d": 128, "ragged": True, "layout": "bnhd"},
        # A training step over long inputs.
        {"name": "cross train long", "op": "train", "dtype": "bf16", "B": 1, "Hq": 32, "Hkv": 32, "n": 4096, "m": 8000,
         "d": 128, "ragged": False, "layout": "bhnd"},
        # A few sequences behind a short common prompt: the call's latency.
        {"name": "prefix token short", "op": "prefix", "dtype": "bf16", "B": 4, "Hq": 32, "Hkv": 8, "n": 1, "P": 700,
         "S": 64, "d": 64, "layout": "bhnd"},
        # Answers to many questions on one document of 32768 rows, one token each.
        {"name": "prefix token batch", "op": "prefix", "dtype": "bf16", "B": 32, "Hq": 32, "Hkv": 8, "n": 1,
         "P": 32768, "S": 512, "d": 128, "layout": "bhnd"},
        # The questions themselves, 100 rows each, over a document of 16384 rows.
        {"name": "prefix questions", "op": "prefix", "dtype": "bf16", "B": 16, "Hq": 32, "Hkv": 8, "n": 100,
         "P": 16384, "S": 128, "d": 128, "layout": "bnhd"},
        # Three tokens a sequence in full precision.
        {"name": "prefix fp32", "op": "prefix", "dtype": "fp32", "B": 4, "Hq": 8, "Hkv": 8, "n": 3, "P": 2000,
         "S": 100, "d": 128, "layout": "bhnd"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "train", "prefix"])
    dtype = "fp32" if rng.random() < 0.25 else "bf16"
    Hkv, group = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 4, 8])
    case = {"op": op, "dtype": dtype, "B": _spread(rng, 1, 32), "Hq": min(32, Hkv * group), "Hkv": Hkv,
            "d": rng.choice([64, 128]), "layout": rng.choice(["bhnd", "bnhd"])}
    if op == "prefix":
        case["n"] = 1 if rng.random() < 0.5 else _spread(rng, 2, 100)
        case["P"] = _spread(rng, 1, 32768)
        case["S"] = case["n"] + _spread(rng, 1, 512)
    else:
        case["n"] = 1 if op == "cross" and rng.random() < 0.4 else _spread(rng, 1, 4096)
        # One key alone has the probability 1: dQ and dK are then zero but for rounding, which says nothing.
        case["m"] = _spread(rng, 32 if op == "train" else 1, 16384)
        case["ragged"] = rng.random() < 0.5
    # No drawn case costs more than the largest listed one of its kind.
    most = {("cross", "bf16"): 1.0e12, ("train", "bf16"): 1.2e12, ("prefix", "bf16"): 4.0e11}
    limit = most.get((op, dtype), 2.0e10)
    while case["B"] > 1 and (work(case)["flops"] > limit or work(case)["bytes"] > 4.0e8):
        case["B"] //= 2
    long = "P" if op == "prefix" else "m"
    while work(case)["flops"] > limit or work(case)["bytes"] > 4.0e8:
        big = long if case[long] >= case["n"] else "n"
        case[big] = max(32 if big == "m" else 1, case[big] * 2 // 3)
        if op == "prefix":
            case["S"] = max(case["S"], case["n"])
    return case


def _key_lengths(case):
    """Valid key rows of each sequence: all, or from all down to half, and one empty from four on."""
    B, m = case["B"], case["m"]
    if not case["ragged"]:
        return [m] * B
    lens = [max(1, m - (b * m) // (2 * B)) for b in range(B)]
    if B >= 4:
        lens[B // 2] = 0
    return lens


def _own_lengths(case):
    """Rows of its own that each sequence has, the n new ones among them."""
    B, S, n = case["B"], case["S"], case["n"]
    return [S - (b * (S - n)) // B for b in range(B)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, B, Hq, Hkv, n, d = DTYPES[case["dtype"]], case["B"], case["Hq"], case["Hkv"], case["n"], case["d"]

    def normal(B, H, rows, scale=1.0):
        """[B, H, rows, d], by the case's layout in memory."""
        if case["layout"] == "bnhd":
            return (torch.randn((B, rows, H, d), generator=gen, device="cuda") * scale).to(dt).transpose(1, 2)
        return (torch.randn((B, H, rows, d), generator=gen, device="cuda") * scale).to(dt)

    # Queries of norm 2 sqrt(d) give logits of standard deviation 2: peaked rows.
    state = {"op": case["op"], "q": normal(B, Hq, n, 2.0), "tau": 1.0 / math.sqrt(d)}
    if case["op"] == "prefix":
        state["kp"], state["vp"] = normal(1, Hkv, case["P"])[0], normal(1, Hkv, case["P"])[0]
        state["ks"], state["vs"] = normal(B, Hkv, case["S"]), normal(B, Hkv, case["S"])
        state["s_len"] = torch.tensor(_own_lengths(case), dtype=torch.int32, device="cuda")
    else:
        state["k"], state["v"] = normal(B, Hkv, case["m"]), normal(B, Hkv, case["m"])
        state["k_len"] = torch.tensor(_key_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if case["op"] == "train":
            state["dout"] = normal(B, Hq, n)
    return state


def _softmax(z, seen):
    """Row probabilities and log-sum-exp of z over what is seen; nothing seen: zeros and -inf."""
    z = z.masked_fill(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    return p / torch.where(total == 0, torch.ones_like(total), total), lse


def _plain_cross(s):
    q, k, v, tau = s["q"].float(), s["k"].float(), s["v"].float(), s["tau"]
    (B, Hq, n, d), (Hkv, m) = q.shape, k.shape[1:3]
    rows = (Hq // Hkv) * n  # the query rows of the heads that share one key head
    q = q.reshape(B, Hkv, rows, d)
    seen = torch.ones((1, 1, 1, m), dtype=torch.bool, device=q.device)
    if s["k_len"] is not None:
        seen = torch.arange(m, device=q.device) < s["k_len"][:, None, None, None]
    p, lse = _softmax(tau * (q @ k.transpose(-1, -2)), seen)
    out = p @ v
    dt = s["q"].dtype
    got = {"out": out.reshape(B, Hq, n, d).to(dt), "lse": lse.reshape(B, Hq, n)}
    if s["op"] == "train":
        do = s["dout"].float().reshape(B, Hkv, rows, d)
        dv = p.transpose(-1, -2) @ do
        dz = p * (do @ v.transpose(-1, -2) - (do * out).sum(-1, keepdim=True))
        got["dq"] = (tau * (dz @ k)).reshape(B, Hq, n, d).to(dt)
        got["dk"] = (tau * (dz.transpose(-1, -2) @ q)).to(dt)
        got["dv"] = dv.to(dt)
    return got


def _plain_prefix(s):
    q, kp, vp, ks, vs = (s[x].float() for x in ("q", "kp", "vp", "ks", "vs"))
    (B, Hq, n, d), (Hkv, P), S = q.shape, kp.shape[:2], ks.shape[2]
    g = Hq // Hkv
    q = q.reshape(B, Hkv, g * n, d)
    # The shared rows: all sequences' queries of a key head against them at once.
    every = q.transpose(0, 1).reshape(Hkv, B * g * n, d)
    zp = (every @ kp.transpose(-1, -2)).reshape(Hkv, B, g * n, P).transpose(0, 1)
    zs = q @ ks.transpose(-1, -2)
    # Query i of the n new rows sees its sequence's own rows up to itself.
    last = s["s_len"].long()[:, None, None, None] - n + torch.arange(n, device=q.device).repeat(g)[:, None]
    seen = torch.cat((torch.ones((B, 1, g * n, P), dtype=torch.bool, device=q.device),
                      torch.arange(S, device=q.device) <= last), -1)
    p, lse = _softmax(s["tau"] * torch.cat((zp, zs), -1), seen)
    mine = p[..., :P].transpose(0, 1).reshape(Hkv, B * g * n, P)
    out = (mine @ vp).reshape(Hkv, B, g * n, d).transpose(0, 1) + p[..., P:] @ vs
    return {"out": out.reshape(B, Hq, n, d).to(s["q"].dtype), "lse": lse.reshape(B, Hq, n)}


def run(state):
    if own:
        from linear_memory_attention_b200 import attention
        if state["op"] == "prefix":
            return attention.prefix_attention(state["q"], state["kp"], state["vp"], state["ks"], state["vs"],
                                              state["s_len"], state["tau"])
        return attention.cross_attention(state["q"], state["k"], state["v"], state["tau"], k_len=state["k_len"],
                                         dout=state.get("dout"))
    return _plain_prefix(state) if state["op"] == "prefix" else _plain_cross(state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, Hq, Hkv, n, d = case["B"], case["Hq"], case["Hkv"], case["n"], case["d"]
    rows = B * Hq * n
    if case["op"] == "prefix":
        lens = _own_lengths(case)
        pairs = Hq * sum(n * case["P"] + n * s - n * (n - 1) // 2 for s in lens)
        keys = Hkv * (case["P"] + sum(lens))
    else:
        lens = _key_lengths(case)
        pairs = Hq * n * sum(lens)
        keys = Hkv * sum(lens)
    # Queries and the valid keys and values in; the output rows and their log-sum-exp out.
    total = {"bytes": e * d * (2 * rows + 2 * keys) + 4 * rows, "flops": 4 * d * pairs}
    if case["op"] == "train":
        # dO in; dQ, and dK and dV of every row, out.  Four more products of the forward's two: dP, dV,
        # dQ and dK.  Computing the logits a second time is a kernel's choice and is not counted.
        total["bytes"] += e * d * (2 * rows + 2 * B * Hkv * case["m"])
        total["flops"] += 8 * d * pairs
    return total


def exact(case, seed):
    s = prepare(case, seed)
    B, Hq, Hkv, n, d, tau = case["B"], case["Hq"], case["Hkv"], case["n"], case["d"], s["tau"]
    g = Hq // Hkv
    f64 = {"dtype": torch.float64, "device": "cuda"}
    got = {"out": torch.zeros((B, Hq, n, d), **f64), "lse": torch.full((B, Hq, n), -math.inf, **f64)}
    if case["op"] == "train":
        got["dq"] = torch.zeros((B, Hq, n, d), **f64)
        got["dk"], got["dv"] = (torch.zeros((B, Hkv, case["m"], d), **f64) for _ in range(2))
    for b in range(B):
        for h in range(Hq):
            q = s["q"][b, h].double()
            if case["op"] == "prefix":
                size = _own_lengths(case)[b]
                k = torch.cat((s["kp"][h // g], s["ks"][b, h // g, :size])).double()
                v = torch.cat((s["vp"][h // g], s["vs"][b, h // g, :size])).double()
                z = tau * torch.einsum("ic,jc->ij", q, k)
                hidden = torch.triu(torch.ones((n, k.shape[0]), dtype=torch.bool, device="cuda"),
                                    diagonal=k.shape[0] - n + 1)
                z[hidden] = -math.inf
            else:
                size = _key_lengths(case)[b]
                if size == 0:
                    continue
                k, v = s["k"][b, h // g, :size].double(), s["v"][b, h // g, :size].double()
                z = tau * torch.einsum("ic,jc->ij", q, k)
            lse = torch.logsumexp(z, -1)
            p = torch.exp(z - lse[:, None])
            got["lse"][b, h] = lse
            got["out"][b, h] = torch.einsum("ij,jc->ic", p, v)
            if case["op"] == "train":
                do = s["dout"][b, h].double()
                dp = torch.einsum("ic,jc->ij", do, v)
                dz = p * (dp - torch.einsum("ij,ij->i", p, dp)[:, None])
                got["dq"][b, h] = tau * torch.einsum("ij,jc->ic", dz, k)
                got["dk"][b, h // g, :size] += tau * torch.einsum("ij,ic->jc", dz, q)
                got["dv"][b, h // g, :size] += torch.einsum("ij,ic->jc", p, do)
    return got
