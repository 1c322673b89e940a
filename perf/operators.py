"""The microscaled 4-bit (MX4) base-weight operators as calls and as plain torch, for measuring one against the other.

MX4: blocks of 32 consecutive columns share one power-of-two scale byte E (value 2^(E - 127), 255 = NaN); each
element is a 4-bit e2m1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign), two per byte, the low nibble first.  A matrix
[rows][cols] is codes uint8 [rows][cols / 2] and scales uint8 [rows][16 ceil(cols / 512)] (16-byte rows, zeros past
cols / 32).  Shapes are those of the repository's workloads: the 8B layer (4096, 1024, 14336), the 14B MLP (5120,
17408) with its mixed batch of 1144 tokens, decode batches, and prompts up to the 8192 tokens one batch may hold.
"""
import math

import torch

own = False

DEV = "cuda:0"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode batch's activations quantised before a 4-bit product: latency
        {"name": "quantize_tokens_16x4096", "op": "quantize", "rows": 16, "cols": 4096, "dtype": "bf16"},
        # a down_proj weight at load, with the dequantised copy that a delta is compressed against
        {"name": "quantize_down_4096x14336", "op": "quantize", "rows": 4096, "cols": 14336, "dtype": "bf16"},
        # a 4-bit checkpoint's gate_proj back to dense bf16 (the dense merge of a hot user)
        {"name": "dequantize_gate_17408x5120", "op": "dequantize", "rows": 17408, "cols": 5120, "dtype": "bf16"},
        # one user typing: q|k|v of one token
        {"name": "gemm_qkv_1", "op": "gemm", "T": 1, "d_in": 4096, "n0": 4096, "n1": 1024, "n2": 1024, "n3": 0},
        # the stack's decode step: gate|up at 512 tokens
        {"name": "gemm_gateup_512", "op": "gemm", "T": 512, "d_in": 4096, "n0": 14336, "n1": 14336, "n2": 0, "n3": 0},
        # the mixed prefill and decode batch, ragged in tokens, over the widest rows
        {"name": "gemm_down_1144", "op": "gemm", "T": 1144, "d_in": 17408, "n0": 5120, "n1": 0, "n2": 0, "n3": 0},
        # 4-bit tokens too: a decode batch through q|k|v (latency), the stack's gate|up, a long prompt's gate
        {"name": "gemm4_qkv_16", "op": "gemm4", "T": 16, "d_in": 4096, "n0": 4096, "n1": 1024, "n2": 1024, "n3": 0},
        {"name": "gemm4_gateup_512", "op": "gemm4", "T": 512, "d_in": 4096, "n0": 14336, "n1": 14336, "n2": 0, "n3": 0},
        {"name": "gemm4_gate_8192", "op": "gemm4", "T": 8192, "d_in": 4096, "n0": 14336, "n1": 0, "n2": 0, "n3": 0},
        # 16 users, one token each, through q_proj: the whole multi-tenant layer in one launch
        {"name": "apply_q_16users_16", "op": "apply", "T": 16, "d_in": 4096, "d_out": 4096, "users": 16,
         "mode": "matrix", "group": 128, "ids": "perm", "tokens": "bf16"},
        # the stack's decode step through o_proj: 512 tokens, Zipf users of 128
        {"name": "apply_o_128users_512", "op": "apply", "T": 512, "d_in": 4096, "d_out": 4096, "users": 128,
         "mode": "matrix", "group": 128, "ids": "zipf", "tokens": "bf16"},
        # the mixed batch through down_proj with column scales, the base product on 4-bit tokens
        {"name": "apply_down_32users_1144", "op": "apply", "T": 1144, "d_in": 17408, "d_out": 5120, "users": 32,
         "mode": "col", "group": 128, "ids": "mixed", "tokens": "mx4"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "gemm", "gemm4", "apply"])
    if op in ("quantize", "dequantize"):
        while True:
            c = {"op": op, "rows": _log(rng, 1, 17408), "cols": 64 * _log(rng, 1, 272),
                 "dtype": rng.choice(["bf16", "f32"])}
            if c["rows"] * c["cols"] * (2 if c["dtype"] == "f32" else 1) <= 4096 * 14336:
                return c
    if op in ("gemm", "gemm4"):
        while True:
            n = rng.randint(1, 4)
            d = [_log(rng, 16, 14336) if i < n else 0 for i in range(4)]
            c = {"op": op, "T": _log(rng, 1, 8192 if op == "gemm4" else 2048), "d_in": 64 * _log(rng, 4, 272),
                 "n0": d[0], "n1": d[1], "n2": d[2], "n3": d[3]}
            f = c["T"] * c["d_in"] * sum(d)
            if f <= (8192 * 4096 * 14336 if op == "gemm4" else 1144 * 17408 * 5120) and sum(d) * c["d_in"] <= 28672 * 4096:
                return c
    while True:
        c = {"op": "apply", "T": _log(rng, 1, 1144), "d_in": 64 * _log(rng, 4, 272), "d_out": _log(rng, 16, 14336),
             "users": _log(rng, 1, 128), "mode": rng.choice(["matrix", "row", "col", "group"]), "group": 128,
             "ids": rng.choice(["uniform", "zipf"]), "tokens": rng.choice(["bf16", "mx4"])}
        if c["mode"] == "group" and c["d_in"] % 128:
            continue
        if c["users"] * c["d_in"] * c["d_out"] <= 128 * 4096 * 4096 and c["T"] * c["d_in"] * c["d_out"] <= 1144 * 17408 * 5120:
            return c


def _outs(case):
    return [case[k] for k in ("n0", "n1", "n2", "n3") if case[k]]


# ------------------------------------------------------------------ MX4 in plain torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], from the bit fields."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22))
    return bits.to(torch.int32).view(torch.float32)


def _quantize(v):
    """Codes uint8 [rows][cols / 2], scales uint8 [rows][16 ceil(cols / 512)] and the values they stand for (fp32)."""
    rows, cols = v.shape
    b = v.float().view(rows, cols // 32, 32)
    amax = b.abs().amax(dim=2, keepdim=True)
    bad = ~torch.isfinite(amax)
    safe = torch.where(bad, torch.zeros_like(amax), amax)
    e = torch.frexp(safe)[1] - 3  # floor(log2 amax) - 2
    e = torch.where(safe == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    r = torch.where(bad, torch.zeros_like(b), b) * _pow2(-e)
    q = r.abs()
    step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0))
    q = (torch.round(q / step) * step).clamp(max=6.0)  # round is half-to-even, as on the e2m1 grid
    code = (torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4))).to(torch.uint8)
    code = code | (torch.signbit(r) & ~bad).to(torch.uint8) << 3
    code = code.view(rows, cols // 2, 2)
    scales = torch.zeros(rows, 16 * ((cols + 511) // 512), dtype=torch.uint8, device=v.device)
    scales[:, :cols // 32] = torch.where(bad, torch.full_like(e, 255), e + 127).squeeze(2).to(torch.uint8)
    val = torch.where(bad, torch.full_like(r, float("nan")), torch.copysign(q, r) * _pow2(e))
    return code[:, :, 0] | code[:, :, 1] << 4, scales, val.view(rows, cols)


def _dequantize(codes, scales):
    rows, cols = codes.shape[0], codes.shape[1] * 2
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float32, device=codes.device)
    v = grid[torch.stack((codes & 15, codes >> 4), dim=2).int()]
    s = scales[:, :cols // 32].int()
    f = torch.where(s == 255, float("nan"), _pow2(s.clamp(max=254) - 127))
    return (v.view(rows, cols // 32, 32) * f.unsqueeze(2)).view(rows, cols)


def _deltas(case, signs, scales, dtype):
    """Every user's dense delta scale (.) sign [U][d_out][d_in], from the packed signs (bit 1 is +1)."""
    U, d_out, d_in = case["users"], case["d_out"], case["d_in"]
    byte = signs.view(torch.uint8).view(U, d_out, d_in // 8, 1)
    bit = byte >> torch.arange(8, dtype=torch.uint8, device=byte.device) & 1
    s = bit.view(U, d_out, d_in).to(dtype) * 2 - 1
    f = scales.to(dtype)
    if case["mode"] == "group":
        return (s.view(U, d_out, -1, case["group"]) * f.view(U, d_out, -1, 1)).view(U, d_out, d_in)
    return s * f.view({"matrix": (U, 1, 1), "row": (U, d_out, 1), "col": (U, 1, d_in)}[case["mode"]])


# ------------------------------------------------------------------ inputs

def _tokens(g, T, d_in):
    """Activations: normal, one channel in 128 eight times as large (the outlier channels of trained models)."""
    x = torch.randn(T, d_in, generator=g, device=DEV)
    loud = torch.rand(d_in, generator=g, device=DEV) < 1 / 128
    return (x * torch.where(loud, 8.0, 1.0)).to(torch.bfloat16)


def _weight(g, d_out, d_in, dtype=torch.bfloat16):
    return (torch.randn(d_out, d_in, generator=g, device=DEV) * 0.02).to(dtype)


def _ids(case, g):
    T, U = case["T"], case["users"]
    if case["ids"] == "perm":
        return torch.randperm(U, generator=g, device=DEV)[:T].int()
    r = torch.rand(T, generator=g, device=DEV, dtype=torch.float64)
    if case["ids"] == "uniform":  # -1 among them: tokens of the base model
        return (r * (U + 1)).long().clamp(max=U).int() - 1
    w = torch.arange(1, U + 1, device=DEV, dtype=torch.float64) ** -1.1  # Zipf(1.1)
    ids = torch.searchsorted(torch.cumsum(w / w.sum(), 0), r).clamp(max=U - 1).int()
    if case["ids"] == "mixed":  # 8 prompt chunks of 128 tokens, then decode tokens
        ids = torch.cat((ids[:8].repeat_interleave(128), ids[1024:]))
    return ids


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    op = case["op"]
    if op == "quantize":
        if case["rows"] <= 64:
            return {"case": case, "v": _tokens(g, case["rows"], case["cols"]).to(dt)}
        return {"case": case, "v": _weight(g, case["rows"], case["cols"], dt)}
    if op == "dequantize":
        return {"case": case, "base": _quantize(_weight(g, case["rows"], case["cols"]))[:2], "dtype": dt}
    x = _tokens(g, case["T"], case["d_in"])
    if op in ("gemm", "gemm4"):
        return {"case": case, "x": x, "bases": [_quantize(_weight(g, n, case["d_in"]))[:2] for n in _outs(case)]}
    U, d_out, d_in = case["users"], case["d_out"], case["d_in"]
    base = _quantize(_weight(g, d_out, d_in))[:2]
    signs = torch.randint(-2 ** 63, 2 ** 63 - 1, (U, d_out, d_in // 64), generator=g, device=DEV)
    per = {"matrix": 1, "row": d_out, "col": d_in, "group": d_out * d_in // case["group"]}[case["mode"]]
    sdt = torch.float16 if case["mode"] in ("row", "col") else torch.float32
    scales = (5e-4 * (0.5 + torch.rand(U, per, generator=g, device=DEV))).to(sdt)
    ids = _ids(case, g)
    # the scheduler's list of each user's tokens (row T: none), as wide as the busiest user's
    host = ids.tolist()
    rows = [[t for t, u in enumerate(host) if u == k] for k in range(U)]
    cap = max(1, max(len(r) for r in rows))
    slots = torch.tensor([r + [case["T"]] * (cap - len(r)) for r in rows], device=DEV)
    return {"case": case, "x": x, "base": base, "signs": signs, "scales": scales, "ids": ids, "slots": slots}


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from tenant_serving_amd import bitdelta as B
        if op == "quantize":
            _, scales, values = B.quantize_mx4(state["v"], values=True)
            return {"values": values, "scales": scales}
        if op == "dequantize":
            return B.dequantize_mx4(*state["base"], out_dtype=state["dtype"])
        if op == "gemm":
            return B.base_gemm_mx4(state["x"], state["bases"])
        if op == "gemm4":
            return B.base_gemm_mx4x4(B.quantize_mx4(state["x"]), state["bases"])
        sd = B.BD_F16 if state["scales"].dtype == torch.float16 else B.BD_F32
        p = B.params(case["mode"], case["group"], 0.0, sd)
        return B.apply_mx4(state["x"], *state["base"], state["signs"], state["scales"], p, state["ids"],
                           y_dtype=torch.bfloat16, tokens=case["tokens"])
    if op == "quantize":
        _, scales, values = _quantize(state["v"])
        return {"values": values.to(state["v"].dtype), "scales": scales}
    if op == "dequantize":
        return _dequantize(*state["base"]).to(state["dtype"])
    x = state["x"].float()
    if op == "gemm":
        return [x @ _dequantize(*b).t() for b in state["bases"]]
    if op == "gemm4":
        xq = _quantize(state["x"])[2]
        return [xq @ _dequantize(*b).t() for b in state["bases"]]
    xb = _quantize(state["x"])[2] if case["tokens"] == "mx4" else x
    y = xb @ _dequantize(*state["base"]).t()
    xpad = torch.cat((x, torch.zeros_like(x[:1])))
    d = torch.bmm(xpad[state["slots"]], _deltas(case, state["signs"], state["scales"], torch.float32).transpose(1, 2))
    ypad = torch.cat((torch.zeros_like(y), torch.zeros_like(y[:1])))
    ypad[state["slots"].flatten()] = d.flatten(0, 1)
    return (y + ypad[:-1]).to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without

def _mx4_bytes(rows, cols):
    return rows * cols // 2 + rows * cols // 32


def work(case):
    op = case["op"]
    if op in ("quantize", "dequantize"):
        el = 4 if case["dtype"] == "f32" else 2
        n = case["rows"] * case["cols"]
        both = 2 if op == "quantize" else 1  # quantize reads the values and writes what the codes stand for
        return {"bytes": both * el * n + _mx4_bytes(case["rows"], case["cols"]), "flops": 3 * n if both == 2 else n}
    T, K = case["T"], case["d_in"]
    if op in ("gemm", "gemm4"):
        N = sum(_outs(case))
        return {"bytes": 2 * T * K + _mx4_bytes(N, K) + 4 * T * N, "flops": 2 * T * N * K}
    N, U = case["d_out"], min(case["users"], T)
    per = {"matrix": 1, "row": N, "col": K, "group": N * K // case["group"]}[case["mode"]]
    el = 2 if case["mode"] in ("row", "col") else 4
    return {"bytes": 2 * T * K + _mx4_bytes(N, K) + U * (N * K // 8 + el * per) + 2 * T * N + 4 * T,
            "flops": 4 * T * N * K}


# ------------------------------------------------------------------ the definition in 64 bits

MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _exact_quantize(v):
    """(values, scale bytes): the nearest of the 16 codes, a tie to the even code, counted against the midpoints."""
    b = v.double().view(v.shape[0], -1, 32)
    a = b.abs().amax(dim=2)
    p = torch.floor(torch.log2(a.clamp(min=2.0 ** -140)))
    p = torch.where(torch.exp2(p) > a, p - 1, p)
    p = torch.where(torch.exp2(p + 1) <= a, p + 1, p) - 2
    p = p.clamp(-127, 127)
    r = b / torch.exp2(p).unsqueeze(2)
    k = sum(((r.abs() > m) | ((r.abs() == m) & (i % 2 == 1))).long() for i, m in enumerate(MIDS))
    val = torch.tensor(GRID, dtype=torch.float64, device=v.device)[k] * torch.sign(r) * torch.exp2(p).unsqueeze(2)
    return val.view(v.shape), p + 127


def _exact_dense(codes, scales):
    rows, half = codes.shape
    v = torch.empty(rows, 2 * half, dtype=torch.float64, device=codes.device)
    for at, c in ((0, codes.long() & 15), (1, codes.long() >> 4)):
        ex, man = (c >> 1) & 3, c & 1
        mag = torch.where(ex == 0, man * 0.5, (1 + man * 0.5) * torch.exp2(ex.double() - 1))
        v[:, at::2] = torch.where(c >= 8, -mag, mag)
    return v * torch.exp2(scales[:, :half // 16].double() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"values": _exact_quantize(s["v"])[0], "scales": None}
    if op == "dequantize":
        return _exact_dense(*s["base"])
    x = s["x"].double()
    xb = _exact_quantize(s["x"])[0] if op == "gemm4" or case.get("tokens") == "mx4" else x
    if op in ("gemm", "gemm4"):
        return [xb @ _exact_dense(*b).t() for b in s["bases"]]
    y = xb @ _exact_dense(*s["base"]).t()
    ids = s["ids"].long()
    for u in sorted(set(ids.tolist()) - {-1}):
        one = dict(case, users=1)
        t = (ids == u).nonzero().flatten()
        d = _deltas(one, s["signs"][u:u + 1].contiguous(), s["scales"][u:u + 1], torch.float64)[0]
        y[t] += x[t] @ d.t()
    return y
