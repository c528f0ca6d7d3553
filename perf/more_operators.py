"""The cases that the MXFP4 products of rows, the gated activation on rows and the 8-bit
checkpoints are measured on.

`run` makes one pass through an operator: with `own` false in plain torch operations (float32,
rounded once at the end), with `own` true through the calls of bit_quantized_mixture_amd.
`exact` gives the same outputs in float64 from the definitions.

Kinds of case:
  product      rows to MXFP4 (gathered by token or in expert order already), then their grouped product
               with an MXFP4 stack: out[p] = x4[p] W4_e^T + bias_e
  glu_step     the activation between the two products and its gradient, with the rows kept in 8 bits between
  glu_grad     that gradient alone, from rows that a forward pass has left in 8 bits
  rows8        rows put into 8 bits and read back
  lora_grad8   the gradients of low-rank adapters whose input rows are kept in 8 bits

4 bits: e2m1 values times a power of two for each 32, the largest value's floor(log2) less 2.
8 bits: int8 times a power of two for each 32, the smallest one that keeps every value within half a step.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one decoded token of the 32-expert layer: gate_up rows of its four experts
        {"name": "product_one_token", "kind": "product", "T": 1, "K": 2880, "N": 5760, "E": 32, "k": 4, "skew": 0.0, "x": "bf16",
         "out": "f32", "bias": True},
        # 64 decoded tokens of the fine-grained layer
        {"name": "product_decode", "kind": "product", "T": 64, "K": 2048, "N": 1536, "E": 128, "k": 8, "skew": 0.0, "x": "bf16",
         "out": "f32", "bias": False},
        # a prompt of odd length through a down projection, rows in expert order, some experts much asked for
        {"name": "product_ragged", "kind": "product", "T": 8168, "K": 1536, "N": 4096, "E": 64, "k": 1, "skew": 0.5, "x": "f32",
         "out": "bf16", "bias": False},
        # the 32-expert layer's gate_up projection over 2048 tokens
        {"name": "product_layer", "kind": "product", "T": 2048, "K": 2880, "N": 5760, "E": 32, "k": 4, "skew": 0.0, "x": "bf16",
         "out": "f32", "bias": True},
        # the 8-expert layer's gate_up projection over 4096 tokens: the largest product
        {"name": "product_wide", "kind": "product", "T": 4096, "K": 4096, "N": 28672, "E": 8, "k": 2, "skew": 0.0, "x": "bf16",
         "out": "bf16", "bias": False},
        # a short training batch of the 32-expert layer
        {"name": "glu_step_short", "kind": "glu_step", "S": 256, "I": 2880, "act": "clamped_glu", "interleaved": True, "rows": "f32",
         "out": "bf16"},
        # training the 8-expert layer over 4096 tokens
        {"name": "glu_step_layer", "kind": "glu_step", "S": 8192, "I": 14336, "act": "swiglu", "interleaved": False, "rows": "f32",
         "out": "bf16"},
        # the backward pass of an odd number of rows, the gradient in float32 as the adapters' backward leaves it
        {"name": "glu_grad_odd", "kind": "glu_grad", "S": 8191, "I": 2880, "act": "clamped_glu", "interleaved": True, "rows": "f32",
         "out": "bf16"},
        # a few rows kept between two passes
        {"name": "rows8_short", "kind": "rows8", "S": 64, "C": 2880, "rows": "bf16"},
        # the gathered rows of the largest prefill, as the adapters' backward wants them
        {"name": "rows8_prefill", "kind": "rows8", "S": 131072, "C": 4096, "rows": "bf16"},
        # training the adapters of the 32-expert layer's down projection
        {"name": "lora_grad8_experts", "kind": "lora_grad8", "S": 8192, "K": 2880, "N": 2880, "r": 32, "groups": 32, "adapters": 32,
         "experts": True, "out": "f32"},
        # training the adapters of the 8-expert layer's gate_up projection
        {"name": "lora_grad8_wide", "kind": "lora_grad8", "S": 8192, "K": 4096, "N": 28672, "r": 16, "groups": 8, "adapters": 8,
         "experts": True, "out": "f32"},
    ]


MOST_BYTES, MOST_FLOPS = 3.3e9, 1.93e12  # of one pass: the largest listed cases


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        kind = rng.choice(["product", "product", "product", "product", "glu_step", "glu_grad", "rows8", "lora_grad8", "lora_grad8"])
        if kind == "product":
            E = _log(rng, 1, 128)
            k = min(E, rng.randint(1, 8))
            case = {"kind": kind, "T": max(1, _log(rng, 1, 16384) // k), "K": 32 * _log(rng, 2, 448),
                    "N": rng.choice([_log(rng, 64, 28672), 8 * _log(rng, 8, 3584), 8 * _log(rng, 8, 3584)]), "E": E, "k": k, "skew": rng.choice([0.0, 0.25, 0.5]), "x": rng.choice(["bf16", "f32"]),
                    "out": rng.choice(["f32", "bf16"]), "bias": rng.random() < 0.5}
            # the plain form decodes the stack to float32 and pads every expert's rows to the longest
            longest = 3 * case["T"] * k * ((1 - case["skew"]) / E + case["skew"] / math.sqrt(E)) + 8
            if E * case["N"] * case["K"] > 1e9 or E * longest * (case["K"] + case["N"]) > 2e9:
                continue
        elif kind == "lora_grad8":
            experts = rng.random() < 0.5
            groups = _log(rng, 1, 64)
            case = {"kind": kind, "S": _log(rng, 16, 16384), "K": 32 * _log(rng, 2, 448), "N": 8 * _log(rng, 8, 3584),
                    "r": 8 * _log(rng, 1, 16), "groups": groups, "adapters": groups if experts else rng.randint(1, groups),
                    "experts": experts, "out": rng.choice(["f32", "bf16"])}
            padded = (2 * case["S"] + 8 * groups) * (case["K"] + case["N"])
            if case["adapters"] * case["r"] * (case["K"] + case["N"]) > 1e8 or padded > 2e9:
                continue
        elif kind == "rows8":
            case = {"kind": kind, "S": _log(rng, 1, 131072), "C": 32 * _log(rng, 2, 448), "rows": rng.choice(["bf16", "f32"])}
        else:
            case = {"kind": kind, "S": _log(rng, 1, 16384), "I": 32 * _log(rng, 2, 448), "act": rng.choice(["swiglu", "clamped_glu"]),
                    "interleaved": rng.random() < 0.5, "rows": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"])}
        cost = work(case)
        if cost["bytes"] <= MOST_BYTES and cost["flops"] <= MOST_FLOPS:
            return case


def work(case):
    """Each input read once, each output written once (an 8-bit checkpoint that a pass leaves and takes up
    again: both)."""
    kind = case["kind"]
    if kind == "product":
        S, K, N, E = case["T"] * case["k"], case["K"], case["N"], min(case["E"], case["T"] * case["k"])
        read = case["T"] * K * SIZE[case["x"]] + E * N * K * 17 / 32 + (4 * E * N if case["bias"] else 0)
        return {"bytes": read + S * N * SIZE[case["out"]], "flops": 2 * S * N * K}
    if kind == "rows8":
        n = case["S"] * case["C"]
        return {"bytes": n * (2 * SIZE[case["rows"]] + 2 * 33 / 32), "flops": 2 * n}
    if kind == "lora_grad8":
        S, K, N, r, n = case["S"], case["K"], case["N"], case["r"], min(case["adapters"], case["S"])
        w = 2 * n * r * (K + N)
        return {"bytes": 2 * S * N + S * K * 33 / 32 + 4 * S * r + w + 2 * SIZE[case["out"]] * S * K + 2 * w,
                "flops": 4 * S * r * (K + N)}
    n, b, o = case["S"] * case["I"], SIZE[case["rows"]], SIZE[case["out"]]
    back = n * (b + 2 * 33 / 32 + 2 * o)
    return {"bytes": back + (n * (2 * b + 2 * 33 / 32 + o) if kind == "glu_step" else 0), "flops": 30 * n}


# ---- the two formats in float32 ------------------------------------------------------------------------------------------

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _blocks(x):
    return x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)


def _two_to(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _floor_log2(amax):
    return torch.where(amax > 0, torch.frexp(amax)[1] - 1, torch.full_like(amax, -200, dtype=torch.int32))


def _to4(x):
    """e2m1 codes [.., K/32, 32] with their signs in bit 3, and exponents [.., K/32]."""
    v = _blocks(x.float())
    e = (_floor_log2(v.abs().amax(-1)) - 2).clamp(-127, 127)
    m = v.abs() * _two_to(-e)[..., None]
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int() + (m >= 3.5).int()
            + (m > 5.0).int())
    return code + 8 * torch.signbit(v).int(), e


def _values4(code, e):
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    return (grid[code] * _two_to(e)[..., None]).flatten(-2)


def _pack4(code, e):
    """The bytes of a packed stack: blocks [.., K/32, 16] (the even element in the low nibble) and scales [.., K/32]."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), (e + 127).to(torch.uint8)


def _unpack4(blocks, scales):
    b = blocks.int()
    return torch.stack([b & 15, b >> 4], -1).flatten(-2), scales.int() - 127


def _to8(x):
    """int8 [.., C] and exponent bytes [.., C/32]."""
    v = _blocks(x.float())
    amax = v.abs().amax(-1)
    e = _floor_log2(amax).clamp_min(-127)
    e = e + (amax * _two_to(-e) >= 127.5 / 64).int()
    q = torch.round(torch.ldexp(v, (6 - e)[..., None])).clamp(-127, 127)
    return q.flatten(-2).to(torch.int8), (e + 127).to(torch.uint8)


def _values8(q, scales):
    return torch.ldexp(_blocks(q.float()), (scales.int() - 133)[..., None]).flatten(-2)


# ---- inputs --------------------------------------------------------------------------------------------------------------


def _lengths(total, groups, skew, rng):
    """Rows of each group, as a router with or without favourites or packed prompts give them (some may be empty)."""
    p = rng.uniform(0.5, 1.5, groups) / (1.0 + np.arange(groups)) ** skew
    return rng.multinomial(total, p / p.sum()).tolist()


def _offsets(lengths):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).to(DEV)


def _places(lengths):
    """Row numbers of every group, padded to the longest with the number of rows: [groups, longest]."""
    ends, longest = np.cumsum(lengths), max(1, max(lengths))
    place = (ends - lengths)[:, None] + np.arange(longest)[None, :]
    return torch.from_numpy(np.where(place < ends[:, None], place, ends[-1]).astype(np.int64)).to(DEV)


def prepare(case, seed):
    gen, rng = torch.Generator(device=DEV), np.random.default_rng(seed)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, device=DEV, generator=gen) * std).to(dtype)

    kind, s = case["kind"], {"case": case}
    if kind == "product":
        T, K, N, E, k = case["T"], case["K"], case["N"], case["E"], case["k"]
        x = torch.randn(T, K, device=DEV, generator=gen)
        x *= torch.exp(0.5 * torch.randn(K, device=DEV, generator=gen))  # some columns are larger than others
        s["x"] = x.to(DTYPES[case["x"]])
        if k > 1:  # tokens in order, each sent to k experts
            logits = torch.randn(T, E, device=DEV, generator=gen) - case["skew"] * torch.log(1.0 + torch.arange(E, device=DEV))
            ids = torch.topk(logits, k, dim=1)[1].reshape(-1)
            s["slots"] = torch.argsort(ids, stable=True).to(torch.int32)
            s["lengths"] = torch.bincount(ids, minlength=E).tolist()
        else:      # rows in expert order already
            s["slots"] = None
            s["lengths"] = _lengths(T, E, case["skew"], rng)
        s["offsets"], s["place"] = _offsets(s["lengths"]), _places([n for n in s["lengths"] if n])
        s["used"] = torch.from_numpy(np.flatnonzero(s["lengths"])).to(DEV)  # experts with rows
        packed = [_pack4(*_to4(normal(N, K, dtype=torch.float32, std=0.02))) for _ in range(E)]
        s["w"], s["ws"] = (torch.stack([p[i] for p in packed]) for i in (0, 1))
        s["bias"] = normal(E, N, dtype=torch.float32, std=0.02) if case["bias"] else None
    elif kind == "rows8":
        s["x"] = normal(case["S"], case["C"], dtype=DTYPES[case["rows"]])
    elif kind == "lora_grad8":
        S, K, N, r, n, G = (case[v] for v in ("S", "K", "N", "r", "adapters", "groups"))
        s["lengths"] = _lengths(S, G, 0.0, rng)
        ids = np.arange(G) if case["experts"] else np.where(rng.random(G) < 0.1, -1, rng.integers(0, n, G))
        s["ids"], s["offsets"], s["place"] = ids.tolist(), _offsets(s["lengths"]), _places(s["lengths"])
        s["ids_long"] = torch.from_numpy(ids.astype(np.int64)).to(DEV)
        s["adapter"] = None if case["experts"] else torch.from_numpy(ids.astype(np.int32)).to(DEV)
        s["q"], s["qs"] = _to8(normal(S, K))
        s["a"], s["b"] = normal(n, r, K, std=K ** -0.5), normal(n, N, r, std=r ** -0.5)
        s["scale"] = torch.rand(n, device=DEV, generator=gen) + 0.5
        s["g"], s["z"] = normal(S, N), normal(S, r, dtype=torch.float32)
        s["gx"] = normal(S, K, dtype=DTYPES[case["out"]])  # the base projection's part
    else:
        S, I = case["S"], case["I"]
        rows = normal(S, 2 * I, dtype=DTYPES[case["rows"]], std=2.0)
        s["g"] = normal(S, I, dtype=DTYPES[case["rows"]])
        if kind == "glu_step":
            s["rows"] = rows
        else:
            s["q"], s["qs"] = _to8(rows)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------------


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import bit_quantized_mixture_amd as e4b

    c, kind = s["case"], s["case"]["kind"]
    if kind == "product":
        x4, xs = e4b.e4b_quantize_act_mxfp4(s["x"], s["slots"], c["k"])
        return e4b.e4b_grouped_gemm_mxfp4(x4, xs, s["w"], s["ws"], s["offsets"], bias=s["bias"], dtype=DTYPES[c["out"]])
    if kind == "rows8":
        q, qs = e4b.e4b_checkpoint_rows(s["x"])
        return e4b.e4b_restore_rows(q, qs, dtype=DTYPES[c["rows"]])
    if kind == "lora_grad8":
        return e4b.e4b_grouped_lora_backward(s["g"], s["q"], s["z"], s["a"], s["b"], s["scale"], s["offsets"], s["adapter"],
                                             gx_base=s["gx"], x_scales=s["qs"])
    act = {"act": c["act"], "interleaved": c["interleaved"]}
    if kind == "glu_grad":
        return e4b.e4b_glu_backward(s["g"], s["q"], s["qs"], dtype=DTYPES[c["out"]], **act)
    h, (q, qs) = e4b.e4b_glu(s["rows"], dtype=DTYPES[c["out"]], checkpoint=True, **act)
    return h, e4b.e4b_glu_backward(s["g"], q, qs, dtype=DTYPES[c["out"]], **act)


def _run_plain(s):
    c, kind = s["case"], s["case"]["kind"]
    if kind == "product":
        return _product_plain(s, c)
    if kind == "rows8":
        return _values8(*_to8(s["x"])).to(DTYPES[c["rows"]])
    if kind == "lora_grad8":
        return _lora_plain(s, c)
    out = DTYPES[c["out"]]
    if kind == "glu_grad":
        return _glu_grad_plain(s["g"].float(), _values8(s["q"], s["qs"]), c).to(out)
    kept = _to8(s["rows"])
    return _glu_plain(s["rows"].float(), c).to(out), _glu_grad_plain(s["g"].float(), _values8(*kept), c).to(out)


def _padded(rows, place):
    """Rows of every group, padded with zeros: [groups, longest, columns] in float32."""
    return torch.cat([rows.float(), torch.zeros_like(rows[:1], dtype=torch.float32)])[place]


def _rows_of(padded, place, S):
    """The padded rows at their places: [S, columns]."""
    out = torch.empty(S + 1, padded.shape[-1], device=padded.device)
    out[place.reshape(-1)] = padded.reshape(-1, padded.shape[-1])
    return out[:S]


def _product_plain(s, c):
    x = s["x"] if s["slots"] is None else s["x"][s["slots"].long() // c["k"]]
    x = _padded(_values4(*_to4(x)), s["place"])
    w = _values4(*_unpack4(s["w"][s["used"]], s["ws"][s["used"]]))
    out = torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2)
    if s["bias"] is not None:
        out = out + s["bias"][s["used"]][:, None, :]
    return _rows_of(out, s["place"], c["T"] * c["k"]).to(DTYPES[c["out"]])


def _halves(rows, c):
    I = c["I"]
    return (rows[:, 0::2], rows[:, 1::2]) if c["interleaved"] else (rows[:, :I], rows[:, I:])


def _glu_plain(rows, c):
    gate, up = _halves(rows, c)
    if c["act"] == "swiglu":
        return gate * torch.sigmoid(gate) * up
    gate = gate.clamp(max=7.0)
    return gate * torch.sigmoid(1.702 * gate) * (up.clamp(-7.0, 7.0) + 1.0)


def _glu_grad_plain(g, rows, c):
    gate, up = _halves(rows, c)
    if c["act"] == "swiglu":
        s = torch.sigmoid(gate)
        d_gate, d_up = g * up * s * (1.0 + gate * (1.0 - s)), g * gate * s
    else:
        low = gate.clamp(max=7.0)
        s = torch.sigmoid(1.702 * low)
        d_gate = torch.where(gate <= 7.0, g * (up.clamp(-7.0, 7.0) + 1.0) * s * (1.0 + 1.702 * low * (1.0 - s)), 0.0)
        d_up = torch.where(up.abs() <= 7.0, g * low * s, 0.0)
    return torch.stack([d_gate, d_up], -1).flatten(-2) if c["interleaved"] else torch.cat([d_gate, d_up], -1)


def _lora_plain(s, c):
    ids, S, n = s["ids_long"].clamp_min(0), c["S"], s["a"].shape[0]
    x, g, z = (_padded(v, s["place"]) for v in (_values8(s["q"], s["qs"]), s["g"], s["z"]))
    a, b = s["a"].float()[ids], s["b"].float()[ids]
    scale = torch.where(s["ids_long"] >= 0, s["scale"][ids], 0.0)[:, None, None]
    u = torch.bmm(g, b) * scale
    gx = s["gx"].float() + _rows_of(torch.bmm(u, a), s["place"], S)
    ga = torch.bmm(u.transpose(1, 2).contiguous(), x)
    gb = torch.bmm(g.transpose(1, 2).contiguous(), z) * scale
    # an adapter's gradient is the sum over the groups that use it
    uses = (s["ids_long"][None, :] == torch.arange(n, device=ga.device)[:, None]).float()
    ga = (uses @ ga.reshape(len(ga), -1)).reshape(s["a"].shape)
    gb = (uses @ gb.reshape(len(gb), -1)).reshape(s["b"].shape)
    return gx.to(DTYPES[c["out"]]), ga, gb


# ---- the definitions in float64 ------------------------------------------------------------------------------------------


def _exact4(x):
    """The nearest of the e2m1 values by their spacing (1/2 up to 2, then 1, then 2), ties to the even one."""
    v = x.double().reshape(-1, 32)
    top = v.abs().max(dim=1, keepdim=True).values
    unit = torch.exp2((torch.floor(torch.log2(top.clamp_min(1e-300))) - 2).clamp_min(-127.0))
    m = (v / unit).abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    return (torch.sign(v) * (torch.round(m / step) * step).clamp(max=6.0) * unit).reshape(x.shape)


def _exact8(x):
    v = x.double().reshape(-1, 32)
    top = v.abs().max(dim=1, keepdim=True).values
    unit = torch.exp2(torch.floor(torch.log2(top.clamp_min(1e-300))).clamp_min(-127.0) - 6)
    unit = torch.where(torch.round(top / unit) > 127, 2 * unit, unit)
    return (torch.round(v / unit) * unit).reshape(x.shape)


def _held4(blocks, scales):
    low, high = (blocks & 15).long(), (blocks >> 4).long()
    code = torch.stack([low, high], dim=-1).reshape(*blocks.shape[:-1], 32)
    mag, exp = code & 1, (code >> 1) & 3
    v = torch.where(exp == 0, 0.5 * mag.double(), (1 + 0.5 * mag.double()) * torch.exp2(exp.double() - 1))
    v = torch.where(code >= 8, -v, v) * torch.exp2(scales.double() - 127)[..., None]
    return v.reshape(*blocks.shape[:-2], -1)


def _held8(q, scales):
    return q.double() * torch.exp2(scales.double() - 133).repeat_interleave(32, dim=-1)


def _exact_glu(rows, c, g=None):
    """h, or with g the gradient of the rows."""
    I = c["I"]
    pick = torch.arange(2 * I, device=rows.device).reshape(I, 2).T if c["interleaved"] else torch.arange(2 * I, device=rows.device).reshape(2, I)
    gate, up = rows.index_select(1, pick[0]), rows.index_select(1, pick[1])
    slope, shift, top = (1.0, 0.0, math.inf) if c["act"] == "swiglu" else (1.702, 1.0, 7.0)
    low, mid = torch.clamp(gate, max=top), torch.clamp(up, -top, top) + shift
    sig = 1.0 / (1.0 + torch.exp(-slope * low))
    if g is None:
        return low * sig * mid
    out = torch.empty_like(rows)
    out[:, pick[0]] = torch.where(gate > top, 0.0, g * mid * (sig + slope * low * sig * torch.exp(-slope * low) * sig))
    out[:, pick[1]] = torch.where(up.abs() > top, 0.0, g * low * sig)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rows8":
        return _exact8(s["x"])
    if kind == "glu_grad":
        return _exact_glu(_held8(s["q"], s["qs"]), case, s["g"].double())
    if kind == "glu_step":
        return _exact_glu(s["rows"].double(), case), _exact_glu(_exact8(s["rows"]), case, s["g"].double())
    if kind == "product":
        x = _exact4(s["x"])
        if s["slots"] is not None:
            x = x.index_select(0, torch.div(s["slots"].long(), case["k"], rounding_mode="floor"))
        parts, lo = [], 0
        for e, n in enumerate(s["lengths"]):
            if n:
                y = torch.mm(x[lo:lo + n], _held4(s["w"][e], s["ws"][e]).T.contiguous())
                parts.append(y if s["bias"] is None else y + s["bias"][e].double())
            lo += n
        return torch.cat(parts)
    gx, ga, gb = s["gx"].double(), torch.zeros_like(s["a"], dtype=torch.float64), torch.zeros_like(s["b"], dtype=torch.float64)
    x, ends = _held8(s["q"], s["qs"]), np.cumsum(s["lengths"])
    for hi, n, i in zip(ends, s["lengths"], s["ids"]):
        if i < 0 or n == 0:
            continue
        rows = slice(int(hi) - n, int(hi))
        g, scale = s["g"][rows].double(), s["scale"][i].double()
        u = scale * torch.mm(g, s["b"][i].double())
        gx[rows] += torch.mm(u, s["a"][i].double())
        ga[i] += torch.mm(u.T, x[rows])
        gb[i] += scale * torch.mm(g.T, s["z"][rows].double())
    return gx, ga, gb
