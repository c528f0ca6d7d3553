"""The cases that the token permutation and the low-rank adapters are measured on.

`run` makes one pass through an operator: with `own` false in plain torch operations (float32,
rounded once at the end), with `own` true through the calls of bit_quantized_mixture_amd.
`exact` gives the same outputs in float64 from the definitions.

Kinds of case:
  permute           rows[p] = x[sorted_slots[p] // k]
  permute_grad      its gradient: the sum of each token's k rows
  combine           out[t] = sum_j w[t, j] * (row of slot t*k + j)
  combine_grad      its gradients: of the rows and of the weights
  lora              out = y + scale_a * (x A_a^T) B_a^T for groups of rows with an adapter a each
  lora_grad         its gradients: of x (added to the base projection's), of A and of B
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
        # one decoded token of the fine-grained layer: eight float32 expert rows into one
        {"name": "combine_one_token", "kind": "combine", "T": 1, "H": 2048, "E": 128, "k": 8, "rows": "f32", "out": "bf16"},
        # the largest prefill: gathering its tokens for the experts, and combining their rows
        {"name": "permute_prefill", "kind": "permute", "T": 16384, "H": 4096, "E": 64, "k": 8, "rows": "bf16", "out": "bf16"},
        {"name": "combine_prefill", "kind": "combine", "T": 16384, "H": 4096, "E": 64, "k": 8, "rows": "f32", "out": "bf16"},
        # a training batch of odd length: the gradient of the gathered copies back to the tokens
        {"name": "permute_grad_odd", "kind": "permute_grad", "T": 4099, "H": 2880, "E": 32, "k": 3, "rows": "bf16", "out": "f32"},
        # a training batch of the 32-expert layer: the gradients of the expert rows and of the router's weights
        {"name": "combine_grad", "kind": "combine_grad", "T": 2048, "H": 2880, "E": 32, "k": 4, "rows": "f32", "out": "bf16"},
        # one decoded token of one request on the dense [14336, 4096] projection
        {"name": "lora_one_token", "kind": "lora", "S": 1, "K": 4096, "N": 14336, "r": 16, "groups": 1, "adapters": 1,
         "experts": False, "none": 0.0, "out": "f32"},
        # 64 requests decode together on that projection, a token each: many adapters, some requests without one
        {"name": "lora_decode_requests", "kind": "lora", "S": 64, "K": 4096, "N": 14336, "r": 16, "groups": 64, "adapters": 48,
         "experts": False, "none": 0.1, "out": "f32"},
        # 64 decoded tokens of the fine-grained layer: an adapter for each of its 128 experts
        {"name": "lora_decode_experts", "kind": "lora", "S": 512, "K": 2048, "N": 1536, "r": 16, "groups": 128, "adapters": 128,
         "experts": True, "none": 0.0, "out": "f32"},
        # prompts of 24 requests packed into one prefill of odd length, larger ranks, a bfloat16 projection
        {"name": "lora_prefill_requests", "kind": "lora", "S": 5003, "K": 2880, "N": 2880, "r": 64, "groups": 24, "adapters": 16,
         "experts": False, "none": 0.1, "out": "bf16"},
        # the down projection of the 8-expert layer over 4096 tokens, an adapter for each expert
        {"name": "lora_prefill_experts", "kind": "lora", "S": 8192, "K": 14336, "N": 4096, "r": 16, "groups": 8, "adapters": 8,
         "experts": True, "none": 0.0, "out": "f32"},
        # training the adapters of the 32-expert layer's down projection
        {"name": "lora_grad_experts", "kind": "lora_grad", "S": 8192, "K": 2880, "N": 2880, "r": 32, "groups": 32, "adapters": 32,
         "experts": True, "none": 0.0, "out": "f32"},
        # training the adapters of the 8-expert layer's gate_up projection: the widest gradient
        {"name": "lora_grad_wide", "kind": "lora_grad", "S": 8192, "K": 4096, "N": 28672, "r": 16, "groups": 8, "adapters": 8,
         "experts": True, "none": 0.0, "out": "f32"},
    ]


MOST_BYTES, MOST_FLOPS = 2.3e9, 1.8e10  # of one pass: the largest listed cases


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        kind = rng.choice(["permute", "permute_grad", "combine", "combine_grad", "lora", "lora", "lora_grad", "lora_grad"])
        if kind.startswith("lora"):
            experts = rng.random() < 0.5
            groups = _log(rng, 1, 128)
            case = {"kind": kind, "S": _log(rng, 1 if kind == "lora" else 16, 16384),
                    "K": 8 * _log(rng, 8, 1792), "N": 8 * _log(rng, 8, 3584), "r": 8 * _log(rng, 1, 16), "groups": groups,
                    "adapters": groups if experts else rng.randint(1, groups), "experts": experts,
                    "none": 0.0 if experts else rng.choice([0.0, 0.1, 0.5]), "out": rng.choice(["f32", "bf16"])}
            # the plain form pads every group to the longest one
            padded = groups * (2 * case["S"] / groups + 8) * (case["K"] + case["N"]) * 4
            if padded > 8e9 or case["adapters"] * case["r"] * (case["K"] + case["N"]) > 2e8:
                continue
        else:
            E = _log(rng, 1, 256)
            case = {"kind": kind, "T": _log(rng, 1, 16384), "H": rng.choice([1, 2, 8, 8, 64]) * _log(rng, 16, 128), "E": E,
                    "k": min(E, rng.randint(1, 8)), "rows": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"])}
            if kind == "permute":
                case["out"] = case["rows"]
        cost = work(case)
        if cost["bytes"] <= MOST_BYTES and cost["flops"] <= MOST_FLOPS:
            return case


def _slots(case):
    return case["T"] * case["k"]


def work(case):
    """Each input read once, each output written once."""
    if case["kind"].startswith("lora"):
        S, K, N, r, n, b = case["S"], case["K"], case["N"], case["r"], case["adapters"], SIZE[case["out"]]
        n = min(n, S)
        w = 2 * n * r * (K + N)
        if case["kind"] == "lora":
            return {"bytes": 2 * S * K + w + 2 * b * S * N, "flops": 2 * S * r * (K + N)}
        return {"bytes": 2 * S * N + 2 * S * K + 4 * S * r + w + 2 * b * S * K + 2 * w, "flops": 4 * S * r * (K + N)}
    T, H, S, rb, ob = case["T"], case["H"], _slots(case), SIZE[case["rows"]], SIZE[case["out"]]
    if case["kind"] == "permute":
        return {"bytes": (T + S) * H * rb + 4 * S, "flops": 0}
    if case["kind"] == "combine_grad":
        return {"bytes": T * H * ob + S * H * (rb + ob) + 12 * S, "flops": 3 * S * H}
    weighted = case["kind"] == "combine"
    return {"bytes": S * H * rb + T * H * ob + (8 if weighted else 4) * S, "flops": (2 if weighted else 1) * S * H}


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(case, rng):
    """Rows of each group: a token each, or what a router or packed prompts give (some of them may be empty)."""
    if case["S"] == case["groups"] and not case["experts"]:
        return [1] * case["groups"]
    p = rng.uniform(0.5, 1.5, case["groups"])
    return rng.multinomial(case["S"], p / p.sum()).tolist()


def prepare(case, seed):
    gen, rng = _generator(seed), np.random.default_rng(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, device=DEV, generator=gen) * std).to(dtype)

    if case["kind"].startswith("lora"):
        S, K, N, r, n, G = case["S"], case["K"], case["N"], case["r"], case["adapters"], case["groups"]
        lengths = _lengths(case, rng)
        offsets = np.concatenate([[0], np.cumsum(lengths)])
        if case["experts"]:
            ids = np.arange(G)
        else:
            ids = np.where(rng.random(G) < case["none"], -1, rng.integers(0, n, G))
        longest = max(1, max(lengths))
        place = offsets[:-1, None] + np.arange(longest)[None, :]
        place = np.where(place < offsets[1:, None], place, S)  # row S: the padding
        state = {
            "case": case, "lengths": lengths, "ids": ids.tolist(),
            "offsets": torch.from_numpy(offsets.astype(np.int32)).to(DEV),
            "adapter": None if case["experts"] else torch.from_numpy(ids.astype(np.int32)).to(DEV),
            "place": torch.from_numpy(place.astype(np.int64)).to(DEV),
            "ids_long": torch.from_numpy(ids.astype(np.int64)).to(DEV),
            "x": normal(S, K), "a": normal(n, r, K, std=K ** -0.5), "b": normal(n, N, r, std=r ** -0.5),
            "scale": torch.rand(n, device=DEV, generator=gen) + 0.5,
        }
        if case["kind"] == "lora":
            state["y"] = normal(S, N, dtype=DTYPES[case["out"]])
        else:
            state["g"] = normal(S, N)
            state["z"] = torch.randn(S, r, device=DEV, generator=gen)  # kept by the forward pass
            state["gx"] = normal(S, K, dtype=DTYPES[case["out"]])      # the base projection's part
        return state
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    logits = torch.randn(T, E, device=DEV, generator=gen)
    if E > 8:  # some experts are asked for more often than others
        logits = logits - 0.5 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    top, ids = torch.topk(logits, k, dim=1)
    state = {"case": case, "slots": torch.argsort(ids.reshape(-1), stable=True).to(torch.int32),
             "w": torch.softmax(top, dim=1)}
    rows_t, out_t = DTYPES[case["rows"]], DTYPES[case["out"]]
    if case["kind"] == "permute":
        state["x"] = normal(T, H, dtype=rows_t)
    else:
        state["rows"] = normal(T * k, H, dtype=rows_t)
    if case["kind"] == "combine_grad":
        state["g"] = normal(T, H, dtype=out_t)
    return state


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import bit_quantized_mixture_amd as e4b

    c, kind = s["case"], s["case"]["kind"]
    if kind == "permute":
        return e4b.e4b_permute_tokens(s["x"], s["slots"], c["k"])
    if kind == "permute_grad":
        return e4b.e4b_combine_tokens(s["rows"], s["slots"], c["k"], dtype=DTYPES[c["out"]])
    if kind == "combine":
        return e4b.e4b_combine_tokens(s["rows"], s["slots"], c["k"], s["w"], dtype=DTYPES[c["out"]])
    if kind == "combine_grad":
        return e4b.e4b_combine_tokens_backward(s["g"], s["rows"], s["slots"], c["k"], s["w"], dtype=DTYPES[c["out"]])
    if kind == "lora":
        return e4b.e4b_grouped_lora(s["x"], s["a"], s["b"], s["scale"], s["offsets"], s["adapter"], y=s["y"])[0]
    return e4b.e4b_grouped_lora_backward(s["g"], s["x"], s["z"], s["a"], s["b"], s["scale"], s["offsets"], s["adapter"],
                                         gx_base=s["gx"])


def _run_plain(s):
    c, kind = s["case"], s["case"]["kind"]
    if kind.startswith("lora"):
        return _lora_plain(s) if kind == "lora" else _lora_grad_plain(s)
    T, H, k, slots = c["T"], c["H"], c["k"], s["slots"].long()
    if kind == "permute":
        return s["x"][slots // k]
    if kind == "combine_grad":
        g, w = s["g"].float()[slots // k], s["w"].reshape(-1)
        g_w = torch.zeros_like(w)
        g_w[slots] = (g * s["rows"].float()).sum(1)
        return (g * w[slots, None]).to(DTYPES[c["out"]]), g_w.reshape(T, k)
    inverse = torch.empty_like(slots)
    inverse[slots] = torch.arange(T * k, device=slots.device)
    rows = s["rows"].float()[inverse].reshape(T, k, H)
    if kind == "combine":
        rows = rows * s["w"][:, :, None]
    return rows.sum(1).to(DTYPES[c["out"]])


def _padded(rows, place):
    """Rows of every group, padded with zeros: [groups, longest, columns] in float32."""
    return torch.cat([rows.float(), torch.zeros_like(rows[:1], dtype=torch.float32)])[place]


def _of_groups(s):
    """The adapters of the groups in float32; a group without one gets scale 0."""
    ids = s["ids_long"].clamp_min(0)
    scale = torch.where(s["ids_long"] >= 0, s["scale"][ids], torch.zeros((), device=ids.device))
    return s["a"].float()[ids], s["b"].float()[ids], scale[:, None, None]


def _back(padded, place, base):
    """base + the padded rows at their places."""
    S, C = base.shape
    out = torch.zeros(S + 1, C, device=base.device)
    out[place.reshape(-1)] = padded.reshape(-1, C)
    return (base.float() + out[:S]).to(base.dtype)


def _lora_plain(s):
    a, b, scale = _of_groups(s)
    z = torch.bmm(_padded(s["x"], s["place"]), a.transpose(1, 2).contiguous())
    return _back(torch.bmm(z, b.transpose(1, 2).contiguous()) * scale, s["place"], s["y"])


def _lora_grad_plain(s):
    a, b, scale = _of_groups(s)
    n = s["a"].shape[0]
    x, g, z = (_padded(s[v], s["place"]) for v in ("x", "g", "z"))
    u = torch.bmm(g, b) * scale
    gx = _back(torch.bmm(u, a), s["place"], s["gx"])
    ga = torch.bmm(u.transpose(1, 2).contiguous(), x)
    gb = torch.bmm(g.transpose(1, 2).contiguous(), z) * scale
    # an adapter's gradient is the sum over the groups that use it
    uses = (s["ids_long"][None, :] == torch.arange(n, device=ga.device)[:, None]).float()
    ga = (uses @ ga.reshape(len(ga), -1)).reshape(s["a"].shape)
    gb = (uses @ gb.reshape(len(gb), -1)).reshape(s["b"].shape)
    return gx, ga, gb


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if not kind.startswith("lora"):
        return _tokens_exact(s, case, kind)
    x, a, b, scale = s["x"].double(), s["a"].double(), s["b"].double(), s["scale"].double()
    ga, gb = torch.zeros_like(a), torch.zeros_like(b)
    out = s["y"].double() if kind == "lora" else s["gx"].double()
    lo = 0
    for length, i in zip(s["lengths"], s["ids"]):
        rows = slice(lo, lo + length)
        lo += length
        if i < 0 or not length:
            continue
        if kind == "lora":
            out[rows] += scale[i] * (x[rows] @ a[i].T @ b[i].T)
        else:
            g = s["g"][rows].double()
            u = scale[i] * (g @ b[i])
            out[rows] += u @ a[i]
            ga[i] += u.T @ x[rows]
            gb[i] += scale[i] * (g.T @ s["z"][rows].double())
    return out if kind == "lora" else (out, ga, gb)


def _tokens_exact(s, case, kind):
    T, H, k = case["T"], case["H"], case["k"]
    token = torch.div(s["slots"].long(), k, rounding_mode="floor")
    if kind == "permute":
        return s["x"].double().index_select(0, token)
    w = s["w"].double().reshape(-1).index_select(0, s["slots"].long())
    if kind == "combine_grad":
        g_rows = s["g"].double().index_select(0, token)
        g_w = torch.empty(T * k, dtype=torch.float64, device=DEV)
        g_w.scatter_(0, s["slots"].long(), torch.einsum("ph,ph->p", g_rows, s["rows"].double()))
        return g_rows * w[:, None], g_w.reshape(T, k)
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    # by pieces of the columns: a float64 copy of all rows is large
    for c0 in range(0, H, 512):
        part = s["rows"][:, c0:c0 + 512].double()
        out[:, c0:c0 + 512].index_add_(0, token, part * w[:, None] if kind == "combine" else part)
    return out
