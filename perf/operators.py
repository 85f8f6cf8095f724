"""What is measured of the training and few-token operators of the MoE layer.

Four operators around the routing path of DeepSeek-V3/V3.2 and Kimi K2:

  combine_backward  gradients of the weighted combine: the expert outputs' rows and the router weights
  gather_backward   gradient of the row gather: each token sums its k sorted rows' gradients
  router_backward   gradients of the gate: from the router weights to the hidden states and the gate weight
  expert_w4         the experts' products on 4-bit weights with group scales, for few tokens

`run` computes the plain form (torch operations in 32 bits) where `own` is false and calls
token_dispatch_fp32_b200 where it is true.  `exact` restates each operator in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one training batch of the full DeepSeek-V3 routing workload: every assignment on 32 hot experts
        {"name": "combine_backward_full", "op": "combine_backward", "T": 16384, "d": 7168, "k": 8, "N_r": 256,
         "dtype": "bf16", "hot": 32},
        # the smallest routing configuration (64 fp32 tokens, top-4 of 64): latency counts
        {"name": "combine_backward_tiny", "op": "combine_backward", "T": 64, "d": 512, "k": 4, "N_r": 64,
         "dtype": "f32", "hot": 0},
        # rows that are no multiple of a vector, an odd number of tokens
        {"name": "combine_backward_odd", "op": "combine_backward", "T": 1999, "d": 1001, "k": 3, "N_r": 40,
         "dtype": "bf16", "hot": 0},
        # the gather's gradient on the same full batch, the shared expert's gradient added on the way
        {"name": "gather_backward_full", "op": "gather_backward", "T": 16384, "d": 7168, "k": 8, "N_r": 256,
         "dtype": "bf16", "hot": 32, "add": True},
        # fp32 rows, a ragged micro-batch
        {"name": "gather_backward_f32", "op": "gather_backward", "T": 1500, "d": 4096, "k": 6, "N_r": 64,
         "dtype": "f32", "hot": 0, "add": False},
        # the gate's gradient of the full DeepSeek-V3 batch, the rows' gradient joined on the way
        {"name": "router_backward_full", "op": "router_backward", "T": 16384, "d": 7168, "k": 8, "N_r": 256,
         "dtype": "bf16", "hot": 32, "softmax": False, "add": True},
        # the Kimi K2 prefill batch: 384 experts, an even load
        {"name": "router_backward_k2", "op": "router_backward", "T": 8192, "d": 7168, "k": 8, "N_r": 384,
         "dtype": "bf16", "hot": 0, "softmax": False, "add": False},
        # the smallest configuration in fp32: latency counts
        {"name": "router_backward_tiny", "op": "router_backward", "T": 64, "d": 512, "k": 4, "N_r": 64,
         "dtype": "f32", "hot": 0, "softmax": False, "add": False},
        # the softmax gate: every logit of a token has a gradient
        {"name": "router_backward_softmax", "op": "router_backward", "T": 4096, "d": 7168, "k": 8, "N_r": 256,
         "dtype": "bf16", "hot": 0, "softmax": True, "add": False},
        # one token of a decode step through one expert layer: eight experts' weights are read
        {"name": "expert_w4_one_token", "op": "expert_w4", "T": 1, "d": 7168, "k": 8, "N_r": 256, "n_out": 2048,
         "group": 32, "scales": "bf16", "hot": 0},
        # a decode batch of 64 positions: nearly every expert is hit, by two rows on average
        {"name": "expert_w4_decode", "op": "expert_w4", "T": 64, "d": 7168, "k": 8, "N_r": 256, "n_out": 2048,
         "group": 32, "scales": "bf16", "hot": 0},
        # a second layer back to wide rows, more tokens, coarser groups, an uneven load
        {"name": "expert_w4_down", "op": "expert_w4", "T": 200, "d": 1408, "k": 6, "N_r": 64, "n_out": 2056,
         "group": 128, "scales": "f32", "hot": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["combine_backward", "gather_backward", "router_backward", "expert_w4"])
    k = rng.randint(1, 8)
    if op == "expert_w4":
        # decode batches: from one token to a few hundred, over weights of up to 256 x 2048 x 7168
        T = _log(rng, 1, 256)
        d = 8 * _log(rng, 64, 896)
        n_out = _log(rng, 256, 2048)
        N_r = max(k, _log(rng, 8, 256))
        return {"op": op, "T": T, "d": d, "k": k, "N_r": N_r, "n_out": n_out,
                "group": rng.choice([32, 64, 128]), "scales": rng.choice(["bf16", "bf16", "f32"]),
                "hot": rng.choice([0, 0, 4])}
    # training batches: from a few tokens to 16384, rows of 256 to 7168 elements, odd ones among them
    T = _log(rng, 16, 16384)
    d = min(7168, 64 * _log(rng, 4, 112) + rng.choice([0, 0, 8, 1]))
    N_r = max(k, 16 * _log(rng, 1, 24), 16)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if dtype == "f32":
        T = max(1, T // 2)
    case = {"op": op, "T": T, "d": d, "k": k, "N_r": N_r, "dtype": dtype,
            "hot": rng.choice([0, 0, 8])}
    if op != "combine_backward":
        case["add"] = rng.choice([False, True])
    if op == "router_backward":
        case["softmax"] = rng.choice([False, False, True])
        if case["softmax"]:
            case["T"] = max(1, case["T"] // 4)
    return case


# ---- inputs -------------------------------------------------------------------------------------------------------


def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _plan(idx, N_r):
    """The dispatch of idx [T,k]: offsets [N_r+1], perm and inv [T*k], as int32."""
    flat = idx.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(perm.numel(), device=perm.device)
    offsets = torch.zeros(N_r + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = torch.bincount(flat, minlength=N_r).cumsum(0)
    return offsets.int(), perm.int(), inv.int()


def _choose(gen, scores, k, hot):
    """k distinct experts per token: the best scores, the first `hot` experts preferred."""
    c = scores.clone()
    if hot:
        c[:, :hot] += 1.0
    return torch.topk(c, k, dim=1).indices


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, d, k, N_r = case["T"], case["d"], case["k"], case["N_r"]
    s = {"case": case}
    if case["op"] in ("combine_backward", "gather_backward"):
        dt = DT[case["dtype"]]
        scores = torch.rand((T, N_r), generator=gen, device="cuda")
        idx = _choose(gen, scores, k, case["hot"])
        s["offsets"], s["perm"], s["inv"] = _plan(idx, N_r)
        if case["op"] == "combine_backward":
            w = scores.gather(1, idx) + 0.05
            s["w"] = w / w.sum(1, keepdim=True) * 2.5
            s["E"] = _rows(gen, T * k, d, dt, 1.0)
            s["dy"] = _rows(gen, T, d, dt, 1e-2)
        else:
            s["dxs"] = _rows(gen, T * k, d, dt, 1e-2)
            s["add"] = _rows(gen, T, d, dt, 1e-2) if case["add"] else None
    elif case["op"] == "router_backward":
        dt = DT[case["dtype"]]
        s["x"] = _rows(gen, T, d, dt, 1.0)
        s["W"] = _randn(gen, (N_r, d), torch.float32, 1.0 / math.sqrt(d))
        s["logits"] = s["x"].float() @ s["W"].t()
        scores = torch.softmax(s["logits"], 1) if case["softmax"] else torch.sigmoid(s["logits"])
        s["idx"] = _choose(gen, scores, k, case["hot"]).int()
        s["offsets"], s["perm"], _ = _plan(s["idx"].long(), N_r)
        s["dw"] = _randn(gen, (T, k), torch.float32, 0.1)
        s["add"] = _rows(gen, T, d, dt, 1e-2) if case["add"] else None
        if own:
            import token_dispatch_fp32_b200 as mr
            flags = mr.MR_SCORE_SOFTMAX if case["softmax"] else 0
            n = mr.mr_router_backward_workspace_size(T, d, N_r, k, flags)
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    else:
        n_out, group = case["n_out"], case["group"]
        scores = torch.rand((T, N_r), generator=gen, device="cuda")
        s["offsets"], s["perm"], _ = _plan(_choose(gen, scores, k, case["hot"]), N_r)
        s["x"] = _rows(gen, T, d, torch.bfloat16, 1.0)
        q = torch.randint(0, 256, (N_r, n_out, d // 2), generator=gen, device="cuda", dtype=torch.uint8)
        n_groups = -(-d // group)
        scales = (torch.rand((N_r, n_out, n_groups), generator=gen, device="cuda") + 0.5) / (4 * math.sqrt(d))
        s["scales"] = scales.to(DT[case["scales"]])
        s["segments"] = s["offsets"].tolist()
        if own:  # the weights are laid out once, when they are loaded
            import token_dispatch_fp32_b200 as mr
            s["W4"] = mr.mr_expert_pack_w4(q, s["scales"], group)
        else:
            s["q"] = q
    return s


def _rows(gen, n, d, dtype, scale):
    """[n, d] normal values, drawn in blocks so that no fp32 copy of the whole is held."""
    out = torch.empty((n, d), dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // d)
    for i in range(0, n, step):
        out[i:i + step] = torch.randn((min(step, n - i), d), generator=gen, device="cuda") * scale
    return out


# ---- the operators ------------------------------------------------------------------------------------------------

EPS = 1e-20
SCALE = 2.5


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import token_dispatch_fp32_b200 as mr
    c = s["case"]
    if c["op"] == "combine_backward":
        return mr.mr_combine_backward(s["dy"], s["E"], s["w"], s["inv"])
    if c["op"] == "gather_backward":
        return mr.mr_gather_rows_backward(s["dxs"], c["k"], s["inv"], add=s["add"])
    if c["op"] == "router_backward":
        return mr.mr_router_backward(s["x"], s["W"], s["logits"], s["idx"], s["dw"], s["perm"], s["offsets"], SCALE,
                                     flags=mr.MR_SCORE_SOFTMAX if c["softmax"] else 0, add=s["add"],
                                     workspace=s["ws"])
    return mr.mr_expert_gemv_gather_w4(s["x"], c["k"], s["perm"], s["offsets"], s["W4"], c["N_r"], c["n_out"],
                                       c["group"], scale_dtype=DT[c["scales"]])


def _run_plain(s):
    c = s["case"]
    k = c["k"]
    if c["op"] == "combine_backward":
        T, d = s["dy"].shape
        inv = s["inv"].long()
        dy = s["dy"].float()
        dE = torch.empty_like(s["E"])
        dE[inv] = (s["w"].reshape(T, k, 1) * dy.reshape(T, 1, d)).reshape(T * k, d).to(dE.dtype)
        dw = (s["E"][inv].float().reshape(T, k, d) * dy.reshape(T, 1, d)).sum(2)
        return dE, dw
    if c["op"] == "gather_backward":
        T, d = s["dxs"].shape[0] // k, s["dxs"].shape[1]
        dx = s["dxs"][s["inv"].long()].float().reshape(T, k, d).sum(1)
        if s["add"] is not None:
            dx = dx + s["add"].float()
        return dx.to(s["dxs"].dtype)
    if c["op"] == "router_backward":
        L, g, idx = s["logits"], s["dw"], s["idx"].long()
        if c["softmax"]:
            p = torch.softmax(L, 1)
            dp = torch.zeros_like(p).scatter_add_(1, idx, g * SCALE)
            dL = p * (dp - (p * dp).sum(1, keepdim=True))
        else:
            l = L.gather(1, idx)
            sc = torch.sigmoid(l)
            den = sc.sum(1, keepdim=True) + EPS
            ds = SCALE / den * (g - (g * sc).sum(1, keepdim=True) / den)
            dL = torch.zeros_like(L).scatter_add_(1, idx, ds * sc * torch.sigmoid(-l))
        dx = dL @ s["W"]
        if s["add"] is not None:
            dx = dx + s["add"].float()
        return dx.to(s["x"].dtype), dL.t() @ s["x"].float()
    out = torch.empty((c["T"] * k, c["n_out"]), dtype=torch.bfloat16, device="cuda")
    seg, tok = s["segments"], s["perm"].long() // k
    for e in range(c["N_r"]):
        a, b = seg[e], seg[e + 1]
        if a < b:
            q = torch.stack((s["q"][e] & 15, s["q"][e] >> 4), 2).reshape(c["n_out"], c["d"])
            sc = s["scales"][e].float().repeat_interleave(c["group"], 1)[:, :c["d"]]
            W = (q.float() - 8) * sc
            out[a:b] = (s["x"][tok[a:b]].float() @ W.t()).bfloat16()
    return out


# ---- what a pass cannot do without --------------------------------------------------------------------------------


def work(case):
    T, d, k, N_r = case["T"], case["d"], case["k"], case["N_r"]
    if case["op"] == "expert_w4":
        n_out = case["n_out"]
        pool = case["hot"] if case["hot"] >= k else N_r
        hit = pool * (1 - (1 - k / pool) ** T)  # experts that some token chose, on average
        weight = n_out * d / 2 + n_out * -(-d // case["group"]) * (2 if case["scales"] == "bf16" else 4)
        return {"bytes": hit * weight + 2 * T * d + 2 * T * k * n_out + 8 * T * k, "flops": 2 * T * k * n_out * d}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "combine_backward":
        return {"bytes": (2 * T * k + T) * d * e + 12 * T * k, "flops": 3 * T * k * d}
    if case["op"] == "gather_backward":
        return {"bytes": (T * k + T + (T if case["add"] else 0)) * d * e + 4 * T * k, "flops": T * k * d}
    rows = T * d * e * (3 if case["add"] else 2)
    logits = 4 * T * (N_r if case["softmax"] else k)
    return {"bytes": rows + 8 * N_r * d + logits + 12 * T * k,
            "flops": 4 * T * (N_r if case["softmax"] else k) * d}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------


def exact(case, seed):
    T, d, k, N_r, op = case["T"], case["d"], case["k"], case["N_r"], case["op"]
    s = prepare(case, seed)
    if op in ("combine_backward", "gather_backward"):
        row = s["inv"].long().view(T, k)
        step = max(1, (1 << 26) // (d * k))
        if op == "combine_backward":
            dE = torch.empty((T * k, d), dtype=torch.float64, device="cuda")
            dw = torch.empty((T, k), dtype=torch.float64, device="cuda")
            for t in range(0, T, step):
                g = s["dy"][t:t + step].double()
                for j in range(k):
                    r = row[t:t + step, j]
                    dw[t:t + step, j] = torch.einsum("td,td->t", g, s["E"][r].double())
                    dE[r] = g * s["w"][t:t + step, j, None].double()
            return dE, dw
        dx = s["add"].double() if case["add"] else torch.zeros((T, d), dtype=torch.float64, device="cuda")
        for t in range(0, T, step):
            for j in range(k):
                dx[t:t + step] += s["dxs"][row[t:t + step, j]].double()
        return dx
    if op == "router_backward":
        L, g, idx = s["logits"].double(), s["dw"].double(), s["idx"].long()
        t = torch.arange(T, device="cuda")
        dL = torch.zeros_like(L)
        if case["softmax"]:
            p = torch.exp(L - torch.logsumexp(L, 1, keepdim=True))
            mean = torch.zeros(T, dtype=torch.float64, device="cuda")
            for j in range(k):
                dL[t, idx[:, j]] += SCALE * g[:, j] * p[t, idx[:, j]]
                mean += SCALE * g[:, j] * p[t, idx[:, j]]
            dL -= p * mean[:, None]
        else:
            u = [1 / (1 + torch.exp(-L[t, idx[:, j]])) for j in range(k)]
            S = sum(u) + EPS
            mean = sum(g[:, j] * u[j] for j in range(k)) / S
            for j in range(k):
                l = L[t, idx[:, j]]
                dL[t, idx[:, j]] += SCALE * (g[:, j] - mean) / S * torch.exp(-l) / (1 + torch.exp(-l)) ** 2
        dx = dL @ s["W"].double()
        if case["add"]:
            dx += s["add"].double()
        dW = torch.zeros((N_r, d), dtype=torch.float64, device="cuda")
        for i in range(0, T, 4096):
            dW += dL[i:i + 4096].t() @ s["x"][i:i + 4096].double()
        return dx, dW
    # expert_w4: the drawn nibbles again (they are laid out otherwise where `own` is true)
    q = s["q"] if "q" in s else _nibbles(case, seed)
    out = torch.empty((T * k, case["n_out"]), dtype=torch.float64, device="cuda")
    group, tok = case["group"], s["perm"].long() // k
    for e in range(N_r):
        a, b = s["segments"][e], s["segments"][e + 1]
        if a == b:
            continue
        xe = s["x"][tok[a:b]].double()
        W = torch.empty((case["n_out"], d), dtype=torch.float64, device="cuda")
        W[:, 0::2] = (q[e] & 15).double() - 8
        W[:, 1::2] = (q[e] >> 4).double() - 8
        for i, c0 in enumerate(range(0, d, group)):
            W[:, c0:c0 + group] *= s["scales"][e, :, i, None].double()
        out[a:b] = xe @ W.t()
    return out


def _nibbles(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, d, N_r, n_out = case["T"], case["d"], case["N_r"], case["n_out"]
    torch.rand((T, N_r), generator=gen, device="cuda")
    _rows(gen, T, d, torch.bfloat16, 1.0)
    return torch.randint(0, 256, (N_r, n_out, d // 2), generator=gen, device="cuda", dtype=torch.uint8)
