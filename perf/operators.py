"""The serving operators beside the MoE layer's batch path, as cases to measure: the whole layer for a
few tokens, and the latent projections with the low-rank adapters of many requests.

``run`` computes each case either in plain torch operations (``own`` false) or with the calls a user of
this package makes (``own`` true), on the same inputs.  The layer's definition (formulas, routing rules,
residual gates) is the one include/moe.h states.
"""
import math

import torch

own = False

# The two layer shapes of this repository's workloads: the Muse latent layer and the Shazeer layer.
MUSE = dict(d=8192, L=4096, I=4096, n=256, k=8, act="swiglu", dtype="bf16", pre=1, norm=1, resid="gate",
            gate="softmax", rf32=0)
SHAZEER = dict(d=512, L=0, I=1024, n=256, k=4, act="relu", dtype="bf16", pre=0, norm=0, resid="none",
               gate="softmax", rf32=0)

EPS, TAU, FLOOR = 1e-6, 0.3, 1e-3


def listed():
    return [
        # one stream decoding alone: every weight byte is read for one token, latency counts
        dict(MUSE, name="few one token", op="few", T=1, nA=0, rank=0),
        # eight streams, or the verification of seven drafted tokens and one more
        dict(MUSE, name="few eight tokens", op="few", T=8, nA=0, rank=0),
        # three requests, two of them with a fine-tune of their own, on the sigmoid router in fp32
        dict(MUSE, name="few sigmoid, adapters", op="few", T=3, nA=5, rank=16, gate="sigmoid", rf32=1),
        # a small layer of many small experts: launches and hand-overs count, not bytes
        dict(SHAZEER, name="few small experts", op="few", T=4, nA=0, rank=0),
        # the smallest layer there is, in fp32
        dict(SHAZEER, name="few tiny fp32", op="few", T=2, nA=0, rank=0, d=64, I=128, n=8, k=2, dtype="f32"),
        # decode of one request with its adapter
        dict(name="down one token", op="down", T=1, d=8192, L=4096, nA=4, rank=16, mix="each", resid="none"),
        # a decode batch in which every request has another adapter
        dict(name="down decode batch", op="down", T=64, d=8192, L=4096, nA=64, rank=16, mix="each", resid="none"),
        # odd widths and rank, tokens of adapters and of none in any order
        dict(name="down odd sizes", op="down", T=333, d=2112, L=1088, nA=7, rank=24, mix="any", resid="none"),
        # prompts of uneven lengths packed into one batch, an adapter for each
        dict(name="down prompts", op="down", T=16384, d=8192, L=4096, nA=32, rank=16, mix="packed", resid="none"),
        # the way up of a decode batch, larger ranks, fewer adapters than requests
        dict(name="up decode batch", op="up", T=48, d=8192, L=4096, nA=12, rank=64, mix="any", resid="gate"),
        # a chunk of a prompt beside decoding requests
        dict(name="up mixed batch", op="up", T=600, d=8192, L=4096, nA=16, rank=8, mix="any", resid="literal"),
        # packed prompts on the way up
        dict(name="up prompts", op="up", T=8192, d=8192, L=4096, nA=24, rank=32, mix="packed", resid="gate"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        c = dict(rng.choice([MUSE, SHAZEER]), op="few", T=rng.randint(1, 8), nA=0, rank=0)
        wide = c["L"] > 0
        top = 4096 if wide else 1024
        c["d"] = 64 * _log(rng, 1, (8192 if wide else 1024) // 64)
        c["L"] = 64 * _log(rng, 1, top // 64) if wide else 0
        c["I"] = 64 * _log(rng, 1, top // 64)
        c["n"] = _log(rng, 8, 256)
        c["k"] = rng.randint(1, 8)
        if wide:
            c["gate"] = rng.choice(["softmax", "sigmoid"])
            c["rf32"] = int(c["gate"] == "sigmoid")
            c["resid"] = rng.choice(["gate", "literal", "none"])
            if rng.random() < 0.5:
                c["nA"], c["rank"] = rng.randint(1, 9), 8 * rng.randint(1, 8)
        else:
            c["dtype"] = rng.choice(["bf16", "f32"])
            c["norm"] = rng.randint(0, 1)
            if c["dtype"] == "f32":
                c["d"], c["I"] = 64 * rng.randint(1, 4), 64 * rng.randint(1, 8)
        return c
    op = rng.choice(["down", "up"])
    return dict(op=op, T=_log(rng, 1, 16384), d=64 * _log(rng, 4, 128), L=64 * _log(rng, 2, 64),
                nA=_log(rng, 1, 64), rank=8 * rng.choice([1, 1, 2, 2, 3, 4, 5, 8]),
                mix=rng.choice(["any", "each", "packed"]),
                resid="none" if op == "down" else rng.choice(["gate", "literal", "none"]))


# ------------------------------------------------------------------ inputs

def _normal(shape, std, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std)


def _tokens_adapters(case, gen):
    """The adapter of every token, -1 for none."""
    T, nA = case["T"], case["nA"]
    any_ = torch.randint(-1, nA, (T,), generator=gen, device="cuda", dtype=torch.int32)
    mix = case.get("mix", "any")
    if mix == "any":
        return any_
    if mix == "each":
        return torch.randperm(max(T, nA), generator=gen, device="cuda")[:T].remainder(nA).int()
    # packed: prompts of uneven lengths, one after the other
    cuts = torch.rand(nA, generator=gen, device="cuda").cumsum(0)
    at = torch.linspace(0, 1, T, device="cuda") * cuts[-1]
    return torch.searchsorted(cuts, at).clamp_(max=nA - 1).int()


def _adapters(case, gen, down=True, up=True):
    nA, r, d, L = case["nA"], case["rank"], case["d"], case["L"]
    a = {"scale": torch.rand(nA, generator=gen, device="cuda") * 0.75 + 0.25}
    if down:
        a["down_a"] = _normal((nA, r, d), d ** -0.5, gen, torch.bfloat16)
        a["down_b"] = _normal((nA, L, r), r ** -0.5, gen, torch.bfloat16)
    if up:
        a["up_a"] = _normal((nA, r, L), L ** -0.5, gen, torch.bfloat16)
        a["up_b"] = _normal((nA, d, r), r ** -0.5, gen, torch.bfloat16)
    return a


def _config(case):
    import sparse_moe_layer_softmax_b200 as moe
    resid = {"none": moe.MOE_RESID_NONE, "gate": moe.MOE_RESID_MUSE_GATE, "literal": moe.MOE_RESID_LITERAL}
    few = case["op"] == "few"
    return moe.make_config(
        T=case["T"], d_model=case["d"], n_experts=case["n"] if few else 1, top_k=case["k"] if few else 1,
        d_ff=case["I"] if few else 64, d_latent=case["L"],
        dtype=moe.MOE_F32 if few and case["dtype"] == "f32" else moe.MOE_BF16,
        expert_act=moe.MOE_ACT_RELU if few and case["act"] == "relu" else moe.MOE_ACT_SWIGLU,
        pre_norm=case["pre"] if few else 0, expert_norm=case["norm"] if few else 0,
        resid_mode=resid[case["resid"]], eps=EPS, tau=TAU, resid_floor=FLOOR,
        gate_mode=moe.MOE_GATE_SIGMOID if few and case["gate"] == "sigmoid" else moe.MOE_GATE_SOFTMAX,
        router_f32=case["rf32"] if few else 0)


def _keys64(u, w, corr):
    """Router keys in 64 bits: what the selection goes by."""
    l = u.double() @ w.double().T
    return l if corr is None else torch.sigmoid(l) + corr.double()


def _layer_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    T, d, L, I, n, k = (case[x] for x in ("T", "d", "L", "I", "n", "k"))
    E = L or d
    w = {"w_router": _normal((n, d), d ** -0.5, gen, torch.float32 if case["rf32"] else dt),
         "w_gu": _normal((n, (2 if case["act"] == "swiglu" else 1) * I, E), E ** -0.5, gen, dt),
         "w_down": _normal((n, E, I), I ** -0.5, gen, dt)}
    if L:
        w["p_down"] = _normal((L, d), d ** -0.5, gen, dt)
        w["p_up"] = _normal((d, L), L ** -0.5, gen, dt)
    if case["pre"]:
        w["gamma_pre"] = _normal((L,), 0.02, gen, torch.float32)
    if case["norm"]:
        w["gamma_expert"] = _normal((E,), 0.02, gen, torch.float32)
    if case["resid"] != "none":
        w["resid_g"] = torch.rand(d, generator=gen, device="cuda")
    if case["gate"] == "sigmoid":
        w["correction_bias"] = _normal((n,), 0.05, gen, torch.float32)
    # As in every workload of this repository, a token whose k-th and (k+1)-th keys nearly tie is drawn
    # again, so that each order of summation selects the same experts: eight tries a token, the first that
    # is clear.
    u = _normal((8, T, d), 1.0, gen, dt)
    if k < n:
        top = _keys64(u, w["w_router"], w.get("correction_bias")).topk(k + 1, dim=-1).values
        clear = (top[..., k - 1] - top[..., k]) > 1e-3 * top.square().mean(-1).sqrt()
        first = clear.float().argmax(0)
    else:
        first = torch.zeros(T, dtype=torch.long, device="cuda")
    return w, u[first, torch.arange(T, device="cuda")].contiguous(), gen


def prepare(case, seed):
    if case["op"] == "few":
        w, u, gen = _layer_inputs(case, seed)
        s = {"case": case, "w": w, "u": u}
        if case["nA"]:
            s["ad"] = _adapters(case, gen)
            s["which"] = _tokens_adapters(case, gen)
        if own:
            import sparse_moe_layer_softmax_b200 as moe
            s["layer"] = moe.MoELayer(_config(case), w, adapters=s.get("ad"))
        return s
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    T, d, L = case["T"], case["d"], case["L"]
    down = case["op"] == "down"
    s = {"case": case,
         "x": _normal((T, d if down else L), 1.0, gen, torch.bfloat16),
         "p": _normal((L, d) if down else (d, L), (d if down else L) ** -0.5, gen, torch.bfloat16),
         "ad": _adapters(case, gen, down=down, up=not down), "which": _tokens_adapters(case, gen)}
    if not down:
        s["r"] = _normal((T, d), 1.0, gen, torch.bfloat16)
        s["g"] = torch.rand(d, generator=gen, device="cuda")
    if own:
        import sparse_moe_layer_softmax_b200 as moe
        s["cfg"] = _config(case)
        s["adapters"] = moe.make_adapters(s["ad"])
        s["ws"] = torch.empty(moe.adapters_workspace_size(s["cfg"], s["adapters"]), dtype=torch.uint8,
                              device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def _resid(case, r, g, b):
    if case["resid"] == "none":
        return b
    if case["resid"] == "literal":
        return r + g * b
    beta = torch.sigmoid(g / TAU)
    alpha = torch.sqrt(torch.clamp(torch.sigmoid(-g / TAU) * (1 + beta), min=FLOOR))
    return alpha * r + beta * b


def _project(x, p, a, b, scale, which):
    """x p^T and every token's adapter: each token's column block of a product with all adapters."""
    x = x.float()
    y = x @ p.float().T
    nA, r, _ = a.shape
    mine = which[:, None] == torch.arange(nA, device=x.device)
    v = (x @ a.float().reshape(nA * r, -1).T).reshape(-1, nA, r) * (mine * scale)[:, :, None]
    return y + v.reshape(-1, nA * r) @ b.float().permute(0, 2, 1).reshape(nA * r, -1)


def _norm(x, gain):
    return x * (1 + gain) / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)


def _few_plain(s):
    case, w, u, ad = s["case"], s["w"], s["u"], s.get("ad")
    k, I = case["k"], case["I"]
    keys = u.double() @ w["w_router"].double().T  # the selection looks at values next to a border
    if case["gate"] == "sigmoid":
        score = torch.sigmoid(keys)
        idx = torch.sort(score + w["correction_bias"].double(), dim=-1, descending=True, stable=True)[1][:, :k]
        picked = score.gather(1, idx)
        wt = picked / (picked.sum(-1, keepdim=True) + 1e-15)
    else:
        idx = torch.sort(keys, dim=-1, descending=True, stable=True)[1][:, :k]
        wt = torch.softmax(keys.gather(1, idx), -1)
    wt = wt.float()
    z = u.float()
    if case["L"]:
        z = (_project(u, w["p_down"], ad["down_a"], ad["down_b"], ad["scale"], s["which"]) if ad
             else z @ w["p_down"].float().T)
        if case["pre"]:
            z = _norm(z, w["gamma_pre"])
    h = (w["w_gu"][idx].float() @ z[:, None, :, None]).squeeze(-1)
    a = torch.nn.functional.silu(h[..., :I]) * h[..., I:] if case["act"] == "swiglu" else torch.relu(h)
    o = (w["w_down"][idx].float() @ a[..., None]).squeeze(-1)
    if case["norm"]:
        o = _norm(o, w["gamma_expert"])
    y = (wt[..., None] * o).sum(1)
    if case["L"]:
        y = (_project(y, w["p_up"], ad["up_a"], ad["up_b"], ad["scale"], s["which"]) if ad
             else y @ w["p_up"].float().T)
        y = _resid(case, u.float(), w.get("resid_g"), y)
    return {"out": y.to(u.dtype), "idx": idx.int(), "w": wt}


def run(s):
    case = s["case"]
    if own:
        import sparse_moe_layer_softmax_b200 as moe
        if case["op"] == "few":
            T, k, u = case["T"], case["k"], s["u"]
            idx = torch.empty((T, k), dtype=torch.int32, device=u.device)
            wt = torch.empty((T, k), dtype=torch.float32, device=u.device)
            out = s["layer"].forward_few(u, topk_idx_out=idx, topk_w_out=wt, token_adapter=s.get("which"))
            return {"out": out, "idx": idx, "w": wt}
        out = torch.empty((case["T"], s["p"].shape[0]), dtype=torch.bfloat16, device=s["x"].device)
        if case["op"] == "down":
            moe.moe_latent_down_adapters(s["cfg"], s["x"], s["p"], s["adapters"], s["which"], out, s["ws"])
        else:
            moe.moe_latent_up_adapters(s["cfg"], s["x"], s["p"], s["adapters"], s["which"], s["r"], s["g"],
                                       out, s["ws"])
        return out
    if case["op"] == "few":
        return _few_plain(s)
    side = case["op"]
    y = _project(s["x"], s["p"], s["ad"][side + "_a"], s["ad"][side + "_b"], s["ad"]["scale"], s["which"])
    if side == "up":
        y = _resid(case, s["r"].float(), s["g"], y)
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    T, d, L, nA, r = case["T"], case["d"], case["L"], case["nA"], case["rank"]
    size = 4 if case.get("dtype") == "f32" else 2
    used = nA * (1 - (1 - 1 / max(nA, 1)) ** T) if nA else 0  # adapters that T tokens use
    if case["op"] != "few":
        rows = T * (d + L) + (T * d if case["resid"] != "none" else 0)
        return {"bytes": int(2 * (d * L + used * r * (d + L) + rows)),
                "flops": int(2 * T * d * L + 2 * T * r * (d + L))}
    E, I, n, k = L or d, case["I"], case["n"], case["k"]
    per = (3 if case["act"] == "swiglu" else 2) * I * E
    experts = n * (1 - (1 - k / n) ** T)  # distinct experts that T tokens select
    router = n * d * (4 if case["rf32"] or size == 4 else 2)
    dense = 2 * d * L + 2 * used * r * (d + L)
    flops = 2 * T * (n * d + k * per + 2 * d * L + 2 * bool(nA) * r * (d + L))
    return {"bytes": int(size * (experts * per + dense + 2 * T * d) + router), "flops": int(flops)}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_rows(x, p, ad, side, which):
    """Token by adapter: groups of the tokens of one adapter, each with its own two products."""
    x = x.double()
    y = torch.matmul(x, p.double().mT)
    if ad is None:
        return y
    for a in sorted(set(which.tolist()) - {-1}):
        t = (which == a).nonzero().flatten()
        inner = torch.matmul(x[t], ad[side + "_a"][a].double().mT)
        y[t] += ad["scale"][a].double() * torch.matmul(inner, ad[side + "_b"][a].double().mT)
    return y


def _exact_resid(case, r, g, b):
    if case["resid"] == "gate":
        g = g.double()
        beta = 1 / (1 + torch.exp(-g / TAU))
        alpha2 = (1 - beta) * (1 + beta)
        return alpha2.clamp(min=FLOOR).sqrt() * r.double() + beta * b
    return r.double() + g.double() * b if case["resid"] == "literal" else b


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "few":
        y = _exact_rows(s["x"], s["p"], s["ad"], case["op"], s["which"])
        return _exact_resid(case, s["r"], s["g"], y) if case["op"] == "up" else y
    w, u, ad, which = s["w"], s["u"], s.get("ad"), s.get("which")
    T, k, I = case["T"], case["k"], case["I"]
    logits = (u.double()[:, None, :] * w["w_router"].double()[None]).sum(-1)
    score = 1 / (1 + torch.exp(-logits)) if case["gate"] == "sigmoid" else logits
    key = score + w["correction_bias"].double() if case["gate"] == "sigmoid" else logits
    z = _exact_rows(u, w["p_down"], ad, "down", which) if case["L"] else u.double()
    if case["pre"]:
        z = z / (z.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * (1 + w["gamma_pre"].double())
    idx = torch.zeros((T, k), dtype=torch.int32)
    wt = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    y = torch.zeros_like(z)
    ranks = key.tolist()
    for t in range(T):
        order = sorted(range(case["n"]), key=lambda e: (-ranks[t][e], e))[:k]
        idx[t] = torch.tensor(order, dtype=torch.int32)
        picked = score[t, order]
        if case["gate"] == "softmax":
            picked = torch.exp(picked - picked.max())
        wt[t] = picked / (picked.sum() + (1e-15 if case["gate"] == "sigmoid" else 0.0))
        for j, e in enumerate(order):
            h = w["w_gu"][e].double() @ z[t]
            if case["act"] == "swiglu":
                h = h[:I] / (1 + torch.exp(-h[:I])) * h[I:]
            else:
                h = h.clamp(min=0)
            o = w["w_down"][e].double() @ h
            if case["norm"]:
                o = o * (1 + w["gamma_expert"].double())
                o = o / (o.pow(2).mean() + EPS).sqrt()
            y[t] += wt[t, j] * o
    if case["L"]:
        y = _exact_resid(case, u, w.get("resid_g"), _exact_rows(y, w["p_up"], ad, "up", which))
    return {"out": y, "idx": idx.cuda(), "w": wt}
