"""Plain 64-bit evaluations of the few-token layer and of the adapted latent projections, for the GPU
tests: the formulas of include/moe.h in torch float64, one token at a time, sharing no code with the
library.  Also the random inputs those tests draw."""
import torch

import sparse_moe_layer_softmax_b200 as moe

RESID = {"none": moe.MOE_RESID_NONE, "gate": moe.MOE_RESID_MUSE_GATE, "literal": moe.MOE_RESID_LITERAL}


def adapted(x, p, a, b, scale, which):
    """x p^T + scale[a] B_a (A_a x) for the tokens whose adapter a is at least 0."""
    x = x.double()
    y = x @ p.double().T
    if a is not None:
        for t, i in enumerate(which.tolist()):
            if i >= 0:
                y[t] += scale[i].double() * (b[i].double() @ (a[i].double() @ x[t]))
    return y


def residual(mode, b, r, g, tau, floor):
    if mode == "none":
        return b
    r, g = r.double(), g.double()
    if mode == "literal":
        return r + g * b
    beta = torch.sigmoid(g / tau)
    return torch.sqrt(torch.clamp(torch.sigmoid(-g / tau) * (1 + beta), min=floor)) * r + beta * b


def centred(x, gamma, eps):
    return (1 + gamma.double()) * x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)


def scaled(x, gamma, eps):
    s = (1 + gamma.double()) * x
    return s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)


def layer(c, w, u, r, ad=None, which=None):
    """The whole layer.  c: a dict of the case's fields.  Returns out [T, d] float64, idx, w, keys."""
    if c.get("input_norm"):
        u = centred(r.double(), w["gamma_in"], 1e-5).to(torch.bfloat16)  # the path's one rounding of u
    l = u.double() @ w["w_router"].double().T
    if c.get("gate") == "sigmoid":
        l = c.get("mult", 1.0) * l
    if w.get("logit_bias") is not None:
        l = l + w["logit_bias"].double()
    score = torch.sigmoid(l) if c.get("gate") == "sigmoid" else l
    keys = score + w["correction_bias"].double() if w.get("correction_bias") is not None else score
    k = c["k"]
    idx = torch.sort(keys, dim=-1, descending=True, stable=True)[1][:, :k]
    sel = score.gather(1, idx)
    wt = sel / (sel.sum(-1, keepdim=True) + 1e-15) if c.get("gate") == "sigmoid" else torch.softmax(sel, -1)
    wt = wt * c.get("routed_scale", 1.0)
    z = u.double()
    if c["L"]:
        z = adapted(u, w["p_down"], ad and ad["down_a"], ad and ad["down_b"], ad and ad["scale"], which)
        if c.get("pre", 1):
            z = centred(z, w["gamma_pre"], 1e-6)
    y = torch.zeros_like(z)
    for t in range(u.shape[0]):
        for j in range(k):
            e = int(idx[t, j])
            h = w["w_gu"][e].double() @ z[t]
            if c["act"] == "swiglu":
                h = torch.nn.functional.silu(h[:c["I"]]) * h[c["I"]:]
            else:
                h = torch.relu(h)
            o = w["w_down"][e].double() @ h
            if c.get("norm", 1):
                o = scaled(o, w["gamma_expert"], 1e-6)
            y[t] += wt[t, j] * o
    if c["L"]:
        b = adapted(y, w["p_up"], ad and ad["up_a"], ad and ad["up_b"], ad and ad["scale"], which)
        if c.get("post_norm"):
            b = scaled(b, w["gamma_post"], 1e-5)
        y = residual(c.get("resid", "none"), b, r, w.get("resid_g"), 0.3, 1e-3)
    return y, idx.int(), wt, keys


def normal(shape, std, gen, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def make_layer(c, seed):
    """Weights and tokens of a case; tokens whose k-th and (k+1)-th router keys nearly tie are drawn
    again, so that fp32 and fp64 sums select the same experts."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f32 = c.get("dtype") == "f32"
    dt = torch.float32 if f32 else torch.bfloat16
    T, d, L, I, n = (c[x] for x in ("T", "d", "L", "I", "n"))
    E = L or d
    w = {"w_router": normal((n, d), d ** -0.5, gen, torch.float32 if c.get("rf32") else dt),
         "w_gu": normal((n, (2 if c["act"] == "swiglu" else 1) * I, E), E ** -0.5, gen, dt),
         "w_down": normal((n, E, I), I ** -0.5, gen, dt)}
    if L:
        w["p_down"] = normal((L, d), d ** -0.5, gen, dt)
        w["p_up"] = normal((d, L), L ** -0.5, gen, dt)
        w["gamma_pre"] = normal((L,), 0.1, gen, torch.float32)
    w["gamma_expert"] = normal((E,), 0.1, gen, torch.float32)
    w["resid_g"] = torch.rand(d, generator=gen, device="cuda")
    w["gamma_in"] = normal((d,), 0.1, gen, torch.float32)
    w["gamma_post"] = normal((d,), 0.1, gen, torch.float32)
    if c.get("gate") == "sigmoid":
        w["correction_bias"] = normal((n,), 0.05, gen, torch.float32)
    if c.get("bias"):
        w["logit_bias"] = normal((n,), 0.5, gen, torch.float32)
    u = normal((T, d), 1.0, gen, dt)
    for _ in range(20):
        probe = dict(c, L=0, I=0)
        src = centred(u.double(), w["gamma_in"], 1e-5).to(dt) if c.get("input_norm") else u
        keys = layer(dict(probe, k=0, input_norm=0), dict(w, w_router=w["w_router"]), src, u)[3]
        if c["k"] >= n:
            break
        top = torch.sort(keys, dim=-1, descending=True)[0]
        near = (top[:, c["k"] - 1] - top[:, c["k"]]) < 2e-3 * keys.square().mean(-1).sqrt()
        if not near.any():
            break
        u[near] = normal((int(near.sum()), d), 1.0, gen, dt)
    return w, u, gen


def make_adapters(c, nA, rank, gen, T=None):
    d, L = c["d"], c["L"]
    ad = {"down_a": normal((nA, rank, d), d ** -0.5, gen), "down_b": normal((nA, L, rank), rank ** -0.5, gen),
          "up_a": normal((nA, rank, L), L ** -0.5, gen), "up_b": normal((nA, d, rank), rank ** -0.5, gen),
          "scale": torch.rand(nA, generator=gen, device="cuda") + 0.25}
    which = torch.randint(-1, nA, (T or c["T"],), generator=gen, device="cuda", dtype=torch.int32)
    return ad, which


def config(c):
    return moe.make_config(
        T=c["T"], d_model=c["d"], n_experts=c["n"], top_k=c["k"], d_ff=c["I"], d_latent=c["L"],
        dtype=moe.MOE_F32 if c.get("dtype") == "f32" else moe.MOE_BF16,
        expert_act=moe.MOE_ACT_SWIGLU if c["act"] == "swiglu" else moe.MOE_ACT_RELU,
        pre_norm=c.get("pre", 1) if c["L"] else 0, expert_norm=c.get("norm", 1),
        resid_mode=RESID[c.get("resid", "none")], routed_scale=c.get("routed_scale", 1.0),
        gate_mode=moe.MOE_GATE_SIGMOID if c.get("gate") == "sigmoid" else moe.MOE_GATE_SOFTMAX,
        router_f32=c.get("rf32", 0), logit_mult=c.get("mult", 1.0),
        input_norm=c.get("input_norm", 0), post_norm=c.get("post_norm", 0))
