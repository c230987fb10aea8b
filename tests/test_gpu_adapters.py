"""moe_latent_down_adapters, moe_latent_up_adapters and moe_layer_forward_adapters against a 64-bit
evaluation.

Tolerances, per element.  Storing bf16 is off by at most 2^-8 of the value.  In batches on the tensor-core
path v = scale A x is rounded to bf16: at most 2^-8 of every product B_fr v_r, so 2^-8 of
sum_r |B_fr v_r|.  The fp32 sums over K products err like 16 sqrt(K) 2^-24 of the row's largest value.  The
way up rounds b to bf16 before the residual update (as moe_latent_up does): beta 2^-8 |b| more.
"""
import pytest

torch = pytest.importorskip("torch")
import sparse_moe_layer_softmax_b200 as moe  # noqa: E402

import serving_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def setup(T, d, L, nA, rank, mix="any", seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(T=T, d=d, L=L, n=1, k=1, I=64, act="swiglu", norm=0)
    ad, which = ref.make_adapters(c, nA, rank, gen)
    if mix == "packed":
        which = torch.arange(T, device="cuda").mul(min(nA, 5)).div(T, rounding_mode="floor").int()
    elif mix == "each":
        which = torch.arange(T, device="cuda").remainder(nA).int()
    elif mix == "one":
        which = torch.full((T,), nA - 1, dtype=torch.int32, device="cuda")
    elif mix == "none":
        which = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    w = {"p_down": ref.normal((L, d), d ** -0.5, gen), "p_up": ref.normal((d, L), L ** -0.5, gen),
         "g": torch.rand(d, generator=gen, device="cuda")}
    x = {"u": ref.normal((T, d), 1.0, gen), "y": ref.normal((T, L), 1.0, gen), "r": ref.normal((T, d), 1.0, gen)}
    return c, ad, which.contiguous(), w, x


def run_down(c, ad, which, w, x, fill=0xFF, stream=None, out=None):
    cfg, a = ref.config(c), moe.make_adapters(ad)
    ws = torch.full((moe.adapters_workspace_size(cfg, a),), fill, dtype=torch.uint8, device="cuda")
    out = torch.full((c["T"], c["L"]), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    moe.moe_latent_down_adapters(cfg, x["u"], w["p_down"], a, which, out, ws, stream=stream)
    return out


def run_up(c, ad, which, w, x, resid, fill=0xFF):
    cfg, a = ref.config(dict(c, resid=resid)), moe.make_adapters(ad)
    ws = torch.full((moe.adapters_workspace_size(cfg, a),), fill, dtype=torch.uint8, device="cuda")
    out = torch.full((c["T"], c["d"]), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_latent_up_adapters(cfg, x["y"], w["p_up"], a, which, x["r"], w["g"], out, ws)
    return out


def definition(x, p, a, b, scale, which):
    """The projection and, for the tolerance, sum_r |B_fr v_r| of every element."""
    x = x.double()
    y = x @ p.double().T
    mag = torch.zeros_like(y)
    for i in set(which.tolist()) - {-1}:
        t = (which == i).nonzero().flatten()
        v = scale[i].double() * (x[t] @ a[i].double().T)
        y[t] += v @ b[i].double().T
        mag[t] = v.abs() @ b[i].double().abs().T
    return y, mag


def check(got, want, mag, K, extra=0.0):
    tol = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -8 * mag + \
        16 * K ** 0.5 * 2.0 ** -24 * want.abs().amax(-1, keepdim=True) + extra
    err = (got.double() - want).abs()
    worst = (err / tol.clamp(min=1e-30)).max().item()
    assert worst <= 1.0, f"error {worst:.2f} of the tolerance"


def check_both(T, d, L, nA, rank, mix="any", seed=1, resid="gate"):
    c, ad, which, w, x = setup(T, d, L, nA, rank, mix, seed)
    want, mag = definition(x["u"], w["p_down"], ad["down_a"], ad["down_b"], ad["scale"], which)
    check(run_down(c, ad, which, w, x), want, mag, d)
    b, mag = definition(x["y"], w["p_up"], ad["up_a"], ad["up_b"], ad["scale"], which)
    want = ref.residual(resid, b, x["r"], w["g"], 0.3, 1e-3)
    beta = {"none": 0.0, "literal": w["g"].double(), "gate": torch.sigmoid(w["g"].double() / 0.3)}[resid]
    scale = 1.0 if resid == "none" else beta
    check(run_up(c, ad, which, w, x, resid), want, mag * scale, L, 2.0 ** -8 * b.abs() * beta)
    assert moe.moe_get_device_status() == 0


CASES = [(T, 256, 128, 3, 16) for T in (1, 2, 17, 63, 64, 65, 128, 129, 256, 257)] + [
    (1, 512, 256, 1, 8), (64, 1024, 512, 64, 16), (50, 512, 384, 7, 24), (33, 256, 256, 2, 128),
    (9, 192, 64, 3, 8), (40, 64, 64, 2, 16), (64, 320, 192, 5, 40),  # widths that split no reduction
    (100, 512, 256, 40, 8), (200, 256, 384, 300, 16), (333, 576, 320, 7, 24), (300, 256, 256, 2, 72),
    (700, 512, 512, 3, 128), (1000, 256, 256, 300, 8), (2047, 256, 256, 6, 64), (2048, 512, 256, 9, 16),
    (2300, 256, 512, 70, 56), (4099, 512, 256, 3, 32), (2500, 128, 128, 4, 120)]


@pytest.mark.parametrize("T,d,L,nA,rank", CASES)
def test_adapted_projections(T, d, L, nA, rank):
    check_both(T, d, L, nA, rank, seed=T + rank)


@pytest.mark.parametrize("mix", ["packed", "each", "one", "none"])
@pytest.mark.parametrize("T", [5, 64, 90, 500, 2600])
def test_adapted_projections_mixes(T, mix):
    check_both(T, 512, 256, 11, 16, mix, seed=T, resid="literal")
    check_both(T, 256, 512, 11, 64, mix, seed=T + 1, resid="none")


def test_adapted_projections_full_width():
    """The Muse widths: a decode batch, a small prompt and a prefill batch."""
    for T, nA, rank, mix in ((1, 4, 16, "each"), (64, 64, 16, "each"), (50, 5, 128, "any"), (64, 64, 128, "each"),
                               (300, 16, 8, "any"), (3000, 8, 32, "packed")):
        check_both(T, 8192, 4096, nA, rank, mix, seed=T)


@pytest.mark.parametrize("T", [1, 30, 64, 65, 200, 600, 2100])
def test_tokens_without_an_adapter_get_the_plain_bits(T):
    c, ad, which, w, x = setup(T, 512, 256, 5, 16)
    cfg = ref.config(dict(c, resid="gate"))
    z, out = torch.empty_like(x["y"]), torch.empty_like(x["r"])
    moe.moe_latent_down(cfg, x["u"], w["p_down"], z)
    moe.moe_latent_up(cfg, x["y"], w["p_up"], x["r"], w["g"], out)
    none = which < 0
    assert torch.equal(run_down(c, ad, which, w, x)[none], z[none])
    assert torch.equal(run_up(c, ad, which, w, x, "gate")[none], out[none])


@pytest.mark.parametrize("T", [7, 64, 150, 400, 2200])
def test_results_repeat_and_ignore_the_workspace(T):
    c, ad, which, w, x = setup(T, 512, 256, 9, 24)
    a = run_down(c, ad, which, w, x)
    assert torch.equal(a, run_down(c, ad, which, w, x, fill=0))
    assert torch.equal(a, run_down(c, ad, which, w, x, fill=0x3C))
    # the order of the adapters in the stack does not matter
    perm = torch.randperm(9, device="cuda")
    moved = {k: v[perm].contiguous() for k, v in ad.items()}
    back = torch.argsort(perm).int()
    at = torch.where(which >= 0, back[which.clamp(min=0).long()], which).int()
    assert torch.equal(a, run_down(c, moved, at, w, x))


@pytest.mark.parametrize("T", [20, 64, 100, 500, 2100])
def test_broken_adapters_stay_with_their_tokens(T):
    c, ad, which, w, x = setup(T, 512, 256, 4, 16, seed=T)
    which[:2] = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    good = run_down(c, ad, which, w, x)
    assert moe.moe_get_device_status() == 0
    ad["down_b"][2, 5, 3] = float("inf")
    ad["down_a"][1, 0, 7] = float("nan")
    got = run_down(c, ad, which, w, x)
    status = moe.moe_get_device_status()
    clean = (which != 1) & (which != 2)
    assert torch.equal(got[clean], good[clean])
    assert got[which == 1].isnan().any(-1).all()  # a broken A reaches all of its tokens' features
    if T > 64:
        assert status == moe.STATUS_CODES["MOE_ERR_DEVICE_CHECK"]
        assert got[which == 2].isfinite().all()
    else:
        assert status == 0
        assert not got[which == 2][:, 5].isfinite().any()
    # an unused adapter may hold anything
    c, ad, which, w, x = setup(T, 512, 256, 4, 16, seed=T)
    which[which == 3] = -1
    good = run_down(c, ad, which, w, x)
    for name in ("down_a", "down_b", "scale"):
        ad[name][3] = float("nan")
    assert torch.equal(run_down(c, ad, which, w, x), good)
    assert moe.moe_get_device_status() == 0


@pytest.mark.parametrize("T", [20, 300])
def test_bad_inputs_rows_stay_alone(T):
    c, ad, which, w, x = setup(T, 512, 256, 4, 16)
    good = run_down(c, ad, which, w, x)
    x["u"][7, 3] = float("nan")
    got = run_down(c, ad, which, w, x)
    keep = torch.arange(T, device="cuda") != 7
    assert torch.equal(got[keep], good[keep]) and got[7].isnan().all()


@pytest.mark.parametrize("T", [20, 300, 2100])
def test_bad_adapter_index_is_latched_and_means_none(T):
    c, ad, which, w, x = setup(T, 512, 256, 4, 16)
    which[3], which[T - 1] = -1, -1
    good = run_down(c, ad, which, w, x)
    assert moe.moe_get_device_status() == 0
    which[3], which[T - 1] = 4, -2
    got = run_down(c, ad, which, w, x)
    assert moe.moe_get_device_status() == moe.STATUS_CODES["MOE_ERR_DEVICE_CHECK"]
    assert torch.equal(got, good)


@pytest.mark.parametrize("T", [30, 100, 600, 2100])
def test_in_a_graph_after_other_work_and_on_two_streams(T):
    """Replays with new tokens and adapters; inputs written by a kernel just before the call; two calls
    at a time on two streams."""
    c, ad, which, w, x = setup(T, 512, 256, 6, 16)
    cfg, a = ref.config(c), moe.make_adapters(ad)
    size = moe.adapters_workspace_size(cfg, a)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    u, wh, out = x["u"].clone(), which.clone(), torch.empty_like(x["y"])

    def call(i, src, dst):
        moe.moe_latent_down_adapters(cfg, src, w["p_down"], a, wh, dst, ws[i])

    call(0, u, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, u, out)
        call(0, u, out)
    for k in range(3):
        u.copy_(x["u"].roll(k, 0))
        wh.copy_(which.roll(2 * k, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run_down(c, ad, wh.clone(), w, {"u": u.clone()}))
    wh.copy_(which)
    want = run_down(c, ad, which, w, x)
    big = torch.randn(4096, 4096, device="cuda")
    for _ in range(5):  # the producer of u runs right before
        u.zero_()
        big = big @ big * 1e-2
        u.copy_(x["u"])
        call(0, u, out)
        got = out.clone()
        assert torch.equal(got, want)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                o = torch.empty_like(out)
                call(i, x["u"], o)
                outs[i].append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs[0] + outs[1])


def test_writes_nothing_beside_its_output():
    for T in (5, 64, 77, 300, 2100):
        c, ad, which, w, x = setup(T, 256, 128, 3, 16)
        cfg, a = ref.config(c), moe.make_adapters(ad)
        need = moe.adapters_workspace_size(cfg, a)
        ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        buf = torch.full((T + 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_latent_down_adapters(cfg, x["u"], w["p_down"], a, which, buf[2:T + 2], ws, workspace_bytes=need)
        torch.cuda.synchronize()
        assert (buf[:2] == 5).all() and (buf[T + 2:] == 5).all() and (ws[need:] == 0xA5).all()


# ------------------------------------------------------------------ as they are used together

LAYER = dict(d=512, L=256, I=192, n=16, k=4, act="swiglu", resid="gate")


@pytest.mark.parametrize("T", [1, 6, 64, 65, 300, 2100])
def test_layer_with_adapters(T):
    """The whole layer with adapters: within the batch path's bar of the definition (2e-2 of a row's
    largest value), from one token to a prompt; the few-token kernel on the same layer agrees."""
    c = dict(LAYER, T=T)
    w, u, gen = ref.make_layer(c, 40 + T)
    ad, which = ref.make_adapters(c, 5, 16, gen)
    layer = moe.MoELayer(ref.config(c), w, adapters=ad)
    idx = torch.empty((T, 4), dtype=torch.int32, device="cuda")
    out = layer.forward(u, topk_idx_out=idx, token_adapter=which)
    assert moe.moe_get_device_status() == 0
    rows = torch.arange(T)[:: max(1, T // 40)]
    want, widx, _, _ = ref.layer(dict(c, T=len(rows)), w, u[rows], u[rows], ad, which[rows])
    assert torch.equal(idx[rows], widx)
    assert ((out[rows].double() - want).abs().amax(-1) <= 2e-2 * want.abs().amax(-1)).all()
    if T <= moe.FEW_MAX_TOKENS:
        few = layer.forward_few(u, token_adapter=which)
        assert ((few.double() - want).abs().amax(-1) <= 2e-2 * want.abs().amax(-1)).all()
    # the layer's own forward is not touched by its adapters
    assert torch.equal(layer.forward(u), moe.MoELayer(ref.config(c), w).forward(u))


def test_layer_with_adapters_and_norms():
    c = dict(LAYER, T=70, input_norm=1, post_norm=1, gate="sigmoid", rf32=1)
    w, h, gen = ref.make_layer(c, 50)
    ad, which = ref.make_adapters(c, 3, 8, gen)
    layer = moe.MoELayer(ref.config(c), w, adapters=ad)
    out = layer.forward(h, r=h, token_adapter=which)
    want = ref.layer(c, w, h, h, ad, which)[0]
    assert ((out.double() - want).abs().amax(-1) <= 2e-2 * want.abs().amax(-1)).all()


def test_decode_steps_with_drafts_and_adapters():
    """A serving loop: a prompt through the batch path, then steps of 1 to 8 tokens through the few-token
    kernel on the same weights and adapters, each against the definition."""
    c = dict(LAYER, T=100)
    w, u, gen = ref.make_layer(c, 60)
    ad, which = ref.make_adapters(c, 5, 16, gen)
    batch = moe.MoELayer(ref.config(c), w, adapters=ad).forward(u, token_adapter=which)
    at = 0
    for T in (1, 8, 3, 5, 1, 7):
        layer = moe.MoELayer(ref.config(dict(c, T=T)), w, adapters=ad)
        got = layer.forward_few(u[at:at + T].contiguous(), token_adapter=which[at:at + T].contiguous())
        # both are within 2e-2 of the definition
        assert ((got.double() - batch[at:at + T].double()).abs().amax(-1)
                <= 2e-2 * batch[at:at + T].double().abs().amax(-1)).all()
        at += T
    assert moe.moe_get_device_status() == 0
