"""moe_layer_forward_few: the whole layer for 1 to 8 tokens in one kernel, against a 64-bit evaluation.

Tolerances.  The layer's intermediates stay in fp32, and enter the products as hi + lo bf16 pairs: a
relative error of at most 2^-17 per activation value, independent from value to value, so a product's
error is about 2^-17 of its rms; SwiGLU passes on at most three times the relative error of its
input; four products in a row give an rms error of at most about 10 * 2^-17 of the result's rms, and no
element of some 10^4 lies beyond five of those: 2^-11 of the row's rms (of its largest value, when the
residual or a norm makes rms smaller).  Storing bf16 adds half a step, 2^-8 of the value.  fp32 layers:
sums of at most 512 products, each with relative error 2^-24 per step, four in a row: 1e-5 of the rms.
"""
import pytest

torch = pytest.importorskip("torch")
import sparse_moe_layer_softmax_b200 as moe  # noqa: E402

import serving_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

MUSE = dict(d=256, L=128, I=192, n=16, k=4, act="swiglu", resid="gate")
SHAZ = dict(d=128, L=0, I=256, n=16, k=4, act="relu", norm=0)


def close(c, out, want):
    f32 = c.get("dtype") == "f32"
    rms = want.square().mean(-1, keepdim=True).sqrt()
    tol = 1e-5 * rms + 2.0 ** -24 * want.abs() if f32 else 2.0 ** -11 * rms + 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8)
    err = (out.double() - want).abs()
    worst = (err / tol.clamp(min=1e-30)).max().item()
    assert worst <= 1.0, f"error {worst:.2f} of the tolerance, max {err.max().item():.3e}"


def run_few(c, w, u, r=None, ad=None, which=None, layer=None, **kw):
    layer = layer or moe.MoELayer(ref.config(c), w, adapters=ad)
    T, k, n = c["T"], c["k"], c["n"]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    wt = torch.full((T, k), -7.0, device="cuda")
    lg = torch.full((T, n), -7.0, device="cuda")
    out = layer.forward_few(u, r, topk_idx_out=idx, topk_w_out=wt, logits_out=lg, token_adapter=which, **kw)
    return out, idx, wt, lg, layer


def check(c, seed, nA=0, rank=0):
    w, u, gen = ref.make_layer(c, seed)
    ad = which = None
    if nA:
        ad, which = ref.make_adapters(c, nA, rank, gen)
    r = u if c.get("input_norm") else ref.normal(u.shape, 1.0, gen, u.dtype)
    out, idx, wt, lg, _ = run_few(c, w, None if c.get("input_norm") else u, r, ad, which,
                                  **({"out": torch.empty_like(u)} if c.get("input_norm") else {}))
    assert moe.moe_get_device_status() == 0
    want, widx, wwt, keys = ref.layer(c, w, u, r, ad, which)
    assert torch.equal(idx, widx)
    torch.testing.assert_close(wt.double(), wwt, rtol=4e-6, atol=1e-7)
    score = keys - w["correction_bias"].double() if w.get("correction_bias") is not None else keys
    torch.testing.assert_close(lg.double(), score, rtol=0, atol=4e-6 * max(1.0, keys.abs().max().item()))
    close(c, out, want)
    return out


CASES = [
    dict(MUSE, T=1), dict(MUSE, T=2), dict(MUSE, T=7), dict(MUSE, T=8),
    dict(MUSE, T=8, k=8, n=13), dict(MUSE, T=3, k=1, n=1), dict(MUSE, T=5, n=256, k=8),
    dict(MUSE, T=4, resid="literal"), dict(MUSE, T=4, resid="none"), dict(MUSE, T=4, pre=0, norm=0),
    dict(MUSE, T=6, act="relu", bias=1, routed_scale=2.5),
    dict(MUSE, T=3, gate="sigmoid", rf32=1, mult=2.0), dict(MUSE, T=8, gate="sigmoid", bias=1),
    dict(MUSE, T=5, rf32=1, d=192), dict(MUSE, T=4, input_norm=1), dict(MUSE, T=5, post_norm=1),
    dict(MUSE, T=8, input_norm=1, post_norm=1, resid="literal"),
    dict(MUSE, T=2, d=64, L=64, I=64, n=3, k=2), dict(MUSE, T=8, d=1984, L=832, I=576, n=40, k=6),
    dict(MUSE, T=8, d=2560, L=1536, I=1088, n=12, k=3),
    dict(SHAZ, T=1), dict(SHAZ, T=8, norm=1), dict(SHAZ, T=5, act="swiglu"), dict(SHAZ, T=4, d=512, I=1024, n=256),
    dict(SHAZ, T=3, dtype="f32", d=64, I=128, n=8, k=2), dict(SHAZ, T=8, dtype="f32", norm=1, act="swiglu"),
    dict(SHAZ, T=2, dtype="f32", d=96, I=160, n=5, k=5, gate="sigmoid"),
]


@pytest.mark.parametrize("c", CASES, ids=[" ".join(f"{k}={v}" for k, v in c.items()) for c in CASES])
def test_few_matches_definition(c):
    check(c, 100 + CASES.index(c))


@pytest.mark.parametrize("T,nA,rank", [(1, 1, 8), (8, 3, 16), (5, 9, 24), (8, 8, 64), (3, 2, 128), (8, 2, 40)])
def test_few_with_adapters(T, nA, rank):
    check(dict(MUSE, T=T), 200 + T + rank, nA, rank)
    check(dict(MUSE, T=T, d=320, L=192, post_norm=1), 300 + T + rank, nA, rank)


def test_few_full_width():
    """The Muse widths with 32 experts: long reductions, every ring slot reused many times."""
    c = dict(MUSE, T=8, d=8192, L=4096, I=4096, n=32, k=8)
    check(c, 11, 5, 16)
    check(dict(c, T=1), 12)


def test_few_ties_take_the_lower_index():
    c = dict(MUSE, T=4, n=32, k=4)
    w, u, gen = ref.make_layer(c, 21)
    w["w_router"][16:] = w["w_router"][:16]  # experts e and e + 16 tie bit for bit
    _, idx, _, _, _ = run_few(c, w, u)
    keys = u.double() @ w["w_router"].double().T
    keys[:, 16:] = keys[:, :16]
    assert torch.equal(idx, torch.sort(keys, dim=-1, descending=True, stable=True)[1][:, :4].int())


def test_few_every_token_on_the_same_experts():
    c = dict(MUSE, T=8, n=32, k=4, bias=1)
    w, u, gen = ref.make_layer(c, 22)
    w["logit_bias"] = torch.zeros(32, device="cuda")
    w["logit_bias"][[3, 9, 17, 30]] = 100.0
    out, idx, _, _, _ = run_few(c, w, u)
    assert all(sorted(row) == [3, 9, 17, 30] for row in idx.tolist())
    close(c, out, ref.layer(c, w, u, u)[0])


@pytest.mark.parametrize("T,d,L,I", [(8, 4096, 2048, 4096), (7, 2048, 2048, 3392), (8, 64, 128, 3392), (6, 8192, 512, 4096)])
def test_few_wide_hidden_layers_with_every_token_on_one_expert(T, d, L, I):
    """The expert stages hold more activations than the dense ones, and the way up's weights are on their
    way while the last expert still multiplies."""
    c = dict(MUSE, T=T, d=d, L=L, I=I, n=8, k=2)
    w, u, gen = ref.make_layer(c, 32)
    w["logit_bias"] = torch.zeros(8, device="cuda")
    w["logit_bias"][[2, 5]] = 100.0
    for _ in range(3):
        close(c, run_few(c, w, u)[0], ref.layer(c, w, u, u)[0])


def test_few_repeats_bit_for_bit_on_any_workspace():
    c = dict(MUSE, T=8)
    w, u, gen = ref.make_layer(c, 23)
    ad, which = ref.make_adapters(c, 3, 16, gen)
    out, idx, wt, lg, layer = run_few(c, w, u, ad=ad, which=which)
    for fill in (0xFF, 0x00, 0x7F):
        layer._few_workspace.fill_(fill)
        again = run_few(c, w, u, ad=ad, which=which, layer=layer)
        for a, b in zip((out, idx, wt, lg), again):
            assert torch.equal(a, b)


def test_few_token_does_not_depend_on_its_neighbours():
    c = dict(MUSE, T=8)
    w, u, gen = ref.make_layer(c, 24)
    out = run_few(c, w, u)[0]
    for t in (0, 3, 7):
        one = run_few(dict(c, T=1), w, u[t:t + 1].contiguous())[0]
        assert torch.equal(one[0], out[t])


def test_few_without_adapters_is_the_same_layer():
    c = dict(MUSE, T=6)
    w, u, gen = ref.make_layer(c, 25)
    ad, _ = ref.make_adapters(c, 3, 16, gen)
    none = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(run_few(c, w, u)[0], run_few(c, w, u, ad=ad, which=none)[0])


def test_few_agrees_with_the_batch_path():
    """moe_layer_forward rounds every intermediate to bf16: its own bar against the definition is 2e-2
    of a row's largest value."""
    c = dict(MUSE, T=8, n=32, k=8)
    w, u, gen = ref.make_layer(c, 26)
    layer = moe.MoELayer(ref.config(c), w)
    a, b = layer.forward(u).double(), layer.forward_few(u).double()
    assert ((a - b).abs().amax(-1) <= 2e-2 * a.abs().amax(-1)).all()


def test_few_nan_stays_with_its_token():
    c = dict(MUSE, T=5)
    w, u, gen = ref.make_layer(c, 27)
    out = run_few(c, w, u)[0]
    assert moe.moe_get_device_status() == 0
    bad = u.clone()
    bad[2, 7] = float("nan")
    got = run_few(c, w, bad, r=u)[0]
    assert moe.moe_get_device_status() == moe.STATUS_CODES["MOE_ERR_DEVICE_CHECK"]
    keep = [0, 1, 3, 4]
    assert torch.equal(got[keep], out[keep])
    assert got[2].isnan().all()


def test_few_unused_weights_may_hold_anything():
    """Experts and adapters that no token selects are not read into any result."""
    c = dict(MUSE, T=2, n=64, k=2)
    w, u, gen = ref.make_layer(c, 28)
    ad, _ = ref.make_adapters(c, 4, 8, gen)
    which = torch.tensor([2, -1], dtype=torch.int32, device="cuda")
    out, idx, *_ = run_few(c, w, u, ad=ad, which=which)
    unused = [e for e in range(64) if e not in set(idx.flatten().tolist())]
    w["w_gu"][unused] = float("nan")
    w["w_down"][unused] = float("inf")
    for name in ("down_a", "down_b", "up_a", "up_b", "scale"):
        ad[name][[0, 1, 3]] = float("nan")
    assert torch.equal(run_few(c, w, u, ad=ad, which=which)[0], out)
    # another token's adapter: its non-finite values stay with its own token
    ad["up_b"][2] = float("nan")
    got = run_few(c, w, u, ad=ad, which=which)[0]
    assert torch.equal(got[1], out[1]) and got[0].isnan().all()


def test_few_bad_adapter_index_is_latched_and_left_out():
    c = dict(MUSE, T=4)
    w, u, gen = ref.make_layer(c, 29)
    ad, _ = ref.make_adapters(c, 3, 16, gen)
    good = torch.tensor([1, -1, -1, 2], dtype=torch.int32, device="cuda")
    bad = torch.tensor([1, 3, -2, 2], dtype=torch.int32, device="cuda")
    out = run_few(c, w, u, ad=ad, which=good)[0]
    assert moe.moe_get_device_status() == 0
    got = run_few(c, w, u, ad=ad, which=bad)[0]
    assert moe.moe_get_device_status() == moe.STATUS_CODES["MOE_ERR_DEVICE_CHECK"]
    assert torch.equal(got, out)


def test_few_in_a_graph_and_on_two_streams():
    c = dict(MUSE, T=4, d=512, L=256, I=256, n=32, k=8)
    w, u, gen = ref.make_layer(c, 30)
    layers = [moe.MoELayer(ref.config(c), w) for _ in range(2)]
    want = layers[0].forward_few(u)
    layers[1].forward_few(u)
    torch.cuda.synchronize()
    static, out = u.clone(), torch.empty_like(u)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers[0].forward_few(static, out=out)
    for k in range(3):  # replays see new inputs
        x = u.roll(k, 0).contiguous()
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want.roll(k, 0))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):  # two calls at a time, each with its own workspace
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(layers[i].forward_few(u))
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o, want)
    assert moe.moe_get_device_status() == 0


def test_few_writes_its_outputs_only():
    c = dict(MUSE, T=3)
    w, u, gen = ref.make_layer(c, 31)
    buf = torch.full((8, c["d"]), 5.0, dtype=torch.bfloat16, device="cuda")
    layer = moe.MoELayer(ref.config(c), w)
    need = moe.few_workspace_size(layer.cfg)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_layer_forward_few(layer.cfg, layer._w, u, u, buf[2:5], workspace=ws, workspace_bytes=need)
    torch.cuda.synchronize()
    assert (buf[:2] == 5).all() and (buf[5:] == 5).all() and (ws[need:] == 0xA5).all()
    close(c, buf[2:5], ref.layer(c, w, u, u)[0])
