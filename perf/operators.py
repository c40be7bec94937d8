"""Measured cases of the recurrent block's operators around the delta rule.

Four families, each as a user's program calls it:

- ``scan``: the per-channel gated linear recurrence h_t = a_t h_{t-1} + w_t x_t, its forward over
  whole sequences (``fwd``), its backward (``bwd``) and one serving token (``step``);
- ``norm``: layer norm's forward and backward with the reduction of the weight's and the bias's
  gradients;
- ``beam``: the best continuations of every group of beams over the vocabulary;
- ``reorder``: the recurrent states follow the beams that were chosen, in place.

With ``own`` false ``run`` computes the operators from elementary torch operations; with it true
it calls this package.
"""
import math

import torch

own = False

CKPT = 64                       # tokens between two saved states of the scan
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST = 4 * 4096 * 2048          # elements of the largest case


def listed():
    return [
        # training: one mixer layer at the bench workload's tokens, 16 heads x 128 channels
        dict(name="scan_fwd_b4_t4096_d2048", op="scan", way="fwd", B=4, T=4096, D=2048, x="bf16", g="f32",
             gate="raw", tied=False, ragged=False),
        # prompt of one long document, few heads (4 x 128), bf16 gates straight from a projection
        dict(name="scan_fwd_b1_t32768_d512", op="scan", way="fwd", B=1, T=32768, D=512, x="bf16", g="bf16",
             gate="slow", tied=True, ragged=False),
        # a padded batch of short documents in 32 bits, an odd number of channels
        dict(name="scan_fwd_ragged_b3_t777_d333", op="scan", way="fwd", B=3, T=777, D=333, x="f32", g="f32",
             gate="log", tied=False, ragged=True),
        # the gradient of the first case
        dict(name="scan_bwd_b4_t4096_d2048", op="scan", way="bwd", B=4, T=4096, D=2048, x="bf16", g="f32",
             gate="raw", tied=False, ragged=False),
        # the gradient of a padded batch, moving-average form, channels that are no power of two
        dict(name="scan_bwd_ragged_b2_t5000_d1000", op="scan", way="bwd", B=2, T=5000, D=1000, x="bf16", g="bf16",
             gate="slow", tied=True, ragged=True),
        # one serving token of 256 sequences (the decode workload's) x 2048 channels
        dict(name="scan_step_n256_d2048", op="scan", way="step", B=256, T=1, D=2048, x="bf16", g="f32",
             gate="raw", tied=False, ragged=False),
        # the norm of every head's output: B4 T4096 H16 rows of 128
        dict(name="norm_fwd_262144x128", op="norm", way="fwd", N=262144, D=128, x="bf16", y="bf16", w="f32", bias=True),
        # the gradient of a block's input norm: B4 T4096 rows of 2048
        dict(name="norm_bwd_16384x2048", op="norm", way="bwd", N=16384, D=2048, x="bf16", y="bf16", w="f32", bias=True),
        # 32 requests of 8 beams (256 sequences), a vocabulary of 32000 in bf16, some beams finished
        dict(name="beam_g32_k8_v32000", op="beam", G=32, K=8, V=32000, M=8, x="bf16", finished=True, first=False),
        # one request of 4 beams, a large odd vocabulary in 32 bits, twice as many candidates as beams
        dict(name="beam_g1_k4_v100003", op="beam", G=1, K=4, V=100003, M=8, x="f32", finished=False, first=False),
        # the decode workload's states (256 sequences x 16 heads x 128 x 128) follow their beams
        dict(name="reorder_n256_16x128x128", op="reorder", L=1, G=32, K=8, E=16 * 128 * 128),
        # the scan's states of 24 layers, 8 requests of 4 beams x 2048 channels
        dict(name="reorder_l24_n32_d2048", op="reorder", L=24, G=8, K=4, E=2048),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "norm", "norm", "beam", "beam", "reorder"])
    if op == "scan":
        way = rng.choice(["fwd", "fwd", "bwd", "bwd", "step"])
        D = _spread(rng, 1, 4096)
        if way == "step":
            B, T = _spread(rng, 1, 512), 1
        else:
            B = _spread(rng, 1, 16)
            T = _spread(rng, 1, min(32768, MOST // (B * D)))
        return dict(op="scan", way=way, B=B, T=T, D=D, x=rng.choice(["bf16", "bf16", "f32"]),
                    g=rng.choice(["f32", "bf16"]), gate=rng.choice(["raw", "slow", "log"]),
                    tied=rng.random() < 0.5, ragged=way != "step" and rng.random() < 0.4)
    if op == "norm":
        D = _spread(rng, 8, 16384)
        x = rng.choice(["bf16", "bf16", "f32"])
        return dict(op="norm", way=rng.choice(["fwd", "bwd"]), N=_spread(rng, 1, min(262144, MOST // D)), D=D, x=x, y=x,
                    w=rng.choice(["f32", "bf16"]), bias=rng.random() < 0.7)
    if op == "beam":
        K = _spread(rng, 1, 16)
        V = _spread(rng, 64, 262144)
        G = _spread(rng, 1, max(1, min(64, MOST // 4 // (K * V))))
        return dict(op="beam", G=G, K=K, V=V, M=rng.choice([K, 2 * K]), x=rng.choice(["bf16", "f32"]),
                    finished=rng.random() < 0.5, first=rng.random() < 0.2)
    K = _spread(rng, 2, 16)
    G = _spread(rng, 1, 64)
    E = _spread(rng, 1, min(16 * 128 * 128, 2 * MOST // (G * K)))
    return dict(op="reorder", L=_spread(rng, 1, max(1, min(32, 2 * MOST // (G * K * E)))), G=G, K=K, E=E)


# ---------------------------------------------------------------- inputs ----


def _gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return gen


def prepare(case, seed):
    gen = _gen(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    s = dict(case)
    if case["op"] == "scan":
        B, T, D = case["B"], case["T"], case["D"]
        shape = (B, D) if case["way"] == "step" else (B, T, D)
        if case["gate"] == "log":       # log-decays themselves: memories of a few to some thousand tokens
            s["gates"] = normal(*shape, std=1.5, mean=-3.0).exp_().neg_().to(DT[case["g"]])
        elif case["gate"] == "slow":    # raw gates of slow decay
            s["gates"] = normal(*shape, mean=-2.0, dtype=DT[case["g"]])
        else:                           # raw gates
            s["gates"] = normal(*shape, dtype=DT[case["g"]])
        s["inputs"] = normal(*shape, dtype=DT[case["x"]])
        s["h"] = normal(B, D, std=0.5)
        s["lengths"] = None
        if case["ragged"]:              # a padded batch: one full row, the others of any length, an empty one among them
            n = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
            n[0] = T
            if B > 2:
                n[-1] = 0
            s["lengths"] = n
        if case["way"] == "bwd":
            s["dh"] = normal(*shape, dtype=DT[case["x"]])
            s["dh_T"] = normal(B, D, std=0.5)
            # the states that the forward of a training step has left behind
            s["ckpt"] = _scan_states(s)[1]
        return s
    if case["op"] == "norm":
        N, D = case["N"], case["D"]
        # rows with an offset and a spread of their own, as residual streams have
        s["inputs"] = (normal(N, D) * normal(N, 1, std=0.5).exp_() + normal(N, 1, std=0.5)).to(DT[case["x"]])
        s["weight"] = normal(D, std=0.2, mean=1.0, dtype=DT[case["w"]])
        s["bias_"] = normal(D, std=0.2, dtype=DT[case["w"]]) if case["bias"] else None
        s["eps"] = 1e-5
        if case["way"] == "bwd":
            s["dy"] = normal(N, D, dtype=DT[case["y"]])
            _, s["mean"], s["rstd"] = _norm(s)
        return s
    if case["op"] == "beam":
        G, K, V = case["G"], case["K"], case["V"]
        logits = normal(G, K, V, std=2.5)
        # some tokens are banned: half with -inf, half with the type's lowest value
        banned = torch.rand((G, K, V), generator=gen, device="cuda") < 0.01
        low = torch.rand((G, K, V), generator=gen, device="cuda") < 0.5
        dt = DT[case["x"]]
        logits = torch.where(banned, torch.where(low, torch.finfo(dt).min, -math.inf), logits)
        s["logits"] = logits.to(dt)
        s["scores"] = normal(G, K, std=1.5, mean=-20.0)
        if case["first"]:               # the first token: one live beam, the others empty
            s["scores"].fill_(-math.inf)
            s["scores"][:, 0] = 0.0
        s["finished_"] = None
        s["eos"] = min(2, V - 1)
        if case["finished"]:
            s["finished_"] = torch.rand((G, K), generator=gen, device="cuda") < 0.2
        return s
    L, G, K, E = case["L"], case["G"], case["K"], case["E"]
    s["states"] = normal(L, G * K, E)
    s["parent"] = torch.randint(0, K, (G, K), generator=gen, device="cuda", dtype=torch.int32)
    return s


# ----------------------------------------------------------- plain forms ----


def _gates(s):
    """The decay a and 1 - a of every token, in 32 bits."""
    a = s["gates"].float()
    if s["gate"] == "log":
        return a.exp(), -torch.expm1(a)
    return 1.0 / (1.0 + a.exp()), 1.0 / (1.0 + (-a).exp())


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t from the zero state, by doubling the reach."""
    a, d, T = a, 1, a.shape[1]
    while d < T:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1) if 2 * d < T else a
        d *= 2
    return b


def _inside(s):
    """Which tokens lie inside their sequence, or None where all do."""
    if s["lengths"] is None:
        return None
    return (torch.arange(s["T"], device="cuda")[None] < s["lengths"][:, None])[..., None]


def _scan_terms(s):
    a, rest = _gates(s)
    b = s["inputs"].float()
    if s["tied"]:
        b = rest * b
    inside = _inside(s)
    if inside is not None:
        a, b = torch.where(inside, a, 1.0), torch.where(inside, b, 0.0)
    return a, b


def _scan_states(s):
    """The state after every token, and the one before every CKPT-th token, in 32 bits."""
    a, b = _scan_terms(s)
    b[:, 0] += a[:, 0] * s["h"]
    h = _scan(a, b)
    ckpt = torch.cat([s["h"][:, None], h[:, CKPT - 1:s["T"] - 1:CKPT]], 1)
    return h, ckpt


def _scan_fwd(s):
    h, ckpt = _scan_states(s)
    last = h[:, -1].clone()
    inside = _inside(s)
    if inside is not None:
        h = torch.where(inside, h, 0.0)
    return h.to(s["inputs"].dtype), last, ckpt


def _scan_bwd(s):
    a, rest = _gates(s)
    x, dh = s["inputs"].float(), s["dh"].float()
    inside = _inside(s)
    h, _ = _scan_states(s)
    before = torch.cat([s["h"][:, None], h[:, :-1]], 1)
    if inside is not None:
        dh, am = torch.where(inside, dh, 0.0), torch.where(inside, a, 1.0)
    else:
        am = a
    # the state's whole gradient, from the last token back: lam_t = dh_t + a_{t+1} lam_{t+1}
    dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dh_T"][:, None]], 1)
    up = torch.cat([am[:, 1:], torch.ones_like(am[:, :1])], 1).flip(1)
    lam = _scan(up, dh.flip(1)).flip(1)
    dx = lam * rest if s["tied"] else lam
    da = lam * (before - x if s["tied"] else before)
    dg = da * a if s["gate"] == "log" else -da * (a * rest)
    if inside is not None:
        dx, dg = torch.where(inside, dx, 0.0), torch.where(inside, dg, 0.0)
    return dx.to(s["inputs"].dtype), dg.to(s["gates"].dtype), am[:, 0] * lam[:, 0]


def _scan_step(s):
    a, rest = _gates(s)
    x = s["inputs"].float()
    s["h"].copy_(a * s["h"] + (rest * x if s["tied"] else x))
    return s["h"].to(s["inputs"].dtype), s["h"]


def _norm(s):
    x = s["inputs"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + s["eps"])
    y = x * rstd * s["weight"].float()
    if s["bias_"] is not None:
        y = y + s["bias_"].float()
    return y.to(DT[s["y"]]), mean[:, 0], rstd[:, 0]


def _norm_bwd(s):
    x, dy = s["inputs"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    wdy = dy * s["weight"].float()
    dx = rstd * (wdy - wdy.mean(1, keepdim=True) - xh * (wdy * xh).mean(1, keepdim=True))
    dw = (dy * xh).sum(0)
    db = dy.sum(0) if s["bias_"] is not None else None
    return dx.to(s["inputs"].dtype), dw, db


def _beam(s):
    # scores next to one another decide whole numbers: in 64 bits
    G, K, V = s["logits"].shape
    x = s["logits"].double()
    top = x.amax(2, keepdim=True)
    lse = (x - top).exp().sum(2, keepdim=True).log() + top
    c = s["scores"].double()[..., None] + (x - lse)
    c = torch.where(torch.isnan(c), -math.inf, c)
    if s["finished_"] is not None:
        at_eos = torch.arange(V, device="cuda") == s["eos"]
        ended = torch.where(at_eos, s["scores"].double()[..., None], -math.inf)
        c = torch.where(s["finished_"][..., None], ended, c)
    best, at = torch.sort(c.view(G, K * V), dim=1, descending=True, stable=True)
    best, at = best[:, :s["M"]], at[:, :s["M"]]
    return best.float(), (at // V).int(), (at % V).int()


def _reorder(s):
    L, G, K, E = (s[k] for k in "LGKE")
    at = (torch.arange(G, device="cuda")[:, None] * K + s["parent"]).view(-1)
    s["states"].copy_(s["states"][:, at])
    return s["states"]


# ------------------------------------------------------------------ run ----


def _run_own(s):
    from recurrent_state_memory_b200 import gdr
    if s["op"] == "scan":
        mode = gdr.GATE_LOGDECAY if s["gate"] == "log" else gdr.GATE_NEG_SOFTPLUS
        if s["way"] == "step":
            o = gdr.scan_step(s["inputs"], s["gates"], s["h"], gate_mode=mode, tied=s["tied"])
            return o, s["h"]
        if s["way"] == "fwd":
            return gdr.scan_fwd(s["inputs"], s["gates"], s["h"], gate_mode=mode, tied=s["tied"], lengths=s["lengths"],
                                want_ckpt=True)
        d = gdr.scan_bwd(s["inputs"], s["gates"], s["ckpt"], s["dh"], s["dh_T"], gate_mode=mode, tied=s["tied"],
                         lengths=s["lengths"])
        return d["x"], d["g"], d["h0"]
    if s["op"] == "norm":
        if s["way"] == "fwd":
            return gdr.layernorm_fwd(s["inputs"], s["weight"], s["bias_"], eps=s["eps"], out_dtype=DT[s["y"]])
        d = gdr.layernorm_bwd(s["inputs"], s["dy"], s["mean"], s["rstd"], s["weight"], with_bias=s["bias_"] is not None)
        return d["x"], d["weight"], d["bias"]
    if s["op"] == "beam":
        return gdr.beam_select(s["logits"], s["scores"], s["M"], finished=s["finished_"], eos=s["eos"])
    return gdr.state_reorder(s["states"], s["parent"], layers=True)


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "scan":
        return {"fwd": _scan_fwd, "bwd": _scan_bwd, "step": _scan_step}[state["way"]](state)
    if state["op"] == "norm":
        return _norm(state) if state["way"] == "fwd" else _norm_bwd(state)
    return _beam(state) if state["op"] == "beam" else _reorder(state)


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "scan":
        n, rows = case["B"] * case["T"] * case["D"], case["B"] * case["D"]
        x, g = size[case["x"]], size[case["g"]]
        if case["way"] == "step":
            return {"bytes": n * (2 * x + g + 8), "flops": 6 * n}
        saved = 4 * rows * -(-case["T"] // CKPT)
        if case["way"] == "fwd":
            return {"bytes": n * (2 * x + g) + saved + 8 * rows, "flops": 6 * n}
        return {"bytes": n * (3 * x + 2 * g) + saved + 8 * rows, "flops": 14 * n}
    if case["op"] == "norm":
        N, D, x, y, w = case["N"], case["D"], size[case["x"]], size[case["y"]], size[case["w"]]
        if case["way"] == "fwd":
            return {"bytes": N * D * (x + y) + 8 * N + (2 if case["bias"] else 1) * D * w, "flops": 8 * N * D}
        return {"bytes": N * D * (2 * x + y) + 8 * N + D * (w + (8 if case["bias"] else 4)), "flops": 14 * N * D}
    if case["op"] == "beam":
        n = case["G"] * case["K"] * case["V"]
        return {"bytes": n * size[case["x"]] + 4 * case["G"] * (case["K"] + 3 * case["M"]), "flops": 4 * n}
    # in place: what is written are the beams with another parent, what is read the states that
    # some other beam takes over (both as expected of parents drawn evenly)
    L, G, K, E = (case[k] for k in "LGKE")
    moved = G * (K - 1)
    read = G * K * (1.0 - (1.0 - 1.0 / K) ** (K - 1))
    return {"bytes": L * 4 * E * (moved + read) + 4 * G * K, "flops": 0}


# ---------------------------------------------------------------- exact ----


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "scan":
        return _exact_scan(case, s)
    if case["op"] == "norm":
        x, w = s["inputs"].double(), s["weight"].double()
        D = case["D"]
        if case["way"] == "fwd":
            mu = x.sum(1) / D
            var = (x - mu[:, None]).square().sum(1) / D
            y = (x - mu[:, None]) / (var + s["eps"]).sqrt()[:, None] * w
            return (y if s["bias_"] is None else y + s["bias_"].double()), mu, (var + s["eps"]).rsqrt()
        mu, r, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
        hat = (x - mu[:, None]) * r[:, None]
        c1, c2 = (dy @ w) / D, ((dy * hat) @ w) / D
        dx = r[:, None] * (dy * w - c1[:, None] - hat * c2[:, None])
        return dx, torch.einsum("nd,nd->d", dy, hat), None if s["bias_"] is None else torch.einsum("nd->d", dy)
    if case["op"] == "beam":
        x = s["logits"].double()
        c = torch.log_softmax(x, 2) + s["scores"].double()[..., None]
        c = torch.nan_to_num(c, nan=-math.inf, neginf=-math.inf)
        if s["finished_"] is not None:
            c[s["finished_"]] = -math.inf
            c[..., s["eos"]] = torch.where(s["finished_"], s["scores"].double(), c[..., s["eos"]])
        return torch.topk(c.view(case["G"], -1), case["M"]).values, None, None
    L, G, K, E = (case[k] for k in "LGKE")
    view = s["states"].view(L, G, K, E)
    return torch.take_along_dim(view, s["parent"].long()[None, :, :, None], 2).double().reshape(L, G * K, E)


def _exact_scan(case, s):
    """Token by token."""
    step = case["way"] == "step"
    B, T, D = case["B"], case["T"], case["D"]
    g, x = s["gates"].double().view(B, T, D), s["inputs"].double().view(B, T, D)
    a = g.exp() if case["gate"] == "log" else torch.sigmoid(-g)
    rest = -torch.expm1(g) if case["gate"] == "log" else torch.sigmoid(g)
    w = rest if case["tied"] else torch.ones_like(rest)
    n = s["lengths"].long()[:, None] if s["lengths"] is not None else torch.full((B, 1), T, device="cuda")
    h = s["h"].double()
    out, ckpt = torch.zeros_like(x), []
    prev = torch.zeros_like(x)
    for t in range(T):
        if t % CKPT == 0:
            ckpt.append(h)
        prev[:, t] = h
        h = torch.where(t < n, a[:, t] * h + w[:, t] * x[:, t], h)
        out[:, t] = torch.where(t < n, h, 0.0)
    if step:
        return out[:, 0], h
    if case["way"] == "fwd":
        return out, h, torch.stack(ckpt, 1)
    lam, dx, dg = s["dh_T"].double(), torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T - 1, -1, -1):
        on = t < n
        here = lam + s["dh"][:, t].double()
        dx[:, t] = torch.where(on, w[:, t] * here, 0.0)
        slope = a[:, t] if case["gate"] == "log" else -a[:, t] * rest[:, t]
        dg[:, t] = torch.where(on, here * (prev[:, t] - (x[:, t] if case["tied"] else 0.0)) * slope, 0.0)
        lam = torch.where(on, here * a[:, t], lam)
    return dx, dg, lam
