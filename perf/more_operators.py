"""What the gated feed-forward block on rows grouped by expert, and the activations that it keeps in
8 bits, are measured on.

  gated   both projections, the activation and the product of each expert's rows in one kernel
          (``ep_expert_gated``): h = act(Wg x) * (Wu x)
  step    the block's forward pass with what its backward pass needs kept (in e4m3 or bf16), then
          the gradient through the down projection and the activation (``ep_expert_gated`` with a
          checkpoint, ``ep_expert_gated_dgrad``)
  keep    rows kept in 8 bits and brought back (``ep_checkpoint_rows``, ``ep_restore_rows``)
  wgrad   the matrices' gradient from rows kept in 8 bits (``ep_expert_gemm_wgrad_checkpoint``)
  block   a training pass of the whole block by autograd (``experts.expert_feed_forward``)

A checkpoint in e4m3 has one power of two for each 16 features of a row, the least 2^k with
amax <= 448 * 2^k (2^-126 for a group of zeros), and the values (rounded to bf16 before) over it.

``run`` computes them in plain torch operations in 32 bits, or (``own``) by the calls above.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 16      # features of a row per power of two


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request decodes one token through a dense block: the weights' stream and latency
        dict(name="gated_one", op="gated", rows=1, K=4096, F=4096, E=1, skew=0.0, act="silu"),
        # a decode step's rows over 32 experts: the weights are what is read
        dict(name="gated_decode", op="gated", rows=251, K=7168, F=2048, E=32, skew=0.5, act="silu"),
        # a small model's prompt, features that are odd multiples of 8, short contraction
        dict(name="gated_odd", op="gated", rows=4229, K=560, F=2616, E=8, skew=0.5, act="gelu"),
        # a prefill over uneven experts
        dict(name="gated_prefill", op="gated", rows=32771, K=7168, F=2048, E=32, skew=0.5, act="silu"),
        # a small model's training step, 8-bit checkpoints, some experts without rows
        dict(name="step_small", op="step", rows=509, K=256, F=512, E=8, skew=0.5, act="gelu", keep="e4m3"),
        # a training step that keeps bf16
        dict(name="step_bf16", op="step", rows=8191, K=2048, F=1368, E=16, skew=0.3, act="silu", keep="bf16"),
        # a training step of large experts that keeps 8 bits
        dict(name="step_train", op="step", rows=16384, K=7168, F=2048, E=32, skew=0.3, act="silu", keep="e4m3"),
        # rows kept for the backward pass and brought back: a few, and a training step's
        dict(name="keep_few", op="keep", rows=128, K=7168),
        dict(name="keep_rows", op="keep", rows=16381, K=7168),
        # gradients of the gate and up matrices from kept rows: small experts, and a training step's
        dict(name="wgrad_small", op="wgrad", rows=509, K=256, F=1024, E=8, skew=0.5),
        dict(name="wgrad_train", op="wgrad", rows=16384, K=7168, F=4096, E=32, skew=0.3),
        # the whole block, forward and every gradient, keeping 8 bits
        dict(name="block_train", op="block", rows=8192, K=4096, F=2048, E=16, skew=0.3, act="silu"),
    ]


def _between(rng, lo, hi):
    """A whole number, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(["gated", "gated", "step", "step", "keep", "wgrad", "block"])
    if op == "keep":
        return dict(op=op, rows=_between(rng, 1, 33000), K=8 * _between(rng, 8, 1024))
    c = dict(op=op, rows=_between(rng, 1, 33000), K=8 * _between(rng, 32, 900), F=8 * _between(rng, 32, 520),
             E=rng.choice([1, 2, 4, 8, 16, 32, 64]), skew=rng.choice([0.0, 0.3, 0.5]))
    if op != "wgrad":
        c["act"] = rng.choice(["silu", "gelu"])
    if op == "step":
        c["keep"] = rng.choice(["e4m3", "e4m3", "bf16"])
    return c


def draw(rng):
    most = [work(c) for c in listed()]
    bytes_, flops = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    c = _draw(rng)
    while work(c)["bytes"] > bytes_ or work(c)["flops"] > flops:
        c = _draw(rng)
    return c


def _kept(features, keep="e4m3"):
    """Bytes of a row's checkpoint."""
    return 2 * features if keep == "bf16" else -(-features // GROUP) * (GROUP + 1)


def work(case):
    c = case
    rows, K = c["rows"], c["K"]
    if c["op"] == "keep":
        return {"bytes": rows * (2 * K + 2 * _kept(K) + 2 * K), "flops": 0}
    F, used = c["F"], min(c["E"], c["rows"])
    if c["op"] == "gated":
        return {"bytes": 2 * (rows * (K + F) + used * 2 * K * F), "flops": 4 * rows * K * F}
    if c["op"] == "step":
        # x, both matrices, h and the checkpoint; then dy, the down matrix, the checkpoint, dg, du and h again
        kept = 2 * rows * _kept(F, c["keep"])
        return {"bytes": 2 * (rows * (K + F) + used * 2 * K * F) + 2 * kept + 2 * (rows * K + used * K * F + 3 * rows * F),
                "flops": 6 * rows * K * F}
    if c["op"] == "wgrad":
        return {"bytes": rows * (_kept(K) + 2 * F) + 2 * c["E"] * K * F, "flops": 2 * rows * K * F}
    # x, dy, y, dx, the matrices and their gradients, the checkpoints written and read
    return {"bytes": 2 * (4 * rows * K + 3 * (used + c["E"]) * K * F) + 2 * rows * (_kept(K) + 2 * _kept(F)),
            "flops": 18 * rows * K * F}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16) * scale


def _rows(g, rows, K):
    """Activations as they leave a layer: some channels and some rows are much larger than the others."""
    wide = torch.exp(torch.randn(K, generator=g, device=DEV) * 0.7)
    tall = torch.exp(torch.randn(rows, 1, generator=g, device=DEV) * 0.5)
    return (torch.randn(rows, K, generator=g, device=DEV) * wide * tall * 0.7).to(torch.bfloat16)


def _inputs(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    rows, K = c["rows"], c["K"]
    s = {"case": c}
    if c["op"] == "keep":
        s["x"] = _rows(g, rows, K)
        return s
    F, E = c["F"], c["E"]
    p = torch.arange(1, E + 1, device=DEV, dtype=torch.float32).pow(-c["skew"])
    p = p[torch.randperm(E, generator=g, device=DEV)]
    if E >= 8:
        p[torch.randint(0, E, (1,), generator=g, device=DEV)] = 0.0     # an expert nobody chose
    n = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=E)
    s["prefix"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    s["prefix"][1:] = n.cumsum(0)
    s["most"] = int(n.max())
    if c["op"] == "wgrad":
        s["dy"] = _normal(g, rows, F)
        s["x"] = _rows(g, rows, K)
        return s
    s["x"] = _normal(g, rows, K)
    s["gate_up"] = _normal(g, E, 2 * F, K, scale=1.5 * K ** -0.5)
    if c["op"] in ("step", "block"):
        s["dy"] = _normal(g, rows, K)
        s["down"] = _normal(g, E, K, F, scale=F ** -0.5)
    return s


def prepare(case, seed):
    """The inputs, and the output buffers, workspace and launch that a caller of the library owns."""
    s = _inputs(case, seed)
    c = case
    rows, K = c["rows"], c["K"]
    like = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if c["op"] == "keep":
        s["q"], s["scales"] = like(rows, _padded(K), dtype=torch.uint8), like(rows, _padded(K) // GROUP, dtype=torch.uint8)
        s["back"] = like(rows, K)
    elif c["op"] == "wgrad":
        s["q"], s["scales"] = _quantised(s.pop("x"))
        s["dw"] = like(c["E"], c["F"], K)
    elif c["op"] == "block":
        for name in ("x", "gate_up", "down"):
            s[name].requires_grad_(True)
    else:
        F = c["F"]
        s["h"] = like(rows, F)
        if c["op"] == "step":
            wide = 2 * _padded(F)
            s["kept"] = like(rows, 2 * F) if c["keep"] == "bf16" else like(rows, wide, dtype=torch.uint8)
            s["scales"] = None if c["keep"] == "bf16" else like(rows, wide // GROUP, dtype=torch.uint8)
            s["dgu"], s["again"] = like(rows, 2 * F), like(rows, F)
    if own:
        import combine_layout_02_gb300 as ep
        from combine_layout_02_gb300 import experts
        s["ep"], s["experts"] = ep, experts
        s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["launch"] = ep.make_launch(error_flags=s["err"])
        if "act" in c:
            s["act"] = {"silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU_TANH}[c["act"]]
        if c["op"] in ("gated", "step"):
            s["shape"] = ep.ep_gemm_shape(rows, c["E"], K, c["F"])
            s["down_shape"] = ep.ep_gemm_shape(rows, c["E"], c["F"], K)
            if c["op"] == "step":
                s["checkpoint"] = ep.make_checkpoint(s["kept"], s["scales"])
        elif c["op"] == "keep":
            s["checkpoint"] = ep.make_checkpoint(s["q"], s["scales"])
        elif c["op"] == "wgrad":
            s["shape"] = ep.ep_gemm_shape(rows, c["E"], K, c["F"])
            s["checkpoint"] = ep.make_checkpoint(s["q"], s["scales"])
            s["workspace"] = like(max(16, ep.ep_wgrad_checkpoint_workspace_size(s["shape"])), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    return (_own if own else _plain)(s["case"]["op"], s)


def _own(op, s):
    ep = s["ep"]
    if op == "gated":
        ep.ep_expert_gated(s["shape"], s["x"], s["gate_up"], s["prefix"], s["act"], s["h"], None, s["launch"])
        return {"h": s["h"]}
    if op == "step":
        ep.ep_expert_gated(s["shape"], s["x"], s["gate_up"], s["prefix"], s["act"], s["h"], s["checkpoint"], s["launch"])
        ep.ep_expert_gated_dgrad(s["down_shape"], s["dy"], s["down"], s["prefix"], s["act"], s["checkpoint"], s["dgu"], s["again"],
                                 s["launch"])
        return {"h": s["h"], "dgu": s["dgu"], "again": s["again"]}
    if op == "keep":
        rows, K = s["x"].shape
        ep.ep_checkpoint_rows(rows, K, s["x"], s["checkpoint"], s["launch"])
        ep.ep_restore_rows(rows, K, s["checkpoint"], s["back"], s["launch"])
        return {"x": s["back"]}
    if op == "wgrad":
        ep.ep_expert_gemm_wgrad_checkpoint(s["shape"], s["dy"], s["checkpoint"], s["prefix"], s["dw"], s["workspace"], s["launch"])
        return {"dw": s["dw"]}
    y = s["experts"].expert_feed_forward(s["x"], s["gate_up"], s["down"], s["prefix"], activation=s["case"]["act"], checkpoint="e4m3",
                                         err=s["err"])
    dx, dgate_up, ddown = torch.autograd.grad(y, (s["x"], s["gate_up"], s["down"]), s["dy"])
    return {"y": y.detach(), "dx": dx, "dgate_up": dgate_up, "ddown": ddown}


def _padded(features):
    return -(-features // GROUP) * GROUP


def _quantised(x):
    """x [rows][features] -> (e4m3 bytes [rows][padded], exponents + 127 [rows][padded / 16])."""
    rows, features = x.shape
    at = torch.zeros(rows, _padded(features), device=x.device)
    at[:, :features] = x.to(torch.bfloat16)
    at = at.view(rows, -1, GROUP)
    bits = at.abs().amax(2).view(torch.int32)
    k = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=1)         # 448 = 1.75 * 2^8
    q = (at * ((254 - k) << 23).view(torch.float32).unsqueeze(2)).to(torch.float8_e4m3fn)
    return q.view(rows, -1).view(torch.uint8), k.to(torch.uint8)


def _values(q, scales, features):
    """What a checkpoint stands for, in 32 bits."""
    v = q.view(torch.float8_e4m3fn).float().view(q.shape[0], -1, GROUP)
    return (v * (scales.int() << 23).view(torch.float32).unsqueeze(2)).flatten(1)[:, :features]


def _as_kept(x, keep):
    x = x.to(torch.bfloat16)
    return x.float() if keep == "bf16" else _values(*_quantised(x), x.shape[1])


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = 2.0 * math.sqrt(2.0 / math.pi)
    s = 1.0 / (1.0 + torch.exp(-c * (g + 0.044715 * g * g * g)))
    return g * s, s + g * s * (1.0 - s) * c * (1.0 + 3 * 0.044715 * g * g)


def _places(prefix, rows, most):
    """The row at each place of [E][most] (and whether there is one), and each row's place."""
    E = len(prefix) - 1
    start = prefix[:-1].long()
    at = start[:, None] + torch.arange(most, device=prefix.device)
    there = at < prefix[1:].long()[:, None]
    row = torch.arange(rows, device=prefix.device)
    e = torch.searchsorted(prefix[1:].long().contiguous(), row, right=True).clamp(max=E - 1)
    return at.clamp(max=rows - 1), there.unsqueeze(-1), e * most + row - start[e]


def _by_expert(x, places):
    """Rows of each expert side by side, zero where it has fewer: [E][most][...] in 32 bits."""
    at, there, _ = places
    return torch.where(there, x.float()[at], torch.zeros((), device=x.device))


def _product(x, weight, places):
    """Each row times its expert's matrix [E][in][out], in 32 bits."""
    return torch.matmul(_by_expert(x, places), weight.float()).flatten(0, 1)[places[2]]


def _plain(op, s):
    c, bf = s["case"], torch.bfloat16
    if op == "keep":
        return {"x": _values(*_quantised(s["x"]), c["K"]).to(bf)}
    places = _places(s["prefix"], c["rows"], s["most"])
    if op == "wgrad":
        x = _values(s["q"], s["scales"], c["K"])
        return {"dw": torch.matmul(_by_expert(s["dy"], places).transpose(1, 2), _by_expert(x, places)).to(bf)}
    x, gate_up = s["x"].detach(), s["gate_up"].detach()
    g, u = _product(x, gate_up.transpose(1, 2), places).chunk(2, dim=1)
    h = _act(g, c["act"])[0] * u
    if op == "gated":
        return {"h": h.to(bf)}
    keep = c.get("keep", "e4m3")
    down = s["down"].detach()
    dh = _product(s["dy"], down, places)
    g, u = _as_kept(g, keep), _as_kept(u, keep)
    a, da = _act(g, c["act"])
    dgu, again = torch.cat([dh * u * da, dh * a], dim=1), a * u
    if op == "step":
        return {"h": h.to(bf), "dgu": dgu.to(bf), "again": again.to(bf)}
    return {"y": _product(h, down.transpose(1, 2), places).to(bf), "dx": _product(dgu, gate_up, places).to(bf),
            "dgate_up": torch.matmul(_by_expert(dgu, places).transpose(1, 2), _by_expert(_as_kept(x, keep), places)).to(bf),
            "ddown": torch.matmul(_by_expert(s["dy"], places).transpose(1, 2), _by_expert(again, places)).to(bf)}


# ------------------------------------------------------------------ in 64 bits

def _two_to(k):
    """2^k exactly (a power taken on the device may be off in the last place)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _kept_exactly(x):
    """x as its checkpoint has it, in 64 bits: the group's power of two by its logarithm, the nearest
    of the type's values (three bits after the first, none below 2^-9) by division and rounding."""
    x = x.to(torch.bfloat16).double()
    rows, features = x.shape
    at = torch.nn.functional.pad(x, (0, _padded(features) - features)).view(rows, _padded(features) // GROUP, GROUP)
    most = at.abs().amax(2, keepdim=True)
    m, e = torch.frexp(most / 448.0)
    k = torch.where(most > 0, torch.where(m > 0.5, e, e - 1), torch.full_like(e, -126)).clamp(min=-126)
    at = at * _two_to(-k)
    step = _two_to((torch.frexp(at)[1] - 1).clamp(min=-6) - 3)
    return (torch.round(at / step) * step * _two_to(k)).flatten(1)[:, :features]


def _derivative(g, act):
    """act and its derivative, in 64 bits, by hyperbolic tangents."""
    if act == "silu":
        s = 0.5 * (1 + torch.tanh(0.5 * g))
        return g * s, s + g * 0.25 * (1 - torch.tanh(0.5 * g) ** 2)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def exact(case, seed):
    """The same outputs from the definitions, expert by expert, in 64 bits."""
    c, s = case, _inputs(case, seed)
    f64 = torch.float64
    if c["op"] == "keep":
        return {"x": _kept_exactly(s["x"])}
    rows, K, F, E, edge = c["rows"], c["K"], c["F"], c["E"], s["prefix"].tolist()
    new = lambda *shape: torch.zeros(*shape, dtype=f64, device=DEV)  # noqa: E731
    if c["op"] == "wgrad":
        dw, x = new(E, F, K), _kept_exactly(s["x"])
        for e in range(E):
            dw[e] = s["dy"][edge[e]:edge[e + 1]].to(f64).t() @ x[edge[e]:edge[e + 1]]
        return {"dw": dw}
    h, dgu, again = new(rows, F), new(rows, 2 * F), new(rows, F)
    if c["op"] == "block":
        y, dx, dgate_up, ddown = new(rows, K), new(rows, K), new(E, 2 * F, K), new(E, K, F)
    for e in range(E):
        at = slice(edge[e], edge[e + 1])
        x, w = s["x"][at].to(f64), s["gate_up"][e].to(f64)
        g, u = x @ w[:F].t(), x @ w[F:].t()
        h[at] = _derivative(g, c["act"])[0] * u
        if c["op"] == "gated":
            continue
        if c.get("keep") == "bf16":
            g, u = g.to(torch.bfloat16).to(f64), u.to(torch.bfloat16).to(f64)
        else:
            g, u = _kept_exactly(g), _kept_exactly(u)
        a, da = _derivative(g, c["act"])
        down, dy = s["down"][e].to(f64), s["dy"][at].to(f64)
        dh = dy @ down
        dgu[at, :F], dgu[at, F:], again[at] = dh * u * da, dh * a, a * u
        if c["op"] == "block":
            y[at], dx[at] = h[at] @ down.t(), dgu[at] @ w
            dgate_up[e], ddown[e] = dgu[at].t() @ _kept_exactly(s["x"][at]), dy.t() @ again[at]
    if c["op"] == "gated":
        return {"h": h}
    if c["op"] == "step":
        return {"h": h, "dgu": dgu, "again": again}
    return {"y": y, "dx": dx, "dgate_up": dgate_up, "ddown": ddown}
