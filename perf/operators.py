"""What the operators on rows grouped by their owner are measured on.

Three operators work on the rows that a dispatch has delivered (or on rows that wait for one):

  sort      received rows brought into expert order (``ep_sort_layout`` + ``ep_sort_rows``), back
            into token order with the routing weights applied (``ep_unsort_rows``), and the
            gradients of both directions (``ep_unsort_rows_backward``, ``ep_unsort_rows`` with
            no weights)
  expert    the product of each expert's rows with that expert's matrix (``ep_expert_gemm``) and
            its two gradients (``ep_expert_gemm_dgrad``, ``ep_expert_gemm_wgrad``)
  adapter   a projection that all rows share plus each row's own low-rank adapter
            (``ep_adapter_gemm``)

``run`` computes them in plain torch operations in 32 bits, or (``own``) by the calls above.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 128     # channels per scale of an e4m3 row


# ------------------------------------------------------------------ cases

def listed():
    return [
        # -- sort: rows a rank received, N of them, k entries each, E local experts
        # a decode step's received rows: launches and latency
        dict(name="sort_decode", op="sort", N=128, H=7168, E=32, k=8, share=0.125, skew=0.0, fp8=False),
        # a prefill's received rows in bf16 (R8 x T4096 tokens, top-8 of 256 experts, 32 on the rank)
        dict(name="sort_prefill", op="sort", N=21673, H=7168, E=32, k=8, share=0.125, skew=0.0, fp8=False),
        # the same after an e4m3 dispatch: quantised rows with their scales, an odd count
        dict(name="sort_fp8", op="sort", N=16381, H=7168, E=32, k=8, share=0.25, skew=0.0, fp8=True),
        # back with the weights, the prefill's experts' outputs
        dict(name="back_prefill", op="back", N=21673, H=7168, E=32, k=8, share=0.125, skew=0.0),
        # both gradients on skewed routing where every entry is local (top-6 of 128 experts)
        dict(name="grad_skewed", op="grad", N=16384, H=4096, E=128, k=6, share=1.0, skew=0.6),
        # -- expert: rows already in expert order, in_features K, out_features F
        # a decode step: few rows an expert, the weights are what is read
        dict(name="expert_decode", op="expert", rows=251, K=7168, F=2048, E=32, skew=0.5),
        # a prefill: uneven experts, the products are what counts
        dict(name="expert_prefill", op="expert", rows=32771, K=7168, F=4096, E=32, skew=0.5),
        # gradients of a small model's experts, some of them without rows
        dict(name="expert_grad_small", op="expert_grad", rows=509, K=256, F=512, E=8, skew=0.5),
        # gradients of a training step's experts
        dict(name="expert_grad_train", op="expert_grad", rows=16384, K=7168, F=2048, E=32, skew=0.3),
        # -- adapter: T rows, L adapters of rank r beside one K -> F projection
        # one request decodes one token
        dict(name="adapter_one", op="adapter", T=1, K=4096, F=4096, L=8, r=16, runs=False),
        # many requests decode together, each with its own adapter
        dict(name="adapter_decode", op="adapter", T=61, K=7168, F=7168, L=64, r=16, runs=False),
        # prompts of several requests, one after another
        dict(name="adapter_prefill", op="adapter", T=8191, K=7168, F=4096, L=16, r=64, runs=True),
    ]


def _between(rng, lo, hi):
    """A whole number, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(["sort", "back", "grad", "expert", "expert_grad", "adapter"])
    if op in ("sort", "back", "grad"):
        E = rng.choice([8, 16, 32, 64, 128, 256])
        c = dict(op=op, N=_between(rng, 1, 30000), H=128 * _between(rng, 2, 64), E=E,
                 k=rng.randint(1, min(8, E)), share=rng.choice([0.125, 0.25, 0.5, 1.0]),
                 skew=rng.choice([0.0, 0.3, 0.6]))
        if op == "sort":
            c["fp8"] = rng.random() < 0.4
        return c
    if op in ("expert", "expert_grad"):
        return dict(op=op, rows=_between(rng, 1, 33000), K=8 * _between(rng, 32, 900), F=8 * _between(rng, 32, 600),
                    E=rng.choice([1, 2, 4, 8, 16, 32, 64]), skew=rng.choice([0.0, 0.3, 0.5]))
    T = _between(rng, 1, 8192)
    return dict(op=op, T=T, K=8 * _between(rng, 32, 900), F=8 * _between(rng, 32, 900),
                L=_between(rng, 1, 64), r=rng.choice([8, 16, 24, 32, 64]), runs=rng.random() < 0.5)


def draw(rng):
    most = [work(c) for c in listed()]
    bytes_, flops = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    c = _draw(rng)
    while work(c)["bytes"] > bytes_ or work(c)["flops"] > flops:
        c = _draw(rng)
    return c


def _valid(c):
    """Expected entries that stay on the rank."""
    return c["N"] * (c["k"] * c["share"] + (1 - c["share"]) ** c["k"])


def work(case):
    c = case
    op = c["op"]
    if op == "sort":
        row = c["H"] + c["H"] // GROUP * 4 if c["fp8"] else 2 * c["H"]
        n = _valid(c)
        return {"bytes": c["N"] * (row + c["k"] * 12) + n * (row + 4), "flops": 0}
    if op == "back":
        n = _valid(c)
        return {"bytes": n * 2 * c["H"] + c["N"] * (2 * c["H"] + c["k"] * 8), "flops": 2 * n * c["H"]}
    if op == "grad":
        # dout, y, dy and the weights' gradients; then the sorted rows' gradients and dx
        n = _valid(c)
        return {"bytes": c["N"] * (2 * c["H"] + c["k"] * 12) + 2 * n * 2 * c["H"] + n * 2 * c["H"] + c["N"] * (2 * c["H"] + c["k"] * 4),
                "flops": 4 * n * c["H"]}
    if op == "expert":
        used = min(c["E"], c["rows"])
        return {"bytes": 2 * (c["rows"] * (c["K"] + c["F"]) + used * c["K"] * c["F"]), "flops": 2 * c["rows"] * c["K"] * c["F"]}
    if op == "expert_grad":
        used = min(c["E"], c["rows"])
        return {"bytes": 2 * (2 * c["rows"] * (c["K"] + c["F"]) + (used + c["E"]) * c["K"] * c["F"]), "flops": 4 * c["rows"] * c["K"] * c["F"]}
    used = min(c["L"], c["T"])
    return {"bytes": 2 * (c["T"] * (c["K"] + c["F"]) + c["K"] * c["F"] + used * c["r"] * (c["K"] + c["F"])) + 8 * c["T"],
            "flops": 2 * c["T"] * (c["K"] * c["F"] + c["r"] * (c["K"] + c["F"]))}


# ------------------------------------------------------------------ inputs

def _routing(c, g):
    """topk_idx [N][k] int64: distinct experts, of which those of this rank keep their local id and
    the others are -1; every row but about 1 % has at least one. How many entries are local goes by
    the case alone (a caller knows it from the counts it has read). Weights: softmax over the entries."""
    N, E, k = c["N"], c["E"], c["k"]
    fixed = torch.Generator(device=DEV).manual_seed(1)
    n = torch.rand(N, k, generator=fixed, device=DEV).lt(c["share"]).sum(1)
    n = torch.where((n == 0) & (torch.rand(N, generator=fixed, device=DEV) > 0.01), torch.ones_like(n), n)
    if N < 100:
        n = n.clamp(min=1)
    n = n[torch.randperm(N, generator=g, device=DEV)]
    p = torch.arange(1, E + 1, device=DEV, dtype=torch.float32).pow(-c["skew"])
    p = p[torch.randperm(E, generator=g, device=DEV)]
    score = p.log() - torch.log(-torch.log(torch.rand(N, E, generator=g, device=DEV).clamp(1e-9, 1 - 1e-6)))
    idx = score.topk(k, dim=1).indices
    place = torch.rand(N, k, generator=g, device=DEV).argsort(1)        # which of the k entries are local
    idx = torch.where(place < n[:, None], idx, torch.full_like(idx, -1))
    w = torch.softmax(torch.randn(N, k, generator=g, device=DEV), -1)
    return idx.contiguous(), w.contiguous()


def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16) * scale


def _inputs(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    if c["op"] in ("sort", "back", "grad"):
        idx, w = _routing(c, g)
        s = dict(idx=idx, w=w, rows=int((idx >= 0).sum()))
        if c["op"] == "sort":
            if c["fp8"]:
                s["x"] = (torch.randn(c["N"], c["H"], generator=g, device=DEV) * 100).to(torch.float8_e4m3fn)
                s["scales"] = torch.rand(c["N"], c["H"] // GROUP, generator=g, device=DEV) * 0.02 + 0.001
            else:
                s["x"] = _normal(g, c["N"], c["H"])
        elif c["op"] == "back":
            s["y"] = _normal(g, s["rows"], c["H"])
        else:
            s["y"] = _normal(g, s["rows"], c["H"])
            s["dout"] = _normal(g, c["N"], c["H"])
            s["dxs"] = _normal(g, s["rows"], c["H"])
        return s
    if c["op"] in ("expert", "expert_grad"):
        p = torch.arange(1, c["E"] + 1, device=DEV, dtype=torch.float32).pow(-c["skew"])
        p = p[torch.randperm(c["E"], generator=g, device=DEV)]
        if c["E"] >= 8:
            p[torch.randint(0, c["E"], (1,), generator=g, device=DEV)] = 0.0     # an expert nobody chose
        n = torch.bincount(torch.multinomial(p, c["rows"], replacement=True, generator=g), minlength=c["E"])
        prefix = torch.zeros(c["E"] + 1, dtype=torch.int32, device=DEV)
        prefix[1:] = n.cumsum(0)
        s = dict(prefix=prefix, most=int(n.max()), weight=_normal(g, c["E"], c["F"], c["K"], scale=c["K"] ** -0.5))
        s["x"] = _normal(g, c["rows"], c["K"])
        if c["op"] == "expert_grad":
            s["dy"] = _normal(g, c["rows"], c["F"])
        return s
    T, K, F, L, r = c["T"], c["K"], c["F"], c["L"], c["r"]
    ids = torch.randint(0, L, (T,), generator=g, device=DEV)
    if c["runs"]:
        ids = ids[torch.randint(0, T, (T,), generator=g, device=DEV).sort().values // max(1, T // (2 * L)) * max(1, T // (2 * L))]
    ids = torch.where(torch.rand(T, generator=g, device=DEV) < (0.0 if c["runs"] else 0.1), torch.full_like(ids, -1), ids)
    return dict(ids=ids, x=_normal(g, T, K), weight=_normal(g, F, K, scale=K ** -0.5), a=_normal(g, L, r, K, scale=K ** -0.5),
                b=_normal(g, L, F, r, scale=r ** -0.5), scales=torch.rand(L, generator=g, device=DEV) + 0.25)


def prepare(case, seed):
    """The inputs, and the output buffers, workspace and launch that a caller of the library owns."""
    s = _inputs(case, seed)
    c = s["case"] = case
    like = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if c["op"] in ("sort", "back", "grad"):
        # the placement: an output of `sort`, what a caller has in hand in the other two
        s["entry_rows"] = like(c["N"], c["k"], dtype=torch.int32)
        s["row_entries"] = like(s["rows"], dtype=torch.int32)
        s["prefix"] = like(c["E"] + 1, dtype=torch.int32)
        if c["op"] == "sort":
            s["xs"] = torch.empty(s["rows"], c["H"], dtype=s["x"].dtype, device=DEV)
            s["xs_scales"] = like(s["rows"], c["H"] // GROUP, dtype=torch.float32) if c["fp8"] else None
        else:
            s["entry_rows"], s["row_entries"], s["prefix"] = _plain_layout(s["idx"], c["E"], s["rows"])
            s["out"] = like(c["N"], c["H"])
        if c["op"] == "grad":
            s["dy"], s["dw"] = like(s["rows"], c["H"]), like(c["N"], c["k"], dtype=torch.float32)
    elif c["op"] == "expert":
        s["y"] = like(c["rows"], c["F"])
    elif c["op"] == "expert_grad":
        s["dx"], s["dw"] = like(c["rows"], c["K"]), like(c["E"], c["F"], c["K"])
    else:
        s["y"] = like(c["T"], c["F"])
    if own:
        import combine_layout_02_gb300 as ep
        from combine_layout_02_gb300.buffers import SortBuffers
        s["ep"] = ep
        s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["launch"] = ep.make_launch(error_flags=s["err"])
        if c["op"] in ("sort", "back", "grad"):
            s["shape"] = ep.make_shape(1, c["N"], c["H"], c["E"], c["k"])
            placed = SortBuffers(s["shape"], s["rows"], DEV)
            for name, t in (("entry_rows", placed.entry_rows), ("row_entries", placed.row_entries), ("prefix", placed.expert_prefix)):
                t.copy_(s[name])
                s[name] = t
            s["handle"], s["workspace"] = placed.handle(), placed.workspace
        elif c["op"] in ("expert", "expert_grad"):
            s["shape"] = ep.ep_gemm_shape(c["rows"], c["E"], c["K"], c["F"])
        else:
            s["shape"] = ep.ep_adapter_shape(c["T"], c["K"], c["F"], c["L"], c["r"])
            s["workspace"] = like(max(16, ep.ep_adapter_workspace_size(s["shape"])), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    return (_own if own else _plain)(s["case"]["op"], s)


def _own(op, s):
    ep = s["ep"]
    if op == "sort":
        ep.ep_sort_layout(s["shape"], s["idx"], s["handle"], s["workspace"], s["launch"])
        fp8 = s["case"]["fp8"]
        ep.ep_sort_rows(s["shape"], s["x"], ep.EP_FP8_E4M3 if fp8 else ep.EP_BF16, s.get("scales"), s["handle"],
                        s["xs"], s["xs_scales"], s["launch"])
        return {"entry_rows": s["entry_rows"], "row_entries": s["row_entries"], "prefix": s["prefix"], "xs": s["xs"], "scales": s["xs_scales"]}
    if op == "back":
        ep.ep_unsort_rows(s["shape"], s["y"], s["w"], s["handle"], s["out"], s["launch"])
        return {"out": s["out"]}
    if op == "grad":
        ep.ep_unsort_rows_backward(s["shape"], s["dout"], s["y"], s["w"], s["handle"], s["dy"], s["dw"], s["launch"])
        ep.ep_unsort_rows(s["shape"], s["dxs"], None, s["handle"], s["out"], s["launch"])
        return {"dy": s["dy"], "dw": s["dw"], "dx": s["out"]}
    if op == "expert":
        ep.ep_expert_gemm(s["shape"], s["x"], s["weight"], s["prefix"], s["y"], s["launch"])
        return {"y": s["y"]}
    if op == "expert_grad":
        ep.ep_expert_gemm_dgrad(s["shape"], s["dy"], s["weight"], s["prefix"], s["dx"], s["launch"])
        ep.ep_expert_gemm_wgrad(s["shape"], s["dy"], s["x"], s["prefix"], s["dw"], s["launch"])
        return {"dx": s["dx"], "dw": s["dw"]}
    ep.ep_adapter_gemm(s["shape"], s["x"], s["weight"], s["a"], s["b"], s["scales"], s["ids"], s["y"], s["workspace"], s["launch"])
    return {"y": s["y"]}


def _plain_layout(idx, E, rows):
    """(entry_rows [N][k], row_entries [rows], prefix [E + 1]): entries by expert, then in order."""
    flat = idx.reshape(-1)
    key = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    order = key.sort(stable=True).indices[:rows]
    entry_rows = torch.full_like(flat, -1, dtype=torch.int32)
    entry_rows[order] = torch.arange(rows, device=idx.device, dtype=torch.int32)
    n = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    prefix = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    prefix[1:] = n[:E].cumsum(0)
    return entry_rows.view(idx.shape), order.to(torch.int32), prefix


def _taken(y, entry_rows):
    """Each entry's row of y in 32 bits, zero where it has none: [N][k][H]."""
    at = entry_rows.long()
    got = y.float()[at.clamp(min=0)]
    return torch.where((at >= 0).unsqueeze(-1), got, torch.zeros((), device=y.device))


def _back(y, entry_rows, w):
    got = _taken(y, entry_rows) if len(y) else torch.zeros(*entry_rows.shape, y.shape[1], device=y.device)
    return (got if w is None else got * w.unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _by_expert(x, prefix, most):
    """Rows of each expert side by side, zero where it has fewer: [E][most][...] in 32 bits, and
    each row's place in the flat [E * most]."""
    E, rows = len(prefix) - 1, len(x)
    start = prefix[:-1].long()
    at = start[:, None] + torch.arange(most, device=x.device)
    there = at < prefix[1:].long()[:, None]
    side = torch.where(there.unsqueeze(-1), x.float()[at.clamp(max=rows - 1)], torch.zeros((), device=x.device))
    row = torch.arange(rows, device=x.device)
    e = torch.searchsorted(prefix[1:].long().contiguous(), row, right=True).clamp(max=E - 1)
    return side, e * most + row - start[e]


def _plain(op, s):
    c = s["case"]
    if op == "sort":
        entry_rows, row_entries, prefix = _plain_layout(s["idx"], c["E"], s["rows"])
        token = row_entries.long() // c["k"]
        if c["fp8"]:
            xs, scales = s["x"].view(torch.uint8)[token].view(torch.float8_e4m3fn), s["scales"][token]
        else:
            xs, scales = s["x"][token], None
        return {"entry_rows": entry_rows, "row_entries": row_entries, "prefix": prefix, "xs": xs, "scales": scales}
    if op == "back":
        return {"out": _back(s["y"], s["entry_rows"], s["w"])}
    if op == "grad":
        entry = s["row_entries"].long()
        dout = s["dout"].float()
        dy = s["w"].reshape(-1)[entry].unsqueeze(-1) * dout[entry // c["k"]]
        dw = torch.zeros(c["N"] * c["k"], device=DEV)
        dw[entry] = (s["y"].float() * dout[entry // c["k"]]).sum(1)
        return {"dy": dy.to(torch.bfloat16), "dw": dw.view(c["N"], c["k"]), "dx": _back(s["dxs"], s["entry_rows"], None)}
    if op == "expert":
        x, place = _by_expert(s["x"], s["prefix"], s["most"])
        return {"y": torch.matmul(x, s["weight"].float().transpose(1, 2)).flatten(0, 1)[place].to(torch.bfloat16)}
    if op == "expert_grad":
        dy, place = _by_expert(s["dy"], s["prefix"], s["most"])
        x, _ = _by_expert(s["x"], s["prefix"], s["most"])
        dx = torch.matmul(dy, s["weight"].float()).flatten(0, 1)[place].to(torch.bfloat16)
        return {"dx": dx, "dw": torch.matmul(dy.transpose(1, 2), x).to(torch.bfloat16)}
    T, L, r = c["T"], c["L"], c["r"]
    x, ids = s["x"].float(), s["ids"]
    mine = (ids[:, None] == torch.arange(L, device=DEV)).float() * s["scales"]      # [T][L], scale or 0
    low = torch.matmul(x, s["a"].float().reshape(L * r, -1).t()).view(T, L, r) * mine.unsqueeze(-1)
    delta = torch.matmul(low.view(T, L * r), s["b"].float().transpose(1, 2).reshape(L * r, -1))
    return {"y": (torch.matmul(x, s["weight"].float().t()) + delta).to(torch.bfloat16)}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The same outputs from the definitions, entry by entry or expert by expert, in 64 bits."""
    c, s = case, _inputs(case, seed)
    f64 = torch.float64
    if c["op"] == "sort":
        return None         # whole numbers and copied bits
    if c["op"] in ("back", "grad"):
        rows_of = torch.full((c["N"] * c["k"],), -1, dtype=torch.int64, device=DEV)
        at, flat = 0, s["idx"].reshape(-1)
        for e in range(c["E"]):
            mine = (flat == e).nonzero().reshape(-1)
            rows_of[mine] = at + torch.arange(len(mine), device=DEV)
            at += len(mine)
        rows_of = rows_of.view(c["N"], c["k"])

        def total(y, w):
            out = torch.zeros(c["N"], c["H"], dtype=f64, device=DEV)
            for j in range(c["k"]):
                t = (rows_of[:, j] >= 0).nonzero().reshape(-1)
                part = y[rows_of[t, j]].to(f64)
                out[t] += part if w is None else part * w[t, j, None].to(f64)
            return out

        if c["op"] == "back":
            return {"out": total(s["y"], s["w"])}
        dy = torch.zeros(s["rows"], c["H"], dtype=f64, device=DEV)
        dw = torch.zeros(c["N"], c["k"], dtype=f64, device=DEV)
        for j in range(c["k"]):
            t = (rows_of[:, j] >= 0).nonzero().reshape(-1)
            d = s["dout"][t].to(f64)
            dy[rows_of[t, j]] = s["w"][t, j, None].to(f64) * d
            dw[t, j] = torch.einsum("th,th->t", d, s["y"][rows_of[t, j]].to(f64))
        return {"dy": dy, "dw": dw, "dx": total(s["dxs"], None)}
    if c["op"] in ("expert", "expert_grad"):
        edge = s["prefix"].tolist()
        if c["op"] == "expert":
            y = torch.zeros(c["rows"], c["F"], dtype=f64, device=DEV)
            for e in range(c["E"]):
                y[edge[e]:edge[e + 1]] = s["x"][edge[e]:edge[e + 1]].to(f64) @ s["weight"][e].to(f64).t()
            return {"y": y}
        dx = torch.zeros(c["rows"], c["K"], dtype=f64, device=DEV)
        dw = torch.zeros(c["E"], c["F"], c["K"], dtype=f64, device=DEV)
        for e in range(c["E"]):
            d = s["dy"][edge[e]:edge[e + 1]].to(f64)
            dx[edge[e]:edge[e + 1]] = d @ s["weight"][e].to(f64)
            dw[e] = d.t() @ s["x"][edge[e]:edge[e + 1]].to(f64)
        return {"dx": dx, "dw": dw}
    x = s["x"].to(f64)
    y = x @ s["weight"].to(f64).t()
    for i in range(c["L"]):
        t = (s["ids"] == i).nonzero().reshape(-1)
        y[t] += s["scales"][i].to(f64) * ((x[t] @ s["a"][i].to(f64).t()) @ s["b"][i].to(f64).t())
    return {"y": y}
