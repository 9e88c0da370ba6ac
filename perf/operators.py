"""Workloads of the operators whose rows pick their weights: routed rows
(sorted by expert, brought back with weights, and the gradient), the experts'
products with their gradients, and low-rank adapters beside a shared
projection.

Each case runs one operator once.  With `own` false `run` computes it from
elementary torch operations in 32 bits; with `own` true it calls this
repository's entry points.
"""
import math

import torch

own = False

ELEM = {"f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # Routing plan and row dispatch.  Decoding: a handful of requests, one
        # token each, 8 of 128 experts; latency is all that counts.
        {"name": "dispatch decode", "op": "dispatch", "tokens": 5, "top_k": 8, "experts": 128,
         "cols": 4096, "elem": "f16", "dropped": 0.0},
        # A prompt batch of one layer, many small experts.
        {"name": "dispatch prompt", "op": "dispatch", "tokens": 8192, "top_k": 8, "experts": 64,
         "cols": 2048, "elem": "f16", "dropped": 0.0},
        # Odd row length and a padded batch whose padding has no expert.
        {"name": "dispatch ragged padded", "op": "dispatch", "tokens": 3001, "top_k": 2, "experts": 8,
         "cols": 4095, "elem": "f32", "dropped": 0.2},
        # Expert outputs (FP32, as the products give them) back to tokens.
        {"name": "combine prompt", "op": "combine", "tokens": 8192, "top_k": 8, "experts": 64,
         "cols": 2048, "elem": "f32", "out": "f16", "weighted": True, "dropped": 0.0},
        # The dispatch's gradient: rows summed without weights.
        {"name": "dispatch gradient", "op": "combine", "tokens": 2000, "top_k": 2, "experts": 8,
         "cols": 4000, "elem": "f16", "out": "f16", "weighted": False, "dropped": 0.1},
        # The combine's gradient in training: rows and weights.
        {"name": "combine gradient", "op": "combine_grad", "tokens": 4096, "top_k": 4, "experts": 32,
         "cols": 4096, "elem": "f32", "out": "f32", "weighted": True, "dropped": 0.0},
        # The experts' products.  Decoding: a few rows for each of many
        # experts, bound by reading the weights.
        {"name": "experts decode", "op": "grouped", "rows": 64, "experts": 32, "k": 2048, "n": 2048,
         "spare": 0},
        # A prompt batch: hundreds of rows for each expert.
        {"name": "experts prompt", "op": "grouped", "rows": 16384, "experts": 16, "k": 4096, "n": 4096,
         "spare": 0},
        # Training: data and weight gradients, with padding rows at the end.
        {"name": "experts gradient", "op": "grouped_grad", "rows": 8192, "experts": 32, "k": 2048,
         "n": 4000, "spare": 100},
        # Adapters beside a shared projection.  Decoding: one token for each
        # of 16 requests, each with an adapter of its own or none.
        {"name": "adapters decode", "op": "lora", "tokens": 16, "k": 4096, "n": 4096, "adapters": 16,
         "rank": 16, "run": 1},
        # A prompt batch: a few hundred tokens of each request.
        {"name": "adapters prompt", "op": "lora", "tokens": 4096, "k": 4096, "n": 4096, "adapters": 8,
         "rank": 64, "run": 400},
        # Short prompts of many requests, odd rank and width.
        {"name": "adapters mixed ragged", "op": "lora", "tokens": 333, "k": 1000, "n": 4095,
         "adapters": 40, "rank": 9, "run": 7},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 or of 8, or any number, equally often."""
    w = _log(rng, lo, hi)
    step = rng.choice((64, 8, 1))
    return max(lo, w // step * step)


def draw(rng):
    """One more case, its cost below that of the largest listed case of its kind."""
    op = rng.choice(("dispatch", "combine", "combine_grad", "grouped", "grouped_grad", "lora"))
    if op in ("dispatch", "combine", "combine_grad"):
        top_k = rng.randint(1, 8)
        case = {"op": op, "tokens": _log(rng, 1, 16384), "top_k": top_k,
                "experts": max(top_k, _log(rng, 2, 256)), "cols": _width(rng, 64, 8192),
                "elem": rng.choice(("f16", "f32")), "dropped": rng.choice((0.0, 0.15))}
        if op != "dispatch":
            case["out"] = rng.choice(("f16", "f32"))
            case["weighted"] = op == "combine_grad" or rng.random() < 0.7
        limit = 8192 * 8 * 2048
        while case["tokens"] * top_k * case["cols"] > limit:
            case["tokens"] = max(1, case["tokens"] // 2 - rng.randint(0, 1))
        return case
    if op in ("grouped", "grouped_grad"):
        case = {"op": op, "rows": _log(rng, 1, 16384), "experts": _log(rng, 1, 64),
                "k": _width(rng, 64, 4096), "n": _width(rng, 64, 4096), "spare": rng.choice((0, 37))}
        limit = 8192 * 2048 * 4000 if op == "grouped_grad" else 16384 * 4096 * 4096
        while case["rows"] * case["k"] * case["n"] > limit:
            case["rows"] = max(1, case["rows"] // 2 - rng.randint(0, 1))
        while case["experts"] * case["k"] * case["n"] > 32 * 2048 * 4000:
            case["experts"] = max(1, case["experts"] // 2)
        return case
    return {"op": op, "tokens": _log(rng, 1, 4096), "k": _width(rng, 64, 4096), "n": _width(rng, 64, 4096),
            "adapters": _log(rng, 1, 64), "rank": rng.choice((4, 8, 9, 16, 32, 33, 64)),
            "run": rng.choice((1, 7, 400))}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _choices(case, g):
    """top_k different experts for every token, some experts liked more than
    others; the last `dropped` share of the tokens is padding (no expert)."""
    logits = _normal(g, case["tokens"], case["experts"]) + 0.5 * _normal(g, case["experts"])
    top = logits.topk(case["top_k"], dim=1)
    ids = top.indices.to(torch.int32)
    pad = int(case["tokens"] * case["dropped"])
    if pad:
        ids[case["tokens"] - pad:] = -1
    return ids.contiguous(), torch.softmax(top.values, dim=1).contiguous()


def _slots(ids, experts):
    """The place of every entry among the rows sorted by expert, -1 for none."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=flat.device)
    return torch.where(key < experts, slots, torch.full_like(slots, -1)).to(torch.int32).reshape(ids.shape)


def _offsets(case, g):
    """Group offsets of `rows` rows over the experts, some liked more."""
    logits = _normal(g, case["rows"], case["experts"]) + 0.3 * _normal(g, case["experts"])
    counts = torch.bincount(logits.argmax(dim=1), minlength=case["experts"])
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return torch.cat((zero, counts.cumsum(0))).to(torch.int32), int(counts.max())


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, H = case["tokens"], case["top_k"], case["cols"]
        st["ids"], st["w"] = _choices(case, g)
        elem = ELEM[case["elem"]]
        # the sorted rows' buffer, with one spare row behind its end
        if op == "dispatch":
            st["x"] = _normal(g, T, H, dtype=elem)
            st["out"] = torch.zeros(T * k + 1, H, dtype=elem, device="cuda")
        else:
            st["slots"] = _slots(st["ids"], case["experts"])
            st["z"] = _normal(g, T * k, H, dtype=elem)
            if op == "combine_grad":
                st["dy"] = _normal(g, T, H, dtype=ELEM[case["out"]])
                st["dz"] = torch.zeros(T * k + 1, H, dtype=elem, device="cuda")
    elif op in ("grouped", "grouped_grad"):
        E, K, N = case["experts"], case["k"], case["n"]
        R = case["rows"] + case["spare"]
        st["offsets"], st["most"] = _offsets(case, g)
        st["x"] = _normal(g, R, K, dtype=torch.float16)
        st["w"] = _normal(g, E, K, N, scale=K ** -0.5, dtype=torch.float16)
        if op == "grouped":
            st["y"] = torch.zeros(R + 1, N, device="cuda")
        else:
            st["dy"] = _normal(g, R, N, dtype=torch.float16)
            st["dx"] = torch.zeros(R + 1, K, device="cuda")
    else:
        T, K, N, n, r = (case[f] for f in ("tokens", "k", "n", "adapters", "rank"))
        st["x"] = _normal(g, T, K, dtype=torch.float16)
        st["w"] = _normal(g, K, N, scale=K ** -0.5, dtype=torch.float16)
        st["down"] = _normal(g, n, K, r, scale=K ** -0.5, dtype=torch.float16)
        st["up"] = _normal(g, n, r, N, scale=r ** -0.5, dtype=torch.float16)
        st["scale"] = torch.rand(n, generator=g, device="cuda") + 0.5
        # requests of `run` tokens; about one in n + 1 has no adapter
        pick = torch.randint(-1, n, (-(-T // case["run"]),), generator=g, device="cuda", dtype=torch.int32)
        st["adapter"] = pick.repeat_interleave(case["run"])[:T].contiguous()
    return st


# ------------------------------------------------------------------ one pass

def _plain_plan(ids, experts):
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < experts)
    key = torch.where(kept, flat, torch.full_like(flat, experts))
    by, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by, torch.arange(experts + 1, device=ids.device))
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=ids.device)
    none = torch.full_like(flat, -1)
    slots = torch.where(kept, slots, none)
    order = torch.where(by < experts, order, none)
    return offsets.to(torch.int32), order.to(torch.int32), slots.to(torch.int32).reshape(ids.shape)


def _plain_dispatch(st):
    offsets, order, slots = _plain_plan(st["ids"], st["case"]["experts"])
    out = st["out"]
    at = torch.where(slots < 0, torch.full_like(slots, out.shape[0] - 1), slots).long()
    out[at] = st["x"][:, None, :].expand(-1, at.shape[1], -1)
    return {"offsets": offsets, "order": order, "slots": slots, "out": out[:-1]}


def _plain_combine(st):
    slots = st["slots"].long()
    rows = st["z"][slots.clamp(min=0)].float()
    if st["case"]["weighted"]:
        rows = rows * st["w"][:, :, None]
    rows = torch.where((slots >= 0)[:, :, None], rows, torch.zeros((), device=rows.device))
    return rows.sum(dim=1).to(ELEM[st["case"]["out"]])


def _plain_combine_grad(st):
    slots, dz = st["slots"].long(), st["dz"]
    dy = st["dy"].float()[:, None, :]
    at = torch.where(slots < 0, torch.full_like(slots, dz.shape[0] - 1), slots)
    dz[at] = (st["w"][:, :, None] * dy).to(dz.dtype)
    dots = (st["z"][slots.clamp(min=0)].float() * dy).sum(dim=2)
    return {"dz": dz[:-1], "dw": torch.where(slots >= 0, dots, torch.zeros_like(dots))}


def _padded(st, x):
    """Each group's rows in a block of its own, `most` rows long, in 32 bits
    and zero behind the group's end; and the rows' places (the spare row
    behind the buffer's end for the padding)."""
    lo, hi = st["offsets"][:-1].long(), st["offsets"][1:].long()
    at = lo[:, None] + torch.arange(st["most"], device=x.device)
    inside = at < hi[:, None]
    rows = x[at.clamp(max=x.shape[0] - 1)].float()
    rows = torch.where(inside[:, :, None], rows, torch.zeros((), device=x.device))
    return rows, torch.where(inside, at, torch.full_like(at, x.shape[0]))


def _plain_grouped(st):
    rows, at = _padded(st, st["x"])
    st["y"][at] = torch.bmm(rows, st["w"].float())
    return st["y"][:-1]


def _plain_grouped_grad(st):
    x, _ = _padded(st, st["x"])
    dy, at = _padded(st, st["dy"])
    st["dx"][at] = torch.bmm(dy, st["w"].float().transpose(1, 2).contiguous())
    return {"dx": st["dx"][:-1], "dw": torch.bmm(x.transpose(1, 2).contiguous(), dy)}


def _plain_lora(st):
    x, down, up, pick = st["x"].float(), st["down"].float(), st["up"].float(), st["adapter"].long()
    n, K, r = down.shape
    low = (x @ down.permute(1, 0, 2).reshape(K, n * r)).reshape(-1, n, r)  # every adapter
    mine = pick[:, None] == torch.arange(n, device=x.device)
    low = torch.where(mine[:, :, None], low * st["scale"][None, :, None], torch.zeros((), device=x.device))
    return x @ st["w"].float() + low.reshape(-1, n * r) @ up.reshape(n * r, -1)


def _own(st):
    import tiled_dense_gemm_loop_amd as tdg
    case = st["case"]
    op = case["op"]
    if op == "dispatch":
        offsets, order, slots = tdg.tdg_route_plan(st["ids"], case["experts"])
        out = tdg.tdg_rows_dispatch(st["x"], slots, out=st["out"][:-1])
        return {"offsets": offsets, "order": order, "slots": slots, "out": out}
    if op == "combine":
        return tdg.tdg_rows_combine(st["z"], st["slots"], st["w"] if case["weighted"] else None,
                                    out_dtype=ELEM[case["out"]])
    if op == "combine_grad":
        dz, dw = tdg.tdg_rows_combine_grad(st["dy"], st["z"], st["slots"], st["w"], dz=st["dz"][:-1])
        return {"dz": dz, "dw": dw}
    if op == "grouped":
        return tdg.gemm_f16f32_grouped(st["x"], st["w"], st["offsets"], C=st["y"][:-1])
    if op == "grouped_grad":
        return {"dx": tdg.gemm_f16f32_grouped_nt(st["dy"], st["w"], st["offsets"], C=st["dx"][:-1]),
                "dw": tdg.gemm_f16f32_grouped_tn(st["x"], st["dy"], st["offsets"])}
    return tdg.gemm_f16f32_lora(st["x"], st["w"], st["down"], st["up"], st["adapter"], st["scale"])


_PLAIN = {"dispatch": _plain_dispatch, "combine": _plain_combine, "combine_grad": _plain_combine_grad,
          "grouped": _plain_grouped, "grouped_grad": _plain_grouped_grad, "lora": _plain_lora}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass needs

def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, H = case["tokens"], case["top_k"], case["cols"]
        kept = (T - int(T * case["dropped"])) * k
        es = 2 if case["elem"] == "f16" else 4
        if op == "dispatch":
            return {"bytes": T * H * es + kept * H * es + 12 * T * k + 4 * (case["experts"] + 1), "flops": 0}
        os = 2 if case["out"] == "f16" else 4
        tables = T * k * (8 if case["weighted"] else 4)
        if op == "combine":
            return {"bytes": kept * H * es + T * H * os + tables, "flops": 2 * kept * H}
        return {"bytes": 2 * kept * H * es + T * H * os + tables + 4 * T * k, "flops": 3 * kept * H}
    if op in ("grouped", "grouped_grad"):
        R, E, K, N = case["rows"], case["experts"], case["k"], case["n"]
        live = min(E, R)  # groups that can have rows
        if op == "grouped":
            return {"bytes": 2 * R * K + 2 * live * K * N + 4 * R * N, "flops": 2 * R * K * N}
        return {"bytes": 2 * R * (K + N) + 2 * live * K * N + 4 * R * K + 4 * E * K * N, "flops": 4 * R * K * N}
    T, K, N, n, r = (case[f] for f in ("tokens", "k", "n", "adapters", "rank"))
    live = min(n, -(-T // case["run"]))
    return {"bytes": 2 * T * K + 2 * K * N + 2 * live * r * (K + N) + 4 * T * N + 4 * T,
            "flops": 2 * T * K * N + 2 * T * r * (K + N)}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        E, k = case["experts"], case["top_k"]
        ids = st["ids"].reshape(-1).cpu()
        of = [(ids == e).nonzero().reshape(-1) for e in range(E)]  # ascending entries of each expert
        order = torch.cat(of)
        ends = torch.tensor([0] + [len(o) for o in of]).cumsum(0)
        if op == "dispatch":
            slots = torch.full((ids.numel(),), -1, dtype=torch.int64)
            slots[order] = torch.arange(order.numel())
            out = torch.zeros(ids.numel(), case["cols"], dtype=torch.float64, device="cuda")
            out[:order.numel()] = st["x"][(order // k).cuda()].double()
            full = torch.full((ids.numel(),), -1, dtype=torch.int64)
            full[:order.numel()] = order
            return {"offsets": ends.to(torch.int32), "order": full.to(torch.int32),
                    "slots": slots.to(torch.int32).reshape(-1, k), "out": out}
        order = order.cuda()
        token = order // k
        w = st["w"].reshape(-1).double()[order]
        z = st["z"][:order.numel()].double()
        if op == "combine":
            y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
            return y.index_add_(0, token, z * w[:, None] if case["weighted"] else z)
        dy = st["dy"].double()[token]
        dz = torch.zeros(ids.numel(), case["cols"], dtype=torch.float64, device="cuda")
        dz[:order.numel()] = dy * w[:, None]
        dw = torch.zeros(ids.numel(), dtype=torch.float64, device="cuda")
        dw[order] = (dy * z).sum(dim=1)
        return {"dz": dz, "dw": dw.reshape(-1, k)}
    if op in ("grouped", "grouped_grad"):
        ends = st["offsets"].tolist()
        K, N, x = case["k"], case["n"], st["x"]
        parts = list(zip(range(case["experts"]), ends, ends[1:]))
        if op == "grouped":
            y = torch.zeros(x.shape[0], N, dtype=torch.float64, device="cuda")
            for e, lo, hi in parts:
                if hi > lo:
                    y[lo:hi] = x[lo:hi].double() @ st["w"][e].double()
            return y
        dx = torch.zeros(x.shape[0], K, dtype=torch.float64, device="cuda")
        dw = torch.zeros(case["experts"], K, N, dtype=torch.float64, device="cuda")
        for e, lo, hi in parts:
            if hi > lo:
                dy = st["dy"][lo:hi].double()
                dx[lo:hi] = dy @ st["w"][e].double().t().contiguous()
                dw[e] = x[lo:hi].double().t().contiguous() @ dy
        return {"dx": dx, "dw": dw}
    x = st["x"].double()
    y = x @ st["w"].double()
    for a in range(case["adapters"]):
        rows = (st["adapter"] == a).nonzero().reshape(-1)
        if rows.numel():
            low = x[rows] @ st["down"][a].double()
            y[rows] += st["scale"][a].double() * (low @ st["up"][a].double())
    return y
