"""Workloads of the 4-bit weights (quantizing them, products with them, the
experts' products with them) and of a whole layer of experts for a few tokens.

Each case runs one operator once.  With `own` false `run` computes it from
elementary torch operations in 32 bits; with `own` true it calls this
repository's entry points.

4-bit weights of a K x N matrix: codes (ceil(K / 128), N, 64) of uint8; the
weight k = 128 b + 32 j + 8 q + i of column n is the nibble at bit
4 (i / 2) + 16 (i % 2) of the little-endian 32-bit word 4 q + j of
codes[b, n]; scales (and zeros) have a row per `group` values of k.  The
weight's value is (code - zero) * scale, zero 8 where there are no zeros.
"""
import math

import torch

own = False

ELEM = {"f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # Making 4-bit weights of a square projection and reading them back
        # (loading a model, or training that rounds its weights).
        {"name": "quantize projection", "op": "quantize", "count": 1, "k": 4096, "n": 4096, "group": 128,
         "zeros": False},
        # A stack of experts' matrices, odd in both sizes, with zero points.
        {"name": "quantize experts ragged", "op": "quantize", "count": 8, "k": 1000, "n": 4095, "group": 64,
         "zeros": True},
        # A projection in decoding, one request: all that counts is reading
        # 8 MB of codes, and latency.
        {"name": "w4 one token", "op": "w4", "rows": 1, "k": 4096, "n": 4096, "group": 128, "zeros": False},
        # A small batch, small groups with zero points, odd sizes.
        {"name": "w4 batch ragged", "op": "w4", "rows": 13, "k": 4000, "n": 4095, "group": 32, "zeros": True},
        # A full batch of requests on a wide projection.
        {"name": "w4 batch wide", "op": "w4", "rows": 32, "k": 4096, "n": 16384, "group": 128, "zeros": False},
        # A piece of a prompt, bound by operations.
        {"name": "w4 prompt", "op": "w4", "rows": 1024, "k": 4096, "n": 4096, "group": 128, "zeros": False},
        # The experts' products.  Decoding: a few rows for each of many.
        {"name": "w4 experts decode", "op": "w4_grouped", "rows": 64, "experts": 32, "k": 2048, "n": 2048,
         "group": 128, "zeros": False, "spare": 0},
        # A prompt batch: hundreds of rows for each expert.
        {"name": "w4 experts prompt", "op": "w4_grouped", "rows": 8192, "experts": 16, "k": 4096, "n": 4096,
         "group": 64, "zeros": False, "spare": 0},
        # Short prompts, odd sizes, zero points, padding rows at the end.
        {"name": "w4 experts ragged", "op": "w4_grouped", "rows": 333, "experts": 9, "k": 1000, "n": 1537,
         "group": 32, "zeros": True, "spare": 37},
        # A whole layer of experts.  One token of one request, 8 of 128
        # experts: two dependent products that read 75 MB.
        {"name": "layer one token", "op": "layer", "tokens": 1, "top_k": 8, "experts": 128, "cols": 2048,
         "inner": 768, "out": "f16", "dropped": 0.0},
        # A batch of requests that reaches most of the experts.
        {"name": "layer batch", "op": "layer", "tokens": 16, "top_k": 8, "experts": 64, "cols": 2048,
         "inner": 1024, "out": "f16", "dropped": 0.0},
        # Few large experts, several rows for each, odd sizes, padding tokens.
        {"name": "layer ragged padded", "op": "layer", "tokens": 33, "top_k": 2, "experts": 8, "cols": 4095,
         "inner": 1001, "out": "f32", "dropped": 0.2},
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
    op = rng.choice(("quantize", "w4", "w4_grouped", "layer"))
    if op == "layer":
        top_k = rng.randint(1, 8)
        case = {"op": op, "tokens": _log(rng, 1, 64), "top_k": top_k, "experts": max(top_k, _log(rng, 4, 128)),
                "cols": _width(rng, 64, 4096), "inner": _width(rng, 64, 4096), "out": rng.choice(("f16", "f32")),
                "dropped": rng.choice((0.0, 0.15))}
        while case["experts"] * case["cols"] * case["inner"] > 128 * 2048 * 768:
            case["inner"] = max(64, case["inner"] // 2 - rng.randint(0, 1))
            case["experts"] = max(top_k, case["experts"] * 3 // 4)
        # each entry at most its expert's three matrices, as the listed batch
        while case["tokens"] * top_k * case["cols"] * case["inner"] > 16 * 8 * 2048 * 1024:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    case = {"op": op, "k": _width(rng, 64, 4096), "n": _width(rng, 64, 4096), "group": rng.choice((32, 64, 96, 128)),
            "zeros": rng.random() < 0.4}
    if op == "quantize":
        case["count"] = _log(rng, 1, 16)
        while case["count"] * case["k"] * case["n"] > 8 * 1000 * 4095:
            case["count"] = max(1, case["count"] // 2)
            case["n"] = max(64, case["n"] * 3 // 4)
        return case
    if op == "w4":
        case["rows"] = _log(rng, 1, 1024)
        return case
    case.update(rows=_log(rng, 1, 8192), experts=_log(rng, 1, 64), spare=rng.choice((0, 37)))
    while case["experts"] * case["k"] * case["n"] > 16 * 4096 * 4096:
        case["experts"] = max(1, case["experts"] // 2)
    return case


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _weights4(case, g, count):
    """Codes, scales and zero points of `count` matrices; the codes behind K,
    which nothing may use, are random too."""
    K, N = case["k"], case["n"]
    groups = -(-K // case["group"])
    codes = torch.randint(0, 256, (count, -(-K // 128), N, 64), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(count, groups, N, generator=g, device="cuda") + 0.5) * (0.2 * K ** -0.5)).half()
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(5, 11, (count, groups, N), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales, zeros


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
    if op == "quantize":
        st["w"] = _normal(g, case["count"], case["k"], case["n"], scale=case["k"] ** -0.5, dtype=torch.float16)
    elif op == "w4":
        codes, scales, zeros = _weights4(case, g, 1)
        st["codes"], st["scales"], st["zeros"] = codes[0], scales[0], None if zeros is None else zeros[0]
        st["x"] = _normal(g, case["rows"], case["k"], dtype=torch.float16)
    elif op == "w4_grouped":
        R = case["rows"] + case["spare"]
        st["codes"], st["scales"], st["zeros"] = _weights4(case, g, case["experts"])
        st["offsets"], st["most"] = _offsets(case, g)
        st["x"] = _normal(g, R, case["k"], dtype=torch.float16)
        st["y"] = torch.zeros(R + 1, case["n"], device="cuda")  # with one spare row behind its end
    else:
        T, k, E, H, I = (case[f] for f in ("tokens", "top_k", "experts", "cols", "inner"))
        top = _normal(g, T, E).topk(k, dim=1)
        st["ids"], st["weights"] = top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1).contiguous()
        pad = int(T * case["dropped"])  # the last tokens are padding: no expert
        if pad:
            st["ids"][T - pad:] = -1
        st["x"] = _normal(g, T, H, dtype=torch.float16)
        st["up"] = _normal(g, E, H, 2 * I, scale=H ** -0.5, dtype=torch.float16)
        st["down"] = _normal(g, E, I, H, scale=I ** -0.5, dtype=torch.float16)
    return st


# ------------------------------------------------------------------ one pass

def _plain_codes(codes, K):
    """The codes of a stack, count x K x N, as 32-bit floats."""
    count, blocks, N, _ = codes.shape
    nib = torch.stack((codes & 15, codes >> 4), dim=-1)
    # byte 16 q + 4 j + 2 b1 + b0, nibble h: k = 32 j + 8 q + 4 b0 + 2 h + b1
    nib = nib.view(count, blocks, N, 4, 4, 2, 2, 2).permute(0, 1, 4, 3, 6, 7, 5, 2)
    return nib.reshape(count, blocks * 128, N)[:, :K].float()


def _plain_values(codes, scales, zeros, K, group):
    each = torch.arange(K, device=codes.device) // group
    q = _plain_codes(codes, K)
    q -= 8.0 if zeros is None else zeros.float()[:, each]
    return q.mul_(scales.float()[:, each])


def _plain_quantize(st):
    case, w = st["case"], st["w"].float()
    count, K, N = w.shape
    group = case["group"]
    groups = -(-K // group)
    zero = torch.zeros((), device=w.device)
    each = torch.arange(K, device=w.device) // group
    padded = torch.cat((w, zero.expand(count, groups * group - K, N)), dim=1).view(count, groups, group, N)
    if case["zeros"]:
        lo, hi = padded.amin(dim=2).clamp(max=0), padded.amax(dim=2).clamp(min=0)
        scales = ((hi - lo) / 15).half()
        s = scales.float()
        zeros = torch.where(s > 0, torch.round(-lo / s), zero).clamp(0, 15)
        least, most, add = -zeros, 15 - zeros, zeros
    else:
        scales = (padded.abs().amax(dim=2) / 7).half()
        s, zeros = scales.float(), None
        least, most = torch.full_like(s, -8), torch.full_like(s, 7)
    q = torch.where(s[:, each] > 0, torch.round(w / s[:, each]), zero)
    q = torch.minimum(torch.maximum(q, least[:, each]), most[:, each])
    out = {"values": (q * s[:, each]).half(), "scales": scales}
    if zeros is not None:
        out["zeros"] = zeros.to(torch.uint8)
    return out


def _plain_w4(st):
    case = st["case"]
    zeros = None if st["zeros"] is None else st["zeros"][None]
    w = _plain_values(st["codes"][None], st["scales"][None], zeros, case["k"], case["group"])
    return st["x"].float() @ w[0]


def _plain_w4_grouped(st):
    case, x = st["case"], st["x"]
    w = _plain_values(st["codes"], st["scales"], st["zeros"], case["k"], case["group"])
    # each group's rows in a block of its own, `most` rows long; what lies
    # behind a group's end goes to the spare row
    lo, hi = st["offsets"][:-1].long(), st["offsets"][1:].long()
    at = lo[:, None] + torch.arange(st["most"], device=x.device)
    inside = at < hi[:, None]
    rows = x[at.clamp(max=x.shape[0] - 1)].float()
    rows = torch.where(inside[:, :, None], rows, torch.zeros((), device=x.device))
    st["y"][torch.where(inside, at, torch.full_like(at, x.shape[0]))] = torch.bmm(rows, w)
    return st["y"][:-1]


def _plain_layer(st):
    case, ids = st["case"], st["ids"].long()
    T, k, E, I = (case[f] for f in ("tokens", "top_k", "experts", "inner"))
    x = st["x"].float()
    kept = (ids >= 0) & (ids < E)
    pick = torch.where(kept, ids, torch.zeros_like(ids)).reshape(-1)
    entry = torch.arange(T * k, device=x.device)
    if T * k <= E:  # each entry's own matrices
        both = torch.bmm(x[entry // k][:, None], st["up"][pick].float())
        h = both[..., :I] / (1 + torch.exp(-both[..., :I])) * both[..., I:]
        z = torch.bmm(h, st["down"][pick].float())[:, 0]
    else:  # every token through every expert
        both = torch.bmm(x.expand(E, -1, -1).contiguous(), st["up"].float())
        h = both[..., :I] / (1 + torch.exp(-both[..., :I])) * both[..., I:]
        z = torch.bmm(h, st["down"].float())[pick, entry // k]
    w = torch.where(kept, st["weights"], torch.zeros((), device=x.device))
    return (z.view(T, k, -1) * w[:, :, None]).sum(dim=1).to(ELEM[case["out"]])


def _own(st):
    import tiled_dense_gemm_loop_amd as tdg
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        codes, scales, zeros = tdg.tdg_w4_quantize(st["w"], case["group"], zeros=case["zeros"])
        values = tdg.tdg_w4_dequantize(codes, scales, zeros, K=case["k"], group=case["group"])
        out = {"values": values, "scales": scales}
        if zeros is not None:
            out["zeros"] = zeros
        return out
    if op == "w4":
        return tdg.gemm_f16w4f32(st["x"], st["codes"], st["scales"], st["zeros"], group=case["group"])
    if op == "w4_grouped":
        return tdg.gemm_f16w4f32_grouped(st["x"], st["codes"], st["scales"], st["offsets"], st["zeros"],
                                         group=case["group"], C=st["y"][:-1])
    return tdg.tdg_expert_layer(st["x"], st["ids"], st["weights"], st["up"], st["down"],
                                out_dtype=ELEM[case["out"]])


_PLAIN = {"quantize": _plain_quantize, "w4": _plain_w4, "w4_grouped": _plain_w4_grouped, "layer": _plain_layer}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass needs

def _bytes4(case):
    """Bytes of one matrix's codes, scales and zero points."""
    K, N = case["k"], case["n"]
    return -(-K * N // 2) + -(-K // case["group"]) * N * (3 if case["zeros"] else 2)


def work(case):
    op = case["op"]
    if op == "quantize":  # codes are written, and read to give the values
        n = case["count"] * case["k"] * case["n"]
        return {"bytes": 4 * n + 2 * case["count"] * _bytes4(case), "flops": 4 * n}
    if op == "w4":
        M, K, N = case["rows"], case["k"], case["n"]
        return {"bytes": 2 * M * K + 4 * M * N + _bytes4(case), "flops": 2 * M * K * N}
    if op == "w4_grouped":
        R, K, N = case["rows"], case["k"], case["n"]
        return {"bytes": 2 * R * K + 4 * R * N + min(case["experts"], R) * _bytes4(case), "flops": 2 * R * K * N}
    T, k, E, H, I = (case[f] for f in ("tokens", "top_k", "experts", "cols", "inner"))
    kept = T - int(T * case["dropped"])
    live = E * (1 - (1 - k / E) ** kept)  # experts that some token picks, on average
    es = 2 if case["out"] == "f16" else 4
    return {"bytes": int(live * 6 * H * I) + T * H * (2 + es) + 8 * T * k, "flops": 6 * kept * k * H * I}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_weights(codes, scales, zeros, K, group):
    """(code - zero) * scale of one matrix, K x N."""
    words = codes.contiguous().view(torch.int32)  # blocks x N x 16
    rows = []
    for k in range(128):
        j, q, i = k // 32, k % 32 // 8, k % 8
        rows.append(words[:, :, 4 * q + j] >> (4 * (i // 2) + 16 * (i % 2)) & 15)
    code = torch.stack(rows, dim=1).reshape(-1, codes.shape[1])[:K].double()
    for g in range(scales.shape[0]):
        part = code[g * group:(g + 1) * group]
        part -= 8 if zeros is None else zeros[g].double()
        part *= scales[g].double()
    return code


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        w, group = st["w"].double(), case["group"]
        values = torch.empty_like(w)
        scales, zeros = [], []
        for at in range(0, case["k"], group):
            part = w[:, at:at + group]
            if case["zeros"]:
                lo, hi = part.amin(dim=1).clamp(max=0), part.amax(dim=1).clamp(min=0)
                s = ((hi - lo) / 15).half().double()
                z = (-lo / s).round().clamp(0, 15)
                zeros.append(z)
            else:
                s = (part.abs().amax(dim=1) / 7).half().double()
                z = torch.full_like(s, 8)
            code = ((part / s[:, None]).round() + z[:, None]).clamp(0, 15)
            values[:, at:at + group] = (code - z[:, None]) * s[:, None]
            scales.append(s)
        out = {"values": values, "scales": torch.stack(scales, dim=1)}
        if zeros:
            out["zeros"] = torch.stack(zeros, dim=1).to(torch.uint8)
        return out
    if op == "w4":
        return st["x"].double() @ _exact_weights(st["codes"], st["scales"], st["zeros"], case["k"], case["group"])
    if op == "w4_grouped":
        ends, x = st["offsets"].tolist(), st["x"]
        y = torch.zeros(x.shape[0], case["n"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                zeros = None if st["zeros"] is None else st["zeros"][e]
                y[lo:hi] = x[lo:hi].double() @ _exact_weights(st["codes"][e], st["scales"][e], zeros, case["k"],
                                                              case["group"])
        return y
    I = case["inner"]
    y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
    ids = st["ids"].long()
    for e in range(case["experts"]):
        token, j = (ids == e).nonzero(as_tuple=True)
        if token.numel():
            both = st["x"][token].double() @ st["up"][e].double()
            h = both[:, :I] * torch.sigmoid(both[:, :I]) * both[:, I:]
            y.index_add_(0, token, (h @ st["down"][e].double()) * st["weights"][token, j].double()[:, None])
    return y
