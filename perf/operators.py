"""The operators of a sparse expert layer and of a token embedding, as a program uses them.

route    the k best experts of each token from its router logits, their weights, and the logits' gradient
experts  tokens sorted by expert (rows copied in that order) and back (rows summed with their weights), and the
         gradients of both
embed    rows of a table looked up by token and scaled, and the table's gradient

Each case runs in a plain form (elementary torch operations in 32 bits, rounded once at the end) or, where `own`
is set, through this package's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases -----------------------------------------------------------------------------------------------------

def route_case(tokens, experts, k, dtype, score, renormalize, masked, train):
    return {"op": "route", "tokens": tokens, "experts": experts, "k": k, "dtype": dtype, "score": score,
            "renormalize": renormalize, "masked": masked, "train": train}


def experts_case(tokens, width, experts, k, dtype, dropped, strided, train):
    return {"op": "experts", "tokens": tokens, "width": width, "experts": experts, "k": k, "dtype": dtype,
            "dropped": dropped, "strided": strided, "train": train}


def embed_case(tokens, vocab, width, dtype, grad, accumulate, train):
    return {"op": "embed", "tokens": tokens, "vocab": vocab, "width": width, "dtype": dtype, "grad": grad,
            "accumulate": accumulate, "train": train}


def listed():
    return [
        # a decode step of a small batch: the call's latency counts
        dict(route_case(8, 64, 2, "f32", "softmax", True, False, False), name="route 8x64 k2 f32"),
        # an odd number of tokens in 16 bits with experts masked out, some tokens (padding) left with none; training
        dict(route_case(4097, 160, 6, "bf16", "sigmoid", True, True, True), name="route 4097x160 k6 bf16 train"),
        # a large training batch, weights from the softmax over all experts
        dict(route_case(65536, 256, 8, "f32", "softmax", False, False, True), name="route 65536x256 k8 f32 train"),
        # a decode step: 16 tokens there and back
        dict(experts_case(16, 2048, 64, 4, "bf16", False, False, False), name="experts 16x2048 of 64 k4 bf16"),
        # ragged: an odd batch, a width that is no power of two, slots without an expert, rows of a wider tensor
        dict(experts_case(1237, 1000, 60, 6, "f32", True, True, True), name="experts 1237x1000 of 60 k6 f32 train"),
        # an ordinary training step
        dict(experts_case(8192, 2048, 128, 8, "bf16", False, False, True), name="experts 8192x2048 of 128 k8 bf16 train"),
        # a large prefill
        dict(experts_case(32768, 4096, 256, 8, "bf16", False, False, False), name="experts 32768x4096 of 256 k8 bf16"),
        # a decode step over a large vocabulary
        dict(embed_case(16, 152064, 2048, "bf16", "bf16", False, False), name="embed 16 of 152064x2048 bf16"),
        # a prefill
        dict(embed_case(16384, 152064, 4096, "bf16", "bf16", False, False), name="embed 16384 of 152064x4096 bf16"),
        # a small training step in 32 bits
        dict(embed_case(2048, 32000, 1024, "f32", "f32", False, True), name="embed 2048 of 32000x1024 f32 train"),
        # odd sizes in 16 bits, the gradient added to a 32-bit one kept over several batches
        dict(embed_case(16383, 50001, 1000, "f16", "f32", True, True), name="embed 16383 of 50001x1000 f16 add"),
        # a large training step
        dict(embed_case(65536, 152064, 4096, "bf16", "bf16", False, True), name="embed 65536 of 152064x4096 bf16 train"),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A row width: mostly a multiple of 64, sometimes of 8, sometimes any."""
    w = _log_uniform(rng, low, high)
    step = rng.choice([64, 64, 64, 8, 1])
    return max(low, w // step * step)


def draw(rng):
    op = rng.choice(["route", "experts", "embed"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    train = rng.random() < 0.5
    if op == "route":
        tokens = _log_uniform(rng, 1, 65535)
        experts = _log_uniform(rng, 8, 256)
        k = rng.randint(1, min(8, experts))
        return route_case(tokens, experts, k, dtype, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5,
                          rng.random() < 0.3, train)
    if op == "experts":
        k = rng.randint(1, 8)
        experts = _log_uniform(rng, 8, 256)
        width = _width(rng, 128, 4096)
        # rows are read and written about six times in training, twice in a forward pass
        room = 32768 * 8 * 4096 * 2 // (3 if train else 1)
        tokens = _log_uniform(rng, 1, min(32768, room // (k * width * BYTES[dtype])))
        return experts_case(tokens, width, experts, k, dtype, rng.random() < 0.3, rng.random() < 0.3, train)
    vocab = _log_uniform(rng, 1000, 152063)
    width = _width(rng, 64, 4096 if dtype != "f32" else 2048)
    tokens = _log_uniform(rng, 1, 65536)
    grad = rng.choice([dtype, "f32"]) if vocab * width <= 152064 * 2048 else dtype
    accumulate = train and grad == "f32" and rng.random() < 0.5
    return embed_case(tokens, vocab, width, dtype, grad, accumulate, train)


# ---- inputs ----------------------------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _router_logits(tokens, experts, g, dtype=torch.float32):
    """Logits as a router gives them: some experts are liked more than others."""
    liked = 0.5 * torch.randn(experts, device="cuda", generator=g)
    return (1.5 * torch.randn(tokens, experts, device="cuda", generator=g) + liked).to(dtype)


def _rows(tokens, width, dtype, g, strided):
    """Activations; where `strided`, a part of the columns of a wider tensor."""
    wide = torch.randn(tokens, width + (24 if strided else 0), device="cuda", generator=g, dtype=dtype)
    return wide[:, 8:8 + width] if strided else wide


def _token_ids(tokens, vocab, g):
    """Ids as text has them: their frequency falls with their rank, and 3 in 100 are the padding token 0."""
    u = torch.rand(tokens, device="cuda", generator=g, dtype=torch.float64)
    ranks = torch.exp(u * math.log(vocab + 1)).long().clamp_(1, vocab) - 1
    ids = (ranks * 7919 + 13) % vocab if vocab % 7919 else ranks
    return torch.where(torch.rand(tokens, device="cuda", generator=g) < 0.03, 0, ids)


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    dtype = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "route":
        logits = _router_logits(c["tokens"], c["experts"], g, dtype)
        if c["masked"]:
            gone = torch.rand(logits.shape, device="cuda", generator=g) < 0.3
            gone |= torch.rand(c["tokens"], 1, device="cuda", generator=g) < 0.02
            logits.masked_fill_(gone, -math.inf)
        s["logits"] = logits
        s["scale"] = 1.0 if c["renormalize"] else 2.5
        if c["train"]:
            s["grad_weights"] = torch.randn(c["tokens"], c["k"], device="cuda", generator=g)
        return s
    if c["op"] == "experts":
        tokens, width, k = c["tokens"], c["width"], c["k"]
        scores, ids = _router_logits(tokens, c["experts"], g).topk(k, dim=1)
        ids = ids.int()
        if c["dropped"]:
            ids = torch.where(torch.rand(ids.shape, device="cuda", generator=g) < 0.1, -1, ids)
        s["expert_ids"] = ids.contiguous()
        s["weights"] = torch.softmax(scores, 1).contiguous()
        s["x"] = _rows(tokens, width, dtype, g, c["strided"])
        # what the experts answer, in the order of the sorted rows
        s["expert_out"] = torch.randn(tokens * k, width, device="cuda", generator=g, dtype=dtype)
        if c["train"]:
            s["grad_out"] = _rows(tokens, width, dtype, g, c["strided"])
            s["grad_rows"] = torch.randn(tokens * k, width, device="cuda", generator=g, dtype=dtype)
        return s
    s["table"] = 0.02 * torch.randn(c["vocab"], c["width"], device="cuda", generator=g, dtype=dtype)
    s["tokens"] = _token_ids(c["tokens"], c["vocab"], g)
    s["scale"] = math.sqrt(c["width"])
    if c["train"]:
        s["grad_out"] = torch.randn(c["tokens"], c["width"], device="cuda", generator=g, dtype=dtype)
        if c["accumulate"]:
            s["grad_table"] = torch.randn(c["vocab"], c["width"], device="cuda", generator=g, dtype=DTYPES[c["grad"]])
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------

def _plain_scores(logits, ids, score, renormalize):
    """Scores of all experts and of the chosen ones, the latter as they are weighted (before the scale)."""
    l = logits.float()
    some = ids >= 0
    at = ids.clamp(min=0).long()
    if score == "softmax":
        high = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(high == -math.inf, 0, high))
        every = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        every = 1 / (1 + torch.exp(-l))
    chosen = torch.where(some, every.gather(1, at), 0)
    if renormalize:
        return every, chosen / chosen.sum(1, keepdim=True).clamp(min=1e-30)
    return every, chosen


def _plain_route(logits, k, score, renormalize, scale):
    l = logits.float()
    order = torch.sort(l, dim=1, descending=True, stable=True)
    ids = torch.where(order.values[:, :k] == -math.inf, -1, order.indices[:, :k]).int()
    return ids, _plain_scores(logits, ids, score, renormalize)[1] * scale


def _plain_route_backward(grad, logits, ids, score, renormalize, scale):
    every, u = _plain_scores(logits, ids, score, renormalize)
    some = ids >= 0
    at = ids.clamp(min=0).long()
    g = torch.where(some, grad, 0) * scale
    if renormalize:
        part = u * (g - (u * g).sum(1, keepdim=True))
        if score == "sigmoid":
            part = part * (1 - every.gather(1, at))
    elif score == "sigmoid":
        part = g * u * (1 - u)
    else:
        part = g * u
    d = torch.zeros_like(every).scatter_add_(1, at, torch.where(some, part, 0))
    if score == "softmax" and not renormalize:
        d = d - every * (u * g).sum(1, keepdim=True)
    return d.to(logits.dtype)


def _plain_group(ids, experts):
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, experts, flat)
    slots = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.empty_like(slots)
    place[slots] = torch.arange(slots.numel(), device=slots.device)
    rows = torch.where(flat < 0, -1, place).int().reshape(ids.shape)
    slots = torch.where(key[slots] == experts, -1, slots).int()
    return offsets, rows, slots


def _plain_dispatch(x, slots, k):
    rows = x[slots.clamp(min=0).long() // k].float()
    return torch.where((slots >= 0)[:, None], rows, 0).to(x.dtype)


def _plain_gather_back(values, rows):
    """The rows of each token's slots, in 32 bits, zeros where a slot has none: [tokens, k, width]."""
    got = values[rows.clamp(min=0).long()].float()
    return torch.where((rows >= 0)[..., None], got, 0)


def _plain_combine_backward(grad_out, expert_out, rows, slots, weights):
    k = rows.shape[1]
    g = grad_out.float()
    grad_weights = (_plain_gather_back(expert_out, rows) * g[:, None, :]).sum(2)
    at = slots.clamp(min=0).long()
    grad_rows = g[at // k] * weights.reshape(-1)[at][:, None]
    return torch.where((slots >= 0)[:, None], grad_rows, 0).to(grad_out.dtype), grad_weights


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        how = (c["score"], c["renormalize"], s["scale"])
        ids, weights = _plain_route(s["logits"], c["k"], *how)
        out = {"expert_ids": ids, "weights": weights}
        if c["train"]:
            out["grad_logits"] = _plain_route_backward(s["grad_weights"], s["logits"], ids, *how)
        return out
    if c["op"] == "experts":
        offsets, rows, slots = _plain_group(s["expert_ids"], c["experts"])
        out = {"offsets": offsets, "row_of_slot": rows, "slot_of_row": slots}
        out["rows"] = _plain_dispatch(s["x"], slots, c["k"])
        back = _plain_gather_back(s["expert_out"], rows)
        out["out"] = (back * s["weights"][..., None]).sum(1).to(s["x"].dtype)
        if c["train"]:
            out["grad_expert_out"], out["grad_weights"] = _plain_combine_backward(
                s["grad_out"], s["expert_out"], rows, slots, s["weights"])
            out["grad_x"] = _plain_gather_back(s["grad_rows"], rows).sum(1).to(s["x"].dtype)
        return out
    out = {"out": (s["table"][s["tokens"]].float() * s["scale"]).to(s["table"].dtype)}
    if c["train"]:
        grad = torch.zeros(c["vocab"], c["width"], device="cuda")
        grad.index_add_(0, s["tokens"], s["grad_out"].float() * s["scale"])
        if c["accumulate"]:
            out["grad_table"] = s["grad_table"].add_(grad)
        else:
            out["grad_table"] = grad.to(DTYPES[c["grad"]])
    return out


# ---- this package ----------------------------------------------------------------------------------------------

_package = None


def _run_own(s):
    global _package
    if _package is None:
        import segmented_radix_top_gb300 as _package
    st = _package
    c = s["case"]
    if c["op"] == "route":
        how = {"score": c["score"], "renormalize": c["renormalize"], "scale": s["scale"]}
        ids, weights = st.route(s["logits"], c["k"], **how)
        out = {"expert_ids": ids, "weights": weights}
        if c["train"]:
            out["grad_logits"] = st.route_backward(s["grad_weights"], s["logits"], ids, **how)
        return out
    if c["op"] == "experts":
        groups = st.group_by_expert(s["expert_ids"], c["experts"])
        out = {"offsets": groups.offsets, "row_of_slot": groups.row_of_slot, "slot_of_row": groups.slot_of_row}
        out["rows"] = st.dispatch(s["x"], groups)
        out["out"] = st.combine(s["expert_out"], groups, s["weights"])
        if c["train"]:
            out["grad_expert_out"], out["grad_weights"] = st.combine_backward(
                s["grad_out"], s["expert_out"], groups, s["weights"])
            out["grad_x"] = st.dispatch_backward(s["grad_rows"], groups)
        return out
    out = {"out": st.embedding(s["table"], s["tokens"], scale=s["scale"])}
    if c["train"]:
        if c["accumulate"]:
            out["grad_table"] = st.embedding_backward(s["grad_out"], s["tokens"], c["vocab"], scale=s["scale"],
                                                      grad_table=s["grad_table"], accumulate=True)
        else:
            out["grad_table"] = st.embedding_backward(s["grad_out"], s["tokens"], c["vocab"], scale=s["scale"],
                                                      dtype=DTYPES[c["grad"]])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without -----------------------------------------------------------------------------

def _distinct(tokens, vocab):
    """Expected number of distinct ids among `tokens` of _token_ids."""
    edge = np.log(np.arange(1, vocab + 2, dtype=np.float64)) / math.log(vocab + 1)
    p = 0.97 * np.diff(edge)
    p[0] += 0.03
    return float((1 - (1 - p) ** tokens).sum())


def work(case):
    c = case
    b = BYTES[c["dtype"]]
    if c["op"] == "route":
        size = c["tokens"] * c["experts"]
        slots = c["tokens"] * c["k"]
        total = size * b + slots * 8
        if c["train"]:
            total += slots * 4 + size * b
        return {"bytes": total, "flops": 4.0 * size * (2 if c["train"] else 1)}
    if c["op"] == "experts":
        slots = c["tokens"] * c["k"]
        kept = slots * (0.9 if c["dropped"] else 1.0)
        one, many = c["tokens"] * c["width"] * b, slots * c["width"] * b
        read = kept * c["width"] * b
        index = slots * 4 + slots * 4 + slots * 8 + (c["experts"] + 1) * 8
        total = index + one + many + read + one
        flops = 2.0 * kept * c["width"]
        if c["train"]:
            total += one + many + slots * 4 + read + one
            flops *= 4
        return {"bytes": total, "flops": flops}
    distinct = _distinct(c["tokens"], c["vocab"])
    out = c["tokens"] * c["width"] * b
    total = c["tokens"] * 8 + distinct * c["width"] * b + out
    flops = 1.0 * c["tokens"] * c["width"]
    if c["train"]:
        row = c["width"] * BYTES[c["grad"]]
        total += out + (2 * distinct * row if c["accumulate"] else c["vocab"] * row)
        flops *= 3
    return {"bytes": total, "flops": flops}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------

def _exact_route(s):
    c = s["case"]
    l = s["logits"].double().cpu().numpy()
    rank = np.argsort(-l, axis=1, kind="stable")[:, :c["k"]]
    x = np.take_along_axis(l, rank, 1)
    ok = np.isfinite(x)
    if c["score"] == "softmax":
        top = np.where(ok[:, :1], x[:, :1], 0)
        e = np.exp(l - top)
        score = e / np.where(ok[:, :1], e.sum(1, keepdims=True), 1)
    else:
        score = 1 / (1 + np.exp(-l))
    a = np.where(ok, np.take_along_axis(score, rank, 1), 0)
    total = a.sum(1, keepdims=True) if c["renormalize"] else np.ones((len(a), 1))
    total = np.where(total > 0, total, 1)
    out = {"expert_ids": None, "weights": torch.from_numpy(s["scale"] * a / total)}
    if c["train"]:
        # through the Jacobian of each step: weights from chosen scores, scores from logits
        gw = np.where(ok, s["grad_weights"].double().cpu().numpy(), 0) * s["scale"]
        ga = gw / total
        if c["renormalize"]:
            ga = ga - (gw * a).sum(1, keepdims=True) / total ** 2
        full = np.zeros_like(l)
        np.put_along_axis(full, rank, np.where(ok, ga, 0), 1)
        if c["score"] == "softmax":
            d = score * (full - (full * score).sum(1, keepdims=True))
        else:
            d = full * score * (1 - score)
        out["grad_logits"] = torch.from_numpy(d)
    return out


def _exact_experts(s):
    c = s["case"]
    ids = s["expert_ids"].cpu().numpy()
    tokens, k = ids.shape
    flat = ids.reshape(-1)
    kept = np.flatnonzero(flat >= 0)
    slots = kept[np.lexsort((kept, flat[kept]))]
    place = np.full(flat.shape, -1, dtype=np.int64)
    place[slots] = np.arange(len(slots))
    slots_t = torch.from_numpy(slots).cuda()
    place_t = torch.from_numpy(place.reshape(ids.shape)).cuda()
    some = place_t >= 0
    w = torch.where(some, s["weights"].double(), 0)
    n, width = tokens * k, c["width"]
    out = {"offsets": None, "row_of_slot": None, "slot_of_row": None}
    x = s["x"].double()
    rows = torch.zeros(n, width, dtype=torch.float64, device="cuda")
    rows[:len(slots)] = x[slots_t // k]
    out["rows"] = rows
    total = torch.zeros_like(x)
    for j in range(k):
        total.addcmul_(s["expert_out"][place_t[:, j].clamp(min=0)].double(), w[:, j:j + 1])
    out["out"] = total
    if c["train"]:
        g = s["grad_out"].double()
        grad = torch.zeros_like(rows)
        grad[:len(slots)] = g[slots_t // k] * w.reshape(-1)[slots_t, None]
        out["grad_expert_out"] = grad
        grad_w = torch.zeros_like(w)
        grad_x = torch.zeros_like(x)
        for j in range(k):
            at, ok = place_t[:, j].clamp(min=0), some[:, j]
            grad_w[:, j] = torch.where(ok, torch.einsum("th,th->t", s["expert_out"][at].double(), g), 0)
            grad_x += s["grad_rows"][at].double() * ok[:, None]
        out["grad_weights"], out["grad_x"] = grad_w, grad_x
    return out


def _exact_embed(s):
    c = s["case"]
    t = s["tokens"]
    out = {"out": s["table"].double()[t] * s["scale"]}
    if c["train"]:
        # each distinct token's sum, by sorted positions
        order = torch.argsort(t, stable=True)
        ids, inverse = torch.unique_consecutive(t[order], return_inverse=True)
        sums = torch.zeros(len(ids), c["width"], dtype=torch.float64, device="cuda")
        sums.index_add_(0, inverse, s["grad_out"].double()[order] * s["scale"])
        if c["accumulate"]:
            grad = s["grad_table"].double()
        else:
            grad = torch.zeros(c["vocab"], c["width"], dtype=torch.float64, device="cuda")
        grad[ids] += sums
        out["grad_table"] = grad
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "embed": _exact_embed}[case["op"]](s)
