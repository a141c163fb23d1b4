"""What stands between the steps of a sparse expert layer, as a program uses it.

norm      layer norm of rows, with the gradients of the rows, the weight and the bias
groups    routing limited to the best groups of experts
quantize  rows in 8-bit floating point with a scale for each block of 128
product8  each expert's matrix product of its rows, both in 8-bit floating point with their blocks' scales
product   the same in 16 bits, with the gradients of the rows and of the weights

Each case runs in a plain form (elementary torch operations in 32 bits, rounded once at the end) or, where `own`
is set, through this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128          # of the scales
LARGEST = 448.0      # of e4m3
SMALLEST = 2.0**-100  # below it a block's largest value counts as this
EPS = 1e-5


# ---- cases -----------------------------------------------------------------------------------------------------

def norm_case(tokens, width, dtype, strided, train):
    return {"op": "norm", "tokens": tokens, "width": width, "dtype": dtype, "strided": strided, "train": train}


def groups_case(tokens, experts, k, num_groups, kept, dtype, score, renormalize, masked):
    return {"op": "groups", "tokens": tokens, "experts": experts, "k": k, "num_groups": num_groups, "kept": kept,
            "dtype": dtype, "score": score, "renormalize": renormalize, "masked": masked}


def quantize_case(tokens, width, dtype, strided):
    return {"op": "quantize", "tokens": tokens, "width": width, "dtype": dtype, "strided": strided}


def product8_case(tokens, k, experts, width, out_width, dtype, dropped):
    return {"op": "product8", "tokens": tokens, "k": k, "experts": experts, "width": width, "out_width": out_width,
            "dtype": dtype, "dropped": dropped}


def product_case(tokens, k, experts, width, out_width, dtype, dropped, train):
    return {"op": "product", "tokens": tokens, "k": k, "experts": experts, "width": width, "out_width": out_width,
            "dtype": dtype, "dropped": dropped, "train": train}


def listed():
    return [
        # a decode step of a small batch: the call's latency counts
        dict(norm_case(16, 2048, "bf16", False, False), name="norm 16x2048 bf16"),
        # an odd batch of odd rows, a part of a wider tensor's columns, in training
        dict(norm_case(1237, 1001, "f32", True, True), name="norm 1237x1001 f32 train"),
        # a large training batch
        dict(norm_case(65536, 4096, "bf16", False, True), name="norm 65536x4096 bf16 train"),
        # a decode step: few tokens, 8 of 256 experts from 4 of 8 groups
        dict(groups_case(64, 256, 8, 8, 4, "bf16", "sigmoid", True, False), name="groups 64x256 4 of 8 k8 bf16"),
        # a large batch whose groups are no powers of two, some experts masked out, some tokens left with none
        dict(groups_case(65535, 160, 6, 8, 3, "f32", "softmax", False, True), name="groups 65535x160 3 of 8 k6 f32"),
        # a decode step's rows
        dict(quantize_case(64, 2048, "bf16", False), name="quantize 64x2048 bf16"),
        # a prefill's rows
        dict(quantize_case(131072, 4096, "bf16", False), name="quantize 131072x4096 bf16"),
        # a decode step: one or two rows for each expert that is used at all
        dict(product8_case(16, 4, 64, 2048, 1024, "bf16", False), name="product8 16 k4 of 64 2048x1024"),
        # ragged: an odd batch, the last block of the width and of the columns in part, slots without an expert
        dict(product8_case(1237, 6, 60, 1040, 1000, "f32", True), name="product8 1237 k6 of 60 1040x1000"),
        # a prefill
        dict(product8_case(16384, 8, 128, 4096, 2048, "bf16", False), name="product8 16384 k8 of 128 4096x2048"),
        # a small training step, ragged in every size
        dict(product_case(1237, 6, 60, 1000, 1096, "f16", True, True), name="product 1237 k6 of 60 1000x1096 f16 train"),
        # an ordinary training step
        dict(product_case(8192, 8, 128, 2048, 1024, "bf16", False, True),
             name="product 8192 k8 of 128 2048x1024 bf16 train"),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high, least):
    """A row width: mostly a multiple of 64, sometimes only of `least`."""
    w = _log_uniform(rng, low, high)
    step = rng.choice([64, 64, 64, 8, 1])
    step = max(step, least)
    return max(low, w // step * step)


def draw(rng):
    op = rng.choice(["norm", "groups", "quantize", "product8", "product8", "product", "product"])
    if op == "norm":
        dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
        width = _width(rng, 64, 8192, 1)
        tokens = _log_uniform(rng, 1, min(65536, 65536 * 4096 * 2 // (width * BYTES[dtype])))
        return norm_case(tokens, width, dtype, rng.random() < 0.3, rng.random() < 0.6)
    if op == "groups":
        num_groups = rng.choice([2, 4, 8, 8, 16])
        size = _log_uniform(rng, 2, 256 // num_groups)
        experts = num_groups * size
        kept = rng.randint(1, num_groups)
        k = rng.randint(1, min(8, kept * size))
        return groups_case(_log_uniform(rng, 1, 65535), experts, k, num_groups, kept, rng.choice(["f32", "bf16"]),
                           rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, rng.random() < 0.3)
    if op == "quantize":
        width = _width(rng, 128, 8192, 16)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        tokens = _log_uniform(rng, 1, min(131072, 131072 * 4096 * 2 // (width * BYTES[dtype])))
        return quantize_case(tokens, width, dtype, rng.random() < 0.3)
    k = rng.randint(1, 8)
    experts = _log_uniform(rng, 8, 256)
    width = _width(rng, 128, 4096, 16 if op == "product8" else 8)
    out_width = _width(rng, 128, 4096, 8)
    while experts * width * out_width > 128 * 4096 * 1024:
        experts = max(8, experts // 2)
    if op == "product8":
        most = 16384 * 8 * 4096 * 2048 // (k * width * out_width)
        return product8_case(_log_uniform(rng, 1, min(16384, most)), k, experts, width, out_width,
                             rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.3)
    train = rng.random() < 0.6
    most = 8192 * 8 * 2048 * 1024 // (k * width * out_width)
    return product_case(_log_uniform(rng, 1, max(1, min(16384, most))), k, experts, width, out_width,
                        rng.choice(["bf16", "bf16", "f16"]), rng.random() < 0.3, train)


# ---- inputs ----------------------------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(*shape, g, dtype=torch.float32):
    return torch.randn(*shape, device="cuda", generator=g, dtype=dtype)


def _router_logits(tokens, experts, g, dtype=torch.float32):
    """Logits as a router gives them: some experts are liked more than others."""
    return (1.5 * _randn(tokens, experts, g=g) + 0.5 * _randn(experts, g=g)).to(dtype)


def _activations(tokens, width, dtype, g, strided):
    """Rows of different sizes with an offset; where `strided`, a part of the columns of a wider tensor."""
    wide = _randn(tokens, width + (32 if strided else 0), g=g, dtype=dtype)
    wide.mul_(torch.exp(0.5 * _randn(tokens, 1, g=g))).add_(0.25)
    return wide[:, 16:16 + width] if strided else wide


def _sorted_slots(c, g):
    """Token slots sorted by expert, as routing leaves them: offsets, row of each slot, slot of each row."""
    tokens, k, experts = c["tokens"], c["k"], c["experts"]
    ids = _router_logits(tokens, experts, g).topk(k, dim=1).indices
    if c["dropped"]:
        ids = torch.where(torch.rand(ids.shape, device="cuda", generator=g) < 0.1, experts, ids)
    flat = ids.reshape(-1)
    slots = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=experts + 1)[:experts]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.empty_like(slots)
    place[slots] = torch.arange(slots.numel(), device="cuda")
    rows = torch.where(flat == experts, -1, place).int().reshape(tokens, k)
    return offsets, rows, torch.where(flat[slots] == experts, -1, slots).int()


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _quantized(x, rows):
    """x in 8 bits with a float32 scale for each block of `rows` by BLOCK values: (values, scales)."""
    lead, (n, width) = x.shape[:-2], x.shape[-2:]
    full = x.new_zeros(*lead, -(-n // rows) * rows, _blocks(width) * BLOCK)
    full[..., :n, :width] = x
    tiles = full.reshape(*lead, full.shape[-2] // rows, rows, full.shape[-1] // BLOCK, BLOCK)
    largest = tiles.abs().amax((-3, -1), keepdim=True).clamp(min=SMALLEST)
    values = (tiles * (LARGEST / largest)).to(torch.float8_e4m3fn).reshape(full.shape)[..., :n, :width].contiguous()
    return values, (largest / LARGEST).squeeze(-1).squeeze(-2).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    dtype = DTYPES[c["dtype"]]
    s = {"case": c}
    tokens = c["tokens"]
    if c["op"] == "norm":
        s["x"] = _activations(tokens, c["width"], dtype, g, c["strided"])
        s["weight"] = (1 + 0.1 * _randn(c["width"], g=g)).to(dtype)
        s["bias"] = (0.1 * _randn(c["width"], g=g)).to(dtype)
        if c["train"]:
            s["grad_out"] = _randn(tokens, c["width"], g=g, dtype=dtype)
        return s
    if c["op"] == "groups":
        logits = _router_logits(tokens, c["experts"], g, dtype)
        if c["masked"]:
            gone = torch.rand(logits.shape, device="cuda", generator=g) < 0.3
            gone |= torch.rand(tokens, 1, device="cuda", generator=g) < 0.02
            logits.masked_fill_(gone, -math.inf)
        s["logits"] = logits
        s["scale"] = 1.0 if c["renormalize"] else 2.5
        return s
    if c["op"] == "quantize":
        s["x"] = _activations(tokens, c["width"], dtype, g, c["strided"])
        return s
    n, experts, width, out_width = tokens * c["k"], c["experts"], c["width"], c["out_width"]
    s["groups"] = _sorted_slots(c, g)
    # for the plain form: the experts' first rows, known on the host
    s["bounds"] = s["groups"][0].tolist()
    if c["op"] == "product8":
        s["rows"], s["row_scales"] = _quantized(_activations(n, width, torch.float32, g, False), 1)
        weights, scales = zip(*(_quantized(0.02 * _randn(out_width, width, g=g), BLOCK) for _ in range(experts)))
        s["weights"], s["weight_scales"] = torch.stack(weights), torch.stack(scales)
        return s
    s["rows"] = _randn(n, width, g=g, dtype=dtype)
    s["weights"] = _randn(experts, out_width, width, g=g, dtype=dtype).mul_(width**-0.5)
    if c["train"]:
        s["grad_out"] = _randn(n, out_width, g=g, dtype=dtype)
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------

def _plain_norm(s):
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    mean = x.sum(1, keepdim=True) / x.shape[1]
    centred = x - mean
    rstd = 1 / torch.sqrt((centred * centred).sum(1, keepdim=True) / x.shape[1] + EPS)
    hat = centred * rstd
    dtype = s["x"].dtype
    out = {"out": (hat * w + b).to(dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if "grad_out" in s:
        g = s["grad_out"].float()
        gw = g * w
        inner = gw - gw.sum(1, keepdim=True) / x.shape[1] - hat * ((gw * hat).sum(1, keepdim=True) / x.shape[1])
        out["grad_x"] = (inner * rstd).to(dtype)
        out["grad_weight"] = (g * hat).sum(0).to(dtype)
        out["grad_bias"] = g.sum(0).to(dtype)
    return out


def _plain_groups(s):
    c = s["case"]
    l = s["logits"].float()
    tokens, experts = l.shape
    best = l.reshape(tokens, c["num_groups"], -1).amax(2)
    order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
    keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
    keep = keep.repeat_interleave(experts // c["num_groups"], dim=1)
    order = torch.sort(torch.where(keep, l, -math.inf), dim=1, descending=True, stable=True)
    ids = torch.where(order.values[:, :c["k"]] == -math.inf, -1, order.indices[:, :c["k"]])
    if c["score"] == "softmax":
        high = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(high == -math.inf, 0, high))
        every = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        every = 1 / (1 + torch.exp(-l))
    chosen = torch.where(ids >= 0, every.gather(1, ids.clamp(min=0)), 0)
    if c["renormalize"]:
        chosen = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-30)
    return {"expert_ids": ids.int(), "weights": chosen * s["scale"]}


def _plain_quantize(s):
    values, scales = _quantized(s["x"].float(), 1)
    return {"values": values, "scales": scales}


def _spread(scales, rows, n, width):
    """Each value's scale: blocks of `rows` by BLOCK values."""
    return scales.repeat_interleave(rows, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :width]


def _full_precision(call):
    """32-bit products in 32 bits, whatever the program has set."""
    def wrapped(*args):
        was = torch.backends.cuda.matmul.allow_tf32
        torch.backends.cuda.matmul.allow_tf32 = False
        try:
            return call(*args)
        finally:
            torch.backends.cuda.matmul.allow_tf32 = was
    return wrapped


@_full_precision
def _plain_product8(s):
    c = s["case"]
    n, width, out_width = s["rows"].shape[0], c["width"], c["out_width"]
    rows = s["rows"].float() * _spread(s["row_scales"], 1, n, width)
    out = torch.zeros(n, out_width, device="cuda", dtype=DTYPES[c["dtype"]])
    for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if b > a:
            w = s["weights"][e].float() * _spread(s["weight_scales"][e], BLOCK, out_width, width)
            out[a:b] = (rows[a:b] @ w.t()).to(out.dtype)
    return {"out": out}


@_full_precision
def _plain_product(s):
    out = torch.zeros(s["rows"].shape[0], s["weights"].shape[1], device="cuda", dtype=s["rows"].dtype)
    got = {"out": out}
    if "grad_out" in s:
        got["grad_rows"] = torch.zeros_like(s["rows"])
        got["grad_weights"] = torch.zeros_like(s["weights"])
    for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if b > a:
            x, w = s["rows"][a:b].float(), s["weights"][e].float()
            out[a:b] = (x @ w.t()).to(out.dtype)
            if "grad_out" in s:
                g = s["grad_out"][a:b].float()
                got["grad_rows"][a:b] = (g @ w).to(out.dtype)
                got["grad_weights"][e] = (g.t() @ x).to(out.dtype)
    return got


PLAIN = {"norm": _plain_norm, "groups": _plain_groups, "quantize": _plain_quantize, "product8": _plain_product8,
         "product": _plain_product}


# ---- this package ----------------------------------------------------------------------------------------------

_package = None


def _run_own(s):
    global _package
    if _package is None:
        import segmented_radix_top_gb300 as _package
    st = _package
    c = s["case"]
    if c["op"] == "norm":
        y, mean, rstd = st.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        out = {"out": y, "mean": mean, "rstd": rstd}
        if c["train"]:
            out["grad_x"], out["grad_weight"], out["grad_bias"] = st.layer_norm_backward(
                s["grad_out"], s["x"], s["weight"], mean, rstd)
        return out
    if c["op"] == "groups":
        ids, weights = st.route(s["logits"], c["k"], score=c["score"], renormalize=c["renormalize"],
                                scale=s["scale"], num_groups=c["num_groups"], groups_kept=c["kept"])
        return {"expert_ids": ids, "weights": weights}
    if c["op"] == "quantize":
        values, scales = st.quantize_rows(s["x"])
        return {"values": values, "scales": scales}
    groups = st.ExpertGroups(*s["groups"])
    if c["op"] == "product8":
        return {"out": st.expert_matmul(s["rows"], s["weights"], groups, row_scales=s["row_scales"],
                                        weight_scales=s["weight_scales"], out_dtype=DTYPES[c["dtype"]])}
    out = {"out": st.expert_matmul(s["rows"], s["weights"], groups)}
    if c["train"]:
        out["grad_rows"], out["grad_weights"] = st.expert_matmul_backward(s["grad_out"], s["rows"], s["weights"],
                                                                          groups)
    return out


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without -----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "norm":
        b, size = BYTES[c["dtype"]], c["tokens"] * c["width"]
        total = 2 * size * b + 2 * c["width"] * b + 8 * c["tokens"]
        if c["train"]:
            total += 2 * size * b + 2 * c["width"] * b  # grad_out, grad_x; weight's and bias's
        return {"bytes": total, "flops": (24.0 if c["train"] else 8.0) * size}
    if c["op"] == "groups":
        size = c["tokens"] * c["experts"]
        return {"bytes": size * BYTES[c["dtype"]] + c["tokens"] * c["k"] * 8, "flops": 4.0 * size}
    if c["op"] == "quantize":
        size = c["tokens"] * c["width"]
        return {"bytes": size * BYTES[c["dtype"]] + size + c["tokens"] * _blocks(c["width"]) * 4, "flops": 3.0 * size}
    rows = c["tokens"] * c["k"] * (0.9 if c["dropped"] else 1.0)
    kept = rows / c["tokens"]
    used = c["experts"] * (1 - (1 - kept / c["experts"]) ** c["tokens"])  # experts with a row
    k, n = c["width"], c["out_width"]
    flops = 2.0 * rows * k * n
    out = c["tokens"] * c["k"] * n * BYTES[c["dtype"]]
    index = (c["experts"] + 1) * 8
    if c["op"] == "product8":
        total = rows * (k + 4 * _blocks(k)) + used * (k * n + 4 * _blocks(k) * _blocks(n)) + out + index
        return {"bytes": total, "flops": flops}
    total = rows * k * 2 + used * k * n * 2 + out + index
    if c["train"]:
        # grad_out, grad_rows and the weights' gradient; rows and weights are read once in all
        total += rows * n * 2 + c["tokens"] * c["k"] * k * 2 + c["experts"] * k * n * 2
        flops *= 3
    return {"bytes": total, "flops": flops}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------

def _exact_norm(s):
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    var, mean = torch.var_mean(x, 1, correction=0)
    rstd = (var + EPS).rsqrt()
    hat = torch.addcmul(-(mean * rstd)[:, None], x, rstd[:, None])
    out = {"out": torch.addcmul(b, hat, w), "mean": mean, "rstd": rstd}
    if "grad_out" in s:
        g = s["grad_out"].double()
        # through the mean and the variance, one after the other
        d_hat = g * w
        d_var = (d_hat * (x - mean[:, None])).sum(1) * -0.5 * rstd**3
        d_mean = -(d_hat.sum(1) * rstd)
        n = x.shape[1]
        out["grad_x"] = d_hat * rstd[:, None] + 2 * (x - mean[:, None]) * (d_var / n)[:, None] + (d_mean / n)[:, None]
        out["grad_weight"] = torch.einsum("tw,tw->w", g, hat)
        out["grad_bias"] = torch.einsum("tw->w", g)
    return out


def _exact_groups(s):
    c = s["case"]
    l = s["logits"].double()
    # a group's and an expert's place: how many are ahead of it
    best = l.view(l.shape[0], c["num_groups"], -1).max(2).values
    low = torch.ones(c["num_groups"], c["num_groups"], device="cuda", dtype=torch.bool).tril(-1)
    ahead = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & low)
    open_ = (ahead.sum(2) < c["kept"]).repeat_interleave(l.shape[1] // c["num_groups"], 1) & (l > -math.inf)
    weights = torch.zeros(l.shape[0], c["k"], device="cuda", dtype=torch.float64)
    left = torch.where(open_, l, -math.inf)
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    for j in range(c["k"]):
        top = left.max(1).values
        at = (left == top[:, None]).double().argmax(1)[:, None]
        weights[:, j] = torch.where(top > -math.inf, score.gather(1, at)[:, 0], 0)
        left.scatter_(1, at, -math.inf)
    if c["renormalize"]:
        total = weights.sum(1, keepdim=True)
        weights = torch.where(total > 0, weights / total, 0)
    return {"expert_ids": None, "weights": weights * s["scale"]}


def _exact_quantize(s):
    x = s["x"].double()
    scales = torch.stack([part.abs().amax(1) for part in x.split(BLOCK, 1)], 1).clamp_(min=SMALLEST) / LARGEST
    # the nearest value with three bits after the leading one (2^-9 apart below 2^-6)
    values = torch.cat([part / scales[:, i:i + 1] for i, part in enumerate(x.split(BLOCK, 1))], 1)
    step = torch.exp2(torch.floor(torch.log2(values.abs().clamp(min=2.0**-6))) - 3)
    return {"values": torch.round(values / step) * step, "scales": scales}


def _exact_product8(s):
    c = s["case"]
    out = torch.zeros(s["rows"].shape[0], c["out_width"], device="cuda", dtype=torch.float64)
    for e in range(c["experts"]):
        a, b = s["bounds"][e:e + 2]
        if a == b:
            continue
        # block by block of the contraction, each with its scales
        for i in range(_blocks(c["width"])):
            at = slice(i * BLOCK, min((i + 1) * BLOCK, c["width"]))
            part = s["rows"][a:b, at].double() @ s["weights"][e, :, at].double().t()
            part *= s["row_scales"][a:b, i:i + 1].double()
            part *= s["weight_scales"][e, :, i].double().repeat_interleave(BLOCK)[:c["out_width"]]
            out[a:b] += part
    return {"out": out}


def _exact_product(s):
    w = s["weights"].double()
    out = torch.zeros(s["rows"].shape[0], w.shape[1], device="cuda", dtype=torch.float64)
    got = {"out": out}
    if s["case"]["train"]:
        got["grad_rows"] = torch.zeros(s["rows"].shape, device="cuda", dtype=torch.float64)
        got["grad_weights"] = torch.zeros_like(w)
    for e in range(len(w)):
        at = slice(*s["bounds"][e:e + 2])
        x = s["rows"][at].double()
        out[at] = torch.einsum("rk,nk->rn", x, w[e])
        if s["case"]["train"]:
            g = s["grad_out"][at].double()
            got["grad_rows"][at] = torch.einsum("rn,nk->rk", g, w[e])
            got["grad_weights"][e] = torch.einsum("rn,rk->nk", g, x)
    return got


EXACT = {"norm": _exact_norm, "groups": _exact_groups, "quantize": _exact_quantize, "product8": _exact_product8,
         "product": _exact_product}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
