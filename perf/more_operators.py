"""Measured cases of the operators of a layer whose weights have 4 bits, and of
its router:

* ``groups``   a weight rounded to 4-bit floats with a power of two for each 32
  values, and read back;
* ``linear``   activations in bf16, fp16 or fp32 times such a weight;
* ``experts``  the same product with a weight per expert, on rows taken from the
  tokens in the order of their experts;
* ``gate``     the router's choice: the largest of each token's logits and their
  weights; with ``train`` also the gradient of the logits;
* ``balance``  the loss that keeps the experts evenly used and the number of
  choices of each expert, with the gradient of the logits.

``run`` computes the plain form in 32 bits with elementary operations, or,
where ``own`` is true, calls the package's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
GROUP = 32                            # values that share a scale
CODE_BYTES = 0.5 + 1.0 / GROUP        # of a value: its code and its part of the scale


def listed():
    return [
        # A decoded 4096 x 4096 weight laid out for serving.
        dict(name="groups 4096", kind="groups", rows=4096, cols=4096, dtype="f32"),
        # The weights of 16 experts of 1536 x 4096 kept in bf16.
        dict(name="groups experts bf16", kind="groups", rows=24576, cols=4096, dtype="bf16"),
        # One token through a 4096 x 4096 projection: the latency of a decode step.
        dict(name="linear decode 1", kind="linear", tokens=1, channels=4096, depth=4096, dtype="bf16"),
        # A decode batch of 24 sequences through the 5632 x 2048 weight.
        dict(name="linear decode 24", kind="linear", tokens=24, channels=5632, depth=2048, dtype="f16"),
        # A prompt of 4096 tokens through the 4096 x 4096 weight: the largest product.
        dict(name="linear prompt 4096", kind="linear", tokens=4096, channels=4096, depth=4096, dtype="bf16"),
        # A ragged prompt in fp32, an odd number of channels and a depth of 49 groups.
        dict(name="linear ragged f32", kind="linear", tokens=1021, channels=2049, depth=1568, dtype="f32"),
        # Decode batch of 16 sequences, 2 of 16 experts each: a few rows per expert.
        dict(name="experts decode", kind="experts", tokens=16, top_k=2, experts=16, channels=1536,
             depth=4096, skew=0.0, dropped=0.0, dtype="bf16"),
        # Prompt of 4096 tokens over 16 experts that are chosen unevenly.
        dict(name="experts prompt skewed", kind="experts", tokens=4096, top_k=2, experts=16,
             channels=1536, depth=4096, skew=1.0, dropped=0.0, dtype="bf16"),
        # The router of a 4-sequence decode step, 8 of 64 experts: the smallest call.
        dict(name="gate decode 4", kind="gate", tokens=4, experts=64, top_k=8, renormalize=True,
             train=False, padded=0.0, masked=0.0, dtype="f32"),
        # The router of a training step, 8 of 64 experts, forward and gradient.
        dict(name="gate train", kind="gate", tokens=16384, experts=64, top_k=8, renormalize=False,
             train=True, padded=0.0, masked=0.0, dtype="f32"),
        # The loss of a small ragged batch: 3 of 13 experts, padded tokens and a switched-off expert.
        dict(name="balance ragged", kind="balance", tokens=1001, experts=13, top_k=3, padded=0.1,
             masked=0.1, dtype="bf16"),
        # The loss of a large training batch, 8 of 256 experts.
        dict(name="balance train", kind="balance", tokens=65536, experts=256, top_k=8, padded=0.0,
             masked=0.0, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _groups(rng, hi):
    """A number of values: whole groups, mostly of 256 as the codec's blocks are."""
    if rng.random() < 0.5:
        return 256 * rng.randint(1, hi // 256)
    return GROUP * rng.randint(4, hi // GROUP)


def _case(rng):
    kind = rng.choice(["groups", "linear", "linear", "experts", "gate", "gate", "balance"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "groups":
        return dict(kind=kind, rows=_log_int(rng, 1, 24576), cols=_groups(rng, 5632), dtype=dtype)
    if kind == "linear":
        return dict(kind=kind, tokens=_log_int(rng, 1, 8192), channels=_log_int(rng, 256, 5632),
                    depth=_groups(rng, 5632), dtype=dtype)
    if kind == "experts":
        return dict(kind=kind, tokens=_log_int(rng, 1, 4096), top_k=rng.randint(1, 8),
                    experts=rng.choice([8, 13, 16, 32, 64]), channels=_log_int(rng, 256, 2048),
                    depth=_groups(rng, 4096), skew=rng.choice([0.0, 0.5, 1.0]),
                    dropped=rng.choice([0.0, 0.0, 0.1]), dtype=dtype)
    experts = _log_int(rng, 4, 512)
    c = dict(kind=kind, tokens=_log_int(rng, 1, 65536), experts=experts,
             top_k=rng.randint(1, min(10, experts)), padded=rng.choice([0.0, 0.0, 0.1]),
             masked=rng.choice([0.0, 0.0, 0.2]), dtype=rng.choice(["bf16", "f16", "f32", "f32"]))
    if kind == "gate":
        c.update(renormalize=rng.random() < 0.5, train=rng.random() < 0.6)
    return c


def draw(rng):
    most = [work(c) for c in listed()]
    bytes_most = max(w["bytes"] for w in most)
    flops_most = max(w["flops"] for w in most)
    while True:
        c = _case(rng)
        w = work(c)
        if w["bytes"] <= bytes_most and w["flops"] <= flops_most:
            return c


def work(case):
    b = BYTES[case["dtype"]]
    if case["kind"] == "groups":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * b + CODE_BYTES), "flops": 4.0 * n}
    t = case["tokens"]
    if case["kind"] == "linear":
        n, k = case["channels"], case["depth"]
        return {"bytes": t * k * b + n * k * CODE_BYTES + t * n * b, "flops": 2.0 * t * n * k}
    if case["kind"] == "experts":
        n, k, e = case["channels"], case["depth"], case["experts"]
        rows = t * case["top_k"]
        # Experts that some token chooses, as expected of an even choice.
        chosen = e * (1.0 - (1.0 - case["top_k"] / e) ** t)
        return {"bytes": t * k * b + 4 * rows + chosen * n * k * CODE_BYTES + rows * n * b,
                "flops": 2.0 * rows * n * k}
    n, rows = t * case["experts"], t * case["top_k"]
    if case["kind"] == "gate":
        moved = n * b + 8 * rows
        if case["train"]:
            moved += 12 * rows + n * b + (0 if case["renormalize"] else n * b)
        return {"bytes": moved, "flops": (8.0 if case["train"] else 4.0) * n}
    return {"bytes": 3 * n * b + 4 * rows + 8 * case["experts"] + 8, "flops": 10.0 * n}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _uniform(shape, g):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(t, k, dtype, g):
    """Normal values with a scale of its own for each token and a few large channels."""
    x = _normal((t, k), g) * torch.exp(0.5 * _normal((t, 1), g))
    x *= 1.0 + 15.0 * (_uniform((1, k), g) < 0.01)
    return x.to(dtype)


def _weight(rows, cols, g):
    """Weights of a trained layer: normal, rows of different size."""
    return 0.02 * _normal((rows, cols), g) * torch.exp(0.3 * _normal((rows, 1), g))


def _logits(case, g):
    """A router's logits: some experts liked more, some switched off, some tokens padding."""
    t, e = case["tokens"], case["experts"]
    l = (1.5 * _normal((t, e), g) + 0.5 * _normal((1, e), g)).to(DTYPES[case["dtype"]])
    if case["masked"]:
        l.masked_fill_(_uniform((1, e), g) < case["masked"], -math.inf)
    if case["padded"]:
        l.masked_fill_(_uniform((t, 1), g) < case["padded"], -math.inf)
    return l


def prepare(case, seed):
    g = _generator(seed)
    dtype, kind = DTYPES[case["dtype"]], case["kind"]
    s = dict(case, dtype=dtype, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if kind == "groups":
        s["w"] = _weight(case["rows"], case["cols"], g).to(dtype)
        return s
    t = case["tokens"]
    if kind == "linear":
        s["x"] = _activations(t, case["depth"], dtype, g)
        s["w"], s["w_scale"] = _codes(_weight(case["channels"], case["depth"], g))
        return s
    if kind == "experts":
        e, n, k = case["experts"], case["channels"], case["depth"]
        s["x"] = _activations(t, k, dtype, g)
        score = case["skew"] * _normal((1, e), g) - torch.log(-torch.log(_uniform((t, e), g).clamp_(1e-9, 1 - 1e-7)))
        choice = torch.topk(score, case["top_k"], dim=1).indices
        if case["dropped"]:
            choice = torch.where(_uniform(choice.shape, g) < case["dropped"], -1, choice)
        s["order"], s["offsets"] = _sort(choice, e)
        # The longest expert's rows: what a batch padded to equal lengths is sized by.
        s["capacity"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
        s["w"] = torch.empty((e, n, k // 2), dtype=torch.uint8, device="cuda")
        s["w_scale"] = torch.empty((e, n, k // GROUP), dtype=torch.uint8, device="cuda")
        for i in range(e):
            s["w"][i], s["w_scale"][i] = _codes(_weight(n, k, g))
        return s
    s["logits"] = _logits(case, g)
    if kind == "balance":
        s["choice"] = _gate(s["logits"], case["top_k"], True)[0]
        s["loss_grad"] = 0.01 * (1.0 + _uniform((), g))
    elif case["train"]:
        s["weights_grad"] = _normal((t, case["top_k"]), g)
    return s


def _sort(choice, experts):
    """The choices in the order of their experts, ties by place; dropped ones (-1) at the end."""
    flat = choice.reshape(-1)
    key = torch.where(flat < 0, experts, flat)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(experts, device=key.device)).sum(dim=0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return order.to(torch.int32), offsets.to(torch.int32)


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _power(exponent):
    """2^exponent for -127..127, by its bits."""
    return torch.where(exponent < -126, 1 << 22, (exponent + 127) << 23).to(torch.int32).view(torch.float32)


def _codes(w):
    """Codes (two in a byte, the first one low) and scale bytes of a weight: the
    scale 2^(byte - 127) is a quarter of the power of two below the group's largest
    magnitude; a code is a sign and the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6, halves
    to the even code."""
    x = w.float().unflatten(1, (-1, GROUP))
    top = x.abs().amax(dim=2)
    exponent = (torch.frexp(top).exponent - 3).clamp(-127, 127)     # frexp: top < 2^exponent
    v = x.abs() * _power(-exponent)[:, :, None]
    # The lowest value of each code, itself included where the code is even.
    code = ((v > 0.25).int() + (v >= 0.75).int() + (v > 1.25).int() + (v >= 1.75).int()
            + (v > 2.5).int() + (v >= 3.5).int() + (v > 5.0).int())
    code = torch.where(torch.signbit(x), code + 8, code).flatten(1)
    scale = torch.where(top > 0, exponent + 127, 0)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), scale.to(torch.uint8)


def _values(codes, scale):
    """What codes and scale bytes stand for, in fp32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    c = codes.int()
    v = table[torch.stack([c % 16, c // 16], dim=-1).flatten(-2)]
    return (v.unflatten(-1, (-1, GROUP)) * _power(scale.int() - 127)[..., None]).flatten(-2)


def _expert_product(x, w, order, offsets, top_k, capacity):
    """Rows padded to `capacity` for each expert, one batched product, rows taken back."""
    rows = order.numel()
    row = torch.arange(rows, device=x.device)
    expert = (row[:, None] >= offsets[None, 1:]).sum(dim=1)           # == experts where dropped
    place = expert * capacity + (row - offsets.long()[expert])
    e, n, k = w.shape
    padded = torch.zeros((e + 1) * capacity + rows, k, device=x.device)
    padded[place] = x.float()[order.long() // top_k]
    wide = torch.bmm(padded[:e * capacity].view(e, capacity, k), w.transpose(1, 2))
    kept = expert < e
    taken = wide.view(e * capacity, n)[torch.where(kept, place, 0)]
    return torch.where(kept[:, None], taken, 0.0)


def _softmax(l):
    """Rows of probabilities; zeros where a row has no finite logit."""
    top = l.amax(dim=1, keepdim=True)
    live = top > -math.inf
    e = torch.where(live, torch.exp(l - torch.where(live, top, 0.0)), 0.0)
    return e / torch.where(live, e.sum(dim=1, keepdim=True), 1.0), live


def _gate(logits, top_k, renormalize):
    """The largest logits' experts, the lowest first where they are equal, and their
    weights; -1 and 0 where no finite logit is left."""
    l = logits.float()
    top, choice = torch.sort(l, dim=1, descending=True, stable=True)
    kept = top[:, :top_k] > -math.inf
    choice = choice[:, :top_k]
    p = torch.where(kept, torch.gather(_softmax(l)[0], 1, choice), 0.0)
    if renormalize:
        p = torch.where(kept, p / p.sum(dim=1, keepdim=True), 0.0)
    return torch.where(kept, choice, -1).to(torch.int32), p


def _gate_grad(grad, logits, choice, weights, renormalize):
    kept = choice >= 0
    gw = grad * weights
    total = gw.sum(dim=1, keepdim=True)
    own_part = gw - weights * total if renormalize else gw
    out = torch.zeros(logits.shape, device=logits.device)
    out.scatter_add_(1, torch.where(kept, choice, 0).long(), torch.where(kept, own_part, 0.0))
    return out if renormalize else out - _softmax(logits.float())[0] * total


def _balance(logits, choice, loss_grad):
    """(loss, counts, tokens that count, gradient of the logits)."""
    experts = logits.shape[1]
    p, live = _softmax(logits.float())
    counts = torch.zeros(experts + 1, dtype=torch.int32, device=choice.device)
    flat = torch.where(choice < 0, experts, choice).reshape(-1).long()
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    counts = counts[:experts]
    tokens = live.sum().to(torch.int32)
    share = counts.double() / counts.sum().clamp(min=1)
    mean = p.double().sum(dim=0) / tokens.clamp(min=1)
    loss = (experts * (share * mean).sum()).float()
    share = share.float()
    inner = share - (p * share).sum(dim=1, keepdim=True)
    grad = p * inner * (loss_grad * experts / tokens.clamp(min=1))
    return loss, counts, tokens, grad


def _plain(s):
    kind, dtype = s["kind"], s["dtype"]
    if kind == "groups":
        return _values(*_codes(s["w"])).to(dtype)
    if kind == "linear":
        return (s["x"].float() @ _values(s["w"], s["w_scale"]).T).to(dtype)
    if kind == "experts":
        return _expert_product(s["x"], _values(s["w"], s["w_scale"]), s["order"], s["offsets"],
                               s["top_k"], s["capacity"]).to(dtype)
    if kind == "gate":
        choice, weights = _gate(s["logits"], s["top_k"], s["renormalize"])
        r = {"choice": choice, "weights": weights}
        if s["train"]:
            r["logits_grad"] = _gate_grad(s["weights_grad"], s["logits"], choice, weights,
                                          s["renormalize"]).to(dtype)
        return r
    loss, counts, tokens, grad = _balance(s["logits"], s["choice"], s["loss_grad"])
    return {"loss": loss, "counts": counts, "tokens": tokens, "logits_grad": grad.to(dtype)}


# ---------------------------------------------------------------------------
# The package's entry points
# ---------------------------------------------------------------------------

def _own(s):
    import ggml_iq_codebook_amd as iq

    kind, report = s["kind"], {"status": s["status"], "check": False}
    if kind == "groups":
        codes, scale = iq.quantize_groups(s["w"], **report)
        return iq.dequantize_groups(codes, scale, dtype=s["dtype"])
    if kind == "linear":
        return iq.fp4_linear(s["x"], s["w"], s["w_scale"])
    if kind == "experts":
        return iq.fp4_expert_linear(s["x"], s["w"], s["w_scale"], s["offsets"], s["order"],
                                    top_k=s["top_k"])
    if kind == "gate":
        choice, weights = iq.expert_gate(s["logits"], s["top_k"], renormalize=s["renormalize"], **report)
        r = {"choice": choice, "weights": weights}
        if s["train"]:
            r["logits_grad"] = iq.expert_gate_backward(s["weights_grad"], s["logits"], choice, weights,
                                                       renormalize=s["renormalize"])
        return r
    loss, counts, tokens = iq.expert_balance(s["logits"], s["choice"], **report)
    grad = iq.expert_balance_backward(s["loss_grad"], s["logits"], counts, tokens)
    return {"loss": loss, "counts": counts, "tokens": tokens, "logits_grad": grad}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _two64(exponent):
    """2^exponent in 64 bits, exactly."""
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _decoded64(codes, scale):
    """Sign, two bits of exponent and one of mantissa, times the group's power of two."""
    c = codes.long()
    c = torch.stack((c & 15, c >> 4), dim=-1).reshape(*codes.shape[:-1], -1)
    exponent, mantissa = (c >> 1) & 3, (c & 1).double()
    size = torch.where(exponent == 0, 0.5 * mantissa, (1.0 + 0.5 * mantissa) * _two64(exponent - 1))
    group = _two64(scale.long() - 127).repeat_interleave(GROUP, dim=-1)
    return torch.where(c >= 8, -size, size) * group


def _rounded64(w):
    """Each value replaced by the nearest that its group can hold."""
    x = w.double().reshape(w.shape[0], -1, GROUP)
    top = x.abs().max(dim=2, keepdim=True).values
    step = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    # log2 may have rounded to a whole number from below, or to less than one.
    step = torch.where(_two64(step) > top, step - 1, step)
    step = torch.where(_two64(step + 1) <= top, step + 1, step)
    unit = _two64((step - 2).clamp(-127, 127))
    size = x.abs() / unit
    # Halves of 1 up to 2, steps of 1 up to 4, of 2 above; torch rounds halves to even.
    near = torch.where(size < 2.0, torch.round(size * 2) / 2,
                       torch.where(size < 4.0, torch.round(size), torch.round(size / 2) * 2))
    return (torch.sign(x) * near.clamp(max=6.0) * unit).reshape(w.shape)


def _rows64(l):
    """Probabilities of each row, zeros where every logit is -inf."""
    p = torch.softmax(l.double(), dim=1)
    return torch.where(torch.isfinite(l).any(dim=1, keepdim=True), p, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "groups":
        return _rounded64(s["w"])
    if kind == "linear":
        return torch.matmul(s["x"].double(), _decoded64(s["w"], s["w_scale"]).T)
    if kind == "experts":
        order, ends = s["order"].long(), s["offsets"].tolist()
        y = torch.zeros((order.numel(), case["channels"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            if ends[e + 1] > ends[e]:
                token = torch.div(order[ends[e]:ends[e + 1]], s["top_k"], rounding_mode="floor")
                y[ends[e]:ends[e + 1]] = torch.matmul(s["x"][token].double(),
                                                      _decoded64(s["w"][e], s["w_scale"][e]).T)
        return y
    p = _rows64(s["logits"])
    if kind == "gate":
        k = s["top_k"]
        # Ranks by counting who goes before: larger, or equal and of a lower index.
        best = torch.argsort(-s["logits"].double(), dim=1, stable=True)[:, :k]
        pick = torch.zeros_like(p).scatter_(1, best, 1.0) * torch.isfinite(s["logits"])
        norm = (p * pick).sum(dim=1, keepdim=True) if s["renormalize"] else 1.0
        dense = torch.where(pick > 0, p / norm, 0.0)
        r = {"choice": None, "weights": torch.gather(dense, 1, best)}
        if s["train"]:
            g = torch.zeros_like(p).scatter_(1, best, s["weights_grad"].double()) * pick
            total = (g * dense).sum(dim=1, keepdim=True)
            r["logits_grad"] = dense * (g - total) if s["renormalize"] else p * (g - total)
        return r
    e, live = case["experts"], torch.isfinite(s["logits"]).any(dim=1)
    counts = torch.stack([(s["choice"] == i).sum() for i in range(e)]).double()
    share = counts / max(1.0, float(counts.sum()))
    factor = e / max(1, int(live.sum()))
    grad = p * (share - torch.matmul(p, share)[:, None]) * (s["loss_grad"].double() * factor)
    return {"loss": (p.sum(dim=0) * share).sum() * factor, "counts": None, "tokens": None, "logits_grad": grad}
