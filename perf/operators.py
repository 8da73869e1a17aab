"""Measured cases of the operators that run a layer on decoded weights: the
8-bit product with a scale per token and per channel, the same product by
expert, and the routing of tokens to experts and back with its gradients.

Each case is real work of one of four paths:

* ``linear``  activations in bf16, fp16 or fp32 are rounded to 8-bit integers
  with one scale per token and multiplied with an 8-bit weight that has one
  scale per output channel (what a served layer does);
* ``product`` the product alone, on activations that are already 8-bit;
* ``experts`` the product by expert: rows taken from the tokens in the order
  of their experts, each expert with its own weight;
* ``layer``   a served expert layer from the router's choice to the weighted
  sum over each token's experts;
* ``route``   tokens sorted by expert, copied there, brought back with the
  router's weights; with ``train`` also the gradients of both copies.

``run`` computes the plain form in 32 bits with elementary operations, or,
where ``own`` is true, calls the package's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # One token through a 4096 x 4096 projection: the latency of a decode step.
        dict(name="linear decode 1", kind="linear", tokens=1, channels=4096, depth=4096, dtype="bf16"),
        # A decode batch of 24 sequences on one 1536 x 4096 weight.
        dict(name="linear decode 24", kind="linear", tokens=24, channels=1536, depth=4096, dtype="f16"),
        # A prompt of 4096 tokens through the 4096 x 4096 weight.
        dict(name="linear prompt 4096", kind="linear", tokens=4096, channels=4096, depth=4096, dtype="bf16"),
        # A ragged prompt in fp32 through the 5632 x 2048 weight.
        dict(name="linear ragged f32", kind="linear", tokens=1021, channels=5632, depth=2048, dtype="f32"),
        # Mid-sized ragged product with an odd number of channels (a pruned head).
        dict(name="product odd", kind="product", tokens=197, channels=2049, depth=1536, dtype="bf16"),
        # Calibration-sized batch: the largest product.
        dict(name="product 16384", kind="product", tokens=16384, channels=4096, depth=4096, dtype="f16"),
        # Decode batch of 16 sequences, 2 of 16 experts each: a few rows per expert.
        dict(name="experts decode", kind="experts", tokens=16, top_k=2, experts=16, channels=1536,
             depth=4096, skew=0.0, dropped=0.0, dtype="bf16"),
        # Prompt of 4096 tokens over 16 experts that are chosen unevenly.
        dict(name="experts prompt skewed", kind="experts", tokens=4096, top_k=2, experts=16,
             channels=1536, depth=4096, skew=1.0, dropped=0.0, dtype="bf16"),
        # A whole served expert layer on a medium batch.
        dict(name="layer 512", kind="layer", tokens=512, top_k=2, experts=16, channels=1536,
             depth=4096, skew=0.5, dropped=0.0, dtype="bf16"),
        # Routing of a 4-sequence decode step: latency of the smallest calls.
        dict(name="route decode 4", kind="route", tokens=4, top_k=2, experts=16, width=4096,
             skew=0.0, dropped=0.0, train=False, dtype="bf16"),
        # A training step's routing, 8 of 64 experts: forward and gradients.
        dict(name="route train", kind="route", tokens=4096, top_k=8, experts=64, width=4096,
             skew=0.5, dropped=0.0, train=True, dtype="bf16"),
        # Odd sizes with dropped choices (a router with a capacity limit), fp32.
        dict(name="route train ragged", kind="route", tokens=1001, top_k=3, experts=13, width=1535,
             skew=1.0, dropped=0.1, train=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _depth(rng):
    # Weights decoded from 256-value blocks have depths that are multiples of
    # 256; products of other 8-bit weights have any depth.
    if rng.random() < 0.75:
        return 256 * rng.randint(1, 22)
    return rng.randint(100, 5632)


def _case(rng):
    kind = rng.choice(["linear", "linear", "product", "experts", "layer", "route", "route"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    tokens = _log_int(rng, 1, 16384)
    if kind in ("linear", "product"):
        return dict(kind=kind, tokens=tokens, channels=_log_int(rng, 256, 5632), depth=_depth(rng),
                    dtype=dtype)
    routing = dict(tokens=_log_int(rng, 1, 8192), experts=rng.choice([8, 13, 16, 32, 64]),
                   top_k=rng.randint(1, 8), skew=rng.choice([0.0, 0.5, 1.0]),
                   dropped=rng.choice([0.0, 0.0, 0.1]))
    if kind == "route":
        return dict(kind=kind, width=rng.randint(128, 4096), train=rng.random() < 0.6, dtype=dtype,
                    **routing)
    return dict(kind=kind, channels=_log_int(rng, 256, 2048), depth=_depth(rng), dtype=dtype,
                **routing)


def draw(rng):
    most = [work(c) for c in listed()]
    bytes_most = max(w["bytes"] for w in most)
    flops_most = max(w["flops"] for w in most)
    while True:
        c = _case(rng)
        w = work(c)
        if w["bytes"] <= bytes_most and w["flops"] <= flops_most / 4 * (4 if c["kind"] == "product" else 1):
            return c


def work(case):
    b, t = BYTES[case["dtype"]], case["tokens"]
    if case["kind"] in ("linear", "product"):
        n, k = case["channels"], case["depth"]
        x = t * k * b if case["kind"] == "linear" else t * (k + 4)
        return {"bytes": x + n * (k + 4) + t * n * b, "flops": 2.0 * t * n * k}
    rows = t * case["top_k"]
    if case["kind"] == "route":
        d = case["width"]
        moved = t * d + rows * d + rows * d + t * d               # dispatch, combine
        if case["train"]:
            moved += t * d + 2 * rows * d + rows * d + t * d      # their gradients
        small = rows * (4 + 4 + 4 + (4 if case["train"] else 0)) + 4 * (case["experts"] + 1)
        return {"bytes": moved * b + small,
                "flops": rows * d * (2.0 + (4.0 if case["train"] else 0.0))}
    n, k = case["channels"], case["depth"]
    # Experts that some token chooses, as expected of an even choice.
    e = case["experts"]
    weights = e * (1.0 - (1.0 - case["top_k"] / e) ** t) * n * (k + 4)
    if case["kind"] == "experts":
        return {"bytes": t * (k + 4) + 4 * rows + weights + rows * n * b, "flops": 2.0 * rows * n * k}
    return {"bytes": t * k * b + 8 * rows + weights + t * n * b,
            "flops": 2.0 * rows * n * k + 2.0 * rows * n}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(t, k, dtype, g):
    """Normal values with a scale of its own for each token and a few large channels."""
    x = _normal((t, k), g) * torch.exp(0.5 * _normal((t, 1), g))
    x *= 1.0 + 15.0 * (torch.rand((1, k), generator=g, device="cuda") < 0.01)
    return x.to(dtype)


def _codes(x):
    """8-bit codes and scale of each row (the last axis)."""
    scale = x.abs().amax(dim=-1) / 127.0
    return torch.round(x / scale[..., None]).clamp_(-127, 127).to(torch.int8), scale


def _weight(shape, g):
    return _codes(0.02 * _normal(shape, g))


def _routing(case, g):
    """The router's choice: distinct experts for each token and their normalised weights."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    liking = case["skew"] * _normal((1, e), g)
    score = liking - torch.log(-torch.log(torch.rand((t, e), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    top, choice = torch.topk(score, k, dim=1)
    weights = torch.softmax(top, dim=1)
    if case["dropped"]:
        choice = torch.where(torch.rand((t, k), generator=g, device="cuda") < case["dropped"], -1, choice)
    return choice.to(torch.int32), weights


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"kind": case["kind"], "dtype": dtype, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    kind, t = case["kind"], case["tokens"]
    if kind in ("linear", "product"):
        s["w"], s["w_scale"] = _weight((case["channels"], case["depth"]), g)
        x = _activations(t, case["depth"], dtype, g)
        if kind == "linear":
            s["x"] = x
        else:
            s["x"], s["x_scale"] = _codes(x.float())
        return s
    s["top_k"], s["experts"] = case["top_k"], case["experts"]
    s["choice"], s["weights"] = _routing(case, g)
    if kind == "route":
        d, rows = case["width"], t * case["top_k"]
        s["train"] = case["train"]
        s["x"] = _activations(t, d, dtype, g)
        s["y"] = _normal((rows, d), g).to(dtype)          # what the experts answer, in their order
        if case["train"]:
            s["out_grad"] = _normal((t, d), g).to(dtype)
            s["x_sorted_grad"] = _normal((rows, d), g).to(dtype)
        return s
    # A weight for each expert, drawn one after another to stay small.
    e, n, k = case["experts"], case["channels"], case["depth"]
    s["w"] = torch.empty((e, n, k), dtype=torch.int8, device="cuda")
    s["w_scale"] = torch.empty((e, n), dtype=torch.float32, device="cuda")
    for i in range(e):
        s["w"][i], s["w_scale"][i] = _weight((n, k), g)
    x = _activations(t, k, dtype, g)
    order, position, offsets = _sort(s["choice"], e)
    # The longest expert's rows: what a batch padded to equal lengths is sized by.
    s["capacity"] = max(1, int((offsets[1:] - offsets[:-1]).max()))
    if kind == "layer":
        s["x"] = x
    else:
        s["x"], s["x_scale"] = _codes(x.float())
        s["order"], s["offsets"] = order, offsets
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _sort(choice, experts):
    """The choices in the order of their experts, ties by place; dropped ones (-1) at the end."""
    flat = choice.reshape(-1)
    key = torch.where(flat < 0, experts, flat)
    order = torch.argsort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=order.device)
    counts = (key[:, None] == torch.arange(experts, device=key.device)).sum(dim=0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return order.to(torch.int32), position.to(torch.int32).reshape(choice.shape), offsets.to(torch.int32)


def _product(x, x_scale, w, w_scale):
    return (x.float() @ w.float().T) * x_scale[:, None] * w_scale


def _expert_product(x, x_scale, w, w_scale, order, offsets, top_k, capacity):
    """Rows padded to `capacity` for each expert, one batched product, rows taken back."""
    rows = order.numel()
    row = torch.arange(rows, device=x.device)
    expert = (row[:, None] >= offsets[None, 1:]).sum(dim=1)           # == experts where dropped
    place = expert * capacity + (row - offsets.long()[expert])
    token = order.long() // top_k
    e, n, k = w.shape
    padded = torch.zeros((e + 1) * capacity + rows, k, device=x.device)
    padded[place] = x.float()[token]
    wide = torch.bmm(padded[:e * capacity].view(e, capacity, k), w.float().transpose(1, 2))
    kept = expert < e
    taken = wide.view(e * capacity, n)[torch.where(kept, place, 0)]
    scale = x_scale[token][:, None] * w_scale[torch.where(kept, expert, 0)]
    return torch.where(kept[:, None], taken * scale, 0.0)


def _dispatch(x, order, offsets, top_k):
    kept = torch.arange(order.numel(), device=x.device) < offsets[-1]
    return torch.where(kept[:, None], x[order.long() // top_k], 0.0)


def _combine(y, position, offsets, weights):
    kept = position < offsets[-1]
    rows = torch.where(kept[:, :, None], y[position.long()].float(), 0.0)
    return (rows * weights[:, :, None]).sum(dim=1)


def _combine_grad(grad, y, position, offsets, weights):
    kept = (position < offsets[-1])[:, :, None]
    at = position.long()
    g = grad.float()[:, None, :]
    y_grad = torch.zeros(y.shape, device=y.device)
    y_grad[at.reshape(-1)] = torch.where(kept, g * weights[:, :, None], 0.0).reshape(y.shape)
    return y_grad, torch.where(kept, g * y[at].float(), 0.0).sum(dim=2)


def _plain(s):
    kind, dtype = s["kind"], s["dtype"]
    if kind == "linear":
        q, scale = _codes(s["x"].float())
        return _product(q, scale, s["w"], s["w_scale"]).to(dtype)
    if kind == "product":
        return _product(s["x"], s["x_scale"], s["w"], s["w_scale"]).to(dtype)
    if kind == "experts":
        return _expert_product(s["x"], s["x_scale"], s["w"], s["w_scale"], s["order"], s["offsets"],
                               s["top_k"], s["capacity"]).to(dtype)
    order, position, offsets = _sort(s["choice"], s["experts"])
    if kind == "layer":
        q, scale = _codes(s["x"].float())
        y = _expert_product(q, scale, s["w"], s["w_scale"], order, offsets, s["top_k"], s["capacity"])
        return _combine(y.to(dtype), position, offsets, s["weights"]).to(dtype)
    r = {"order": order, "position": position, "offsets": offsets,
         "x_sorted": _dispatch(s["x"], order, offsets, s["top_k"]),
         "out": _combine(s["y"], position, offsets, s["weights"]).to(dtype)}
    if s["train"]:
        y_grad, r["weights_grad"] = _combine_grad(s["out_grad"], s["y"], position, offsets, s["weights"])
        r["y_grad"] = y_grad.to(dtype)
        r["x_grad"] = _combine(s["x_sorted_grad"], position, offsets,
                               torch.ones_like(s["weights"])).to(dtype)
    return r


# ---------------------------------------------------------------------------
# The package's entry points
# ---------------------------------------------------------------------------

def _own(s):
    import ggml_iq_codebook_amd as iq

    kind, dtype = s["kind"], s["dtype"]
    report = {"status": s["status"], "check": False}
    if kind == "linear":
        return iq.int8_linear(s["x"], s["w"], s["w_scale"], **report)
    if kind == "product":
        return iq.int8_matmul(s["x"], s["x_scale"], s["w"], s["w_scale"], dtype=dtype)
    if kind == "experts":
        return iq.int8_expert_matmul(s["x"], s["x_scale"], s["w"], s["w_scale"], s["offsets"],
                                     s["order"], top_k=s["top_k"], dtype=dtype)
    order, position, offsets = iq.expert_sort(s["choice"], s["experts"], **report)
    if kind == "layer":
        q, scale = iq.quantize_rows(s["x"], **report)
        y = iq.int8_expert_matmul(q, scale, s["w"], s["w_scale"], offsets, order, top_k=s["top_k"],
                                  dtype=dtype)
        return iq.expert_combine(y, position, offsets, s["weights"])
    r = {"order": order, "position": position, "offsets": offsets,
         "x_sorted": iq.expert_dispatch(s["x"], position, offsets),
         "out": iq.expert_combine(s["y"], position, offsets, s["weights"])}
    if s["train"]:
        r["y_grad"], r["weights_grad"] = iq.expert_combine_backward(s["out_grad"], s["y"], position,
                                                                    offsets, s["weights"])
        r["x_grad"] = iq.expert_dispatch_backward(s["x_sorted_grad"], position, offsets)
    return r


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _codes64(x):
    """code = the integer nearest to x * 127 / max|row|, scale = max|row| / 127."""
    x = x.double()
    top = x.abs().max(dim=1, keepdim=True).values
    return torch.round(x / (top / 127.0)), top / 127.0


def _rows64(x, x_scale, s, experts):
    """y[t, j] = the product of token t with the weight of its j-th expert, expert by expert."""
    t, k = s["choice"].shape
    y = torch.zeros((t, k, s["w"].shape[1]), dtype=torch.float64, device=x.device)
    for e in range(experts):
        token, slot = torch.nonzero(s["choice"] == e, as_tuple=True)
        if token.numel():
            w = s["w"][e].double() * s["w_scale"][e].double()[:, None]
            y[token, slot] = torch.matmul(x[token] * x_scale[token], w.T)
    return y


def _by_expert(choice):
    """Place of each choice when they are counted expert by expert, and whether it is kept."""
    flat = choice.reshape(-1).cpu().tolist()
    places = sorted(range(len(flat)), key=lambda i: (flat[i] if flat[i] >= 0 else 1 << 30, i))
    return torch.tensor(places, device=choice.device), choice.reshape(-1) >= 0


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "linear":
        q, scale = _codes64(s["x"])
        return torch.matmul(q * scale, (s["w"].double() * s["w_scale"].double()[:, None]).T)
    if kind == "product":
        return torch.matmul(s["x"].double() * s["x_scale"].double()[:, None],
                            (s["w"].double() * s["w_scale"].double()[:, None]).T)
    places, kept = _by_expert(s["choice"])
    if kind == "experts":
        y = _rows64(s["x"].double(), s["x_scale"].double()[:, None], s, case["experts"])
        return y.reshape(-1, y.shape[2])[places]
    t, k = s["choice"].shape
    keep = kept.view(t, k, 1).double()
    weight = s["weights"].double()[:, :, None]
    if kind == "layer":
        q, scale = _codes64(s["x"])
        return (_rows64(q, scale, s, case["experts"]) * weight).sum(dim=1)
    back = torch.empty_like(places)
    back[places] = torch.arange(places.numel(), device=places.device)
    y = s["y"].double()[back].view(t, k, -1)
    r = {"order": None, "position": None, "offsets": None,
         "x_sorted": (s["x"].double()[:, None, :] * keep).expand(t, k, -1).reshape(t * k, -1)[places],
         "out": (y * keep * weight).sum(dim=1)}
    if case["train"]:
        g = s["out_grad"].double()[:, None, :] * keep
        r["weights_grad"] = (g * y).sum(dim=2)
        r["y_grad"] = (g * weight).reshape(t * k, -1)[places]
        r["x_grad"] = (s["x_sorted_grad"].double()[back].view(t, k, -1) * keep).sum(dim=1)
    return r
