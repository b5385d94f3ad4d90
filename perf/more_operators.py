"""Cases and plain forms of the 4-bit weight operators for few tokens with BF16 activations:
the dual-component layer (fused_linear_a16), the choice of experts from a router's logits
(moe_route), the chosen experts' gated products (moe_experts), and both in one call (moe_layer).

Weights are in the layer's packed format: codes in [-7, 7], two to a byte, with one fp32 scale
per output column and 128 elements of the reduction; D() multiplies them out.

    fused_linear_a16  h = bf16(x D(L1))        y = x D(R) + h L2
    moe_route         ids: the k largest logits of a row (ties: the lowest index; a NaN is larger
                      than any number), a logit of -inf is not chosen: id -1, weight 0
                      weights: softmax of the row at these ids, over all logits or over the chosen
    moe_experts       [g u] = x D(R1) + bf16(x D(L11)) L12        a = silu(g) u
                      y_e = a D(R2) + bf16(a D(L21)) L22
                      y = base + sum over a token's slots of weight * y_e
                      (an id outside [0, count) adds nothing)
"""
import math

import torch

own = False

GROUP = 128  # elements of the reduction per scale


def listed():
    return [
        # one token through an attention output projection of rank 128
        dict(name="linear_1", op="linear", b=1, m=4096, n=4096, r=128),
        # a few sequences' decode step, gate/up projection that was packed without low-rank factors
        dict(name="linear_4", op="linear", b=4, m=4096, n=14336, r=0),
        # a full decode batch, down projection of the highest rank
        dict(name="linear_16", op="linear", b=16, m=14336, n=4096, r=256),
        # the largest batch, gate/up of the largest layer, odd number of tokens
        dict(name="linear_61", op="linear", b=61, m=5120, n=25600, r=64),
        # one decode step's choice, fp32 logits
        dict(name="route_1", op="route", b=1, count=128, k=8, bf16=False, renorm=True, masked=0),
        # a prefill batch, BF16 logits (many ties), some experts masked, weights over all experts
        dict(name="route_8192", op="route", b=8192, count=256, k=8, bf16=True, renorm=False, masked=13),
        # one rank's share of the experts: three in four ids are another rank's, residual added
        dict(name="experts_24", op="experts", b=24, m=4096, f=1024, r=32, rd=32, count=32, k=8,
             spread=128, base=True),
        # few large experts, two per token, decode of four sequences
        dict(name="experts_4", op="experts", b=4, m=4096, f=14336, r=0, rd=0, count=8, k=2, spread=8,
             base=False),
        # the smallest layer call: one token, small experts
        dict(name="layer_1", op="layer", b=1, m=2048, f=768, r=0, rd=0, count=128, k=8, bf16=False,
             renorm=True, masked=0, base=True),
        # one token, experts with low-rank factors in both products
        dict(name="layer_lowrank_1", op="layer", b=1, m=2048, f=1024, r=64, rd=64, count=64, k=4,
             bf16=False, renorm=True, masked=0, base=True),
        # a ragged decode batch over many small experts
        dict(name="layer_13", op="layer", b=13, m=2048, f=768, r=16, rd=16, count=128, k=8, bf16=True,
             renorm=True, masked=0, base=True),
        # the largest batch: most experts in use, some by many tokens
        dict(name="layer_64", op="layer", b=64, m=4096, f=1024, r=32, rd=0, count=128, k=8, bf16=False,
             renorm=False, masked=5, base=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "route", "experts", "layer", "layer"])
    if op == "route":
        count = _log_int(rng, 2, 512)
        return dict(op=op, b=_log_int(rng, 1, 8192), count=count, k=rng.randint(1, min(count, 16)),
                    bf16=rng.random() < 0.5, renorm=rng.random() < 0.5,
                    masked=rng.choice([0, 0, count // 3, count - 1]))
    b = _log_int(rng, 1, 64)
    if op == "linear":
        m, n = GROUP * _log_int(rng, 1, 200), GROUP * _log_int(rng, 1, 200)
        while m * n > 5120 * 25600:
            n = GROUP * max(1, n // GROUP // 2)
        return dict(op=op, b=b, m=m, n=n, r=16 * rng.choice([0, 0, 1, 2, 3, 4, 8, 8, 12, 16]))
    count = _log_int(rng, 2, 128)
    k = rng.randint(1, min(count, 8))
    m, f = GROUP * _log_int(rng, 1, 40), GROUP * _log_int(rng, 1, 112)
    while count * m * f > 128 * 4096 * 1024:
        f = GROUP * max(1, f // GROUP // 2)
        count = max(k, count * 3 // 4)
    r, rd = (16 * rng.choice([0, 0, 1, 2, 4, 8]) for _ in range(2))
    case = dict(op=op, b=b, m=m, f=f, r=r, rd=rd, count=count, k=k, base=rng.random() < 0.7)
    if op == "experts":
        case.update(spread=count * rng.choice([1, 1, 2, 4]))
    else:
        case.update(bf16=rng.random() < 0.3, renorm=rng.random() < 0.7,
                    masked=rng.choice([0, 0, count // 4]))
    return case


def _codes(shape, gen, device):
    """Packed codes as Eq. (1) leaves them: bell-shaped, from a table of pairs of codes."""
    c = torch.round(torch.randn((2, 4096), generator=gen, device=device) * 2.3).clamp(-7, 7).to(torch.int32)
    table = ((c[0] & 15) | ((c[1] & 15) << 4)).to(torch.uint8)
    return table[torch.randint(0, 4096, shape, generator=gen, device=device, dtype=torch.int32)]


def _weights(lead, m, n, r, gen, device):
    """Packed weights of `lead` layers (or of one) as a dict of the format's five tensors. Scales
    spread over columns and groups; products keep the size of their inputs."""
    def scales(*shape, std):
        return (0.5 + torch.rand(shape, generator=gen, device=device)) * (std / 2.3)

    return dict(
        m=m, n=n, r=r,
        rq=_codes((*lead, n, m // 2), gen, device), sr=scales(*lead, m // GROUP, n, std=m ** -0.5),
        l1q=_codes((*lead, r, m // 2), gen, device), sl1=scales(*lead, m // GROUP, r, std=m ** -0.5),
        l2t=(torch.randn((*lead, n, r), generator=gen, device=device)
             * (0.4 / max(r, 1) ** 0.5)).to(torch.bfloat16))


def _logits(case, gen, host, device):
    lo = torch.randn((case["b"], case["count"]), generator=gen, device=device) * 1.5
    for _ in range(1 if case["masked"] else 0):
        lo[:, torch.randperm(case["count"], generator=host)[:case["masked"]].to(device)] = -math.inf
    return lo.to(torch.bfloat16) if case["bf16"] else lo


def prepare(case, seed):
    device = torch.device("cuda")
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=device).manual_seed(seed)
    op, b = case["op"], case["b"]
    state = dict(op=op, case=case)
    if op in ("route", "layer"):
        state["logits"] = _logits(case, gen, host, device)
    if op != "route":
        m = case["m"]
        # activations as the layer meets them: 1% of the channels 30 times the others
        hot = torch.ones(m, device=device)
        hot[torch.randperm(m, generator=host)[:max(1, m // 100)].to(device)] = 30.0
        state["x"] = (torch.randn((b, m), generator=gen, device=device) * hot).to(torch.bfloat16)
    if op == "linear":
        state["w"] = _weights((), m, case["n"], case["r"], gen, device)
    elif op != "route":
        f, count, k = case["f"], case["count"], case["k"]
        state["up"] = _weights((count,), m, 2 * f, case["r"], gen, device)
        state["down"] = _weights((count,), f, m, case["rd"], gen, device)
        state["base"] = torch.randn((b, m), generator=gen, device=device).to(torch.bfloat16) if case["base"] else None
    if op == "experts":
        # each token's experts are different ones of `spread`; those from count on are elsewhere
        pick = torch.rand((b, case["spread"]), generator=gen, device=device).argsort(dim=1)[:, :k]
        state["ids"] = pick.to(torch.int32).contiguous()
        state["weights"] = torch.softmax(torch.randn((b, k), generator=gen, device=device), dim=1)
    if own:
        # what a program keeps: views of the packed weights, its buffers
        from rank_residual_w4a4_b200 import twq
        if op in ("route", "layer"):
            state["out"] = dict(ids=torch.empty((b, case["k"]), dtype=torch.int32, device=device),
                                weights=torch.empty((b, case["k"]), dtype=torch.float32, device=device))
        if op == "linear":
            state["packed"] = twq.Weights(**state["w"])
            state["out"] = dict(
                y=torch.empty((b, case["n"]), dtype=torch.bfloat16, device=device),
                h=torch.empty((b, case["r"]), dtype=torch.bfloat16, device=device) if case["r"] else None)
        elif op != "route":
            ex = state["packed"] = twq.Experts(twq.Weights(**state["up"]), twq.Weights(**state["down"]))
            state.setdefault("out", {}).update(
                y=torch.empty((b, m), dtype=torch.bfloat16, device=device),
                workspace=torch.empty(twq.moe_workspace_bytes(b, k, ex), dtype=torch.uint8, device=device))
    return state


def _dequant(q, s):
    """Codes (..., n, m/2) and scales (..., m/128, n) -> fp32 (..., n, m)."""
    c = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).to(torch.int8)
    c = ((c ^ 8) - 8).float().unflatten(-1, (-1, GROUP))
    return (c * s.transpose(-1, -2).unsqueeze(-1)).flatten(-2)


def _product(x, w, at=None):
    """x (..., m) fp32 through the dual-component weights, or through those of the layers `at`."""
    rq, sr, l1q, sl1, l2t = (w[k] if at is None else w[k][at] for k in ("rq", "sr", "l1q", "sl1", "l2t"))
    y = x @ _dequant(rq, sr).transpose(-1, -2)
    if not w["r"]:
        return y
    h = (x @ _dequant(l1q, sl1).transpose(-1, -2)).to(torch.bfloat16).float()
    return y + h @ l2t.float().transpose(-1, -2)


def _plain_route(state):
    case, lo = state["case"], state["logits"].float()
    top = torch.where(lo.isnan(), torch.inf, lo)
    order = torch.sort(top, dim=1, descending=True, stable=True).indices[:, :case["k"]]
    picked = lo.gather(1, order)
    e = torch.exp(picked - top.amax(dim=1, keepdim=True))
    e = torch.where(picked == -torch.inf, 0.0, e)
    over = e if case["renorm"] else torch.exp(lo - top.amax(dim=1, keepdim=True))
    weights = torch.where(picked == -torch.inf, 0.0, e / over.sum(dim=1, keepdim=True))
    return torch.where(picked == -torch.inf, -1, order).to(torch.int32), weights


def _plain_experts(state, ids, weights):
    x, count = state["x"].float(), state["case"]["count"]
    used = torch.unique(ids[(ids >= 0) & (ids < count)]).long()
    p = torch.where(ids[:, :, None] == used[None, None, :], weights[:, :, None], 0.0).sum(dim=1)
    gu = _product(x.expand(used.shape[0], -1, -1), state["up"], used)
    g, u = gu.chunk(2, dim=-1)
    y = _product(g / (1.0 + torch.exp(-g)) * u, state["down"], used)
    y = (y * p.t()[:, :, None]).sum(dim=0)
    if state["base"] is not None:
        y = y + state["base"].float()
    return y.to(torch.bfloat16)


def run(state):
    op, case = state["op"], state["case"]
    if not own:
        if op == "linear":
            return _product(state["x"].float(), state["w"]).to(torch.bfloat16)
        if op == "experts":
            return _plain_experts(state, state["ids"], state["weights"])
        ids, weights = _plain_route(state)
        if op == "route":
            return ids, weights
        return _plain_experts(state, ids, weights), ids, weights
    from rank_residual_w4a4_b200 import twq
    out = state["out"]
    if op == "linear":
        return twq.fused_linear_a16(state["x"], state["packed"], **out)
    if op == "route":
        return twq.moe_route(state["logits"], case["k"], renormalize=case["renorm"], **out)
    if op == "experts":
        return twq.moe_experts(state["x"], state["ids"], state["weights"], state["packed"],
                               base=state["base"], **out)
    return twq.moe_layer(state["x"], state["logits"], case["k"], state["packed"],
                         renormalize=case["renorm"], base=state["base"], **out)


def _weight_bytes(m, n, r):
    return (n * m + r * m) // 2 + 4 * (m // GROUP) * (n + r) + 2 * n * r


def work(case):
    op, b = case["op"], case["b"]
    if op == "linear":
        m, n, r = case["m"], case["n"], case["r"]
        return {"bytes": _weight_bytes(m, n, r) + 2 * b * (m + n), "flops": 2 * b * (m * n + r * (m + n))}
    k, count = case["k"], case["count"]
    if op == "route":
        return {"bytes": b * count * (2 if case["bf16"] else 4) + 8 * b * k, "flops": 0}
    m, f, r, rd = case["m"], case["f"], case["r"], case["rd"]
    # experts in use: as many as different ones that b draws of k of them leave on average
    among = case["spread"] if op == "experts" else count - case["masked"]
    pairs = b * min(k, among) * min(count, among) / among
    used = min(count, among) * (1.0 - (1.0 - min(k, among) / among) ** b)
    one = _weight_bytes(m, 2 * f, r) + _weight_bytes(f, m, rd)
    io = 2 * b * m * (3 if case["base"] else 2) + 8 * b * k
    if op == "layer":
        io += b * count * (2 if case["bf16"] else 4)
    return {"bytes": used * one + io,
            "flops": pairs * 2 * (3 * m * f + r * (m + 2 * f) + rd * (m + f))}


def _exact_weights(w, e):
    """One layer's (R, L1, L2) in 64 bits, R and L1 as (m, n) and (m, r)."""
    def one(q, s):
        q, s = (q, s) if e is None else (q[e], s[e])
        n, half = q.shape
        v = torch.empty((n, 2 * half), dtype=torch.float64, device=q.device)
        lo, hi = (q & 15).double(), (q >> 4).double()
        v[:, 0::2] = torch.where(lo > 7, lo - 16, lo)
        v[:, 1::2] = torch.where(hi > 7, hi - 16, hi)
        return (v * s.double().t().repeat_interleave(GROUP, dim=1)).t()

    l2 = (w["l2t"] if e is None else w["l2t"][e]).double().t()
    return one(w["rq"], w["sr"]), one(w["l1q"], w["sl1"]), l2


def _exact_product(x, w, e=None):
    big, l1, l2 = _exact_weights(w, e)
    y = torch.einsum("im,mn->in", x, big)
    if w["r"]:
        y += torch.einsum("ir,rn->in", torch.einsum("im,mr->ir", x, l1).to(torch.bfloat16).double(), l2)
    return y


def exact(case, seed):
    """The same outputs in 64 bits; experts one by one, each on its own tokens."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_product(s["x"].double(), s["w"])
    if op == "experts":
        ids, weights = s["ids"], s["weights"].double()
    else:
        lo, k = s["logits"].double().cpu(), case["k"]
        ids = torch.full((case["b"], k), -1, dtype=torch.int32)
        weights = torch.zeros((case["b"], k), dtype=torch.float64)
        share = torch.softmax(lo, dim=1)
        # stable sorts of the negated values keep equal ones in the order of their indices
        for i, row in enumerate((-lo).sort(dim=1, stable=True).indices[:, :k].tolist()):
            row = [j for j in row if lo[i, j] != -math.inf]
            ids[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
            p = share[i, row]
            weights[i, :len(row)] = p / p.sum() if case["renorm"] else p
        ids, weights = ids.to(s["logits"].device), weights.to(s["logits"].device)
    if op == "route":
        return ids, weights
    x = s["x"].double()
    y = torch.zeros_like(x) if s["base"] is None else s["base"].double()
    for e in range(case["count"]):
        rows, slots = (ids == e).nonzero(as_tuple=True)
        if not rows.numel():
            continue
        gu = _exact_product(x[rows], s["up"], e)
        g, u = gu[:, :case["f"]], gu[:, case["f"]:]
        y.index_add_(0, rows, _exact_product(torch.sigmoid(g) * g * u, s["down"], e) * weights[rows, slots, None])
    return y if op == "experts" else (y, ids, weights)
