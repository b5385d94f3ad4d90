"""Cases and plain forms of the low-rank adapter operators: rows grouped by adapter
(group_rows), the adapters of many requests beside the shared layer (adapter_linear)
and their gradients (adapter_backward), on BF16 activations and on 8-bit codes.

Row i of a batch uses adapter ids[i] in [0, count), or none (-1). With A (r x m),
B (n x r) and the fp32 factor s of that adapter:

    adapter_linear    h = x A^T               y = base + s h B^T
    adapter_backward  dh = s dy B             dx = dx_base + dh A
                      dA = sum over rows of dh^T x,  dB = sum of s dy^T h

A row without an adapter has h = 0, y = base, dx = dx_base; an adapter without rows has
zero gradients. X is BF16, or int8 codes with one fp32 scale per row and 128 columns.
"""
import math

import torch

own = False

GROUP = 128  # columns per activation scale


def listed():
    return [
        # one decode step of a server: 48 sequences, each with its own request's adapter
        dict(name="group_decode", op="group", b=48, count=32, used=20, plain=4, order="mixed"),
        # a large prefill batch: rows of a request stand together, some without an adapter
        dict(name="group_prefill", op="group", b=16384, count=64, used=40, plain=1024, order="runs"),
        # the smallest call: one token of one request, attention output projection
        dict(name="decode_1", op="linear", b=1, m=4096, n=4096, r=16, count=8, used=1, plain=0,
             order="mixed", codes=False),
        # decode of a full batch with many adapters in flight, gate/up projection
        dict(name="decode_48", op="linear", b=48, m=4096, n=14336, r=16, count=32, used=20, plain=4,
             order="mixed", codes=False),
        # a ragged mixed step: a few short prompts and decode rows, odd batch, odd rank
        dict(name="mixed_333", op="linear", b=333, m=5120, n=5120, r=24, count=16, used=11, plain=17,
             order="runs", codes=False),
        # prefill of the gate/up projection, four prompts
        dict(name="prefill_2048", op="linear", b=2048, m=4096, n=14336, r=32, count=8, used=4,
             plain=0, order="runs", codes=False),
        # prefill of the down projection on the 8-bit codes that the layer itself reads
        dict(name="prefill_codes", op="linear", b=4096, m=14336, n=4096, r=16, count=8, used=6,
             plain=100, order="runs", codes=True),
        # the largest prefill: MLP of a large model, high rank
        dict(name="prefill_8192", op="linear", b=8192, m=5120, n=25600, r=64, count=4, used=4,
             plain=0, order="runs", codes=False),
        # a small training step: short sequences, three adapters of which one has no rows
        dict(name="train_257", op="backward", b=257, m=512, n=512, r=8, count=3, used=2, plain=9,
             order="runs", codes=False),
        # fine-tuning of one adapter on an attention projection
        dict(name="train_4096", op="backward", b=4096, m=4096, n=4096, r=16, count=1, used=1, plain=0,
             order="runs", codes=False),
        # several adapters trained together from 8-bit checkpoints of X, gate/up projection
        dict(name="train_codes", op="backward", b=8192, m=4096, n=14336, r=32, count=6, used=5,
             plain=0, order="mixed", codes=True),
        # the largest training step, high rank
        dict(name="train_8192", op="backward", b=8192, m=5120, n=25600, r=64, count=4, used=4, plain=0,
             order="runs", codes=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["group", "linear", "linear", "backward", "backward"])
    count = _log_int(rng, 1, 64)
    if op == "group":
        b = _log_int(rng, 1, 16384)
        case = dict(op=op, b=b, count=count)
    else:
        m = GROUP * _log_int(rng, 2, 112)
        n = GROUP * _log_int(rng, 2, 112)
        r = 8 * rng.choice([1, 1, 2, 2, 3, 4, 4, 6, 8, 8, 12, 16])
        b = _log_int(rng, 1 if op == "linear" else 64, 8192)
        while r * (m + n) * count > 1 << 25:  # the bank and its gradients stay small beside X and Y
            count //= 2
        while b * (6 * m + 4 * n) > 8192 * (6 * 5120 + 4 * 25600) or b * r > 8192 * 64:
            b //= 2
        case = dict(op=op, b=b, m=m, n=n, r=r, count=count, codes=rng.random() < 0.4)
    plain = rng.choice([0, 0, b // 16, b // 4])
    used = rng.randint(1, count)
    case.update(used=min(used, b - plain), plain=plain, order=rng.choice(["runs", "mixed"]))
    return case


def _ids(case, gen, device):
    """ids of b rows: `used` adapters of `count`, each on one row at least, `plain` rows
    with none; a request's rows stand together ("runs") or anywhere ("mixed")."""
    b, used, rows = case["b"], case["used"], case["b"] - case["plain"]
    which = torch.randperm(case["count"], generator=gen)[:used]
    cuts = torch.randperm(rows - 1, generator=gen)[:used - 1].sort().values + 1
    seg = torch.zeros(rows, dtype=torch.int64)
    seg[cuts] = 1
    ids = torch.full((b,), -1, dtype=torch.int32)
    ids[:rows] = which[seg.cumsum(0)].to(torch.int32)
    if case["order"] == "mixed":
        ids = ids[torch.randperm(b, generator=gen)]
    return ids.to(device)


def prepare(case, seed):
    device = torch.device("cuda")
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=device).manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape, std):
        return (torch.randn(shape, generator=gen, device=device) * std).to(bf16)

    ids = _ids(case, host, device)
    state = dict(op=case["op"], ids=ids, count=case["count"])
    if own:
        from rank_residual_w4a4_b200 import twq
    if case["op"] == "group":
        return state
    b, m, n, r, count = (case[k] for k in ("b", "m", "n", "r", "count"))
    codes = case["codes"]
    # activations as the layer meets them: 1% of the channels 30 times the others
    hot = torch.ones(m, device=device)
    hot[torch.randperm(m, generator=host)[:max(1, m // 100)].to(device)] = 30.0
    x = (torch.randn((b, m), generator=gen, device=device) * hot).to(bf16)
    if codes:  # what quantize_act_a8 leaves: s = max|x| / 127, code = round(x / s)
        g = x.float().view(b, m // GROUP, GROUP)
        s = g.abs().amax(dim=2, keepdim=True) / 127.0
        state["xq8"] = torch.round(g / s).clamp(-127, 127).to(torch.int8).view(b, m)
        state["sx"] = s.view(b, m // GROUP).contiguous()
    else:
        state["x"] = x
    state["a"] = normal(count, r, m, std=m ** -0.5)
    state["b"] = normal(count, n, r, std=0.02)
    # alpha / rank, not the same for every adapter
    state["scale"] = 2.0 / (1.0 + torch.arange(count, device=device, dtype=torch.float32) % 3)
    if case["op"] == "linear":
        state["base"] = normal(b, n, std=3.0)
    else:
        state["dy"] = normal(b, n, std=0.01)
        state["dx_base"] = normal(b, m, std=0.01)
        state["h"] = normal(b, r, std=3.0)  # kept from the forward pass
    if own:
        # what a program keeps: the bank's view, the grouping of this batch, its buffers
        state["adapters"] = twq.Adapters(state["a"], state["b"], state["scale"])
        state["groups"] = twq.group_rows(ids, count)
        if case["op"] == "linear":
            state["out"] = dict(y=torch.empty_like(state["base"]),
                                h=torch.empty((b, r), dtype=bf16, device=device))
        else:
            state["out"] = dict(
                dx=torch.empty_like(state["dx_base"]), da=torch.empty_like(state["a"]),
                db=torch.empty_like(state["b"]),
                workspace=torch.empty(twq.adapter_backward_workspace_bytes(b, m, n, r, count),
                                      dtype=torch.uint8, device=device))
    else:
        # the same knowledge for the plain form: the rows of each adapter that has any
        cpu = ids.cpu()
        state["rows"] = [(int(k), (cpu == k).nonzero().flatten().to(device))
                         for k in cpu.unique().tolist() if k >= 0]
    return state


def _x32(state, rows):
    if "x" in state:
        return state["x"][rows].float()
    q, s = state["xq8"][rows].float(), state["sx"][rows]
    return (q.view(q.shape[0], -1, GROUP) * s[:, :, None]).view(q.shape)


def _plain_group(state):
    ids, count = state["ids"], state["count"]
    key = torch.where((ids < 0) | (ids >= count), count, ids)
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    bounds = torch.arange(count + 1, device=ids.device)
    offsets = (key[:, None] < bounds[None, :]).sum(dim=0).to(torch.int32)
    return order, offsets


def _plain_linear(state):
    base, a, b = state["base"], state["a"], state["b"]
    y = base.clone()
    h = torch.zeros((base.shape[0], a.shape[1]), dtype=torch.bfloat16, device=base.device)
    for k, rows in state["rows"]:
        hk = _x32(state, rows) @ a[k].float().t()
        h[rows] = hk.to(torch.bfloat16)
        y[rows] = (base[rows].float() + state["scale"][k] * (hk @ b[k].float().t())).to(torch.bfloat16)
    return y, h


def _plain_backward(state):
    dy, h, a, b = state["dy"], state["h"], state["a"], state["b"]
    dx = state["dx_base"].clone()
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for k, rows in state["rows"]:
        dyk = dy[rows].float() * state["scale"][k]
        dh = dyk @ b[k].float()
        dx[rows] = (dx[rows].float() + dh @ a[k].float()).to(torch.bfloat16)
        da[k] = (dh.t() @ _x32(state, rows)).to(torch.bfloat16)
        db[k] = (dyk.t() @ h[rows].float()).to(torch.bfloat16)
    return dx, da, db


def run(state):
    if not own:
        return {"group": _plain_group, "linear": _plain_linear,
                "backward": _plain_backward}[state["op"]](state)
    from rank_residual_w4a4_b200 import twq
    if state["op"] == "group":
        g = twq.group_rows(state["ids"], state["count"])
        return g.order, g.offsets
    ad, groups, out = state["adapters"], state["groups"], state["out"]
    if state["op"] == "linear":
        if "x" in state:
            return twq.adapter_linear(state["x"], ad, groups, base=state["base"], **out)
        return twq.adapter_linear_i8(state["xq8"], state["sx"], ad, groups, base=state["base"], **out)
    if "x" in state:
        return twq.adapter_backward(state["dy"], state["x"], state["h"], ad, groups,
                                    dx_base=state["dx_base"], **out)
    return twq.adapter_backward_i8(state["dy"], state["xq8"], state["sx"], state["h"], ad, groups,
                                   dx_base=state["dx_base"], **out)


def work(case):
    b, count, used = case["b"], case["count"], case["used"]
    if case["op"] == "group":
        return {"bytes": 8 * b + 4 * (count + 1), "flops": 0}
    m, n, r, rows = case["m"], case["n"], case["r"], case["b"] - case["plain"]
    x = rows * (m + 4 * (m // GROUP)) if case["codes"] else 2 * rows * m
    bank = 2 * used * r * (m + n)
    if case["op"] == "linear":
        return {"bytes": x + bank + 4 * b * n + 2 * b * r, "flops": 2 * rows * r * (m + n)}
    return {"bytes": x + bank + 2 * rows * n + 4 * b * m + 2 * rows * r + 2 * count * r * (m + n),
            "flops": 4 * rows * r * (m + n)}


def exact(case, seed):
    """The same outputs in 64 bits, row blocks and einsum over the adapters' own rows."""
    s = prepare(case, seed)
    ids = s["ids"].cpu().tolist()
    count = case["count"]
    rows_of = [[] for _ in range(count + 1)]
    for i, k in enumerate(ids):
        rows_of[k if 0 <= k < count else count].append(i)
    dev = s["ids"].device
    if case["op"] == "group":
        order = [i for rows in rows_of for i in rows]
        offsets = [0]
        for rows in rows_of[:count]:
            offsets.append(offsets[-1] + len(rows))
        return (torch.tensor(order, dtype=torch.int32, device=dev),
                torch.tensor(offsets, dtype=torch.int32, device=dev))
    f64 = torch.float64

    def x64(idx):
        if not case["codes"]:
            return s["x"][idx].to(f64)
        return s["xq8"][idx].to(f64) * s["sx"][idx].to(f64).repeat_interleave(GROUP, dim=1)

    if case["op"] == "linear":
        y = s["base"].to(f64)
        h = torch.zeros((case["b"], case["r"]), dtype=f64, device=dev)
    else:
        y = s["dx_base"].to(f64)
        da = torch.zeros(s["a"].shape, dtype=f64, device=dev)
        db = torch.zeros(s["b"].shape, dtype=f64, device=dev)
    for k in range(count):
        a64, b64, f = s["a"][k].to(f64), s["b"][k].to(f64), s["scale"][k].to(f64)
        for at in range(0, len(rows_of[k]), 2048):
            idx = torch.tensor(rows_of[k][at:at + 2048], device=dev)
            if case["op"] == "linear":
                hk = torch.einsum("im,cm->ic", x64(idx), a64)
                h[idx] = hk
                y[idx] += f * torch.einsum("ic,nc->in", hk, b64)
            else:
                dyk = s["dy"][idx].to(f64)
                dh = f * torch.einsum("in,nc->ic", dyk, b64)
                y[idx] += torch.einsum("ic,cm->im", dh, a64)
                da[k] += torch.einsum("ic,im->cm", dh, x64(idx))
                db[k] += f * torch.einsum("in,ic->nc", dyk, s["h"][idx].to(f64))
    return (y, h) if case["op"] == "linear" else (y, da, db)
