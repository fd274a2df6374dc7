"""The operators around the FP8 linears, as cases to be timed and compared.

Four operators that sit beside the block-scaled linears of this library:

  route    top-k choice of experts from router logits, with the counts per expert,
           the balance loss and the gradient of both weights and loss
  group    rows sorted by group (expert or adapter): the segment starts that the
           grouped linear and the adapters take, and the order that leads there
  combine  the experts' output rows weighted and summed back to their tokens, and
           the gradient of that
  lora     low-rank adapters of many requests at once, added to a shared projection

`run` computes each in a plain form (elementary torch operations in 32 bits, long
sums in 64) where `own` is false, and through the library's entry points where it
is true.  `exact` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

F32, F64, I32, I64, BF16 = torch.float32, torch.float64, torch.int32, torch.int64, torch.bfloat16
TYPES = {"bf16": BF16, "fp32": F32}


# ------------------------------------------------------------------- cases

def _route(T, E, k, dtype, scoring, renorm, balance, masked, closed, train, **more):
    return dict(more, op="route", T=T, E=E, k=k, dtype=dtype, scoring=scoring, renorm=renorm,
                scale=2.5 if scoring == "sigmoid" else 1.0, balance=balance, masked=masked,
                closed=closed, train=train)


def _group(T, k, groups, dropped, **more):
    return dict(more, op="group", T=T, k=k, groups=groups, dropped=dropped)


def _combine(T, k, H, base, dropped, back, **more):
    return dict(more, op="combine", T=T, k=k, H=H, base=base, dropped=dropped, back=back)


def _lora(M, N, K, R, L, requests, bare, **more):
    return dict(more, op="lora", M=M, N=N, K=K, R=R, L=L, requests=requests, bare=bare)


def listed():
    return [
        # one token of a decode step through a 256-expert router
        _route(1, 256, 8, "bf16", "sigmoid", True, 0.0, False, 0, False, name="route one token"),
        # a training batch of the 16-expert workload: an odd number of rows, padding, one expert off
        _route(4093, 16, 2, "bf16", "softmax", False, 0.01, True, 1, True, name="route train 16"),
        # a large training batch over 256 experts
        _route(16384, 256, 8, "fp32", "sigmoid", True, 0.001, True, 0, True, name="route train 256"),
        # a decode batch sorted by its requests' adapters, some requests without one
        _group(64, 1, 48, 4, name="group 64 rows by adapter"),
        # the entries of a long prompt sorted by expert
        _group(16384, 8, 256, 97, name="group 131072 entries by expert"),
        # a decode batch's expert rows summed on top of the shared expert's output
        _combine(32, 8, 7168, True, 0, False, name="combine decode"),
        # a prompt's expert rows, an odd number of tokens, some entries dropped
        _combine(4093, 8, 7168, False, 211, False, name="combine prompt"),
        # the gradient of a training batch
        _combine(2048, 8, 7168, False, 64, True, name="combine gradient"),
        # one request, one adapter, the attention output projection
        _lora(1, 4096, 4096, 16, 1, 1, 0, name="lora one token"),
        # a decode batch of many adapters beside gate and up
        _lora(64, 28672, 4096, 16, 48, 60, 4, name="lora decode 64"),
        # prompts of a few requests beside down, an odd number of rows
        _lora(5003, 4096, 14336, 16, 5, 9, 64, name="lora prompt down"),
        # prompts beside gate and up at a large rank
        _lora(4096, 28672, 4096, 64, 8, 12, 0, name="lora prompt gate up"),
    ]


def _spread(rng, lo, hi):
    """An integer between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(("route", "route", "group", "combine", "lora", "lora"))
    if op == "route":
        E = rng.choice((_spread(rng, 2, 1024), 8, 16, 64, 128, 256))
        k = min(E, rng.randint(1, 10))
        return _route(_spread(rng, 1, 32768), E, k, rng.choice(("bf16", "fp32")),
                      rng.choice(("softmax", "sigmoid")), rng.random() < 0.5, rng.choice((0.001, 0.01, 0.1)),
                      rng.random() < 0.5, rng.choice((0, 0, 1, max(0, (E - k) // 2))) if E > k else 0,
                      rng.random() < 0.6)
    if op == "group":
        T, k = _spread(rng, 1, 65536), rng.randint(1, 8)
        return _group(T, k, _spread(rng, 1, 1024), rng.choice((0, rng.randint(0, T * k))))
    if op == "combine":
        T, k = _spread(rng, 1, 8192), rng.randint(1, 10)
        return _combine(T, k, 8 * _spread(rng, 8, 1024), rng.random() < 0.5,
                        rng.choice((0, rng.randint(0, T * k))), rng.random() < 0.4)
    M = _spread(rng, 1, 8192)
    L = _spread(rng, 1, 64)
    bare = rng.choice((0, M // 16, M // 4))
    requests = rng.randint(min(L, M - bare), max(L, M - bare)) if M <= 128 else rng.randint(L, 3 * L)
    N, K = rng.choice(((4096, 4096), (1024, 4096), (28672, 4096), (4096, 14336),
                       (8 * _spread(rng, 16, 2048), 8 * _spread(rng, 16, 1024))))
    return _lora(M, N, K, 8 * _spread(rng, 1, 16), L, min(requests, M - bare), bare)


def draw(rng):
    most = max(max(w["bytes"], w["flops"] / 50) for w in map(work, listed()))
    while True:
        c = _draw(rng)
        w = work(c)
        # the plain forms of the adapters multiply by all of them at once
        if max(w["bytes"], w["flops"] / 50) <= most and c.get("L", 1) * c.get("R", 1) <= 4096:
            return c


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k, size = c["T"], c["E"], c["k"], 2 if c["dtype"] == "bf16" else 4
        b = T * E * size + T * k * 8 + 4 * E + 4 + (T if c["masked"] else 0)
        f = 6 * T * E
        if c["train"]:  # read the logits, ids and weight gradients again, write the gradient
            b += T * E * size * 2 + T * k * 8 + 4 * E
            f += 8 * T * E
        return {"bytes": b, "flops": f}
    if c["op"] == "group":
        n = c["T"] * c["k"]
        return {"bytes": 12 * n + 4 * (c["groups"] + 1), "flops": n}
    if c["op"] == "combine":
        T, k, H = c["T"], c["k"], c["H"]
        rows = T * k - c["dropped"]
        b = rows * H * 2 + T * H * 2 * (2 if c["base"] and not c["back"] else 1) + T * k * 8
        if c["back"]:  # the experts' rows and the tokens' gradients in, the rows' and the weights' gradients out
            b += T * k * H * 2 + T * k * 4
        return {"bytes": b, "flops": (4 if c["back"] else 2) * rows * H}
    rows, used = c["M"] - c["bare"], min(c["L"], c["requests"])
    b = rows * c["K"] * 2 + c["M"] * c["N"] * 4 + used * (c["N"] + c["K"]) * c["R"] * 2 + c["M"] * 4
    return {"bytes": b, "flops": 2 * rows * c["R"] * (c["N"] + c["K"])}


# ------------------------------------------------------------------ inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _sorted_rows(ids, groups):
    """(offsets, order, slot) of ids sorted by group, rows of no group last."""
    flat = ids.reshape(-1).to(I64)
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(groups + 1, dtype=I64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([count.new_zeros(1), torch.cumsum(count[:groups], 0)])
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=ids.device)
    slot = torch.where(key < groups, slot, -1)
    return offsets.to(I32), order.to(I32), slot.to(I32).reshape(ids.shape)


def _some(g, n, count):
    """A truth value for each of n places, `count` of them true."""
    at = torch.zeros(n, dtype=torch.bool, device="cuda")
    at[torch.randperm(n, generator=g, device="cuda")[:count]] = True
    return at


def prepare(case, seed):
    c, g = case, _rng(seed)
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        # some experts are more popular than others, in every token
        z = _randn(g, T, E, scale=1.5) + _randn(g, E, scale=0.7)
        z[:, torch.randperm(E, generator=g, device="cuda")[:c["closed"]]] = -math.inf
        mask = torch.rand(T, generator=g, device="cuda") < 0.93 if c["masked"] else None
        dev = {"device": "cuda"}
        return dict(case=c, logits=z.to(TYPES[c["dtype"]]), mask=mask, d_weights=_randn(g, T, k, scale=0.1),
                    d_loss=_randn(g, 1).abs() + 0.5,
                    ids=torch.empty(T, k, dtype=I32, **dev), weights=torch.empty(T, k, **dev),
                    counts=torch.empty(E, dtype=I32, **dev), loss=torch.empty(1, **dev),
                    loss_grad=torch.empty(E, **dev), d_logits=torch.empty(T, E, dtype=TYPES[c["dtype"]], **dev),
                    workspace=torch.empty(4 << 20, dtype=torch.uint8, **dev))
    if c["op"] == "group":
        T, k, G = c["T"], c["k"], c["groups"]
        popular = _randn(g, G, scale=0.7)
        ids = torch.multinomial(torch.softmax(popular, 0), T * k, replacement=True, generator=g)
        ids = torch.where(_some(g, T * k, c["dropped"]), -1, ids).to(I32).reshape(T, k)
        return dict(case=c, ids=ids, offsets=torch.empty(G + 1, dtype=I32, device="cuda"),
                    order=torch.empty(T * k, dtype=I32, device="cuda"), slot=torch.empty_like(ids),
                    workspace=torch.empty(4 << 20, dtype=torch.uint8, device="cuda"))
    if c["op"] == "combine":
        T, k, H = c["T"], c["k"], c["H"]
        ids = torch.randint(0, 64, (T * k,), generator=g, device="cuda")
        ids = torch.where(_some(g, T * k, c["dropped"]), -1, ids).to(I32).reshape(T, k)
        offsets, _, slot = _sorted_rows(ids, 64)
        y = _randn(g, T * k, H, dtype=BF16)
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        s = dict(case=c, y=y, weights=w / w.sum(1, keepdim=True), slot=slot, offsets=offsets)
        if c["back"]:
            return dict(s, d_out=_randn(g, T, H, scale=0.1, dtype=BF16), d_y=torch.empty_like(y),
                        d_weights=torch.empty(T, k, device="cuda"))
        return dict(s, base=_randn(g, T, H, dtype=BF16) if c["base"] else None,
                    out=torch.empty(T, H, dtype=BF16, device="cuda"))
    M, N, K, R, L = (c[n] for n in "MNKRL")
    # contiguous rows for each request, requests in any order of adapters, every
    # adapter in use where there are requests enough; `bare` rows have none
    rows, n = M - c["bare"], c["requests"]
    cut = np.sort(np.random.default_rng(seed).choice(np.arange(1, rows), n - 1, replace=False)) if rows > 1 else []
    lengths = torch.tensor(np.diff(np.concatenate([[0], cut, [rows]])), dtype=I64, device="cuda")
    owner = (torch.randperm(n, generator=g, device="cuda") % L).repeat_interleave(lengths)
    ids = torch.cat([owner, owner.new_full((c["bare"],), -1)]).to(I32)
    offsets, order, _ = _sorted_rows(ids, L)
    return dict(case=c, ids=ids, offsets=offsets, order=order, x=_randn(g, M, K, dtype=BF16),
                a=_randn(g, L, R, K, scale=K ** -0.5, dtype=BF16), b=_randn(g, L, N, R, scale=R ** -0.5, dtype=BF16),
                scales=torch.rand(L, generator=g, device="cuda") + 0.5, y=_randn(g, M, N, dtype=BF16),
                out=torch.empty(M, N, dtype=BF16, device="cuda"),
                workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------- plain forms

def _route_plain(s):
    c, z = s["case"], s["logits"].float()
    T, E, k = c["T"], c["E"], c["k"]
    top, at = torch.sort(z, dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    chosen = top > -math.inf
    if s["mask"] is not None:
        chosen = chosen & s["mask"][:, None]
    row = chosen[:, :1]
    ids = torch.where(chosen, at, -1)
    safe = torch.where(row, z, 0.0)
    if c["scoring"] == "softmax":
        e = torch.exp(safe - safe.amax(1, keepdim=True))
        score = share = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-safe))
        share = score / score.sum(1, keepdim=True)
    picked = torch.where(chosen, score.gather(1, at), 0.0)
    part = torch.where(chosen, picked / picked.sum(1, keepdim=True), 0.0) if c["renorm"] else picked
    counts = torch.zeros(T, E, device=z.device).scatter_add_(1, at, chosen.float()).sum(0, dtype=F64)
    n = row.sum().double().clamp(min=1)
    slope = c["balance"] * E * counts / (c["k"] * n * n)
    loss = (slope * torch.where(row, share, 0.0).sum(0, dtype=F64)).sum().float().reshape(1)
    out = [ids.to(I32), c["scale"] * part, counts.to(I32), loss]
    if not c["train"]:
        return out
    up = slope.float() * s["d_loss"]
    down = torch.where(chosen, s["d_weights"] * c["scale"], 0.0)
    d = share * (up - (share * up).sum(1, keepdim=True))
    if c["renorm"]:
        back = part * (down - (part * down).sum(1, keepdim=True))
    else:
        back = picked * down
        if c["scoring"] == "softmax":
            d = d - score * back.sum(1, keepdim=True)
    d = d.scatter_add(1, at, back)
    if c["scoring"] == "sigmoid":
        d = d * (1 - score)
    return out + [torch.where(row, d, 0.0).to(s["logits"].dtype)]


def _combine_plain(s):
    c, slot = s["case"], s["slot"].to(I64)
    T, k, H = c["T"], c["k"], c["H"]
    used = (slot >= 0)
    w = torch.where(used, s["weights"], 0.0)
    rows = s["y"].float()[slot.clamp(min=0)]
    if not c["back"]:
        out = (torch.where(used[..., None], rows, 0.0) * w[..., None]).sum(1)
        return [(out + s["base"].float() if s["base"] is not None else out).to(BF16)]
    d_out = s["d_out"].float()
    d_w = torch.where(used, (rows * d_out[:, None]).sum(2), 0.0)
    d_y = torch.zeros(T * k + 1, H, device=d_out.device)
    d_y[torch.where(used, slot, T * k).reshape(-1)] = (w[..., None] * d_out[:, None]).reshape(T * k, H)
    return [d_y[:-1].to(BF16), d_w]


def _lora_plain(s):
    c = s["case"]
    M, N, K, R, L = (c[n] for n in "MNKRL")
    inner = (s["x"].float() @ s["a"].float().reshape(L * R, K).T).reshape(M, L, R)
    mine = s["ids"][:, None] == torch.arange(L, dtype=I32, device="cuda")
    inner = inner * (mine * s["scales"])[..., None]
    return [(s["y"].float() + inner.reshape(M, L * R) @ s["b"].float().permute(0, 2, 1).reshape(L * R, N)).to(BF16)]


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "route":
        return _route_plain(s)
    if c["op"] == "group":
        return list(_sorted_rows(s["ids"], c["groups"]))
    return _combine_plain(s) if c["op"] == "combine" else _lora_plain(s)


def _run_own(s, c):
    import fine_grained_block_token_b200 as fp8
    if c["op"] == "route":
        ids, weights, counts, loss, loss_grad = fp8.route(
            s["logits"], c["k"], scoring=c["scoring"], renormalize=c["renorm"], scale=c["scale"],
            balance=c["balance"], mask=s["mask"], ids=s["ids"], weights=s["weights"], counts=s["counts"],
            loss=s["loss"], loss_grad=s["loss_grad"], workspace=s["workspace"])
        if not c["train"]:
            return [ids, weights, counts, loss]
        d = fp8.route_backward(s["logits"], ids, s["d_weights"], loss_grad, s["d_loss"], scoring=c["scoring"],
                               renormalize=c["renorm"], scale=c["scale"], d_logits=s["d_logits"])
        return [ids, weights, counts, loss, d]
    if c["op"] == "group":
        return list(fp8.group_rows(s["ids"], c["groups"], offsets=s["offsets"], order=s["order"], slot=s["slot"],
                                   workspace=s["workspace"]))
    if c["op"] == "combine":
        if c["back"]:
            return list(fp8.combine_rows_backward(s["d_out"], s["y"], s["weights"], s["slot"], s["offsets"],
                                                  d_y=s["d_y"], d_weights=s["d_weights"]))
        return [fp8.combine_rows(s["y"], s["weights"], s["slot"], base=s["base"], out=s["out"])]
    return [fp8.lora_add(s["y"], s["x"], s["a"], s["b"], s["offsets"], s["order"], scales=s["scales"], out=s["out"],
                         workspace=s["workspace"])]


# -------------------------------------------------------------- 64 bits

def _route_exact(s):
    """The definition row by row in 64 bits; the gradient by reverse differentiation."""
    c, dtype = s["case"], s["logits"].dtype
    E, k = c["E"], c["k"]
    z = s["logits"].double().requires_grad_()
    live = torch.isfinite(z).any(1)
    if s["mask"] is not None:
        live = live & s["mask"]
    p = torch.softmax(z[live], 1) if c["scoring"] == "softmax" else torch.sigmoid(z[live])
    share = p if c["scoring"] == "softmax" else p / p.sum(1, keepdim=True)
    rank = torch.argsort(z.detach()[live], dim=1, descending=True, stable=True)[:, :k]
    open_ = torch.isfinite(z.detach()[live].gather(1, rank))
    w = torch.where(open_, p.gather(1, rank), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    weights = torch.zeros(c["T"], k, dtype=F64, device=z.device).index_put((live.nonzero()[:, 0],), w)
    counts = torch.bincount(rank[open_], minlength=E).double()
    n = max(1, int(live.sum()))
    loss = c["balance"] * E * ((counts / (k * n)) * (share.sum(0) / n)).sum().reshape(1)
    if not c["train"]:
        return [None, weights.detach(), None, loss.detach()]
    total = (weights * s["d_weights"].double()).sum() + (loss * s["d_loss"].double()).sum()
    d, = torch.autograd.grad(total, z)
    return [None, weights.detach(), None, loss.detach(), d]


def _combine_exact(s):
    c, slot = s["case"], s["slot"].to(I64)
    T, k, H = c["T"], c["k"], c["H"]
    out = s["base"].double() if not c["back"] and s["base"] is not None else torch.zeros(T, H, dtype=F64, device="cuda")
    d_y = torch.zeros(T * k, H, dtype=F64, device="cuda")
    d_w = torch.zeros(T, k, dtype=F64, device="cuda")
    for j in range(k):
        t = (slot[:, j] >= 0).nonzero()[:, 0]
        at, w = slot[t, j], s["weights"][t, j].double()[:, None]
        if c["back"]:
            d_y[at] = w * s["d_out"][t].double()
            d_w[t, j] = (s["y"][at].double() * s["d_out"][t].double()).sum(1)
        else:
            out[t] += w * s["y"][at].double()
    return [d_y, d_w] if c["back"] else [out]


def _lora_exact(s):
    out = s["y"].double()
    for i in range(s["case"]["L"]):
        at = (s["ids"] == i).nonzero()[:, 0]
        if at.numel():
            inner = s["x"][at].double() @ s["a"][i].double().T
            out[at] += s["scales"][i].double() * (inner @ s["b"][i].double().T)
    return [out]


def exact(case, seed):
    if case["op"] == "group":
        return None  # whole numbers alone
    s = prepare(case, seed)
    return {"route": _route_exact, "combine": _combine_exact, "lora": _lora_exact}[case["op"]](s)
