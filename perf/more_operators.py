"""Workloads of the routing on given logits and of the lm_head's losses: inputs, the plain torch form of each, its 64-bit
definition and the work that it cannot avoid.

Three operators, in the order in which a decoder's last layer meets them:

select    logits of the experts -> the chosen experts and their weights: softmax or sigmoid scores, a bias that moves the
          choice only, groups of which the best are kept, top-k, renormalised weights (select); with `grad` the gradient
          of the logits too (select_backward)
loss      cross entropy over the vocabulary of an NVFP4 lm_head (lmhead_loss); with `grad` the gradient of x too
distill   divergence from a teacher of which each token's largest logits are known (lmhead_distill); with `grad` the
          gradient of x too

x and the lm_head's weights are NVFP4 tensors: E2M1 codes (two a byte, the even element in the low nibble), an E4M3 scale
for 16 elements and an fp32 scale for the tensor.
"""

import torch

own = False  # True: the framework's operators, False: the plain torch forms

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DEV = "cuda"


def listed():
    """The measured cases."""
    routed = dict(E=256, k=8, dtype="fp32", scoring="sigmoid", bias=True, groups=8, kept=4, top=2, renorm=True)
    plain = dict(E=384, k=8, dtype="fp32", scoring="softmax", bias=False, groups=1, kept=1, top=1, renorm=True)
    head = dict(D=7168, N=129280)
    return [
        # One decoded token, before every expert layer: four of eight groups, then eight experts.
        dict(routed, name="select_T1", op="select", T=1, grad=False),
        # A large prefill's choice, all experts in one group.
        dict(plain, name="select_T32768", op="select", T=32768, grad=False),
        # A training step's tokens: the choice, and the gradient that its weights send back.
        dict(routed, name="select_grad_T8192", op="select", T=8192, grad=True),
        # A softmax router that does not renormalise, odd sizes: its gradient reaches every expert.
        dict(name="select_grad_T1003", op="select", T=1003, E=96, k=6, dtype="bf16", scoring="softmax", bias=False,
             groups=6, kept=3, top=1, renorm=False, grad=True),
        # The log-probability of one token, as a verifier of drafted text asks for it: the weights are streamed once.
        dict(head, name="loss_T1", op="loss", T=1, grad=False),
        # A prompt scored in one call (perplexity).
        dict(head, name="loss_T4096", op="loss", T=4096, grad=False),
        # A training step on a micro-batch.
        dict(head, name="loss_grad_T4096", op="loss", T=4096, grad=True),
        # A short text under a small odd vocabulary.
        dict(name="loss_grad_T203", op="loss", T=203, D=2080, N=32003, grad=True),
        # A few tokens measured against the unquantized model's 64 best.
        dict(head, name="distill_T32", op="distill", T=32, K=64, dtype="fp32", tau=1.0, grad=False),
        # A prompt measured likewise.
        dict(head, name="distill_T1024", op="distill", T=1024, K=64, dtype="bf16", tau=1.0, grad=False),
        # A training step that follows the teacher.
        dict(head, name="distill_grad_T1024", op="distill", T=1024, K=64, dtype="bf16", tau=2.0, grad=True),
        # A handful of tokens, odd sizes.
        dict(name="distill_grad_T21", op="distill", T=21, K=37, dtype="fp32", tau=1.5, D=1056, N=50021, grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    """A case of the listed ones' ranges: one token to thousands, odd counts, small and large vocabularies."""
    op = rng.choice(["select", "loss", "distill"])
    case = dict(op=op, grad=rng.random() < 0.5)
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 6, 8])
        E = groups * _log_int(rng, max(4, 8 // groups), 384 // groups)
        kept = rng.randint(1, groups)
        case.update(T=_log_int(rng, 1, 32768), E=E, k=rng.randint(1, min(E // groups * kept, 8)),
                    dtype=rng.choice(["fp32", "bf16"]), scoring=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.random() < 0.5, groups=groups, kept=kept, top=rng.choice([1, 2]), renorm=rng.random() < 0.7)
        return case
    case.update(T=_log_int(rng, 1, 4096), D=32 * rng.randint(8, 224), N=_log_int(rng, 2000, 129280))
    if op == "distill":
        case.update(K=_log_int(rng, 1, 128), dtype=rng.choice(["fp32", "bf16"]), tau=rng.choice([0.5, 1.0, 2.0, 4.0]))
    return case


# --- inputs -----------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _quantize(x):
    """[..., C] fp32 -> NVFP4 codes [..., C/2], scales [..., C/16] and the global scale, as a checkpoint holds them."""
    gs = x.abs().max() / 2688.0
    b = x.reshape(*x.shape[:-1], -1, 16)
    scale = (b.abs().amax(-1) / (6.0 * gs)).clamp(max=448.0).to(torch.float8_e4m3fn)
    q = b / (scale.float() * gs).clamp(min=1e-30).unsqueeze(-1)
    mag = torch.bucketize(q.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device),
                          out_int32=True).to(torch.uint8)
    code = (mag | ((q < 0).to(torch.uint8) << 3)).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8), gs.reshape(1)


def prepare(case, seed):
    g = _gen(seed)
    s = _prepare_select(case, g) if case["op"] == "select" else _prepare_head(case, g)
    if own and case["op"] != "select":
        from nvfp4_block_scaled_06_amd import router as rt

        s["ws"] = rt.Workspace(rt.lmhead_loss_workspace_bytes(case["T"], case["D"], case["N"], case["grad"]))
        s["xq"] = rt.NVFP4Tensor(*s["x"])
        s["wq"] = rt.NVFP4Tensor(*s["w"])
    return s


def _prepare_select(case, g):
    T, E = case["T"], case["E"]
    s = dict(case=case)
    logits = 1.5 * torch.randn((T, E), generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    s["logits"] = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
    s["bias"] = None
    if case["bias"]:  # moved by small equal steps during training, to even out the experts' loads
        s["bias"] = 0.001 * torch.randint(-100, 101, (E,), generator=g, device=DEV).float()
    s["scale"] = 2.5 if case["renorm"] else 1.0
    if case["grad"]:
        s["grad_w"] = torch.randn((T, case["k"]), generator=g, device=DEV) / T
    return s


def _prepare_head(case, g):
    T, D, N = case["T"], case["D"], case["N"]
    s = dict(case=case)
    s["x"] = _quantize(torch.randn((T, D), generator=g, device=DEV) * torch.exp(
        0.3 * torch.randn((T, 1), generator=g, device=DEV)))
    s["w"] = _quantize(0.02 * torch.randn((N, D), generator=g, device=DEV))
    # The tokens that take part are weighted alike; a prompt's own are left out.
    s["weight"] = torch.full((T,), 1.0 / T, device=DEV)
    if case["op"] == "loss":
        y = torch.randint(0, N, (T,), generator=g, device=DEV)
        out = torch.rand(T, generator=g, device=DEV) < (0.1 if T > 1 else 0.0)
        s["targets"] = torch.where(out, -100, y).to(torch.int32)
        return s
    # The teacher's K best, from the best downwards; its shorter lists are filled up with -1.
    K = case["K"]
    first = torch.randint(0, N, (T, 1), generator=g, device=DEV)
    step = torch.randint(1, N // K + 1, (T, K), generator=g, device=DEV)
    tokens = (first + step.cumsum(1)) % N  # distinct: the steps of a row sum to N at most
    t = 12.0 + 2.0 * torch.randn((T, K), generator=g, device=DEV).sort(dim=1, descending=True).values
    length = torch.randint((K + 1) // 2, K + 1, (T, 1), generator=g, device=DEV)
    s["tokens"] = torch.where(torch.arange(K, device=DEV) < length, tokens, -1).to(torch.int32)
    s["teacher"] = t.to(torch.bfloat16) if case["dtype"] == "bf16" else t
    return s


# --- one pass ---------------------------------------------------------------


def run(s):
    c = s["case"]
    if own:
        from nvfp4_block_scaled_06_amd import router as rt

        if c["op"] == "select":
            idx, w = rt.select(s["logits"], c["k"], bias=s["bias"], scoring=c["scoring"], groups=c["groups"],
                               topk_groups=c["kept"], group_top=c["top"], renormalize=c["renorm"],
                               routed_scale=s["scale"])
            if not c["grad"]:
                return [idx, w]
            return [idx, w, rt.select_backward(s["logits"], idx, s["grad_w"], scoring=c["scoring"],
                                               renormalize=c["renorm"], routed_scale=s["scale"])]
        if c["op"] == "loss":
            loss, lse, dx = rt.lmhead_loss(s["xq"], s["wq"], s["targets"], s["ws"], weight=s["weight"],
                                           want_grad=c["grad"])
            return [loss, lse, dx] if c["grad"] else [loss, lse]
        loss, lse, logq, dx = rt.lmhead_distill(s["xq"], s["wq"], s["tokens"], s["teacher"], s["ws"],
                                                temperature=c["tau"], weight=s["weight"], want_grad=c["grad"])
        return [loss, lse, logq, dx] if c["grad"] else [loss, lse, logq]
    return {"select": _plain_select, "loss": _plain_loss, "distill": _plain_distill}[c["op"]](s)


def _plain_select(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    # The choice in 64 bits: among thousands of rows some keys differ by less than 32 bits tell apart.
    x = s["logits"].double()
    if c["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    key = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        in_group = key.reshape(T, c["groups"], -1)
        best = in_group.sort(dim=2, descending=True).values[:, :, :c["top"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros((T, c["groups"]), dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = torch.where(keep.unsqueeze(2), in_group, float("-inf")).reshape(T, E)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k]  # ties to the lower expert
    score = score.float()
    chosen = score.gather(1, idx)
    total = chosen.sum(1, keepdim=True) if c["renorm"] else torch.ones((), device=x.device)
    w = s["scale"] * chosen / total
    if not c["grad"]:
        return [idx.to(torch.int32), w]
    dw = s["scale"] * s["grad_w"]
    if c["renorm"]:
        dw = (dw - (dw * (chosen / total)).sum(1, keepdim=True)) / total
    ds = torch.zeros((T, E), device=x.device).scatter_(1, idx, dw)
    if c["scoring"] == "sigmoid":
        dx = ds * score * (1.0 - score)
    else:
        dx = score * (ds - (ds * score).sum(1, keepdim=True))
    return [idx.to(torch.int32), w, dx.to(s["logits"].dtype)]


def _values(codes, scales):
    """Code values times block scales, fp32 (exact)."""
    lut = torch.tensor(E2M1, dtype=torch.float32, device=codes.device)
    q = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), dim=-1).reshape(codes.shape[0], -1, 16)
    return (q * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).reshape(codes.shape[0], -1)


def _plain_loss(s):
    c = s["case"]
    xc, xs, gsa = s["x"]
    wc, ws, gsw = s["w"]
    w = _values(wc, ws)
    z = (_values(xc, xs) @ w.t()) * (gsa * gsw)
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    y = s["targets"].long().unsqueeze(1)
    valid = (y >= 0) & (y < c["N"])
    y = torch.where(valid, y, 0)
    loss = torch.where(valid, lse - z.gather(1, y), 0.0).reshape(-1)
    if not c["grad"]:
        return [loss, lse.reshape(-1)]
    p = torch.exp(z - lse).scatter_add_(1, y, torch.full_like(lse, -1.0))
    dx = torch.where(valid, (p @ w) * (gsw * s["weight"].unsqueeze(1)), 0.0)
    return [loss, lse.reshape(-1), dx.to(torch.bfloat16)]


def _plain_distill(s):
    c = s["case"]
    tau = c["tau"]
    xc, xs, gsa = s["x"]
    wc, ws, gsw = s["w"]
    w = _values(wc, ws)
    z = (_values(xc, xs) @ w.t()) * (gsa * gsw / tau)
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    tok = s["tokens"].long()
    valid = (tok >= 0) & (tok < c["N"])
    tok = torch.where(valid, tok, 0)
    t = torch.where(valid, s["teacher"].float() / tau, float("-inf"))
    t = t - t.amax(1, keepdim=True)
    logp = t - torch.log(torch.exp(t).sum(1, keepdim=True))
    p = torch.exp(logp)
    logq = torch.where(valid, z.gather(1, tok) - lse, 0.0)
    loss = tau * tau * torch.where(valid, p * (logp - logq), 0.0).sum(1)
    if not c["grad"]:
        return [loss, lse.reshape(-1), logq]
    q = torch.exp(z - lse).scatter_add_(1, tok, -p)
    dx = (q @ w) * (gsw * tau * s["weight"].unsqueeze(1))
    return [loss, lse.reshape(-1), logq, dx.to(torch.bfloat16)]


# --- the operators' definitions in 64 bits ------------------------------------


def exact(case, seed):
    """What run() returns, unrounded."""
    s = prepare(case, seed)
    return _exact_select(case, s) if case["op"] == "select" else _exact_head(case, s)


def _exact_select(case, s):
    """By repeated maxima, and the gradient through the scores' Jacobian."""
    T, E, k = case["T"], case["E"], case["k"]
    x = s["logits"].double()
    score = torch.special.expit(x) if case["scoring"] == "sigmoid" else torch.exp(
        x - torch.logsumexp(x, 1, keepdim=True))
    key = score.clone()
    if s["bias"] is not None:
        key += s["bias"].double()
    size = E // case["groups"]
    if case["groups"] > 1:
        best = torch.stack([key[:, a:a + size].topk(min(case["top"], size), dim=1).values.sum(1)
                            for a in range(0, E, size)], dim=1)
        keep = torch.zeros_like(best)
        for _ in range(case["kept"]):
            at = best.argmax(1, keepdim=True)
            keep.scatter_(1, at, 1.0)
            best.scatter_(1, at, float("-inf"))
        key[keep.repeat_interleave(size, dim=1) == 0] = float("-inf")
    chosen = []
    for _ in range(k):
        at = key.argmax(1, keepdim=True)
        chosen.append(at)
        key.scatter_(1, at, float("-inf"))
    idx = torch.cat(chosen, 1)
    v = score.gather(1, idx)
    S = v.sum(1, keepdim=True)
    w = s["scale"] * (v / S if case["renorm"] else v)
    outs = [idx.to(torch.int32), w]
    if case["grad"]:
        u = s["grad_w"].double()
        dv = s["scale"] * ((u - (u * (v / S)).sum(1, keepdim=True)) / S if case["renorm"] else u)
        if case["scoring"] == "sigmoid":
            d = torch.zeros_like(x).scatter_(1, idx, dv * v * torch.special.expit(-x.gather(1, idx)))
        else:
            d = -score * (dv * v).sum(1, keepdim=True)
            d.scatter_add_(1, idx, dv * v)
        outs.append(d)
    return outs


def _decode64(codes, scales, gs):
    """x[i] = value(code) * block scale * global scale, from the bits of the formats."""
    nib = torch.stack((codes % 16, codes // 16), dim=-1).flatten(-2).to(torch.int32)
    sign, ex, man = 1 - 2 * (nib // 8), (nib // 2) % 4, nib % 2
    q = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man.double()) * 2.0 ** (ex.double() - 1)) * sign
    sc = scales.to(torch.int64)
    ex, man = sc // 8, (sc % 8).double()
    v = torch.where(ex == 0, man * 2.0 ** -9, (8.0 + man) * 2.0 ** (ex.double() - 10))
    return q * v.repeat_interleave(16, dim=-1) * gs.double()


def _exact_head(case, s):
    """Both losses: the vocabulary in pieces, first the sums, then the gradient."""
    T, N, tau, piece = case["T"], case["N"], case.get("tau", 1.0), 16384
    x = _decode64(*s["x"])
    wc, ws, gsw = s["w"]
    z = torch.empty((T, N), dtype=torch.float64, device=DEV)
    for a in range(0, N, piece):
        z[:, a:a + piece] = torch.mm(x, _decode64(wc[a:a + piece], ws[a:a + piece], gsw).t().contiguous()) / tau
    lse = torch.logsumexp(z, 1)
    if case["op"] == "loss":
        tok = s["targets"].long().unsqueeze(1)
        valid = tok >= 0
        p = valid.double()
        logp = torch.zeros_like(p)
    else:
        tok = s["tokens"].long()
        valid = tok >= 0
        logp = torch.log_softmax((s["teacher"].double() / tau).masked_fill(~valid, float("-inf")), dim=1)
        p = torch.exp(logp)
        logp = logp.masked_fill(~valid, 0.0)
    logq = (z.gather(1, tok.clamp(min=0)) - lse.unsqueeze(1)).masked_fill(~valid, 0.0)
    outs = [tau ** 2 * (p * (logp - logq)).sum(1), lse]
    if case["op"] == "distill":
        outs.append(logq)
    if case["grad"]:
        z.sub_(lse.unsqueeze(1)).exp_()
        z.scatter_add_(1, tok.clamp(min=0), -p)
        dx = torch.zeros_like(x)
        for a in range(0, N, piece):
            dx += torch.mm(z[:, a:a + piece].contiguous(), _decode64(wc[a:a + piece], ws[a:a + piece], gsw))
        dx *= tau * s["weight"].double().unsqueeze(1)
        outs.append(dx * valid.any(1, keepdim=True))
    return outs


def work(case):
    """Bytes: each tensor that the pass needs once. Operations: the multiplications and additions of the products (the
    gradient's included, without a second computation of the logits), or a few for each logit of a choice."""
    T = case["T"]
    if case["op"] == "select":
        E, k, size = case["E"], case["k"], 4 if case["dtype"] == "fp32" else 2
        b = T * (E * size + 8 * k) + (4 * E if case["bias"] else 0)
        if case["grad"]:  # the logits, the choice and its gradient in, the logits' gradient out
            b += T * (E * size + 4 * k)
        return {"bytes": b, "flops": (8 if case["grad"] else 4) * T * E}
    D, N = case["D"], case["N"]
    b = (N + T) * D * 9 // 16 + 8 * T
    if case["op"] == "loss":
        b += 4 * T
    else:
        b += T * case["K"] * (8 + (4 if case["dtype"] == "fp32" else 2))
    if case["grad"]:
        b += 2 * T * D + 4 * T
    return {"bytes": b, "flops": (4 if case["grad"] else 2) * T * N * D}
