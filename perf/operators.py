"""Workloads of the expert layer's and the logits' operators: inputs, the plain
torch form of each, its 64-bit definition and the work that it cannot avoid.

Four operators, in the order in which a decoding step calls them:

plan      the router's chosen experts -> rows sorted by expert (grouped_plan)
swiglu    gathered rows x gate and up weights of their experts, bias, SwiGLU
          (grouped_swiglu)
combine   rows x down weights, bias, weighted sum of each token's rows,
          residual (grouped_combine)
penalize  repetition, frequency and presence penalties, token biases and a
          grammar mask on logits, and the greedy token (lmhead_penalize)

Activations and weights are NVFP4 tensors: E2M1 codes (two a byte, the even
element in the low nibble), an E4M3 scale for 16 elements and an fp32 scale
for the tensor (activations) or the expert (weights).
"""

import torch

own = False  # True: the framework's operators, False: the plain torch forms

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DEV = "cuda"


def listed():
    """The measured cases. E experts are routed over; G of them, from `first` on, are held here."""
    full = dict(k=8, E=256, first=0, G=256)
    expert = dict(D=7168, F=2048)
    vocab = dict(N=129280, dtype="fp32", prompt=0.5)
    return [
        # One token's eight experts, before every expert layer of a decoding step.
        dict(full, name="plan_T1", op="plan", T=1),
        # The large prefill's routing result, all experts on this GPU.
        dict(name="plan_T32768", op="plan", T=32768, k=8, E=384, first=0, G=384),
        # Decoding one sequence: eight experts' gate and up weights are streamed.
        dict(full, **expert, name="swiglu_T1", op="swiglu", T=1, bias=False),
        # Batched decoding: most experts are hit, by two rows on average.
        dict(full, **expert, name="swiglu_T64", op="swiglu", T=64, bias=False),
        # Prefill: 65536 rows, about 256 for each expert, unevenly.
        dict(full, **expert, name="swiglu_T8192", op="swiglu", T=8192, bias=False),
        # One rank of an expert-parallel group, odd sizes: 24 of 96 experts held here, most rows go elsewhere.
        dict(name="swiglu_part_T1003", op="swiglu", T=1003, k=6, E=96, first=17, G=24, D=2080, F=1360, bias=True),
        dict(full, **expert, name="combine_T1", op="combine", T=1, bias=False, residual=True),
        dict(full, **expert, name="combine_T64", op="combine", T=64, bias=False, residual=True),
        dict(full, **expert, name="combine_T8192", op="combine", T=8192, bias=False, residual=True),
        # The same rank: partial sums for the exchange between ranks, so no residual; many tokens have no row here.
        dict(name="combine_part_T1003", op="combine", T=1003, k=6, E=96, first=17, G=24, D=2080, F=1376, bias=True,
             residual=False),
        # One sequence with some history.
        dict(vocab, name="penalize_T1", op="penalize", T=1, L=1024, nbias=32, mask=False),
        # A full serving batch, long histories, a grammar for every row.
        dict(vocab, name="penalize_T256", op="penalize", T=256, L=4096, nbias=300, mask=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    """A case of the listed ones' ranges: one token to thousands, odd counts, all experts or a rank's part of them."""
    op = rng.choice(["plan", "swiglu", "swiglu", "combine", "combine", "penalize"])
    if op == "penalize":
        return dict(op=op, T=_log_int(rng, 1, 256), N=_log_int(rng, 4000, 129280), dtype=rng.choice(["fp32", "bf16"]),
                    prompt=rng.random(), L=_log_int(rng, 1, 4096), nbias=rng.choice([0, rng.randint(1, 300)]),
                    mask=rng.random() < 0.5)
    E = _log_int(rng, 8, 384 if op == "plan" else 256)
    k = rng.randint(1, min(E, 8))
    G = E if rng.random() < 0.5 else rng.randint(1, E)
    case = dict(op=op, T=_log_int(rng, 1, 32768 if op == "plan" else 8192), k=k, E=E, first=rng.randint(0, E - G), G=G)
    if op == "plan":
        return case
    case.update(D=32 * rng.randint(8, 224), F=32 * rng.randint(4, 64), bias=rng.random() < 0.5)
    if op == "combine":
        case["residual"] = rng.random() < 0.5
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


def _weights(case, rows, cols, g):
    """[G, rows, cols] expert weights ~ N(0, 0.02^2), each expert with a global scale of its own."""
    G = case["G"]
    codes = torch.empty((G, rows, cols // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((G, rows, cols // 16), dtype=torch.uint8, device=DEV)
    gs = torch.empty(G, dtype=torch.float32, device=DEV)
    for e in range(G):
        codes[e], scales[e], gs[e:e + 1] = _quantize(0.02 * torch.randn((rows, cols), generator=g, device=DEV))
    return codes, scales, gs


def _routing(case, g):
    """The k experts of each token, some of them more popular than others, and their weights (sum 2.5)."""
    T, E, k = case["T"], case["E"], case["k"]
    score = torch.randn((T, E), generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    val, idx = torch.topk(torch.sigmoid(score), k, dim=1)
    return idx.to(torch.int32).contiguous(), (2.5 * val / val.sum(1, keepdim=True)).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "penalize":
        return _prepare_penalize(case, g)
    T, k, G = case["T"], case["k"], case["G"]
    idx, w = _routing(case, g)
    s = dict(case=case, topk_idx=idx, topk_w=w)
    if case["op"] != "plan":
        s["plan"] = _plain_plan(idx, case["first"], G)
        kept = case["D"] if case["op"] == "swiglu" else case["F"]
        rows = T if case["op"] == "swiglu" else T * k
        x = torch.randn((rows, kept), generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
        if case["op"] == "combine":  # a gated product of two projections
            x *= torch.sigmoid(x) * torch.randn((rows, kept), generator=g, device=DEV)
            x[int(s["plan"][0][-1]):] = 0.0
        s["x"] = _quantize(x)
        del x
        N = 2 * case["F"] if case["op"] == "swiglu" else case["D"]
        s["w"] = _weights(case, N, kept, g)
        s["bias"] = 0.1 * torch.randn((G, N), generator=g, device=DEV) if case["bias"] else None
        if case["op"] == "combine":
            s["residual"] = None
            if case["residual"]:
                s["residual"] = torch.randn((T, N), generator=g, device=DEV).to(torch.bfloat16)
    if own:
        from nvfp4_block_scaled_06_amd import router as rt

        nbytes = rt.grouped_workspace_bytes(T, k, G, case.get("D", 32), case.get("F", 32))
        s["ws"] = rt.Workspace(nbytes)
        if case["op"] != "plan":
            s["xq"] = rt.NVFP4Tensor(*s["x"])
            s["wg"] = rt.GroupedWeights(*s["w"])
            s["rt_plan"] = rt.GroupedPlan(*s["plan"], T, k)
    return s


def _prepare_penalize(case, g):
    T, N, L = case["T"], case["N"], case["L"]
    s = dict(case=case)
    logits = 3.0 * torch.randn((T, N), generator=g, device=DEV)
    s["logits"] = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
    s["out"] = torch.empty_like(s["logits"])
    # Text repeats itself: few tokens make most of it.
    u = torch.rand((T, L), generator=g, device=DEV)
    s["history"] = (N ** u - 1.0).to(torch.int32).clamp(0, N - 1)
    s["lengths"] = torch.randint((L + 1) // 2, L + 1, (T,), generator=g, device=DEV).to(torch.int32)
    s["prompt"] = (s["lengths"].float() * case["prompt"]).to(torch.int32)
    s["repetition"] = 1.0 + 0.3 * torch.rand(T, generator=g, device=DEV)
    s["frequency"] = 0.5 * torch.rand(T, generator=g, device=DEV)
    s["presence"] = 0.5 * torch.rand(T, generator=g, device=DEV)
    s["bias"] = None
    if case["nbias"]:
        n = case["nbias"]
        tok = torch.topk(torch.rand((T, N), generator=g, device=DEV), n, dim=1).indices.to(torch.int32)
        s["bias"] = (torch.arange(0, T * n + 1, n, device=DEV, dtype=torch.int32), tok.reshape(-1).contiguous(),
                     2.0 * torch.randn(T * n, generator=g, device=DEV))
    s["mask"] = None
    if case["mask"]:  # one bit a token, set where the grammar allows it
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (T, (N + 31) // 32), generator=g, device=DEV).to(torch.int32)
    if own:
        from nvfp4_block_scaled_06_amd import router as rt

        s["ws"] = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N))
    return s


# --- one pass ---------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        from nvfp4_block_scaled_06_amd import router as rt

        c = s["case"]
        if op == "plan":
            p = rt.grouped_plan(s["topk_idx"], c["G"], s["ws"], first_expert=c["first"])
            return [p.offsets, p.rows, p.pos]
        if op == "swiglu":
            return rt.grouped_swiglu(s["xq"], s["wg"], s["rt_plan"], bias=s["bias"])
        if op == "combine":
            return rt.grouped_combine(s["xq"], s["wg"], s["rt_plan"], s["topk_w"], s["ws"], bias=s["bias"],
                                      residual=s["residual"])
        idx, logit, logits = rt.lmhead_penalize(
            s["logits"], s["ws"], history=s["history"], prompt=s["prompt"], lengths=s["lengths"],
            repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias=s["bias"],
            mask=s["mask"], out=s["out"])
        return [idx, logit, logits]
    if op == "plan":
        return list(_plain_plan(s["topk_idx"], s["case"]["first"], s["case"]["G"]))
    return {"swiglu": _plain_swiglu, "combine": _plain_combine, "penalize": _plain_penalize}[op](s)


def _plain_plan(idx, first, G):
    """Slots (token k + choice) sorted by expert, those of one expert in slot order: the experts' offsets, the slot
    of each row (-1 behind the last one) and the row of each slot (-1 for experts held elsewhere)."""
    e = idx.reshape(-1).long() - first
    e = torch.where((e >= 0) & (e < G), e, G)
    order = torch.argsort(e, stable=True)
    offsets = torch.searchsorted(e[order].contiguous(), torch.arange(G + 1, device=idx.device))
    place = torch.arange(e.numel(), device=idx.device)
    kept = place < offsets[G]
    rows = torch.where(kept, order, -1)
    pos = torch.empty_like(place)
    pos[order] = torch.where(kept, place, -1)
    return offsets.to(torch.int32), rows.to(torch.int32), pos.to(torch.int32)


def _values(codes, scales):
    """Code values times block scales, fp32 (exact)."""
    lut = torch.tensor(E2M1, dtype=torch.float32, device=codes.device)
    q = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), dim=-1).reshape(codes.shape[0], -1, 16)
    return (q * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).reshape(codes.shape[0], -1)


def _plain_swiglu(s):
    c = s["case"]
    offsets, rows, _ = s["plan"]
    xc, xs, gsa = s["x"]
    wc, ws, gsw = s["w"]
    F, off = c["F"], offsets.tolist()
    x = _values(xc, xs)
    out = torch.zeros((c["T"] * c["k"], F), dtype=torch.bfloat16, device=xc.device)
    for e in range(c["G"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        y = (x[rows[a:b].long() // c["k"]] @ _values(wc[e], ws[e]).t()) * (gsa * gsw[e])
        if s["bias"] is not None:
            y = y + s["bias"][e]
        gate, up = y[:, :F], y[:, F:]
        out[a:b] = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)
    return out


def _plain_combine(s):
    c = s["case"]
    offsets, rows, _ = s["plan"]
    hc, hs, gsh = s["x"]
    wc, ws, gsw = s["w"]
    off = offsets.tolist()
    slots = torch.zeros((c["T"] * c["k"], c["D"]), dtype=torch.float32, device=hc.device)
    w = s["topk_w"].reshape(-1, 1)
    for e in range(c["G"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        y = (_values(hc[a:b], hs[a:b]) @ _values(wc[e], ws[e]).t()) * (gsh * gsw[e])
        if s["bias"] is not None:
            y = y + s["bias"][e]
        slot = rows[a:b].long()
        slots[slot] = w[slot] * y
    out = slots.reshape(c["T"], c["k"], c["D"]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(torch.bfloat16)


def _plain_penalize(s):
    c = s["case"]
    T, N, L = c["T"], c["N"], c["L"]
    x = s["logits"].float()
    place = torch.arange(L, device=x.device)
    tok = s["history"].long()
    used = place < s["lengths"].unsqueeze(1)
    made = used & (place >= s["prompt"].unsqueeze(1))
    seen = torch.zeros((T, N), device=x.device).scatter_add_(1, tok, used.float())
    count = torch.zeros((T, N), device=x.device).scatter_add_(1, tok, made.float())
    r = s["repetition"].unsqueeze(1)
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = torch.where(count > 0, x - s["frequency"].unsqueeze(1) * count, x)
    x = torch.where(count > 0, x - s["presence"].unsqueeze(1), x)
    if s["bias"] is not None:
        start, t, v = s["bias"]
        row = torch.arange(T, device=x.device).repeat_interleave((start[1:] - start[:-1]).long(),
                                                                 output_size=t.numel())
        x[row, t.long()] += v
    if s["mask"] is not None:
        bit = (s["mask"].unsqueeze(2) >> torch.arange(32, device=x.device, dtype=torch.int32)) & 1
        x = torch.where(bit.reshape(T, -1)[:, :N] == 1, x, float("-inf"))
    top = x.amax(1)  # the choice comes before the rounding of the stored logits
    at = torch.where(x == top.unsqueeze(1), torch.arange(N, device=x.device), N).amin(1)
    at = torch.where(top > float("-inf"), at, -1)
    return [at.to(torch.int32), top, x.to(s["logits"].dtype)]


# --- the operators' definitions in 64 bits ------------------------------------


def _decode64(codes, scales, gs):
    """x[i] = value(code) * block scale * global scale, from the bits of the formats."""
    nib = torch.stack((codes % 16, codes // 16), dim=-1).flatten(-2).to(torch.int64)
    sign, ex, man = 1 - 2 * (nib // 8), (nib // 2) % 4, nib % 2
    q = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man.double()) * 2.0 ** (ex.double() - 1)) * sign
    sc = scales.to(torch.int64)
    ex, man = sc // 8, (sc % 8).double()
    v = torch.where(ex == 0, man * 2.0 ** -9, (8.0 + man) * 2.0 ** (ex.double() - 10))
    return q * v.repeat_interleave(16, dim=-1) * gs.double()


def exact(case, seed):
    """What run() returns, unrounded, expert by expert over the tokens that chose it."""
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(case, s)
    if case["op"] == "penalize":
        return _exact_penalize(case, s)
    T, k, F, D = case["T"], case["k"], case["F"], case["D"]
    idx = s["topk_idx"].long() - case["first"]
    xc, xs, gx = s["x"]
    wc, ws, gw = s["w"]
    n = 0
    if case["op"] == "swiglu":
        out = torch.zeros((T * k, F), dtype=torch.float64, device=DEV)
    else:
        out = torch.zeros((T, D), dtype=torch.float64, device=DEV)
        if s["residual"] is not None:
            out += s["residual"].double()
    for e in range(case["G"]):
        tok, choice = (idx == e).nonzero(as_tuple=True)
        m = tok.numel()
        if m == 0:
            continue
        W = _decode64(wc[e], ws[e], gw[e])
        b = 0.0 if s["bias"] is None else s["bias"][e].double()
        if case["op"] == "swiglu":
            y = torch.mm(_decode64(xc[tok], xs[tok], gx), W.t().contiguous()) + b
            out[n:n + m] = y[:, :F] * torch.special.expit(y[:, :F]) * y[:, F:]
        else:
            y = torch.mm(_decode64(xc[n:n + m], xs[n:n + m], gx), W.t().contiguous()) + b
            out.index_add_(0, tok, y * s["topk_w"][tok, choice].double().unsqueeze(1))
        n += m
    return out


def _exact_plan(case, s):
    idx = s["topk_idx"].reshape(-1)
    slots = [(idx == case["first"] + e).nonzero().reshape(-1) for e in range(case["G"])]
    sizes = torch.tensor([0] + [x.numel() for x in slots], device=DEV)
    rows = torch.full((idx.numel(),), -1, device=DEV)
    pos = rows.clone()
    kept = torch.cat(slots)
    rows[:kept.numel()] = kept
    pos[kept] = torch.arange(kept.numel(), device=DEV)
    return [sizes.cumsum(0).to(torch.int32), rows.to(torch.int32), pos.to(torch.int32)]


def _exact_penalize(case, s):
    """Row by row with the tokens' counts."""
    outs = []
    for t in range(case["T"]):
        x = s["logits"][t].double()
        h = s["history"][t, :int(s["lengths"][t])].long()
        seen = torch.unique(h)
        r = s["repetition"][t].double()
        x[seen] = torch.where(x[seen] > 0, x[seen] / r, x[seen] * r)
        made, times = torch.unique(h[int(s["prompt"][t]):], return_counts=True)
        x[made] -= s["frequency"][t].double() * times + s["presence"][t].double()
        if s["bias"] is not None:
            a, b = int(s["bias"][0][t]), int(s["bias"][0][t + 1])
            x[s["bias"][1][a:b].long()] += s["bias"][2][a:b].double()
        if s["mask"] is not None:
            n = torch.arange(case["N"], device=DEV)
            x[(s["mask"][t][n // 32] >> (n % 32).int()) & 1 == 0] = float("-inf")
        outs.append(x)
    x = torch.stack(outs)
    top, at = x.max(1)
    return [at.to(torch.int32), top, x]


def work(case):
    """Bytes: each tensor that the pass needs once, with the weights of the experts expected to be hit. Operations:
    multiply and add of the rows held here."""
    op, T = case["op"], case["T"]
    if op == "penalize":
        size = 4 if case["dtype"] == "fp32" else 2
        per_row = 2 * case["N"] * size + 3 * case["L"] + 8 * case["nbias"] + (case["N"] // 8 if case["mask"] else 0)
        return {"bytes": T * per_row, "flops": 2 * T * case["N"]}
    k, E, G = case["k"], case["E"], case["G"]
    slots = T * k
    if op == "plan":
        return {"bytes": 4 * (3 * slots + G + 1), "flops": slots}
    D, F = case["D"], case["F"]
    rows = slots * G / E  # held here, on average
    hit = G * (1.0 - (1.0 - k / E) ** T)
    nvfp4 = 9 / 16
    if op == "swiglu":
        b = hit * 2 * F * D * nvfp4 + min(T, rows) * D * nvfp4 + 2 * slots * F + 4 * slots
        return {"bytes": int(b), "flops": int(rows * 2 * 2 * F * D)}
    b = hit * F * D * nvfp4 + rows * F * nvfp4 + 2 * T * D * (2 if case["residual"] else 1) + 12 * slots
    return {"bytes": int(b), "flops": int(rows * 2 * F * D)}
