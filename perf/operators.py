"""Cases of the mixture-of-experts operators around the grouped FP8 products: routing, the move of
tokens into and out of the experts' layouts, and the FP8 weight gradient.

Every case has an "op":
  route     scores of T tokens over E experts -> chosen experts and their weights; with "train", the
            gradient of the weights with respect to the scores as well.
  dispatch  chosen experts -> the layout of the grouped products, and the tokens cast to FP8 in it.
  combine   the experts' results back in token order, weighted; with "train", the gradients of the
            results and of the weights as well.
  wgrad     the gradient of the experts' weights: both operands cast to FP8 per channel over blocks of
            128 tokens, then multiplied per expert.
"""
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


# ---- cases -------------------------------------------------------------------------------------
def _route(T, E, topk, scores, groups=1, topk_groups=1, group_top=1, bias=False, renorm=True, scale=1.0,
           bf16=False, train=False):
    return dict(op="route", T=T, E=E, topk=topk, scores=scores, groups=groups, topk_groups=topk_groups,
                group_top=group_top, bias=bias, renorm=renorm, scale=scale, bf16=bf16, train=train)


def _dispatch(T, E, G, topk, H, masked, bf16=True, ue8m0=False):
    return dict(op="dispatch", T=T, E=E, G=G, topk=topk, H=H, masked=masked, bf16=bf16, ue8m0=ue8m0)


def _combine(T, E, G, topk, H, masked, train=False):
    return dict(op="combine", T=T, E=E, G=G, topk=topk, H=H, masked=masked, train=train)


def _wgrad(T, G, topk, N, K, ue8m0=False, bf16=True, accumulate=False):
    return dict(op="wgrad", T=T, G=G, topk=topk, N=N, K=K, ue8m0=ue8m0, bf16=bf16, accumulate=accumulate)


def listed():
    named = {
        # one generated token: nothing but latency
        "route_token": _route(1, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5),
        # an odd decode batch of a softmax router that keeps its probabilities, scores in bf16
        "route_decode_softmax": _route(67, 64, 6, "softmax", renorm=False, bf16=True),
        # a training step's routing of a long batch, with biases for balance and expert groups
        "route_train": _route(16384, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5, train=True),
        # a softmax router in training, groups by their best expert, odd token and expert counts
        "route_train_softmax": _route(5001, 160, 6, "softmax", 8, 3, 1, renorm=False, bf16=True, train=True),
        # decode on one of eight devices: 128 tokens, 32 of the 256 experts here, the masked layout
        "dispatch_decode": _dispatch(128, 256, 32, 8, 7168, True),
        # a prompt of 4096 tokens over experts that are all here, the contiguous layout
        "dispatch_prefill": _dispatch(4096, 32, 32, 8, 7168, False),
        # the way back at decode
        "combine_decode": _combine(128, 256, 32, 8, 7168, True),
        # the way back in training, with its gradients
        "combine_train": _combine(4096, 32, 32, 8, 7168, False, train=True),
        # a small expert layer with ragged groups: latency of the three launches
        "wgrad_small": _wgrad(301, 4, 2, 256, 384),
        # eight experts' down projections over 8192 routed rows, power-of-two scales
        "wgrad_experts": _wgrad(4096, 8, 2, 7168, 2048, ue8m0=True),
        # many experts with few rows each, added to the gradient of earlier micro-batches
        "wgrad_many": _wgrad(1024, 32, 8, 4096, 2048, accumulate=True),
        # a dense layer over a batch that ends inside a block, fp32 scales
        "wgrad_dense": _wgrad(4001, 1, 1, 7168, 18432),
    }
    return [dict(case, name=name) for name, case in named.items()]


def _log_int(rng, low, high):
    return min(high, int(round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(("route", "dispatch", "combine", "wgrad"))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        E = groups * max(8, _log_int(rng, 8, 384) // groups)
        topk_groups = groups if groups == 1 else rng.randint(2, groups)
        topk = rng.randint(1, 8)
        sigmoid = rng.random() < 0.5
        return _route(_log_int(rng, 1, 16384 * 256 // max(E, 256)), E, topk, "sigmoid" if sigmoid else "softmax",
                      groups, topk_groups, 2 if sigmoid else 1, bias=sigmoid and rng.random() < 0.7,
                      renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), bf16=rng.random() < 0.5,
                      train=rng.random() < 0.5)
    H = BLOCK * rng.randint(2, 56)
    if op in ("dispatch", "combine"):
        masked = rng.random() < 0.5
        topk = rng.randint(1, 8)
        G = rng.randint(8, 64)
        E = G * rng.choice((1, 1, 2, 8))
        T = _log_int(rng, 1, 256 if masked else 4096)
        if op == "dispatch":
            return _dispatch(T, E, G, topk, H, masked, bf16=rng.random() < 0.7, ue8m0=rng.random() < 0.4)
        return _combine(T, E, G, topk, H, masked, train=not masked and rng.random() < 0.6)
    G = rng.choice((1, rng.randint(2, 32)))
    topk = 1 if G == 1 else rng.randint(1, min(G, 8))
    N = BLOCK * rng.randint(2, 32)
    K = BLOCK * rng.randint(2, max(2, min(56, 12288 // G // (N // BLOCK))))
    return _wgrad(_log_int(rng, 16, 8192 // topk), G, topk, N, K, ue8m0=rng.random() < 0.5,
                  bf16=rng.random() < 0.7, accumulate=rng.random() < 0.4)


def _rows(case):
    """Rows of the layouts that hold a token: as many as the choices that fall on the experts here."""
    return case["T"] * case["topk"] * case["G"] / case.get("E", case["G"])


def _layout_rows(case):
    """Rows of the contiguous layout's buffers: what any routing of these choices can need."""
    pairs = case["T"] * case["topk"]
    some = min(case["G"], pairs)
    return BLOCK * (some + (pairs - some) // BLOCK)


def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k, size = case["E"], case["topk"], 2 if case["bf16"] else 4
        both = 2 if case["train"] else 1
        return {"bytes": both * T * E * size + T * k * (12 if case["train"] else 8) + 4 * E * case["bias"],
                "flops": both * 8 * T * E}
    rows = _rows(case)
    if case["op"] == "dispatch":
        H = case["H"]
        return {"bytes": T * H * (2 if case["bf16"] else 4) + rows * (H + H / 32) + 8 * T * case["topk"],
                "flops": 4 * rows * H}
    if case["op"] == "combine":
        H, k = case["H"], case["topk"]
        read = rows * H * 2 + T * k * 8
        back = (T * H * 2 + rows * H * 2 + T * k * 4) if case["train"] else 0
        return {"bytes": read + T * H * 2 + back, "flops": (5 if case["train"] else 2) * rows * H}
    N, K, size = case["N"], case["K"], 2 if case["bf16"] else 4
    out = case["G"] * N * K * 4
    return {"bytes": rows * N * size + T * K * size + out * (2 if case["accumulate"] else 1),
            "flops": 2 * rows * N * K}


# ---- inputs ------------------------------------------------------------------------------------
def _choices(gen, T, E, topk):
    """Chosen experts of T tokens: distinct per token, some experts more popular than others."""
    popular = torch.randn(E, generator=gen, device="cuda") * 0.5
    noise = torch.rand((T, E), generator=gen, device="cuda").clamp_(1e-7, 1 - 1e-7)
    gumbel = -torch.log(-torch.log(noise))
    return torch.topk(gumbel + popular, topk, dim=1).indices.to(torch.int32)


def _tokens(gen, shape, bf16):
    """Activations: normal, a few channels much larger than the rest."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= 1 + 15 * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.01)
    return x.to(torch.bfloat16) if bf16 else x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    state = {"case": case}
    T = case["T"]
    if case["op"] == "route":
        E = case["E"]
        logits = torch.randn((T, E), generator=gen, device="cuda") * 1.5
        state["logits"] = logits.to(torch.bfloat16) if case["bf16"] else logits
        # a balancing bias moves by a fixed step per training step
        state["bias"] = torch.randint(-50, 51, (E,), generator=gen, device="cuda") * 1e-3 if case["bias"] else None
        state["dweights"] = torch.randn((T, case["topk"]), generator=gen, device="cuda") if case["train"] else None
        return state
    G, topk = case["G"], case["topk"]
    ids = _choices(gen, T, case.get("E", G), topk)
    if case["op"] == "dispatch":
        state["ids"] = ids
        state["x"] = _tokens(gen, (T, case["H"]), case["bf16"])
        H = case["H"]
        # the layout's buffers, kept from step to step; rows without a token are not written
        if case["masked"]:
            lead, scales = (G, T), (G, H // BLOCK, T)
        else:
            lead, scales = (_layout_rows(case),), (H // BLOCK, _layout_rows(case))
        state["q"] = torch.zeros(lead + (H,), dtype=torch.uint8, device="cuda")
        state["sf"] = torch.zeros(scales, device="cuda")
        return state
    pos, row_pair, _, counts, offsets = _layout(ids, G, T if case.get("masked") else 0)
    state |= {"pos": pos, "row_pair": row_pair, "offsets": offsets}
    if case["op"] == "combine":
        H = case["H"]
        state["weights"] = torch.rand((T, topk), generator=gen, device="cuda")
        y = torch.randn((row_pair.numel(), H), generator=gen, device="cuda").to(torch.bfloat16)
        state["y"] = y.view(row_pair.shape + (H,))
        if case["train"]:
            state["dout"] = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
            state["dy"] = torch.zeros_like(state["y"])
        return state
    N, K = case["N"], case["K"]
    state["x"] = _tokens(gen, (T, K), case["bf16"])
    if G == 1 and topk == 1:
        state["dy"] = (torch.randn((T, N), generator=gen, device="cuda") * 1e-3).to(state["x"].dtype)
    else:
        dy = torch.randn((row_pair.numel(), N), generator=gen, device="cuda") * 1e-3
        dy[row_pair < 0] = 0  # as the gradient of the combine leaves its padding rows
        state["dy"] = dy.to(state["x"].dtype)
    state["longest"] = -(-int(counts.max()) // BLOCK) * BLOCK
    state["dw"] = torch.randn((G, N, K), generator=gen, device="cuda") * 0.05 if case["accumulate"] else None
    return state


# ---- plain forms -------------------------------------------------------------------------------
def _layout(ids, G, m_max):
    """Stable order of the choices by expert. m_max = 0: the contiguous layout (every expert's rows
    padded to a multiple of 128), else the masked one. -> pos, row_pair, m_indices, counts, offsets."""
    T, topk = ids.shape
    pairs = T * topk
    flat = ids.reshape(-1).long()
    here = (flat >= 0) & (flat < G)
    expert = flat.clamp(0, G - 1)
    chosen = (expert[:, None] == torch.arange(G, device=ids.device)) & here[:, None]
    rank = chosen.cumsum(0).gather(1, expert[:, None])[:, 0] - 1
    counts = chosen.sum(0)
    if m_max:
        rows = G * m_max
        offsets = torch.arange(G + 1, device=ids.device) * m_max
    else:
        some = min(G, pairs)
        rows = BLOCK * (some + (pairs - some) // BLOCK)
        offsets = torch.cat((counts.new_zeros(1), ((counts + BLOCK - 1) // BLOCK * BLOCK).cumsum(0)))
    pos = torch.where(here, offsets[expert] + rank, -1)
    # one row more than there are takes what is not here
    at = torch.where(here, pos, rows)
    row_pair = pos.new_full((rows + 1,), -1).scatter(0, at, torch.arange(pairs, device=ids.device))[:rows]
    m_indices = pos.new_full((rows + 1,), -1).scatter(0, at, expert)[:rows]
    pos, row_pair, m_indices = (t.to(torch.int32) for t in (pos, row_pair, m_indices))
    return pos.view(T, topk), row_pair.view(G, m_max) if m_max else row_pair, m_indices, counts.to(torch.int32), offsets.to(torch.int32)


def _pow2_at_least(v):
    m, e = torch.frexp(v)
    return torch.ldexp(torch.ones_like(v), torch.where(m == 0.5, e - 1, e)).clamp(min=2.0 ** -126)


def _cast(x, ue8m0):
    """e4m3 codes (as what they stand for, before the scale) and scales of x over runs of 128 of its last axis."""
    v = x.float().unflatten(-1, (-1, BLOCK))
    amax = v.abs().amax(-1)
    s = amax / torch.full_like(amax, E4M3_MAX)  # a division: by a Python number it would be a product with 1/448
    if ue8m0:
        s = _pow2_at_least(s)
    q = torch.where(s[..., None] == 0, 0.0, v / s[..., None]).to(torch.float8_e4m3fn)
    return q.flatten(-2), s


def _scores(state):
    case, x = state["case"], state["logits"].float()
    if case["scores"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(state):
    case, x = state["case"], state["logits"].float()
    T, E, k = case["T"], case["E"], case["topk"]
    s = _scores(state)
    key = s
    if state["bias"] is not None:
        key = s + state["bias"]
    elif case["groups"] == 1 or case["group_top"] == 1:
        key = x  # the same order, without the rounding of the scores
    if case["groups"] > 1:
        each = key.view(T, case["groups"], -1)
        best = torch.topk(each, case["group_top"], dim=2).values.sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter(1, keep, True)
        key = torch.where(allowed[:, :, None], each, float("-inf")).view(T, E)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = s.gather(1, ids)
    w = chosen / chosen.sum(1, keepdim=True) if case["renorm"] else chosen
    out = {"ids": ids.to(torch.int32), "weights": w * case["scale"]}
    if case["train"]:
        g = state["dweights"] * case["scale"]
        if case["renorm"]:
            total = chosen.sum(1, keepdim=True)
            g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
        ds = torch.zeros_like(s).scatter(1, ids, g)
        if case["scores"] == "sigmoid":
            dx = ds * s * (1.0 - s)
        else:
            dx = s * (ds - (ds * s).sum(1, keepdim=True))
        out["dlogits"] = dx.to(state["logits"].dtype)
    return out


def _plain_dispatch(state):
    case = state["case"]
    G, T = case["G"], case["T"]
    pos, row_pair, m_indices, counts, offsets = _layout(state["ids"], G, T if case["masked"] else 0)
    q, s = _cast(state["x"], case["ue8m0"])
    token = (row_pair.long() // case["topk"]).clamp(min=0)
    empty = (row_pair < 0)[..., None]
    q = q.view(torch.uint8)[token].masked_fill(empty, 0).view(torch.float8_e4m3fn)
    s = s[token].masked_fill(empty, 0).transpose(-1, -2).contiguous()
    if case["masked"]:
        return {"pos": pos, "masked_m": counts, "q": q, "sf": s}
    return {"pos": pos, "m_indices": m_indices, "offsets": offsets, "q": q, "sf": s}


def _plain_combine(state):
    case, pos, w = state["case"], state["pos"].long(), state["weights"]
    H = case["H"]
    rows = state["y"].view(-1, H)
    picked = rows[pos.clamp(min=0)].float().masked_fill((pos < 0)[..., None], 0)
    out = {"out": (picked * w[..., None]).sum(1).to(torch.bfloat16)}
    if case["train"]:
        dout = state["dout"].float()
        out["dweights"] = (picked * dout[:, None]).sum(2)
        pair = state["row_pair"].long()
        weight = torch.where(pair < 0, 0.0, w.reshape(-1)[pair.clamp(min=0)])
        out["dy"] = (dout[(pair // case["topk"]).clamp(min=0)] * weight[:, None]).to(torch.bfloat16)
    return out


def _per_channel(rows, ue8m0):
    """Rows as the FP8 codes and scales of each channel over blocks of 128 rows stand for them."""
    q, s = _cast(rows.t().contiguous(), ue8m0)
    return (q.float().unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2).t()


def _plain_wgrad(state):
    case = state["case"]
    G, topk, T = case["G"], case["topk"], case["T"]
    if G == 1 and topk == 1:
        pad = -T % BLOCK
        x = torch.nn.functional.pad(state["x"], (0, 0, 0, pad))
        dy = torch.nn.functional.pad(state["dy"], (0, 0, 0, pad))
    else:
        pair = state["row_pair"].long()
        x = state["x"][(pair // topk).clamp(min=0)].masked_fill((pair < 0)[:, None], 0)
        dy = state["dy"]
    a, b = _per_channel(dy, case["ue8m0"]), _per_channel(x, case["ue8m0"])
    # every expert's rows, as many as the longest has
    first, last = state["offsets"][:-1].long(), state["offsets"][1:].long()
    at = first[:, None] + torch.arange(state["longest"], device=first.device)
    past = (at >= last[:, None])[..., None]
    at = at.clamp(max=a.shape[0] - 1)
    dw = torch.matmul(a[at].masked_fill(past, 0).transpose(1, 2).contiguous(), b[at].masked_fill(past, 0))
    return {"dw": dw if state["dw"] is None else state["dw"] + dw}


# ---- one pass ----------------------------------------------------------------------------------
def _own(state):
    import moe_grouped_gemm_e4m3_amd as dg
    case = state["case"]
    if case["op"] == "route":
        scores = dg.SCORES_SIGMOID if case["scores"] == "sigmoid" else dg.SCORES_SOFTMAX
        ids, weights = dg.moe_route(state["logits"], case["topk"], scores, bias=state["bias"], groups=case["groups"],
                                    topk_groups=case["topk_groups"], group_top=case["group_top"],
                                    renormalise=case["renorm"], scale=case["scale"])
        out = {"ids": ids, "weights": weights}
        if case["train"]:
            out["dlogits"] = dg.moe_route_backward(state["logits"], ids, state["dweights"], scores,
                                                   renormalise=case["renorm"], scale=case["scale"])
        return out
    if case["op"] == "dispatch":
        if case["masked"]:
            pos, row_pair, masked_m = dg.moe_layout_masked(state["ids"], case["G"], case["T"])
            out = {"pos": pos, "masked_m": masked_m}
        else:
            pos, row_pair, m_indices, offsets = dg.moe_layout_contiguous(state["ids"], case["G"])
            out = {"pos": pos, "m_indices": m_indices, "offsets": offsets}
        q, sf = dg.moe_dispatch_fp8(state["x"], pos, row_pair, q=state["q"], sf=state["sf"], ue8m0=case["ue8m0"])
        return out | {"q": q.view(torch.float8_e4m3fn), "sf": sf}
    if case["op"] == "combine":
        out = {"out": dg.moe_combine(state["y"], state["pos"], state["weights"])}
        if case["train"]:
            out["dy"], out["dweights"] = dg.moe_combine_backward(state["dout"], state["y"], state["pos"],
                                                                 state["row_pair"], state["weights"], dy=state["dy"])
        return out
    if case["G"] == 1 and case["topk"] == 1:
        a, sa = dg.cast_fp8_per_channel(state["dy"], ue8m0=case["ue8m0"])
        b, sb = dg.cast_fp8_per_channel(state["x"], ue8m0=case["ue8m0"])
        offsets = None
    else:
        offsets = state["offsets"]
        a, sa = dg.cast_fp8_per_channel(state["dy"], offsets=offsets, ue8m0=case["ue8m0"])
        b, sb = dg.cast_fp8_per_channel(state["x"], row_pair=state["row_pair"], topk=case["topk"], offsets=offsets,
                                        ue8m0=case["ue8m0"])
    return {"dw": dg.grouped_gemm_wgrad(a, sa, b, sb, offsets, c=state["dw"], ue8m0=case["ue8m0"])}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine,
            "wgrad": _plain_wgrad}[state["case"]["op"]](state)


# ---- in 64 bits --------------------------------------------------------------------------------
def _exact_fp8(x, ue8m0):
    """x [R, C] in 64 bits, runs of 128 along C -> (what the codes stand for, scales [R, C/128]). The scale and the
    quotient that is coded are 32-bit numbers by their definition; each is rounded once, from 64 bits."""
    runs = x.view(x.shape[0], -1, BLOCK)
    s = (runs.abs().max(2).values / torch.tensor(E4M3_MAX, dtype=torch.float64, device=x.device)).float().double()
    if ue8m0:
        s = torch.exp2(torch.ceil(torch.log2(s))).clamp(min=2.0 ** -126)
    r = torch.where(s[:, :, None] > 0, runs / s[:, :, None], torch.zeros_like(runs)).float().double()
    # steps of e4m3: 2^(floor(log2 |r|) - 3), 2^-9 below 2^-6; round() takes ties to even
    step = torch.exp2(torch.frexp(r).exponent.double().sub(1).clamp(min=-6) - 3)
    return torch.round(r / step).mul(step).clamp(-E4M3_MAX, E4M3_MAX).view(x.shape), s


def _exact_route(case, state):
    x = state["logits"].double()
    s = torch.sigmoid(x) if case["scores"] == "sigmoid" else torch.softmax(x, 1)
    key = s if state["bias"] is None else s + state["bias"].double()
    n = case["groups"]
    if n > 1:
        best = key.view(len(x), n, -1).sort(dim=2, descending=True).values[:, :, :case["group_top"]].sum(2)
        place = best.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
        key = key.masked_fill((place >= case["topk_groups"]).repeat_interleave(case["E"] // n, 1), -1e300)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :case["topk"]]
    top = torch.take_along_dim(s, ids, 1)
    S = top.sum(1, keepdim=True)
    c = case["scale"]
    out = {"ids": None, "weights": c * top / S if case["renorm"] else c * top}
    if case["train"]:
        # the Jacobian's two halves: from weights to scores, from scores to logits
        d = c * state["dweights"].double()
        dtop = d / S - (d * top).sum(1, keepdim=True) / S ** 2 if case["renorm"] else d
        if case["scores"] == "sigmoid":
            out["dlogits"] = torch.zeros_like(x).scatter_(1, ids, dtop * top * (1 - top))
        else:
            inner = (dtop * top).sum(1, keepdim=True)
            out["dlogits"] = (-s * inner).scatter_add_(1, ids, dtop * top)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, state)
    G, topk = case["G"], case["topk"]
    if case["op"] == "dispatch":
        q, s = _exact_fp8(state["x"].double(), case["ue8m0"])
        # the rows of each expert in the order of the choices, found by sorting (expert, choice)
        flat = state["ids"].long().view(-1)
        order = torch.argsort(torch.where(flat < G, flat, G), stable=True)
        count = torch.bincount(flat, minlength=G)[:G]
        order = order[:int(count.sum())]
        start = count.cumsum(0) - count
        width = state["q"].shape[1] if case["masked"] else None
        padded = -(-count // BLOCK) * BLOCK
        base = torch.arange(G, device=flat.device) * width if case["masked"] else padded.cumsum(0) - padded
        row = base[flat[order]] + torch.arange(len(order), device=flat.device) - start[flat[order]]
        full = torch.zeros((state["q"].numel() // case["H"], case["H"]), dtype=torch.float64, device=flat.device)
        scales = torch.zeros((len(full), case["H"] // BLOCK), dtype=torch.float64, device=flat.device)
        full[row], scales[row] = q[order // topk], s[order // topk]
        if case["masked"]:
            return {"pos": None, "masked_m": None, "q": full.view(state["q"].shape),
                    "sf": scales.view(G, width, -1).transpose(1, 2).contiguous()}
        return {"pos": None, "m_indices": None, "offsets": None, "q": full, "sf": scales.t().contiguous()}
    if case["op"] == "combine":
        # row by row of the layout, added up per token
        H = case["H"]
        pair = state["row_pair"].view(-1).long()
        used = pair >= 0
        token = pair[used] // topk
        w = state["weights"].double().view(-1)[pair[used]][:, None]
        y = state["y"].view(-1, H)[used].double()
        out = {"out": torch.zeros((case["T"], H), dtype=torch.float64, device=y.device).index_add_(0, token, y * w)}
        if case["train"]:
            g = state["dout"].double()[token]
            out["dy"] = torch.zeros(state["dy"].shape, dtype=torch.float64, device=y.device)
            out["dy"][used] = g * w
            out["dweights"] = torch.zeros(case["T"] * topk, dtype=torch.float64, device=y.device)
            out["dweights"][pair[used]] = (g * y).sum(1)
            out["dweights"] = out["dweights"].view(case["T"], topk)
        return out
    ends = state["offsets"].tolist()
    dw = torch.zeros((G, case["N"], case["K"]), dtype=torch.float64, device="cuda")
    for g in range(G):
        rows = slice(ends[g], ends[g + 1])
        if rows.start == rows.stop:
            continue
        if G == 1 and topk == 1:
            x, dy = (torch.zeros((rows.stop, t.shape[1]), dtype=torch.float64, device="cuda") for t in (state["x"], state["dy"]))
            x[:case["T"]], dy[:case["T"]] = state["x"].double(), state["dy"].double()
        else:
            pair = state["row_pair"][rows].long()
            x = state["x"].double()[pair.clamp(min=0) // topk] * (pair >= 0)[:, None]
            dy = state["dy"][rows].double()
        (qa, sa), (qb, sb) = (_exact_fp8(t.t().contiguous(), case["ue8m0"]) for t in (dy, x))
        a, b = qa * sa.repeat_interleave(BLOCK, 1), qb * sb.repeat_interleave(BLOCK, 1)
        dw[g] = a @ b.t()
    return {"dw": dw if state["dw"] is None else state["dw"].double() + dw}
