"""The layer's 8-bit and few-token operators as a user calls them, beside their plain forms.

Three operators:

* ``matmul``: a product in 8-bit integers with one scale per token and one per output channel, over one weight matrix or
  a stack of them (one per group of rows).  The tokens come in bf16 or fp32 and are quantised within the call.
* ``layer``: the whole mixture-of-experts layer with 8-bit integer experts (tokens and the intermediate quantised row by
  row, weights stored as codes with a scale per output channel).
* ``few``: the whole layer for at most 16 tokens, as a server runs it between two sampled tokens, with bf16, 8-bit or
  4-bit experts.

Quantising a row: scale = max|x| / 127, code = x * 127 / max|x| rounded to the nearest integer, ties to even; a row of
zeros has scale 0 and codes 0.  The 8-bit layer keeps its intermediate in bf16, as the layer does with other weights,
and quantises that.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------- cases

def _mm(name, T, N, K, groups=1, x="bf16", out="bf16"):
    return dict(name=name, op="matmul", T=T, N=N, K=K, groups=groups, x=x, out=out)


def _layer(name, op, T, d, F, E, k, weights, router="softmax_topk", n_group=1, topk_group=1, cf=0.0, act="swiglu",
           shared=0, skew=False):
    return dict(name=name, op=op, T=T, d=d, F=F, E=E, k=k, weights=weights, router=router, n_group=n_group,
                topk_group=topk_group, cf=cf, act=act, shared=shared, skew=skew)


def listed():
    return [
        # one token through a square projection: latency
        _mm("mm_one_token", 1, 4096, 4096),
        # an odd batch, odd output width, fp32 in and out
        _mm("mm_ragged_f32", 777, 2051, 1424, x="f32", out="f32"),
        # eight weight matrices, ragged groups of rows, one group empty, unused rows at the end
        _mm("mm_grouped", 2048, 4096, 2048, groups=8),
        # a prefill batch through the widest projection of the Mixtral-style layer
        _mm("mm_prefill", 4096, 14336, 4096),
        # a decode batch over many small experts
        _layer("layer_decode", "layer", 64, 2048, 768, 128, 8, "i8"),
        # ragged sizes, ReLU, drops
        _layer("layer_ragged", "layer", 333, 208, 144, 4, 2, "i8", cf=1.25, act="relu"),
        # the Switch-style batch: top-1, skewed experts, drops
        _layer("layer_switch", "layer", 8192, 2048, 8192, 64, 1, "i8", cf=1.0, act="relu", skew=True),
        # the Mixtral-style prefill, with a capacity
        _layer("layer_prefill", "layer", 4096, 4096, 14336, 8, 2, "i8", cf=1.25),
        # a small layer with grouped sigmoid routing and a shared expert: latency
        _layer("few_small", "few", 2, 448, 256, 32, 8, "bf16", "sigmoid_group", 8, 4, shared=256),
        # one token through the Mixtral-style layer
        _layer("few_one_token", "few", 1, 4096, 14336, 8, 2, "bf16"),
        # 16 sequences decoding through 4-bit experts
        _layer("few_q4", "few", 16, 2048, 768, 128, 8, "q4"),
        # four sequences decoding through the DeepSeek-style layer with 8-bit experts and its bf16 shared expert
        _layer("few_deepseek_i8", "few", 4, 7168, 2048, 256, 8, "i8", "sigmoid_group", 8, 4, shared=2048),
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("matmul", "layer", "few"))
    if op == "matmul":
        while True:
            c = dict(op=op, T=_log(rng, 1, 4096), N=_log(rng, 33, 14336), K=_log(rng, 64, 14336, 16),
                     groups=rng.choice((1, 1, 2, 5, 8)), x=rng.choice(("bf16", "bf16", "f32")),
                     out=rng.choice(("bf16", "bf16", "f32")))
            if c["T"] * c["N"] * c["K"] * c["groups"] <= 4096 * 14336 * 4096 and c["groups"] * c["N"] * c["K"] <= 1 << 29:
                return c
    while True:
        weights = "i8" if op == "layer" else rng.choice(("bf16", "i8", "q4"))
        step = 64 if weights == "q4" else 16
        router = rng.choice(("softmax_topk", "sigmoid_group"))
        n_group = rng.choice((2, 4, 8)) if router == "sigmoid_group" else 1
        per = rng.choice((4, 8, 16, 32))
        E = n_group * per if n_group > 1 else rng.choice((2, 6, 8, 40, 64, 100, 128))
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(8, E * topk_group // n_group))
        c = dict(op=op, T=_log(rng, 17, 4096) if op == "layer" else rng.randint(1, 16), d=_log(rng, 64, 4096, step),
                 F=_log(rng, 64, 8192, step), E=E, k=k, weights=weights, router=router, n_group=n_group,
                 topk_group=topk_group, cf=rng.choice((0.0, 1.0, 1.25, 2.0)),
                 act="swiglu" if weights == "q4" else rng.choice(("swiglu", "swiglu", "relu")),
                 shared=_log(rng, 64, 2048, 16) if op == "few" and weights != "q4" and rng.random() < 0.4 else 0,
                 skew=False)
        each = c["d"] * c["F"]
        if c["E"] * each <= 4e8 and (c["T"] * c["k"] * each <= 1.9e9 if op == "few" else c["E"] * _room(c) * each <= 6e11):
            return c


def _capacity(c):
    return max(1, int(c["T"] * c["k"] / c["E"] * c["cf"])) if c["cf"] else None


def _room(c):
    """Rows that one expert can hold."""
    return min(c["T"], _capacity(c) or c["T"])


def work(case):
    c = case
    if c["op"] == "matmul":
        size = {"bf16": 2, "f32": 4}
        nbytes = c["T"] * c["K"] * size[c["x"]] + c["groups"] * c["N"] * (c["K"] + 4) + c["T"] * c["N"] * size[c["out"]]
        return {"bytes": nbytes, "flops": 2 * c["T"] * c["N"] * c["K"]}
    T, d, F, E, k = c["T"], c["d"], c["F"], c["E"], c["k"]
    mats = 3 if c["act"] == "swiglu" else 2
    touched = E * (1 - (1 - k / E) ** T)          # experts that some token chooses, if all are chosen alike
    per_weight = {"bf16": 2.0, "i8": 1.0, "q4": 0.5625}[c["weights"]]
    nbytes = touched * mats * d * F * per_weight + E * d * 4 + 2 * T * d * 2 + 3 * c["shared"] * d * 2
    return {"bytes": nbytes, "flops": 2 * T * (k * mats * d * F + 3 * d * c["shared"] + d * E)}


# --------------------------------------------------------------------------------------------------------- inputs

def _codes(gen, rows, cols, std=0.02):
    """A drawn weight matrix as 8-bit codes with a scale per row."""
    w = torch.randn((rows, cols), generator=gen, device="cuda") * std
    top = w.abs().amax(1, keepdim=True)
    return torch.round(w * (127.0 / top)).to(torch.int8), (top / 127.0).squeeze(1)


def _stack_codes(gen, n, rows, cols):
    q = torch.empty((n, rows, cols), dtype=torch.int8, device="cuda")
    s = torch.empty((n, rows), device="cuda")
    for e in range(n):
        q[e], s[e] = _codes(gen, rows, cols)
    return q, s


def _stack_bf16(gen, n, rows, cols, std=0.02):
    w = torch.empty((n, rows, cols), dtype=torch.bfloat16, device="cuda")
    for e in range(n):
        w[e] = torch.randn((rows, cols), generator=gen, device="cuda") * std
    return w


def _stack_q4(gen, n, rows, cols):
    """Codes 0..15, eight per int32 word from the low bits up; a bf16 scale and bias per 64 of them."""
    bits = torch.randint(-2 ** 31, 2 ** 31, (n, rows, cols // 8), generator=gen, device="cuda", dtype=torch.int64)
    s = (torch.randn((n, rows, cols // 64), generator=gen, device="cuda") * 0.0005 + 0.002).to(torch.bfloat16)
    return bits.to(torch.int32), s, (s.float() * -7.5).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case=c)
    if c["op"] == "matmul":
        x = torch.randn((c["T"], c["K"]), generator=gen, device="cuda")
        x *= torch.exp(0.5 * torch.randn((c["T"], 1), generator=gen, device="cuda"))     # rows of unlike size
        state["x"] = x.to(DTYPES[c["x"]])
        state["wq"], state["ws"] = _stack_codes(gen, c["groups"], c["N"], c["K"])
        state["out"] = torch.zeros((c["T"], c["N"]), dtype=DTYPES[c["out"]], device="cuda")
        state["offsets"] = None
        if c["groups"] > 1:
            cut = torch.sort(torch.randint(0, c["T"] + 1, (c["groups"],), generator=gen, device="cuda")).values
            cut[1] = cut[0]                       # one group is empty; the rows behind the last cut belong to none
            state["offsets"] = torch.cat([cut.new_zeros(1), cut]).to(torch.int32)
        return state
    T, d, F, E = c["T"], c["d"], c["F"], c["E"]
    state["x"] = torch.randn((T, d), generator=gen, device="cuda").to(torch.bfloat16)
    state["w_router"] = torch.randn((E, d), generator=gen, device="cuda") * 0.02
    state["bias"] = None
    if c["skew"]:
        state["bias"] = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -1.1
    elif c["router"] == "sigmoid_group":
        state["bias"] = (torch.rand((E,), generator=gen, device="cuda") * 2 - 1) * 0.05
    w = state["w"] = {}
    for i, (rows, cols) in (("1", (F, d)), ("2", (F, d)), ("3", (d, F))):
        if i == "2" and c["act"] == "relu":
            continue
        if c["weights"] == "bf16":
            w["w" + i] = _stack_bf16(gen, E, rows, cols)
        elif c["weights"] == "i8":
            w["w" + i], w["s" + i] = _stack_codes(gen, E, rows, cols)
        else:
            w["w" + i], w["s" + i], w["b" + i] = _stack_q4(gen, E, rows, cols)
    if c["shared"]:
        for i, (rows, cols) in (("1", (c["shared"], d)), ("2", (c["shared"], d)), ("3", (d, c["shared"]))):
            w["ws" + i] = _stack_bf16(gen, 1, rows, cols)[0]
    return state


# ---------------------------------------------------------------------------------------------- the framework's calls

def _own_matmul(state):
    from mixture_experts_layer_41_b200 import api
    c = state["case"]
    if "ws8" not in state:                        # what a program keeps: the codes' buffer and a workspace
        state["xq"] = torch.empty((c["T"], c["K"]), dtype=torch.int8, device="cuda")
        state["xs"] = torch.empty((c["T"],), device="cuda")
        n = api.moe_quantized_matmul_workspace_size(c["groups"], c["T"], c["N"], c["K"])
        state["ws8"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
    api.moe_quantize_rows(state["x"], state["xq"], state["xs"])
    api.moe_quantized_matmul(state["xq"], state["xs"], state["wq"], state["ws"], state["out"], state["ws8"],
                             group_offsets=state["offsets"])
    return state["out"]


def _own_layer(state):
    from mixture_experts_layer_41_b200 import api
    c = state["case"]
    if "layer" not in state:                      # what a program keeps: the layer with its weights and workspace
        cfg = api.make_config(num_tokens=c["T"], hidden=c["d"], intermediate=c["F"], num_experts=c["E"], top_k=c["k"],
                              router=c["router"], routed_scaling=2.5 if c["router"] == "sigmoid_group" else 1.0,
                              n_group=c["n_group"], topk_group=c["topk_group"], capacity_factor=c["cf"], act=c["act"],
                              weight_dtype={"bf16": "bf16", "i8": "i8_channel", "q4": "q4_affine_g64"}[c["weights"]],
                              shared_intermediate=c["shared"])
        state["layer"] = api.MoELayer(cfg, state["w_router"], state["w"], router_bias=state["bias"])
    layer = state["layer"]
    o = layer.forward_few(state["x"]) if c["op"] == "few" else layer.forward(state["x"])
    return dict(out=o.out, ids=o.topk_ids, weights=o.topk_w, kept=o.kept_counts, prob_sum=o.prob_sum)


# --------------------------------------------------------------------------------------------------- plain forms

def _quantize(x):
    """Codes (as fp32 values) and scales of the last axis; in 64 bits, where a value may lie next to a border."""
    top = x.abs().amax(-1, keepdim=True)
    wide = top.double()
    q = torch.round(x.double() * 127.0 / torch.where(wide > 0, wide, 1.0)).float()
    return q, top.float() / 127.0


def _plain_matmul(state):
    x, out = state["x"].float(), state["out"]
    q, s = _quantize(x)
    y = torch.matmul(q, state["wq"].float().transpose(1, 2)) * s * state["ws"][:, None, :]     # [groups, T, N]
    if state["offsets"] is None:
        return y[0].to(out.dtype)
    rows = torch.arange(x.shape[0], device="cuda")
    group = torch.searchsorted(state["offsets"][1:].contiguous(), rows.to(torch.int32), right=True)
    valid = group < y.shape[0]
    picked = y[group.clamp(max=y.shape[0] - 1), rows].to(out.dtype)
    return torch.where(valid[:, None], picked, out)


def _route(state):
    """Chosen experts, their weights and every expert's summed probability, in 64 bits (ids turn on small gaps)."""
    c = state["case"]
    logits = state["x"].double() @ state["w_router"].double().t()
    bias = 0.0 if state["bias"] is None else state["bias"].double()
    if c["router"] == "softmax_topk":
        p = torch.softmax(logits + bias, 1)
        rank = p
    else:
        p = torch.sigmoid(logits)
        rank = p + bias
        g = rank.view(c["T"], c["n_group"], -1)
        best = torch.sort(torch.sort(g, dim=2, descending=True).values[:, :, :2].sum(2), dim=1, descending=True,
                          stable=True).indices[:, :c["topk_group"]]
        live = torch.zeros(g.shape[:2], dtype=torch.bool, device="cuda").scatter_(1, best, True)
        rank = torch.where(live[:, :, None], g, -math.inf).view(c["T"], -1)
    ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * (2.5 if c["router"] == "sigmoid_group" else 1.0)
    return ids, w, p.sum(0)


def _places(c, ids):
    """Each slot's place among its expert's slots in token order, whether it is kept, and the kept counts."""
    flat = ids.reshape(-1)
    hot = torch.zeros((flat.numel(), c["E"]), dtype=torch.int32, device="cuda").scatter_(1, flat[:, None], 1)
    place = torch.cumsum(hot, 0, dtype=torch.int32).gather(1, flat[:, None]).squeeze(1) - 1
    room = _capacity(c) or c["T"]
    return place, place < room, hot.sum(0).clamp(max=room).to(torch.int32)


def _activate(c, gate, up):
    return torch.relu(gate) if c["act"] == "relu" else gate * torch.sigmoid(gate) * up


def _unpack(w, i, at):
    """Chosen 4-bit matrices in fp32: scale * code + bias."""
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    codes = ((w["w" + i][at][..., None] >> shift) & 15).flatten(-2).float()
    s, b = (w[k + i][at].float().repeat_interleave(64, dim=-1) for k in "sb")
    return s * codes + b


def _product(c, w, i, at, x):
    """x [n, rows, K] times the chosen experts' matrices."""
    if c["weights"] == "i8":
        q, s = _quantize(x)
        return torch.matmul(q, w["w" + i][at].float().transpose(1, 2)) * s * w["s" + i][at][:, None, :]
    m = w["w" + i][at].float() if c["weights"] == "bf16" else _unpack(w, i, at)
    return torch.matmul(x, m.transpose(1, 2))


def _experts(c, w, at, x):
    gate = _product(c, w, "1", at, x)
    h = _activate(c, gate, _product(c, w, "2", at, x) if c["act"] == "swiglu" else None)
    if c["weights"] == "i8":
        h = h.to(torch.bfloat16).float()
    return _product(c, w, "3", at, h)


def _plain_layer(state):
    c, w = state["case"], state["w"]
    T, d, E, k = c["T"], c["d"], c["E"], c["k"]
    x = state["x"].float()
    ids, wts, prob_sum = _route(state)
    place, keep, kept = _places(c, ids)
    flat = ids.reshape(-1)
    if c["op"] == "few":                          # a few tokens: every slot with a copy of its expert
        y = _experts(c, w, flat, x.repeat_interleave(k, 0)[:, None, :]).squeeze(1)
    else:                                         # every expert with room for its rows
        room = _room(c)
        rows = torch.where(keep, flat * room + place, E * room)
        xp = torch.zeros((E * room + 1, d), device="cuda").index_copy_(0, rows, x.repeat_interleave(k, 0))
        y = _experts(c, w, slice(None), xp[:-1].view(E, room, d)).reshape(E * room, d)[rows.clamp(max=E * room - 1)]
    y = torch.where(keep[:, None], y, 0.0).view(T, k, d)
    out = (wts.float()[:, :, None] * y).sum(1)
    if c["shared"]:
        g, u = x @ w["ws1"].float().t(), x @ w["ws2"].float().t()
        out = out + (g * torch.sigmoid(g) * u) @ w["ws3"].float().t()
    return dict(out=out.to(torch.bfloat16), ids=ids.to(torch.int32), weights=wts.float(), kept=kept, prob_sum=prob_sum.float())


def run(state):
    if state["case"]["op"] == "matmul":
        if own:
            return _own_matmul(state)
        return _plain_matmul(state)
    if own:
        return _own_layer(state)
    return _plain_layer(state)


# -------------------------------------------------------------------------------------------- 64-bit evaluation

def _exact_codes(x):
    """x [rows, K] in float64: the values that the codes stand for."""
    top = x.abs().max(1).values
    step = (top / 127.0).unsqueeze(1)
    codes = torch.round(torch.where(step > 0, x * 127.0, x) / torch.where(step > 0, top.unsqueeze(1), 1.0))
    return codes * step


def exact(case, seed):
    c = case
    state = prepare(case, seed)
    if c["op"] == "matmul":
        x = _exact_codes(state["x"].double())
        out = state["out"].double()
        ends = [0, c["T"]] if state["offsets"] is None else state["offsets"].tolist()
        for g in range(c["groups"]):
            a, b = ends[g], ends[g + 1]
            out[a:b] = x[a:b] @ (state["wq"][g].double() * state["ws"][g].double()[:, None]).t()
        return out
    T, E, k, w = c["T"], c["E"], c["k"], state["w"]
    x = state["x"].double()
    score = torch.einsum("td,ed->te", x, state["w_router"].double())
    shift = torch.zeros(E, dtype=torch.float64, device="cuda") if state["bias"] is None else state["bias"].double()
    if c["router"] == "softmax_topk":
        e = torch.exp(score + shift - (score + shift).max(1, keepdim=True).values)
        prob = e / e.sum(1, keepdim=True)
        key = prob.clone()
    else:
        prob = 1.0 / (1.0 + torch.exp(-score))
        key = prob + shift
        size = E // c["n_group"]
        for t in range(T):
            rows = key[t].view(c["n_group"], size)
            marks = torch.topk(rows, 2, dim=1).values.sum(1).tolist()
            order = sorted(range(c["n_group"]), key=lambda g: (-marks[g], g))
            for g in order[c["topk_group"]:]:
                key[t, g * size:(g + 1) * size] = -math.inf
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    wts = torch.gather(prob, 1, ids)
    wts = wts / wts.sum(1, keepdim=True)
    if c["router"] == "sigmoid_group":
        wts = wts * 2.5
    room = _capacity(c)
    out = torch.zeros((T, c["d"]), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if room is not None:
            t, j = t[:room], j[:room]
        if not t.numel():
            continue
        m = {}
        for i in "123":
            if "w" + i not in w:
                continue
            if c["weights"] == "bf16":
                m[i] = w["w" + i][e].double()
            elif c["weights"] == "i8":
                m[i] = w["w" + i][e].double() * w["s" + i][e].double()[:, None]
            else:
                words = w["w" + i][e].to(torch.int64) & 0xFFFFFFFF
                code = torch.stack([(words >> (4 * n)) % 16 for n in range(8)], dim=2).reshape(words.shape[0], -1, 64)
                m[i] = (code.double() * w["s" + i][e].double()[:, :, None] + w["b" + i][e].double()[:, :, None]).flatten(1)
        a = _exact_codes(x[t]) if c["weights"] == "i8" else x[t]
        g = a @ m["1"].t()
        h = g.clamp(min=0) if c["act"] == "relu" else g / (1 + torch.exp(-g)) * (a @ m["2"].t())
        if c["weights"] == "i8":
            h = _exact_codes(h.to(torch.bfloat16).double())
        out.index_add_(0, t, (h @ m["3"].t()) * wts[t, j][:, None])
    if c["shared"]:
        s1, s2, s3 = (w["ws" + i].double() for i in "123")
        g = x @ s1.t()
        out += (g / (1 + torch.exp(-g)) * (x @ s2.t())) @ s3.t()
    return dict(out=out, ids=None, weights=wts, kept=None, prob_sum=prob.sum(0))
