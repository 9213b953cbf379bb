"""The routed experts beside the shared expert, and the products in 8 bits they are made of: cases to measure.

Three operators of ``moe_shared_expert_gb300``:

* ``route``: ``moe_route``, from the router's logits to each token's experts and their weights;
* ``linear``: ``fp8_block_linear``, y = x W^T with W in e4m3 and one scale for each block of 128 x 128, x rounded to
  e4m3 with one scale for each token and block of 128;
* ``experts``: ``moe_experts_forward``, the weighted sum of each token's routed SwiGLU experts (weights as in
  ``linear``) plus the shared expert's output.

``run`` computes them in their plain form (elementary torch operations in 32 bits, rounded once at the end) or, where
``own`` is true, with the framework's calls.

Rounding to e4m3 (``B`` a block of x): a = max(max |B|, 2^-100), s = a / 448, q = e4m3(448 B / a), B ~ q s.  For B
in bf16 a quotient that is a tie of e4m3 is exact in 32 bits and every other one is far from a tie, so q has one value.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
MASKED_FROM = -3.3895313892515355e38  # the lowest finite bf16: a logit at or below it takes its expert out of the choice


# ------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one generated token at the router: latency only
        {"name": "route one token", "op": "route", "T": 1, "E": 256, "k": 8, "scoring": "sigmoid", "bias": True,
         "n_group": 8, "topk_group": 4, "renormalise": True, "scale": 2.5, "dtype": "f32", "masked": False},
        # a decode batch, logits in bf16, some experts closed to some tokens
        {"name": "route decode batch", "op": "route", "T": 64, "E": 128, "k": 4, "scoring": "softmax", "bias": False,
         "n_group": 1, "topk_group": 1, "renormalise": True, "scale": 1.0, "dtype": "bf16", "masked": True},
        # the prompt of the prefill workload
        {"name": "route prompt", "op": "route", "T": 8192, "E": 384, "k": 8, "scoring": "sigmoid", "bias": True,
         "n_group": 1, "topk_group": 1, "renormalise": True, "scale": 2.0, "dtype": "f32", "masked": False},
        # many packed prompts, groups of an odd size, softmax scores with a bias
        {"name": "route packed prompts", "op": "route", "T": 65536, "E": 160, "k": 6, "scoring": "softmax",
         "bias": True, "n_group": 8, "topk_group": 3, "renormalise": False, "scale": 16.0, "dtype": "bf16",
         "masked": False},
        # the merged latent projection (2112 x 7168) for one token: the weights are read once, little else happens
        {"name": "linear one token 2112x7168", "op": "linear", "T": 1, "N": 2112, "K": 7168},
        # the shared expert's gate_up at the decode batch
        {"name": "linear decode 12288x7168", "op": "linear", "T": 64, "N": 12288, "K": 7168},
        # a short prompt against sizes that divide by nothing
        {"name": "linear ragged 2111x6100", "op": "linear", "T": 333, "N": 2111, "K": 6100},
        # the shared expert's gate_up over the whole prompt
        {"name": "linear prompt 12288x7168", "op": "linear", "T": 8192, "N": 12288, "K": 7168},
        # one generated token through its eight experts
        {"name": "experts one token", "op": "experts", "T": 1, "E": 32, "total": 32, "k": 8, "H": 7168, "I": 2048,
         "shared": True},
        # a decode batch on one rank that holds a quarter of the experts: most pairs belong to other ranks
        {"name": "experts decode quarter", "op": "experts", "T": 64, "E": 32, "total": 128, "k": 8, "H": 7168,
         "I": 2048, "shared": True},
        # small experts whose sizes divide by nothing
        {"name": "experts ragged", "op": "experts", "T": 300, "E": 10, "total": 10, "k": 3, "H": 1000, "I": 700,
         "shared": False},
        # a prompt: about a thousand tokens for each expert
        {"name": "experts prompt", "op": "experts", "T": 4096, "E": 32, "total": 32, "k": 8, "H": 7168, "I": 2048,
         "shared": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "linear", "experts"])
    if op == "route":
        n_group = rng.choice([1, 1, 4, 8])
        E = n_group * rng.randint(max(4, 16 // n_group), 512 // n_group)
        topk_group = rng.randint(max(1, n_group // 2), n_group) if n_group > 1 else 1
        T = min(_log_int(rng, 1, 65536), 65536 * 160 // E)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(10, topk_group * (E // n_group))),
                "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "n_group": n_group,
                "topk_group": topk_group, "renormalise": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]),
                "dtype": rng.choice(["f32", "bf16"]), "masked": rng.random() < 0.3}
    if op == "linear":
        N, K = _log_int(rng, 256, 12288), _log_int(rng, 512, 7168)
        if rng.random() < 0.6:  # sizes as models have them
            N, K = max(BLOCK, N // 64 * 64), max(BLOCK, K // 128 * 128)
        return {"op": op, "T": _log_int(rng, 1, 8192), "N": N, "K": K}
    total = rng.choice([8, 16, 32, 64, 128])
    E = min(32, total)
    H, I = _log_int(rng, 768, 7168), _log_int(rng, 384, 2048)
    if rng.random() < 0.6:
        H, I = H // 128 * 128, I // 128 * 128
    return {"op": op, "T": _log_int(rng, 1, 4096), "E": E, "total": total, "k": rng.randint(1, 8), "H": H, "I": I,
            "shared": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------------ the inputs

def _pad16(n):
    return (n + 15) // 16 * 16


def _blocks(n):
    return -(-n // BLOCK)


def _weights(shape, gen, sigma):
    """A weight [.., N, K] in e4m3 (rows of a pitch of 16 bytes) and its scales [.., N / 128, K / 128]."""
    *lead, N, K = shape
    nb, kb = _blocks(N), _blocks(K)
    w = torch.zeros(*lead, nb * BLOCK, kb * BLOCK, dtype=torch.bfloat16, device="cuda")
    w[..., :N, :K].normal_(0.0, sigma, generator=gen)
    w = w.view(*lead, nb, BLOCK, kb, BLOCK)
    s = w.abs().amax(dim=(-3, -1)).float().clamp_min(AMAX_FLOOR) / E4M3_MAX
    w = (w / s[..., :, None, :, None]).to(torch.float8_e4m3fn).view(*lead, nb * BLOCK, kb * BLOCK)
    q = torch.zeros(*lead, N, _pad16(K), dtype=torch.uint8, device="cuda")
    q[..., :K] = w[..., :N, :K].view(torch.uint8)
    return q.view(torch.float8_e4m3fn)[..., :K], s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, T = case["op"], case["T"]
    st = {"case": case}

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * sigma

    if op == "route":
        E = case["E"]
        # a router's logits: a spread of about 1.5 and experts that are more popular than others
        logits = normal(T, E, sigma=1.5) + normal(E, sigma=0.5)
        if case["masked"]:  # a tenth of the experts closed to a token, and now and then all of them
            logits = logits.masked_fill(torch.rand(T, E, generator=gen, device="cuda") < 0.1, -math.inf)
            logits[torch.rand(T, generator=gen, device="cuda") < 0.02] = -math.inf
        st["logits"] = logits.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        st["bias"] = normal(E, sigma=0.05) if case["bias"] else None
    elif op == "linear":
        N, K = case["N"], case["K"]
        st["x"] = normal(T, K).to(torch.bfloat16)
        st["w"], st["s"] = _weights((N, K), gen, 1 / math.sqrt(K))
    else:
        E, H, I, k = case["E"], case["H"], case["I"], case["k"]
        st["x"] = normal(T, H).to(torch.bfloat16)
        scores = torch.sigmoid(normal(T, case["total"], sigma=1.5) + normal(case["total"], sigma=0.5))
        top = scores.topk(k, dim=1)
        st["ids"] = top.indices.to(torch.int32)
        st["weights"] = top.values / top.values.sum(1, keepdim=True)
        # gate rows, then up rows, each with blocks of its own
        w, s = _weights((E, 2, I, H), gen, 1 / math.sqrt(H))
        st["w_gate_up"], st["s_gate_up"] = w.flatten(1, 2), s.flatten(1, 2)
        st["w_down"], st["s_down"] = _weights((E, H, I), gen, 1 / math.sqrt(I))
        st["shared"] = normal(T, H, sigma=0.5).to(torch.bfloat16) if case["shared"] else None
        st["first"] = (case["total"] - E) // 2  # this rank's experts lie in the middle of all of them
    return st


# ------------------------------------------------------------------------------------------------ the plain forms

def _rounded(x):
    """x [.., K] in 32 bits, rounded to e4m3 in blocks of 128 along K: the values q s that it stands for."""
    K = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    q = (b * (E4M3_MAX / 512) / a * 512).to(torch.float8_e4m3fn).float()  # 448 B / a without overflow
    return (q * (a / E4M3_MAX)).flatten(-2)[..., :K]


def _spread(s, N, K):
    """Block scales [.., N / 128, K / 128] for each element [.., N, K]."""
    return s.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]


def _plain_route(st):
    c, k = st["case"], st["case"]["k"]
    l = st["logits"].float()
    open_ = l > MASKED_FROM
    l = l.masked_fill(~open_, -math.inf)
    if c["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
        # the sum in 64 bits, rounded to 32: the choice compares scores, so they may not depend on an order of summation
        score = e / e.double().sum(1, keepdim=True).float().clamp_min(1e-30)
    choice = score if st["bias"] is None else score + st["bias"]
    choice = choice.masked_fill(~open_, -math.inf)
    G = c["n_group"]
    if G > 1:
        per = choice.view(choice.shape[0], G, -1).sort(dim=2, descending=True).values[:, :, :2]
        second = per[:, :, 1].masked_fill(per[:, :, 1] == -math.inf, 0.0)  # a closed expert adds nothing
        group = per[:, :, 0] + second if c["bias"] else per[:, :, 0]
        best = group.sort(dim=1, descending=True, stable=True).indices[:, : c["topk_group"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, best, True)
        choice = choice.masked_fill(~keep.repeat_interleave(c["E"] // G, 1), -math.inf)
    top = choice.sort(dim=1, descending=True, stable=True)
    ids, found = top.indices[:, :k], top.values[:, :k] > -math.inf
    w = score.gather(1, ids) * found
    if c["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return {"ids": torch.where(found, ids, -1).to(torch.int32), "weights": w * c["scale"]}


def _plain_linear(st):
    N, K = st["w"].shape
    return {"y": (_rounded(st["x"].float()) @ (st["w"].float() * _spread(st["s"], N, K)).t()).to(torch.bfloat16)}


def _plain_experts(st):
    E, H, I = st["case"]["E"], st["case"]["H"], st["case"]["I"]
    x = _rounded(st["x"].float())
    wg = st["w_gate_up"].float().view(E, 2, I, H) * _spread(st["s_gate_up"].view(E, 2, -1, _blocks(H)), I, H)
    gu = x @ wg.flatten(1, 2).transpose(1, 2)                                     # [E, T, 2 I]: every expert on every token
    g, u = gu[..., :I], gu[..., I:]
    h = _rounded(g / (1.0 + torch.exp(-g)) * u)
    o = h @ (st["w_down"].float() * _spread(st["s_down"], H, I)).transpose(1, 2)  # [E, T, H]
    chosen = st["ids"][:, :, None] == torch.arange(E, device="cuda") + st["first"]
    y = torch.einsum("te,eth->th", (chosen * st["weights"][:, :, None]).sum(1), o)
    return {"y": (y if st["shared"] is None else st["shared"].float() + y).to(torch.bfloat16)}


def _kept(st):
    """The workspace and the outputs that a program keeps from pass to pass."""
    if "workspace" not in st:
        import moe_shared_expert_gb300 as mse
        c, T = st["case"], st["case"]["T"]
        if c["op"] == "route":
            st["workspace"] = None
            st["ids"] = torch.empty(T, c["k"], dtype=torch.int32, device="cuda")
            st["weights"] = torch.empty(T, c["k"], dtype=torch.float32, device="cuda")
        elif c["op"] == "linear":
            st["workspace"] = mse.new_fp8_linear_workspace(T, c["N"], c["K"])
            st["y"] = torch.empty(T, c["N"], dtype=torch.bfloat16, device="cuda")
        else:
            st["workspace"] = mse.new_moe_workspace(T, c["k"], c["E"], c["H"], c["I"])
            st["y"] = torch.empty(T, c["H"], dtype=torch.bfloat16, device="cuda")
    return st["workspace"]


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"route": _plain_route, "linear": _plain_linear, "experts": _plain_experts}[c["op"]](st)
    import moe_shared_expert_gb300 as mse
    ws = _kept(st)
    if c["op"] == "route":
        ids, w = mse.moe_route(st["logits"], c["k"], scoring=c["scoring"], bias=st["bias"], n_group=c["n_group"],
                               topk_group=c["topk_group"], group_top=2 if c["bias"] else 1,
                               renormalise=c["renormalise"], scale=c["scale"], ids=st["ids"], weights=st["weights"])
        return {"ids": ids, "weights": w}
    if c["op"] == "linear":
        return {"y": mse.fp8_block_linear(st["x"], st["w"], st["s"], y=st["y"], workspace=ws)}
    return {"y": mse.moe_experts_forward(st["x"], st["ids"], st["weights"], st["w_gate_up"], st["s_gate_up"],
                                         st["w_down"], st["s_down"], first_expert=st["first"], shared=st["shared"],
                                         y=st["y"], workspace=ws)}


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        E, k = case["E"], case["k"]
        # logits and bias in, ids and weights out; a score and a comparison for each choice of each logit
        return {"bytes": T * E * (4 if case["dtype"] == "f32" else 2) + 4 * E * case["bias"] + 8 * T * k,
                "flops": T * E * (4 + k)}
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": N * K + 4 * _blocks(N) * _blocks(K) + 2 * T * (K + N), "flops": 2 * T * N * K}
    E, H, I, k, total = (case[n] for n in ("E", "H", "I", "k", "total"))
    pairs = T * min(k, total) * E / total                             # expected to stay on this rank
    read = E * (1 - (1 - min(k, total) / total) ** T)                 # experts that expect a token
    expert = 3 * H * I + 4 * 3 * _blocks(H) * _blocks(I)
    return {"bytes": read * expert + T * H * (4 + 2 * case["shared"]) + 8 * T * k, "flops": 6 * pairs * H * I}


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits

def _e4m3_64(v):
    """The nearest e4m3 value (ties to even) of v in 64 bits, |v| < 464: 3 fraction bits, exponents from -6."""
    exponent = (torch.frexp(v).exponent - 1).clamp_min(-6)
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.round(v / step) * step


def _rounded_64(x):
    out = torch.empty_like(x)
    for k in range(0, x.shape[-1], BLOCK):
        b = x[..., k:k + BLOCK]
        a = b.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
        out[..., k:k + BLOCK] = _e4m3_64(E4M3_MAX * b / a) * (a / E4M3_MAX)
    return out


def _weight_64(w, s):
    out = w.double()
    for n in range(s.shape[0]):
        for k in range(s.shape[1]):
            out[n * BLOCK:(n + 1) * BLOCK, k * BLOCK:(k + 1) * BLOCK] *= s[n, k].double()
    return out


def _exact_route(st):
    c, E, k = st["case"], st["case"]["E"], st["case"]["k"]
    l = st["logits"].double()
    closed = ~(l > MASKED_FROM)
    l = torch.where(closed, torch.full_like(l, -math.inf), l)
    if c["scoring"] == "sigmoid":
        score = torch.sigmoid(l)
    else:
        score = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
    # scores and choices are held in 32 bits, so that is where ties are
    choice = score.float() + (st["bias"] if st["bias"] is not None else 0.0)
    choice[closed] = -math.inf
    if c["n_group"] > 1:
        size = E // c["n_group"]
        parts = [choice[:, g * size:(g + 1) * size] for g in range(c["n_group"])]
        if c["bias"]:
            two = torch.stack([p.topk(2, 1).values for p in parts], 1)
            of = two[:, :, 0] + torch.where(two[:, :, 1] == -math.inf, 0.0, two[:, :, 1])
        else:
            of = torch.stack([p.amax(1) for p in parts], 1)
        order = torch.argsort(of, dim=1, descending=True, stable=True)
        rank = torch.argsort(order, dim=1)
        for g, p in enumerate(parts):
            p[rank[:, g] >= c["topk_group"]] = -math.inf
    ids = torch.argsort(choice, dim=1, descending=True, stable=True)[:, :k]
    w = torch.where(choice.gather(1, ids) == -math.inf, 0.0, score.gather(1, ids))
    if c["renormalise"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return {"ids": None, "weights": w * c["scale"]}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(st)
    x = _rounded_64(st["x"].double())
    if case["op"] == "linear":
        return {"y": x @ _weight_64(st["w"], st["s"]).t()}
    I, nb = case["I"], _blocks(case["I"])
    y = torch.zeros_like(x) if st["shared"] is None else st["shared"].double()
    for e in range(case["E"]):
        token, slot = torch.nonzero(st["ids"] == e + st["first"], as_tuple=True)
        if not token.numel():
            continue
        rows = x[token]
        w, s = st["w_gate_up"][e], st["s_gate_up"][e]
        g, u = rows @ _weight_64(w[:I], s[:nb]).t(), rows @ _weight_64(w[I:], s[nb:]).t()
        h = _rounded_64(torch.nn.functional.silu(g) * u)
        o = h @ _weight_64(st["w_down"][e], st["s_down"][e]).t()
        y.index_add_(0, token, o * st["weights"][token, slot].double()[:, None])
    return {"y": y}
