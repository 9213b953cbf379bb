"""Tokens sorted by expert and back, with their gradients, and products in 8-bit integers: cases to measure.

Five operators of ``moe_shared_expert_gb300``:

* ``sort``: ``moe_sort``, each token's row copied to the rows of its experts, experts one after another, pairs of a token
  and an expert in their order within each;
* ``unsort``: ``moe_unsort``, y[t] = base[t] + sum_j weights[t, j] rows[place[t, j]];
* ``gradient``: ``moe_unsort_backward`` (drows[place[t, j]] = weights[t, j] dy[t], dweights[t, j] = <rows[place[t, j]], dy[t]>)
  and ``moe_sort_backward`` (dx[t] = sum_j drows[place[t, j]]) of what the experts made of the first one's rows;
* ``linear``: ``int8_linear``, y = x W^T with W in 8-bit integers and one scale for each of its rows, x rounded to 8-bit
  integers with one scale for each token;
* ``grouped``: ``int8_grouped_matmul``, the same product of sorted rows with their experts' weights; with ``swiglu`` the rows
  are ``int8_quantise`` of silu(gate) up.

``run`` computes them in their plain form (elementary torch operations in 32 bits, rounded once at the end) or, where ``own``
is true, with the framework's calls.

Rounding to 8-bit integers (``r`` a row of x): a = max(max |r|, 2^-100), s = a / 127, q = rint(127 r / a), r ~ q s.  For r in
bf16 a quotient halfway between two integers is exact in 32 bits and every other one is far from that, so q has one value.
"""
import math

import torch

own = False

LEVELS = 127.0
AMAX_FLOOR = 2.0 ** -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}


# ------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one generated token to its experts: latency only
        {"name": "sort one token", "op": "sort", "T": 1, "E": 32, "total": 32, "k": 8, "H": 7168, "dtype": "bf16"},
        # the prompt of the prefill workload, in 8-bit integers with their scales, on a rank that holds half of the experts
        {"name": "sort prompt", "op": "sort", "T": 8192, "E": 64, "total": 128, "k": 8, "H": 7168, "dtype": "int8"},
        # a decode batch on one rank that holds a quarter of the experts, on top of the shared expert's output
        {"name": "unsort decode quarter", "op": "unsort", "T": 64, "E": 32, "total": 128, "k": 8, "H": 7168, "dtype": "bf16",
         "base": True},
        # a prompt whose experts are all here
        {"name": "unsort prompt", "op": "unsort", "T": 4096, "E": 32, "total": 32, "k": 8, "H": 7168, "dtype": "bf16",
         "base": True},
        # a short training batch in 32 bits, sizes that divide by nothing
        {"name": "gradient ragged", "op": "gradient", "T": 333, "E": 10, "total": 10, "k": 3, "H": 1001, "dtype": "f32"},
        # a training step's tokens
        {"name": "gradient prompt", "op": "gradient", "T": 4096, "E": 32, "total": 32, "k": 8, "H": 7168, "dtype": "bf16"},
        # the merged latent projection (2112 x 7168) for one token: the weights are read once, little else happens
        {"name": "linear one token 2112x7168", "op": "linear", "T": 1, "N": 2112, "K": 7168},
        # the shared expert's gate_up at the decode batch
        {"name": "linear decode 12288x7168", "op": "linear", "T": 64, "N": 12288, "K": 7168},
        # the shared expert's gate_up over the whole prompt
        {"name": "linear prompt 12288x7168", "op": "linear", "T": 8192, "N": 12288, "K": 7168},
        # one generated token through the gate and up weights of its eight experts
        {"name": "grouped one token", "op": "grouped", "T": 1, "E": 32, "total": 32, "k": 8, "N": 4096, "K": 7168,
         "swiglu": False},
        # small experts whose sizes divide by nothing: activation and down projection
        {"name": "grouped ragged swiglu", "op": "grouped", "T": 300, "E": 10, "total": 10, "k": 3, "N": 1000, "K": 700,
         "swiglu": True},
        # a prompt's down projection after the activation: about a thousand tokens for each expert
        {"name": "grouped prompt swiglu", "op": "grouped", "T": 2048, "E": 16, "total": 16, "k": 8, "N": 7168, "K": 2048,
         "swiglu": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _experts(rng):
    total = rng.choice([8, 16, 32, 64, 128, 256])
    return {"E": total // rng.choice([1, 1, 2, 4]), "total": total, "k": rng.randint(1, 8)}


def _busy(case):
    """A rank that would hardly see a pair holds all experts (as far as they are at most 32) instead."""
    if case["T"] * case["k"] * case["E"] < 4 * case["total"]:
        case["total"] = case["E"] = max(8, min(case["total"], 32))
    return case


def draw(rng):
    op = rng.choice(["sort", "unsort", "gradient", "linear", "grouped"])
    if op in ("sort", "unsort", "gradient"):
        H = _log_int(rng, 256, 7168)
        if rng.random() < 0.6:  # sizes as models have them
            H = max(256, H // 128 * 128)
        case = {"op": op, "T": _log_int(rng, 1, 8192 if op == "sort" else 4096), **_experts(rng), "H": H}
        case["dtype"] = rng.choice(["int8", "bf16", "f32"] if op == "sort" else ["bf16", "f32"])
        if op == "unsort":
            case["base"] = rng.random() < 0.5
        if case["dtype"] == "f32":
            case["T"] = max(1, case["T"] // 2)
        return _busy(case)
    N, K = _log_int(rng, 256, 12288), _log_int(rng, 384, 7168)
    if rng.random() < 0.6:
        N, K = max(256, N // 64 * 64), max(384, K // 128 * 128)
    if op == "linear":
        return {"op": op, "T": _log_int(rng, 1, 8192), "N": N, "K": K}
    case = {"op": op, "T": _log_int(rng, 1, 2048), **_experts(rng), "N": min(N, 7168), "K": K, "swiglu": rng.random() < 0.5}
    # no more products, in all experts, than the largest listed case has
    limit = 2048 * 8 * 16 * 7168 * 2048
    case["E"] = min(case["E"], 32)
    while case["T"] > 1 and case["T"] * case["k"] * case["E"] * case["N"] * case["K"] > limit:
        case["T"] //= 2
    return _busy(case)


# ------------------------------------------------------------------------------------------------ the inputs

def _pad16(n):
    return (n + 15) // 16 * 16


def _ids(case, gen):
    """Each token's experts, int32 [T, k]: some experts are more popular than others, and a batch ends in padding."""
    T, total, k = case["T"], case["total"], case["k"]
    score = torch.randn(T, total, generator=gen, device="cuda") * 1.5 + torch.randn(total, generator=gen, device="cuda") * 0.5
    ids = score.topk(k, dim=1).indices.to(torch.int32)
    ids[T - T // 16:] = -1  # a padded token has no expert
    return ids


def _rounded(x):
    """Rows x [.., K] in 32 bits, as 8-bit integers (held in 32 bits), and their scales [.., 1]."""
    a = x.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    return torch.round(x * (LEVELS / 512) / a * 512), a / LEVELS  # 127 x / a without overflow


def _weights(shape, gen):
    """A weight [.., N, K] in 8-bit integers (rows of a pitch of 16 bytes) and its scales [.., N]."""
    *lead, K = shape
    q = torch.zeros(*lead, _pad16(K), dtype=torch.int8, device="cuda")
    s = torch.empty(*lead, dtype=torch.float32, device="cuda")
    for i in range(lead[0] if len(lead) > 1 else 1):
        part = (q[i], s[i]) if len(lead) > 1 else (q, s)
        w, scale = _rounded(torch.randn(lead[-1], K, generator=gen, device="cuda") / math.sqrt(K))
        part[0][..., :K] = w.to(torch.int8)
        part[1].copy_(scale[..., 0])
    return q[..., :K], s


def _plan(st):
    """For each pair its place among the sorted rows (-1: not of this rank), the pair of each row, the first row of each expert."""
    c = st["case"]
    first, E = st["first"], c["E"]
    expert = st["ids"].flatten().long() - first
    expert = torch.where((expert >= 0) & (expert < E), expert, E)
    pair = expert.sort(stable=True).indices
    here = expert[pair] < E
    place = torch.full_like(expert, -1)
    place[pair] = torch.where(here, torch.arange(len(pair), device="cuda"), -1)
    counts = (expert[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return place.view(st["ids"].shape).to(torch.int32), pair, here, offsets.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, T = case["op"], case["T"]
    st = {"case": case}

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    if op != "linear":
        st["ids"] = _ids(case, gen)
        st["first"] = (case["total"] - case["E"]) // 2  # this rank's experts lie in the middle of all of them
        P = T * case["k"]
    if op == "linear":
        st["x"] = normal(T, case["K"])
        st["w"], st["ws"] = _weights((case["N"], case["K"]), gen)
    elif op == "grouped":
        N, K = case["N"], case["K"]
        st["offsets"] = _plan(st)[3]
        if case["swiglu"]:
            st["gate_up"] = normal(P, 2 * K)
        else:
            q, s = _rounded(normal(P, K).float())
            st["x"] = torch.zeros(P, _pad16(K), dtype=torch.int8, device="cuda")[:, :K]
            st["x"].copy_(q)
            st["xs"] = s[:, 0].contiguous()
        st["w"], st["ws"] = _weights((case["E"], N, K), gen)
        st["out"] = torch.zeros(P, N, dtype=torch.bfloat16, device="cuda")  # rows behind the last expert's stay as they are
    else:
        H, dtype = case["H"], DTYPES[case["dtype"]]
        if op == "sort":
            if dtype is torch.int8:
                q, s = _rounded(normal(T, H).float())
                st["x"], st["xs"] = q.to(dtype), s[:, 0].contiguous()
            else:
                st["x"], st["xs"] = normal(T, H, dtype=dtype), None
            st["rows"] = torch.zeros(P, H, dtype=dtype, device="cuda")
            st["row_scales"] = None if st["xs"] is None else torch.zeros(P, device="cuda")
        else:
            st["place"] = _plan(st)[0]
            w = torch.rand(T, case["k"], generator=gen, device="cuda") + 0.1
            st["weights"] = w / w.sum(1, keepdim=True)
            st["rows"] = normal(P, H, dtype=dtype)
            if op == "unsort":
                st["base"] = normal(T, H, dtype=dtype) if case["base"] else None
            else:
                st["dy"] = normal(T, H, dtype=dtype)
                st["dx_rows"] = normal(P, H, dtype=dtype)  # from the experts' own backward pass
                st["drows"] = torch.zeros(P, H, dtype=dtype, device="cuda")
    return st


# ------------------------------------------------------------------------------------------------ the plain forms

def _plain_sort(st):
    place, pair, here, offsets = _plan(st)
    of = pair // st["case"]["k"]
    out = {"rows": torch.where(here[:, None], st["x"][of], torch.zeros_like(st["x"][:1])), "place": place, "offsets": offsets}
    if st["xs"] is not None:
        out["row_scales"] = torch.where(here, st["xs"][of], 0.0)
    return out


def _gathered(rows, place, j):
    """rows[place[:, j]] in 32 bits, 0 where a pair has no place."""
    at = place[:, j].long()
    return torch.where(at[:, None] >= 0, rows[at.clamp_min(0)].float(), 0.0)


def _plain_unsort(st):
    rows, place, w = st["rows"], st["place"], st["weights"]
    y = torch.zeros(place.shape[0], rows.shape[1], device="cuda") if st["base"] is None else st["base"].float()
    for j in range(place.shape[1]):
        y = y + w[:, j, None] * _gathered(rows, place, j)
    return {"y": y.to(rows.dtype)}


def _plain_gradient(st):
    rows, place, w, dy = st["rows"], st["place"], st["weights"], st["dy"].float()
    P, H = rows.shape
    k = place.shape[1]
    drows = torch.zeros(P + 1, H, dtype=rows.dtype, device="cuda")  # the last row takes what has no place
    dw = torch.zeros_like(w)
    dx = torch.zeros_like(dy)
    for j in range(k):
        at = place[:, j].long()
        drows[torch.where(at >= 0, at, P)] = (w[:, j, None] * dy).to(rows.dtype)
        dw[:, j] = (_gathered(rows, place, j) * dy).sum(1)
        dx = dx + _gathered(st["dx_rows"], place, j)
    return {"drows": drows[:P], "dweights": dw, "dx": dx.to(rows.dtype)}


def _plain_linear(st):
    q, s = _rounded(st["x"].float())
    return {"y": (q @ st["w"].float().t() * s * st["ws"]).to(torch.bfloat16)}


def _swiglu(gate_up):
    g, u = gate_up.float().chunk(2, -1)
    return g / (1.0 + torch.exp(-g)) * u


def _plain_grouped(st):
    if st["case"]["swiglu"]:
        q, s = _rounded(_swiglu(st["gate_up"]))
    else:
        q, s = st["x"].float(), st["xs"][:, None]
    offsets = st["offsets"]
    row = torch.arange(len(q), device="cuda")[:, None]
    y = torch.zeros(len(q), st["case"]["N"], device="cuda")
    for e in range(st["case"]["E"]):  # every expert on every row
        of = q @ st["w"][e].float().t() * s * st["ws"][e]
        y = torch.where((row >= offsets[e]) & (row < offsets[e + 1]), of, y)
    return {"y": y.to(torch.bfloat16)}


def _kept(st):
    """The workspace and the outputs that a program keeps from pass to pass."""
    if "kept" not in st:
        import moe_shared_expert_gb300 as mse
        c, T = st["case"], st["case"]["T"]
        st["kept"] = k = {}
        if c["op"] == "sort":
            k["place"] = torch.empty(T, c["k"], dtype=torch.int32, device="cuda")
            k["offsets"] = torch.empty(c["E"] + 1, dtype=torch.int32, device="cuda")
            k["workspace"] = mse.new_moe_sort_workspace(T, c["k"], c["E"])
        elif c["op"] == "unsort":
            k["y"] = torch.empty(T, c["H"], dtype=st["rows"].dtype, device="cuda")
        elif c["op"] == "gradient":
            k["dweights"] = torch.empty(T, c["k"], dtype=torch.float32, device="cuda")
            k["dx"] = torch.empty_like(st["dy"])
        elif c["op"] == "linear":
            k["y"] = torch.empty(T, c["N"], dtype=torch.bfloat16, device="cuda")
            k["workspace"] = mse.new_int8_workspace(T, c["N"], c["K"])
        else:
            P = T * c["k"]
            k["workspace"] = mse.new_int8_workspace(P, c["N"], c["K"], groups=c["E"])
            if c["swiglu"]:
                k["q"] = torch.empty(P, _pad16(c["K"]), dtype=torch.int8, device="cuda")[:, :c["K"]]
                k["scales"] = torch.empty(P, dtype=torch.float32, device="cuda")
    return st["kept"]


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"sort": _plain_sort, "unsort": _plain_unsort, "gradient": _plain_gradient, "linear": _plain_linear,
                "grouped": _plain_grouped}[c["op"]](st)
    import moe_shared_expert_gb300 as mse
    k = _kept(st)
    if c["op"] == "sort":
        rows, place, offsets, scales = mse.moe_sort(st["x"], st["ids"], c["E"], first_expert=st["first"], scales=st["xs"],
                                                    rows=st["rows"], row_scales=st["row_scales"], **k)
        out = {"rows": rows, "place": place, "offsets": offsets}
        if scales is not None:
            out["row_scales"] = scales
        return out
    if c["op"] == "unsort":
        return {"y": mse.moe_unsort(st["rows"], st["place"], st["weights"], base=st["base"], **k)}
    if c["op"] == "gradient":
        drows, dweights = mse.moe_unsort_backward(st["dy"], st["place"], st["rows"], st["weights"], drows=st["drows"],
                                                  dweights=k["dweights"])
        return {"drows": drows, "dweights": dweights, "dx": mse.moe_sort_backward(st["dx_rows"], st["place"], dx=k["dx"])}
    if c["op"] == "linear":
        return {"y": mse.int8_linear(st["x"], st["w"], st["ws"], **k)}
    if c["swiglu"]:
        x, xs = mse.int8_quantise(st["gate_up"], swiglu=True, offsets=st["offsets"], q=k["q"], scales=k["scales"])
    else:
        x, xs = st["x"], st["xs"]
    return {"y": mse.int8_grouped_matmul(x, xs, st["offsets"], st["w"], st["ws"], out=st["out"], workspace=k["workspace"])}


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, T = case["op"], case["T"]
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": N * K + 4 * N + 2 * T * (K + N), "flops": 2 * T * N * K}
    E, k, total = case["E"], case["k"], case["total"]
    tokens = T - T // 16                                     # without the padding
    pairs = tokens * k * E / total                           # expected to stay on this rank
    if op == "grouped":
        N, K = case["N"], case["K"]
        read = E * (1 - (1 - k / total) ** tokens)           # experts that expect a token
        return {"bytes": read * (N * K + 4 * N) + pairs * ((4 if case["swiglu"] else 1) * K + 2 * N),
                "flops": 2 * pairs * N * K}
    H, size = case["H"], {"bf16": 2, "f32": 4, "int8": 1}[case["dtype"]]
    some = tokens * (1 - (1 - E / total) ** k)               # tokens that expect an expert here
    if op == "sort":
        return {"bytes": (some + pairs) * H * size + 8 * T * k + 4 * E, "flops": T * k}
    if op == "unsort":
        return {"bytes": (pairs + T * (1 + case["base"])) * H * size + 8 * T * k, "flops": 2 * pairs * H}
    return {"bytes": (3 * pairs + some + T) * H * size + 12 * T * k, "flops": 4 * pairs * H}


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits

def _rounded_64(x):
    a = torch.maximum(x.abs().amax(-1, keepdim=True), torch.full((), AMAX_FLOOR, dtype=torch.float64, device="cuda"))
    return torch.round(LEVELS * x / a), a / LEVELS


def exact(case, seed):
    if case["op"] == "sort":
        return None  # copies and whole numbers: nothing is computed
    st = prepare(case, seed)
    if case["op"] == "linear":
        y = torch.empty(case["T"], case["N"], dtype=torch.float64, device="cuda")
        q, s = _rounded_64(st["x"].double())
        for n in range(0, case["N"], 1024):
            y[:, n:n + 1024] = s * (q @ st["w"][n:n + 1024].double().t()) * st["ws"][n:n + 1024].double()
        return {"y": y}
    if case["op"] == "grouped":
        y = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        at = st["offsets"].tolist()
        for e in range(case["E"]):
            rows = slice(at[e], at[e + 1])
            if case["swiglu"]:
                gu = st["gate_up"][rows].double()
                q, s = _rounded_64(torch.nn.functional.silu(gu[:, :case["K"]]) * gu[:, case["K"]:])
            else:
                q, s = st["x"][rows].double(), st["xs"][rows, None].double()
            if len(q):
                y[rows] = (q @ st["w"][e].double().t()) * s * st["ws"][e].double()
        return {"y": y}
    place = st["place"].long()
    token, slot = torch.nonzero(place >= 0, as_tuple=True)
    at = place[token, slot]
    w = st["weights"][token, slot].double()[:, None]
    if case["op"] == "unsort":
        y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda") if st["base"] is None else st["base"].double()
        return {"y": y.index_add_(0, token, w * st["rows"][at].double())}
    dy = st["dy"].double()
    drows = torch.zeros(st["rows"].shape, dtype=torch.float64, device="cuda")
    dweights = torch.zeros(place.shape, dtype=torch.float64, device="cuda")
    drows[at] = w * dy[token]
    dweights[token, slot] = torch.linalg.vecdot(st["rows"][at].double(), dy[token])
    return {"drows": drows, "dweights": dweights,
            "dx": torch.zeros_like(dy).index_add_(0, token, st["dx_rows"][at].double())}
