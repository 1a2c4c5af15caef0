"""Workloads of the gated feed-forward block and of the orthogonalised update, with their plain forms.

  gated   h = act(x Wg + bg) * (x Wu + bu) and its gradients: the first half of a gated feed-forward
          block, the largest matrices that a sharded unit is gathered for;
  muon    one step of an optimizer whose update of a matrix is orthogonalised: the ranks' 16-bit
          contributions are averaged into the momentum, the momentum (with the gradient ahead of it)
          is brought near the closest matrix with orthonormal rows or columns by Newton-Schulz
          products, and the fp32 parameters and their 16-bit copy are updated.

`run` computes an operator in plain torch operations where `own` is false, and through the package
where it is true; `exact` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ACTIVATIONS = ("none", "relu", "gelu_tanh", "gelu", "silu")

# the optimizer's constants: momentum with the gradient ahead, five products with the usual quintic
LR, MOMENTUM, WEIGHT_DECAY, EPS, STEPS = 2e-4, 0.95, 0.1, 1e-7, 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
BLOCK = 256                       # each matrix's momentum starts on a multiple of it


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through the gate and up projections of a 4096 -> 11008 block: reading the weights is all
        dict(name="gated one token", op="gated", back=False, rows=1, inner=4096, outer=11008, layout="out_in",
             act="silu", bias=False, keep=False, dtype="bf16"),
        # a batch of 24 sequences decoded together, weights stored (in, out), with biases
        dict(name="gated 24 tokens", op="gated", back=False, rows=24, inner=2048, outer=8192, layout="in_out",
             act="gelu_tanh", bias=True, keep=False, dtype="bf16"),
        # a training pass over four sequences of 2048 tokens, both projections kept for the gradients
        dict(name="gated 8192 tokens", op="gated", back=False, rows=8192, inner=4096, outer=11008, layout="out_in",
             act="silu", bias=False, keep=True, dtype="bf16"),
        # its gradients: the largest products
        dict(name="gated grad 8192 tokens", op="gated", back=True, rows=8192, inner=4096, outer=11008,
             layout="out_in", act="silu", bias=False, keep=True, dtype="bf16"),
        # one sequence of the 2048-wide model, weights stored (in, out), with biases
        dict(name="gated grad 2048 tokens", op="gated", back=True, rows=2048, inner=2048, outer=8192,
             layout="in_out", act="gelu_tanh", bias=True, keep=True, dtype="bf16"),
        # odd sizes: no operand has rows on the 16-byte grid
        dict(name="gated grad 777x1001x1603", op="gated", back=True, rows=777, inner=1001, outer=1603,
             layout="out_in", act="gelu", bias=True, keep=True, dtype="fp16"),
        # the matrices of a three-layer 256-wide network over four ranks: a call whose latency counts
        dict(name="muon 256 wide", op="muon", sizes="gpt", layers=3, d=256, n_d=4, dtype="bf16"),
        # two layers of the 2048-wide GPT, sixteen ranks' contributions
        dict(name="muon 2048 wide", op="muon", sizes="gpt", layers=2, d=2048, n_d=16, dtype="bf16"),
        # an attention and a feed-forward matrix of the 4096-wide model, one rank's view of eight
        dict(name="muon 4096 wide", op="muon", sizes="llama", layers=1, d=4096, n_d=8, dtype="bf16"),
        # matrices of any shape, vectors among them, rows off the 16-byte grid
        dict(name="muon ragged", op="muon", sizes="ragged", n=8, hi=2000, pick=8, n_d=3, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _even(rng, value, share):
    return max(64, value // 64 * 64) if rng.random() < share else value


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if rng.random() < 0.45:
        kind, n_d = rng.choice(("gpt", "llama", "ragged", "ragged")), rng.choice((1, 2, 3, 4, 7, 8))
        if kind == "ragged":
            return dict(op="muon", sizes=kind, n=rng.randint(2, 12), hi=_log(rng, 64, 2500), pick=rng.randrange(1 << 16),
                        n_d=n_d, dtype=dtype)
        d = _even(rng, _log(rng, 64, 1900 if kind == "gpt" else 3600), 0.7)
        return dict(op="muon", sizes=kind, layers=rng.randint(1, 4 if d < 1024 else 1), d=d, n_d=n_d, dtype=dtype)
    inner, outer = (_even(rng, _log(rng, 64, 8192), 0.7) for _ in range(2))
    rows = _log(rng, 1, max(1, min(8192, 3.0e11 / (inner * outer))))
    back = rng.random() < 0.5
    return dict(op="gated", back=back, rows=rows, inner=inner, outer=outer, layout=rng.choice(("in_out", "out_in")),
                act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.5, keep=back or rng.random() < 0.6, dtype=dtype)


def shapes(case):
    """(count, rows, columns) of a muon case's matrices, by shape."""
    if case["sizes"] == "gpt":           # attention's input and output, the feed-forward's two
        d, n = case["d"], case["layers"]
        return [(n, d, 3 * d), (n, d, d), (n, d, 4 * d), (n, 4 * d, d)]
    if case["sizes"] == "llama":         # an attention matrix and a gate projection, stored (out, in)
        d, n = case["d"], case["layers"]
        return [(n, d, d), (n, d * 43 // 16, d)]
    u = np.random.RandomState(case["pick"]).random_sample((case["n"], 2))
    sizes = np.floor(16 * (case["hi"] / 16) ** u).astype(int)
    sizes[3::4, 0] = 1                   # a vector now and then
    return [(1, int(r), int(c)) for r, c in sizes]


def work(case):
    if case["op"] == "gated":
        m, k, n = case["rows"], case["inner"], case["outer"]
        if not case["back"]:
            return {"bytes": 2 * (m * k + 2 * k * n + m * n * (3 if case["keep"] else 1)), "flops": 4 * m * n * k}
        return {"bytes": 2 * (2 * m * k + 4 * k * n + 3 * m * n), "flops": 8 * m * n * k}
    elems = flops = 0
    for count, r, c in shapes(case):
        m, n = min(r, c), max(r, c)
        elems += count * r * c
        # X X^T and the square of it are symmetric: half of each is enough; the product with X is whole
        flops += count * STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    # contributions, momentum and parameters read and written, 16-bit parameters and direction written
    return {"bytes": elems * (2 * case["n_d"] + 8 + 8 + 2 + 2), "flops": flops}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    s = dict(case=case)
    (_prepare_muon if case["op"] == "muon" else _prepare_gated)(s, case, normal)
    return s


def _prepare_gated(s, case, normal):
    t, m, k, n = DTYPES[case["dtype"]], case["rows"], case["inner"], case["outer"]
    shape = (n, k) if case["layout"] == "out_in" else (k, n)
    s["x"] = normal(m, k, dtype=t)
    for name in ("w_gate", "w_up"):
        s[name] = normal(*shape, std=k ** -0.5, dtype=t)
    for name in ("b_gate", "b_up"):
        s[name] = normal(n, std=0.1, dtype=t) if case["bias"] else None
    if case["back"]:
        s["gate"], s["up"] = normal(m, n, dtype=t), normal(m, n, dtype=t)
        s["dh"] = normal(m, n, std=0.01, dtype=t)
    if own:
        import zero_sharded_mixed_03_gb300 as Z
        if case["back"]:
            s["out"] = {"d" + k: torch.empty_like(s[k]) if s[k] is not None else None
                        for k in ("x", "w_gate", "w_up", "b_gate", "b_up")}
            names = ("x", "w_gate", "w_up", "gate", "up", "dh")
        else:
            s["out"] = {k: torch.empty(m, n, dtype=t, device="cuda") if k == "h" or case["keep"] else None
                        for k in ("h", "gate", "up")}
            names = ("x", "w_gate", "w_up", "b_gate", "b_up")
        s["args"] = Z.zero_gated_t(
            rows=m, in_features=k, out_features=n, dtype16=Z.ZERO_BF16 if t == torch.bfloat16 else Z.ZERO_FP16,
            layout=Z.ZERO_WEIGHT_OUT_IN if case["layout"] == "out_in" else Z.ZERO_WEIGHT_IN_OUT,
            activation=(Z.ZERO_ACT_NONE, Z.ZERO_ACT_RELU, Z.ZERO_ACT_GELU_TANH, Z.ZERO_ACT_GELU,
                        Z.ZERO_ACT_SILU)[ACTIVATIONS.index(case["act"])],
            **{k: s[k].data_ptr() for k in names if s[k] is not None},
            **{k: v.data_ptr() for k, v in s["out"].items() if v is not None})
        s["workspace"] = torch.empty(max(16, Z.zero_gated_workspace(s["args"], case["back"])), dtype=torch.uint8, device="cuda")


def _prepare_muon(s, case, normal):
    """Gradients as they come in training: a signal of few directions, the same on every rank and kept by the
    momentum, and noise of each rank's own."""
    t, n_d, groups = DTYPES[case["dtype"]], case["n_d"], shapes(case)
    s["param"], s["grad"], momentum = [], [], []
    for count, r, c in groups:
        rank = max(1, min(r, c) // 8)
        falling = 2.0 ** -torch.linspace(0, 4, rank, device="cuda")
        signal = (normal(count, r, rank) * falling) @ normal(count, rank, c) * (1e-3 / rank ** 0.5)
        s["param"].append(normal(count, r, c, std=0.02))
        s["grad"].append(torch.stack([(signal + normal(count, r, c, std=1e-3)).to(t) for _ in range(n_d)]))
        momentum.append(0.9 * signal + normal(count, r, c, std=3e-4))
    s["param16"] = [p.to(t) for p in s["param"]]
    s["momentum"] = momentum
    if not own:
        return
    import zero_sharded_mixed_03_gb300 as Z
    each = [(r, c) for count, r, c in groups for _ in range(count)]
    h = Z.zero_muon_create([r for r, _ in each], [c for _, c in each], n_d,
                           Z.ZERO_BF16 if t == torch.bfloat16 else Z.ZERO_FP16)
    info = Z.zero_muon_info(h)
    s["update"] = [torch.empty_like(p) for p in s["param16"]]
    # both halves of the momentum, and each group's matrices in them
    halves = [torch.zeros(info.state_elems, device="cuda") for _ in range(2)]
    s["halves"], at = [[], []], 0
    for (count, r, c), m in zip(groups, momentum):
        step = -(-r * c // BLOCK) * BLOCK
        for k in range(2):
            s["halves"][k].append(torch.as_strided(halves[k], (count, r, c), (step, c, 1), at))
        s["halves"][0][-1].copy_(m)
        at += count * step
    s["workspace"] = torch.zeros(info.workspace_bytes, dtype=torch.uint8, device="cuda")

    def pointers(tensors):
        return [v[i].data_ptr() for v in tensors for i in range(len(v))]

    Z.zero_muon_bind(h, pointers(s["param"]), pointers(s["param16"]), pointers(s["update"]),
                     [p for r in range(n_d) for p in pointers([g[r] for g in s["grad"]])],
                     [v.data_ptr() for v in halves], s["workspace"].data_ptr(), 0,
                     torch.cuda.current_stream().cuda_stream)
    s["handle"], s["current"], s["buffers"] = h, 0, halves
    s["hyper"] = Z.muon_hyper(lr=LR, momentum=MOMENTUM, weight_decay=WEIGHT_DECAY, eps=EPS, steps=STEPS,
                              coefficients=COEFFICIENTS, nesterov=True, scale=Z.ZERO_MUON_SCALE_RMS)


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return (_plain_muon if state["case"]["op"] == "muon" else _plain_gated)(state)


def _run_own(s):
    import zero_sharded_mixed_03_gb300 as Z
    stream = torch.cuda.current_stream().cuda_stream
    if s["case"]["op"] == "muon":
        Z.zero_muon_step(s["handle"], s["hyper"], 1.0, stream)
        s["current"] ^= 1                # the gradients are finite, so no step is left out
        return {"param": s["param"], "param16": s["param16"], "momentum": s["halves"][s["current"]],
                "update": s["update"]}
    ws = s["workspace"]
    if s["case"]["back"]:
        Z.zero_gated_backward(s["args"], ws.data_ptr(), ws.numel(), stream)
    else:
        Z.zero_gated(s["args"], ws.data_ptr(), ws.numel(), stream)
    return s["out"]


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z * torch.sigmoid(z) if act == "silu" else z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        sg = torch.sigmoid(z)
        return sg * (1 + z * (1 - sg))
    return torch.ones_like(z)


def _plain_gated(s):
    case, t = s["case"], s["x"].dtype
    x, wg, wu = (s[k].float() for k in ("x", "w_gate", "w_up"))
    if case["layout"] == "out_in":
        wg, wu = wg.t(), wu.t()                              # (in, out)
    if not case["back"]:
        g, u = x @ wg, x @ wu
        if case["bias"]:
            g, u = g + s["b_gate"].float(), u + s["b_up"].float()
        keep = case["keep"]
        return {"h": (_act(g, case["act"]) * u).to(t), "gate": g.to(t) if keep else None, "up": u.to(t) if keep else None}
    g, u, dh = s["gate"].float(), s["up"].float(), s["dh"].float()
    dg, du = dh * u * _act_grad(g, case["act"]), dh * _act(g, case["act"])
    out = {"dx": dg @ wg.t() + du @ wu.t()}
    for name, d in (("gate", dg), ("up", du)):
        out["dw_" + name] = d.t() @ x if case["layout"] == "out_in" else x.t() @ d
        out["db_" + name] = d.sum(0) if case["bias"] else None
    return {k: v.to(t) if v is not None else None for k, v in out.items()}


def _plain_muon(s):
    """m = mu m + (1 - mu) g;  u = mu m + (1 - mu) g;  O = orthogonalised u;  p -= lr (wd p + 0.2 sqrt(max(r, c)) O)"""
    t, n_d = DTYPES[s["case"]["dtype"]], s["case"]["n_d"]
    a, b, c = COEFFICIENTS
    out = {"param": [], "param16": [], "momentum": [], "update": []}
    for p, grad, m in zip(s["param"], s["grad"], s["momentum"]):
        g = grad.float().sum(0) / n_d
        m = MOMENTUM * m + (1 - MOMENTUM) * g
        x = MOMENTUM * m + (1 - MOMENTUM) * g
        tall = x.shape[1] > x.shape[2]
        if tall:
            x = x.transpose(1, 2)
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
        for _ in range(STEPS):
            gram = x @ x.transpose(1, 2)
            x = a * x + (b * gram + c * (gram @ gram)) @ x
        if tall:
            x = x.transpose(1, 2)
        p = p - (LR * WEIGHT_DECAY) * p - (LR * 0.2 * max(p.shape[1:]) ** 0.5) * x
        for k, v in (("param", p), ("param16", p.to(t)), ("momentum", m), ("update", x.to(t))):
            out[k].append(v)
    s["param"], s["momentum"] = out["param"], out["momentum"]
    return out


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return (_exact_muon if case["op"] == "muon" else _exact_gated)(s, case)


def _exact_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    return z / (1 + torch.exp(-z)) if act == "silu" else z * 1.0


def _exact_gated(s, case):
    x, wg, wu = (s[k].double() for k in ("x", "w_gate", "w_up"))
    mk = "nk" if case["layout"] == "out_in" else "kn"
    if not case["back"]:
        g, u = torch.einsum("mk,%s->mn" % mk, x, wg), torch.einsum("mk,%s->mn" % mk, x, wu)
        if case["bias"]:
            g, u = g + s["b_gate"].double(), u + s["b_up"].double()
        return {"h": _exact_act(g, case["act"]) * u, "gate": g if case["keep"] else None, "up": u if case["keep"] else None}
    g, u = (s[k].double().requires_grad_(True) for k in ("gate", "up"))
    dg, du = torch.autograd.grad(_exact_act(g, case["act"]) * u, (g, u), s["dh"].double())
    out = {"dx": torch.einsum("mn,%s->mk" % mk, dg, wg) + torch.einsum("mn,%s->mk" % mk, du, wu)}
    for name, d in (("gate", dg), ("up", du)):
        out["dw_" + name] = torch.einsum("mn,mk->%s" % mk, d, x)
        out["db_" + name] = d.sum(0) if case["bias"] else None
    return out


def _exact_muon(s, case):
    a, b, c = COEFFICIENTS
    out = {"param": [], "param16": [], "momentum": [], "update": []}
    for p, grad, m in zip(s["param"], s["grad"], s["momentum"]):
        g = torch.zeros(p.shape, dtype=torch.float64, device="cuda")
        for contribution in grad:
            g += contribution.double() / case["n_d"]
        m = torch.lerp(g, m.double(), MOMENTUM)
        u = torch.lerp(g, m, MOMENTUM)
        direction = torch.empty_like(u)
        for i in range(len(u)):
            x = u[i] / (torch.linalg.matrix_norm(u[i]) + EPS)
            wide = x.shape[0] <= x.shape[1]
            for _ in range(STEPS):           # whichever side has the smaller Gram matrix
                gram = x @ x.mT if wide else x.mT @ x
                poly = gram @ (c * gram)
                poly += b * gram
                poly.diagonal().add_(a)
                x = poly @ x if wide else x @ poly
            direction[i] = x
        p = p.double()
        p = p - LR * (WEIGHT_DECAY * p + 0.2 * math.sqrt(max(p.shape[1:])) * direction)
        for k, v in (("param", p), ("param16", p), ("momentum", m), ("update", direction)):
            out[k].append(v)
    return out
