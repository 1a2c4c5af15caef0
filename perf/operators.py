"""Workloads of the operators around a sharded training step, with each operator's plain form.

Three operators that a program calls next to the sharded AdamW step, each over the range it meets:

  linear      y = act(x W + b) + residual and its gradients: what a gathered unit's weights are
              gathered for, and what fills a rank's 16-bit gradient contribution;
  block_norm  y = x + s * gate * Norm_post(h), z = Norm_pre(y) and its gradients: the norms after
              one block and before the next, with the block's gate and residual scale;
  adamw       one AdamW step over many separately held tensors (what is not sharded: norms,
              biases, replicated modules), first and second moments in 8 or 32 bits.

`run` computes an operator in plain torch operations where `own` is false, and through the
package where it is true; `exact` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256                       # elements that share one pair of 8-bit scales
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu_tanh", "gelu", "silu")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # norm gains and biases of the 24-layer GPT (d = 2048), kept replicated: many short tensors,
        # a call whose latency counts
        dict(name="adamw8 gains and biases", op="adamw", bits=8, sizes="vectors", layers=24, d=2048,
             grad="bf16", packed=False, clip=False),
        # all 148 tensors of GPT-2 small as one unsharded fp16 step
        dict(name="adamw8 gpt2 small fp16", op="adamw", bits=8, sizes="gpt", layers=12, d=768,
             grad="fp16", packed=False, clip=False),
        # ten thousand ragged tensors (1 to 65,536 elements) packed back to back, so that most start
        # off the 16-byte grid; clipped by the global norm
        dict(name="adamw8 ragged clipped", op="adamw", bits=8, sizes="ragged", n=10000, hi=16,
             grad="bf16", packed=True, clip=True),
        # the same kind of step with states in 32 bits and fp32 gradients
        dict(name="adamw32 ragged fp32 grads", op="adamw", bits=32, sizes="ragged", n=10000, hi=16,
             grad="fp32", packed=False, clip=False),
        # one token of a d = 4096 model
        dict(name="block_norm one token", op="block_norm", back=False, rows=1, dim=4096, layer=False,
             post=True, gate_rows=1, dtype="bf16"),
        # 8 sequences of 2048 tokens of the 1.3B GPT, LayerNorm, one learned gate per channel
        dict(name="block_norm gpt 16384x2048", op="block_norm", back=False, rows=16384, dim=2048,
             layer=True, post=True, gate_rows=16384, dtype="bf16"),
        # the backward pass of 8 sequences of a d = 4096 RMSNorm model, one gate per sequence
        dict(name="block_norm grad 16384x4096", op="block_norm", back=True, rows=16384, dim=4096,
             layer=False, post=True, gate_rows=2048, dtype="bf16"),
        # odd sizes: no row starts on the 16-byte grid, gates of 7 tokens with a ragged last group
        dict(name="block_norm grad 1001x1023", op="block_norm", back=True, rows=1001, dim=1023,
             layer=True, post=True, gate_rows=7, dtype="fp16"),
        # a single token through the 1.3B GPT's first feed-forward matrix
        dict(name="linear one token", op="linear", back=False, rows=1, inner=2048, outer=8192,
             layout="in_out", act="gelu_tanh", bias=True, residual=False, dtype="bf16"),
        # four sequences through the 1.3B GPT's second feed-forward matrix, onto the residual stream
        dict(name="linear gpt down 8192", op="linear", back=False, rows=8192, inner=8192, outer=2048,
             layout="in_out", act="none", bias=True, residual=True, dtype="bf16"),
        # the gradients of a 4096 -> 11008 gate projection over 8192 tokens: the largest product
        dict(name="linear grad llama gate 8192", op="linear", back=True, rows=8192, inner=4096,
             outer=11008, layout="out_in", act="silu", bias=False, residual=False, dtype="bf16"),
        # odd sizes: no operand has rows on the 16-byte grid
        dict(name="linear grad 777x1001x1603", op="linear", back=True, rows=777, inner=1001, outer=1603,
             layout="out_in", act="gelu", bias=True, residual=False, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("adamw", "block_norm", "linear"))
    if op == "adamw":
        kind = rng.choice(("vectors", "gpt", "ragged"))
        case = dict(op=op, bits=rng.choice((8, 8, 32)), sizes=kind, grad=rng.choice(("bf16", "fp16", "fp32")),
                    packed=rng.random() < 0.4, clip=rng.random() < 0.4)
        if kind == "ragged":
            case.update(n=_log(rng, 20, 10000), hi=rng.randint(10, 16))
        elif kind == "gpt":
            case.update(layers=rng.randint(1, 12), d=_log(rng, 100, 768))
        else:
            case.update(layers=rng.randint(2, 48), d=_log(rng, 100, 4096))
        return case
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op == "block_norm":
        dim = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            dim = max(64, dim // 64 * 64)
        rows = _log(rng, 1, min(16384, 64_000_000 // dim))
        gate = rng.choice((0, 1, _log(rng, 1, rows), rows))
        return dict(op=op, back=rng.random() < 0.5, rows=rows, dim=dim, layer=rng.random() < 0.5,
                    post=rng.random() < 0.7, gate_rows=gate, dtype=dtype)
    inner, outer = _log(rng, 64, 11008), _log(rng, 64, 11008)
    if rng.random() < 0.7:
        inner, outer = max(64, inner // 64 * 64), max(64, outer // 64 * 64)
    rows = _log(rng, 1, max(1, min(8192, 3.6e11 / (inner * outer))))
    for v in (inner, outer, rows):
        if v == 3072:
            return draw(rng)
    return dict(op=op, back=rng.random() < 0.5, rows=rows, inner=inner, outer=outer,
                layout=rng.choice(("in_out", "out_in")), act=rng.choice(ACTIVATIONS),
                bias=rng.random() < 0.6, residual=rng.random() < 0.5, dtype=dtype)


def tensor_sizes(case):
    """Element counts of an adamw case's tensors."""
    if case["sizes"] == "ragged":        # log-uniform over 1 .. 2^hi
        u = np.random.RandomState(7).random_sample(case["n"])
        return [int(s) for s in np.clip(np.floor(2.0 ** (case["hi"] * u)), 1, 1 << case["hi"])]
    d, layers = case["d"], case["layers"]
    if case["sizes"] == "vectors":       # two norms and four biases a layer, and the final norm
        return [d, d, 3 * d, d, d, d, 4 * d, d] * layers + [d, d]
    block = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, 4 * d * d, 4 * d, 4 * d * d, d]
    return [50257 * d, 1024 * d] + block * layers + [d, d]


def work(case):
    if case["op"] == "adamw":
        n = sum(tensor_sizes(case))
        g = 4 if case["grad"] == "fp32" else 2
        # gradient, master read and written, 16-bit copy written, moments read and written;
        # 8 bits: one byte each and a pair of scales a block, and the exported values written
        state = (2 + 2 + 4 / BLOCK + 4) if case["bits"] == 8 else 16
        return {"bytes": n * (g + 8 + 2 + state), "flops": 20 * n}
    if case["op"] == "block_norm":
        n, gates = case["rows"] * case["dim"], _gates(case) * case["dim"]
        # forward: h, x, y, z; backward: dz, dy, y, dx, dh, and h where a norm or gate needs it
        streams = 4 if not case["back"] else 5 + bool(case["post"] or case["gate_rows"])
        return {"bytes": 2 * (n * streams + gates * (2 if case["back"] else 1)), "flops": (16 if not case["back"] else 34) * n}
    m, k, n = case["rows"], case["inner"], case["outer"]
    if not case["back"]:
        return {"bytes": 2 * (m * k + k * n + m * n * (2 + case["residual"])), "flops": 2 * m * n * k}
    return {"bytes": 2 * (2 * m * k + 2 * k * n + m * n * (2 if case["act"] != "none" else 1)), "flops": 4 * m * n * k}


def _gates(case):
    return -(-case["rows"] // case["gate_rows"]) if case["gate_rows"] else 0


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    s = dict(case=case)
    {"adamw": _prepare_adamw, "block_norm": _prepare_norm, "linear": _prepare_linear}[case["op"]](s, case, normal)
    return s


HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
MAX_NORM, STEPS_BEFORE = 1.0, 10


def _prepare_adamw(s, case, normal):
    sizes = np.array(tensor_sizes(case), dtype=np.int64)
    blocks = -(-sizes // BLOCK)
    padded = blocks * BLOCK
    first = np.concatenate([[0], np.cumsum(padded)[:-1]])       # each tensor's first state element
    offset = np.concatenate([[0], np.cumsum(sizes)[:-1]]) if case["packed"] else first
    n_blocks, n = int(blocks.sum()), int(sizes.sum() if case["packed"] else padded.sum())
    grad_t = DTYPES[case["grad"]]
    p16_t = grad_t if grad_t != torch.float32 else torch.bfloat16
    # tensors differ in scale, as layers do
    t_sizes = torch.from_numpy(sizes).cuda()
    place = torch.arange(int(sizes.sum()), device="cuda") + torch.repeat_interleave(
        torch.from_numpy(first - (np.cumsum(sizes) - sizes)).cuda(), t_sizes)   # element -> state element
    at = torch.arange(n, device="cuda") if case["packed"] else place
    scale = torch.repeat_interleave(torch.exp2(normal(len(sizes)) * 1.5), t_sizes)

    def flat(values, dtype=torch.float32):
        out = torch.zeros(n, dtype=dtype, device="cuda")
        out[at] = values.to(dtype)
        return out

    def state(values):
        out = torch.zeros(n_blocks * BLOCK, device="cuda")
        out[place] = values
        return out

    count = place.numel()
    s["param"] = flat(normal(count, std=0.02))
    s["param16"] = s["param"].to(p16_t)
    s["grad"] = flat(normal(count, std=1e-3) * scale, grad_t)
    m, v = state(normal(count, std=3e-4) * scale), state((normal(count, std=1e-3) * scale) ** 2)
    if case["bits"] == 8:
        m8, me = _encode_m(m)
        r8, re = _encode_root(v.sqrt())
        s["m"], s["v"], s["scales"] = m8, r8, torch.stack([me, re], 1).contiguous()
        s["m_out"] = torch.empty(n_blocks * BLOCK, dtype=torch.bfloat16, device="cuda")
        s["root_out"] = torch.empty_like(s["m_out"])
    else:
        s["m"], s["v"], s["scales"] = m, v, None
    s["place"] = place if case["packed"] else None
    s["t"] = STEPS_BEFORE
    if own:
        import zero_sharded_mixed_03_gb300 as Z
        kinds = {torch.bfloat16: Z.ZERO_BF16, torch.float16: Z.ZERO_FP16, torch.float32: Z.ZERO_FP32}
        h = Z.zero_adamw_create(sizes.tolist(), case["bits"], kinds[p16_t], kinds[grad_t])
        s["workspace"] = torch.zeros(Z.zero_adamw_info(h).workspace_bytes, dtype=torch.uint8, device="cuda")
        # each tensor is an allocation of its own to the operator: a pointer a tensor
        ptrs = [[t.data_ptr() + int(o) * t.element_size() for o in offset] for t in (s["param"], s["param16"], s["grad"])]
        Z.zero_adamw_bind(h, *ptrs, s["m"].data_ptr(), s["v"].data_ptr(),
                          s["scales"].data_ptr() if s["scales"] is not None else None,
                          s["workspace"].data_ptr(), STEPS_BEFORE, torch.cuda.current_stream().cuda_stream)
        s["handle"], s["hyper"] = h, Z.hyper(max_grad_norm=MAX_NORM if case["clip"] else 0.0, **HYPER)


def _prepare_norm(s, case, normal):
    t, rows, dim = DTYPES[case["dtype"]], case["rows"], case["dim"]
    channels = torch.exp2(normal(dim))               # some channels are much larger than others
    s["h"] = (normal(rows, dim) * channels).to(t)
    s["x"] = normal(rows, dim, std=2.0, dtype=t)
    s["gate"] = normal(_gates(case), dim, std=0.5, mean=0.5, dtype=t) if case["gate_rows"] else None
    for name in ("post_w", "pre_w"):
        s[name] = normal(dim, std=0.1, mean=1.0, dtype=t)
    for name in ("post_b", "pre_b"):
        s[name] = normal(dim, std=0.1, dtype=t) if case["layer"] else None
    if not case["post"]:
        s["post_w"] = s["post_b"] = None
    if case["back"]:
        s["y"] = normal(rows, dim, std=2.0, dtype=t)
        s["dz"], s["dy"] = normal(rows, dim, std=0.01, dtype=t), normal(rows, dim, std=0.01, dtype=t)
    if own:
        import zero_sharded_mixed_03_gb300 as Z
        ptr = lambda name: s[name].data_ptr() if s.get(name) is not None else None  # noqa: E731
        new = lambda like: torch.empty_like(s[like]) if s.get(like) is not None else None  # noqa: E731
        if case["back"]:
            s["out"] = {"d" + k: new(k) for k in ("h", "x", "gate", "post_w", "post_b", "pre_w", "pre_b")}
            names = ("h", "y", "gate", "post_w", "post_b", "pre_w", "pre_b", "dy", "dz")
        else:
            s["out"] = {"y": new("x"), "z": new("x")}
            names = ("h", "x", "gate", "post_w", "post_b", "pre_w", "pre_b")
        s["args"] = Z.zero_block_norm_t(
            rows=rows, dim=dim, dtype16=Z.ZERO_BF16 if t == torch.bfloat16 else Z.ZERO_FP16,
            kind=Z.ZERO_NORM_LAYER if case["layer"] else Z.ZERO_NORM_RMS,
            norms=Z.ZERO_NORM_PRE | (Z.ZERO_NORM_POST if case["post"] else 0), rows_per_gate=case["gate_rows"],
            eps=NORM_EPS, residual_scale=RESIDUAL_SCALE, **{k: ptr(k) for k in names},
            **{k: v.data_ptr() for k, v in s["out"].items() if v is not None})
        s["workspace"] = torch.empty(max(16, Z.zero_block_norm_workspace(s["args"])) if case["back"] else 16,
                                     dtype=torch.uint8, device="cuda")


NORM_EPS, RESIDUAL_SCALE = 1e-5, 0.7


def _prepare_linear(s, case, normal):
    t, m, k, n = DTYPES[case["dtype"]], case["rows"], case["inner"], case["outer"]
    s["x"] = normal(m, k, dtype=t)
    shape = (n, k) if case["layout"] == "out_in" else (k, n)
    s["w"] = normal(*shape, std=k ** -0.5, dtype=t)
    s["bias"] = normal(n, std=0.1, dtype=t) if case["bias"] else None
    s["residual"] = normal(m, n, dtype=t) if case["residual"] and not case["back"] else None
    if case["back"]:
        s["pre"] = normal(m, n, dtype=t) if case["act"] != "none" else None
        s["dy"] = normal(m, n, std=0.01, dtype=t)
    if own:
        import zero_sharded_mixed_03_gb300 as Z
        if case["back"]:
            s["out"] = {"dx": torch.empty_like(s["x"]), "dw": torch.empty_like(s["w"]),
                        "dbias": torch.empty_like(s["bias"]) if case["bias"] else None}
            names = ("x", "w", "pre", "dy")
        else:
            s["out"] = {"y": torch.empty(m, n, dtype=t, device="cuda"),
                        "pre": torch.empty(m, n, dtype=t, device="cuda")}
            names = ("x", "w", "bias", "residual")
        s["args"] = Z.zero_linear_t(
            rows=m, in_features=k, out_features=n, dtype16=Z.ZERO_BF16 if t == torch.bfloat16 else Z.ZERO_FP16,
            layout=Z.ZERO_WEIGHT_OUT_IN if case["layout"] == "out_in" else Z.ZERO_WEIGHT_IN_OUT,
            activation=(Z.ZERO_ACT_NONE, Z.ZERO_ACT_RELU, Z.ZERO_ACT_GELU_TANH, Z.ZERO_ACT_GELU,
                        Z.ZERO_ACT_SILU)[ACTIVATIONS.index(case["act"])],
            **{name: s[name].data_ptr() for name in names if s[name] is not None},
            **{name: v.data_ptr() for name, v in s["out"].items() if v is not None})
        s["workspace"] = torch.empty(max(16, Z.zero_linear_workspace(s["args"], case["back"])),
                                     dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"adamw": _plain_adamw, "block_norm": _plain_norm, "linear": _plain_linear}[state["case"]["op"]](state)


def _run_own(s):
    import zero_sharded_mixed_03_gb300 as Z
    case, stream = s["case"], torch.cuda.current_stream().cuda_stream
    if case["op"] == "adamw":
        Z.zero_adamw_step(s["handle"], s["hyper"], 1.0, stream)
        if case["bits"] == 8:
            Z.zero_adamw_export(s["handle"], s["m_out"].data_ptr(), s["root_out"].data_ptr(), stream)
            return {"param": s["param"], "param16": s["param16"], "m": s["m_out"], "root": s["root_out"]}
        return {"param": s["param"], "param16": s["param16"], "m": s["m"], "v": s["v"]}
    ws = s["workspace"]
    if case["op"] == "block_norm":
        if case["back"]:
            Z.zero_block_norm_backward(s["args"], ws.data_ptr(), ws.numel(), stream)
        else:
            Z.zero_block_norm(s["args"], stream)
    elif case["back"]:
        Z.zero_linear_backward(s["args"], ws.data_ptr(), ws.numel(), stream)
    else:
        Z.zero_linear(s["args"], ws.data_ptr(), ws.numel(), stream)
    return s["out"]


# 8-bit moments, in blocks of 256 elements of one tensor.  First moment: e4m3 times 2^(e - 127),
# e = (exponent field of the block's largest magnitude) - 7, at least 1.  Second moment: its root
# as an unsigned float of 4 exponent and 4 fraction bits (code c: fraction c % 16; exponent field
# c // 16, 14 for [1, 2)) times 2^(e - 127), e = the exponent field of the block's largest root; a
# root above 0 is never stored as 0.

def _power(e):
    """2^(e - 127) of a float32 exponent field e (1 .. 254)."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _top_field(x):
    return x.reshape(-1, BLOCK).abs().amax(1).view(torch.int32) >> 23


def _encode_m(m):
    e = (_top_field(m) - 7).clamp(min=1)
    codes = (m.reshape(-1, BLOCK) * _power(254 - e)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(-1), e.to(torch.uint8)


def _decode_m(codes, e):
    return (codes.view(torch.float8_e4m3fn).to(torch.float32).reshape(-1, BLOCK) * _power(e)[:, None]).reshape(-1)


def _encode_root(r):
    e = _top_field(r)
    y = r.reshape(-1, BLOCK) * _power(254 - e)[:, None]
    bits = y.view(torch.int32)
    normal = ((bits + 0x3FFFF + ((bits >> 19) & 1)) >> 19) - (113 << 4)
    codes = torch.where(y >= 2.0 ** -13, normal, (y * 2.0 ** 17).round().to(torch.int32))
    codes = torch.where((codes == 0) & (y > 0), 1, codes)
    return codes.to(torch.uint8).reshape(-1), e.to(torch.uint8)


def _decode_root(codes, e):
    c = codes.to(torch.int32).reshape(-1, BLOCK)
    y = torch.where(c >= 16, ((c + (113 << 4)) << 19).view(torch.float32), c.to(torch.float32) * 2.0 ** -17)
    return (y * _power(e)[:, None]).reshape(-1)


def _plain_adamw(s):
    """m = b1 m + (1-b1) g; v = b2 v + (1-b2) g^2; p -= lr wd p; p -= lr/(1-b1^t) m / (sqrt(v)/sqrt(1-b2^t) + eps)

    The inputs are finite, so no step is left out."""
    case, h = s["case"], HYPER
    s["t"] += 1
    f = lambda x: float(np.float32(x))  # noqa: E731
    g, p = s["grad"].float(), s["param"]
    if case["clip"]:
        norm = (g * g).sum(dtype=torch.float64).sqrt()
        g = g * (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
    if case["packed"]:
        spread = torch.zeros(2, s["m"].numel(), device="cuda")
        spread[0, s["place"]], spread[1, s["place"]] = g, p
        g, p = spread[0], spread[1]
    if case["bits"] == 8:
        m = _decode_m(s["m"], s["scales"][:, 0])
        root = _decode_root(s["v"], s["scales"][:, 1])
        v = root * root
    else:
        m, v = s["m"], s["v"]
    m = m * f(h["beta1"]) + g * f(1 - h["beta1"])
    v = v * f(h["beta2"]) + (g * g) * f(1 - h["beta2"])
    root = v.sqrt()
    d = root / torch.full((), f(math.sqrt(1 - h["beta2"] ** s["t"])), device="cuda") + f(h["eps"])
    p = p - p * f(h["lr"] * h["weight_decay"])
    p = p - (m / d) * f(h["lr"] / (1 - h["beta1"] ** s["t"]))
    s["param"] = p[s["place"]] if case["packed"] else p
    s["param16"] = s["param"].to(s["param16"].dtype)
    out = {"param": s["param"], "param16": s["param16"]}
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
        return {**out, "m": m, "v": v}
    m8, me = _encode_m(m)
    r8, re = _encode_root(root)
    s["m"], s["v"], s["scales"] = m8, r8, torch.stack([me, re], 1)
    return {**out, "m": _decode_m(m8, me).to(torch.bfloat16), "root": _decode_root(r8, re).to(torch.bfloat16)}


def _norm(x, layer, w, b):
    if layer:
        x = x - x.mean(1, keepdim=True)
    hat = x * (x * x).mean(1, keepdim=True).add(NORM_EPS).rsqrt()
    return hat, hat * w + b if b is not None else hat * w


def _norm_grad(x, layer, w, dout):
    """(dx, normalised x)"""
    if layer:
        x = x - x.mean(1, keepdim=True)
    rstd = (x * x).mean(1, keepdim=True).add(NORM_EPS).rsqrt()
    hat, g = x * rstd, dout * w
    dx = g - hat * (g * hat).mean(1, keepdim=True)
    return (dx - g.mean(1, keepdim=True) if layer else dx) * rstd, hat


def _plain_norm(s):
    case, t = s["case"], s["h"].dtype
    f = {k: s[k].float() if s.get(k) is not None else None for k in ("h", "x", "gate", "post_w", "post_b", "pre_w", "pre_b", "y", "dy", "dz")}
    group = torch.arange(case["rows"], device="cuda") // case["gate_rows"] if case["gate_rows"] else None
    gate = RESIDUAL_SCALE * f["gate"][group] if group is not None else RESIDUAL_SCALE
    hat, u = _norm(f["h"], case["layer"], f["post_w"], f["post_b"]) if case["post"] else (None, f["h"])
    if not case["back"]:
        y = f["x"] + gate * u
        return {"y": y.to(t), "z": _norm(y, case["layer"], f["pre_w"], f["pre_b"])[1].to(t)}
    g, pre_hat = _norm_grad(f["y"], case["layer"], f["pre_w"], f["dz"])
    dx = f["dy"] + g
    du = dx * gate
    dh = _norm_grad(f["h"], case["layer"], f["post_w"], du)[0] if case["post"] else du
    out = {"dx": dx, "dh": dh, "dpre_w": (f["dz"] * pre_hat).sum(0), "dgate": None, "dpost_w": None,
           "dpre_b": f["dz"].sum(0) if case["layer"] else None, "dpost_b": None}
    if group is not None:
        out["dgate"] = torch.zeros_like(f["gate"]).index_add_(0, group, RESIDUAL_SCALE * dx * u)
    if case["post"]:
        out["dpost_w"] = (du * hat).sum(0)
        out["dpost_b"] = du.sum(0) if case["layer"] else None
    return {k: v.to(t) if v is not None else None for k, v in out.items()}


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
    sg = torch.sigmoid(z)
    return sg * (1 + z * (1 - sg))


def _plain_linear(s):
    case, t = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    w = w.t() if case["layout"] == "out_in" else w           # (in, out)
    if not case["back"]:
        z = x @ w
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(t), "pre": z.to(t)}
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_grad(s["pre"].float(), case["act"])
    dw = dz.t() @ x if case["layout"] == "out_in" else x.t() @ dz
    return {"dx": (dz @ w.t()).to(t), "dw": dw.to(t), "dbias": dz.sum(0).to(t) if case["bias"] else None}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"adamw": _exact_adamw, "block_norm": _exact_norm, "linear": _exact_linear}[case["op"]](s, case)


def _exact_adamw(s, case):
    """The moments in 8 bits have no exact value: theirs is the unrounded one, which they are near."""
    h, t = HYPER, STEPS_BEFORE + 1
    if case["bits"] == 8:
        m = _decode_m(s["m"], s["scales"][:, 0]).double()
        v = _decode_root(s["v"], s["scales"][:, 1]).double() ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    place = s["place"] if case["packed"] else slice(None)
    g, p = torch.zeros_like(m), torch.zeros_like(m)
    g[place], p[place] = s["grad"].double(), s["param"].double()
    if case["clip"]:
        g = g * min(1.0, MAX_NORM / (float(torch.linalg.vector_norm(g)) + 1e-6))
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    step = m / (1 - h["beta1"] ** t) / ((v / (1 - h["beta2"] ** t)).sqrt() + h["eps"])
    p = (p - h["lr"] * (h["weight_decay"] * p + step))[place]
    out = {"param": p, "param16": p, "m": m}
    out["root" if case["bits"] == 8 else "v"] = v.sqrt() if case["bits"] == 8 else v
    return out


def _exact_norm(s, case):
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    n = case["rows"]

    def leaf(name):
        return d[name].requires_grad_(case["back"]) if name in d else None

    h, gate = leaf("h"), leaf("gate")
    weights = {k: leaf(k) for k in ("post_w", "post_b", "pre_w", "pre_b")}

    def norm(v, w, b):
        centred = v - v.mean(-1, keepdim=True) if case["layer"] else v
        var = (centred ** 2).mean(-1, keepdim=True)
        return centred / torch.sqrt(var + NORM_EPS) * w + (b if b is not None else 0.0)

    u = norm(h, weights["post_w"], weights["post_b"]) if case["post"] else h
    if gate is not None:
        u = u * gate.repeat_interleave(case["gate_rows"], 0)[:n]
    u = RESIDUAL_SCALE * u
    if not case["back"]:
        y = d["x"] + u
        return {"y": y, "z": norm(y, weights["pre_w"], weights["pre_b"])}
    y = leaf("y")
    z = norm(y, weights["pre_w"], weights["pre_b"])
    pre = [w for w in (weights["pre_w"], weights["pre_b"]) if w is not None]
    into_y = torch.autograd.grad(z, [y] + pre, d["dz"])
    dx = d["dy"] + into_y[0]
    names = [k for k in ("h", "gate", "post_w", "post_b") if k in d]
    grads = dict(zip(names, torch.autograd.grad(u, [d[k] for k in names], dx)))
    out = {"d" + k: grads.get(k) for k in ("h", "gate", "post_w", "post_b")}
    out.update(dx=dx, dpre_w=into_y[1], dpre_b=into_y[2] if len(pre) > 1 else None)
    return out


def _exact_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _exact_linear(s, case):
    x, w = s["x"].double(), s["w"].double()
    if not case["back"]:
        z = torch.einsum("mk,nk->mn" if case["layout"] == "out_in" else "mk,kn->mn", x, w)
        z = z + s["bias"].double() if s["bias"] is not None else z
        y = _exact_act(z, case["act"])
        return {"y": y + s["residual"].double() if s["residual"] is not None else y, "pre": z}
    dz = s["dy"].double()
    if case["act"] != "none":
        z = s["pre"].double().requires_grad_(True)
        dz = torch.autograd.grad(_exact_act(z, case["act"]), z, dz)[0]
    if case["layout"] == "out_in":
        dx, dw = dz @ w, torch.einsum("mn,mk->nk", dz, x)
    else:
        dx, dw = torch.einsum("mn,kn->mk", dz, w), torch.einsum("mk,mn->kn", x, dz)
    return {"dx": dx, "dw": dw, "dbias": dz.sum(0) if case["bias"] else None}
