"""The operators of a layer's products next to its parameter shards: cases, plain forms, exact values.

Three operators of one training or serving step around the collectives (FSDP2 places a layer's
weights, the layer runs, its gradients are reduce-scattered):

  act8      an activation kept in 8 bits for the backward pass: e4m3 values, one power-of-two scale
            for each 32 consecutive columns of a row; "pack" writes it, "unpack" gives bf16 back
  linear    y = act(x W^T + bias) + residual on a placed weight W [N, K], optionally keeping the
            pre-activation z = x W^T + bias as such a checkpoint
  backward  from dy and the checkpoints of x and z: dz = dy act'(z), dx = dz W, dW = dz^T x,
            dbias = the sum of dz over the tokens; dW and dbias are the bf16 gradients that the
            reduce-scatter reads

Where `own` is false, `run` computes them with elementary torch operations in 32 bits; where it is
true, it makes the calls a user makes.  `exact` gives the same results from the definitions in 64
bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32            # columns that share a scale
E4M3_MAX = 448.0
MIN_EXP = -110        # the smallest scale is 2^-110: every value stays a normal bf16 number
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # one token's activation of a wide model in decode or at the end of a sequence: latency
        dict(name="pack 1x8192", op="pack", rows=1, cols=8192),
        # the input of a layer kept for its backward pass, a few thousand tokens
        dict(name="pack 8192x8192", op="pack", rows=8192, cols=8192),
        # an odd width: the last block of every row is partial and rows start unaligned
        dict(name="pack 4099x1001", op="pack", rows=4099, cols=1001),
        # a short sequence's checkpoint read back
        dict(name="unpack 333x2048", op="unpack", rows=333, cols=2048),
        # the widest activation of the 8192-wide layer read back
        dict(name="unpack 8192x28672", op="unpack", rows=8192, cols=28672),
        # one new token through the widest weight: the weight's bytes bound it
        dict(name="linear 1x28672x8192 silu", op="linear", T=1, N=28672, K=8192, act="silu",
             bias=False, res=False, keep=False),
        # a few tokens through an output projection with its bias and residual
        dict(name="linear 24x5120x5120 res", op="linear", T=24, N=5120, K=5120, act="none",
             bias=True, res=True, keep=False),
        # a ragged batch through a ragged parameter, keeping z
        dict(name="linear 1003x1001x8192 gelu", op="linear", T=1003, N=1001, K=8192, act="gelu",
             bias=True, res=False, keep=True),
        # a training sequence through the widest weight, keeping z: the largest forward product
        dict(name="linear 4096x28672x8192 silu", op="linear", T=4096, N=28672, K=8192, act="silu",
             bias=False, res=False, keep=True),
        # one expert's share of a batch
        dict(name="backward 77x768x2048 silu", op="backward", T=77, N=768, K=2048, act="silu",
             bias=False),
        # a feed-forward input projection of a 5120-wide block, bias and gelu
        dict(name="backward 2048x13824x5120 gelu", op="backward", T=2048, N=13824, K=5120,
             act="gelu_tanh", bias=True),
        # the down projection of the 8192-wide layer: the largest backward products
        dict(name="backward 4096x8192x28672", op="backward", T=4096, N=8192, K=28672, act="none",
             bias=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A tensor width: most models' are multiples of 8 or 64, some are odd."""
    w = _log_int(rng, lo, hi)
    q = rng.choice((64, 64, 8, 1))
    return max(q, w // q * q)


def draw(rng):
    op = rng.choice(("pack", "unpack", "linear", "linear", "backward", "backward"))
    if op in ("pack", "unpack"):
        cols = _width(rng, 33, 28672)
        return dict(op=op, rows=_log_int(rng, 1, min(32768, 8192 * 28672 // cols)), cols=cols)
    N, K = _width(rng, 65, 28672), _width(rng, 65, 28672)
    T = _log_int(rng, 1, min(8192, 4096 * 28672 * 8192 // (N * K)))
    act = rng.choice(ACTS)
    case = dict(op=op, T=T, N=N, K=K, act=act, bias=rng.random() < 0.5)
    if op == "linear":
        case.update(res=rng.random() < 0.5, keep=act != "none" and rng.random() < 0.5)
    return case


def work(case):
    if case["op"] in ("pack", "unpack"):
        n, blocks = case["rows"] * case["cols"], case["rows"] * -(-case["cols"] // BLOCK)
        return {"bytes": 3 * n + blocks, "flops": 2 * n}
    T, N, K = case["T"], case["N"], case["K"]
    kept = lambda c: T * c + T * -(-c // BLOCK)  # noqa: E731  bytes of a [T, c] checkpoint
    bias = 2 * N if case["bias"] else 0
    if case["op"] == "linear":
        return {"bytes": 2 * (T * K + N * K + T * N) + bias + (2 * T * N if case["res"] else 0)
                + (kept(N) if case["keep"] else 0), "flops": 2 * T * N * K}
    return {"bytes": 2 * (T * N + N * K) + kept(K) + (kept(N) if case["act"] != "none" else 0)
            + 2 * (T * K + N * K) + bias, "flops": 4 * T * N * K}


# ---- plain forms in 32 bits --------------------------------------------------------------------

def _quantise(x):
    """(e4m3 values [rows, cols], scales [rows, blocks]) of a float32 matrix, and its padded width."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    v = torch.nn.functional.pad(x, (0, pad)).reshape(rows, -1, BLOCK)
    amax = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(-1)
    m, e = torch.frexp(amax)                     # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m > E4M3_MAX / 512, e - 8, e - 9)   # the smallest with amax <= 448 * 2^e
    e = torch.where(amax > 0, e, MIN_EXP).clamp(min=MIN_EXP)
    q = torch.where(torch.isfinite(v), torch.ldexp(v, -e[..., None]), math.nan)
    q = q.to(torch.float8_e4m3fn).reshape(rows, cols + pad)
    scales = torch.ldexp(torch.ones_like(amax), e).to(torch.float8_e8m0fnu)
    return q, scales


def _values(q, scales):
    """The float32 values that a checkpoint's padded e4m3 values and scales stand for."""
    rows, padded = q.shape
    v = q.to(torch.float32).reshape(rows, -1, BLOCK) * scales.to(torch.float32)[..., None]
    return v.reshape(rows, padded)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0 * z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


# ---- inputs ------------------------------------------------------------------------------------

def _normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def _activation(gen, rows, cols):
    """An activation: channels of unequal size, a few of them large, the last rows padding."""
    channel = torch.exp(0.5 * torch.randn(cols, generator=gen, device=DEV))
    channel = torch.where(torch.rand(cols, generator=gen, device=DEV) < 0.002, 20.0, channel)
    x = torch.randn(rows, cols, generator=gen, device=DEV) * channel
    x[rows - rows // 64:] = 0
    return x.to(torch.bfloat16)


def _make(case, seed):
    """A case's tensors from its seed, checkpoints as (padded e4m3 values, scales)."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = {}
    if case["op"] in ("pack", "unpack"):
        t["x"] = _activation(gen, case["rows"], case["cols"])
        if case["op"] == "unpack":
            t["x8"] = _quantise(t.pop("x").float())
        return t
    T, N, K = case["T"], case["N"], case["K"]
    t["w"] = _normal(gen, N, K, scale=1 / math.sqrt(K))
    t["bias"] = _normal(gen, N, scale=0.1) if case["bias"] else None
    x = _activation(gen, T, K)
    if case["op"] == "linear":
        t["x"] = x
        t["res"] = _normal(gen, T, N) if case["res"] else None
        return t
    t["x8"] = _quantise(x.float())
    del x
    t["z8"] = _quantise(torch.randn(T, N, generator=gen, device=DEV)) if case["act"] != "none" else None
    t["dy"] = _normal(gen, T, N, scale=1e-3)
    return t


def prepare(case, seed):
    t = _make(case, seed)
    state = {"case": case, "t": t}
    if own:
        from shard_placement_amd.linear import Act8, Linear

        # what a program keeps from the forward pass: checkpoints in buffers of its own
        for name, cols in (("x8", case.get("cols", case.get("K"))), ("z8", case.get("N"))):
            if t.get(name) is not None:
                kept = Act8(t[name][0].shape[0], cols, device=DEV)
                kept.data.copy_(t[name][0])
                kept.scales.copy_(t[name][1])
                state[name] = kept
        if case["op"] == "pack":
            state["x8"] = Act8(case["rows"], case["cols"], device=DEV)
        elif case["op"] == "linear":
            state["layer"] = Linear(t["w"], bias=t["bias"], act=case["act"])
            state["z8"] = Act8(case["T"], case["N"], device=DEV) if case["keep"] else None
        elif case["op"] == "backward":
            # the gradients lie where the reduce-scatter reads them
            state["layer"] = Linear(t["w"], bias=t["bias"], act=case["act"],
                                    weight_grad=torch.empty_like(t["w"]),
                                    bias_grad=None if t["bias"] is None else torch.empty_like(t["bias"]))
            state.setdefault("z8", None)
    return state


# ---- one pass ----------------------------------------------------------------------------------

def _run_own(state):
    case, t = state["case"], state["t"]
    if case["op"] == "pack":
        x8 = state["x8"]
        x8.pack(t["x"])
        return {"q": x8.data[:, :case["cols"]], "scales": x8.scales}
    if case["op"] == "unpack":
        return {"x": state["x8"].unpack()}
    layer = state["layer"]
    if case["op"] == "linear":
        z8 = state["z8"]
        out = {"y": layer.forward(t["x"], residual=t["res"], z=z8)}
        if z8 is not None:
            out.update(q=z8.data[:, :case["N"]], scales=z8.scales)
        return out
    out = {"dx": layer.backward(t["dy"], x=state["x8"], z=state["z8"]), "dw": layer.weight_grad}
    if case["bias"]:
        out["db"] = layer.bias_grad
    return out


def run(state):
    if own:
        return _run_own(state)
    case, t = state["case"], state["t"]
    bf16 = torch.bfloat16
    if case["op"] == "pack":
        q, scales = _quantise(t["x"].float())
        return {"q": q[:, :case["cols"]], "scales": scales}
    if case["op"] == "unpack":
        return {"x": _values(*t["x8"])[:, :case["cols"]].to(bf16)}
    if case["op"] == "linear":
        z = t["x"].float() @ t["w"].float().T
        if case["bias"]:
            z = z + t["bias"].float()
        y = _act(z, case["act"])
        if case["res"]:
            y = y + t["res"].float()
        out = {"y": y.to(bf16)}
        if case["keep"]:
            q, scales = _quantise(z)
            out.update(q=q[:, :case["N"]], scales=scales)
        return out
    dz = t["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_grad(_values(*t["z8"])[:, :case["N"]], case["act"])
    out = {"dx": (dz @ t["w"].float()).to(bf16),
           "dw": (dz.T @ _values(*t["x8"])[:, :case["K"]]).to(bf16)}
    if case["bias"]:
        out["db"] = dz.sum(0).to(bf16)
    return out


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_checkpoint(z, cols):
    """An e4m3 value is a whole number of steps, a step being an eighth of the value's power of two
    and at least 2^-9; halves go to the even number of steps."""
    rows = z.shape[0]
    q = torch.zeros(rows, -(-cols // BLOCK) * BLOCK, dtype=torch.float64, device=z.device)
    q[:, :cols] = z
    q = q.view(rows, -1, BLOCK)
    top = q.abs().nan_to_num(0.0, 0.0, 0.0).max(dim=-1, keepdim=True).values
    e = torch.ceil(torch.log2(top / E4M3_MAX))
    e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)          # log2 rounded down
    e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)     # log2 rounded up
    e = e.clamp(min=MIN_EXP)
    u = q / torch.exp2(e)
    exponent = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    u = torch.round(u / step) * step
    return u.reshape(rows, -1)[:, :cols], torch.exp2(e).reshape(rows, -1)


def _exact_values(kept, cols):
    q, scales = kept[0].double(), kept[1].float().double()
    return (q.unflatten(1, (-1, BLOCK)) * scales.unsqueeze(2)).flatten(1)[:, :cols]


def exact(case, seed):
    t = _make(case, seed)
    if case["op"] == "pack":
        q, scales = _exact_checkpoint(t["x"].double(), case["cols"])
        return {"q": q, "scales": scales}
    if case["op"] == "unpack":
        return {"x": _exact_values(t["x8"], case["cols"])}
    act = case["act"]
    if case["op"] == "linear":
        z = t["x"].double().matmul(t["w"].double().t())
        if t["bias"] is not None:
            z += t["bias"].double()
        y = {"none": lambda: z.clone(), "relu": lambda: z.clamp(min=0),
             "gelu": lambda: z * torch.special.erfc(-z / math.sqrt(2)) / 2,
             "gelu_tanh": lambda: z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)),
             "silu": lambda: z * torch.sigmoid(z)}[act]()
        if t["res"] is not None:
            y += t["res"].double()
        out = {"y": y}
        if case["keep"]:
            out["q"], out["scales"] = _exact_checkpoint(z, case["N"])
        return out
    dz = t["dy"].double()
    if act != "none":
        z = _exact_values(t["z8"], case["N"])
        if act == "relu":
            dz = torch.where(z > 0, dz, 0.0)
        elif act == "gelu":
            dz *= torch.special.erfc(-z / math.sqrt(2)) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        else:
            # z sigmoid(g(z)): sigmoid(g) + z sigmoid(g) sigmoid(-g) g'
            if act == "silu":
                g, slope = z, torch.ones_like(z)
            else:
                g = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
                slope = math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
            s = torch.sigmoid(g)
            dz *= s + z * s * torch.sigmoid(-g) * slope
    out = {"dx": dz.matmul(t["w"].double()),
           "dw": dz.t().matmul(_exact_values(t["x8"], case["K"]))}
    if case["bias"]:
        out["db"] = dz.sum(dim=0)
    return out
