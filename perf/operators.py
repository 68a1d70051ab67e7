"""The operators around the weight matrices that Muon steps, as measured cases.

A transformer block's matrices, norms and biases are what `muon_step` and `adamw_step`
update; the operators here run those layers forward and produce their gradients in the
form the two steps read (fp32, in place, summed over micro-batches where asked):

  layer_norm            y = (x - mean) rstd gain + bias, and the two statistics
  layer_norm_backward   dx (with the skip path's gradient added), dgain, dbias
  linear                y = act(x W^T + bias) + residual, optionally with x W^T + bias kept
  linear_backward       dx (times the derivative of the activation that made x), dW, dbias
  activation_backward   dz = dy act'(z)

With `own` false, run() is the plain form (elementary torch operations in 32 bits, rounded
once); with it true, the calls of newton_schulz_11_b200.api.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short chat turn's tokens through a 768-wide norm: latency
        dict(name="ln-8x768", op="layer_norm", tokens=8, width=768, x="bf16", p="f32", pad=0),
        # a micro-batch of 8 sequences of 4096 tokens at width 4096
        dict(name="ln-32768x4096", op="layer_norm", tokens=32768, width=4096, x="bf16", p="f32", pad=0),
        # ragged: an odd number of packed tokens, an odd width inside a wider fp32 buffer
        dict(name="ln-bwd-1001x1023-f32", op="layer_norm_backward", tokens=1001, width=1023, x="f32", p="f32",
             pad=9, skip=False, accumulate=True),
        # a micro-batch of 16 sequences of 1024 tokens at width 768, in the residual stream
        dict(name="ln-bwd-16384x768", op="layer_norm_backward", tokens=16384, width=768, x="bf16", p="bf16",
             pad=0, skip=True, accumulate=False),
        # one token through the up projection of a 1024-wide block
        dict(name="lin-1x1024x4096", op="linear", tokens=1, k=1024, n=4096, x="bf16", w="bf16", act="gelu_tanh",
             bias=True, residual=False, keep=False, pad=0),
        # 16 sequences of 1024 tokens through an attention output projection, into the residual stream
        dict(name="lin-16384x768x768", op="linear", tokens=16384, k=768, n=768, x="bf16", w="bf16", act="none",
             bias=True, residual=True, keep=False, pad=0),
        # the largest: 8 x 1024 tokens through the up projection of a 4096-wide block, kept for the backward pass
        dict(name="lin-8192x4096x14336", op="linear", tokens=8192, k=4096, n=14336, x="bf16", w="bf16",
             act="relu2", bias=False, residual=False, keep=True, pad=0),
        # ragged and in fp32 throughout, as a numerics check of a small model runs it
        dict(name="lin-bwd-515x770x1030-f32", op="linear_backward", tokens=515, k=770, n=1030, x="f32", w="f32",
             act="silu", bias=True, skip=False, accumulate=False, pad=3),
        # the down projection of a 1024-wide block, second micro-batch: gradients are summed
        dict(name="lin-bwd-8192x4096x1024", op="linear_backward", tokens=8192, k=4096, n=1024, x="bf16", w="bf16",
             act="gelu_tanh", bias=True, skip=False, accumulate=True, pad=0),
        # a short batch through a query projection whose input gradient joins the other projections'
        dict(name="lin-bwd-256x768x768", op="linear_backward", tokens=256, k=768, n=768, x="bf16", w="f32",
             act="none", bias=True, skip=True, accumulate=False, pad=0),
        # the derivative alone: a small head, and a 1024-wide block's hidden layer
        dict(name="act-bwd-100x1000", op="activation_backward", tokens=100, width=1000, x="f32", act="gelu", pad=1),
        dict(name="act-bwd-16384x4096", op="activation_backward", tokens=16384, width=4096, x="bf16",
             act="gelu_tanh", pad=0),
    ]


def _size(rng, low, high):
    """Spread over the logarithm; half of the sizes are whole multiples of 64 where they can be."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if n >= 64 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(("layer_norm", "layer_norm_backward", "linear", "linear", "linear_backward", "linear_backward",
                     "activation_backward"))
    x = rng.choice(("bf16", "bf16", "f32"))
    c = dict(op=op, x=x, pad=rng.choice((0, 0, 8, rng.randint(1, 9))))
    if op in ("layer_norm", "layer_norm_backward", "activation_backward"):
        c["tokens"] = _size(rng, 1, 32768)
        c["width"] = _size(rng, 16, min(8192, 4096 * 32768 // c["tokens"] // (2 if x == "bf16" else 4)))
        if op == "activation_backward":
            c["act"] = rng.choice(ACTS[1:])
        else:
            c["p"] = rng.choice(("f32", "bf16"))
        if op == "layer_norm_backward":
            c.update(skip=rng.random() < 0.5, accumulate=rng.random() < 0.5)
        return c
    c["w"] = rng.choice(("bf16", "f32")) if x == "bf16" else "f32"
    c["tokens"] = _size(rng, 1, 8192)
    c["k"] = _size(rng, 16, 8192)
    # the largest listed case's products, over the directions and the plain form's passes
    most = 8192 * 4096 * 14336 // 8
    c["n"] = _size(rng, 16, max(16, min(8192, most // (c["tokens"] * c["k"]))))
    c["act"] = rng.choice(ACTS)
    c["bias"] = rng.random() < 0.7
    if op == "linear":
        c.update(residual=rng.random() < 0.4, keep=c["act"] != "none" and rng.random() < 0.5)
    else:
        c.update(skip=rng.random() < 0.3, accumulate=rng.random() < 0.3)
    return c


# ------------------------------------------------------------------ inputs

def _maker(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)

    def make(rows, cols, dtype, std=1.0, shift=0.0, pad=0):
        """rows x cols, inside rows of cols + pad elements."""
        t = torch.randn(rows, cols + pad, generator=g, device="cuda")
        return t.mul_(std).add_(shift).to(dtype)[:, :cols]

    return make


def prepare(case, seed):
    make = _maker(seed)
    op, T, pad, xt = case["op"], case["tokens"], case["pad"], DTYPES[case["x"]]
    s = {"case": case}
    if op in ("layer_norm", "layer_norm_backward"):
        D, pt = case["width"], DTYPES[case["p"]]
        # the residual stream: not centred, and a few channels much larger than the others
        x = make(T, D, torch.float32, 1.0, 0.3, pad)
        x *= 1.0 + 7.0 * (torch.arange(D, device="cuda") % 97 == 5)
        s["x"] = x._base.to(xt)[:, :D] if pad else x.to(xt)
        s["gain"] = make(1, D, pt, 0.1, 1.0)[0]
        s["bias"] = make(1, D, pt, 0.1)[0]
        if op == "layer_norm_backward":
            xd = s["x"].double()
            s["mean"] = xd.mean(1).float()
            s["rstd"] = (xd.var(1, unbiased=False) + EPS).rsqrt().float()
            s["dy"] = make(T, D, xt, 1e-2, 0.0, pad)
            s["skip"] = make(T, D, xt, 1e-2) if case["skip"] else None
            acc = case["accumulate"]
            s["dgain"] = make(1, D, torch.float32, 0.1)[0] if acc else torch.empty(D, device="cuda")
            s["dbias"] = make(1, D, torch.float32, 0.1)[0] if acc else torch.empty(D, device="cuda")
    elif op == "linear":
        K, N, wt = case["k"], case["n"], DTYPES[case["w"]]
        s["x"] = make(T, K, xt, 1.0, 0.0, pad)
        s["w"] = make(N, K, wt, 0.02)
        s["bias"] = make(1, N, wt, 0.1)[0] if case["bias"] else None
        s["residual"] = make(T, N, xt) if case["residual"] else None
    elif op == "linear_backward":
        K, N, wt = case["k"], case["n"], DTYPES[case["w"]]
        s["dy"] = make(T, N, xt, 1e-2, 0.0, pad)
        s["w"] = make(N, K, wt, 0.02)
        if case["act"] == "none":
            s["z"], s["x"] = None, make(T, K, xt, 1.0, 0.0, pad)
        else:  # x is the activation's output, as the forward pass left it
            s["z"] = make(T, K, xt, 1.0, 0.0, pad)
            s["x"] = _act(s["z"].float(), case["act"]).to(xt)
        s["skip"] = make(T, K, xt, 1e-2) if case["skip"] else None
        acc = case["accumulate"]
        s["dw"] = make(N, K, torch.float32, 0.1) if acc else torch.empty(N, K, device="cuda")
        s["db"] = None
        if case["bias"]:
            s["db"] = make(1, N, torch.float32, 0.1)[0] if acc else torch.empty(N, device="cuda")
    else:
        s["dy"] = make(T, case["width"], xt, 1e-2, 0.0, pad)
        s["z"] = make(T, case["width"], xt, 1.0, 0.0, pad)
    return s


# ------------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "relu2":
        r = torch.where(z < 0, torch.zeros_like(z), z)
        return r * r
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2.0 * torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain_layer_norm(s):
    x = s["x"].float()
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / x.shape[1] + EPS)
    y = d * rstd[:, None] * s["gain"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_layer_norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    n = x.shape[1]
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gain"].float()
    dx = s["rstd"][:, None] * (g - (g.sum(1) / n)[:, None] - xhat * ((g * xhat).sum(1) / n)[:, None])
    if s["skip"] is not None:
        dx = dx + s["skip"].float()
    dgain, dbias = (dy * xhat).sum(0), dy.sum(0)
    if s["case"]["accumulate"]:
        s["dgain"] += dgain
        s["dbias"] += dbias
    else:
        s["dgain"].copy_(dgain)
        s["dbias"].copy_(dbias)
    return dx.to(s["x"].dtype), s["dgain"], s["dbias"]


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(s["x"].dtype)
    return (y, z.to(s["x"].dtype)) if c["keep"] else y


def _plain_linear_backward(s):
    c = s["case"]
    dy = s["dy"].float()
    dx = dy @ s["w"].float()
    if s["z"] is not None:
        dx = dx * _act_grad(s["z"].float(), c["act"])
    if s["skip"] is not None:
        dx = dx + s["skip"].float()
    dw = dy.t() @ s["x"].float()
    db = dy.sum(0) if c["bias"] else None
    if c["accumulate"]:
        s["dw"] += dw
        if c["bias"]:
            s["db"] += db
    else:
        s["dw"].copy_(dw)
        if c["bias"]:
            s["db"].copy_(db)
    return dx.to(s["x"].dtype), s["dw"], s["db"]


def _plain_activation_backward(s):
    return (s["dy"].float() * _act_grad(s["z"].float(), s["case"]["act"])).to(s["dy"].dtype)


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"layer_norm": _plain_layer_norm, "layer_norm_backward": _plain_layer_norm_backward,
                "linear": _plain_linear, "linear_backward": _plain_linear_backward,
                "activation_backward": _plain_activation_backward}[op](s)
    from newton_schulz_11_b200 import api

    if op == "layer_norm":
        return api.layer_norm(s["x"], s["gain"], s["bias"], eps=EPS)
    if op == "layer_norm_backward":
        return api.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gain"], skip=s["skip"],
                                       dgain=s["dgain"], dbias=s["dbias"], accumulate=c["accumulate"])
    if op == "linear":
        return api.linear(s["x"], s["w"], s["bias"], act=c["act"], residual=s["residual"], save_preact=c["keep"])
    if op == "linear_backward":
        return api.linear_backward(s["dy"], s["x"], s["w"], in_act=c["act"], in_preact=s["z"], skip=s["skip"],
                                   dw=s["dw"], db=s["db"], need_db=c["bias"], accumulate=c["accumulate"])
    return api.activation_backward(s["dy"], s["z"], c["act"])


def work(case):
    T, xb = case["tokens"], BYTES[case["x"]]
    op = case["op"]
    if op == "layer_norm":
        D = case["width"]
        return {"bytes": 2 * T * D * xb + 2 * D * BYTES[case["p"]] + 8 * T, "flops": 8 * T * D}
    if op == "layer_norm_backward":
        D = case["width"]
        grads = 8 * D * (2 if case["accumulate"] else 1)
        return {"bytes": (4 if case["skip"] else 3) * T * D * xb + D * BYTES[case["p"]] + grads + 8 * T,
                "flops": 13 * T * D}
    if op == "activation_backward":
        return {"bytes": 3 * T * case["width"] * xb, "flops": 12 * T * case["width"]}
    K, N, wb = case["k"], case["n"], BYTES[case["w"]]
    if op == "linear":
        outs = 1 + bool(case["residual"]) + bool(case["keep"])
        return {"bytes": (T * K + outs * T * N) * xb + (N * K + N * bool(case["bias"])) * wb, "flops": 2 * T * K * N}
    reads = T * N + T * K * (1 + (case["act"] != "none") + bool(case["skip"]))
    grads = 4 * (N * K + N * bool(case["bias"])) * (2 if case["accumulate"] else 1)
    return {"bytes": (reads + T * K) * xb + N * K * wb + grads, "flops": 4 * T * K * N}


# ------------------------------------------------------------------ the definition in 64 bits

def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_act(z, act):
    """act(z) and act'(z) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act in ("relu", "relu2"):
        r = torch.clamp(z, min=0)
        return (r, (z > 0).double()) if act == "relu" else (r.square(), 2 * r)
    if act == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
        a = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(a * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * a * (1 + 0.134145 * z.square())
    p = torch.sigmoid(z)
    return z * p, p + z * p * (1 - p)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    if op == "layer_norm":
        mean = d["x"].mean(1, keepdim=True)
        var = (d["x"] - mean).square().mean(1, keepdim=True)
        y = (d["x"] - mean) / torch.sqrt(var + EPS) * d["gain"] + d["bias"]
        return y, mean[:, 0], (var + EPS)[:, 0] ** -0.5
    if op == "layer_norm_backward":
        # dx is the projection of g off the constant and off xhat, as the statistics given define them
        xhat = (d["x"] - d["mean"][:, None]) * d["rstd"][:, None]
        g = d["dy"] * d["gain"]
        dx = d["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        dx = dx + d["skip"] if "skip" in d else dx
        dgain, dbias = torch.einsum("td,td->d", d["dy"], xhat), d["dy"].sum(0)
        return (dx, dgain + d["dgain"], dbias + d["dbias"]) if case["accumulate"] else (dx, dgain, dbias)
    if op == "linear":
        z = torch.nn.functional.linear(d["x"], d["w"], d.get("bias"))
        y = _exact_act(z, case["act"])[0]
        y = y + d["residual"] if "residual" in d else y
        return (y, z) if case["keep"] else y
    if op == "linear_backward":
        dx = torch.einsum("tn,nk->tk", d["dy"], d["w"])
        dx = dx * _exact_act(d["z"], case["act"])[1] if "z" in d else dx
        dx = dx + d["skip"] if "skip" in d else dx
        dw = torch.einsum("tn,tk->nk", d["dy"], d["x"])
        db = d["dy"].sum(0) if case["bias"] else None
        if case["accumulate"]:
            return dx, dw + d["dw"], db + d["db"] if case["bias"] else None
        return dx, dw, db
    return d["dy"] * _exact_act(d["z"], case["act"])[1]
