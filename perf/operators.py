"""Cases of the dense linear operators (a matrix product with bias, activation
and residual in its epilogue, and its backward) and of gradient clipping over
many tensors: inputs, the plain form of each operator and its definition in
float64.

Tensors are dense and row-major: x [tokens, d_in], W [d_out, d_in], y, u,
residual [tokens, d_out], bias [d_out] float32; an INT8 weight is
diag(w_scale) q. With act one of ACTIVATIONS:

  forward   u = x W^T + bias,  y = act(u) + residual  (u returned where a
            training step keeps it)
  backward  g_u = g_y act'(u),  g_x = g_u W,  g_W = g_u^T x,
            g_bias = the column sums of g_u
  clip      norm = sqrt(sum of squares over every tensor),
            out = grad min(1, max_norm / norm)
"""
import math

import torch

own = False

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_C, _A = math.sqrt(2.0 / math.pi), 0.044715  # gelu_tanh: u (1 + tanh(C (u + A u^3))) / 2


def _fwd(name, tokens, d_in, d_out, dtype="bf16", activation="none", bias=False, residual=False,
         save=False):
    c = dict(op="forward", tokens=tokens, d_in=d_in, d_out=d_out, dtype=dtype,
             activation=activation, bias=bias, residual=residual, save=save)
    return dict(c, name=name) if name else c


def _bwd(name, tokens, d_in, d_out, dtype="bf16", activation="none", g_weight=False, g_bias=False):
    c = dict(op="backward", tokens=tokens, d_in=d_in, d_out=d_out, dtype=dtype,
             activation=activation, g_weight=g_weight, g_bias=g_bias)
    return dict(c, name=name) if name else c


def _clip(name, layers, block, odd, clipped=True):
    c = dict(op="clip", layers=layers, block=block, odd=odd, clipped=clipped)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a gate projection of the 8B layer set: the weight's bytes
        _fwd("fwd_gate_1tok", 1, 4096, 14336, activation="silu"),
        # a batch of decoded tokens, INT8 weight, added to the residual stream
        _fwd("fwd_down_int8_16tok", 16, 14336, 4096, dtype="int8", residual=True),
        # a larger serving batch through an output projection
        _fwd("fwd_o_100tok", 100, 4096, 4096, bias=True, residual=True),
        # a ragged prompt through a 1B-class projection, training's saved u
        _fwd("fwd_1b_777tok", 777, 2048, 2048, activation="gelu", bias=True, save=True),
        # the 8B MLP up-projection of a training step
        _fwd("fwd_up_8192tok", 8192, 4096, 14336, activation="silu", bias=True, save=True),
        # float32 storage
        _fwd("fwd_f32_512tok", 512, 2048, 2048, dtype="f32", activation="gelu_tanh", bias=True,
             residual=True),
        # the backward of that up-projection with its weight frozen
        _bwd("bwd_up_8192tok", 8192, 4096, 14336, activation="silu", g_bias=True),
        # a ragged batch through a 1B-class projection with a trained weight
        _bwd("bwd_1b_1000tok", 1000, 2048, 2048, activation="gelu", g_weight=True, g_bias=True),
        # the smallest float32 layer: launch latency
        _bwd("bwd_f32_64tok", 64, 256, 256, dtype="f32", activation="relu", g_weight=True,
             g_bias=True),
        # the generators of one 1B-class layer
        _clip("clip_1b_layer", 0, 256, 1),
        # the generators of one 8B layer set (seven linears), b = 256
        _clip("clip_8b_set", 1, 256, 3),
        # of a whole 8B model, 32 layer sets
        _clip("clip_8b_model", 32, 256, 3),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Tokens from 1 to 8192, widths from 128 to 14336 in steps of 8 (a third
    of them multiples of 256), every type, activation and epilogue; clips of
    every block size and up to 16 layer sets."""
    kind = rng.choice(("forward",) * 5 + ("backward",) * 3 + ("clip",) * 2)
    if kind == "clip":
        return _clip(None, rng.randint(0, 16), rng.choice((32, 64, 128, 256, 512)),
                     rng.randint(0, 9), rng.random() < 0.7)
    step = rng.choice((8, 8, 256))
    d_in, d_out = (max(step, _log(rng, 128, 14336) // step * step) for _ in range(2))
    tokens = _log(rng, 1, 8192)
    # (int8 has no weight gradient)
    dtype = rng.choice(("bf16",) * 7 + ("f32",) * 2 + ("int8",))
    most = 8192 * 4096 * 14336 // (12 if dtype == "f32" else 3 if kind == "backward" else 1)
    tokens = max(1, min(tokens, most // (d_in * d_out)))
    act = rng.choice(ACTIVATIONS)
    if kind == "forward":
        return _fwd(None, tokens, d_in, d_out, dtype, act, rng.random() < 0.6, rng.random() < 0.5,
                    rng.random() < 0.4)
    return _bwd(None, tokens, d_in, d_out, dtype, act, dtype != "int8" and rng.random() < 0.5,
                rng.random() < 0.7)


def _sizes(case):
    """Elements of each float32 gradient (generator gradients, in pairs R, P)
    and of each bf16 one (`odd` norm weights and biases per layer set)."""
    b, tri = case["block"], case["block"] * (case["block"] - 1) // 2
    if case["layers"] == 0:  # one 2048 x 2048 projection
        shapes, times = [(2048, 2048)], 1
    else:  # q, k, v, o, gate, up, down
        shapes = [(4096, 4096), (1024, 4096), (1024, 4096), (4096, 4096), (14336, 4096),
                  (14336, 4096), (4096, 14336)]
        times = case["layers"]
    f32 = [d // b * tri for shape in shapes for d in shape] * times
    bf16 = [1024 * (i + 1) + 2 * i + 1 for i in range(case["odd"])] * times
    return f32, bf16


def _randn(gen, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "clip":
        f32, bf16 = _sizes(case)
        flat = {}
        for key, dt, sizes in (("f32", torch.float32, f32), ("bf16", torch.bfloat16, bf16)):
            # a training program's gradients: views of one flat buffer each
            # (and a second flat buffer for the clipped ones)
            flat[key] = _randn(gen, sum(sizes), scale=1e-2, dtype=dt)
            s["grad_" + key] = flat[key]
            s["out_" + key] = torch.zeros_like(flat[key])
        s["grads"] = list(flat["f32"].split(f32)) + (list(flat["bf16"].split(bf16)) if bf16 else [])
        s["outs"] = list(s["out_f32"].split(f32)) + (list(s["out_bf16"].split(bf16)) if bf16 else [])
        # (the expected norm is 1e-2 sqrt(n))
        s["max_norm"] = (0.3 if case["clipped"] else 3.0) * 1e-2 * math.sqrt(sum(f32) + sum(bf16))
        return s
    n, m, t = case["d_in"], case["d_out"], case["tokens"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    if case["dtype"] == "int8":
        s["W"] = torch.randint(-127, 128, (m, n), generator=gen, device="cuda", dtype=torch.int8)
        s["w_scale"] = (0.5 + torch.rand(m, generator=gen, device="cuda")) / (73.0 * math.sqrt(n))
    else:
        s["W"] = _randn(gen, m, n, scale=1.0 / math.sqrt(n), dtype=dt)
        s["w_scale"] = None
    if case["op"] == "forward":
        s["x"] = _randn(gen, t, n, dtype=dt)
        s["bias"] = _randn(gen, m, scale=0.5) if case["bias"] else None
        s["residual"] = _randn(gen, t, m, dtype=dt) if case["residual"] else None
    else:
        s["g_y"] = _randn(gen, t, m, scale=1e-2, dtype=dt)
        # what the forward kept: x for a trained weight, u for an activation
        s["x"] = _randn(gen, t, n, dtype=dt) if case["g_weight"] else None
        s["u"] = _randn(gen, t, m, dtype=dt) if case["activation"] != "none" else None
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"forward": _own_forward, "backward": _own_backward, "clip": _own_clip}[op](s)
    return {"forward": _plain_forward, "backward": _plain_backward, "clip": _plain_clip}[op](s)


def _own_forward(s):
    from orthogonal_equivalence_amd.dense import dense_forward
    c = s["case"]
    y, u = dense_forward(s["x"], s["W"], bias=s["bias"], residual=s["residual"],
                         activation=c["activation"], w_scale=s["w_scale"], save_u=c["save"])
    return {"y": y, "u": u}


def _own_backward(s):
    from orthogonal_equivalence_amd.dense import dense_backward
    c = s["case"]
    g_x, g_W, g_bias = dense_backward(s["g_y"], s["W"], x=s["x"], u=s["u"],
                                      activation=c["activation"], w_scale=s["w_scale"],
                                      need_g_W=c["g_weight"], need_g_bias=c["g_bias"])
    return {"g_x": g_x, "g_W": g_W, "g_bias": g_bias}


def _own_clip(s):
    from orthogonal_equivalence_amd.grads import clip_grads
    norm = clip_grads(s["grads"], s["max_norm"], outs=s["outs"])
    return {"norm": norm, "f32": s["out_f32"], "bf16": s["out_bf16"]}


def _act(u, name):
    if name == "relu":
        return torch.where(u > 0, u, torch.zeros_like(u))
    if name == "gelu":
        return 0.5 * u * (1.0 + torch.erf(u * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * u * (1.0 + torch.tanh(_C * (u + _A * u * u * u)))
    if name == "silu":
        return u / (1.0 + torch.exp(-u))
    return u


def _act_slope(u, name):
    if name == "relu":
        return (u > 0).to(u.dtype)
    if name == "gelu":
        return (0.5 * (1.0 + torch.erf(u * math.sqrt(0.5)))
                + u * torch.exp(-0.5 * u * u) * (1.0 / math.sqrt(2.0 * math.pi)))
    if name == "gelu_tanh":
        t = torch.tanh(_C * (u + _A * u * u * u))
        return 0.5 * (1.0 + t) + 0.5 * u * (1.0 - t * t) * _C * (1.0 + 3.0 * _A * u * u)
    p = 1.0 / (1.0 + torch.exp(-u))  # silu
    return p * (1.0 + u * (1.0 - p))


def _plain_forward(s):
    c, dt = s["case"], s["x"].dtype
    u = s["x"].float() @ s["W"].float().t()
    if s["w_scale"] is not None:
        u = u * s["w_scale"]
    if s["bias"] is not None:
        u = u + s["bias"]
    y = _act(u, c["activation"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(dt), "u": u.to(dt) if c["save"] else None}


def _plain_backward(s):
    c, dt = s["case"], s["g_y"].dtype
    g_u = s["g_y"].float()
    if c["activation"] != "none":
        g_u = g_u * _act_slope(s["u"].float(), c["activation"])
    g_q = g_u if s["w_scale"] is None else g_u * s["w_scale"]
    return {"g_x": (g_q @ s["W"].float()).to(dt),
            "g_W": (g_u.t() @ s["x"].float()).to(dt) if c["g_weight"] else None,
            "g_bias": g_u.sum(0) if c["g_bias"] else None}


def _plain_clip(s):
    # (squares in float64: a sum over hundreds of millions of values)
    norm = (s["grad_f32"].double().square().sum() + s["grad_bf16"].double().square().sum()).sqrt()
    k = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    return {"norm": norm.float(), "f32": s["grad_f32"] * k,
            "bf16": (s["grad_bf16"].float() * k).to(torch.bfloat16)}


def work(case):
    """Every input read once, every output written once; the products' flops
    (the elementwise work is not counted)."""
    if case["op"] == "clip":
        f32, bf16 = _sizes(case)
        n32, n16 = sum(f32), sum(bf16)
        return {"bytes": 2 * (4 * n32 + 2 * n16) + 4, "flops": 3.0 * (n32 + n16)}
    n, m, t = case["d_in"], case["d_out"], case["tokens"]
    es = 4 if case["dtype"] == "f32" else 2
    nbytes = m * n * (1 if case["dtype"] == "int8" else es) + (4 * m if case["dtype"] == "int8" else 0)
    if case["op"] == "forward":
        nbytes += t * n * es + t * m * es * (1 + case["residual"] + case["save"]) + 4 * m * case["bias"]
        return {"bytes": nbytes, "flops": 2.0 * t * n * m}
    nbytes += t * m * es * (1 + (case["activation"] != "none")) + t * n * es  # g_y, u; g_x
    nbytes += (t * n + m * n) * es * case["g_weight"] + 4 * m * case["g_bias"]
    return {"bytes": nbytes, "flops": 2.0 * t * n * m * (1 + case["g_weight"])}


def _exact_act(u, name):
    """act(u) and act'(u) in float64, from the normal distribution's and the
    logistic function's own definitions."""
    if name == "none":
        return u, torch.ones_like(u)
    if name == "relu":
        return u.clamp(min=0), torch.heaviside(u, torch.zeros_like(u))
    if name == "gelu":
        cdf = torch.special.ndtr(u)
        return u * cdf, cdf + u * torch.exp(-0.5 * u.square()) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":  # (1 + tanh z) / 2 is the logistic function of 2 z
        p = torch.special.expit(2 * _C * (u + _A * u ** 3))
        return u * p, p + u * p * (1 - p) * 2 * _C * (1 + 3 * _A * u.square())
    p = torch.special.expit(u)
    return u * p, p + u * p * (1 - p)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        flats = [s["grad_f32"], s["grad_bf16"]]
        norm = math.sqrt(sum(torch.linalg.vector_norm(f, dtype=torch.float64).item() ** 2
                             for f in flats if f.numel()))
        k = min(1.0, s["max_norm"] / norm)
        return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"),
                "f32": flats[0].double() * k, "bf16": flats[1].double() * k}
    W = s["W"].double()
    if s["w_scale"] is not None:
        W = W * s["w_scale"].double()[:, None]
    if case["op"] == "forward":
        u = torch.mm(s["x"].double(), W.t())
        u = u + s["bias"].double() if s["bias"] is not None else u
        y = _exact_act(u, case["activation"])[0]
        y = y + s["residual"].double() if s["residual"] is not None else y
        return {"y": y, "u": u if case["save"] else None}
    g_u = s["g_y"].double()
    if s["u"] is not None:
        g_u = g_u * _exact_act(s["u"].double(), case["activation"])[1]
    return {"g_x": torch.mm(g_u, W),
            "g_W": torch.mm(g_u.t(), s["x"].double()) if case["g_weight"] else None,
            "g_bias": g_u.sum(0) if case["g_bias"] else None}
