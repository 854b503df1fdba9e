"""Cases of the two losses that end in a projection onto a large vocabulary,
neither of which keeps the logits: softmax cross entropy, and distillation
from a teacher's top logits. Inputs, the plain form of each operator and its
definition in float64.

x [tokens, d] and W [vocab, d] share a type, z = x W^T are the logits, and
every row t carries a weight of its own in the backward:

  cross entropy   lse = log sum_j exp(z_j),  loss = lse - z[target]
                  g_z = (g_loss + g_lse) exp(z - lse) - g_loss [j = target]
                  (a target below 0: the row takes no part)
  distillation    p = softmax over the row's listed teacher logits / T,
                  lse = log sum_j exp(z_j / T),
                  loss = T^2 sum_k p_k (log p_k - z[id_k] / T + lse)
                  g_z = g_loss T (exp(z / T - lse) - sum_k p_k [j = id_k])
                  (an id below 0: the entry takes no part; a row without any
                  takes none itself)
  both            g_x = g_z W,  g_W = g_z^T x

The forward returns what the backward takes: lse, and for distillation the
student's logits at the listed ids.
"""
import math

import torch

own = False


def _case(name, op, tokens, d, vocab, dtype="bf16", ignored=0.0, g_weight=False, z_loss=False,
          top=0, temperature=1.0):
    c = dict(op=op, tokens=tokens, d=d, vocab=vocab, dtype=dtype, ignored=ignored)
    if op == "ce_backward":
        c.update(g_weight=g_weight, z_loss=z_loss)
    if op.startswith("distill"):
        c.update(top=top, temperature=temperature)
    if op == "distill_backward":
        c.update(g_weight=g_weight)
    return dict(c, name=name) if name else c


def listed():
    return [
        # scoring one token's continuation: the weight's bytes
        _case("ce_fwd_1tok", "ce_forward", 1, 4096, 131072),
        # a ragged validation batch of a small model, a vocabulary of odd size
        _case("ce_fwd_777tok", "ce_forward", 777, 2048, 50001, ignored=0.2),
        # a training step of an 8B-class model
        _case("ce_fwd_8192tok", "ce_forward", 8192, 4096, 131072),
        # its backward, head and activations
        _case("ce_bwd_8192tok", "ce_backward", 8192, 4096, 131072, ignored=0.05, g_weight=True),
        # a fine-tuning batch whose prompts are ignored, with a term on lse
        _case("ce_bwd_1000tok", "ce_backward", 1000, 2048, 50001, ignored=0.4, g_weight=True,
              z_loss=True),
        # a frozen head: the activations' gradient alone
        _case("ce_bwd_frozen_2048tok", "ce_backward", 2048, 4096, 32768),
        # the smallest, in float32: launch latency
        _case("ce_bwd_f32_64tok", "ce_backward", 64, 256, 1000, dtype="f32", g_weight=True),
        # a distillation step of a 1B-class student, 64 kept logits a token
        _case("distill_fwd_4096tok", "distill_forward", 4096, 2048, 65536, ignored=0.1, top=64,
              temperature=2.0),
        # a small ragged batch in float32
        _case("distill_fwd_f32_100tok", "distill_forward", 100, 1024, 5003, dtype="f32",
              ignored=0.1, top=8, temperature=1.0),
        # the backward of that step
        _case("distill_bwd_4096tok", "distill_backward", 4096, 2048, 65536, ignored=0.1,
              g_weight=True, top=64, temperature=2.0),
        # a ragged batch, few logits a token, frozen head
        _case("distill_bwd_500tok", "distill_backward", 500, 4096, 32001, ignored=0.3, top=16,
              temperature=1.5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Tokens from 1 to 8192, widths from 128 to 4096 in steps of 8 (a third
    of them multiples of 256), vocabularies from 200 to 131072 of any size, up
    to 128 teacher logits a token; bf16, and float32 at a twelfth of the work."""
    op = rng.choice(("ce_forward", "ce_backward", "distill_forward", "distill_backward"))
    step = rng.choice((8, 8, 256))
    d = max(step, _log(rng, 128, 4096) // step * step)
    vocab = _log(rng, 200, 131072)
    if rng.random() < 0.3:
        vocab = max(256, vocab // 256 * 256)
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    most = (8192 * 4096 * 131072 if op[:2] == "ce" else 4096 * 2048 * 65536) // (
        12 if dtype == "f32" else 1)
    tokens = max(1, min(_log(rng, 1, 8192), most // (d * vocab)))
    return _case(None, op, tokens, d, vocab, dtype, rng.choice((0.0, 0.1, 0.5)),
                 rng.random() < 0.6, rng.random() < 0.3, min(vocab, _log(rng, 1, 128)),
                 rng.choice((1.0, 1.5, 2.0, 4.0)))


def _pieces(vocab, n=16384):
    return [(v, min(v + n, vocab)) for v in range(0, vocab, n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, d, v, op = case["tokens"], case["d"], case["vocab"], case["op"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": case}
    # logits of standard deviation 2, and a part of each row along its target's
    # weights: target logits up to ~12, as a model in training has them
    s["W"] = randn(v, d).mul_(2.0 / math.sqrt(d)).to(dt)
    target = (v * rand(t) ** 2).long().clamp_(max=v - 1)
    s["x"] = (randn(t, d) + 2.5 * rand(t, 1) * s["W"][target].float()).to(dt)
    out = rand(t) < case["ignored"]  # prompts, padding
    if t > 1:
        out[t // 2] = False
    else:
        out[:] = False
    temp = case.get("temperature", 1.0)
    if op.startswith("ce"):
        s["targets"] = torch.where(out, torch.full_like(target, -100), target)
    else:
        # distinct ids in no order, the target first; some rows hold fewer
        k = case["top"]
        stride = 1 + (rand(t, 1) * max(1, (v - 1) // max(k, 1) - 1)).long()
        at = torch.arange(k, device="cuda")
        s["ids"] = (target[:, None] + at * stride) % v
        held = 1 + (rand(t, 1) * 1.5 * k).long()
        s["ids"] = torch.where((at >= held) | out[:, None], -1, s["ids"])
        fall = 12.0 * (at + rand(t, k)) / k
        s["teacher"] = 14.0 - fall.sqrt() * 3.0
    if op.endswith("backward"):
        s["g_loss"] = (0.5 + rand(t)) / t  # per-token weights of a mean
        m = torch.full((t,), -math.inf, device="cuda", dtype=torch.float32)
        e = torch.zeros(t, device="cuda")
        xf = s["x"].float()
        for a, b in _pieces(v):
            z = (xf @ s["W"][a:b].float().t()).div_(temp)
            m2 = torch.maximum(m, z.max(1).values)
            e = e * torch.exp(m - m2) + torch.exp(z.sub_(m2[:, None])).sum(1)
            m = m2
        s["lse"] = torch.where(out, torch.zeros_like(m), m + torch.log(e))
        if op == "ce_backward":
            s["g_lse"] = 2e-4 * s["lse"] / t if case["z_loss"] else None
        else:
            z = torch.empty(t, k, device="cuda")
            for i in range(k):
                z[:, i] = (xf * s["W"][s["ids"][:, i].clamp(min=0)].float()).sum(1)
            s["z"] = torch.where(s["ids"] >= 0, z, torch.zeros_like(z))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"ce_forward": _own_ce_forward, "ce_backward": _own_ce_backward,
                "distill_forward": _own_distill_forward,
                "distill_backward": _own_distill_backward}[op](s)
    return {"ce_forward": _plain_ce_forward, "ce_backward": _plain_ce_backward,
            "distill_forward": _plain_distill_forward,
            "distill_backward": _plain_distill_backward}[op](s)


def _own_ce_forward(s):
    from orthogonal_equivalence_amd.losses import cross_entropy_forward
    loss, lse = cross_entropy_forward(s["x"], s["W"], s["targets"])
    return {"loss": loss, "lse": lse}


def _own_ce_backward(s):
    from orthogonal_equivalence_amd.losses import cross_entropy_backward
    g_x, g_W = cross_entropy_backward(s["g_loss"], s["x"], s["W"], s["targets"], s["lse"],
                                      g_lse=s["g_lse"], need_g_W=s["case"]["g_weight"])
    return {"g_x": g_x, "g_W": g_W}


def _own_distill_forward(s):
    from orthogonal_equivalence_amd.losses import distill_forward
    loss, lse, z = distill_forward(s["x"], s["W"], s["ids"], s["teacher"],
                                   temperature=s["case"]["temperature"])
    return {"loss": loss, "lse": lse, "z": z}


def _own_distill_backward(s):
    from orthogonal_equivalence_amd.losses import distill_backward
    g_x, g_W = distill_backward(s["g_loss"], s["x"], s["W"], s["ids"], s["teacher"], s["lse"],
                                s["z"], temperature=s["case"]["temperature"],
                                need_g_W=s["case"]["g_weight"])
    return {"g_x": g_x, "g_W": g_W}


def _plain_lse(z):
    m = z.max(1, keepdim=True).values
    return (m + torch.log(torch.exp(z - m).sum(1, keepdim=True)))[:, 0]


def _plain_ce_forward(s):
    z = s["x"].float() @ s["W"].float().t()
    lse, y = _plain_lse(z), s["targets"]
    part = y >= 0
    loss = lse - z.gather(1, y.clamp(min=0)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return {"loss": torch.where(part, loss, zero), "lse": torch.where(part, lse, zero)}


def _plain_gradients(s, g_z):
    dt = s["x"].dtype
    return {"g_x": (g_z @ s["W"].float()).to(dt),
            "g_W": (g_z.t() @ s["x"].float()).to(dt) if s["case"]["g_weight"] else None}


def _plain_ce_backward(s):
    y = s["targets"]
    zero = torch.zeros_like(s["lse"])
    g = torch.where(y >= 0, s["g_loss"], zero)
    a = g if s["g_lse"] is None else torch.where(y >= 0, s["g_loss"] + s["g_lse"], zero)
    g_z = torch.exp(s["x"].float() @ s["W"].float().t() - s["lse"][:, None]) * a[:, None]
    g_z.scatter_add_(1, y.clamp(min=0)[:, None], -g[:, None])
    return _plain_gradients(s, g_z)


def _plain_teacher(s):
    """p and log p (0 where an entry takes no part), and the rows that do."""
    t = s["teacher"] / s["case"]["temperature"]
    held = s["ids"] >= 0
    part = held.any(1)
    t = torch.where(held, t, torch.full_like(t, -math.inf))
    m = torch.where(part, t.max(1).values, torch.zeros_like(t[:, 0]))[:, None]
    e = torch.exp(t - m)
    total = torch.where(part, e.sum(1), torch.ones_like(m[:, 0]))[:, None]
    log_p = torch.where(held, t - m - torch.log(total), torch.zeros_like(t))
    return e / total, log_p, part


def _plain_distill_forward(s):
    temp = s["case"]["temperature"]
    z = s["x"].float() @ s["W"].float().t()
    p, log_p, part = _plain_teacher(s)
    at = torch.where(s["ids"] >= 0, z.gather(1, s["ids"].clamp(min=0)), torch.zeros_like(p))
    lse = torch.where(part, _plain_lse(z / temp), torch.zeros_like(z[:, 0]))
    loss = temp * temp * (p * (log_p - at / temp + lse[:, None])).sum(1)
    return {"loss": loss, "lse": lse, "z": at}


def _plain_distill_backward(s):
    temp = s["case"]["temperature"]
    p, _, part = _plain_teacher(s)
    g = torch.where(part, s["g_loss"], torch.zeros_like(s["g_loss"]))[:, None] * temp
    g_z = torch.exp((s["x"].float() @ s["W"].float().t()) / temp - s["lse"][:, None]) * g
    g_z.scatter_add_(1, s["ids"].clamp(min=0), -g * p)
    return _plain_gradients(s, g_z)


def work(case):
    """Each input read once, each output written once; one product forward,
    and backward that product again (no logits are kept) beside one for each
    gradient. The elementwise work is not counted."""
    t, d, v = case["tokens"], case["d"], case["vocab"]
    es = 4 if case["dtype"] == "f32" else 2
    k = case.get("top", 0)
    nbytes = (t * d + v * d) * es + t * 8 * max(k, 1) + 4 * t * k
    if case["op"].endswith("forward"):
        return {"bytes": nbytes + 8 * t + 4 * t * k, "flops": 2.0 * t * d * v}
    gw = case["g_weight"]
    nbytes += 8 * t + 4 * t * k + 4 * t * case.get("z_loss", False) + (t * d + v * d * gw) * es
    return {"bytes": nbytes, "flops": 2.0 * t * d * v * (2 + gw)}


def _exact_teacher(s):
    held = s["ids"] >= 0
    t = torch.where(held, s["teacher"].double() / s["case"]["temperature"], -math.inf)
    part = held.any(1)
    log_p = t[part].log_softmax(1).masked_fill(~held[part], 0.0)
    p = t[part].softmax(1)
    full = [torch.zeros_like(t), torch.zeros_like(t)]
    full[0][part], full[1][part] = p, log_p
    return full[0], full[1], part


def exact(case, seed):
    s = prepare(case, seed)
    x, v, temp = s["x"].double(), case["vocab"], case.get("temperature", 1.0)
    ce = case["op"].startswith("ce")
    if ce:
        ids = s["targets"][:, None]
        part = s["targets"] >= 0
        p = part.double()[:, None]
        log_p = torch.zeros_like(p)
    else:
        ids = s["ids"]
        p, log_p, part = _exact_teacher(s)
    if case["op"].endswith("forward"):
        parts, z_at = [], torch.zeros_like(p)
        for a, b in _pieces(v):
            z = x @ s["W"][a:b].double().t()
            here = (ids >= a) & (ids < b)
            z_at = torch.where(here, z.gather(1, (ids - a).clamp(0, b - a - 1)), z_at)
            parts.append((z / temp).logsumexp(1))
        lse = torch.stack(parts).logsumexp(0)
        loss = temp ** 2 * (p * (log_p - z_at / temp + lse[:, None])).sum(1)
        got = {"loss": loss * part, "lse": lse * part}
        return got if ce else dict(got, z=z_at)
    g = s["g_loss"].double() * part * temp
    a_t = g
    if ce and s["g_lse"] is not None:
        a_t = g + s["g_lse"].double() * part
    g_x = torch.zeros_like(x)
    g_W = []
    for a, b in _pieces(v):
        w = s["W"][a:b].double()
        g_z = (x @ w.t() / temp - s["lse"].double()[:, None]).exp_() * a_t[:, None]
        rows, cols = ((ids >= a) & (ids < b)).nonzero(as_tuple=True)
        g_z.index_put_((rows, ids[rows, cols] - a), -(g[:, None] * p)[rows, cols], accumulate=True)
        g_x += g_z @ w
        if case["g_weight"]:
            g_W.append(g_z.t() @ x)
    return {"g_x": g_x, "g_W": torch.cat(g_W) if g_W else None}
