"""Sizes that run every kernel variant the dense linear's plans choose, and
operands of small integers, whose products and sums float32 holds exactly in
any order: the outputs are compared bit for bit.

A case is (float type, INT8 weight, tokens, d_in, d_out), float type 0 float32
and 1 bfloat16."""
import torch

F32, BF16 = 0, 1
DTYPE = {F32: torch.float32, BF16: torch.bfloat16}

# a small cover of the variants of 150 000 drawn products (1 .. 8192 tokens,
# widths 8 .. 14336), and ordinary sizes behind it
CASES = [
    (0, 0, 1, 40, 40), (0, 0, 9, 336, 4384), (0, 0, 43, 9392, 1024), (0, 0, 317, 1792, 2560),
    (0, 0, 1255, 40, 1224), (0, 0, 1362, 1408, 376), (0, 0, 1525, 1144, 40),
    (0, 0, 3417, 136, 4920), (0, 0, 4523, 8, 11056), (0, 1, 1, 72, 40), (0, 1, 1, 552, 552),
    (0, 1, 445, 1240, 1208), (0, 1, 6172, 256, 256), (1, 0, 1, 48, 40), (1, 0, 1, 336, 4320),
    (1, 0, 9, 80, 9376), (1, 0, 10, 8368, 192), (1, 0, 130, 6144, 8448), (1, 0, 336, 328, 3768),
    (1, 0, 445, 208, 14128), (1, 0, 518, 10000, 472), (1, 0, 644, 64, 13984),
    (1, 0, 717, 11040, 96), (1, 0, 940, 3496, 72), (1, 0, 1305, 56, 40), (1, 0, 2304, 4712, 32),
    (1, 0, 2828, 8, 3632), (1, 0, 2978, 9080, 40), (1, 0, 4247, 472, 752), (1, 0, 4618, 9144, 152),
    (1, 0, 4657, 272, 72), (1, 0, 5872, 72, 3408), (1, 0, 6098, 136, 328), (1, 1, 1, 40, 40),
    (1, 1, 1, 64, 1224), (1, 1, 13, 40, 40), (1, 1, 33, 3712, 1040), (1, 1, 35, 608, 7032),
    (1, 1, 66, 3048, 2112), (1, 1, 67, 40, 11912), (1, 1, 74, 3656, 3440), (1, 1, 75, 11048, 40),
    (1, 1, 80, 4328, 4432), (1, 1, 107, 328, 9560), (1, 1, 146, 8704, 4608), (1, 1, 150, 48, 11656),
    (1, 1, 157, 5576, 8648), (1, 1, 171, 9856, 40), (1, 1, 528, 96, 13424), (1, 1, 1207, 48, 3712),
    (1, 1, 1470, 3640, 40), (1, 1, 1508, 72, 4008), (1, 1, 1688, 128, 6144), (1, 1, 2335, 3696, 96),
    (1, 1, 2816, 12336, 1408), (1, 1, 4751, 648, 392), (1, 1, 5888, 136, 424), (1, 1, 6280, 48, 144),
    (1, 1, 7039, 584, 696),
    (0, 0, 14, 200, 1768), (0, 0, 40, 9752, 10152), (0, 0, 309, 11104, 11672), (0, 0, 1024, 2048, 2048),
    (1, 0, 43, 848, 3504), (1, 0, 54, 5280, 1872), (1, 0, 80, 152, 12176), (1, 0, 100, 4096, 4096),
    (1, 0, 173, 11048, 2968), (1, 0, 190, 13568, 7168), (1, 0, 195, 360, 14272),
    (1, 0, 443, 640, 13432), (1, 1, 284, 2448, 952), (1, 1, 376, 1872, 4288),
    (1, 1, 397, 1184, 11648),
]


def variants(case, plan):
    """What the calls of a case run, by the fields of test_dense_plan.plans: the
    forward, g_x alone, g_W alone, and both."""
    t, int8, tokens, d_in, _ = case
    kind = ("f32", "bf16")[t] + (" int8" if int8 else "")
    if plan["stream"]:
        found = {("forward", kind, "stream", d_in % 16 == 0 if int8 else None)}
    elif plan["dense"]:
        found = {("forward", kind, "256 x 256", plan["widen"], plan["w_tiled"])}
    else:
        found = {("forward", kind, plan["widen"], plan["shape"], plan["split"] > 1)}
    if plan["b_dense"]:
        found.add(("g_x", kind, "256 x 256", tokens % 256 == 0))
    else:
        found.add(("g_x", kind, plan["gx_shape"], plan["gx_split"] > 1))
    if not int8:
        found.add(("g_W", kind, plan["gw_shape"], plan["gw_split"] > 1))
        if plan["paired"]:
            found.add(("both", kind, plan["px_shape"], plan["px_split"] > 1, plan["pw_split"] > 1))
    return found


def integers(gen, shape, top, share, device):
    """int16: about `share` of them integers of 1 .. top in size, the rest 0."""
    v = torch.randint(1, top + 1, shape, generator=gen, device=device, dtype=torch.int16)
    v *= torch.randint(0, 2, shape, generator=gen, device=device, dtype=torch.int16) * 2 - 1
    if share < 1:
        v *= torch.randint(0, 1000, shape, generator=gen, device=device,
                           dtype=torch.int16) < int(1000 * share)
    return v


def operands(gen, t, n, left, right, device):
    """Two operands of sums over n products whose absolute values add up to less
    than 2^24, and to some hundreds where that is enough (so that bfloat16
    shows the last unit too): bfloat16 of sizes up to 2, float32 up to 4095
    (more bits than any shorter type keeps) and 2."""
    share = min(1.0, (300 / n) ** 0.5)
    top = 2 if t == BF16 else 4095
    return (integers(gen, left, top, share, device).to(DTYPE[t]),
            integers(gen, right, 2, share, device).to(DTYPE[t]))
