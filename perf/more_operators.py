"""The operators of a stack's plain layers and of its training step, as they are measured: the gated projections and the
matrix product with an epilogue, the gradients of both, and the AdamW step over many tensors.

`run` computes a case in plain torch (own = False) or through the library's entry points (own = True); both take the
same tensors. `exact` gives the same outputs in 64 bits from the definitions.

Definitions (rows t, channels c; a' the derivative of the activation a):
  linear       p = x W^T + b,  y = r + s a(p)
  linear_grad  q = s dy a'(p),  dx = q W,  dW = q^T x,  db = sum of q over the rows
  gated        g = x Wg^T + bg,  u = x Wu^T + bu,  z = a(g) u
  gated_grad   dg = dz u a'(g),  du = dz a(g),  dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x, and their sums
  adamw        g' = g min(1, tau / N),  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2,
               w' = w (1 - lr wd) - lr (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps)
               with 8-bit states m' and v' are then held as codes (`encode` below) and come back as their values
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ADAM = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
BLOCK = 256  # elements of an 8-bit state that share a scale


def size(name):
    return 4 if name == "f32" else 2


# ---------------------------------------------------------------- cases


def listed():
    return [
        # the down projection of one decoded token, into an fp32 residual stream: latency
        dict(name="linear 1 token", op="linear", M=1, K=9728, N=2560, t="bf16", y="f32", act="none", bias=False,
             res=True, s=1.0),
        # the down projection of a layer of the 36-layer stack: 2 x 16384 tokens, fp32 residual stream
        dict(name="linear 32768 tokens", op="linear", M=32768, K=9728, N=2560, t="bf16", y="f32", act="none",
             bias=False, res=True, s=1.0),
        # a projection with bias and activation over a ragged batch of odd widths
        dict(name="linear 4099 tokens, odd", op="linear", M=4099, K=1021, N=2047, t="bf16", y="bf16", act="gelu",
             bias=True, res=False, s=1.0),
        # its backward pass at the width of the four-sequence workload
        dict(name="linear_grad 8192 tokens, gelu", op="linear_grad", M=8192, K=1024, N=4096, t="bf16", y="bf16",
             act="gelu", bias=True, s=1.0),
        # the backward pass of a small fp32 projection over a short ragged batch
        dict(name="linear_grad 3x411, fp32", op="linear_grad", M=1233, K=1024, N=512, t="f32", y="f32", act="none",
             bias=True, s=0.5),
        # eight sequences that each decode one token: the weights' bytes count
        dict(name="gated 8 tokens", op="gated", M=8, d=2560, f=9728, t="bf16", act="silu", bias=False, keep=False),
        # a training step's forward pass of a layer of the stack, with what its backward pass needs
        dict(name="gated 32768 tokens", op="gated", M=32768, d=2560, f=9728, t="bf16", act="silu", bias=False,
             keep=True),
        # its backward pass
        dict(name="gated_grad 32768 tokens", op="gated_grad", M=32768, d=2560, f=9728, t="bf16", act="silu",
             bias=False),
        # a small layer in fp32 with biases, forward and backward of a few documents
        dict(name="gated_grad 2000 tokens, fp32", op="gated_grad", M=2000, d=512, f=1365, t="f32", act="gelu",
             bias=True),
        # norm weights, gates and target taps of 36 layers: many small tensors, fp32 states, clipped
        dict(name="adamw 144 small tensors", op="adamw", layers=36, d=2560, f=0, vocab=0, w="f32", g="f32", bits=32,
             clip=True),
        # two layers of the 4B class, bf16 gradients, fp32 weights and states with bf16 copies for the next pass
        dict(name="adamw 2 layers, 32 bits", op="adamw", layers=2, d=2560, f=9728, vocab=0, w="f32", g="bf16", bits=32,
             clip=True),
        # the same with the token table, weights in bf16 and states in 8 bits
        dict(name="adamw 2 layers and table, 8 bits", op="adamw", layers=2, d=2560, f=9728, vocab=50000, w="bf16",
             g="bf16", bits=8, clip=False),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, its logarithm uniform."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def width(rng, hi):
    """A width: mostly a multiple of 64, now and then of 8, now and then any number."""
    d = spread(rng, 64, hi)
    kind = rng.random()
    return max(64, d // 64 * 64) if kind < 0.6 else max(64, d // 8 * 8) if kind < 0.8 else d


MOST = 32768 * 2560 * 9728  # products of a drawn case


def draw(rng):
    op = rng.choice(["linear", "linear_grad", "gated", "gated_grad", "adamw"])
    t = "f32" if rng.random() < 0.2 else "bf16"
    act = rng.choice(["none", "silu", "gelu", "relu"])
    if op.startswith("linear"):
        K, N = width(rng, 10240), width(rng, 10240)
        M = spread(rng, 1, max(1, min(32768, MOST // (K * N) // (4 if t == "f32" else 1))))
        y = "f32" if t == "f32" else rng.choice(["bf16", "f32"])
        case = dict(op=op, M=M, K=K, N=N, t=t, y=y, act=act, bias=rng.random() < 0.5, s=rng.choice([1.0, 0.5]))
        if op == "linear":
            case["res"] = rng.random() < 0.6
        return case
    if op.startswith("gated"):
        d, f = width(rng, 4096), width(rng, 10240)
        M = spread(rng, 1, max(1, min(32768, MOST // (d * f) // (4 if t == "f32" else 1))))
        act = "silu" if act == "none" else act
        case = dict(op=op, M=M, d=d, f=f, t=t, act=act, bias=rng.random() < 0.3)
        if op == "gated":
            case["keep"] = rng.random() < 0.5
        return case
    bits = rng.choice([8, 32])
    case = dict(op=op, layers=rng.randint(1, 12), d=width(rng, 2560), f=rng.choice([0, spread(rng, 64, 9728)]),
                vocab=rng.choice([0, spread(rng, 256, 32768)]), w=rng.choice(["f32", "bf16"]),
                g=rng.choice(["f32", "bf16"]), bits=bits, clip=rng.random() < 0.5)
    while weights(case) > 250_000_000:
        case["layers"] -= 1
    return case


def shapes(case):
    """The parameters: per layer two norm weights, a gate, five target taps and, with f, the three matrices; with
    vocab, the token table."""
    d, f, v = case["d"], case["f"], case["vocab"]
    layer = [(d,), (d,), (d,), (5, d)] + ([(f, d), (f, d), (d, f)] if f else [])
    return layer * case["layers"] + ([(v, d)] if v else [])


def weights(case):
    return sum(math.prod(s) for s in shapes(case))


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(DT[dtype])

    s, op = dict(case), case["op"]
    if op.startswith("linear"):
        M, K, N, t = case["M"], case["K"], case["N"], case["t"]
        s["in"] = normal((M, K), t)
        s["W"] = normal((N, K), t, K ** -0.5)
        s["b"] = normal((N,), t, 0.2) if case["bias"] else None
        if op == "linear":
            s["r"] = normal((M, N), case["y"], 2.0) if case["res"] else None
        else:
            s["dy"] = normal((M, N), case["y"], 1e-3)
            s["p"] = None if case["act"] == "none" else normal((M, N), t)  # as the forward pass kept it
        return s
    if op.startswith("gated"):
        M, d, f, t = case["M"], case["d"], case["f"], case["t"]
        s["in"] = normal((M, d), t)
        s["Wg"], s["Wu"] = normal((f, d), t, d ** -0.5), normal((f, d), t, d ** -0.5)
        s["bg"], s["bu"] = (normal((f,), t, 0.2), normal((f,), t, 0.2)) if case["bias"] else (None, None)
        if op == "gated_grad":
            s["dz"] = normal((M, f), t, 1e-3)
            s["g"], s["u"] = normal((M, f), t), normal((M, f), t)  # as the forward pass kept them
        return s
    # parameters and states as a training program holds them: views of flat buffers
    at, spans = 0, []
    for sh in shapes(case):
        spans.append((at, sh))
        at += math.prod(sh)

    def views(flat):
        return [flat[i:i + math.prod(sh)].view(sh) for i, sh in spans]

    s["flat_w"], s["flat_g"] = normal((at,), case["w"], 0.02), normal((at,), case["g"], 1e-3)
    s["ws"], s["gs"] = views(s["flat_w"]), views(s["flat_g"])
    m, v = normal((at,), "f32", 3e-4), normal((at,), "f32", 1e-3).square_()
    if case["bits"] == 32:
        s["flat_m"], s["flat_v"] = m, v
    else:
        s["flat_m"], s["flat_v"] = (torch.empty((at,), dtype=torch.uint8, device="cuda") for _ in range(2))
        s["tops"] = []
        for x, cm, cv, a, b in zip(s["ws"], views(s["flat_m"]), views(s["flat_v"]), views(m), views(v)):
            top = torch.empty((2, -(-x.numel() // BLOCK)), dtype=torch.int16, device="cuda")
            zero = torch.zeros((x.numel(),), dtype=torch.int64, device="cuda")
            cm.copy_(encode(a.reshape(-1), zero, True, top[0]).view(x.shape))
            cv.copy_(encode(b.reshape(-1), zero, False, top[1]).view(x.shape))
            s["tops"].append(top)
        s["val_m"], s["val_v"] = torch.zeros_like(m), torch.zeros_like(v)
        s["vms"], s["vvs"] = views(s["val_m"]), views(s["val_v"])
    del m, v
    s["ms"], s["vs"] = views(s["flat_m"]), views(s["flat_v"])
    # fp32 weights keep a bf16 copy for the next forward pass
    s["flat_c"] = s["flat_w"].bfloat16() if case["w"] == "f32" else None
    s["cs"] = None if s["flat_c"] is None else views(s["flat_c"])
    s["step"], s["seed"] = 100, seed % 65536
    s["norm"] = s["flat_g"].float().norm().reshape(1) if case["clip"] else None
    s["tau"] = 0.5e-3 * math.sqrt(weights(case)) if case["clip"] else math.inf
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import chunk_wise_weight_amd as ttt

    op = s["op"]
    act = s.get("act")
    act = None if act == "none" else act
    if op == "linear":
        return ttt.ttt_linear(s["in"], s["W"], s["b"], act=act, residual=s["r"], scale=s["s"], dtype=DT[s["y"]])
    if op == "linear_grad":
        got = ttt.ttt_linear_grad(s["dy"], s["in"], s["W"], act=act, pre=s["p"], scale=s["s"], bias=s["bias"])
        return {k: v for k, v in got._asdict().items() if v is not None}
    if op == "gated":
        if s["keep"]:
            z, g, u = ttt.ttt_gated(s["in"], s["Wg"], s["Wu"], s["bg"], s["bu"], act=act, keep=True)
            return {"z": z, "g": g, "u": u}
        return {"z": ttt.ttt_gated(s["in"], s["Wg"], s["Wu"], s["bg"], s["bu"], act=act)}
    if op == "gated_grad":
        got = ttt.ttt_gated_grad(s["dz"], s["in"], s["Wg"], s["Wu"], s["g"], s["u"], act=act, bias=s["bias"])
        return {k: v for k, v in got._asdict().items() if v is not None}
    more = {} if s["bits"] == 32 else {"tops": s["tops"], "seed": s["seed"]}
    ttt.ttt_adamw(s["ws"], s["gs"], s["ms"], s["vs"], s["step"], copies=s["cs"], norm=s["norm"], tau=s["tau"], **ADAM,
                  **more)
    if s["bits"] == 8:
        ttt.ttt_adamw_values(s["ms"], s["tops"], 1, out=s["vms"])
        ttt.ttt_adamw_values(s["vs"], s["tops"], 2, out=s["vvs"])
    return adam_outputs(s)


def adam_outputs(s):
    names = ("flat_m", "flat_v") if s["bits"] == 32 else ("val_m", "val_v")
    got = {"w": s["flat_w"], "m": s[names[0]], "v": s[names[1]]}
    if s["flat_c"] is not None:
        got["copy"] = s["flat_c"]
    return got


C0, C1 = math.sqrt(2 / math.pi), 0.044715


def activate(p, act):
    """The activation and its derivative."""
    if act == "none":
        return p, torch.ones_like(p)
    if act == "relu":
        return p.clamp(min=0), (p > 0).to(p.dtype)
    if act == "silu":
        h = 1 / (1 + torch.exp(-p))
        return p * h, h * (1 + p * (1 - h))
    # gelu by tanh: p sigmoid(2 w), w = C0 (p + C1 p^3)
    h = 1 / (1 + torch.exp(-2 * C0 * (p + C1 * p * p * p)))
    return p * h, h + p * h * (1 - h) * 2 * C0 * (1 + 3 * C1 * p * p)


def run_plain(s):
    op = s["op"]
    if op == "adamw":
        return plain_adamw(s)
    t, x = s["in"].dtype, s["in"].float()
    if op == "linear":
        p = x @ s["W"].float().T
        if s["b"] is not None:
            p = p + s["b"].float()
        y = activate(p, s["act"])[0] if s["act"] != "none" else p
        if s["s"] != 1.0:
            y = y * s["s"]
        return (y if s["r"] is None else y + s["r"].float()).to(DT[s["y"]])
    if op == "linear_grad":
        q = s["dy"].float()
        if s["act"] != "none":
            q = q * activate(s["p"].float(), s["act"])[1]
        if s["s"] != 1.0:
            q = q * s["s"]
        out = {"dx": (q @ s["W"].float()).to(t), "dw": (q.T @ x).to(t)}
        if s["bias"]:
            out["dbias"] = q.sum(0)
        return out
    if op == "gated":
        g, u = x @ s["Wg"].float().T, x @ s["Wu"].float().T
        if s["bg"] is not None:
            g, u = g + s["bg"].float(), u + s["bu"].float()
        z = (activate(g, s["act"])[0] * u).to(t)
        return {"z": z, "g": g.to(t), "u": u.to(t)} if s["keep"] else {"z": z}
    a, da = activate(s["g"].float(), s["act"])
    dz = s["dz"].float()
    dg, du = dz * s["u"].float() * da, dz * a
    out = {"dx": (dg @ s["Wg"].float() + du @ s["Wu"].float()).to(t), "dw_gate": (dg.T @ x).to(t),
           "dw_up": (du.T @ x).to(t)}
    if s["bias"]:
        out["db_gate"], out["db_up"] = dg.sum(0), du.sum(0)
    return out


# 8-bit states. A block of 256 elements has a top T, the smallest multiple of 2^20 that no |x| of the block passes as an
# fp32 bit pattern (3 mantissa bits and the exponent), in units of 2^20. A code c > 0 stands for the pattern
# (T - most + c) << 20 (0 where that is not positive), most = 127 for m (whose code has the sign above) and 255 for v;
# code 0 for 0. |x| is rounded to one of its two neighbours at random, by 16 random bits, so that its expectation is kept.


def blocks(x):
    pad = -x.numel() % BLOCK
    return torch.cat([x, x.new_zeros(pad)]).view(-1, BLOCK) if pad else x.view(-1, BLOCK)


def value(k):
    """The fp32 number of pattern k << 20, 0 for k <= 0."""
    return (k.clamp(min=0) << 20).to(torch.int32).view(torch.float32)


def encode(x, r, signed, top):
    """Codes of the fp32 vector x with 16 random bits r per element; the blocks' tops go into `top`."""
    most = 127 if signed else 255
    n, x, r = x.numel(), blocks(x), blocks(r)
    mag = x.abs().contiguous().view(torch.int32).long()
    T = (mag.amax(1, keepdim=True) + 0xFFFFF) >> 20
    top.copy_(T.view(-1))
    c = ((mag + (r << 4)) >> 20) - T + most
    if signed:
        low = (x.abs() >= (r + 0.5).float() * 2.0 ** -16 * value(T - most + 1)).long()
    else:
        low = torch.ones_like(c)  # a second moment that is not 0 is not held as 0: the step divides by it
    c = torch.where(mag == 0, 0, torch.where(c < 1, low, c))
    if signed:
        c = c + ((x < 0) & (c > 0)).long() * 128
    return c.to(torch.uint8).view(-1)[:n]


def decode(codes, top, signed):
    most = 127 if signed else 255
    c = blocks(codes.reshape(-1)).int()
    k = c & most
    v = torch.where(k > 0, value(top.int()[:, None] - most + k), 0.0)
    return (torch.where(c >= 128, -v, v) if signed else v).view(-1)[:codes.numel()]


def mix(h):
    h = ((h ^ (h >> 16)) * 0x6C8E9CF5) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0x51ED2701) & 0xFFFFFFFF
    return h ^ (h >> 16)


def random_bits(seed, step, tensor, n, device):
    """32 bits for each of n elements (n up to 2^32) of a tensor of the list."""
    key = mix((seed + 0x9E3779B1 * mix(step & 0xFFFFFFFF)) & 0xFFFFFFFF)
    key = mix((key + 0x9E3779B1 * (tensor + 1)) & 0xFFFFFFFF)
    e = torch.arange(n, device=device)
    return mix((key + e * 0x9E3779B1) & 0xFFFFFFFF)


def plain_adamw(s):
    b1, b2 = ADAM["betas"]
    lr, eps, wd, t = ADAM["lr"], ADAM["eps"], ADAM["weight_decay"], s["step"]
    c1, c2 = 1 - b1 ** t, 1 - b2 ** t
    clip = None if s["norm"] is None else (s["tau"] / s["norm"].double()).clamp(max=1.0)

    def apply(w, m, v, copy):
        x = w.float()
        x = x * (1 - lr * wd) - (lr / c1) * m / ((v / c2).sqrt() + eps)
        w.copy_(x)
        if copy is not None:
            copy.copy_(x)

    if s["bits"] == 32:
        g = s["flat_g"].float() if clip is None else (s["flat_g"].double() * clip).float()
        s["flat_m"].mul_(b1).add_(g * (1 - b1))
        s["flat_v"].mul_(b2).add_(g * g * (1 - b2))
        apply(s["flat_w"], s["flat_m"], s["flat_v"], s["flat_c"])
        return adam_outputs(s)
    # in 64 bits up to the rounding: values next to a border between two codes
    for i, (w, g, m, v, top) in enumerate(zip(s["ws"], s["gs"], s["ms"], s["vs"], s["tops"])):
        g = g.reshape(-1).double()
        g = g if clip is None else g * clip
        m1 = (b1 * decode(m, top[0], True).double() + (1 - b1) * g).float()
        v1 = (b2 * decode(v, top[1], False).double() + (1 - b2) * g * g).float()
        apply(w.view(-1), m1, v1, None if s["cs"] is None else s["cs"][i].view(-1))
        r = random_bits(s["seed"], t, i, g.numel(), g.device)
        m.view(-1).copy_(encode(m1, r & 0xFFFF, True, top[0]))
        v.view(-1).copy_(encode(v1, r >> 16, False, top[1]))
        s["vms"][i].view(-1).copy_(decode(m, top[0], True))
        s["vvs"][i].view(-1).copy_(decode(v, top[1], False))
    return adam_outputs(s)


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    """From the definitions; gradients by differentiation."""
    s = prepare(case, seed)
    op = s["op"]

    def double(name):
        return None if s[name] is None else s[name].double()

    def act(p):
        if case["act"] == "silu":
            return p * torch.sigmoid(p)
        if case["act"] == "gelu":
            return 0.5 * p * (1 + torch.tanh(C0 * (p + C1 * p ** 3)))
        return torch.relu(p) if case["act"] == "relu" else p

    def through(inputs, f):
        """Gradient of f with respect to its inputs, given that of its outputs, elementwise functions only."""
        leaves = [x.requires_grad_() for x in inputs]
        return torch.autograd.grad(f(*leaves), leaves)

    if op == "linear":
        p = torch.mm(double("in"), double("W").T)
        p = p if s["b"] is None else p + double("b")
        y = case["s"] * act(p)
        return y if s["r"] is None else y + double("r")
    if op == "linear_grad":
        if case["act"] == "none":
            q = double("dy") * case["s"]
        else:
            q, = through([double("p")], lambda p: (case["s"] * act(p) * double("dy")).sum())
        out = {"dx": torch.mm(q, double("W")), "dw": torch.mm(q.T.contiguous(), double("in"))}
        return {**out, "dbias": q.sum(0)} if case["bias"] else out
    if op == "gated":
        g, u = torch.mm(double("in"), double("Wg").T), torch.mm(double("in"), double("Wu").T)
        if case["bias"]:
            g, u = g + double("bg"), u + double("bu")
        return {"z": act(g) * u, "g": g, "u": u} if case["keep"] else {"z": act(g) * u}
    if op == "gated_grad":
        dg, du = through([double("g"), double("u")], lambda g, u: (act(g) * u * double("dz")).sum())
        out = {"dx": torch.mm(dg, double("Wg")) + torch.mm(du, double("Wu")),
               "dw_gate": torch.mm(dg.T.contiguous(), double("in")), "dw_up": torch.mm(du.T.contiguous(), double("in"))}
        return {**out, "db_gate": dg.sum(0), "db_up": du.sum(0)} if case["bias"] else out
    b1, b2 = ADAM["betas"]
    t, factor = s["step"], 1.0
    if s["norm"] is not None:
        factor = min(1.0, s["tau"] / float(s["norm"].double()))
    out = {k: torch.zeros(s["flat_w"].shape, dtype=torch.float64, device="cuda") for k in ("w", "m", "v")}
    for i, w in enumerate(s["ws"]):
        at = slice(w.storage_offset(), w.storage_offset() + w.numel())
        g = s["gs"][i].double().view(-1) * factor
        if case["bits"] == 32:
            m, v = s["ms"][i].double().view(-1), s["vs"][i].double().view(-1)
        else:
            m, v = decode(s["ms"][i], s["tops"][i][0], True).double(), decode(s["vs"][i], s["tops"][i][1], False).double()
        m, v = torch.lerp(g, m, b1), torch.lerp(g ** 2, v, b2)
        step = (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + ADAM["eps"])
        out["w"][at] = w.double().view(-1) * (1 - ADAM["lr"] * ADAM["weight_decay"]) - ADAM["lr"] * step
        if case["bits"] == 32:
            out["m"][at], out["v"][at] = m, v
    if case["bits"] == 8:
        out["m"] = out["v"] = None  # drawn among two neighbours: held to the plain form's
    if s["flat_c"] is not None:
        out["copy"] = out["w"]
    return out


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op.startswith("linear"):
        M, K, N, t, y = case["M"], case["K"], case["N"], size(case["t"]), size(case["y"])
        bias = N * t if case["bias"] else 0
        if op == "linear":
            return {"bytes": (M * K + N * K) * t + bias + M * N * y * (2 if case["res"] else 1), "flops": 2 * M * N * K}
        kept = 0 if case["act"] == "none" else M * N * t
        return {"bytes": 2 * (M * K + N * K) * t + M * N * y + kept + 2 * bias, "flops": 4 * M * N * K}
    if op.startswith("gated"):
        M, d, f, t = case["M"], case["d"], case["f"], size(case["t"])
        if op == "gated":
            return {"bytes": (M * d + 2 * f * d + M * f * (3 if case["keep"] else 1)) * t, "flops": 4 * M * d * f}
        return {"bytes": (2 * M * d + 4 * f * d + 3 * M * f) * t, "flops": 8 * M * d * f}
    n, state = weights(case), case["bits"] // 8
    copy = 2 if case["w"] == "f32" else 0
    # the values of 8-bit states are asked for too: codes read again, 4 bytes each written
    values = 0 if case["bits"] == 32 else 2 * (1 + 4)
    return {"bytes": n * (2 * size(case["w"]) + size(case["g"]) + 4 * state + copy + values), "flops": 16 * n}
