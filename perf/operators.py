"""The operators around the layer, as they are measured: token embedding and its gradient, the norms between layers
with gate and residual scale, and the global gradient norm with clipping.

`run` computes a case in plain torch (own = False) or through the library's entry points (own = True); both take the
same tensors. `exact` gives the same outputs in 64 bits from the definitions.

Definitions (t a token row, c a channel; mean over c):
  embed        x[t] = scale * E[ids[t]], a zero row for an id outside [0, vocab)
  embed_grad   dE[v] = scale * sum of dx[t] over the t with ids[t] = v
  norm_pre     x = w * h * r(h),  r(h) = (mean h^2 + eps)^(-1/2)
  norm_post    o = alpha h + beta a * w * y * r(y),  x = w_next * o * r(o)   (a: a gate per channel, per token, or none)
  ..._grad     their gradients, for the gradients of x and, from the rows after, of h or o
  clip         g * min(1, tau / N),  N = the 2-norm of all gradients together, into a copy or in place
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def size(name):
    return 4 if name == "f32" else 2


# ---------------------------------------------------------------- cases


def listed():
    return [
        # eight sequences that each decode one token: latency
        dict(name="embed 8 single tokens", op="embed", B=8, T=1, vocab=151936, d=2560, table="bf16", x="f32"),
        # the long stream of the layer benchmark, into an fp32 residual stream
        dict(name="embed 131072 tokens", op="embed", B=1, T=131072, vocab=151936, d=2560, table="bf16", x="f32"),
        # a small table in fp32 and a short ragged batch
        dict(name="embed_grad 3x411, small table", op="embed_grad", B=3, T=411, vocab=512, d=1024, dx="f32", dE="f32"),
        # a training step of two sequences of 16384 tokens on the large table
        dict(name="embed_grad 2x16384 tokens", op="embed_grad", B=2, T=16384, vocab=151936, d=2560, dx="bf16",
             dE="f32"),
        # one decoded token before its first layer: latency
        dict(name="norm_pre 1 token", op="norm_pre", rows=1, d=2560, h="f32", x="bf16", w="f32"),
        # between two layers of the 36-layer stack: 2 x 16384 tokens, fp32 residual stream, a learned gate per channel
        dict(name="norm_post 32768 tokens", op="norm_post", rows=32768, d=2560, h="f32", y="bf16", x="bf16", w="f32",
             gate="channel", alpha=1.0, beta=0.5, next=True),
        # a ragged batch of an odd width, all in bf16, a gate per token
        dict(name="norm_post 4099 tokens, d 1023", op="norm_post", rows=4099, d=1023, h="bf16", y="bf16", x="bf16",
             w="bf16", gate="token", alpha=1.0, beta=1.0, next=True),
        # the backward pass of a first norm: four sequences of 8192 tokens
        dict(name="norm_pre_grad 32768 tokens", op="norm_pre_grad", rows=32768, d=1024, h="bf16", x="bf16", w="bf16"),
        # the backward pass between two layers of the stack
        dict(name="norm_post_grad 32768 tokens", op="norm_post_grad", rows=32768, d=2560, h="f32", y="bf16", x="bf16",
             w="f32", gate="channel", alpha=1.0, beta=0.5, next=True),
        # the norm weights, gates and target taps of 36 layers: many small tensors
        dict(name="clip 144 small tensors", op="clip", layers=36, d=2560, f=0, vocab=0, g="f32", pad=8, tau=0.5,
             place=False),
        # two layers of the 4B class and the token table, clipped into a copy
        dict(name="clip 2 layers and table", op="clip", layers=2, d=2560, f=9728, vocab=151936, g="f32", pad=8,
             tau=0.5, place=False),
        # a step that stays under the threshold, in place: bf16 gradients that lie in one buffer without padding
        dict(name="clip in place, bf16, ragged", op="clip", layers=3, d=1021, f=4093, vocab=32003, g="bf16", pad=1,
             tau=2.0, place=True),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, its logarithm uniform."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def width(rng):
    """A model width: mostly a multiple of 64, now and then of 8, now and then any number."""
    d = spread(rng, 64, 8192)
    kind = rng.random()
    return max(64, d // 64 * 64) if kind < 0.6 else max(64, d // 8 * 8) if kind < 0.8 else d


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm_pre", "norm_post", "norm_pre_grad", "norm_post_grad", "clip"])
    d = width(rng)
    if op in ("embed", "embed_grad"):
        B = rng.randint(1, 8)
        T = spread(rng, 1, max(1, min(131072, 131072 * 2560 // d) // B))
        vocab = spread(rng, 256, min(151936, 151936 * 2560 // d))
        if op == "embed":
            return dict(op=op, B=B, T=T, vocab=vocab, d=d, table=rng.choice(["bf16", "f32"]),
                        x=rng.choice(["bf16", "f32"]))
        return dict(op=op, B=B, T=T, vocab=vocab, d=d, dx=rng.choice(["bf16", "f32"]), dE=rng.choice(["bf16", "f32"]))
    if op.startswith("norm"):
        rows = spread(rng, 1, 32768 * 2560 // d)
        h, y, x = rng.choice([("f32", "f32", "f32"), ("f32", "bf16", "bf16"), ("f32", "f32", "bf16"),
                              ("bf16", "bf16", "bf16")])
        w = "f32" if x == "f32" else rng.choice(["f32", "bf16"])
        case = dict(op=op, rows=rows, d=d, h=h, x=x, w=w)
        if "post" in op:
            case.update(y=y, gate=rng.choice(["none", "channel", "token"]), alpha=rng.choice([1.0, 0.75]),
                        beta=rng.choice([1.0, 0.25]), next=rng.random() < 0.75)
        return case
    d = min(d, 2560)
    case = dict(op=op, layers=rng.randint(1, 14), d=d, f=rng.choice([0, spread(rng, d, 9728)]),
                vocab=rng.choice([0, spread(rng, 256, 32768)]), g=rng.choice(["f32", "bf16"]),
                pad=rng.choice([1, 8]), place=rng.random() < 0.3)
    while weights(case) > 500_000_000:
        case["layers"] -= 1
    # in place a clipped pass would leave nothing to clip for the next one, so there the norm stays under tau
    case["tau"] = 2.0 if case["place"] else rng.choice([0.5, 2.0])
    return case


STD = 1e-3  # of the gradients


def shapes(case):
    """The parameters' gradients: per layer two norm weights, a gate, five target taps and, with f, the three matrices;
    with vocab, the token table."""
    d, f, v = case["d"], case["f"], case["vocab"]
    layer = [(d,), (d,), (d,), (5, d)] + ([(f, d), (f, d), (d, f)] if f else [])
    return layer * case["layers"] + ([(v, d)] if v else [])


def weights(case):
    return sum(math.prod(s) for s in shapes(case))


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(DT[dtype])

    op, d = case["op"], case["d"]
    s = dict(case)
    if op in ("embed", "embed_grad"):
        B, T, vocab = case["B"], case["T"], case["vocab"]
        # token frequencies fall as 1 / rank; a document end now and then (-1), and one look-ahead id per sequence
        u = torch.rand((B, T + 1), generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(vocab)) - 1).long().clamp_(0, vocab - 1)
        ids[torch.rand((B, T + 1), generator=g, device="cuda") < 1 / 2048] = -1
        s["ids"] = ids.int()[:, :T]
        s["scale"] = math.sqrt(d)
        if op == "embed":
            s["E"] = normal((vocab, d), case["table"], 0.02)
        else:
            s["grad"] = normal((B, T, d), case["dx"], 1e-3)
        return s
    if op.startswith("norm"):
        n = case["rows"]
        s["w"] = normal((d,), case["w"], 0.1, 1.0)
        if "post" in op:
            s["branch"] = normal((n, d), case["y"], 0.5)
            s["a"] = (None if case["gate"] == "none" else normal((d,), case["w"], 0.1, 0.5)
                      if case["gate"] == "channel" else torch.sigmoid(normal((n, d), "f32")).to(DT[case["y"]]))
            s["w_next"] = normal((d,), case["w"], 0.1, 1.0) if case["next"] else None
        s["hid"] = normal((n, d), case["h"], 2.0)  # the residual stream: h, or o where gradients are taken
        if op.endswith("grad"):
            s["dh"] = normal((n, d), case["h"], 1e-3)
            s["dx"] = normal((n, d), case["x"], 1e-3) if case.get("next", True) else None
        return s
    # gradients as a training program holds them: views of one flat buffer
    at, spans = 0, []
    for sh in shapes(case):
        spans.append((at, sh))
        at += -(-math.prod(sh) // case["pad"]) * case["pad"]
    flat = normal((at,), case["g"], STD)
    s["flat"] = flat
    s["grads"] = [flat[i:i + math.prod(sh)].view(sh) for i, sh in spans]
    s["tau"] = case["tau"] * STD * math.sqrt(weights(case))  # in the case it is a share of the norm to be expected
    s["flat_out"] = flat if case["place"] else torch.zeros_like(flat)
    s["out"] = None if case["place"] else [s["flat_out"][i:i + math.prod(sh)].view(sh) for i, sh in spans]
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import chunk_wise_weight_amd as ttt

    op = s["op"]
    if op == "embed":
        return ttt.ttt_embed(s["E"], s["ids"], scale=s["scale"], dtype=DT[s["x"]])
    if op == "embed_grad":
        return ttt.ttt_embed_grad(s["grad"], s["ids"], s["vocab"], scale=s["scale"], dtype=DT[s["dE"]])
    if op == "norm_pre":
        return ttt.ttt_norm_pre(s["hid"], s["w"], eps=EPS, dtype=DT[s["x"]])
    if op == "norm_pre_grad":
        dh, dw = ttt.ttt_norm_pre_grad(s["dx"], s["hid"], s["w"], eps=EPS, dh_in=s["dh"])
        return {"dh": dh, "dw": dw}
    if op == "norm_post":
        o, x = ttt.ttt_norm_post(s["hid"], s["branch"], s["w"], gate=s["a"], alpha=s["alpha"], beta=s["beta"], eps=EPS,
                                 w_next=s["w_next"], next_norm=s["next"], dtype=DT[s["x"]])
        return {"o": o, "x": x} if s["next"] else {"o": o}
    if op == "norm_post_grad":
        got = ttt.ttt_norm_post_grad(s["dh"], s["dx"], s["hid"], s["branch"], s["w"], gate=s["a"], alpha=s["alpha"],
                                     beta=s["beta"], eps=EPS, w_next=s["w_next"])
        return {k: v for k, v in got._asdict().items() if v is not None}
    return {"norm": ttt.ttt_clip_grads(s["grads"], s["tau"], out=s["out"]), "out": s["flat_out"]}


def rms(h):
    return torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)


def norm_back(g, n, r):
    """The gradient of h for n = h r(h), given g, the gradient of n."""
    return r * (g - n * (g * n).mean(-1, keepdim=True))


def run_plain(s):
    op = s["op"]
    if op == "embed":
        known = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
        x = s["E"][s["ids"].clamp(0, s["vocab"] - 1)].float() * s["scale"]
        return (x * known[..., None]).to(DT[s["x"]])
    if op == "embed_grad":
        ids = s["ids"].reshape(-1)
        known = (ids >= 0) & (ids < s["vocab"])
        dx = s["grad"].reshape(-1, s["d"]).float() * s["scale"]
        dE = torch.zeros((s["vocab"], s["d"]), device=dx.device)
        return dE.index_add_(0, ids.clamp(0, s["vocab"] - 1), dx * known[:, None]).to(DT[s["dE"]])
    if op == "norm_pre":
        h = s["hid"].float()
        return (h * rms(h) * s["w"].float()).to(DT[s["x"]])
    if op == "norm_pre_grad":
        h, dx = s["hid"].float(), s["dx"].float()
        r = rms(h)
        n = h * r
        dh = s["dh"].float() + norm_back(dx * s["w"].float(), n, r)
        return {"dh": dh.to(DT[s["h"]]), "dw": (dx * n).sum(0)}
    if op == "norm_post":
        h, y, w = s["hid"].float(), s["branch"].float(), s["w"].float()
        b = y * rms(y) * w
        o = s["alpha"] * h + s["beta"] * (b if s["a"] is None else b * s["a"].float())
        out = {"o": o.to(DT[s["h"]])}
        if s["next"]:
            out["x"] = (o * rms(o) * s["w_next"].float()).to(DT[s["x"]])
        return out
    if op == "norm_post_grad":
        o, y, w, do = s["hid"].float(), s["branch"].float(), s["w"].float(), s["dh"].float()
        out = {}
        if s["next"]:
            r = rms(o)
            n, dx = o * r, s["dx"].float()
            do = do + norm_back(dx * s["w_next"].float(), n, r)
            out["dw_next"] = (dx * n).sum(0)
        r = rms(y)
        n, t = y * r, s["beta"] * do
        a = None if s["a"] is None else s["a"].float()
        if a is not None:
            da = t * w * n
            out["dgate"] = da.sum(0) if s["gate"] == "channel" else da.to(s["branch"].dtype)
            t = t * a
        out["dw"] = (t * n).sum(0)
        out["dy"] = norm_back(t * w, n, r).to(s["branch"].dtype)
        out["dh"] = (s["alpha"] * do).to(DT[s["h"]])
        return out
    total = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt().reshape(1)
    c = torch.where(total > s["tau"], s["tau"] / total, 1.0)
    for g, o in zip(s["grads"], s["out"] or s["grads"]):
        o.copy_(g.float() * c)
    return {"norm": total, "out": s["flat_out"]}


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    """From the definitions; gradients by differentiation."""
    s = prepare(case, seed)
    op, d = s["op"], s["d"]

    def leaf(t):
        return None if t is None else t.double().requires_grad_()

    def normed(h, w):
        return w * h / torch.sqrt(torch.mean(h ** 2, dim=-1, keepdim=True) + EPS)

    if op in ("embed", "embed_grad"):
        # an extra last row, zero, takes the ids outside the table
        at = torch.where((s["ids"] < 0) | (s["ids"] >= s["vocab"]), s["vocab"], s["ids"]).long()
        if op == "embed":
            return torch.cat([s["E"].double(), torch.zeros((1, d), device="cuda", dtype=torch.float64)])[at] * s["scale"]
        E = torch.zeros((s["vocab"] + 1, d), device="cuda", dtype=torch.float64, requires_grad=True)
        return torch.autograd.grad((E[at] * s["scale"] * s["grad"].double()).sum(), E)[0][:-1]
    if op in ("norm_pre", "norm_pre_grad"):
        h, w = leaf(s["hid"]), leaf(s["w"])
        x = normed(h, w)
        if op == "norm_pre":
            return x.detach()
        dh, dw = torch.autograd.grad((x * s["dx"].double()).sum() + (h * s["dh"].double()).sum(), [h, w])
        return {"dh": dh, "dw": dw}
    if op in ("norm_post", "norm_post_grad"):
        y, w, a, wn = leaf(s["branch"]), leaf(s["w"]), leaf(s["a"]), leaf(s["w_next"])
        branch = normed(y, w) * (1.0 if a is None else a)
        if op == "norm_post":
            o = (s["alpha"] * s["hid"].double() + s["beta"] * branch).detach()
            return {"o": o, "x": normed(o, wn).detach()} if s["next"] else {"o": o}
        # h is whatever gives the stored o; its gradient does not depend on it
        o = s["hid"].double()
        h = ((o - s["beta"] * branch.detach()) / s["alpha"]).requires_grad_()
        o = s["alpha"] * h + s["beta"] * branch
        loss = (o * s["dh"].double()).sum()
        if s["next"]:
            loss = loss + (normed(o, wn) * s["dx"].double()).sum()
        names = {"dw_next": wn, "dgate": a, "dw": w, "dy": y, "dh": h}
        names = {k: v for k, v in names.items() if v is not None}
        return dict(zip(names, torch.autograd.grad(loss, list(names.values()))))
    total = torch.linalg.vector_norm(torch.cat([g.reshape(-1) for g in s["grads"]]), dtype=torch.float64).reshape(1)
    scaled = s["flat"].double() * torch.clamp(s["tau"] / total, max=1.0)
    return {"norm": total, "out": scaled if case["place"] else scaled * marked(s["flat"], s["grads"])}


def marked(flat, parts):
    """1 where flat belongs to one of its views, 0 in the padding between them."""
    m = torch.zeros_like(flat, dtype=torch.float64)
    for p in parts:
        at = p.storage_offset()
        m[at:at + p.numel()] = 1.0
    return m


# ---------------------------------------------------------------- what a pass cannot do without


def distinct(tokens, vocab):
    """Expected number of different ids among that many tokens."""
    k = torch.arange(1, vocab + 1, dtype=torch.float64)
    p = torch.log1p(1 / k) / math.log(vocab)
    p[-1] = 0
    return float((1 - torch.pow(1 - p, tokens)).sum())


def work(case):
    op, d = case["op"], case["d"]
    if op in ("embed", "embed_grad"):
        n = case["B"] * case["T"]
        if op == "embed":
            return {"bytes": n * (4 + d * size(case["x"])) + distinct(n, case["vocab"]) * d * size(case["table"]),
                    "flops": n * d}
        return {"bytes": n * (4 + d * size(case["dx"])) + case["vocab"] * d * size(case["dE"]), "flops": 2 * n * d}
    if op.startswith("norm"):
        e, h, x = case["rows"] * d, size(case["h"]), size(case["x"])
        if op == "norm_pre":
            return {"bytes": e * (h + x) + d * size(case["w"]), "flops": 4 * e}
        if op == "norm_pre_grad":
            return {"bytes": e * (3 * h + x) + d * (size(case["w"]) + 4), "flops": 12 * e}
        y, a = size(case["y"]), size(case["y"]) if case["gate"] == "token" else 0
        nx = x if case["next"] else 0
        if op == "norm_post":
            return {"bytes": e * (2 * h + y + a + nx) + 3 * d * size(case["w"]), "flops": 10 * e}
        return {"bytes": e * (3 * h + 2 * y + 2 * a + nx) + 3 * d * (size(case["w"]) + 4), "flops": 30 * e}
    n = weights(case)
    # gradients that are not scaled stay where they are; a copy reads each once and writes it once
    return {"bytes": (1 if case["place"] else 2) * n * size(case["g"]), "flops": (2 if case["place"] else 3) * n}
