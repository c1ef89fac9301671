"""The many-tensor operators of the library that a first-order training step uses, with cases to measure
them on: the clipping of a gradient list to a global norm (GradClip), and the AdamW step with its two
moments in float32 or in 8 bits (AdamW).

A case's tensors come from one of the workloads' parameter sets (a 64 x 32 weight, ResNet-50's 161 weights, a
Transformer layer at 1024 / 4096, the Transformer-Big set of 285M parameters) or are drawn over a
logarithmic range of sizes.  The definitions:

  norm   = sqrt(sum of g^2 over the parameters whose gradient is finite); a parameter whose gradient
           holds a NaN or an infinity is skipped: its weights, moments, step count and gradient stay
  c      = max_norm / norm where norm > max_norm, else 1;  g <- c g
  t      <- t + 1 (per parameter)
  m      <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2
  w      <- w (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
  copy   <- bfloat16(w), where the model computes on a bfloat16 copy of its weights

With 8-bit moments, m and r = sqrt(v) are kept as e4m3 codes over one power of two per 256 elements, the
smallest that brings the block's largest magnitude to 448 or less.  The rounding to a code is stochastic, from
16 bits of a counter-based hash of (seed, t, element) each, so that it needs no generator's state: m
rounds up with the probability of its fraction, r with the one that leaves the mean of r^2 = v.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 256           # elements per 8-bit scale; every tensor's moments start at a multiple of it
B1, B2, EPS, LR = 0.9, 0.999, 1e-8, 1e-3
DECAY = 0.01          # weight decay of the tensors with more than 4096 elements (the others: 0)
SEED = 0x5EED0BADF00D  # of the stochastic rounding
LARGEST = 285_212_672  # elements of the largest set


def listed():
    return [
        # the smallest step there is: one 64 x 32 weight, where the launches are all of the time
        dict(name="clip 64x32 f32", op="clip", set="single", grad="f32"),
        # ResNet-50's weights, batch-norm scales and biases: 161 tensors from 64 to 2.4M elements
        dict(name="clip resnet50 f32", op="clip", set="resnet50", grad="f32"),
        # the largest set, with the gradients that a bfloat16 backward pass leaves
        dict(name="clip big bf16", op="clip", set="big", grad="bf16"),
        dict(name="adamw 64x32 f32", op="adamw", set="single", grad="f32", clip=False, copy=False),
        # one Transformer layer, bfloat16 gradients, clipped, and the bfloat16 weights for the next forward pass
        dict(name="adamw layer bf16 copy", op="adamw", set="layer", grad="bf16", clip=True, copy=True),
        dict(name="adamw resnet50 f32", op="adamw", set="resnet50", grad="f32", clip=True, copy=False),
        # the largest set in full precision, no clipping
        dict(name="adamw big f32", op="adamw", set="big", grad="f32", clip=False, copy=False),
        dict(name="adamw8 64x32 f32", op="adamw8", set="single", grad="f32", clip=False, copy=False),
        dict(name="adamw8 layer bf16 copy", op="adamw8", set="layer", grad="bf16", clip=True, copy=True),
        # tensors of odd sizes in one buffer without gaps, so that hardly one starts on a 16-byte boundary, and
        # one of them with a NaN in its gradient
        dict(name="adamw8 odd packed f32", op="adamw8", set="log", tensors=57, total=9_876_543, shapes=3, grad="f32",
             clip=True, copy=False, packed=True, nan=True),
        dict(name="adamw8 resnet50 f32", op="adamw8", set="resnet50", grad="f32", clip=True, copy=False),
        # the largest set with 8-bit moments, as it is trained where memory is short
        dict(name="adamw8 big bf16 copy", op="adamw8", set="big", grad="bf16", clip=True, copy=True),
    ]


def draw(rng):
    case = dict(op=rng.choice(["clip", "adamw", "adamw8"]), set="log", shapes=rng.randrange(1 << 30),
                grad=rng.choice(["f32", "bf16"]), packed=rng.random() < 0.3, nan=rng.random() < 0.2)
    case["tensors"] = int(math.exp(rng.uniform(0.0, math.log(300))))
    # packed tensors need an index of eight bytes an element in the plain form: fewer of them
    most = 40_000_000 if case["packed"] else LARGEST // 2
    case["total"] = int(math.exp(rng.uniform(math.log(4 * case["tensors"] + 1), math.log(most))))
    if case["op"] != "clip":
        case["clip"] = rng.random() < 0.6
        case["copy"] = rng.random() < 0.4
    return case


def sizes(case):
    """The tensors' element counts."""
    if case["set"] == "single":
        return [64 * 32]
    if case["set"] == "layer":
        return [1024 * 1024] * 4 + [1024 * 4096] * 2 + [1024] * 2
    if case["set"] == "big":
        return ([1024 * 1024] * 4 + [1024 * 8192] * 2) * 12 + [32768 * 1024]
    if case["set"] == "resnet50":
        mats, vecs, cin = [147 * 64], [64, 64], 64
        for w, blocks in ((64, 3), (128, 4), (256, 6), (512, 3)):
            for i in range(blocks):
                for rows, cols in [(cin, w), (9 * w, w), (w, 4 * w)] + ([(cin, 4 * w)] if i == 0 else []):
                    mats.append(rows * cols)
                    vecs += [cols, cols]
                cin = 4 * w
        return mats + [2048 * 1000] + vecs + [1000]
    rng = random.Random(case["shapes"])
    part = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(case["tensors"])]
    return [max(1, int(case["total"] * p / sum(part))) for p in part]


def layout(case):
    """(sizes, where each tensor's moments start, elements with the gaps)."""
    n = sizes(case)
    at, end = [], 0
    for k in n:
        at.append(end)
        end += -(-k // BLOCK) * BLOCK
    return n, at, end


def work(case):
    n = sum(sizes(case))
    g = 2 if case["grad"] == "bf16" else 4
    if case["op"] == "clip":
        return {"bytes": 2 * g * n, "flops": 3 * n}
    moments = 16 if case["op"] == "adamw" else 4 + 4 / BLOCK
    return {"bytes": (8 + g + moments + (2 if case["copy"] else 0)) * n, "flops": (16 if case["op"] == "adamw" else 40) * n}


def prepare(case, seed):
    n, at, total = layout(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    owner = torch.from_numpy(np.repeat(np.arange(len(n)), [-(-k // BLOCK) for k in n])).to(dev)
    used = torch.zeros(total, dtype=torch.bool, device=dev)
    for k, o in zip(n, at):
        used[o:o + k] = True
    # gradients of very different scales from tensor to tensor, as from layer to layer, and a tenth of the
    # blocks without any (rows of an embedding that the batch does not touch)
    std = torch.exp(torch.empty(len(n), device=dev).uniform_(math.log(1e-5), math.log(1e-2), generator=gen))
    std = std[owner] * ((torch.rand(len(owner), device=dev, generator=gen) > 0.1) | (len(owner) < 8))
    g = torch.randn(total, device=dev, generator=gen).view(-1, BLOCK).mul_(std[:, None]).view(-1).mul_(used)
    w = torch.randn(total, device=dev, generator=gen).mul_(0.02).mul_(used)
    gtype = torch.bfloat16 if case["grad"] == "bf16" else torch.float32
    norm = math.sqrt(float(g.to(gtype).double().square().sum()))
    if case.get("nan"):
        g[at[len(n) // 2] + n[len(n) // 2] - 1] = math.nan
    s = {"case": case, "n": n, "at": at, "total": total, "owner": owner, "passes": 0,
         "packed": bool(case.get("packed")), "max_norm": 0.4 * norm if case.get("clip", True) else 0.0}
    start = at
    if s["packed"]:   # without gaps, from the second element of a buffer on
        start = [1 + sum(n[:i]) for i in range(len(n))]
        s["place"] = used.nonzero().view(-1)
        lead = torch.zeros(1, device=dev)
        g, w = torch.cat([lead, g[used]]), torch.cat([lead, w[used]])
    s["g"], s["w"] = g.to(gtype), w
    s["copy"] = w.to(torch.bfloat16) if case.get("copy") else None
    s["grads"] = [s["g"][o:o + k] for o, k in zip(start, n)]
    s["params"] = [s["w"][o:o + k] for o, k in zip(start, n)]
    s["copies"] = [s["copy"][o:o + k] for o, k in zip(start, n)] if case.get("copy") else None
    if case["op"] == "clip":
        if own:
            from shampoo_second_order_b200 import GradClip
            s["clip"] = GradClip([(k,) for k in n], grad_dtype=case["grad"])
        return s
    # moments as some hundred steps leave them
    s["decay"] = [DECAY if k > 4096 else 0.0 for k in n]
    live = std[:, None].clamp(min=1e-7)
    m = (torch.randn(total, device=dev, generator=gen).view(-1, BLOCK) * (0.3 * live)).view(-1).mul_(used)
    v = (torch.rand(total, device=dev, generator=gen).add_(0.5).view(-1, BLOCK) * live.square()).view(-1).mul_(used)
    step = torch.randint(100, 1000, (len(n),), device=dev, generator=gen, dtype=torch.int32)
    if case["op"] == "adamw":
        state = {"m": m, "v": v, "step": step}
    else:
        state = {"step": step}
        for name, x in (("m", m), ("r", v.sqrt_())):
            e = scale_exponent(x.view(-1, BLOCK).abs().amax(1))
            state[name] = torch.ldexp(x.view(-1, BLOCK), -e[:, None]).view(-1).to(torch.float8_e4m3fn)
            state[name + "_scale"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    if own:
        from shampoo_second_order_b200 import AdamW
        opt = AdamW([(k,) for k in n], beta1=B1, beta2=B2, eps=EPS, weight_decay=s["decay"],
                    state="f32" if case["op"] == "adamw" else "8bit", grad_dtype=case["grad"],
                    max_norm=s["max_norm"], seed=SEED)
        for name, x in opt.state_tensors().items():
            raw(x).copy_(raw(state[name]))
        s["opt"] = opt
    else:
        s["state"] = state
    return s


def raw(x):
    """A tensor of 8-bit floats as its bytes, any other one as it is."""
    return x.view(torch.uint8) if x.element_size() == 1 else x


def run(s):
    if s["case"]["op"] == "clip":
        # a user's gradients are new at every step; here the bound falls a little from pass to pass, so that
        # every pass has to scale
        bound = s["max_norm"] * 0.999 ** s["passes"]
        s["passes"] += 1
        if own:
            return {"g": s["g"], "norm": s["clip"].clip(s["grads"], bound)}
        return plain_clip(s, bound)
    if own:
        s["opt"].step(s["params"], s["grads"], LR, copies=s["copies"])
        out = dict(s["opt"].state_tensors(), w=s["w"], norm=s["opt"].grad_norm())
    else:
        out = plain_adamw(s)
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def spread(s, x):
    """A list's buffer in float32 with every tensor at its place, as rows of BLOCK elements."""
    x = x.float()
    if s["packed"]:
        x = torch.zeros(s["total"], device=x.device).index_copy_(0, s["place"], x[1:])
    return x.view(-1, BLOCK)


def put(s, buffer, x):
    """Writes rows of BLOCK elements back into the list's buffer, rounded to its type."""
    if s["packed"]:
        buffer[1:] = x.reshape(-1)[s["place"]].to(buffer.dtype)
    else:
        buffer.copy_(x.view(-1))


def finite_norm(s, g, bound):
    """(per tensor: is its gradient finite, the norm over those, the factor that brings it to the bound)."""
    bad = (~torch.isfinite(g)).any(1)
    skip = torch.zeros(len(s["n"]), dtype=torch.int32, device=g.device)
    keep = skip.scatter_reduce(0, s["owner"], bad.int(), "amax") == 0
    squares = g.square().sum(1).double()   # 256 terms in 32 bits, the many blocks in 64
    norm = torch.where(keep[s["owner"]], squares, 0.0).sum().sqrt()
    factor = torch.where(norm > bound, bound / norm, 1.0) if bound > 0 else torch.ones_like(norm)
    return keep, norm.float(), factor.float()


def plain_clip(s, bound):
    g = spread(s, s["g"])
    keep, norm, factor = finite_norm(s, g, bound)
    put(s, s["g"], torch.where(keep[s["owner"]][:, None], g * factor, g))
    return {"g": s["g"], "norm": norm}


def hash32(x):
    """Two multiply-xorshift rounds on the low 32 bits (held in 64: the products wrap without harm)."""
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(seed, step, total):
    """32 bits for every element: step holds the step number of each block of elements."""
    key = (seed & 0xFFFFFFFF) + hash32(torch.tensor(seed >> 32, device=step.device)) + step.long() * 0x632BE5AB
    key = hash32(key & 0xFFFFFFFF)[:, None]
    j = torch.arange(total, device=step.device).view(-1, BLOCK)
    return hash32(((j & 0xFFFFFFFF) * 0x9E3779B1 + (j >> 32) * 0x85EBCA77 + key) & 0xFFFFFFFF)


def scale_exponent(largest):
    """The smallest e with largest <= 448 * 2^e, and at least -126."""
    bits = largest.view(torch.int32)
    return (((bits + 0x1FFFFF) >> 23) - 8).clamp(min=1) - 127


def to_codes(x, bits, square):
    """(e4m3 codes, exponent of each block's scale) of x, rounded with 16 random bits an element."""
    e = scale_exponent(x.abs().amax(1))
    a = torch.ldexp(x.abs(), -e[:, None])
    # below 2^-6 the steps of e4m3 are 2^-9 throughout, as they are from 2^-6 to 2^-5: lift a into that range
    lift = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)
    word = (a + lift).view(torch.int32)
    if square:
        low = (word & -0x100000).view(torch.float32) - lift
        step = (word & 0x7F800000).view(torch.float32) * 0.125
        up = (a - low) * (a + low) > bits.float() * 2.0 ** -16 * (step * (2.0 * low + step))
        y = torch.where(up, low + step, low)
    else:
        y = ((word + (bits.int() << 4)) & -0x100000).view(torch.float32) - lift
    return torch.copysign(y, x).to(torch.float8_e4m3fn).view(-1), e


def plain_adamw(s):
    state, eight = s["state"], s["case"]["op"] == "adamw8"
    g, w = spread(s, s["g"]), spread(s, s["w"])
    keep, norm, factor = finite_norm(s, g, s["max_norm"])
    g = g * factor
    step = state["step"] + keep.int()
    at = s["owner"]
    # the decay of the moments to the t-th power in 64 bits: 1 - b^t loses digits where t is small
    first = (LR / (1.0 - B1 ** step.double())).float()[at][:, None]
    second = (1.0 / (1.0 - B2 ** step.double()).sqrt()).float()[at][:, None]
    shrink = (1.0 - LR * torch.tensor(s["decay"], dtype=torch.float64, device=g.device)).float()[at][:, None]
    if eight:
        m = state["m"].float().view(-1, BLOCK) * state["m_scale"].float()[:, None]
        v = (state["r"].float().view(-1, BLOCK) * state["r_scale"].float()[:, None]).square()
    else:
        m, v = state["m"].view(-1, BLOCK), state["v"].view(-1, BLOCK)
    m = B1 * m + (1.0 - B1) * g
    v = (B2 * v + (1.0 - B2) * g * g).clamp(max=torch.finfo(torch.float32).max)
    r = v.sqrt()
    new = w * shrink - first * (m / (r * second + EPS))
    rows = keep[at]
    new = torch.where(rows[:, None], new, w)
    put(s, s["w"], new)
    if s["copy"] is not None:
        put(s, s["copy"], torch.where(rows[:, None], new, spread(s, s["copy"])))
    if eight:
        bits = random_bits(SEED, step[at], s["total"])
        for name, x, b in (("m", m, bits & 0xFFFF), ("r", r, bits >> 16)):
            codes, e = to_codes(x, b, name == "r")
            codes, old = codes.view(torch.uint8).view(-1, BLOCK), raw(state[name])
            old.copy_(torch.where(rows[:, None], codes, old.view(-1, BLOCK)).view(-1))
            scale = raw(state[name + "_scale"])
            scale.copy_(torch.where(rows, (e + 127).to(torch.uint8), scale))
    else:
        for name, x in (("m", m), ("v", v)):
            state[name].view(-1, BLOCK).copy_(torch.where(rows[:, None], x, state[name].view(-1, BLOCK)))
    state["step"].copy_(step)
    return dict(state, w=s["w"], norm=norm)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits, tensor by tensor
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    grads = [x.double() for x in s["grads"]]
    fine = [bool(torch.isfinite(x).all()) for x in grads]
    norm = math.sqrt(sum(float(x.square().sum()) for x, ok in zip(grads, fine) if ok))
    c = s["max_norm"] / norm if 0 < s["max_norm"] < norm else 1.0
    if case["op"] == "clip":
        out = s["g"].double()
        for x, to, ok in zip(grads, views(s, out), fine):
            to.copy_(x * c if ok else x)
        return {"g": out, "norm": torch.tensor(norm, dtype=torch.float64)}
    state = {k: x.clone() if k == "step" else x.double() for k, x in s["state"].items()}
    out = dict(state, w=s["w"].double(), norm=torch.tensor(norm, dtype=torch.float64))
    weights = views(s, out["w"])
    if case["copy"]:
        out["copy"] = s["copy"].double()
        copies = views(s, out["copy"])
    for i, (k, o) in enumerate(zip(s["n"], s["at"])):
        if not fine[i]:
            continue
        out["step"][i] += 1
        t = int(out["step"][i])
        g = grads[i] * c
        b0, b1 = o // BLOCK, -(-(o + k) // BLOCK)
        if case["op"] == "adamw":
            m, v = out["m"][o:o + k], out["v"][o:o + k]
        else:
            m = (out["m"][b0 * BLOCK:b1 * BLOCK].view(-1, BLOCK) * out["m_scale"][b0:b1, None]).view(-1)[:k]
            v = (out["r"][b0 * BLOCK:b1 * BLOCK].view(-1, BLOCK) * out["r_scale"][b0:b1, None]).view(-1)[:k] ** 2
        m = m + (1 - B1) * (g - m)
        v = v + (1 - B2) * (g * g - v)
        weights[i].mul_(1 - LR * s["decay"][i]).sub_(
            LR / (1 - B1 ** t) * m / (v.sqrt() / math.sqrt(1 - B2 ** t) + EPS))
        if case["copy"]:
            copies[i].copy_(weights[i])
        if case["op"] == "adamw":
            out["m"][o:o + k], out["v"][o:o + k] = m, v
            continue
        lot = lots(SEED, t, o, (b1 - b0) * BLOCK)
        for name, x, u in (("m", m, lot & 0xFFFF), ("r", v.sqrt(), lot >> 16)):
            full = torch.zeros((b1 - b0) * BLOCK, dtype=torch.float64, device=x.device)
            full[:k] = x
            code, scale = rounded(full.view(-1, BLOCK), u.view(-1, BLOCK), name == "r")
            out[name][b0 * BLOCK:b1 * BLOCK] = code.view(-1)
            out[name + "_scale"][b0:b1] = scale
    return out


def views(s, x):
    """Each tensor's part of a list's buffer."""
    got, end = [], 1
    for k, o in zip(s["n"], s["at"]):
        got.append(x[end:end + k] if s["packed"] else x[o:o + k])
        end += k
    return got


def mixed(x):
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = ((x ^ (x >> shift)) * factor) % (1 << 32)
    return x ^ (x >> 16)


def lots(seed, t, start, count):
    """The 32 random bits of `count` elements from element `start` on, at step t."""
    key = mixed((seed % (1 << 32) + mixed(seed >> 32) + t * 0x632BE5AB) % (1 << 32))
    j = torch.arange(start, start + count, device="cuda")
    return mixed(((j % (1 << 32)) * 0x9E3779B1 + (j // (1 << 32)) * 0x85EBCA77 + key) % (1 << 32))


def rounded(x, u, square):
    """(values of the e4m3 codes, scale of each row) of rows x, by the probabilities of the definition."""
    top = x.abs().amax(1)
    e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0)   # -inf for an empty row
    scale = torch.exp2(e)
    a = x.abs() / scale[:, None]
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6.0) - 3.0)
    low = torch.floor(a / step) * step
    chance = u.double() / 65536.0
    if square:
        up = a ** 2 - low ** 2 > chance * ((low + step) ** 2 - low ** 2)
    else:
        up = (a - low) / step + chance >= 1.0
    return torch.copysign(low + step * up, x), scale
