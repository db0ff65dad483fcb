"""Workloads of the training operators: the AdamW step over many tensors (32- and
8-bit states, with the global gradient clip) and LayerNorm forward and backward.

``run`` is one pass through an operator: with ``own`` false its plain form in
elementary torch operations, with ``own`` true the framework's own call.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 256            # elements that share a scale in the 8-bit states
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.999, 1e-8, 0.01, 1e-4
SEED = 20240917        # key of the 8-bit states' stochastic rounding
LN_EPS = 1e-6
MASK = 0xFFFFFFFF


# ----------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------
def listed():
    return [
        # the shape-check model's expert: 27 small tensors, a step is launch latency; first step, zero states, clipped
        dict(name="adamw_tiny", op="adamw", layout="tiny", p="f32", g="f32", bits=32, copy=True, clip=1.0, step=1),
        # tensors of odd sizes at odd offsets (no vector access is aligned), bf16 weights without a master copy
        dict(name="adamw_ragged", op="adamw", layout="ragged", count=61, total=8_000_003, lseed=5, p="bf16", g="f32",
             bits=32, copy=False, clip=0.0, step=37),
        # the fine-tune of the 16-layer action expert: fp32 master weights, the bf16 copy the next step reads, clipped
        dict(name="adamw_expert", op="adamw", layout="expert", p="f32", g="f32", bits=32, copy=True, clip=1.0, step=1000),
        # the same with 8-bit states
        dict(name="adamw_expert_8bit", op="adamw", layout="expert", p="f32", g="f32", bits=8, copy=True, clip=1.0,
             step=1000),
        # the prefix language model unfrozen, bf16 weights and gradients, 8-bit states
        dict(name="adamw_prefix_8bit", op="adamw", layout="prefix", p="bf16", g="bf16", bits=8, copy=False, clip=0.0,
             step=1000),
        # one token of the prefix width: latency
        dict(name="ln_token", op="ln", M=1, D=960, x="f32", y="bf16", w="bf16", pad=0),
        # two camera images of one query (32 x 32 patches each) at the vision width
        dict(name="ln_images", op="ln", M=2048, D=768, x="bf16", y="bf16", w="bf16", pad=0),
        # a batch of 32 queries, fp32 residual stream in, bf16 operand out
        dict(name="ln_batch", op="ln", M=65536, D=768, x="f32", y="bf16", w="f32", pad=0),
        # the norm of one action chunk at the expert width
        dict(name="ln_bwd_chunk", op="ln_bwd", M=50, D=720, x="f32", y="bf16", w="bf16", pad=0),
        # an odd width with padded rows, fp32 throughout
        dict(name="ln_bwd_odd", op="ln_bwd", M=3001, D=1283, x="f32", y="f32", w="f32", pad=5),
        # eight queries' images in bf16
        dict(name="ln_bwd_images", op="ln_bwd", M=16384, D=768, x="bf16", y="bf16", w="bf16", pad=0),
        # a wide layer, many rows
        dict(name="ln_bwd_wide", op="ln_bwd", M=16384, D=4096, x="bf16", y="bf16", w="f32", pad=0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.4:
        count, total = log(1, 200), log(1000, 100_000_000)
        bits = rng.choice([8, 32])
        p = rng.choice(["f32", "bf16"])
        return dict(op="adamw", layout="ragged", count=count, total=max(total, count), lseed=rng.randrange(1 << 20), p=p,
                    g=rng.choice(["f32", "bf16"]), bits=bits, copy=p == "f32" and rng.random() < 0.5,
                    clip=rng.choice([0.0, 0.5, 1e4]), step=log(1, 100_000))
    D = log(1, 16384)
    M = log(1, min(131072, 60_000_000 // D))
    return dict(op=rng.choice(["ln", "ln_bwd"]), M=M, D=D, x=rng.choice(["f32", "bf16"]), y=rng.choice(["f32", "bf16"]),
                w=rng.choice(["f32", "bf16"]), pad=rng.choice([0, 0, 1, 8]))


def layer(width, heads, kv_heads, hd, ffn, kv_in):
    """(size, is a matrix) of one layer's tensors, in the order of the weight blob."""
    q, kv = heads * hd, kv_heads * hd
    return [(width, 0), (q * width, 1), (kv * kv_in, 1), (kv * kv_in, 1), (width * q, 1), (width, 0),
            (ffn * width, 1), (ffn * width, 1), (width * ffn, 1)]


def sizes_of(case):
    """(sizes, weight decay applies) of the case's tensors."""
    kind = case["layout"]
    if kind == "prefix":
        both = [t for _ in range(16) for t in layer(960, 15, 5, 64, 2560, 960)]
    elif kind == "ragged":
        r = random.Random(case["lseed"])
        share = [math.exp(r.uniform(0.0, 7.0)) for _ in range(case["count"])]
        rest = case["total"] - case["count"]
        cut = [1 + int(rest * s / sum(share)) for s in share]
        cut[0] += case["total"] - sum(cut)
        both = [(n, r.randrange(2)) for n in cut]
    else:
        E, heads, kv_heads, hd, ffn, A, layers, cross = (
            (96, 4, 2, 32, 192, 8, 2, 64) if kind == "tiny" else (720, 15, 5, 64, 2048, 32, 16, 320))
        both = [t for n in range(layers) for t in layer(E, heads, kv_heads, hd, ffn, cross if n % 2 else E)]
        both += [(E, 0), (E * A, 1), (E, 0), (2 * E * E, 1), (E, 0), (E * E, 1), (E, 0), (A * E, 1), (A, 0)]
    return [n for n, _ in both], [bool(d) for _, d in both]


# ----------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if case["op"] == "adamw":
        sizes, decay = sizes_of(case)
        total = sum(sizes)
        st = dict(case=case, sizes=sizes, decay=decay, t=case["step"] - 1)
        st["p"] = normal(total).mul_(0.02).to(DTYPES[case["p"]])
        # gradients of tensors differ in size by orders of magnitude
        size = torch.tensor(sizes, device=DEV)
        spread = torch.repeat_interleave(normal(len(sizes)).mul_(1.5).exp_().mul_(1e-3), size)
        st["g"] = (normal(total) * spread).to(DTYPES[case["g"]])
        st["copy"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
        blocks = sum(-(-n // BLOCK) for n in sizes)
        first = case["step"] == 1
        m = normal(total) * spread * (0.0 if first else 0.25)
        v = (normal(total) * spread).square_() * (0.0 if first else 0.6)
        st["m_scale"] = st["v_scale"] = None
        if case["bits"] == 8:
            # codes as a run leaves them: a power of two a block, no subnormal codes
            at, _, _ = padded(sizes)
            for name, x, top, least, dt in (("m", m, 7, 2.0 ** -6, torch.float8_e4m3fn),
                                            ("v", v, 14, 2.0 ** -14, torch.float8_e5m2)):
                most = to_blocks(x.abs(), at, blocks).amax(1)
                scale = torch.where(most > 0, torch.ldexp(torch.ones_like(most), torch.frexp(most)[1] - 1 - top), 0.0)
                y = x / torch.repeat_interleave(scale, BLOCK)[at].clamp(min=1e-38)
                y = torch.where(y.abs() < least, torch.zeros_like(y), y)
                st[name], st[name + "_scale"] = y.to(dt), scale
        else:
            st["m"], st["v"] = m, v
        st["norm"] = torch.zeros(1, device=DEV)
        del m, v, spread
        if own:  # the optimiser that a training program keeps, over its tensors
            from vision_language_action_b200.runtime import AdamW

            def cut(x):
                return None if x is None else list(x.split(sizes))

            per = [-(-n // BLOCK) for n in sizes]
            scales = [None if st[k] is None else list(st[k].split(per)) for k in ("m_scale", "v_scale")]
            st["grads"] = cut(st["g"])
            st["opt"] = AdamW(cut(st["p"]), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, decay=decay,
                              state_bits=case["bits"], max_norm=case["clip"], copies=cut(st["copy"]), seed=SEED,
                              step=case["step"] - 1, state=(cut(st["m"]), cut(st["v"]), scales[0], scales[1]))
        return st

    M, D, pad = case["M"], case["D"], case["pad"]

    def rows(kind, scale=1.0, shift=0.0):
        x = torch.zeros(M, D + pad, dtype=DTYPES[kind], device=DEV)
        x[:, :D] = normal(M, D).mul_(scale) + shift
        return x[:, :D]

    # a residual stream: rows of different size, a mean of their own
    x = rows(case["x"], normal(M, 1).mul_(0.5).exp_(), normal(M, 1).mul_(0.2) + 0.3)
    st = dict(case=case, x=x, gamma=(1 + 0.2 * normal(D)).to(DTYPES[case["w"]]))
    if case["op"] == "ln":
        st["beta"] = normal(D).mul_(0.2).to(DTYPES[case["w"]])
        st["y"] = rows(case["y"])
        st["mean"], st["rstd"] = torch.zeros(M, device=DEV), torch.zeros(M, device=DEV)
    else:
        st["dy"] = rows(case["y"], 0.01)
        xd = x.double()
        st["mean"] = xd.mean(1).float()
        st["rstd"] = torch.rsqrt(xd.var(1, unbiased=False) + LN_EPS).float()
        st["dx"] = rows(case["x"])
        st["dgamma"], st["dbeta"] = torch.zeros(D, device=DEV), torch.zeros(D, device=DEV)
    return st


# ----------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        from vision_language_action_b200 import runtime

        if op == "adamw":
            st["opt"].step(st["grads"])
            if st["case"]["clip"]:
                st["norm"] = st["opt"].grad_norm
        elif op == "ln":
            runtime.op_layernorm(st["x"], st["gamma"], st["beta"], st["y"], LN_EPS, st["mean"], st["rstd"])
        else:
            runtime.op_layernorm_backward(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"], st["dx"],
                                          st["dgamma"], st["dbeta"])
    elif op == "adamw":
        adamw_plain(st)
    elif op == "ln":
        layernorm_plain(st)
    else:
        layernorm_backward_plain(st)
    if op == "adamw":
        keys = ["p", "m", "v"] + ["copy"] * st["case"]["copy"] + ["norm"] * bool(st["case"]["clip"])
        keys += ["m_scale", "v_scale"] * (st["case"]["bits"] == 8)
    else:
        keys = ["y", "mean", "rstd"] if op == "ln" else ["dx", "dgamma", "dbeta"]
    return {k: st[k] for k in keys}


def padded(sizes):
    """Place of each element when every tensor begins a new block of 256; each block's tensor and number in it."""
    size = torch.tensor(sizes, device=DEV)
    per = (size + BLOCK - 1) // BLOCK
    shift = (torch.cumsum(per, 0) - per) * BLOCK - (torch.cumsum(size, 0) - size)
    at = torch.arange(sum(sizes), device=DEV) + torch.repeat_interleave(shift, size)
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), per)
    number = torch.arange(tensor.numel(), device=DEV) - torch.repeat_interleave(torch.cumsum(per, 0) - per, per)
    return at, tensor, number


def to_blocks(x, at, blocks):
    out = torch.zeros(blocks * BLOCK, dtype=x.dtype, device=x.device)
    out[at] = x
    return out.view(blocks, BLOCK)


def random16(tensor, number, step):
    """16 random bits of every element of the blocks: Philox4x32-10, one draw for 8 elements."""
    octet = number[:, None] * (BLOCK // 8) + torch.arange(BLOCK // 8, device=DEV)
    c0, c1 = octet & MASK, octet >> 32
    c2, c3 = torch.full_like(c0, step & MASK), tensor[:, None].expand_as(c0)
    k0, k1 = SEED & MASK, SEED >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & MASK) ^ c1 ^ k0, b & MASK, ((a >> 32) & MASK) ^ c3 ^ k1, a & MASK
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    words = torch.stack((c0, c1, c2, c3), 2)
    return torch.stack((words & 0xFFFF, words >> 16), 3).view(number.numel(), BLOCK)


def to_8bit(x, at, blocks, rnd, mantissa, top, floor_at_least):
    """Codes and scales of x: magnitude bits of the fp32 value, rounded up where its dropped bits and the random ones carry."""
    bits = x.abs().view(torch.int32)
    most = to_blocks(bits, at, blocks).amax(1) >> 23
    low = torch.repeat_interleave(((most - top).clamp(min=0) << mantissa), BLOCK)[at]
    drop = 23 - mantissa
    code = ((bits + (rnd << (drop - 16))) >> drop) - low
    least = 1 << mantissa
    if floor_at_least:
        code = torch.where(bits > 0, code.clamp(min=least), 0)
    else:
        code = torch.where(code < least, 0, code)
    return torch.where((x < 0) & (code > 0), code + 128, code).to(torch.uint8), most


def adamw_plain(st):
    case = st["case"]
    st["t"] += 1
    t, size = st["t"], torch.tensor(st["sizes"], device=DEV)
    g = st["g"].float()
    if case["clip"]:
        norm = g.double().square().sum().sqrt()
        g = g * torch.clamp(case["clip"] / (norm + 1e-6), max=1.0).float()
        st["norm"].copy_(norm)
    m, v = st["m"].float(), st["v"].float()
    if case["bits"] == 8:
        at, tensor, number = padded(st["sizes"])
        blocks = tensor.numel()
        m = m * torch.repeat_interleave(st["m_scale"], BLOCK)[at]
        v = v * torch.repeat_interleave(st["v_scale"], BLOCK)[at]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    # divisions by a number are products with its reciprocal, made in 64 bits
    denom = v.sqrt() * (1 / math.sqrt(1 - BETA2 ** t)) + EPS
    keep = torch.repeat_interleave(torch.where(torch.tensor(st["decay"], device=DEV), 1 - LR * DECAY, 1.0), size)
    p = st["p"].float() * keep - (m / denom) * (LR / (1 - BETA1 ** t))
    st["p"].copy_(p)
    if case["copy"]:
        st["copy"].copy_(p)
    if case["bits"] == 8:
        rnd = random16(tensor, number, t).view(-1)[at].to(torch.int32)
        for name, x, mantissa, top, floor, dt in (("m", m, 3, 14, False, torch.float8_e4m3fn),
                                                  ("v", v, 2, 29, True, torch.float8_e5m2)):
            code, most = to_8bit(x, at, blocks, rnd, mantissa, top, floor)
            st[name].copy_(code.view(dt))
            # the scale that makes the codes' own exponents (bias 7 and 15) into the value's; 0 where all is 0
            bias = 7 if name == "m" else 15
            any_code = to_blocks(x.abs(), at, blocks).amax(1) > 0
            e = (most - top).clamp(min=0) - 127 + bias
            st[name + "_scale"].copy_(torch.where(any_code, torch.ldexp(torch.ones_like(e, dtype=torch.float32), e), 0.0))
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)


def layernorm_plain(st):
    x = st["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt(c.square().mean(1, keepdim=True) + LN_EPS)
    st["y"].copy_(c * rstd * st["gamma"].float() + st["beta"].float())
    st["mean"].copy_(mean[:, 0])
    st["rstd"].copy_(rstd[:, 0])


def layernorm_backward_plain(st):
    dy, r = st["dy"].float(), st["rstd"][:, None]
    xh = (st["x"].float() - st["mean"][:, None]) * r
    w = dy * st["gamma"].float()
    st["dx"].copy_(r * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True)))
    st["dgamma"].copy_((dy * xh).sum(0))
    st["dbeta"].copy_(dy.sum(0))


# ----------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------
def work(case):
    if case["op"] == "adamw":
        n = float(sum(sizes_of(case)[0]))
        wide = {"f32": 4, "bf16": 2}
        each = 2 * wide[case["p"]] + wide[case["g"]] + 2 * case["copy"] + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        return {"bytes": n * each, "flops": n * (14 + 2 * bool(case["clip"]))}
    M, D = float(case["M"]), float(case["D"])
    wide = {"f32": 4, "bf16": 2}
    if case["op"] == "ln":
        return {"bytes": M * D * (wide[case["x"]] + wide[case["y"]]) + 8 * M + 2 * D * wide[case["w"]], "flops": 8 * M * D}
    return {"bytes": M * D * (2 * wide[case["x"]] + wide[case["y"]]) + 8 * M + D * (wide[case["w"]] + 8),
            "flops": 15 * M * D}


# ----------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ----------------------------------------------------------------------
def exact(case, seed):
    keep, globals()["own"] = own, False
    try:
        st = prepare(case, seed)
    finally:
        globals()["own"] = keep
    if case["op"] == "ln":
        x = st["x"].double()
        mean = x.sum(1) / case["D"]
        var = ((x - mean[:, None]) ** 2).sum(1) / case["D"]
        rstd = 1 / torch.sqrt(var + LN_EPS)
        y = torch.addcmul(st["beta"].double(), (x - mean[:, None]) * rstd[:, None], st["gamma"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "ln_bwd":
        D, r = case["D"], st["rstd"].double()[:, None]
        dy, z = st["dy"].double(), (st["x"].double() - st["mean"].double()[:, None]) * r
        dz = dy * st["gamma"].double()
        dx = (D * dz - dz.sum(1, True) - z * (dz * z).sum(1, True)) * (r / D)
        return {"dx": dx, "dgamma": torch.einsum("md,md->d", dy, z), "dbeta": dy.sum(0)}
    # AdamW, tensor by tensor
    t = case["step"]
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in st["g"].split(st["sizes"])))
    c = min(1.0, case["clip"] / (norm + 1e-6)) if case["clip"] else 1.0
    out = {k: [] for k in ("p", "m", "v")}
    at = sat = 0
    for n, (size, dec) in enumerate(zip(st["sizes"], st["decay"])):
        cut, blocks = slice(at, at + size), -(-size // BLOCK)
        scut = slice(sat, sat + blocks)
        at, sat = at + size, sat + blocks
        m, v = st["m"][cut].double(), st["v"][cut].double()
        if case["bits"] == 8:
            m = m * st["m_scale"][scut].double().repeat_interleave(BLOCK)[:size]
            v = v * st["v_scale"][scut].double().repeat_interleave(BLOCK)[:size]
        g = st["g"][cut].double() * c
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        step = LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
        out["p"].append(st["p"][cut].double() * (1 - LR * DECAY * dec) - step)
        if case["bits"] == 8:
            u = uniform(size, n, t)
            for name, x, digits, top, least in (("m", m, 3, 7, 2.0 ** -6), ("v", v, 2, 14, 2.0 ** -14)):
                a = torch.zeros(blocks * BLOCK, dtype=torch.float64, device=DEV)
                a[:size] = x.abs()
                most = a.view(blocks, BLOCK).amax(1)
                scale = torch.where(most > 0, torch.exp2(torch.floor(torch.log2(most.clamp(min=1e-300))) - top), 0.0)
                y = a[:size] / scale.repeat_interleave(BLOCK)[:size].clamp(min=1e-300)
                grid = torch.exp2(torch.floor(torch.log2(y.clamp(min=1e-300))) - digits)
                y = torch.floor(y / grid + u) * grid
                low = torch.full_like(y, least) if name == "v" else torch.zeros_like(y)
                y = torch.where(y < least, torch.where(a[:size] > 0, low, 0.0), y)
                out[name].append(torch.where(x < 0, -y, y))
        else:
            out["m"].append(m)
            out["v"].append(v)
    said = {k: torch.cat(x) for k, x in out.items()}
    if case["bits"] == 8:
        # a scale is a step function of its block's largest value, and the operator takes that value in 32 bits: next
        # to a power of two it has no value in 64 bits that a result has to be near
        said["m_scale"] = said["v_scale"] = None
    if case["copy"]:
        said["copy"] = said["p"]
    if case["clip"]:
        said["norm"] = torch.tensor([norm], dtype=torch.float64)
    return said


def uniform(size, tensor, step):
    """The random numbers in [0, 1) of one tensor's elements, with 32-bit products made of 16-bit halves."""
    n = -(-size // 8)
    q = torch.arange(n, device=DEV)
    c = [q % 2 ** 32, q // 2 ** 32, torch.full_like(q, step % 2 ** 32), torch.full_like(q, tensor)]
    key = [SEED % 2 ** 32, SEED // 2 ** 32]

    def product(x, y):
        low, high = x * (y % 65536), x * (y // 65536)      # below 2^48
        whole = low + (high % 65536) * 65536               # below 2^49
        return whole % 2 ** 32, high // 65536 + whole // 2 ** 32

    for _ in range(10):
        l0, h0 = product(c[0], 0xD2511F53)
        l1, h1 = product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    halves = [x for word in c for x in (word % 65536, word // 65536)]
    return torch.stack(halves, 1).reshape(-1)[:size].double() / 65536
