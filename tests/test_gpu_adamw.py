"""svla_op_adamw and svla_train_update on the GPU against the oracle.

What is compared how:
  * moments in 32 bits, codes and scales in 8: bit for bit against the oracle in
    float32 (every product and sum is one IEEE operation on both sides);
  * parameters: against the oracle in float64 started from those same values,
    with every rounding counted in units of 2^-24. m' may cancel, so its error
    is relative to A = |b1 m| + |c1 g'|: the clip factor, g c, a coefficient and
    a product for each summand and the sum make at most 5 A. denom: g'^2 has
    twice (clip factor, product), square, coefficient and product, v the sum: 8,
    of which the root halves to 4; the root, 1 / sqrt(1 - b2^t), its product
    and the sum with eps: 8 in all. Quotient, step size and product: 3.
    Together 16 units of A lr / (1 - b1^t) / denom. p (1 - lr wd) has the
    factor, the product, and p' the last rounding: 2 |p| + |p'| (4 of each
    allowed). bf16 parameters and copies add half a bf16 step: 2^-8 |p'|.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import synth  # noqa: E402
from oracle import optim as oo  # noqa: E402
from vision_language_action_b200 import _abi  # noqa: E402
from vision_language_action_b200.runtime import AdamW, SmolVLA  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def np64(t):
    return t.detach().double().cpu().numpy()


def make(sizes, p="f32", g="f32", bits=32, seed=0, offset=0, fresh=False, spread=1.0):
    """Tensors of the sizes as parts of flat buffers that begin `offset` elements in."""
    gen = torch.Generator().manual_seed(seed)
    n = sum(sizes)

    def flat(x, dt):
        buf = torch.empty(n + offset, dtype=dt, device=DEV)
        buf[offset:] = x.to(dt).to(DEV)
        return list(buf[offset:].split(list(sizes)))

    rnd = lambda s: torch.randn(n, generator=gen) * s
    st = dict(p=flat(rnd(0.05), DT[p]), g=flat(rnd(1e-3) * torch.exp(spread * rnd(1.0)), DT[g]))
    if bits == 32:
        st["m"] = flat(rnd(0.0 if fresh else 3e-4), torch.float32)
        st["v"] = flat(rnd(0.0 if fresh else 1e-3) ** 2, torch.float32)
        st["ms"] = st["vs"] = None
    else:
        # any code but NaN and infinity is a legal start, subnormal ones too
        codes = torch.randint(0, 256, (n,), generator=gen, dtype=torch.int64)
        m = torch.where((codes & 0x7F) == 0x7F, 0, codes)
        v = torch.randint(0, 0x7C, (n,), generator=gen, dtype=torch.int64)
        per = [(k + 255) // 256 for k in sizes]
        exps = torch.randint(-24, -14, (sum(per),), generator=gen).float()
        st["m"] = flat((m * (not fresh)).to(torch.uint8).view(torch.float8_e4m3fn), torch.float8_e4m3fn)
        st["v"] = flat((v * (not fresh)).to(torch.uint8).view(torch.float8_e5m2), torch.float8_e5m2)
        st["ms"] = list((2.0 ** exps).to(DEV).split(per))
        st["vs"] = list((2.0 ** (2 * exps + 8)).to(DEV).split(per))
    return st


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def start_moments(st, bits):
    if bits == 32:
        return [x.cpu().numpy() for x in st["m"]], [x.cpu().numpy() for x in st["v"]]
    out = []
    for c, s, fmt in ((st["m"], st["ms"], oo.E4M3), (st["v"], st["vs"], oo.E5M2)):
        out.append([(oo.decode(codes_of(x), fmt) * np.repeat(s_.cpu().numpy().astype(np.float64), 256)[:x.numel()])
                    .astype(np.float32) for x, s_ in zip(c, s)])
    return out


def check_step(st, before, bits, hp, step, decay, seed, max_norm, copies=None, tensor0=0):
    """`before`: (p, g, m, v) numpy lists from before the step."""
    P, G, M, V = before
    norm = oo.grad_norm(G)
    c = float(np.float32(oo.clip_factor(norm, max_norm)))
    for i, (p, g, m, v) in enumerate(zip(P, G, M, V)):
        if p.size == 0:
            continue
        p32, m1, v1 = oo.adamw(p, g, m, v, *hp, step, decay[i], c, dtype=np.float32)
        if bits == 32:
            assert np.array_equal(st["m"][i].cpu().numpy(), m1), i
            assert np.array_equal(st["v"][i].cpu().numpy(), v1), i
        else:
            u = oo.random16(p.size, tensor0 + i, step, seed)
            for got, scale, x, fmt, keep in ((st["m"][i], st["ms"][i], m1, oo.E4M3, False),
                                             (st["v"][i], st["vs"][i], v1, oo.E5M2, True)):
                codes, s = oo.encode(x, u, fmt, keep)
                assert np.array_equal(scale.cpu().numpy(), s), i
                assert np.array_equal(codes_of(got), codes), i
        p1, _, _ = oo.adamw(p, g, m, v, *hp, step, decay[i], oo.clip_factor(norm, max_norm))
        lr, b1, b2, eps = hp[:4]
        gc = np.asarray(g, np.float64) * c
        v64 = b2 * v.astype(np.float64) + (1 - b2) * gc * gc
        moved = (b1 * np.abs(m.astype(np.float64)) + (1 - b1) * np.abs(gc)) * lr / (1 - b1 ** float(step)) / (
            np.sqrt(v64 / (1 - b2 ** float(step))) + eps)
        tol = U * 4 * (np.abs(p) + np.abs(p1)) + 16 * U * moved + 1e-45
        got = np64(st["p"][i])
        if st["p"][i].dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(p1)
        # where float32 has no g'^2 any more (from 1.8e19 up) v is infinite and the quotient 0 (then NaN): the float32
        # value is the definition there
        over = ~np.isfinite(v1)
        assert np.array_equal(got[over], p32[over].astype(np.float64), equal_nan=True), i
        ok = ~over
        assert (np.abs(got - p1) <= tol)[ok].all(), (i, np.max((np.abs(got - p1) / tol)[ok]))
        if copies is not None and copies[i] is not None:
            assert torch.equal(copies[i], st["p"][i].to(torch.bfloat16)), i
    return norm


def run_case(sizes, p="f32", g="f32", bits=32, max_norm=0.0, step=1, seed=11, offset=0, fresh=False, copy=True,
             hp=(1e-3, 0.9, 0.999, 1e-8, 0.1), spread=1.0, steps=1):
    st = make(sizes, p, g, bits, seed, offset, fresh, spread)
    n = len(sizes)
    decay = [(i * 7 + 1) % 3 != 0 for i in range(n)]
    copies = [torch.zeros(k, dtype=torch.bfloat16, device=DEV) if i % 4 != 3 else None for i, k in enumerate(sizes)] \
        if copy else None
    opt = AdamW(st["p"], lr=hp[0], betas=hp[1:3], eps=hp[3], weight_decay=hp[4], state_bits=bits, max_norm=max_norm,
                copies=copies, decay=decay, seed=(seed << 33) + 5, step=step - 1,
                state=(st["m"], st["v"], st["ms"], st["vs"]))
    for k in range(steps):
        M, V = start_moments(st, bits)
        before = ([x.float().cpu().numpy() for x in st["p"]], [x.float().cpu().numpy() for x in st["g"]], M, V)
        opt.step(st["g"])
        norm = check_step(st, before, bits, hp, step + k, decay, (seed << 33) + 5, max_norm, copies)
        if max_norm:
            assert abs(float(opt.grad_norm) - norm) <= U * norm
    return st, opt


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_types_and_alignments(p, g, bits, offset):
    run_case([256, 1, 255, 257, 4096, 8, 2048 + 13, 31], p, g, bits, step=3, offset=offset, seed=offset + 1)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[1], [7], [256], [255], [257], [0, 5, 0], [0, 0, 300, 0], [100_003], [1 << 20]])
def test_sizes(sizes, bits):
    run_case(sizes, bits=bits, step=2, max_norm=0.5)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [399, 400, 401, 1203])
def test_many_tensors(count, bits):
    """More tensors than one launch's table holds, empty ones among them; the norm goes over all of them."""
    rng = np.random.default_rng(count)
    sizes = [int(x) for x in rng.integers(0, 600, count)]
    run_case(sizes, bits=bits, max_norm=0.3, step=5, spread=0.5)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [1e-6, 0.2, 1e6, float("inf")])
def test_clip(max_norm, bits):
    run_case([5000, 3, 777, 64 * 256], bits=bits, max_norm=max_norm, step=2)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p", ["f32", "bf16"])
def test_from_zero_over_several_steps(p, bits):
    run_case([1000, 33, 512], p=p, bits=bits, fresh=True, steps=6, max_norm=1.0)


@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 6, 2 ** 31 + 3, 2 ** 33 + 1])
def test_step_numbers(step):
    run_case([300, 9], bits=8, step=step)


@pytest.mark.parametrize("hp", [(0.0, 0.9, 0.999, 1e-8, 0.1), (1e-2, 0.0, 0.0, 1e-3, 0.0), (1e-3, 0.5, 0.9999, 1e-15, 10.0),
                                (3.0, 0.9, 0.95, 1.0, 0.0)])
def test_settings(hp):
    for bits in (32, 8):
        run_case([700, 3], bits=bits, step=4, hp=hp, spread=0.3)


def test_wide_gradient_range_in_8_bits():
    """Magnitudes from far below float32's normal range to far above one: zero, tiny, huge in one block and apart."""
    st, _ = run_case([512, 256, 256], bits=8, spread=0.1, step=3)
    for scale in (1e-30, 1e-24, 1e12):
        st = make([512, 300], bits=8, fresh=True, seed=4)
        for g in st["g"]:
            g.mul_(scale)
            g[::7] = 0
        st["g"][1].zero_()
        opt = AdamW(st["p"], state_bits=8, seed=9, state=(st["m"], st["v"], st["ms"], st["vs"]))
        M, V = start_moments(st, 8)
        before = ([x.cpu().numpy() for x in st["p"]], [x.cpu().numpy() for x in st["g"]], M, V)
        opt.step(st["g"])
        with np.errstate(all="ignore"):
            check_step(st, before, 8, (1e-3, 0.9, 0.999, 1e-8, 1e-2), 1, [True, True], 9, 0.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_gradients_that_are_not_finite(bad, bits):
    """Without a clip only the element concerned is lost; with one the whole step is skipped."""
    sizes = [600, 300]
    ref = make(sizes, bits=bits, seed=6)
    opt = AdamW(ref["p"], state_bits=bits, seed=1, state=(ref["m"], ref["v"], ref["ms"], ref["vs"]))
    opt.step(ref["g"])
    st = make(sizes, bits=bits, seed=6)
    st["g"][0][300] = bad
    AdamW(st["p"], state_bits=bits, seed=1, state=(st["m"], st["v"], st["ms"], st["vs"])).step(st["g"])
    for i in range(2):
        keep = torch.ones(sizes[i], dtype=torch.bool, device=DEV)
        if i == 0:
            keep[300] = False
            assert torch.isnan(st["p"][0][300])
            if bits == 8:
                assert int(st["m"][0].view(torch.uint8)[300]) == 0x7F and int(st["v"][0].view(torch.uint8)[300]) == 0x7F
                keep[256:512] = False  # its block's scale may lose its largest element
        assert torch.equal(st["p"][i][keep], ref["p"][i][keep]) or bits == 8
        assert torch.equal(st["m"][i].view(torch.uint8).view(sizes[i], -1)[keep],
                           ref["m"][i].view(torch.uint8).view(sizes[i], -1)[keep])
    skip, untouched = make(sizes, bits=bits, seed=6), make(sizes, bits=bits, seed=6)
    skip["g"][0][300] = bad
    copies = [torch.full((k,), 7.0, dtype=torch.bfloat16, device=DEV) for k in sizes]
    opt = AdamW(skip["p"], state_bits=bits, max_norm=1.0, copies=copies, state=(skip["m"], skip["v"], skip["ms"], skip["vs"]))
    opt.step(skip["g"])
    assert not torch.isfinite(opt.grad_norm).item()
    for k in ("p", "m", "v", "ms", "vs"):
        for a, b in zip(skip[k] or [], untouched[k] or []):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert all((c == 7).all() for c in copies)


def test_nothing_beside_the_tensors_is_written():
    """Neighbours in the same buffers keep their bytes, in front and behind."""
    for bits in (32, 8):
        for lo, n in ((0, 250), (8, 256), (3, 513), (16, 2048), (1, 1)):
            total = lo + n + 40
            p, m32 = torch.full((total,), 3.0, device=DEV), torch.zeros(total, device=DEV)
            codes = torch.zeros(total, dtype=torch.uint8, device=DEV)
            g = torch.ones(total, device=DEV)
            per = (n + 255) // 256
            scales = torch.full((per + 2,), 5.0, device=DEV)
            scales2, copy = scales.clone(), torch.full((total,), 9.0, dtype=torch.bfloat16, device=DEV)
            cut = slice(lo, lo + n)
            if bits == 32:
                v32 = m32.clone()
                state = ([m32[cut]], [v32[cut]], None, None)
            else:
                vc = codes.clone()
                state = ([codes[cut].view(torch.float8_e4m3fn)], [vc[cut].view(torch.float8_e5m2)],
                         [scales[1:1 + per]], [scales2[1:1 + per]])
            AdamW([p[cut]], state_bits=bits, copies=[copy[cut]], state=state).step([g[cut]])
            outside = torch.ones(total, dtype=torch.bool, device=DEV)
            outside[cut] = False
            assert (p[outside] == 3).all() and (copy[outside] == 9).all() and (p[cut] != 3).all()
            if bits == 32:
                assert (m32[outside] == 0).all() and (v32[outside] == 0).all() and (m32[cut] > 0).all()
            else:
                assert (codes[outside] == 0).all() and (vc[outside] == 0).all() and (codes[cut] > 0).all()
                assert scales[0] == scales[-1] == 5 and scales2[0] == scales2[-1] == 5


def test_results_do_not_depend_on_alignment_or_company():
    """The same tensor alone and aligned, in a list, and at an odd address: the same bits."""
    for bits in (32, 8):
        outs = []
        for offset in (0, 3):
            st = make([5000], bits=bits, seed=2, offset=offset)
            opt = AdamW(st["p"], state_bits=bits, seed=4, state=(st["m"], st["v"], st["ms"], st["vs"]))
            for _ in range(3):
                opt.step(st["g"])
            outs.append(st)
        for k in ("p", "m", "v"):
            assert torch.equal(outs[0][k][0].view(torch.uint8), outs[1][k][0].view(torch.uint8)), (bits, k)


def test_owned_state_and_shared_gradients():
    """Moments that the optimiser allocates itself start at zero; one gradient may serve two parameters."""
    g = torch.randn(1000, device=DEV) * 1e-3
    for bits in (32, 8):
        ps = [torch.ones(1000, device=DEV), torch.ones(1000, device=DEV)]
        opt = AdamW(ps, lr=1e-2, weight_decay=0.0, state_bits=bits)
        opt.step([g, g])
        assert torch.equal(ps[0], ps[1])
        # from zero moments the first step is lr g / (|g| + eps) whatever the betas
        g64 = g.double()
        assert (ps[0].double() - (1 - 1e-2 * g64 / (g64.abs() + 1e-8))).abs().max() <= 4 * U + 16 * U * 1e-2


def test_stream_and_repeatability():
    a, b = make([70_000, 11], bits=8, seed=3), make([70_000, 11], bits=8, seed=3)
    side = torch.cuda.Stream()
    for st, stream in ((a, None), (b, side)):
        opt = AdamW(st["p"], state_bits=8, max_norm=0.1, state=(st["m"], st["v"], st["ms"], st["vs"]))
        torch.cuda.synchronize()
        for _ in range(3):
            opt.step(st["g"], stream=stream)
        torch.cuda.synchronize()
    for k in ("p", "m", "v"):
        for x, y in zip(a[k], b[k]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_count_on(bits):
    """A captured step, replayed: the device counter and the device learning rate make each replay the next step."""
    lr = torch.full((1,), 1e-3, dtype=torch.float64, device=DEV)
    a, b = make([3000, 500], bits=bits, seed=8), make([3000, 500], bits=bits, seed=8)
    kw = dict(state_bits=bits, max_norm=0.5, seed=3)
    eager = AdamW(a["p"], state=(a["m"], a["v"], a["ms"], a["vs"]), **kw)
    graphed = AdamW(b["p"], lr=lr, capturable=True, state=(b["m"], b["v"], b["ms"], b["vs"]), **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        graphed.step(b["g"])
    for k in range(4):
        rate = 1e-3 * (k + 1)
        lr.fill_(rate)
        graph.replay()
        eager.step(a["g"], lr=rate)
    torch.cuda.synchronize()
    assert int(graphed.step_tensor) == 4
    for k in ("m", "v"):
        for x, y in zip(a[k], b[k]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for x, y in zip(a["p"], b["p"]):
        # the device's pow may round the last bit of 1 - beta^t apart from the host's: 2 steps of the update
        assert torch.allclose(x, y, rtol=2 ** -22, atol=1e-3 * 2 ** -20)


def test_python_refusals():
    p = [torch.zeros(10, device=DEV), torch.zeros(6, device=DEV)]
    g = [torch.zeros(10, device=DEV), torch.zeros(6, device=DEV)]
    with pytest.raises(ValueError):
        AdamW([p[0], p[1].to(torch.bfloat16)])
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4, 6, device=DEV).t()])
    with pytest.raises(ValueError):
        AdamW(p, state_bits=16)
    with pytest.raises(ValueError):
        AdamW(p, decay=[True])
    with pytest.raises(ValueError):
        AdamW(p, copies=[torch.zeros(10, device=DEV), None])
    with pytest.raises(ValueError):
        AdamW(p, state=([torch.zeros(10, device=DEV)] * 2, g, None, None))
    with pytest.raises(ValueError):
        AdamW(p, lr=torch.zeros(1, device=DEV))
    opt = AdamW(p)
    for bad in ([g[0]], [g[0], g[0]], [g[0], g[1].to(torch.bfloat16)], [g[0], g[1].cpu()], [g[0].half(), g[1].half()]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(_abi.SvlaError):
        AdamW([p[0], p[0]]).step([g[0], g[0]])
    assert opt.steps == 0


# ----------------------------------------------------------------------
# the expert's fine-tune: train_step -> train_update -> train_step
# ----------------------------------------------------------------------
def tiny_case(B=2, L=24, Hc=8, seed=7):
    s = synth.SHAPES["tiny"]
    wb = synth.gen_weights(s, seed, random_affine=True)
    rng = np.random.default_rng(seed)
    kv = torch.from_numpy(rng.standard_normal((2, s.p_layers, B, L, s.p_kv_width)).astype(np.float32)).to(DEV)
    valid = torch.ones(B, L, dtype=torch.uint8, device=DEV)
    f = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV)
    return s, wb, (kv.to(torch.bfloat16), valid, f(B, Hc, s.action_dim), f(B, Hc, s.action_dim),
                   torch.tensor([0.3, 0.8], device=DEV)[:B])


@pytest.mark.parametrize("bits", [32, 8])
def test_train_update_runs_with_the_training_step(bits):
    s, wb, batch = tiny_case()
    m = SmolVLA(s, synth.pack_blob(s, wb), max_batch=2, max_prefix=24, max_chunk=8, train=True)
    other = None
    try:
        names = [(k, shp) for k, shp in synth.manifest(s) if not k.startswith("p")]
        sizes = [int(np.prod(shp)) for _, shp in names]
        decay = [len(shp) == 2 for _, shp in names]
        assert sum(sizes) == m.train_weights().numel()
        start = np.concatenate([wb[k].ravel() for k, _ in names])
        assert np.array_equal(m.train_weights().view(torch.int16).cpu().numpy().view(np.uint16), start)
        master = m.train_weights().float()
        mom = m.new_moments(bits)
        norm = torch.zeros(1, device=DEV)
        hp = dict(lr=5e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, max_norm=0.05, seed=77)
        # the same steps through the list of tensors
        ref = master.clone()
        copy = torch.zeros_like(ref, dtype=torch.bfloat16)
        per = [(n + 255) // 256 for n in sizes]
        mom2 = [None if x is None else x.clone() for x in mom]
        parts = lambda x, k: None if x is None else list(x.split(k))
        opt = AdamW(parts(ref, sizes), lr=5e-3, betas=(0.9, 0.95), weight_decay=0.1, max_norm=0.05, seed=77,
                    state_bits=bits, decay=decay, copies=parts(copy, sizes),
                    state=(parts(mom2[0], sizes), parts(mom2[1], sizes), parts(mom2[2], per), parts(mom2[3], per)))
        for step in range(1, 4):
            loss, grads = m.train_step(*batch)
            m.train_update(master, grads, mom, step, grad_norm=norm, **hp)
            opt.step(list(grads.split(sizes)))
            assert torch.equal(master, ref) and torch.equal(m.train_weights(), copy)
            assert torch.equal(norm, opt.grad_norm) and float(norm) > 0.05
            for x, y in zip(mom, mom2):
                assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        # the next training step is that of a handle created from the updated weights, biases included
        loss, grads = m.train_step(*batch)
        new, at = dict(wb), 0
        bitsw = m.train_weights().view(torch.int16).cpu().numpy().view(np.uint16)
        for (k, shp), n in zip(names, sizes):
            new[k] = bitsw[at:at + n].reshape(shp).copy()
            at += n
        assert all(not np.array_equal(new[k], wb[k]) for k, _ in names)
        other = SmolVLA(s, synth.pack_blob(s, new), max_batch=2, max_prefix=24, max_chunk=8, train=True)
        loss2, grads2 = other.train_step(*batch)
        assert torch.equal(loss, loss2) and torch.equal(grads, grads2)
        # what the handle answers with is unchanged
        noise = batch[3]
        a, _ = m.denoise(batch[0], batch[1], noise, 2)
        fresh = SmolVLA(s, synth.pack_blob(s, wb), max_batch=2, max_prefix=24, max_chunk=8)
        b, _ = fresh.denoise(batch[0], batch[1], noise, 2)
        assert torch.equal(a, b)
        fresh.close()
        # a gradient that is not finite skips the step
        before = master.clone()
        grads[5] = float("nan")
        m.train_update(master, grads, mom, 4, grad_norm=norm, **hp)
        assert torch.equal(master, before) and torch.isnan(norm).item()
    finally:
        m.close()
        if other is not None:
            other.close()


def test_train_update_refusals():
    s, wb, batch = tiny_case()
    plain = SmolVLA(s, synth.pack_blob(s, wb), max_batch=2, max_prefix=24, max_chunk=8)
    lib, p = plain.lib, ctypes.c_void_p(256)
    a = _abi.SvlaAdamwArgs()
    a.state_bits, a.eps, a.step = 32, 1e-8, 1
    assert lib.svla_train_update(plain.h, p, p, p, p, None, None, ctypes.byref(a), None, None) == _abi.SVLA_ERR_UNSUPPORTED
    assert lib.svla_train_weights(plain.h, p, None) == _abi.SVLA_ERR_UNSUPPORTED
    assert lib.svla_train_scale_elems(plain.h) == 0
    plain.close()
    m = SmolVLA(s, synth.pack_blob(s, wb), max_batch=2, max_prefix=24, max_chunk=8, train=True)
    try:
        master, mom = m.train_weights().float(), m.new_moments(8)
        g = torch.zeros_like(master)
        call = lambda **kw: lib.svla_train_update(
            m.h, *(ctypes.c_void_p(t.data_ptr()) for t in (master, g, mom[0], mom[1])), None, None,
            ctypes.byref(setattrs(a, **kw)), None, None)
        setattrs = lambda x, **kw: [setattr(x, k, v) for k, v in kw.items()] and x
        assert call(state_bits=8) == _abi.SVLA_ERR_ARG          # no scales
        assert call(state_bits=16) == _abi.SVLA_ERR_ARG
        assert call(state_bits=32, param_type=1) == _abi.SVLA_ERR_ARG
        assert call(param_type=0, step=0) == _abi.SVLA_ERR_ARG
        assert b"step" in lib.svla_last_error(m.h)
        with pytest.raises(ValueError):
            m.train_update(master[:-1], g, mom, 1)
        with pytest.raises(ValueError):
            m.train_update(master, g.to(torch.bfloat16), mom, 1)
        with pytest.raises(_abi.SvlaError):
            m.train_update(master, master, mom, 1)
        with pytest.raises(ValueError):
            m.train_weights(master)
    finally:
        m.close()


@pytest.mark.parametrize("scale", [1e-22, 1e-19, 1e16, 1e18, 1e19])
def test_moments_near_the_ends_of_float32(scale):
    """Blocks that leave the kernel's usual case: v underflows, or passes 2^100 (where float32 has no more room for its
    square): all elements so, or one in a block."""
    for one in (False, True):
        st = make([256, 512, 100], bits=8, fresh=True, seed=12)
        for g in st["g"]:
            if one:
                g[5] = scale
            else:
                g.mul_(1e3 * scale)
        opt = AdamW(st["p"], state_bits=8, seed=9, state=(st["m"], st["v"], st["ms"], st["vs"]))
        for step in (1, 2):
            M, V = start_moments(st, 8)
            before = ([x.cpu().numpy() for x in st["p"]], [x.cpu().numpy() for x in st["g"]], M, V)
            opt.step(st["g"])
            with np.errstate(all="ignore"):
                check_step(st, before, 8, (1e-3, 0.9, 0.999, 1e-8, 1e-2), step, [True] * 3, 9, 0.0)


def test_a_negative_second_moment_stays_in_its_element():
    """No step makes one; one given makes its element NaN (the root has no value) and leaves its neighbours alone."""
    a, b = make([512], bits=8, seed=3), make([512], bits=8, seed=3)
    b["v"][0].view(torch.uint8)[40] = 0x80 | 100
    b["g"][0][40] = a["g"][0][40] = 0.0
    for st in (a, b):
        st["vs"][0].fill_(2.0 ** -40)
        AdamW(st["p"], state_bits=8, state=(st["m"], st["v"], st["ms"], st["vs"])).step(st["g"])
    keep = torch.arange(512, device=DEV) != 40
    assert torch.isnan(b["p"][0][40]) and int(b["v"][0].view(torch.uint8)[40]) == 0x7F
    assert torch.equal(a["m"][0].view(torch.uint8), b["m"][0].view(torch.uint8))
    assert torch.equal(a["v"][0].view(torch.uint8)[keep][256:], b["v"][0].view(torch.uint8)[keep][256:])
    assert torch.allclose(a["p"][0][keep], b["p"][0][keep], rtol=1e-6)


@pytest.mark.parametrize("N", [16, 64, 4096])
@pytest.mark.parametrize("max_norm", [0.0, 1.0])
def test_copies_as_the_weights_of_the_next_product(N, max_norm):
    """The bf16 copy taken as the W of svla_op_gemm right behind the step, which fetches it as early as it may. As a
    graph, without the host's time between."""
    from vision_language_action_b200.runtime import op_gemm
    K = 1024
    gen = torch.Generator().manual_seed(2)
    start, g = torch.randn(N, K, generator=gen).to(DEV), torch.randn(N, K, generator=gen).to(DEV)
    lhs = torch.randn(64, K, generator=gen).to(torch.bfloat16).to(DEV)
    p, copy, out = start.clone(), torch.zeros(N, K, dtype=torch.bfloat16, device=DEV), torch.empty(64, N, device=DEV)
    opt = AdamW([p], lr=0.5, max_norm=max_norm, copies=[copy], capturable=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step([g])
        op_gemm("f32", lhs, copy, out, splits=1)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        early = out.clone()
        assert torch.equal(early, op_gemm("f32", lhs, copy, out, splits=1))


def test_train_weights_into_a_given_tensor():
    s, wb, _ = tiny_case()
    m = SmolVLA(s, synth.pack_blob(s, wb), max_batch=2, max_prefix=24, max_chunk=8, train=True)
    try:
        want = m.train_weights()
        out = torch.zeros_like(want)
        assert m.train_weights(out) is out and torch.equal(out, want)
        for bad in (torch.zeros(2 * want.numel(), dtype=torch.bfloat16, device=DEV)[::2], out.cpu(), out[:-1], out.float()):
            with pytest.raises(ValueError):
                m.train_weights(bad)
    finally:
        m.close()


def test_parameters_whose_storage_was_replaced():
    """`.data = ..` between steps, as moving or reloading a module does: the step goes to the storage of the moment,
    never to the old one, and refuses one of another type or size."""
    p, q, g = torch.ones(100, device=DEV), torch.ones(100, device=DEV), torch.full((100,), 0.1, device=DEV)
    copy = torch.zeros(100, dtype=torch.bfloat16, device=DEV)
    opt, ref = AdamW([p], lr=1e-2, copies=[copy]), AdamW([q], lr=1e-2)
    opt.step([g]), ref.step([g])
    old, old_copy = p.data, copy.data
    keep, keep_copy = old.clone(), old_copy.clone()
    p.data, copy.data = old.clone(), torch.zeros_like(copy)
    opt.step([g]), ref.step([g])
    assert torch.equal(old, keep) and torch.equal(old_copy, keep_copy)
    assert torch.equal(p, q) and torch.equal(copy, q.to(torch.bfloat16))
    for bad in (torch.ones(100, dtype=torch.bfloat16, device=DEV), torch.ones(99, device=DEV),
                torch.ones(200, device=DEV)[::2], torch.ones(100)):
        other = torch.ones(100, device=DEV)
        opt = AdamW([other])
        other.data = bad
        with pytest.raises(ValueError):
            opt.step([g])


def test_a_missing_gradient_is_refused():
    p = [torch.zeros(10, device=DEV), torch.zeros(6, device=DEV)]
    opt = AdamW(p)
    with pytest.raises(ValueError):
        opt.step([torch.zeros(10, device=DEV), None])
    assert opt.steps == 0 and not p[0].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_past_32_bits_of_elements(bits):
    """2^32 + 300 elements, zero but for a stretch across 2^32 and the tensor's end, which follows the oracle with the
    random bits of its own element numbers."""
    from oracle.philox import philox4x32_10
    first, n = 2 ** 32 - 512, 2 ** 32 + 300
    k, seed, hp = n - first, 7, (1e-3, 0.9, 0.999, 1e-8, 0.1)
    if torch.cuda.mem_get_info()[1] < 80 << 30:
        pytest.skip("needs 60 GB")
    part = make([k], "bf16", "bf16", bits, seed=21)
    big = lambda dt: torch.zeros(n, dtype=torch.uint8 if dt.itemsize == 1 else dt, device=DEV).view(dt)
    st = {key: [big(part[key][0].dtype)] for key in ("p", "g", "m", "v")}
    per = (n + 255) // 256
    st["ms"] = [torch.zeros(per, device=DEV)] if bits == 8 else None
    st["vs"] = [torch.zeros(per, device=DEV)] if bits == 8 else None
    raw = lambda t: t.view(torch.uint8)
    for key in ("p", "g", "m", "v"):
        raw(st[key][0])[first * st[key][0].element_size():] = raw(part[key][0])
    if bits == 8:
        for key in ("ms", "vs"):
            st[key][0][first // 256:] = part[key][0]
    M, V = start_moments(part, bits)
    p, g = part["p"][0].float().cpu().numpy(), part["g"][0].float().cpu().numpy()
    AdamW(st["p"], lr=hp[0], weight_decay=hp[4], state_bits=bits, seed=seed, step=4,
          state=(st["m"], st["v"], st["ms"], st["vs"])).step(st["g"])
    torch.cuda.synchronize()
    for key in ("p", "m", "v"):
        assert not raw(st[key][0])[:first * st[key][0].element_size()].any()
    p32, m1, v1 = oo.adamw(p, g, M[0], V[0], *hp, 5, True, 1.0, dtype=np.float32)
    tail = {key: st[key][0][first:] for key in ("p", "m", "v")}
    if bits == 32:
        assert np.array_equal(tail["m"].cpu().numpy(), m1) and np.array_equal(tail["v"].cpu().numpy(), v1)
    else:
        q = np.arange(first // 8, (n + 7) // 8, dtype=np.uint64)
        c = (q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), np.full_like(q, 5), np.zeros_like(q))
        words = np.stack(philox4x32_10(c, (seed, 0)), axis=1)
        u = np.stack([words & 0xFFFF, words >> 16], axis=2).reshape(-1)[:k].astype(np.int64)
        for key, scale, x, fmt, keep in (("m", "ms", m1, oo.E4M3, False), ("v", "vs", v1, oo.E5M2, True)):
            codes, s = oo.encode(x, u, fmt, keep)
            assert np.array_equal(codes_of(tail[key]), codes)
            assert np.array_equal(st[scale][0][first // 256:].cpu().numpy(), s) and not st[scale][0][:first // 256].any()
    # bf16 parameters: half a step, beside float32's own error of the step (the docstring's bound is far below it)
    assert (np.abs(np64(tail["p"]) - p32.astype(np.float64)) <= 2.0 ** -8 * np.abs(p32) + 1e-6).all()
    del st, tail
    torch.cuda.empty_cache()


def test_two_threads_at_once():
    """Two host threads, each with its own stream, optimiser and norm, give what each gives alone."""
    import threading
    from vision_language_action_b200.runtime import op_layernorm, op_layernorm_backward

    def work(seed, out, stream):
        gen = torch.Generator().manual_seed(seed)
        p, g, xs = ([torch.randn(n, generator=gen).to(DEV) for n in ns]
                    for ns in ((1000, 70000, 33), (1000, 70000, 33), (500 * 768, 500 * 768, 768)))
        x, dy, gain = xs[0].view(500, 768), xs[1].view(500, 768), xs[2]
        res = [torch.zeros_like(t) for t in (x, x, gain, gain)]
        mean, rstd = torch.zeros(500, device=DEV), torch.zeros(500, device=DEV)
        opt = AdamW(p, state_bits=8, max_norm=1.0, seed=seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(50):
                opt.step(g)
                op_layernorm(x, gain, None, res[0], 1e-5, mean, rstd)
                op_layernorm_backward(dy, x, gain, mean, rstd, *res[1:])
        stream.synchronize()
        out[seed] = p + res

    alone, together = {}, {}
    for seed in (1, 2):
        work(seed, alone, torch.cuda.Stream())
    threads = [threading.Thread(target=work, args=(s, together, torch.cuda.Stream())) for s in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for seed in (1, 2):
        assert all(torch.equal(a, b) for a, b in zip(alone[seed], together[seed]))


@pytest.mark.parametrize("exponent", [90, 93, 100, 117, 118, 119])
def test_a_first_moment_near_the_end_of_float32(exponent):
    """m from 2^97 up to 2^127 beside an ordinary v, as no run of gradients leaves it but a given state may: the codes
    and scales of the definition all the same. (p is beyond what m / sqrt(v) keeps in float32 and is not looked at.)"""
    n = 700
    gen = torch.Generator().manual_seed(exponent)
    mc = torch.randint(0x60, 0x7F, (n,), generator=gen, dtype=torch.int64) | 0x80 * torch.randint(0, 2, (n,), generator=gen)
    vc = torch.randint(0x20, 0x70, (n,), generator=gen, dtype=torch.int64)
    st = dict(p=[torch.zeros(n, device=DEV)], g=[torch.randn(n, generator=gen).to(DEV)],
              m=[mc.to(torch.uint8).to(DEV).view(torch.float8_e4m3fn)],
              v=[vc.to(torch.uint8).to(DEV).view(torch.float8_e5m2)],
              ms=[torch.full((3,), 2.0 ** exponent, device=DEV)], vs=[torch.full((3,), 2.0 ** -10, device=DEV)])
    M, V = start_moments(st, 8)
    g = st["g"][0].cpu().numpy()
    AdamW(st["p"], state_bits=8, seed=9, step=2, state=(st["m"], st["v"], st["ms"], st["vs"])).step(st["g"])
    _, m1, v1 = oo.adamw(np.zeros(n), g, M[0], V[0], 1e-3, 0.9, 0.999, 1e-8, 1e-2, 3, dtype=np.float32)
    u = oo.random16(n, 0, 3, 9)
    for got, scale, x, fmt, keep in ((st["m"][0], st["ms"][0], m1, oo.E4M3, False),
                                     (st["v"][0], st["vs"][0], v1, oo.E5M2, True)):
        codes, s = oo.encode(x, u, fmt, keep)
        assert np.array_equal(scale.cpu().numpy(), s)
        assert np.array_equal(codes_of(got), codes)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_first_step_on_another_stream_beside_queued_work(bits):
    """The moments' zeros, the norm and the workspace are made on the stream current at construction, behind what is
    queued there; the first step runs on another."""
    n = 300_000
    g = torch.randn(n, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) * 1e-3
    ref, p = torch.ones(n, device=DEV), torch.ones(n, device=DEV)
    kw = dict(lr=1e-2, state_bits=bits, max_norm=0.1, capturable=True)
    AdamW([ref], **kw).step([g])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # about 10 ms
    tmp = torch.empty(8 * n, dtype=torch.uint8, device=DEV).fill_(255)
    del tmp
    opt = AdamW([p], **kw)
    assert torch.cuda.current_stream().query()
    opt.step([g], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(p, ref) and int(opt.step_tensor) == 1


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("step", [3, 2 ** 32, 2 ** 32 + 1, 2 ** 53 - 1])
def test_a_device_learning_rate_beside_the_hosts_step(step, bits):
    """lr_device without step_device: the bias corrections are those of the whole step number, as with a host's rate."""
    lib, n = _abi.load(), 3000
    outs = []
    for on_device in (False, True):
        st = make([n], bits=bits, seed=12)
        t, a = _abi.SvlaAdamwTensor(), _abi.SvlaAdamwArgs()
        t.param, t.grad, t.m, t.v = (st[k][0].data_ptr() for k in ("p", "g", "m", "v"))
        if bits == 8:
            t.m_scale, t.v_scale = st["ms"][0].data_ptr(), st["vs"][0].data_ptr()
        t.n, t.decay = n, 1
        lr = torch.full((1,), 1e-2, dtype=torch.float64, device=DEV)
        a.state_bits, a.lr, a.beta1, a.beta2, a.eps, a.weight_decay, a.step = bits, 1e-2, 0.9, 0.999, 1e-8, 0.1, step
        if on_device:
            a.lr, a.lr_device = 0.0, lr.data_ptr()
        _abi.check(lib.svla_op_adamw(ctypes.byref(t), 1, ctypes.byref(a), None, 0, None,
                                     torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        outs.append(st)
    host, dev = outs
    for k in ("m", "v"):
        assert torch.equal(host[k][0].view(torch.uint8), dev[k][0].view(torch.uint8))
    # the three coefficients may differ by a unit of either side's arithmetic: two units of the step, which is no larger
    # than |p0| + |p|, and one of p0 (1 - lr wd); p itself is rounded on both sides: 3 |p0| + 4 |p| units
    p0, p, q = make([n], bits=bits, seed=12)["p"][0].double(), host["p"][0].double(), dev["p"][0].double()
    assert torch.isfinite(q).all() and ((p - q).abs() <= 4 * U * (p0.abs() + p.abs())).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_stay_where_they_were_at_construction(bits):
    """A moment given other storage, or dropped from its list: the steps go on with the memory of the construction,
    which is not given back, and what is allocated since then keeps its values."""
    n = 300_000
    a, b = make([n], bits=bits, seed=3), make([n], bits=bits, seed=3)
    ref = AdamW(a["p"], state_bits=bits, state=(a["m"], a["v"], a["ms"], a["vs"]))
    opt = AdamW(b["p"], state_bits=bits, state=(b["m"], b["v"], b["ms"], b["vs"]))
    p = b["p"]
    # parts of one buffer each: tensors of their own from here on
    columns = [opt.m, opt.v] + ([opt.m_scale, opt.v_scale] if bits == 8 else [])
    for c in columns:
        c[0] = c[0].clone()
    own = AdamW(p, state_bits=bits, state=(opt.m, opt.v, opt.m_scale, opt.v_scale))
    size = [c[0].numel() * c[0].element_size() for c in columns]
    b = opt = None
    for k, c in enumerate((own.m, own.v) + ((own.m_scale, own.v_scale) if bits == 8 else ())):
        if k % 2:
            c[0].data = torch.zeros_like(c[0])
        else:
            c[0] = torch.zeros_like(c[0])
        columns[k] = None
    fresh = [torch.full((s,), 7, dtype=torch.uint8, device=DEV) for s in size]
    for _ in range(3):
        ref.step(a["g"])
        own.step(a["g"])
    torch.cuda.synchronize()
    assert torch.equal(p[0], a["p"][0]) and all((t == 7).all() for t in fresh)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e25, 2e30, 1e38, 3e38])
def test_an_eps_near_the_end_of_float32(eps, bits):
    """The quotient m / (root + eps) where eps is all of the denominator and its reciprocal no normal number. Gradients of
    1e12 keep the quotient itself a normal number, and the learning rate brings it back to the size of the parameters."""
    st = make([3000], bits=bits, seed=15)
    p = st["p"][0].cpu().numpy()
    st["g"][0].mul_(1e15)
    (m,), (v,) = start_moments(st, bits)
    hp = dict(lr=eps * 1e-13, betas=(0.9, 0.999), eps=eps, weight_decay=0.0)
    AdamW(st["p"], state_bits=bits, seed=1, step=9, state=(st["m"], st["v"], st["ms"], st["vs"]), **hp).step(st["g"])
    g = np64(st["g"][0])
    want, _, _ = oo.adamw(p.astype(np.float64), g, m.astype(np.float64), v.astype(np.float64), hp["lr"], 0.9, 0.999, eps, 0.0, 10)
    A = np.abs(0.9 * m.astype(np.float64)) + np.abs(0.1 * g)
    tol = 16 * U * A * hp["lr"] / (1 - 0.9 ** 10) / eps + 4 * U * (np.abs(p) + np.abs(want))
    moved = np.abs(want - p).max()
    assert moved > 1e-3 and (np.abs(np64(st["p"][0]) - want) <= tol).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [(0,), (300,), (255, 256), (599,)])
def test_the_neighbours_of_a_gradient_that_is_not_finite(at, bad, bits):
    """Only the elements concerned are lost: the others of their 256 step as the oracle's do, to codes and scales that
    leave the lost ones out, and every other 256 bit for bit as without them (with 32 bits every other element)."""
    sizes, hp = [600, 300], (1e-3, 0.9, 0.999, 1e-8, 1e-2)
    ref, st = (make(sizes, bits=bits, seed=6) for _ in range(2))
    for i in at:
        st["g"][0][i] = bad
    M, V = start_moments(st, bits)
    before = ([x.cpu().numpy() for x in st["p"]], [x.cpu().numpy() for x in st["g"]], M, V)
    for s in (ref, st):
        AdamW(s["p"], state_bits=bits, seed=1, state=(s["m"], s["v"], s["ms"], s["vs"])).step(s["g"])
    if bits == 8:
        with np.errstate(all="ignore"):
            check_step(st, before, bits, hp, 1, [True, True], 1, 0.0)
    lost = torch.zeros(sizes[0], dtype=torch.bool, device=DEV)
    lost[list(at)] = True
    assert torch.isnan(st["p"][0][lost]).all() and torch.isfinite(st["p"][0][~lost]).all()
    apart = ~lost
    for i in at if bits == 8 else ():
        apart[i // 256 * 256:i // 256 * 256 + 256] = False
    for i, keep in ((0, apart), (1, torch.ones(sizes[1], dtype=torch.bool, device=DEV))):
        assert keep.any()
        for k in ("p", "m", "v"):
            x, y = (s[k][i].view(torch.uint8).view(sizes[i], -1)[keep] for s in (st, ref))
            assert torch.equal(x, y), (i, k)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_first_tensor_in_lists_of_every_length(bits):
    """Alone, in a list of one launch's short table, past it, and past the long one: the same bits."""
    outs = []
    for count in (1, 32, 33, 400, 401, 900):
        st = make([5000], bits=bits, seed=2)
        more = [make([k], bits=bits, seed=20) for k in (300, 1, 0, 2049)]
        lists = {k: None if st[k] is None else list(st[k]) for k in ("p", "g", "m", "v", "ms", "vs")}
        for i in range(1, count):
            for k in lists:
                if lists[k] is not None:
                    t = more[i % 4][k][0]
                    lists[k].append(t if k == "g" else t.clone())
        opt = AdamW(lists["p"], state_bits=bits, seed=4, state=(lists["m"], lists["v"], lists["ms"], lists["vs"]))
        for _ in range(3):
            opt.step(lists["g"])
        outs.append(st)
    for st in outs[1:]:
        for k in ("p", "m", "v") + (("ms", "vs") if bits == 8 else ()):
            assert torch.equal(outs[0][k][0].view(torch.uint8), st[k][0].view(torch.uint8)), k
