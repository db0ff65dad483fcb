"""svla_op_layernorm and its backward pass on the GPU against the oracle in float64.

Tolerances. A sum of n float32 terms over a tree of depth d is off by at most
d 2^-24 sum|terms|; a thread adds up to 32 terms in turn, then 5 shuffles and up
to 16 warps: d <= 64. So |mean - exact| <= 64 2^-24 mean|x|, and rstd's relative
error, half of the variance's, is at most 64 2^-24 (1 + 2 max|x| rstd ..) plus two
units of the root: with the rows here (|x| / sigma < 8) 1e-5 covers both with a
wide margin. y and dx are then products of a few such factors: 2e-5 of the row's
scale, plus half a step of the output's type (bf16 2^-8 of the value). The
column sums of dgamma and dbeta add at most M terms: M / 296 / rows-a-block of
them in turn and then at most 64 partial ones: (M / 296 + 64) 2^-24 sum|terms|,
beside the 2e-5 that a term of dgamma carries from xh.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import optim as oo  # noqa: E402
from vision_language_action_b200 import _abi  # noqa: E402
from vision_language_action_b200.runtime import AdamW, op_gemm, op_layernorm, op_layernorm_backward  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def np64(t):
    return t.detach().double().cpu().numpy()


def rows(M, D, dt, gen, pad=0, scale=1.0, shift=0.0):
    buf = torch.full((M, D + pad), 77.0, dtype=dt, device=DEV)
    buf[:, :D] = (torch.randn(M, D, generator=gen) * scale + shift).to(dt).to(DEV)
    return buf[:, :D]


def make(M, D, x="f32", y="f32", w="f32", pad=0, seed=0):
    gen = torch.Generator().manual_seed(seed * 1000 + D)
    return dict(
        x=rows(M, D, DT[x], gen, pad, 1.3, 0.4), dy=rows(M, D, DT[y], gen, pad, 0.1),
        gamma=(1 + 0.3 * torch.randn(D, generator=gen)).to(DT[w]).to(DEV),
        beta=(0.3 * torch.randn(D, generator=gen)).to(DT[w]).to(DEV),
        y=rows(M, D, DT[y], gen, pad), dx=rows(M, D, DT[x], gen, pad),
        mean=torch.full((M,), 9.0, device=DEV), rstd=torch.full((M,), 9.0, device=DEV),
        dgamma=torch.full((D,), 9.0, device=DEV), dbeta=torch.full((D,), 9.0, device=DEV))


def untouched_pad(t, pad):
    if pad:
        whole = t.as_strided((t.shape[0], t.shape[1] + pad), t.stride(), t.storage_offset())
        assert (whole[:, t.shape[1]:] == 77).all()


def check(M, D, eps=1e-5, beta=True, **kw):
    a = make(M, D, **kw)
    pad = kw.get("pad", 0)
    op_layernorm(a["x"], a["gamma"], a["beta"] if beta else None, a["y"], eps, a["mean"], a["rstd"])
    x, g, b = np64(a["x"]), np64(a["gamma"]), np64(a["beta"]) if beta else 0.0
    y, mean, rstd = oo.layernorm(x, g, b, eps)
    assert (np.abs(np64(a["mean"]) - mean) <= 64 * 2.0 ** -24 * np.abs(x).mean(1) + 1e-30).all()
    if D > 1:
        assert (np.abs(np64(a["rstd"]) / rstd - 1) <= 1e-5).all()
    scale = np.abs((x - mean[:, None]) * rstd[:, None] * g) + 1.0
    tol = 2e-5 * scale + HALF[a["y"].dtype] * np.abs(y) + (1e-3 if D == 1 else 0.0)
    assert (np.abs(np64(a["y"]) - y) <= tol).all(), np.max(np.abs(np64(a["y"]) - y) / tol)
    untouched_pad(a["y"], pad)
    # backward, from the statistics that the forward left
    op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"], a["dgamma"], a["dbeta"])
    dy = np64(a["dy"])
    dx, dg, db = oo.layernorm_backward(dy, x, g, np64(a["mean"]), np64(a["rstd"]))
    w = np.abs(dy * g)
    xh = np.abs((x - np64(a["mean"])[:, None]) * np64(a["rstd"])[:, None])
    scale = np64(a["rstd"])[:, None] * (w + w.mean(1, keepdims=True) + xh * (w * xh).mean(1, keepdims=True))
    tol = 2e-5 * scale + HALF[a["dx"].dtype] * np.abs(dx)
    assert (np.abs(np64(a["dx"]) - dx) <= tol).all(), np.max(np.abs(np64(a["dx"]) - dx) / tol)
    untouched_pad(a["dx"], pad)
    chain = (M / 296 + 64) * 2.0 ** -24
    assert (np.abs(np64(a["dgamma"]) - dg) <= (chain + 1e-6) * (np.abs(dy) * xh).sum(0) + 1e-30).all()
    assert (np.abs(np64(a["dbeta"]) - db) <= chain * np.abs(dy).sum(0) + 1e-30).all()
    return a


# each width class of the kernels: one to four units of 8 a lane of one warp, two a thread of several, shared-memory sums
WIDTHS = [1, 2, 7, 8, 31, 32, 255, 256, 257, 512, 513, 720, 768, 960, 1000, 1024, 1025, 1283, 2048, 4096, 5000, 8192, 8193,
          8200, 12345, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("M", [1, 13])
def test_widths(M, D):
    check(M, D, seed=M)


@pytest.mark.parametrize("D", [768, 771, 2048, 16384])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("w", ["f32", "bf16"])
def test_types(D, x, y, w):
    check(37, D, x=x, y=y, w=w, seed=3)


@pytest.mark.parametrize("pad", [1, 4, 8, 24])
@pytest.mark.parametrize("D", [64, 768, 1283, 8200])
def test_strides(pad, D):
    """Rows further apart than their width; the elements between them are neither read nor written."""
    check(21, D, pad=pad, x="bf16", y="f32")
    check(21, D, pad=pad, x="f32", y="bf16")


@pytest.mark.parametrize("M,D", [(2, 768), (8, 768), (9, 768), (296 * 8, 768), (296 * 8 + 1, 768), (50, 720), (5001, 33),
                                 (701, 2048), (1000, 4096), (300, 16384)])
def test_row_counts(M, D):
    check(M, D, seed=5)


def test_no_beta_and_optional_outputs():
    a = check(40, 768, beta=False)
    y2 = torch.empty_like(a["y"])
    op_layernorm(a["x"], a["gamma"], None, y2, 1e-5)
    assert torch.equal(y2, a["y"])
    for dg, db in ((None, None), (a["dgamma"].clone(), None), (None, a["dbeta"].clone())):
        dx = torch.empty_like(a["dx"])
        for t in (dg, db):
            if t is not None:
                t.fill_(5.0)
        op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], dx, dg, db)
        assert torch.equal(dx, a["dx"])
        assert dg is None or torch.equal(dg, a["dgamma"])
        assert db is None or torch.equal(db, a["dbeta"])


def test_no_rows():
    a = make(0, 768)
    op_layernorm(a["x"], a["gamma"], a["beta"], a["y"], 1e-5, a["mean"], a["rstd"])
    op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"], a["dgamma"], a["dbeta"])
    assert not a["dgamma"].any() and not a["dbeta"].any()


@pytest.mark.parametrize("M,D", [(100, 768), (77, 2048), (30, 771), (20, 16384)])
def test_in_place(M, D):
    a = make(M, D, seed=9)
    keep = a["x"].clone()
    op_layernorm(a["x"], a["gamma"], a["beta"], a["y"], 1e-5, a["mean"], a["rstd"])
    op_layernorm(keep, a["gamma"], a["beta"], keep, 1e-5)
    assert torch.equal(keep, a["y"])
    op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"], a["dgamma"], a["dbeta"])
    for over in ("x", "dy"):
        b = {k: v.clone() for k, v in a.items()}
        op_layernorm_backward(b["dy"], b["x"], b["gamma"], b["mean"], b["rstd"], b[over], b["dgamma"], b["dbeta"])
        assert torch.equal(b[over], a["dx"]) and torch.equal(b["dgamma"], a["dgamma"])


def test_constant_rows_and_large_offsets():
    """A constant row has no variance: y is beta; a mean far from zero costs no more than the mean's own rounding."""
    x = torch.full((5, 768), 3.0, device=DEV)
    a = make(5, 768)
    op_layernorm(x, a["gamma"], a["beta"], a["y"], 1e-5, a["mean"], a["rstd"])
    assert torch.allclose(a["y"], a["beta"].expand(5, 768), atol=1e-3) and (a["mean"] - 3).abs().max() < 1e-6
    gen = torch.Generator().manual_seed(1)
    x = rows(6, 768, torch.float32, gen, scale=1.0, shift=1000.0)
    op_layernorm(x, a["gamma"], a["beta"], a["y"].new_empty(6, 768), 1e-5, m := torch.empty(6, device=DEV),
                 r := torch.empty(6, device=DEV))
    _, mean, rstd = oo.layernorm(np64(x), 1.0, 0.0, 1e-5)
    # the differences to a mean that is off by e add e^2 to a variance of 1: e <= 64 2^-24 1000
    assert np.abs(np64(m) - mean).max() <= 64 * 2.0 ** -24 * 1000 and np.abs(np64(r) / rstd - 1).max() <= 2e-5


def test_values_that_are_not_finite_stay_in_their_row():
    for bad in (float("nan"), float("inf")):
        for D in (768, 2048, 771):
            a, b = make(20, D, seed=4), make(20, D, seed=4)
            b["x"][7, 5] = bad
            for t in (a, b):
                op_layernorm(t["x"], t["gamma"], t["beta"], t["y"], 1e-5, t["mean"], t["rstd"])
                op_layernorm_backward(t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"], t["dx"], t["dgamma"], t["dbeta"])
            keep = [i for i in range(20) if i != 7]
            assert torch.equal(a["y"][keep], b["y"][keep]) and torch.equal(a["dx"][keep], b["dx"][keep])
            assert not torch.isfinite(b["y"][7]).any() and torch.equal(a["dbeta"], b["dbeta"])


def test_repeatable_on_another_stream_and_in_a_graph():
    a = make(3000, 768, x="bf16", y="bf16")
    fwd = lambda t, s=None: op_layernorm(t["x"], t["gamma"], t["beta"], t["y"], 1e-5, t["mean"], t["rstd"], stream=s)
    bwd = lambda t, s=None: op_layernorm_backward(t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"], t["dx"], t["dgamma"],
                                                  t["dbeta"], stream=s)
    fwd(a), bwd(a)
    ref = {k: v.clone() for k, v in a.items()}
    side = torch.cuda.Stream()
    for k in ("y", "dx", "dgamma", "dbeta", "mean", "rstd"):
        a[k].fill_(1.0)
    torch.cuda.synchronize()
    fwd(a, side), bwd(a, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], ref[k]) for k in ref)
    graphs = []
    for _ in range(2):  # each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fwd(a), bwd(a)
        graphs.append(g)
    for g in graphs:
        for k in ("y", "dx", "dgamma", "dbeta", "mean", "rstd"):
            a[k].fill_(1.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], ref[k]) for k in ref)


def test_python_refusals():
    a = make(4, 64)
    with pytest.raises(ValueError):
        op_layernorm(a["x"].half(), a["gamma"], None, a["y"])
    with pytest.raises(ValueError):
        op_layernorm(a["x"].t(), a["gamma"], None, a["y"])
    with pytest.raises(ValueError):
        op_layernorm(a["x"], a["gamma"][:-1], None, a["y"])
    with pytest.raises(ValueError):
        op_layernorm(a["x"], a["gamma"], a["beta"].to(torch.bfloat16), a["y"])
    with pytest.raises(ValueError):
        op_layernorm(a["x"][:1].expand(4, 64), a["gamma"], None, a["y"])
    with pytest.raises(ValueError):
        op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"][:-1], a["rstd"], a["dx"])
    with pytest.raises(ValueError):
        op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"].to(torch.bfloat16))
    with pytest.raises(_abi.SvlaError):
        op_layernorm(a["x"], a["gamma"], None, a["y"], eps=0.0)


def test_norm_backward_and_optimiser_together():
    """A layer norm trained as it would be: forward, backward, AdamW on gain and bias (bf16 copies that the next
    forward reads), against the same three steps in float64."""
    M, D = 600, 768
    a = make(M, D, x="bf16", y="bf16", w="bf16", seed=2)
    gain, bias = a["gamma"].float(), a["beta"].float()
    opt = AdamW([gain, bias], lr=1e-2, weight_decay=0.0, copies=[a["gamma"], a["beta"]], max_norm=1.0)
    x, dy = np64(a["x"]), np64(a["dy"])
    p = [np64(gain), np64(bias)]
    mom = [[np.zeros(D), np.zeros(D)], [np.zeros(D), np.zeros(D)]]
    for step in range(1, 4):
        op_layernorm(a["x"], a["gamma"], a["beta"], a["y"], 1e-5, a["mean"], a["rstd"])
        g16 = [np64(a["gamma"]), np64(a["beta"])]
        y, mean, rstd = oo.layernorm(x, g16[0], g16[1], 1e-5)
        assert np.abs(np64(a["y"]) - y).max() <= 2.0 ** -8 * np.abs(y).max() + 1e-4
        op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"], a["dgamma"], a["dbeta"])
        opt.step([a["dgamma"], a["dbeta"]])
        _, dg, db = oo.layernorm_backward(dy, x, g16[0], mean, rstd)
        c = oo.clip_factor(oo.grad_norm([dg, db]), 1.0)
        for i, g in enumerate((dg, db)):
            p[i], mom[i][0], mom[i][1] = oo.adamw(p[i], g, *mom[i], 1e-2, 0.9, 0.999, 1e-8, 0.0, step, c=c)
        # m / sqrt(v) keeps the gradients' relative error (1e-6 of sum|terms|, up to 1e-3 of a sum that cancels)
        assert np.abs(np64(gain) - p[0]).max() <= 1e-2 * step * 2e-3 and np.abs(np64(bias) - p[1]).max() <= 1e-2 * step * 2e-3
        assert torch.equal(a["gamma"], gain.to(torch.bfloat16)) and torch.equal(a["beta"], bias.to(torch.bfloat16))


@pytest.mark.parametrize("M", [16, 64, 4096])
def test_outputs_as_the_weights_of_the_next_product(M):
    """svla_op_gemm fetches W before the kernel ahead of it has ended, where that one lets it start early: y and dx
    taken as W right behind the call give what they give after a wait. As graphs, without the host's time between."""
    D = 1024
    a = make(M, D, x="bf16", y="bf16", seed=4)
    lhs = (torch.randn(64, D, generator=torch.Generator().manual_seed(1)) * 0.1).to(torch.bfloat16).to(DEV)
    out = torch.empty(64, M, device=DEV)
    calls = [lambda: op_layernorm(a["x"], a["gamma"], a["beta"], a["y"], 1e-5, a["mean"], a["rstd"]),
             lambda: op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"]),
             lambda: op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"], a["dgamma"],
                                           a["dbeta"])]
    for call, name in zip(calls, ("y", "dx", "dx")):
        call()
        torch.cuda.synchronize()
        want = op_gemm("f32", lhs, a[name], out, splits=1).clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
            op_gemm("f32", lhs, a[name], out, splits=1)
        for _ in range(5):
            a[name].fill_(3.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


@pytest.mark.parametrize("D", [8, 100, 768, 1100, 1283, 5000, 8200, 12288])
@pytest.mark.parametrize("value", [1e-30, 1.0, 2e19, 1e30])
def test_constant_rows_of_any_size(D, value):
    """The mean of a constant row is the value within the sum's rounding, 64 2^-24 of it, and its differences from that
    mean are no larger; where their squares are within float32, so is all that follows."""
    x = torch.full((3, D), value, device=DEV)
    y, mean, rstd = torch.empty_like(x), torch.empty(3, device=DEV), torch.empty(3, device=DEV)
    op_layernorm(x, torch.ones(D, device=DEV), None, y, 1e-5, mean, rstd)
    assert (mean.double() / value - 1).abs().max() <= 64 * 2.0 ** -24
    off = 64 * 2.0 ** -24 * value
    if off < 1e18:
        assert torch.isfinite(y).all() and torch.isfinite(rstd).all()
        assert (rstd.double() * (1e-5 ** 0.5)).max() <= 1 + 1e-5 and rstd.double().min() >= (off ** 2 + 1e-5) ** -0.5 * (1 - 1e-5)


@pytest.mark.parametrize("D", [64, 771, 2048])
@pytest.mark.parametrize("order", [(0, 1, 2), (2, 0, 1), (1, 2, 0)])
def test_parts_of_one_wider_matrix(D, order):
    """x, dy and the output as the column blocks of one buffer, in any order: their rows lie between each other's."""
    M = 33
    a = make(M, D, seed=6)
    wide = torch.full((M, 3 * D), 5.0, device=DEV)
    x, dy, out = (wide[:, k * D:(k + 1) * D] for k in order)
    x.copy_(a["x"])
    dy.copy_(a["dy"])
    op_layernorm(a["x"], a["gamma"], a["beta"], a["y"], 1e-5, a["mean"], a["rstd"])
    op_layernorm(x, a["gamma"], a["beta"], out, 1e-5)
    tol = dict(rtol=0, atol=2e-5 * float(a["y"].abs().max()))  # odd widths: other threads hold the elements
    assert torch.allclose(out, a["y"], **tol)
    op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"])
    op_layernorm_backward(dy, x, a["gamma"], a["mean"], a["rstd"], out)
    assert torch.allclose(out, a["dx"], rtol=0, atol=2e-5 * float(a["dx"].abs().max()))
    assert torch.equal(x, a["x"]) and torch.equal(dy, a["dy"])
    with pytest.raises(_abi.SvlaError):
        op_layernorm(x, a["gamma"], a["beta"], wide[:, 1 + order[0] * D:1 + order[0] * D + D] if order[0] < 2 else
                     wide[:, D + D // 2:2 * D + D // 2], 1e-5)


def test_row_counts_and_strides_at_the_end_of_32_bits():
    buf = torch.zeros(2 ** 31 + 64, dtype=torch.bfloat16, device=DEV)
    one, beta = torch.ones(1, device=DEV), torch.full((1,), 0.5, device=DEV)
    x = buf[:2 ** 31 - 100].view(-1, 1)
    op_layernorm(x, one, beta, x, 1e-5)  # a row of one element has no variance: y = beta
    assert (x[:1000] == 0.5).all() and (x[-1000:] == 0.5).all() and (x[2 ** 30:2 ** 30 + 1000] == 0.5).all()
    assert not buf[2 ** 31 - 100:].any()
    g8 = torch.ones(8, device=DEV)
    for bad, g in ((buf.view(-1, 1), one), (buf.as_strided((2, 8), (2 ** 31 + 8, 1)), g8)):
        with pytest.raises(ValueError):
            op_layernorm(bad, g, None, bad)
    # rows that lie further than 2^32 bytes apart
    far = buf.as_strided((2, 8), (2 ** 31 - 8, 1))
    v = torch.randn(2, 8, device=DEV).to(torch.bfloat16)
    far.copy_(v)
    y = torch.empty_like(v)
    op_layernorm(v, g8, None, y)
    op_layernorm(far, g8, None, far)
    assert torch.equal(far, y)


@pytest.mark.parametrize("D", [16, 51, 100, 720, 771, 1024, 2048, 12296, 16384])
def test_few_rows_in_the_backward(D):
    """One block, one cluster of 2 to 8 blocks, and the first count past it, for every number of rows a block takes."""
    units = (D + 7) // 8
    T = 1 << (units - 1).bit_length() if units <= 16 else 32
    R = 256 // T if D <= 768 else 1
    for M in sorted({1, 2, 3, R, R + 1, 2 * R, 5 * R - 1, 8 * R, 8 * R + 1}):
        check(M, D, y="bf16", seed=M)


def test_missing_arguments_are_refused():
    a = make(4, 64)
    with pytest.raises(ValueError):
        op_layernorm(a["x"], None, a["beta"], a["y"])
    with pytest.raises(ValueError):
        op_layernorm_backward(a["dy"], a["x"], None, a["mean"], a["rstd"], a["dx"])
    with pytest.raises(_abi.SvlaError):
        op_layernorm_backward(a["dy"], a["x"], a["gamma"], None, a["rstd"], a["dx"])
    with pytest.raises(ValueError):
        op_layernorm(a["x"].reshape(2, 2, 64), a["gamma"], None, a["y"].reshape(2, 2, 64))


def test_workspaces_on_a_given_stream_beside_queued_work():
    """A temporary of the workspace's size, given back while the current stream's work on it is still queued: a call on
    another stream meanwhile takes other memory, and neither result changes. (The products' split-K scratch likewise.)"""
    M, D = 3000, 768
    a = make(M, D, x="bf16", y="bf16")
    op_layernorm(a["x"], a["gamma"], a["beta"], a["y"], 1e-5, a["mean"], a["rstd"])
    bwd = lambda s: op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"], a["dgamma"],
                                          a["dbeta"], stream=s)
    gen = torch.Generator().manual_seed(3)
    lhs, w = (torch.randn(m, 4096, generator=gen).to(torch.bfloat16).to(DEV) for m in (64, 512))
    out = torch.empty(64, 512, device=DEV)
    gemm = lambda s: op_gemm("f32", lhs, w, out, splits=16, stream=s)
    lib = _abi.load()
    sizes = [int(lib.svla_op_layernorm_backward_workspace_bytes(M, D)), int(lib.svla_op_gemm_workspace_bytes(64, 512, 4096, 16))]
    assert min(sizes) > 0
    bwd(None), gemm(None)
    torch.cuda.synchronize()
    want = [t.clone() for t in (a["dx"], a["dgamma"], a["dbeta"], out)]
    side = torch.cuda.Stream()
    for call, n, outs in ((bwd, sizes[0], (a["dx"], a["dgamma"], a["dbeta"])), (gemm, sizes[1], (out,))):
        for t in outs:
            t.fill_(7.0)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # about 10 ms
        tmp = torch.empty(n, dtype=torch.uint8, device=DEV)
        kept = [tmp.fill_(k).sum(dtype=torch.int64) for k in range(1, 40)]
        del tmp
        call(side)
        torch.cuda.synchronize()
        assert [int(k) for k in kept] == [n * k for k in range(1, 40)]
    assert all(torch.equal(x, y) for x, y in zip((a["dx"], a["dgamma"], a["dbeta"], out), want))


@pytest.mark.parametrize("widths", [(768, 12288), (6400, 8192)])
def test_two_threads_with_two_widths_of_one_kernel(widths):
    """Widths that share a kernel and differ in the shared memory that it takes, in two threads at once: every call
    launches and gives what it gives alone."""
    import threading
    calls, errors, outs = 4000, [], {}
    start = threading.Barrier(2)

    def work(D, stream):
        try:
            with torch.cuda.stream(stream):
                a = make(9, D, x="bf16", y="bf16", seed=1)
                op_layernorm(a["x"], a["gamma"], a["beta"], a["y"], 1e-5, a["mean"], a["rstd"])
                start.wait(60)
                for _ in range(calls):
                    op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"], a["dgamma"], a["dbeta"])
                stream.synchronize()
                outs[D] = a
        except Exception as e:  # noqa: BLE001
            errors.append(f"{D}: {e}")

    threads = [threading.Thread(target=work, args=(D, torch.cuda.Stream())) for D in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for D in widths:
        a = outs[D]
        want = make(9, D, x="bf16", y="bf16", seed=1)
        op_layernorm_backward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], want["dx"], want["dgamma"], want["dbeta"])
        assert all(torch.equal(a[k], want[k]) for k in ("dx", "dgamma", "dbeta"))


def rows_a_block(D):
    """Rows of a block of the backward's kernel: 256 threads of as many as a row's columns take."""
    units = (D + 7) // 8
    if units <= 16:
        T = 1 << (units - 1).bit_length()
    elif D <= 768:
        T = 32
    else:
        nu = 2 if D <= 8192 else 3
        T = min(512, 32 * -(-units // (32 * nu)))
    return max(1, 256 // T)


@pytest.mark.parametrize("D", [8, 96, 769, 771, 1024, 1025, 1536, 2048, 2056, 4096, 8200])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_blocks_of_the_backward_at_every_width(D, x):
    """The full cluster of 8 blocks and the first count past it, rows of several warps and several such rows a block."""
    R = rows_a_block(D)
    need = [int(_abi.load().svla_op_layernorm_backward_workspace_bytes(m, D)) for m in (8 * R, 8 * R + 1)]
    assert need[0] == 0 and need[1] > 0
    for M in sorted({7 * R + 1, 8 * R - 1, 8 * R, 8 * R + 1, 16 * R + 1}):
        check(M, D, x=x, y="bf16", seed=M)
