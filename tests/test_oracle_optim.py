"""Pins of the optimiser's and LayerNorm's oracle against things other than
itself: closed forms, torch's AdamW in float64, exhaustive codes, the mean over
all random bits, and differences."""
import numpy as np
import pytest

from oracle import optim as oo

torch = pytest.importorskip("torch")


def test_first_step_moves_by_the_learning_rate():
    g = np.array([3.0, -0.02, 1e-6])
    p, m, v = oo.adamw(np.zeros(3), g, np.zeros(3), np.zeros(3), 0.1, 0.9, 0.999, 1e-12, 0.0, 1)
    assert np.allclose(p, -0.1 * np.sign(g), rtol=1e-5)
    assert np.allclose(m, 0.1 * g) and np.allclose(v, 1e-3 * g * g)


def test_matches_torch_adamw_in_float64():
    rng = np.random.default_rng(3)
    p = rng.standard_normal(50)
    t = torch.tensor(p.copy(), requires_grad=True)
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.8, 0.95), eps=1e-7, weight_decay=0.1, foreach=False)
    m = v = np.zeros(50)
    for step in range(1, 7):
        g = rng.standard_normal(50)
        t.grad = torch.tensor(g)
        norm = float(torch.nn.utils.clip_grad_norm_([t], 2.0))
        assert abs(norm - oo.grad_norm([g[:20], g[20:]])) < 1e-12
        opt.step()
        p, m, v = oo.adamw(p, g, m, v, 1e-2, 0.8, 0.95, 1e-7, 0.1, step, c=oo.clip_factor(norm, 2.0))
        assert np.allclose(p, t.detach().numpy(), rtol=1e-12, atol=1e-14), step


def test_decay_flag_and_float32_rounding():
    p, m, v = oo.adamw([2.0], [0.0], [0.0], [0.0], 0.5, 0.9, 0.99, 1e-8, 0.1, 4, decay=True)
    assert p[0] == 2.0 * 0.95 and oo.adamw([2.0], [0.0], [0.0], [0.0], 0.5, 0.9, 0.99, 1e-8, 0.1, 4, decay=False)[0][0] == 2
    rng = np.random.default_rng(1)
    a = [rng.standard_normal(1000).astype(np.float32) for _ in range(3)]
    x = [abs(rng.standard_normal(1000)).astype(np.float32)]
    lo, hi = (oo.adamw(a[0], a[1], a[2], x[0], 1e-3, 0.9, 0.999, 1e-8, 0.01, 7, dtype=d) for d in (np.float32, np.float64))
    for s, e in zip(lo, hi):
        assert s.dtype == np.float32 and np.abs(s - e).max() < 1e-6


@pytest.mark.parametrize("fmt,dtype", [(oo.E4M3, torch.float8_e4m3fn), (oo.E5M2, torch.float8_e5m2)])
def test_codes_are_the_torch_types_and_round_trip(fmt, dtype):
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(dtype).double().numpy()
    mine = oo.decode(codes, fmt)
    ok = np.isfinite(ref)
    assert np.array_equal(mine[ok], ref[ok])
    # values on the grid keep their code whatever the random bits
    digits, bias, top, _ = fmt
    normal = codes[(codes & 0x7F) >= (1 << digits)]
    normal = normal[np.isfinite(ref[normal])]
    x = ref[normal]
    x = x[np.abs(x) < 2.0 ** (top + 1)]
    for u in (0, 1, 40000, 65535):
        got, scale = oo.encode(x, np.full(x.size, u), fmt, False)
        assert scale[0] == 1.0 and np.array_equal(oo.decode(got, fmt), x)


@pytest.mark.parametrize("fmt,keep", [(oo.E4M3, False), (oo.E5M2, True)])
def test_rounding_is_right_in_the_mean(fmt, keep):
    """Over all 65536 draws the decoded mean is the value, to one draw of the spacing."""
    digits, _, top, _ = fmt
    u = np.arange(65536)
    for x in (1.0, 1.03, 1.9999, 3.7 * 2.0 ** -3, 0.777 * 2.0 ** (top - 9)):
        big = 2.0 ** top
        got = np.empty(65536)
        for s in range(0, 65536, BLOCK_FILL):
            block = np.full(BLOCK_FILL + 1, x)
            block[0] = big  # fixes the scale at 1
            codes, scale = oo.encode(block, np.concatenate([[0], u[s:s + BLOCK_FILL]]), fmt, keep)
            got[s:s + BLOCK_FILL] = oo.decode(codes, fmt)[1:]
        spacing = 2.0 ** (np.floor(np.log2(x)) - digits)
        assert scale[0] == 1.0 and abs(got.mean() - x) <= spacing / 65536, (fmt, x)


BLOCK_FILL = 128


def test_small_and_special_values():
    x = np.zeros(256)
    codes, scale = oo.encode(x, np.full(256, 65535), oo.E5M2, True)
    assert not codes.any() and scale[0] == 0
    x[0], x[1], x[2] = 1.0, 1e-30, np.nan
    codes, scale = oo.encode(x, np.zeros(256, int), oo.E5M2, True)
    assert scale[0] == 2.0 ** -14 and oo.decode(codes, oo.E5M2)[1] == 2.0 ** -14 and codes[2] == 0x7F and codes[3] == 0
    x[2] = -np.inf
    codes, scale = oo.encode(x, np.full(256, 65535), oo.E4M3, False)
    assert scale[0] == 2.0 ** -7 and codes[1] == 0 and codes[2] == 0x7F
    # the next block has its own scale; float32's smallest magnitudes keep a legal scale
    y = np.concatenate([np.full(256, 3.0), np.full(44, 2.0 ** -149)])
    codes, scale = oo.encode(y, np.zeros(300, int), oo.E5M2, True)
    assert scale.size == 2 and scale[0] == 2.0 ** -13 and scale[1] == 2.0 ** -112
    assert (oo.decode(codes, oo.E5M2)[256:] == 2.0 ** -14).all()


def test_random_bits_follow_the_published_generator():
    """Element k: half k % 8 of the draw with counter (k / 8, step, tensor)."""
    from oracle.philox import philox4x32_10
    r = oo.random16(40, 5, 9, (7 << 32) | 3)
    w = philox4x32_10(([2], [0], [9], [5]), (3, 7))
    assert [int(r[16 + 2 * i]) | int(r[17 + 2 * i]) << 16 for i in range(4)] == [int(x[0]) for x in w]


def test_nearest_rounding_would_freeze_v():
    """Why the rounding is stochastic: v's mean over many elements follows its float32 course."""
    rng = np.random.default_rng(0)
    n, steps = 2048, 200
    v = codes = np.zeros(n)
    exact = np.zeros(n)
    nearest = np.zeros(n)
    for step in range(1, steps + 1):
        g = rng.standard_normal(n)
        exact = 0.99 * exact + 0.01 * g * g
        v = 0.99 * v + 0.01 * g * g
        codes, scale = oo.encode(v, oo.random16(n, 0, step, 1), oo.E5M2, True)
        v = oo.decode(codes, oo.E5M2) * np.repeat(scale, 256)
        nearest = 0.99 * nearest + 0.01 * g * g
        codes, scale = oo.encode(nearest, np.full(n, 32768), oo.E5M2, True)
        nearest = oo.decode(codes, oo.E5M2) * np.repeat(scale, 256)
    assert abs(v.mean() / exact.mean() - 1) < 0.05
    assert nearest.mean() / exact.mean() < 0.8


def test_layernorm_against_differences_and_closed_forms():
    rng = np.random.default_rng(2)
    x, gamma, beta, dy = (rng.standard_normal(s) for s in ((4, 9), 9, 9, (4, 9)))
    y, mean, rstd = oo.layernorm(x, gamma, beta, 1e-5)
    assert np.allclose(((y - beta) / gamma).mean(1), 0) and np.allclose((((y - beta) / gamma) ** 2).mean(1), 1, atol=1e-4)
    assert np.allclose(oo.layernorm(x + 5.0, gamma, beta, 1e-5)[0], y)
    dx, dg, db = oo.layernorm_backward(dy, x, gamma, mean, rstd)
    loss = lambda a, g, b: float((oo.layernorm(a, g, b, 1e-5)[0] * dy).sum())
    h = 1e-5
    for i in range(4):
        for j in range(9):
            e = np.zeros((4, 9))
            e[i, j] = h
            assert abs((loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(9):
        e = np.zeros(9)
        e[j] = h
        assert abs((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h) - dg[j]) < 1e-7
        assert abs((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h) - db[j]) < 1e-7
    one = oo.layernorm(np.array([[3.0]]), np.array([2.0]), np.array([0.5]), 1e-5)
    assert one[0][0, 0] == 0.5
