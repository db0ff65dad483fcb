"""Refusals of the training operators: arguments that are wrong are rejected on
the host, before any CUDA work (so these run without a GPU)."""
import ctypes

import pytest

from vision_language_action_b200 import _abi

ARG, SHAPE = _abi.SVLA_ERR_ARG, _abi.SVLA_ERR_SHAPE
F32, BF16 = _abi.TYPE_F32, _abi.TYPE_BF16
BASE = 1 << 40  # addresses that are never read


def tensor(at=0, n=1000, bits=32, **kw):
    """One tensor whose ranges lie apart from those of every other `at`."""
    t = _abi.SvlaAdamwTensor()
    room = BASE + at * (1 << 30)
    for i, name in enumerate(("param", "grad", "m", "v", "copy", "m_scale", "v_scale")):
        if bits == 8 or "scale" not in name:
            setattr(t, name, room + i * (1 << 26))
    t.n, t.decay = n, 1
    for k, x in kw.items():
        setattr(t, k, x)
    return t


def args(**kw):
    a = _abi.SvlaAdamwArgs()
    a.state_bits, a.lr, a.beta1, a.beta2, a.eps, a.weight_decay, a.step = 32, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1
    for k, x in kw.items():
        setattr(a, k, x)
    return a


def adamw(ts, a, ws=None, ws_bytes=0, norm=None, n=None):
    lib = _abi.load()
    arr = (_abi.SvlaAdamwTensor * max(1, len(ts)))(*ts)
    st = lib.svla_op_adamw(arr, len(ts) if n is None else n, ctypes.byref(a) if a is not None else None, ws, ws_bytes,
                           norm, None)
    return st, lib.svla_last_error(None).decode()


@pytest.mark.parametrize("kw,status", [
    (dict(param_type=2), ARG), (dict(grad_type=-1), ARG), (dict(state_bits=16), ARG), (dict(lr=-1.0), ARG),
    (dict(lr=float("nan")), ARG), (dict(lr=float("inf")), ARG), (dict(beta1=1.0), ARG), (dict(beta1=-0.1), ARG),
    (dict(beta2=1.0), ARG), (dict(beta2=float("nan")), ARG), (dict(eps=0.0), ARG), (dict(eps=1e-60), ARG),
    (dict(eps=1e60), ARG), (dict(weight_decay=-0.1), ARG), (dict(max_norm=-1.0), ARG),
    (dict(max_norm=float("nan")), ARG), (dict(step=0), ARG), (dict(step=-5), ARG),
])
def test_adamw_settings(kw, status):
    assert adamw([tensor()], args(**kw))[0] == status


@pytest.mark.parametrize("bits,kw,status", [
    (32, dict(n=-1), SHAPE), (32, dict(n=(1 << 40) + 1), SHAPE), (32, dict(param=None), ARG), (32, dict(grad=None), ARG),
    (32, dict(m=None), ARG), (32, dict(v=None), ARG), (8, dict(m_scale=None), ARG), (8, dict(v_scale=None), ARG),
    (32, dict(param=BASE + 2), ARG), (32, dict(m=BASE + (1 << 27) + 1), ARG), (32, dict(copy=BASE + (1 << 28) + 1), ARG),
    (8, dict(m_scale=BASE + (5 << 26) + 2), ARG),
])
def test_adamw_tensors(bits, kw, status):
    st, msg = adamw([tensor(0, bits=bits), tensor(1, bits=bits, **kw)], args(state_bits=bits))
    assert st == status and "tensor 1" in msg


def test_adamw_null_count_and_workspace():
    assert adamw([], None)[0] == ARG
    assert adamw([tensor()], args(), n=-1)[0] == ARG
    lib = _abi.load()
    assert lib.svla_op_adamw(None, 1, ctypes.byref(args()), None, 0, None, None) == ARG
    need = lib.svla_op_adamw_workspace_bytes(1)
    assert need > 0 and lib.svla_op_adamw_workspace_bytes(401) == 2 * need == lib.svla_op_adamw_workspace_bytes(800)
    assert lib.svla_op_adamw_workspace_bytes(-1) == 0 and lib.svla_op_adamw_workspace_bytes(0) == need
    clip = args(max_norm=1.0)
    assert adamw([tensor()], clip)[0] == ARG
    assert adamw([tensor()], clip, BASE - 4096 * 16, need - 1)[0] == ARG
    assert adamw([tensor()], clip, BASE - 4096 * 16 + 4, need)[0] == ARG
    # the empty list is a step over nothing, and so are empty tensors' pointers
    assert adamw([], args())[0] == _abi.SVLA_OK


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("name", ["param", "m", "v", "copy", "grad", "m_scale"])
def test_adamw_overlaps(name, bits):
    """Memory that is written may not be listed twice, nor read through another name."""
    if name == "m_scale" and bits == 32:
        pytest.skip("no scales")
    a, b = tensor(0, bits=bits), tensor(1, bits=bits)
    # the last element of the first tensor's parameters
    setattr(b, name, a.param + 4 * 999 if name not in ("m", "v") or bits == 32 else a.param + 3999)
    st, msg = adamw([a, b], args(state_bits=bits))
    assert st == ARG and "overlaps" in msg
    assert adamw([a, a], args(state_bits=bits))[0] == ARG
    # a tensor's own moments may not share memory either
    c = tensor(0, bits=bits)
    c.v = c.m
    assert adamw([c], args(state_bits=bits))[0] == ARG


def test_adamw_norm_and_workspace_overlaps():
    a = tensor()
    need = _abi.load().svla_op_adamw_workspace_bytes(1)
    assert adamw([a], args(max_norm=1.0), a.m, need)[0] == ARG
    assert adamw([a], args(max_norm=1.0), BASE - 4096 * 16, need, a.param)[0] == ARG
    assert adamw([a], args(max_norm=1.0), BASE - 4096 * 16, need, a.grad + 8)[0] == ARG


def ln(**kw):
    """svla_op_layernorm with ranges that lie apart, and the arguments given in place of the usual ones."""
    a = dict(x=BASE, xt=F32, ldx=64, g=BASE + (1 << 24), b=BASE + (2 << 24), wt=F32, M=10, D=64, eps=1e-5,
             y=BASE + (3 << 24), yt=F32, ldy=64, mean=BASE + (4 << 24), rstd=BASE + (5 << 24))
    a.update(kw)
    return _abi.load().svla_op_layernorm(a["x"], a["xt"], a["ldx"], a["g"], a["b"], a["wt"], a["M"], a["D"], a["eps"],
                                         a["y"], a["yt"], a["ldy"], a["mean"], a["rstd"], None)


def ln_bwd(**kw):
    a = dict(dy=BASE, yt=F32, lddy=64, x=BASE + (1 << 24), xt=F32, ldx=64, g=BASE + (2 << 24), wt=F32,
             mean=BASE + (3 << 24), rstd=BASE + (4 << 24), M=1000, D=64, dx=BASE + (5 << 24), lddx=64,
             dg=BASE + (6 << 24), db=BASE + (7 << 24), ws=BASE + (8 << 24), n=1 << 23)
    a.update(kw)
    return _abi.load().svla_op_layernorm_backward(
        a["dy"], a["yt"], a["lddy"], a["x"], a["xt"], a["ldx"], a["g"], a["wt"], a["mean"], a["rstd"], a["M"], a["D"],
        a["dx"], a["lddx"], a["dg"], a["db"], a["ws"], a["n"], None)


COMMON = [
    (dict(xt=2), ARG), (dict(yt=-1), ARG), (dict(wt=7), ARG), (dict(M=-1), SHAPE), (dict(D=0), SHAPE),
    (dict(D=16385, ldx=1 << 15), SHAPE), (dict(ldx=63), SHAPE), (dict(g=None), ARG), (dict(x=None), ARG),
    (dict(x=BASE + 2), ARG), (dict(g=BASE + (1 << 24) + 2), ARG),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(ldy=63), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(y=None), ARG),
    (dict(y=BASE + (3 << 24) + 1), ARG), (dict(mean=BASE + (4 << 24) + 2), ARG),
    # overlaps: y in x but not x itself, y over the weights or the statistics, the statistics over an input
    (dict(y=BASE + 64 * 4), ARG), (dict(y=BASE, ldy=65), ARG), (dict(y=BASE, yt=BF16), ARG),
    (dict(y=BASE + (1 << 24) - 2000), ARG), (dict(b=BASE + (3 << 24)), ARG), (dict(mean=BASE + (3 << 24) + 4), ARG),
    (dict(rstd=BASE + 8), ARG), (dict(mean=BASE + (5 << 24) + 36), ARG), (dict(mean=BASE + (1 << 24) + 4), ARG),
])
def test_layernorm_refusals(kw, status):
    assert ln(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(lddy=63), SHAPE), (dict(lddx=63), SHAPE), (dict(dy=None), ARG), (dict(dx=None), ARG), (dict(mean=None), ARG),
    (dict(rstd=None), ARG), (dict(dg=BASE + (6 << 24) + 2), ARG), (dict(ws=None), ARG), (dict(n=1000), ARG),
    (dict(ws=BASE + (8 << 24) + 2), ARG),
    (dict(dx=BASE + 4 * 64), ARG), (dict(dx=BASE + (1 << 24), lddx=72), ARG), (dict(dx=BASE + (2 << 24)), ARG),
    (dict(dx=BASE + (3 << 24)), ARG), (dict(dg=BASE + (7 << 24) + 4), ARG), (dict(db=BASE + 400), ARG),
    (dict(dg=BASE + (1 << 24)), ARG), (dict(ws=BASE + (5 << 24) + 64), ARG), (dict(db=BASE + (2 << 24) + 8), ARG),
    (dict(dg=BASE + (8 << 24) + 16), ARG),
])
def test_layernorm_backward_refusals(kw, status):
    assert ln_bwd(**kw) == status


def test_layernorm_workspace_sizes():
    lib = _abi.load()
    f = lib.svla_op_layernorm_backward_workspace_bytes
    assert f(0, 64) == f(10, 0) == f(-3, 64) == f(10, 16385) == 0
    assert f(1, 64) == 0  # one block writes the gradients itself
    assert f(1 << 20, 768) % (2 * 768 * 4) == 0 and f(1 << 20, 768) == f(1 << 24, 768) > 0
    # no rows: nothing to do, and the pointers are not looked at
    assert ln(M=0, x=None, y=None) == _abi.SVLA_OK


def test_train_update_null_and_missing_handle():
    lib = _abi.load()
    p = ctypes.c_void_p(64)
    assert lib.svla_train_update(None, p, p, p, p, None, None, ctypes.byref(args()), None, None) == ARG
    assert lib.svla_train_weights(None, p, None) == ARG
    assert lib.svla_train_scale_elems(None) == 0


def test_python_face_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    from vision_language_action_b200 import runtime as rt
    x, g = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError):
        rt.op_layernorm(x, g, None, torch.empty_like(x))
    with pytest.raises(ValueError):
        rt.op_layernorm_backward(x, x, g, torch.zeros(4), torch.zeros(4), torch.empty_like(x))
    with pytest.raises(ValueError):
        rt.AdamW([x])
    with pytest.raises(ValueError):
        rt.AdamW([])


class FakeStream:
    cuda_stream = 77


@pytest.fixture
def given_stream(monkeypatch):
    """Streams without a GPU: yields (stream, made), the list of (bytes of a tensor made, the stream current then)."""
    import contextlib
    torch = pytest.importorskip("torch")
    now, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    def record(make):
        def made_by(*size, **kw):
            t = make(*size, **dict(kw, device="cpu"))
            made.append((t.numel() * t.element_size(), now[0]))
            return t
        return made_by

    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, record(getattr(torch, name)))
    yield FakeStream(), made


def test_workspaces_come_from_the_pool_of_the_stream_they_are_used_on(given_stream, monkeypatch):
    """A block that another stream's tensor gave back may still be in use there: the current stream's pool is not
    asked for a workspace of a call on a stream given."""
    import torch
    from vision_language_action_b200 import runtime as rt
    stream, made = given_stream
    assert rt._scratch(0, "cpu", stream) is None and not made
    rt._scratch(100, "cpu", stream), rt._scratch(50, "cpu", None)
    assert made == [(100, stream), (50, None)]
    # the product's split-K scratch, through a library that does nothing
    del made[:]
    calls = []

    class Lib:
        def svla_op_gemm_workspace_bytes(self, *a):
            return 4096

        def svla_op_gemm(self, *a):
            calls.append(a)
            return 0

    monkeypatch.setattr(_abi, "load", Lib)
    monkeypatch.setattr(rt, "_ptr", lambda t: None if t is None else t.data_ptr())
    a = torch.ones(4, 64)
    rt.op_gemm("f32", a, a, torch.ones(4, 4), splits=4, stream=stream)
    assert made == [(4096, stream)] and calls[0][-1].value == stream.cuda_stream


class AnyLib:
    """A library whose every function does nothing and returns `value`."""

    def __init__(self, value=0):
        self.value, self.calls = value, []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 12 if name.endswith("_elems") else self.value
        return call


def handle_without_gpu(rt, lib):
    import types
    m = rt.SmolVLA.__new__(rt.SmolVLA)
    m.lib, m.h, m.device, m.action_dim, m.asm = lib, 1, 0, 8, (4, 2)
    m.cfg = types.SimpleNamespace(p_layers=2, p_kv_heads=1, head_dim=4, p_width=6)
    return m


def test_outputs_come_from_the_pool_of_the_stream_that_writes_them(given_stream, monkeypatch):
    """Every output that a call on a stream given allocates itself, likewise; the caller's stream is told to the
    allocator."""
    import torch
    from vision_language_action_b200 import runtime as rt
    stream, made = given_stream
    told = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: told.append(s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(rt, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(rt, "_vec", lambda t, *a: t.data_ptr())
    lib = AnyLib()
    monkeypatch.setattr(_abi, "load", lambda: lib)
    m = handle_without_gpu(rt, lib)
    z = torch.ones
    f, pad, kv = z(2, 3, 8), z(2, 5), z(4)
    calls = [
        (lambda: m.new_kv_cache(2, 5, stream=stream), 1), (lambda: m.prefill(f, pad, stream=stream), 1),
        (lambda: m.denoise(kv, pad, f, 4, trace=True, stream=stream), 2),
        (lambda: m.denoise_prefix(kv, pad, f, 4, z(2, 1, 8), trace=True, stream=stream), 2),
        (lambda: m.sample(f, pad, 3, 3, 4, return_noise=True, stream=stream), 3),
        (lambda: m.assemble_prefix(z(2, 1, 16, 4), z(2, 5, 6), z(2, 5), z(2, 3), stream=stream), 2),
        (lambda: m.train_step(kv, pad, f, f, z(2), stream=stream), 2), (lambda: m.train_weights(stream=stream), 1),
        (lambda: rt.op_quantize_affine8(z(8, 64), stream=stream), 2)]
    for call, n in calls:
        del made[:], told[:]
        call()
        assert [s for _, s in made] == [stream] * n and told == ["current"] * n
    m.h = None


def test_handle_calls_take_the_current_stream_of_the_handles_device(monkeypatch):
    """Whatever the current device: another device's stream does not order the handle's work."""
    torch = pytest.importorskip("torch")
    import types
    from vision_language_action_b200 import runtime as rt
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=(device, "s")))
    monkeypatch.setattr(ctypes, "c_void_p", lambda x: x)
    monkeypatch.setattr(rt, "_ptr", lambda t: None if t is None else 8)
    monkeypatch.setattr(rt, "_vec", lambda *a: 8)
    monkeypatch.setattr(rt, "_new", lambda stream, shape, dtype, device: torch.empty(shape, dtype=dtype))
    lib = AnyLib()
    m = handle_without_gpu(rt, lib)
    m.device = 3
    z = torch.ones
    f, pad, kv = z(2, 3, 8), z(2, 5), z(4)
    for call in (lambda: m.prefill(f, pad), lambda: m.denoise(kv, pad, f, 4),
                 lambda: m.denoise_prefix(kv, pad, f, 4, z(2, 1, 8)), lambda: m.sample(f, pad, 3, 3, 4),
                 lambda: m.assemble_prefix(z(2, 1, 16, 4), z(2, 5, 6), z(2, 5), z(2, 3)),
                 lambda: m.train_step(kv, pad, f, f, z(2)), lambda: m.train_weights(),
                 lambda: m.train_update(f, f, (f, f, None, None), 1), lambda: m.device_status()):
        call()
        assert lib.calls[-1][1][-1] == (3, "s"), lib.calls[-1]
    m.h = None


def test_adamw_scalars_on_the_device():
    """grad_norm, step_device and lr_device: aligned to their types, and none in memory that the step writes."""
    a, room = tensor(), BASE - 4096 * 16
    need = _abi.load().svla_op_adamw_workspace_bytes(1)
    for bad in (1, 2, 3):
        st, msg = adamw([a], args(max_norm=1.0), room, need, room - 64 + bad)
        assert st == ARG and "aligned" in msg
    for bad in (4, 1):
        for kw in (dict(step_device=room - 128 + bad), dict(lr_device=room - 128 + bad)):
            st, msg = adamw([a], args(**kw))
            assert st == ARG and "aligned" in msg
    for inside in (a.param, a.m + 8, a.v, a.copy):
        for kw in (dict(step_device=inside), dict(lr_device=inside)):
            st, msg = adamw([a], args(**kw))
            assert st == ARG and "overlaps" in msg
    for kw in (dict(step_device=room), dict(lr_device=room + need - 8), dict(lr_device=room - 64)):
        st, msg = adamw([a], args(max_norm=1.0, **kw), room, need, room - 60)
        assert st == ARG and "overlaps" in msg
