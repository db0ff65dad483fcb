"""Weights that the call before has written: the matrix of a product, its int8 codes and the gains of a norm may be the
output of any operator right before on the stream. Each pair runs as a graph, without the host's time between the two,
and gives bit for bit what it gives with a wait between them."""
import pytest

torch = pytest.importorskip("torch")

from vision_language_action_b200 import _abi  # noqa: E402
from vision_language_action_b200 import runtime as rt  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"
BF = torch.bfloat16


def rand(*shape, dtype=BF, seed=0, scale=1.0):
    gen = torch.Generator().manual_seed(seed + sum(shape))
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(DEV)


def rmsnorm_writes_w(N):
    x, y, lhs, out = rand(N, 960, dtype=torch.float32), rand(N, 960), rand(64, 960), rand(64, N, dtype=torch.float32)
    g = rand(960, seed=1)
    return lambda: rt.op_rmsnorm(x, g, y), y, lambda: rt.op_gemm("f32", lhs, y, out, splits=1), out


def gemm_writes_w(N):
    a, b, c, lhs, out = rand(N, 512), rand(960, 512), rand(N, 960), rand(64, 960, seed=2), rand(64, N, dtype=torch.float32)
    return (lambda: rt.op_gemm("bf16", a, b, c, splits=1), c, lambda: rt.op_gemm("f32", lhs, c, out, splits=1), out)


def attention_writes_w(N):
    q, k, v, o = rand(1, N, 960), rand(1, 177, 320), rand(1, 177, 320, seed=3), rand(1, N, 960)
    lhs, out = rand(64, 960, seed=4), rand(64, N, dtype=torch.float32)
    return (lambda: rt.op_attention(q, k, v, o, 15, 5, 64), o, lambda: rt.op_gemm("f32", lhs, o[0], out, splits=1), out)


def gemm_writes_the_gain(N):
    a, b, c = rand(1, 512), rand(960, 512), rand(1, 960)
    x, y = rand(N, 960, dtype=torch.float32), rand(N, 960)
    return lambda: rt.op_gemm("bf16", a, b, c, splits=1), c, lambda: rt.op_rmsnorm(x, c[0], y), y


def adamw_writes_the_gain(N):
    p, grad, copy = rand(960, dtype=torch.float32), rand(960, dtype=torch.float32), rand(960)
    x, y = rand(N, 960, dtype=torch.float32), rand(N, 960)
    opt = rt.AdamW([p], lr=0.0, weight_decay=0.0, copies=[copy])  # the same step at every call
    return lambda: opt.step([grad]), copy, lambda: rt.op_rmsnorm(x, copy, y), y


def quantiser_writes_codes(N):
    lib = _abi.load()
    w, lhs, out = rand(N, 960), rand(64, 960, seed=5), rand(64, N, dtype=torch.float32)
    q, ab = rt.op_quantize_affine8(w)

    def quantise():
        _abi.check(lib.svla_op_quantize_affine8(w.data_ptr(), 960, N, 960, q.data_ptr(), 960, ab.data_ptr(),
                                                torch.cuda.current_stream().cuda_stream))
    return quantise, q, lambda: rt.op_gemm_w8("f32", lhs, q, ab, out), out


def gemm_writes_the_gain_of_codes(N):
    a, b, c = rand(1, 512), rand(960, 512), rand(1, 960)
    q, ab = rt.op_quantize_affine8(rand(N, 960))
    lhs, out = rand(64, 960, seed=6), rand(64, N, dtype=torch.float32)
    return lambda: rt.op_gemm("bf16", a, b, c, splits=1), c, lambda: rt.op_gemm_w8("f32", lhs, q, ab, out, gain=c[0]), out


@pytest.mark.parametrize("N", [16, 64, 4096])
@pytest.mark.parametrize("pair", [rmsnorm_writes_w, gemm_writes_w, attention_writes_w, gemm_writes_the_gain,
                                  adamw_writes_the_gain, quantiser_writes_codes, gemm_writes_the_gain_of_codes])
def test_what_the_call_before_wrote(pair, N):
    write, weights, use, out = pair(N)
    write()
    torch.cuda.synchronize()
    use()
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        write()
        use()
    for _ in range(5):
        weights.fill_(3)
        out.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("epilogue", ["f32", "bf16", "add_f32", "silu_bf16"])
def test_weights_said_to_be_ready(epilogue):
    """The flag changes when W may be fetched, not the product."""
    lib, epi = _abi.load(), {"f32": 0, "bf16": 1, "add_f32": 2, "silu_bf16": 3}[epilogue]
    a, w = rand(50, 960), rand(720, 960)
    outs = [torch.ones(50, 720, dtype=torch.float32 if "f32" in epilogue else BF, device=DEV) for _ in range(2)]
    for flag, c in zip((0, _abi.GEMM_W_READY), outs):
        _abi.check(lib.svla_op_gemm(epi | flag, a.data_ptr(), 960, w.data_ptr(), 960, 50, 720, 960, c.data_ptr(), 720, None, 1,
                                    None, 0, None, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(*outs) and not (outs[0] == 1).all()


def test_an_unknown_epilogue_is_refused_with_the_flag_too():
    p = 4096
    for epi in (4 | _abi.GEMM_W_READY, 0x200, -1):
        assert _abi.load().svla_op_gemm(epi, p, 64, p, 64, 4, 4, 64, p, 4, None, 0, None, 0, None, None) == _abi.SVLA_ERR_ARG
