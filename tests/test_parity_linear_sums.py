"""How accurate the sums of moe_linear and of its gradients are over long contractions, in the 2-norm
and by bounds that do not grow with the length.

The tensor core adds 16 products to its fp32 sum and truncates, which takes up to 2^-23 of the sum
at each step, always towards zero.  fp32 outputs are promoted every 512 elements (32 steps): with
random signs a run's sums grow like the root of the steps, so a run adds 2^-24.5 (the mean of half
a last place, relative) of sqrt(16 i / K) over i = 1 .. 32, 1.2e-5 / sqrt(K) of an output of size 1, and the K / 512
runs' errors, independent in sign, 9e-7 together; without the promotion one run of K / 16 steps
adds 1.2e-5 at K = 7168.  2e-6 lies between.

16-bit outputs are rounded once, by half a step of the type at most (2^-11 of the value in fp16, 2^-8 in
bf16).  Terms of one sign lose about half a last place of the growing sum at each step of 16, or two where
the hardware adds the 16 in groups: 2^-23 of the final sum a step (1.2e-7; measured 1.0e-7).  fp16 sums are left in the tensor
core for 8192 elements, 512 steps: 2^-14.  bf16 sums for 16384: 2^-13.  Longer ones are sums of such runs
with one fp32 rounding each: 122 of them at a million elements in fp16, of 2^-25 of the growing sum each, are
3.6e-6 at most, within the 8e-6 that the measured loss a step leaves of 2^-14."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SLACK = {BF: 2.0 ** -13, HF: 2.0 ** -14}


@pytest.mark.parametrize("M,N,K", [(16, 256, 4096), (64, 256, 7168), (4096, 256, 7168), (300, 5120, 4096), (520, 1032, 7168)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_fp32_outputs_are_good_to_fp32(cuda_dev, M, N, K, dtype):
    """Split and whole sums, one CTA and pairs."""
    g = torch.Generator(device=cuda_dev).manual_seed(M + N)
    x = torch.randn((M, K), generator=g, device=cuda_dev).to(dtype)
    w = (torch.randn((N, K), generator=g, device=cuda_dev) / K ** 0.5).to(dtype)
    got = moe.moe_linear(x, w, out_dtype=F32).double()
    ref = x.double() @ w.double().T
    assert moe.moe_device_status() == moe.MOE_OK
    assert (got - ref).norm() <= 2e-6 * ref.norm()


def _positive(g, *shape, dtype):
    return (torch.rand(shape, generator=g, device="cuda") * 0.5 + 0.75).to(dtype)


@pytest.mark.parametrize("C", [16384, 200_000, 1_000_000])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("P,Q", [(64, 72), (200, 264)])
def test_long_sums_of_one_sign(cuda_dev, C, dtype, P, Q):
    """Terms of one sign, where truncation adds up: dw over C tokens, a 16-bit output over K = C, dx over N = C."""
    g = torch.Generator(device=cuda_dev).manual_seed(C)
    half = torch.finfo(dtype).eps / 2
    # (outputs of about 1: in the range of either type)
    a, b = _positive(g, C, P, dtype=dtype), (_positive(g, C, Q, dtype=F32) / C).to(dtype)
    if dtype == HF:  # (1 / C is subnormal in fp16: the scale lies in both)
        a, b = (a.float() * 2.0 ** -8).to(dtype), (_positive(g, C, Q, dtype=F32) * (2.0 ** 8 / C)).to(dtype)
    ref = a.double().T @ b.double()  # [P, Q]

    def near(got, what):
        err = (got.double() - ref).abs() / ref
        assert float(err.max()) <= half + SLACK[dtype], f"{what}: {float(err.max()):.3e}"

    at, bt = a.T.contiguous(), b.T.contiguous()
    _, dw, _ = moe.moe_linear_backward(a, b, torch.zeros((P, Q), dtype=dtype, device=cuda_dev), need_dx=False)
    near(dw, "dw")
    near(moe.moe_linear(at, bt), "out")
    if C <= 1 << 21 and P % 8 == 0:
        dx, _, _ = moe.moe_linear_backward(at, torch.zeros((P, Q), dtype=dtype, device=cuda_dev), b, need_dw=False)
        near(dx, "dx")
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("C", [8192, 16384, 65536])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_long_sums_of_one_sign_in_one_piece(cuda_dev, C, dtype):
    """So many tiles that none splits its sum over CTAs: dw, and a 16-bit output."""
    P = 2048
    g = torch.Generator(device=cuda_dev).manual_seed(C + 1)
    a, b = ((_positive(g, C, P, dtype=F32) * 2.0 ** e).to(dtype) for e in (-8, 8 - C.bit_length() + 1))
    ref = a[:, :128].double().T @ b.double()
    _, dw, _ = moe.moe_linear_backward(a, b, torch.zeros((P, P), dtype=dtype, device=cuda_dev), need_dx=False)
    out = moe.moe_linear(a.T.contiguous(), b.T.contiguous())
    assert moe.moe_device_status() == moe.MOE_OK
    for got in (dw, out):
        err = (got[:128].double() - ref).abs() / ref
        assert float(err.max()) <= torch.finfo(dtype).eps / 2 + SLACK[dtype], f"{float(err.max()):.3e}"


def test_fp32_gradients_in_two_parts(cuda_dev):
    """dout in two 16-bit parts as 2M rows over x twice: dw and dx are then off by their own rounding alone, 1.7e-3
    in the 2-norm for normally distributed values in bf16; dz rounded to bf16 adds as much again (2.3e-3)."""
    M, N, K = 1024, 256, 1000
    g = torch.Generator(device=cuda_dev).manual_seed(9)
    dout, x, w = (torch.randn(s, generator=g, device=cuda_dev) for s in ((M, N), (M, K), (N, K)))
    x, w, hi = x.to(BF), w.to(BF), dout.to(BF)
    both = torch.cat([hi, (dout - hi.float()).to(BF)])
    dx, dw, _ = moe.moe_linear_backward(both, torch.cat([x, x]), w)
    dx = dx[:M].float() + dx[M:].float()
    assert moe.moe_device_status() == moe.MOE_OK
    for got, ref in ((dw, dout.double().T @ x.double()), (dx, dout.double() @ w.double())):
        assert (got.double() - ref).norm() <= 2e-3 * ref.norm()


def test_host_threads_at_once(moelib):
    """The library's first products may come from several host threads at once, each on its stream."""
    import os
    import subprocess
    import sys
    code = (
        "import threading, torch\n"
        "from mixture_experts_layer_tokens_gb300 import moe\n"
        "torch.manual_seed(0)\n"
        "shapes = [(64, 256, 4096), (300, 1000, 1024), (16, 264, 7168), (1030, 520, 512)]\n"
        "ops = [((torch.randn((m, k), device='cuda') / 8).bfloat16(), (torch.randn((n, k), device='cuda') / 8).bfloat16()) for m, n, k in shapes]\n"
        "torch.cuda.synchronize()\n"
        "outs, start = [None] * 4, threading.Barrier(4)\n"
        "def work(i):\n"
        "    s = torch.cuda.Stream()\n"
        "    start.wait()\n"
        "    with torch.cuda.stream(s):\n"
        "        for _ in range(5):\n"
        "            o = moe.moe_linear(*ops[i])\n"
        "            g = moe.moe_linear_backward(o, *ops[i])\n"
        "    s.synchronize()\n"
        "    outs[i] = [o, *g[:2]]\n"
        "ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]\n"
        "[t.start() for t in ts]; [t.join() for t in ts]\n"
        "for i in range(4):\n"
        "    o = moe.moe_linear(*ops[i])\n"
        "    g = moe.moe_linear_backward(o, *ops[i])\n"
        "    assert all(torch.equal(a, b) for a, b in zip(outs[i], [o, *g[:2]])), i\n"
        "assert moe.moe_device_status() == 0\n"
        "print('same')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_first_promoted_products_under_capture(moelib):
    """The first product that promotes its sums may be a captured one."""
    import os
    import subprocess
    import sys
    code = (
        "import torch\n"
        "from mixture_experts_layer_tokens_gb300 import moe\n"
        "x, w = torch.randn((300, 4096), device='cuda').bfloat16(), torch.randn((264, 4096), device='cuda').bfloat16()\n"
        "a, b = torch.rand((300000, 64), device='cuda').bfloat16(), torch.rand((300000, 72), device='cuda').bfloat16()\n"
        "o, dw, v = torch.empty((300, 264), device='cuda'), torch.empty_like(b[:64]), torch.zeros_like(b[:64])\n"
        "ws = torch.empty(1 << 26, device='cuda', dtype=torch.uint8)\n"
        "def step():\n"
        "    moe.moe_linear(x, w, out=o)\n"
        "    moe.moe_linear_backward(a, b, v, dw=dw, ws=ws, need_dx=False)\n"
        "torch.cuda.synchronize()\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    step()\n"
        "g.replay(); torch.cuda.synchronize()\n"
        "got = [o.clone(), dw.clone()]\n"
        "step(); torch.cuda.synchronize()\n"
        "assert torch.equal(got[0], o) and torch.equal(got[1], dw) and moe.moe_device_status() == 0\n"
        "assert (o.double() - x.double() @ w.double().T).norm() <= 2e-6 * o.double().norm()\n"
        "print('same')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
