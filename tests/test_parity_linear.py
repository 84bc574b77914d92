"""moe_linear and its gradients against their fp64 definition, element by element.

Tolerances: a product sum over K is accumulated in fp32 by tensor-core steps of 16 products;
each step's additions lose at most 2^-22 of the terms' magnitudes so far (an fp32 step is 2^-23,
truncation included, doubled for the alignment of the 16 products), so a sum is within
2^-22 (K / 16 + 16) sum |x||w|; the epilogue's functions are within 2^-20 (1 + |z|) and have
slopes below 1.2; an output is rounded once (half a step: finfo.eps / 2 of the value)."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from oracle import router_ref as rr

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _half_step(ref, dtype):
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps


def _within(got, ref, tol, what):
    got = got.cpu().double()
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() - tol
    assert (bad <= 0).all(), f"{what}: {int((bad > 0).sum())} of {bad.numel()} beyond, worst excess {bad.max():.3e}"


def _make(M, N, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g).to(dtype)
    w = (torch.randn((N, K), generator=g) / K ** 0.5).to(dtype)
    return g, x, w


def _forward(dev, M, N, K, dtype=BF, act="none", bias=False, residual=False, preact=False, out_dtype=None, inplace=False):
    g, x, w = _make(M, N, K, dtype, M * 7 + N * 3 + K)
    odt = out_dtype or dtype
    b = torch.randn((N,), generator=g).to(dtype) if bias else None
    res = torch.randn((M, N), generator=g).to(odt) if residual else None
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    pre = torch.full((M, N), 7.0, dtype=dtype, device=dev) if preact else None
    resd = d(res)
    # (a guard row behind the output stays as it was)
    store = torch.full((M + 1, N), 7.0, dtype=odt, device=dev)
    out = store[:M]
    if inplace:
        out.copy_(res)
        resd = out
    got = moe.moe_linear(d(x), d(w), d(b), resd, act, out=out, preact=pre)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == moe.MOE_OK
    ref, z, mag = rr.linear(x, w, b, res, act)
    acc = 2.0 ** -22 * (K / 16 + 16) * mag
    fun = 0 if act == "none" else 2.0 ** -20 * (1 + z.abs())
    _within(got, ref, 1.2 * acc + fun + 2.0 ** -23 * ref.abs() + _half_step(ref, odt), "out")
    if preact:
        _within(pre, z, acc + _half_step(z, dtype), "preact")
    assert (store[M] == 7.0).all()


# one row to several tiles; N and K beside the tile sizes; few and many K blocks
SHAPES = [(1, 1, 8), (1, 256, 7168), (2, 77, 264), (3, 130, 1032), (4, 8, 64), (5, 8, 64), (7, 33, 72), (16, 256, 2048),
          (33, 500, 200), (127, 129, 520), (128, 256, 64), (129, 257, 128), (200, 64, 4096), (300, 1000, 136),
          (513, 384, 1024), (1030, 72, 640)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_shapes(cuda_dev, M, N, K):
    _forward(cuda_dev, M, N, K)
    _forward(cuda_dev, M, N, K, HF, "none", True, True, True, F32)


@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (3, 41, 256), (40, 264, 512), (150, 41, 96), (150, 200, 3000 // 8 * 8)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
def test_linear_epilogues(cuda_dev, M, N, K, act):
    _forward(cuda_dev, M, N, K, BF, act, True, True, True)
    _forward(cuda_dev, M, N, K, HF, act, True, False, False)
    _forward(cuda_dev, M, N, K, BF, act, False, True, True, F32, inplace=True)
    _forward(cuda_dev, M, N, K, HF, act, False, True, False, inplace=True)


def test_linear_large_grid(cuda_dev):
    """More tiles than SMs (persistent CTAs run several), ragged in every dimension."""
    _forward(cuda_dev, 2500, 2050, 328, BF, "silu", True, True, True)
    _forward(cuda_dev, 2500, 2056, 328, HF, "none", True, False, True, F32)


def test_linear_nonfinite_rows_stay_apart(cuda_dev):
    for M in (4, 40, 300):
        _, x, w = _make(M, 200, 256, BF, 5)
        clean = moe.moe_linear(x.to(cuda_dev), w.to(cuda_dev))
        x[1, 7] = float("nan")
        x[2, 9] = float("inf")
        got = moe.moe_linear(x.to(cuda_dev), w.to(cuda_dev))
        assert torch.isnan(got[1]).all()
        assert not torch.isfinite(got[2]).any()
        keep = [r for r in range(M) if r not in (1, 2)]
        assert torch.equal(got[keep], clean[keep])


def _backward(dev, M, N, K, dtype=BF, act="none", ddt=None, need=(True, True, True)):
    g, x, w = _make(M, N, K, dtype, M * 5 + N * 3 + K + 1)
    ddt = ddt or dtype
    dout = (torch.randn((M, N), generator=g) * 0.5).to(ddt)
    pre = None if act == "none" else (torch.randn((M, N), generator=g) * 2).to(dtype)
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    got = moe.moe_linear_backward(d(dout), d(x), d(w), d(pre), act, need_dx=need[0], need_dw=need[1], need_dbias=need[2])
    torch.cuda.synchronize()
    assert moe.moe_device_status() == moe.MOE_OK
    refs, mags, dmags = rr.linear_backward(dout, x, w, pre, act)
    # dz is rounded to the operands' type where it is computed or comes in fp32; act' is within 2^-20 (absolute:
    # it vanishes where its terms do not) and its product with dout rounds once more
    rounded = act != "none" or ddt != dtype
    dz_err = (torch.finfo(dtype).eps / 2 if rounded else 0) + 2.0 ** -24
    act_err = 2.0 ** -20 if act != "none" else 0
    sub = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps if rounded else 0
    for name, v, ref, mag, dmag, n, needed in zip(("dx", "dw", "dbias"), got, refs, mags, dmags, (N, M, M), need):
        if not needed:
            assert v is None
            continue
        if name == "dbias":
            # a chunk of 8 to 64 rows: at most 8 rows a thread, then 8 threads; then 8 sums over up to M / 8
            # chunks, and those: 8 + 8 + M / 64 + 8 additions in a row at most
            tol = 2.0 ** -24 * (32 + M / 64) * mag + act_err * dmag
        else:
            other = x.double().abs().sum(0)[None] if name == "dw" else w.double().abs().sum(0)[None]
            tol = (2.0 ** -22 * (n / 16 + 16) + dz_err) * mag + 1.01 * act_err * dmag + sub * other
        _within(v, ref, tol + _half_step(ref, dtype), name)


@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (1, 256, 512), (5, 33, 72), (64, 8, 64), (100, 64, 256), (129, 130, 136),
                                   (300, 257, 520), (1000, 256, 1024), (70, 1000, 2048)])
def test_linear_backward_shapes(cuda_dev, M, N, K):
    _backward(cuda_dev, M, N, K)
    _backward(cuda_dev, M, N, K, HF, "silu", F32)
    _backward(cuda_dev, M, N, K, BF, "none", F32)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_backward_activations(cuda_dev, act, dtype):
    _backward(cuda_dev, 150, 200, 264, dtype, act)
    _backward(cuda_dev, 150, 201, 264, dtype, act, F32)


def test_linear_backward_parts_and_large_grid(cuda_dev):
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
        _backward(cuda_dev, 90, 96, 128, BF, "gelu", None, need)
        _backward(cuda_dev, 90, 96, 128, BF, "none", None, need)
    _backward(cuda_dev, 2100, 1100, 1800, BF, "silu")


def test_linear_gradients_are_the_differences_of_the_projection(cuda_dev):
    """d/dt <dout, linear(x + t u)> against <dx, u>, in fp32 outputs: the tensor cores' sums of bf16
    products are good to 2^-22 (K/16 + 16) of their magnitudes and dx to half a bf16 step, random over
    its elements; the step of 2^-3 of a linear map has no truncation error."""
    M, N, K = 64, 96, 128
    g, x, w = _make(M, N, K, BF, 8)
    u = (torch.randint(-4, 5, (M, K), generator=g).float() * 0.125)
    x = (x.float() * 16).round().clamp(-64, 64) / 16  # so that x +- u are exact in bf16
    dout = (torch.randn((M, N), generator=g)).to(BF)
    f = lambda v: (moe.moe_linear(v.to(BF).to(cuda_dev), w.to(cuda_dev), out_dtype=F32).cpu().double() * dout.double()).sum()  # noqa: E731
    dx, _, _ = moe.moe_linear_backward(dout.to(cuda_dev), x.to(BF).to(cuda_dev), w.to(cuda_dev))
    want = (dx.cpu().double() * u.double()).sum()
    mag = (dx.cpu().double() * u.double()).abs().sum()
    acc = 2.0 ** -22 * (K / 16 + 16) * (x.abs().double() @ w.double().abs().T * dout.double().abs()).sum()
    assert abs((f(x + u) - f(x - u)) / 2 - want) <= acc + 2.0 ** -8 * mag


def test_linear_empty_batch(cuda_dev):
    x = torch.empty((0, 64), dtype=BF, device=cuda_dev)
    w = torch.ones((8, 64), dtype=BF, device=cuda_dev)
    assert moe.moe_linear(x, w).shape == (0, 8)
    dw = torch.ones_like(w)
    _, _, db = moe.moe_linear_backward(torch.empty((0, 8), dtype=BF, device=cuda_dev), x, w, dw=dw, need_dbias=True)
    assert (dw == 0).all() and (db == 0).all()


def test_linear_is_the_same_twice_and_under_a_graph(cuda_dev):
    for M, N, K in ((1, 256, 2048), (64, 256, 4096), (600, 512, 512)):
        _, x, w = _make(M, N, K, BF, 2)
        x, w = x.to(cuda_dev), w.to(cuda_dev)
        out = torch.empty((M, N), dtype=F32, device=cuda_dev)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ws = torch.empty(moe.linear_backward_workspace_size(M, N, K), dtype=torch.uint8, device=cuda_dev)

        def step():
            moe.moe_linear(x, w, out=out)
            moe.moe_linear_backward(out, x, w, dx=dx, dw=dw, ws=ws)

        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (out, dx, dw)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in (out, dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, dx, dw), want))


def test_linear_on_another_stream(cuda_dev):
    _, x, w = _make(200, 256, 1024, BF, 3)
    x, w = x.to(cuda_dev), w.to(cuda_dev)
    want = moe.moe_linear(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_linear(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_linear_offsets_past_32_bits(cuda_dev):
    """M * N past 2^31 elements: rows at both ends against the definition."""
    M, N, K = 160_000, 14336, 64
    g, x, w = _make(64, N, K, BF, 4)
    big = torch.zeros((M, K), dtype=BF, device=cuda_dev)
    big[:32], big[-32:] = x[:32].to(cuda_dev), x[32:].to(cuda_dev)
    out = moe.moe_linear(big, w.to(cuda_dev), activation="silu")
    ref, z, mag = rr.linear(x, w, None, None, "silu")
    tol = 1.2 * 2.0 ** -22 * (K / 16 + 16) * mag + 2.0 ** -20 * (1 + z.abs()) + _half_step(ref, BF)
    _within(torch.cat([out[:32], out[-32:]]), ref, tol, "out")
    # dw and dbias of a gradient that is zero but for those rows; dx of the last
    d = torch.randn((64, N), generator=g).to(BF)
    out.zero_()
    out[:32], out[-32:] = d[:32].to(cuda_dev), d[32:].to(cuda_dev)
    dx, dw, db = moe.moe_linear_backward(out, big, w.to(cuda_dev), need_dbias=True)
    refs, mags, _ = rr.linear_backward(d, x, w)
    # (zeros add nothing: the sums hold 64 terms)
    for v, r, m, n in ((torch.cat([dx[:32], dx[-32:]]), refs[0], mags[0], N), (dw, refs[1], mags[1], M), (db, refs[2], mags[2], M)):
        _within(v, r, 2.0 ** -22 * (n / 16 + 16) * m + _half_step(r, BF), "gradient")


def test_linear_first_call_under_capture():
    """The library's first call in a process may be a captured one."""
    import subprocess
    import sys
    code = (
        "import torch\n"
        "from mixture_experts_layer_tokens_gb300 import moe\n"
        "x, w = (torch.randn(s, device='cuda').bfloat16() for s in ((300, 512), (264, 512)))\n"
        "o = torch.empty((300, 264), device='cuda', dtype=torch.bfloat16)\n"
        "dx, dw = torch.empty_like(x), torch.empty_like(w)\n"
        "l, ids, ws = torch.randn((300, 264), device='cuda'), torch.empty((300, 6), device='cuda', dtype=torch.int32), torch.empty((300, 6), device='cuda')\n"
        "dl, dn = torch.empty_like(l), torch.randn((50, 512), device='cuda').bfloat16()\n"
        "y, dy = (torch.randn((300, 512), device='cuda').bfloat16() for _ in range(2))\n"
        "wf = torch.rand((50, 6), device='cuda')\n"
        "tmp = torch.empty(1 << 24, device='cuda', dtype=torch.uint8)\n"
        "outs = [torch.empty((50, 6), device='cuda'), torch.empty_like(dn), torch.empty(512, device='cuda')]\n"
        "def step():\n"
        "    moe.moe_linear(x, w, out=o)\n"
        "    moe.moe_linear_backward(o, x, w, preact=o, activation='silu', dx=dx, dw=dw, ws=tmp)\n"
        "    moe.moe_route_grouped(l, 6, n_group=8, topk_group=3, group_top=2, topk_ids=ids, topk_weights=ws)\n"
        "    moe.moe_route_grouped_backward(ws, l, ids, dlogits=dl)\n"
        "    moe.moe_finalize_backward(dn, y, wf, 6, residual_out=y[:50], rms_weight=y[50], dy=dy, dweights=outs[0], dsum=outs[1], drms=outs[2], ws=tmp)\n"
        "all_of = [o, dx, dw, ids, ws, dl, dy] + outs\n"
        "torch.cuda.synchronize()\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    step()\n"
        "g.replay(); torch.cuda.synchronize()\n"
        "got = [t.clone() for t in all_of]\n"
        "step(); torch.cuda.synchronize()\n"
        "assert all(torch.equal(a, b) for a, b in zip(got, all_of)) and moe.moe_device_status() == 0\n"
        "print('same')\n")
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("M,N,K", [(256, 1024, 1000), (256, 5120, 512), (300, 5120, 4096), (2050, 2560, 4096), (40, 136, 4104)])
def test_linear_cuts(cuda_dev, M, N, K):
    """Sizes whose cuts differ: split K in clusters of 2, 4 and 8, pairs, a split last wave."""
    _forward(cuda_dev, M, N, K, BF, "none", True, False, False, F32)
    _backward(cuda_dev, M, N, K)


@pytest.mark.parametrize("N", [9, 31, 33, 34, 35, 62, 63, 65, 97, 126, 130, 257, 290, 319])
def test_linear_widths_beside_the_vectors(cuda_dev, N):
    """Rows that start anywhere: every parity of row and width, tiles whose last columns are few, in place."""
    for M, out_dtype in ((37, None), (133, F32), (300, None)):
        _forward(cuda_dev, M, N, 136, BF, "gelu", True, True, True, out_dtype, inplace=True)
        _forward(cuda_dev, M, N, 136, HF, "silu", False, False, True, out_dtype)
        _forward(cuda_dev, M, N, 136, BF, "none", False, True, False, out_dtype)


@pytest.mark.parametrize("M,N,K", [(3, 4100, 2056), (4, 4096, 2048), (5, 24, 512), (8, 1000, 2496), (8, 1000, 2504), (6, 33, 5000),
                                   (7, 129, 6448), (1, 4100, 8192), (2, 4100, 4160)])
def test_linear_few_rows(cuda_dev, M, N, K):
    """Both kernels for a few rows, either side of the choice."""
    _forward(cuda_dev, M, N, K, BF, "silu", True, True, True, F32)
    _forward(cuda_dev, M, N, K, HF, "none", True, False, False)
