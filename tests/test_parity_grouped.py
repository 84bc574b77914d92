"""moe_grouped_linear and its gradients against their fp64 definitions, element by element.

Tolerances: a sum over C is accumulated in fp32 by tensor-core steps of 16 products; each step's additions lose at most
2^-22 of the terms' magnitudes so far (an fp32 step is 2^-23, truncation included, doubled for the alignment of the 16
products), so a sum is within 2^-22 (C / 16 + 16) of the sum of magnitudes; an output is rounded once (half a step:
finfo.eps / 2 of the value)."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from oracle import experts_ref as er

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _tol(ref, mag, C, dtype, rel=1.0):
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) * 1.01 + fi.smallest_normal * fi.eps + mag * rel * 2 ** -22 * (C / 16 + 16)


def _within(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() - tol
    assert (bad <= 0).all(), f"{what}: {int((bad > 0).sum())} of {bad.numel()} beyond, worst excess {bad.max():.3e}"


class Problem:
    """Rows counts of the groups; `over` more sorted rows belong to none."""

    def __init__(self, counts, N, K, top_k=1, dtype=BF, x_rows="sorted", rows="sorted", d_rows="sorted", over=0, seed=0):
        g = torch.Generator().manual_seed(seed * 77 + sum(counts) * 5 + N * 3 + K)
        self.S, self.E, self.N, self.K, self.top_k = sum(counts) + over, len(counts), N, K, top_k
        self.dtype, self.x_rows, self.rows, self.d_rows, self.over = dtype, x_rows, rows, d_rows, over
        self.offsets = torch.tensor([0] + list(counts)).cumsum(0).to(torch.int32)
        self.slots = torch.randperm(self.S, generator=g).to(torch.int32)
        T = self.S // top_k
        self.x = torch.randn((T if x_rows == "token" else self.S, K), generator=g).to(dtype)
        self.dout = (torch.randn((T if d_rows == "token" else self.S, N), generator=g)).to(dtype)
        self.w = (torch.randn((self.E, N, K), generator=g) / K ** 0.5).to(dtype)
        if over:  # rows of no group: nothing may read them into a result
            end = int(self.offsets[-1])
            for t, order in ((self.x, x_rows), (self.dout, d_rows)):
                if order != "token":
                    t[self.slots[end:].long() if order == "slot" else slice(end, None)] = float("nan")
            if x_rows == "sorted" and rows == "sorted" and d_rows == "sorted":
                self.slots[end:] = 1 << 30  # (not read)

    def index(self):
        return self.slots if "slot" in (self.rows, self.x_rows, self.d_rows) or "token" in (self.x_rows, self.d_rows) else None

    def dev(self, dev):
        sl = self.index()
        return [t.to(dev) for t in (self.x, self.w, self.offsets)] + [None if sl is None else sl.to(dev)]

    def forward(self, dev, **kw):
        x, w, o, sl = self.dev(dev)
        self.store = torch.full((self.S + 1, self.N), 7.0, dtype=self.dtype, device=dev)
        return moe.moe_grouped_linear(x, w, o, sl, self.top_k, x_rows=self.x_rows, out_rows=self.rows,
                                      out=self.store[:self.S], **kw)

    def check_forward(self, out):
        ref, mag = er.grouped_linear(self.x, self.w, self.offsets, self.index(), self.top_k, self.x_rows, self.rows)
        some = ~torch.isnan(ref[:, 0]) if self.N else None
        out = out.cpu()
        _within(out[some], ref[some], _tol(ref, mag, self.K, self.dtype)[some], "out")
        assert bool((out[~some] == 7).all()) and bool((self.store[self.S] == 7).all())

    def backward(self, dev, wdt=None, accumulate=False, **kw):
        x, w, o, sl = self.dev(dev)
        wdt = wdt or self.dtype
        self.dx_store = torch.full((self.S + 1, self.K), 7.0, dtype=self.dtype, device=dev)
        self.dw_store = torch.full((self.E + 1, self.N, self.K), 7.0, dtype=wdt, device=dev)
        if accumulate:
            g = torch.Generator().manual_seed(4)
            self.old = (torch.randn((self.E, self.N, self.K), generator=g) * 3).to(wdt)
            self.dw_store[:self.E] = self.old.to(dev)
        return moe.moe_grouped_linear_backward(self.dout.to(dev), x, w, o, sl, self.top_k, dout_rows=self.d_rows,
                                               x_rows=self.x_rows, dx_rows=self.rows, dx=self.dx_store[:self.S],
                                               dw=self.dw_store[:self.E], accumulate=accumulate, **kw)

    def check_backward(self, dx, dw, accumulate=False):
        ref, mag, wref, wmag = er.grouped_linear_backward(self.dout, self.x, self.w, self.offsets, self.index(), self.top_k,
                                                          self.d_rows, self.x_rows, self.rows)
        some = ~torch.isnan(ref[:, 0])
        dx = dx.cpu()
        _within(dx[some], ref[some], _tol(ref, mag, self.N, self.dtype)[some], "dx")
        assert bool((dx[~some] == 7).all()) and bool((self.dx_store[self.S] == 7).all())
        if accumulate:
            wref, wmag = wref + self.old.double(), wmag + self.old.double().abs()
        most = max(int((self.offsets[1:] - self.offsets[:-1]).max()), 1)
        _within(dw, wref, _tol(wref, wmag, most, dw.dtype), "dw")
        assert bool((self.dw_store[self.E] == 7).all())
        if not accumulate:
            empty = (self.offsets[1:] == self.offsets[:-1]).nonzero().flatten()
            assert bool((dw[empty.to(dw.device)] == 0).all())


ORDERS = [("sorted", "sorted", "sorted"), ("token", "sorted", "slot"), ("slot", "slot", "token"), ("sorted", "slot", "sorted")]

# (group sizes, N, K): one row, empty groups, tiles that end everywhere, one group with all, many small ones
SHAPES = [
    ([1], 8, 8),
    ([0, 1, 0, 0, 3], 16, 72),
    ([64, 128, 0, 256], 256, 128),
    ([63, 65, 1, 127, 129, 255], 136, 200),
    ([300, 0, 17, 481, 2], 520, 264),
    ([0, 0, 700, 0], 264, 64),
    ([2] * 40 + [0] * 30 + [5] * 9, 128, 320),
    ([33] * 6 + [31] * 3 + [32], 72, 24),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("orders", ORDERS)
@pytest.mark.parametrize("shape", SHAPES)
def test_grouped(cuda_dev, shape, orders, dtype):
    counts, N, K = shape
    x_rows, rows, d_rows = orders
    S = sum(counts)
    top_k = 2 if S % 2 == 0 and "token" in orders else 1
    p = Problem(counts, N, K, top_k, dtype, x_rows, rows, d_rows)
    p.check_forward(p.forward(cuda_dev))
    wdt = F32 if (N + len(orders[0])) % 3 else dtype
    p.check_backward(*p.backward(cuda_dev, wdt))
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("orders", ORDERS)
@pytest.mark.parametrize("counts,N,K", [([30, 0, 50], 264, 4104), ([200, 130], 72, 1600), ([30, 1, 49], 4104, 136),
                                        ([3], 520, 8200), ([700, 300], 16, 3080)])
def test_few_tiles(cuda_dev, counts, N, K, orders):
    """Tiles so few, and sums so long, that several CTAs share a tile's sum (forward, dx or both): right, and the same bits
    each time."""
    x_rows, rows, d_rows = orders
    p = Problem(counts, N, K, 1, HF, x_rows, rows, d_rows)
    out = p.forward(cuda_dev)
    p.check_forward(out)
    first = out.clone()
    for _ in range(3):
        assert torch.equal(p.forward(cuda_dev), first)
    dx, dw = p.backward(cuda_dev)
    p.check_backward(dx, dw)
    first = dx.clone()
    assert torch.equal(p.backward(cuda_dev)[0], first)
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("orders", ORDERS)
def test_rows_of_no_group(cuda_dev, orders):
    """Sorted rows behind the last group, NaN here, are neither used nor written."""
    x_rows, rows, d_rows = orders
    if "token" in orders:
        x_rows, d_rows = ("slot" if o == "token" else o for o in (x_rows, d_rows))
    for counts in ([70, 0, 33], [5, 6, 7], [0, 0, 0]):
        p = Problem(counts, 136, 72, 1, BF, x_rows, rows, d_rows, over=13)
        p.check_forward(p.forward(cuda_dev))
        p.check_backward(*p.backward(cuda_dev))
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("dtype,wdt", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("counts", [[70, 0, 200, 1], [600, 3]])
def test_accumulated_gradient(cuda_dev, counts, dtype, wdt):
    p = Problem(counts, 264, 136, 1, dtype)
    dx, dw = p.backward(cuda_dev, wdt, accumulate=True)
    p.check_backward(dx, dw, accumulate=True)


@pytest.mark.parametrize("counts,N,K,dtype,wdt", [
    ([40, 3], 8, 8264, HF, HF),        # forward sums over 8192 in fp16
    ([40, 3], 16, 16456, BF, BF),      # and over 16384 in bf16
    ([20, 33], 8264, 16, HF, HF),      # dx
    ([20, 300], 16456, 16, BF, BF),
    ([8300, 0, 45], 16, 24, HF, HF),   # dw
    ([16500, 700], 8, 16, BF, F32),
    ([1030, 511, 513, 512], 72, 264, BF, F32),
])
def test_long_sums(cuda_dev, counts, N, K, dtype, wdt):
    p = Problem(counts, N, K, 1, dtype)
    p.check_forward(p.forward(cuda_dev))
    p.check_backward(*p.backward(cuda_dev, wdt))


@pytest.mark.parametrize("counts,N,K,over", [([2000, 0, 40], 2056, 2072, 0), ([1000, 1045], 2072, 2056, 9)])
def test_many_rows_off_128_bytes(cuda_dev, counts, N, K, over):
    """Sorted rows that start on no multiple of 128 bytes, enough of them that they are moved to such a pitch first."""
    p = Problem(counts, N, K, 1, BF, over=over)
    assert moe.grouped_linear_workspace_size(p.S, p.E, N, K) == (p.S * 2112 * 2 + 255) // 256 * 256
    p.check_forward(p.forward(cuda_dev))
    p.check_backward(*p.backward(cuda_dev, F32))


@pytest.mark.parametrize("dtype,wdt", [(BF, BF), (HF, F32)])
@pytest.mark.parametrize("N,K", [(8, 8), (264, 1000), (72, 136)])
def test_gradient_of_experts_without_rows(cuda_dev, N, K, dtype, wdt):
    """Zeros in every place and nowhere else, whatever the sizes leave over."""
    for counts in ([0, 3, 0], [0, 0, 0, 0, 9], [1, 0]):
        p = Problem(counts, N, K, 1, dtype)
        p.check_backward(*p.backward(cuda_dev, wdt))


def test_sums_of_one_sign(cuda_dev):
    """Terms of one sign, where truncation would add up: 32 steps of 16 terms lose at most 2^-23 of the part so far
    each, 16.5 2^-23 of a part of 512, and 40 parts are added in fp32 with a half step of the sum so far each, 20.5
    2^-24 in all: within 27 2^-23 < 3.3e-6."""
    p = Problem([20000], 64, 64, 1, BF)
    p.x, p.dout = torch.ones_like(p.x) * 1.0078125, torch.ones_like(p.dout) * 1.0078125
    _, dw = p.backward(cuda_dev, F32, need_dx=True)
    exact = 20000 * 1.0078125 ** 2
    assert ((dw.double().cpu() - exact).abs() <= 3.3e-6 * exact).all()


def test_not_a_number_stays(cuda_dev):
    """A row with a NaN or an infinity changes its row of out and dx, and its expert's dw, alone."""
    p = Problem([70, 60, 0, 130], 136, 200, 1, BF)
    clean, (cdx, cdw) = p.forward(cuda_dev).clone(), [t.clone() for t in p.backward(cuda_dev)]
    p.x[69, 5], p.x[130, 0], p.dout[69, 3] = float("nan"), float("inf"), float("nan")
    out, (dx, dw) = p.forward(cuda_dev), p.backward(cuda_dev)
    keep = torch.ones(p.S, dtype=torch.bool, device=cuda_dev)
    keep[69] = keep[130] = False
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[69]).all()
    keep[130] = True
    assert torch.equal(dx[keep], cdx[keep]) and torch.isnan(dx[69]).all()
    assert torch.equal(dw[1], cdw[1]) and torch.equal(dw[2], cdw[2]) and torch.isnan(dw[0]).any()
    assert not torch.isfinite(dw[3]).all()


@pytest.mark.parametrize("rows", ["sorted", "slot"])
@pytest.mark.parametrize("counts", [[40, 25], [5, 7, 0, 1], [200, 300]])
def test_slots_out_of_range_are_left_out(cuda_dev, counts, rows):
    """A slot outside [0, S) is recorded, its rows are not written and have no share in dw; the others are as they were."""
    p = Problem(counts, 136, 72, 1, BF, "slot", rows, "slot")
    good, bad = p.slots.clone(), [3, sum(counts) - 1]
    ref = p.forward(cuda_dev).clone()
    dref, _ = (t.clone() for t in p.backward(cuda_dev))
    p.slots[bad[0]], p.slots[bad[1]] = -1, p.S
    out = p.forward(cuda_dev)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG and moe.moe_device_status() == moe.MOE_OK
    dx, dw = p.backward(cuda_dev)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    left = good[bad].long().to(cuda_dev) if rows == "slot" else torch.tensor(bad, device=cuda_dev)
    keep = torch.ones(p.S, dtype=torch.bool, device=cuda_dev)
    keep[left] = False
    assert torch.equal(out[keep], ref[keep]) and bool((out[left] == 7).all())
    assert torch.equal(dx[keep], dref[keep]) and bool((dx[left] == 7).all())
    p.slots = good
    p.dout[good[bad].long()] = 0
    _, want = p.backward(cuda_dev)
    assert torch.equal(dw, want) and moe.moe_device_status() == moe.MOE_OK


def test_a_bad_slot_stops_nothing_else(cuda_dev):
    """A bad slot is recorded while the kernels' waits are long, and stays recorded through later calls: neither makes a
    wait give up."""
    g = torch.Generator(device=cuda_dev).manual_seed(0)
    S, E, N, K = 16384, 8, 4096, 4096
    x = torch.randn((S, K), generator=g, device=cuda_dev).to(BF)
    w = (torch.randn((E, N, K), generator=g, device=cuda_dev) / 64).to(BF)
    o = torch.arange(E + 1, dtype=torch.int32, device=cuda_dev) * (S // E)
    slots = torch.randperm(S, generator=g, device=cuda_dev).to(torch.int32)
    kw = dict(x_rows="slot", out_rows="slot")
    want = moe.moe_grouped_linear(x, w, o, slots, **kw)
    bad = slots.clone()
    bad[5], bad[S - 7] = S + 3, -4
    keep = torch.ones(S, dtype=torch.bool, device=cuda_dev)
    keep[slots[[5, S - 7]].long()] = False
    for _ in range(2):
        assert torch.equal(moe.moe_grouped_linear(x, w, o, bad, **kw)[keep], want[keep])
    assert torch.equal(moe.moe_grouped_linear(x, w, o, slots, **kw), want)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG and moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("offsets", [[0, 30, 20, 70], [-5, 30, 40, 70], [0, 30, 40, 90]])
def test_offsets_out_of_order_are_recorded(cuda_dev, offsets):
    """Groups that do not fit are cut to the rows there are, and the call says so; the rows of a sound group are right."""
    p = Problem([30, 10, 30], 136, 72, 1, BF, "slot", "slot", "slot")
    want, (dx, dw) = p.forward(cuda_dev).clone(), [t.clone() for t in p.backward(cuda_dev)]
    p.offsets = torch.tensor(offsets, dtype=torch.int32)
    out = p.forward(cuda_dev)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG and bool((p.store[p.S] == 7).all())
    dx2, dw2 = p.backward(cuda_dev)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    assert bool((p.dx_store[p.S] == 7).all()) and bool((p.dw_store[p.E] == 7).all())
    rows = p.slots[:30 if offsets[0] == 0 and offsets[2] == 40 else 20].long().to(cuda_dev)
    assert torch.equal(out[rows], want[rows]) and torch.equal(dx2[rows], dx[rows])


def test_parts_of_the_gradients(cuda_dev):
    """dx or dw alone are what both together are; without rows dw is zeros, or what it was."""
    p = Problem([70, 0, 33], 136, 72, 1, BF, "slot", "slot", "slot")
    dx, dw = p.backward(cuda_dev)
    x, w, o, sl = p.dev(cuda_dev)
    kw = dict(dout_rows="slot", x_rows="slot", dx_rows="slot")
    only, none = moe.moe_grouped_linear_backward(p.dout.to(cuda_dev), None, w, o, sl, need_dw=False, **kw)
    assert none is None and torch.equal(only, dx)
    none, only = moe.moe_grouped_linear_backward(p.dout.to(cuda_dev), x, w, o, sl, need_dx=False, **kw)
    assert none is None and torch.equal(only, dw)
    zero = torch.zeros(4, dtype=torch.int32, device=cuda_dev)
    dx, dw = moe.moe_grouped_linear_backward(p.dout[:0].to(cuda_dev), x[:0], w, zero)
    assert dx.shape == (0, 72) and bool((dw == 0).all())
    kept = torch.ones_like(dw)
    moe.moe_grouped_linear_backward(p.dout[:0].to(cuda_dev), x[:0], w, zero, dw=kept, accumulate=True)
    assert bool((kept == 1).all())
    assert moe.moe_grouped_linear(x[:0], w, zero).shape == (0, 136)


def test_same_bits_and_capture(cuda_dev):
    """The same inputs give the same bits; a captured call follows its inputs, the groups among them."""
    p = Problem([300, 5, 0, 129], 264, 520, 2, BF, "token", "slot", "slot")
    x, w, o, sl = p.dev(cuda_dev)
    d = p.dout.to(cuda_dev)
    S, E, N, K = p.S, p.E, p.N, p.K
    ws = torch.full((moe.grouped_linear_workspace_size(S, E, N, K, "token"),), 255, dtype=torch.uint8, device=cuda_dev)
    wb = torch.full((moe.grouped_linear_backward_workspace_size(S, E, N, K, "slot", "token"),), 255, dtype=torch.uint8,
                    device=cuda_dev)
    p.store = torch.full((S + 1, N), 7.0, dtype=BF, device=cuda_dev)
    p.dx_store = torch.full((S + 1, K), 7.0, dtype=BF, device=cuda_dev)
    p.dw_store = torch.full((E + 1, N, K), 7.0, dtype=BF, device=cuda_dev)

    def call(stream=None):
        out = moe.moe_grouped_linear(x, w, o, sl, 2, x_rows="token", out_rows="slot", out=p.store[:S], ws=ws, stream=stream)
        return (out, *moe.moe_grouped_linear_backward(d, x, w, o, sl, 2, dout_rows="slot", x_rows="token", dx_rows="slot",
                                                      dx=p.dx_store[:S], dw=p.dw_store[:E], ws=wb, stream=stream))

    first = [t.clone() for t in call()]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    q = Problem([0, 250, 184, 0], 264, 520, 2, BF, "token", "slot", "slot", seed=8)
    assert q.S == S
    for t, v in ((x, q.x), (w, q.w), (o, q.offsets), (sl, q.slots), (d, q.dout)):
        t.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    q.store, q.dx_store, q.dw_store = p.store, p.dx_store, p.dw_store
    q.check_forward(p.store[:S])
    q.check_backward(p.dx_store[:S], p.dw_store[:E])


def test_gradients_by_differences(cuda_dev):
    """<dout, out(x + h) - out(x - h)> / 2h against dx, and the same for dw, on values that 16 bits hold exactly, so
    that the differences of the linear map are exact but for the roundings of out (half a step each)."""
    p = Problem([20, 13], 24, 40, 1, HF)
    x, w, o, _ = p.dev(cuda_dev)
    dx, dw = p.backward(cuda_dev)
    d = p.dout.to(cuda_dev).double()
    for t, grad in ((x, dx), (w, dw)):
        flat, g = t.view(-1), grad.double().view(-1)
        for i in (0, 17, flat.numel() - 1):
            old = flat[i].clone()
            flat[i] = old + 1
            up, hi = moe.moe_grouped_linear(x, w, o).double(), flat[i].double()
            flat[i] = old - 1
            down, lo = moe.moe_grouped_linear(x, w, o).double(), flat[i].double()
            flat[i] = old
            got = float((d * (up - down)).sum() / (hi - lo))
            moved = (up - down).abs() > 0
            tol = float((d.abs() * moved * (up.abs() + down.abs()) * 2 ** -11).sum() / (hi - lo)) + abs(float(g[i])) * 2 ** -10
            assert abs(got - float(g[i])) <= tol + 1e-3, (got, float(g[i]), tol)


@pytest.mark.parametrize("S,E,N,K", [(2, 1024, 8, 16), (4096, 1024, 64, 72)])
def test_many_experts(cuda_dev, S, E, N, K):
    g = torch.Generator().manual_seed(0)
    counts = torch.bincount(torch.randint(0, E, (S,), generator=g), minlength=E).tolist()
    p = Problem(counts, N, K)
    p.check_forward(p.forward(cuda_dev))
    p.check_backward(*p.backward(cuda_dev, F32))


def test_with_moe_align(cuda_dev):
    """The groups of moe_align, expert by expert against plain products."""
    g = torch.Generator().manual_seed(1)
    T, top_k, E, N, K = 300, 4, 16, 256, 128
    ids = torch.rand((T, E), generator=g).argsort(1)[:, :top_k].to(torch.int32)
    x, w = torch.randn((T, K), generator=g).to(BF), (torch.randn((E, N, K), generator=g) / K ** 0.5).to(BF)
    al = moe.moe_align(ids.to(cuda_dev), E)
    out = moe.moe_grouped_linear(x.to(cuda_dev), w.to(cuda_dev), al.expert_offsets, al.sorted_slot, top_k, x_rows="token",
                                 out_rows="slot")
    ref = torch.einsum("tnk,tk->tn", w.double()[ids.view(-1).long()], x.double().repeat_interleave(top_k, 0))
    mag = torch.einsum("tnk,tk->tn", w.double().abs()[ids.view(-1).long()], x.double().abs().repeat_interleave(top_k, 0))
    _within(out, ref, _tol(ref, mag, K, BF), "out")
