"""Layer norm on the GPU against fp64, element by element within the bounds of
layer_reference, at widths on both sides of every layout the kernels choose (a row per
warp, a row per CTA, rows longer than the registers of a CTA)."""
import pytest
import torch

import layer_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NONFINITE = 4


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from manifold_constrained_hyper_token_b200 import build
    build.build()
    import manifold_constrained_hyper_token_b200 as m
    return m


def _case(T, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    x = (n(T, C) * (torch.rand(T, 1, generator=g) * 3 + 0.1) + n(T, 1)).to(dtype)
    return x, 1 + 0.3 * n(C), 0.3 * n(C), n(T, C).to(dtype)


SHAPES = [(1, 8), (3, 16), (1, 256), (9, 264), (130, 512), (17, 1000), (5, 1024), (33, 1032),
          (7, 2056), (300, 4096), (4, 4104), (2, 7168), (301, 7168), (3, 8200), (2, 16384),
          (3, 16392), (2, 32776), (70, 40000), (1, 100000)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C", SHAPES)
def test_norm(mhc, T, C, dtype):
    x, w, b, _ = _case(T, C, dtype, T + C)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bias in (b, None):
        y = mhc.mhc_layer_norm(x.cuda(), w.cuda(), None if bias is None else b.cuda(),
                               dev_status=st)
        R.assert_within(y, R.norm(x, w, bias, 1e-6), R.norm_bound(x, w, bias, 1e-6, dtype), "y")
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C", SHAPES + [(5000, 64), (1999, 1024), (700, 2048), (401, 12288)])
def test_norm_backward(mhc, T, C, dtype):
    x, w, _, gy = _case(T, C, dtype, T + C)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mhc.mhc_layer_norm_backward(x.cuda(), w.cuda(), gy.cuda(), dev_status=st)
    ref, bound = R.norm_grad(x, w, gy, 1e-6), R.norm_grad_bound(x, w, gy, 1e-6, dtype)
    for g, r, d, name in zip(got, ref, bound, ("grad_x", "grad_weight", "grad_bias")):
        R.assert_within(g, r, d, name)
    assert int(st.item()) == 0


@pytest.mark.parametrize("T,C", [(2368, 1032), (2369, 520), (2400, 2048), (2501, 1024),
                                 (2501, 1032), (2369, 4104), (2369, 7168), (2369, 8192),
                                 (2369, 8200)])
def test_many_rows(mhc, T, C):
    """From 2368 bf16 rows on (16 to an SM) two rows go through a CTA or warp at a time: an odd
    last row, one to eight warps to a row, a row that is not finite beside one that is, and rows
    before and behind the output, which keep their bytes."""
    x, w, b, _ = _case(T, C, BF16, T + C)
    xd, wd, bd = x.cuda(), w.cuda(), b.cuda()
    ref, bound = R.norm(x, w, b, 1e-6), R.norm_bound(x, w, b, 1e-6, BF16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(2):
        y = torch.full((T + 2, C), 7.0, dtype=BF16, device="cuda")
        mhc.mhc_layer_norm(xd, wd, bd, out=y[1:-1], dev_status=st)
        assert int(st.item()) == 0
        assert bool((y[0] == 7).all()) and bool((y[-1] == 7).all())
        assert first is None or torch.equal(first, y)
        first = y
    R.assert_within(y[1:-1], ref, bound, "y")
    R.assert_within(mhc.mhc_layer_norm(xd, wd), R.norm(x, w, None, 1e-6),
                    R.norm_bound(x, w, None, 1e-6, BF16), "y without bias")
    for bad in (T - 1, T - 2, 0):
        spoilt = xd.clone()
        spoilt[bad, C - 1] = float("nan")
        st.zero_()
        got = mhc.mhc_layer_norm(spoilt, wd, bd, dev_status=st)
        assert int(st.item()) == NONFINITE
        keep = [t for t in range(T) if t != bad]
        assert torch.equal(got[keep], y[1:-1][keep])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C", [(4, 64), (3, 2048), (2, 40000)])
def test_rows_far_from_zero(mhc, T, C, dtype):
    """Mean 300 times the deviation: the variance is taken about the mean."""
    g = torch.Generator().manual_seed(C)
    x = (300 + torch.randn(T, C, generator=g)).to(dtype)
    w, gy = torch.ones(C), torch.randn(T, C, generator=g).to(dtype)
    y = mhc.mhc_layer_norm(x.cuda(), w.cuda())
    R.assert_within(y, R.norm(x, w, None, 1e-6), R.norm_bound(x, w, None, 1e-6, dtype), "y")
    got = mhc.mhc_layer_norm_backward(x.cuda(), w.cuda(), gy.cuda())
    for a, r, d, n in zip(got, R.norm_grad(x, w, gy, 1e-6),
                          R.norm_grad_bound(x, w, gy, 1e-6, dtype), ("gx", "gw", "gb")):
        R.assert_within(a, r, d, n)


@pytest.mark.parametrize("C", [64, 2048, 40000])
def test_constant_rows(mhc, C):
    """A constant row has no deviation: y is the bias, and grad_x the centred a / sqrt(eps)."""
    x = torch.full((3, C), 2.0)
    w, b = torch.full((C,), 1.5), torch.linspace(-1, 1, C)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = mhc.mhc_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=1e-4, dev_status=st)
    assert torch.equal(y.cpu(), b.expand(3, C)) and int(st.item()) == 0
    mhc.mhc_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=0.0, dev_status=st)
    assert int(st.item()) == NONFINITE


# a row per warp, per CTA, beyond the registers; pairs of rows (2368 bf16 rows and more), odd
CLOSE = [(3, 72), (5, 264), (2, 520), (3, 1032), (2, 4104), (3, 7168), (2, 14344), (3, 16392),
         (2369, 520), (2501, 1032), (2369, 7168)]


@pytest.mark.parametrize("dtype,value", [(BF16, 3.0), (BF16, 7.0), (BF16, 100.0), (BF16, -100.5),
                                         (F32, 7.0), (F32, 100.0), (F32, 100.1), (F32, 0.3)])
@pytest.mark.parametrize("T,C", CLOSE)
def test_rows_of_one_value(mhc, T, C, dtype, value):
    """The mean of equal values is that value, whatever C is: y is the bias and grad_weight
    zero to the bit although s is 1000, and without eps the row is reported."""
    x = torch.full((T, C), value, dtype=dtype)
    g = torch.Generator().manual_seed(C)
    w, b = 1 + torch.rand(C, generator=g), torch.linspace(-1, 1, C)
    gy = torch.randn(T, C, generator=g).to(dtype)
    xd, wd, bd, gd = x.cuda(), w.cuda(), b.cuda(), gy.cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = mhc.mhc_layer_norm(xd, wd, bd, dev_status=st)
    assert torch.equal(y.cpu(), b.to(dtype).expand(T, C))
    gx, gw, _ = mhc.mhc_layer_norm_backward(xd, wd, gd, dev_status=st)
    assert int(st.item()) == 0 and not bool(gw.any())
    keep = slice(T - 3 if T > 3 else 0, T)
    R.assert_within(gx[keep], R.norm_grad(x[keep], w, gy[keep], 1e-6)[0],
                    R.norm_grad_bound(x[keep], w, gy[keep], 1e-6, dtype)[0], "grad_x")
    for call in (lambda: mhc.mhc_layer_norm(xd, wd, bd, eps=0.0, dev_status=st),
                 lambda: mhc.mhc_layer_norm_backward(xd, wd, gd, eps=0.0, dev_status=st)):
        st.zero_()
        call()
        assert int(st.item()) == NONFINITE


@pytest.mark.parametrize("dtype,value", [(BF16, 7.0), (BF16, 100.0), (F32, 100.0), (F32, 1000.1)])
@pytest.mark.parametrize("T,C", CLOSE)
def test_rows_of_nearly_one_value(mhc, T, C, dtype, value):
    """One value in 50 a step of its type away, another value in each row.  The mean is rounded
    once, u |mean|, which s (up to 1000) carries into every xh; the rounding also adds
    (u mean)^2 to the variance, half of (s u mean)^2 of s.  All else is relative to xh: 64 u for
    the variance's sum as elsewhere, 8 u for the square root, the difference and the product."""
    g = torch.Generator().manual_seed(T + C)
    x = (value * (1 + torch.arange(T) / T)).to(dtype)[:, None].repeat(1, C)
    step = torch.finfo(dtype).eps * x.abs()
    x = torch.where(torch.rand(T, C, generator=g) < 0.02, (x + step).to(dtype), x)
    w, b = 1 + torch.rand(C, generator=g), torch.linspace(-1, 1, C)
    y = mhc.mhc_layer_norm(x.cuda(), w.cuda(), b.cuda())
    xd = x.double()
    m = xd.mean(1, keepdim=True)
    s = 1 / torch.sqrt(((xd - m) ** 2).mean(1, keepdim=True) + 1e-6)
    xh = (xd - m) * s
    dm = 1.01 * R.U * s * m.abs()
    dxh = dm + (72 * R.U + dm * dm) * xh.abs()
    ref = R.norm(x, w, b, 1e-6)
    bound = w.double() * dxh + 4 * R.U * (ref.abs() + b.double().abs())
    R.assert_within(y, ref, bound + R.HALF_STEP[dtype] * (ref.abs() + bound), "y")
    # backward: the same xh in grad_weight, and in grad_x beside its own sums (64 u each)
    gy = torch.randn(T, C, generator=g).to(dtype)
    gx, gw, gb = mhc.mhc_layer_norm_backward(x.cuda(), w.cuda(), gy.cuda())
    rx, rw, rb = R.norm_grad(x, w, gy, 1e-6)
    a = gy.double() * w.double()
    c1, c2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    dc1 = 64 * R.U * a.abs().mean(1, keepdim=True)
    dc2 = (64 * R.U * (a * xh).abs() + a.abs() * dxh).mean(1, keepdim=True)
    bx = s * (dc1 + xh.abs() * dc2 + c2.abs() * dxh
              + (72 * R.U + dm * dm) * (a.abs() + c1.abs() + (xh * c2).abs()))
    R.assert_within(gx, rx, bx + R.HALF_STEP[dtype] * (rx.abs() + bx), "grad_x")
    ga = gy.double().abs()
    R.assert_within(gw, rw, (ga * dxh).sum(0) + (T + 16) * R.U * (ga * xh.abs()).sum(0), "grad_w")
    R.assert_within(gb, rb, (T + 16) * R.U * ga.sum(0), "grad_b")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C", [64, 1032, 40000])
def test_nonfinite_rows_stay_alone(mhc, C, dtype, bad):
    x, w, b, gy = _case(5, C, dtype, C)
    x[2, C // 2] = bad
    keep = [0, 1, 3, 4]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = mhc.mhc_layer_norm(x.cuda(), w.cuda(), b.cuda(), dev_status=st).cpu()
    assert int(st.item()) == NONFINITE
    R.assert_within(y[keep], R.norm(x[keep], w, b, 1e-6),
                    R.norm_bound(x[keep], w, b, 1e-6, dtype), "y")
    st.zero_()
    gx = mhc.mhc_layer_norm_backward(x.cuda(), w.cuda(), gy.cuda(), dev_status=st)[0].cpu()
    assert int(st.item()) == NONFINITE
    R.assert_within(gx[keep], R.norm_grad(x[keep], w, gy[keep], 1e-6)[0],
                    R.norm_grad_bound(x[keep], w, gy[keep], 1e-6, dtype)[0], "grad_x")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C", [(5, 64), (5, 1032), (2500, 1024), (2500, 1032), (5, 40000)])
def test_squares_beyond_fp32_are_reported(mhc, T, C, dtype):
    """Deviations of 2^70 have squares that fp32 cannot hold; 2^40 fits."""
    x, w, b, gy = _case(T, C, dtype, C)
    xd, wd, bd, gd = x.cuda(), w.cuda(), b.cuda(), gy.cuda()
    for scale, want in ((2.0 ** 40, 0), (2.0 ** 70, NONFINITE)):
        big = xd.clone()
        big[T - 2] *= scale
        st = torch.zeros(2, dtype=torch.int32, device="cuda")
        y = mhc.mhc_layer_norm(big, wd, bd, dev_status=st[:1]).cpu()
        mhc.mhc_layer_norm_backward(big, wd, gd, dev_status=st[1:])
        assert st.tolist() == [want, want]
        keep = [t for t in range(T) if want == 0 or t != T - 2]
        xs = big.cpu()[keep]
        R.assert_within(y[keep], R.norm(xs, w, b, 1e-6), R.norm_bound(xs, w, b, 1e-6, dtype), "y")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C", [(5, 1024), (5, 7168), (2501, 7168), (5, 40000)])
def test_sums_beyond_fp32_are_reported(mhc, T, C, dtype):
    """A row of 1e36 has a finite mean and no deviation, but its sum leaves fp32: it is reported
    and stays alone."""
    x, w, b, gy = _case(T, C, dtype, C)
    x[T - 2] = 1e36
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = mhc.mhc_layer_norm(x.cuda(), w.cuda(), b.cuda(), dev_status=st[:1]).cpu()
    mhc.mhc_layer_norm_backward(x.cuda(), w.cuda(), gy.cuda(), dev_status=st[1:])
    assert st.tolist() == [NONFINITE, NONFINITE]
    keep = [t for t in range(T) if t != T - 2]
    R.assert_within(y[keep], R.norm(x[keep], w, b, 1e-6),
                    R.norm_bound(x[keep], w, b, 1e-6, dtype), "y")


@pytest.mark.parametrize("T,C", [(1000, 64), (777, 7168), (70, 40000)])
def test_repeats_bit_for_bit_and_writes_nothing_else(mhc, T, C):
    x, w, b, gy = _case(T, C, BF16, 3)
    xd, wd, bd, gd = x.cuda(), w.cuda(), b.cuda(), gy.cuda()
    n = mhc.mhc_layer_norm_backward_workspace_size(T, C, BF16)
    first = None
    for fill in (0, 255):
        # outputs inside larger buffers: the rows around them keep their bytes
        y = torch.full((T + 2, C), 7.0, dtype=BF16, device="cuda")
        gx = y.clone()
        gwb = torch.full((4, C), 7.0, device="cuda")
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
        mhc.mhc_layer_norm(xd, wd, bd, out=y[1:-1])
        mhc.mhc_layer_norm_backward(xd, wd, gd, out=(gx[1:-1], gwb[1], gwb[2]), workspace=ws[:n])
        for t in (y, gx, gwb):
            assert bool((t[0] == 7).all()) and bool((t[-1] == 7).all())
        assert bool((ws[n:] == fill).all())
        out = [t.cpu() for t in (y, gx, gwb)]
        assert first is None or all(torch.equal(a, c) for a, c in zip(first, out))
        first = out


def test_other_stream_and_graph(mhc):
    """The call runs on the stream it is given; captured calls replay on new inputs."""
    T, C = 600, 1024
    x, w, b, gy = (t.cuda() for t in _case(T, C, BF16, 5))
    want = mhc.mhc_layer_norm(x, w, b), *mhc.mhc_layer_norm_backward(x, w, gy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mhc.mhc_layer_norm(x, w, b, stream=s), *mhc.mhc_layer_norm_backward(x, w, gy, stream=s)
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    xs, gs = torch.zeros_like(x), torch.zeros_like(gy)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = mhc.mhc_layer_norm(xs, w, b)
        grads = mhc.mhc_layer_norm_backward(xs, w, gs)
    for _ in range(2):
        xs.copy_(x)
        gs.copy_(gy)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, (y, *grads)))


def test_largest_offsets(mhc):
    """More than 2^31 elements: the last rows are addressed in 64 bits."""
    T, C = 70000, 32768
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 15 GB")
    x = torch.zeros(T, C, dtype=BF16, device="cuda")
    g = torch.Generator().manual_seed(0)
    last = torch.randn(4, C, generator=g).to(BF16)
    x[-4:] = last.cuda()
    w, b = torch.ones(C), torch.zeros(C)
    y = mhc.mhc_layer_norm(x, w.cuda(), b.cuda())
    R.assert_within(y[-4:], R.norm(last, w, b, 1e-6), R.norm_bound(last, w, b, 1e-6, BF16), "y")
    assert bool((y[:8] == 0).all())
    gx, gw, gb = mhc.mhc_layer_norm_backward(x, w.cuda(), x)
    ref = R.norm_grad(last, w, last, 1e-6)
    bnd = R.norm_grad_bound(last, w, last, 1e-6, BF16)
    R.assert_within(gx[-4:], ref[0], bnd[0], "grad_x")
    R.assert_within(gw, ref[1], bnd[1], "grad_weight")
    R.assert_within(gb, ref[2], bnd[2], "grad_bias")
