"""The gated feed-forward block on the GPU against fp64.

Every element is held to the bound that layer_reference propagates (rigorous, so it grows
with the length of the sums); bf16 results also to the 2-norm: each stored value is off by
at most 2^-8 of itself, independently, and a result sees at most four such roundings on its
way (g or u, then a, dg or du, then itself), so |error| <= sqrt(4) 2^-8 |result|.
"""
import pytest
import torch

import layer_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TIMEOUT = 5
GRADS = ("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down")


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from manifold_constrained_hyper_token_b200 import build
    build.build()
    import manifold_constrained_hyper_token_b200 as m
    return m


def _case(T, C, F, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return ((1.5 * n(T, C)).to(dtype), (n(F, C) * C ** -0.5).to(dtype),
            (n(F, C) * C ** -0.5).to(dtype), (n(C, F) * F ** -0.5).to(dtype), n(T, C).to(dtype))


def _check_fwd(y, x, wg, wu, wd, act, dtype):
    ref = R.ffn(x, wg, wu, wd, act)
    R.assert_within(y, ref, R.ffn_bound(x, wg, wu, wd, act, dtype), "y")
    if dtype == BF16:
        assert R.norm_rel(y, ref) < 2.0 ** -7


def _check_bwd(got, x, wg, wu, wd, gy, act, dtype):
    ref = R.ffn_grad(x, wg, wu, wd, gy, act)
    bnd = R.ffn_grad_bound(x, wg, wu, wd, gy, act, dtype)
    for g, r, b, name in zip(got, ref, bnd, GRADS):
        R.assert_within(g, r, b, name)
        if dtype == BF16:
            assert R.norm_rel(g, r) < 2.0 ** -7, name


# (T, C, F): one element blocks, single tokens, widths that end inside every tile, each side
# of 64, 128 and 256 tokens, several tiles in every direction
SHAPES = [(1, 8, 8), (1, 64, 64), (1, 512, 1368), (2, 72, 200), (3, 1000, 264), (8, 256, 512),
          (15, 136, 1032), (16, 520, 248), (17, 64, 2048), (31, 328, 136), (33, 128, 128),
          (48, 1024, 264), (63, 200, 392), (64, 256, 256), (65, 264, 520), (100, 72, 8),
          (127, 8, 1000), (128, 512, 512), (129, 136, 264), (130, 512, 1368), (200, 1032, 96),
          (255, 320, 184), (256, 256, 1024), (257, 264, 776), (300, 1288, 648), (513, 520, 1032),
          (777, 64, 72), (1025, 384, 520)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,F", SHAPES)
def test_ffn(mhc, T, C, F, dtype):
    x, wg, wu, wd, _ = _case(T, C, F, dtype, T * 7 + C + F)
    for act in ("silu", "gelu"):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = mhc.mhc_ffn(x, wg, wu, wd, act=act, dev_status=st)
        assert int(st.item()) == 0
        _check_fwd(y, x, wg, wu, wd, act, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,F", SHAPES)
def test_ffn_backward(mhc, T, C, F, dtype):
    x, wg, wu, wd, gy = _case(T, C, F, dtype, T * 7 + C + F)
    for act in ("silu", "gelu"):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = mhc.mhc_ffn_backward(x, wg, wu, wd, gy, act=act, dev_status=st)
        assert int(st.item()) == 0
        _check_bwd(got, x, wg, wu, wd, gy, act, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,F", [(1, 4096, 8200), (40, 7168, 1024), (1500, 1000, 2728),
                                   (5000, 264, 520), (2100, 2056, 1032)])
def test_larger(mhc, T, C, F, dtype):
    """Long sums in each direction, and more tiles than SMs."""
    x, wg, wu, wd, gy = _case(T, C, F, dtype, 5)
    _check_fwd(mhc.mhc_ffn(x, wg, wu, wd), x, wg, wu, wd, "silu", dtype)
    _check_bwd(mhc.mhc_ffn_backward(x, wg, wu, wd, gy), x, wg, wu, wd, gy, "silu", dtype)


@pytest.mark.parametrize("T", [3, 300])
def test_saturated_gates(mhc, T):
    """Gates of several hundred either way: the activation's limits, without overflow."""
    x, wg, wu, wd, gy = _case(T, 64, 96, F32, 9)
    wg = wg * 200
    for act in ("silu", "gelu"):
        _check_fwd(mhc.mhc_ffn(x, wg, wu, wd, act=act), x, wg, wu, wd, act, F32)
        _check_bwd(mhc.mhc_ffn_backward(x, wg, wu, wd, gy, act=act), x, wg, wu, wd, gy, act, F32)
        b = [t.to(BF16) for t in (x, wg, wu, wd, gy)]
        y = mhc.mhc_ffn(*b[:4], act=act)
        ref = R.ffn(*b[:4], act)
        R.assert_within(y, ref, R.ffn_bound(*b[:4], act, BF16), "y")
        for g, r, d, n in zip(mhc.mhc_ffn_backward(*b, act=act), R.ffn_grad(*b, act),
                              R.ffn_grad_bound(*b, act, BF16), GRADS):
            R.assert_within(g, r, d, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,F", [(5, 136, 200), (100, 136, 200), (300, 136, 392)])
def test_nonfinite_tokens_stay_alone(mhc, T, C, F, dtype):
    """A token that is not finite spoils its own rows of y and grad_x and no others."""
    x, wg, wu, wd, gy = _case(T, C, F, dtype, 4)
    bad = x.clone()
    bad[2, 5] = float("nan")
    bad[T - 1, 0] = float("inf")
    keep = [t for t in range(T) if t not in (2, T - 1)]
    y, want = mhc.mhc_ffn(bad, wg, wu, wd), mhc.mhc_ffn(x, wg, wu, wd)
    assert torch.equal(y[keep], want[keep])
    assert bool(y[2].isnan().all()) and not bool(y[T - 1].isfinite().any())
    gx = mhc.mhc_ffn_backward(bad, wg, wu, wd, gy)[0]
    want = mhc.mhc_ffn_backward(x, wg, wu, wd, gy)[0]
    assert torch.equal(gx[keep], want[keep]) and bool(gx[2].isnan().all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,F", [(1, 136, 264), (33, 264, 520), (300, 520, 264)])
def test_repeats_bit_for_bit_and_writes_nothing_else(mhc, T, C, F, dtype):
    x, wg, wu, wd, gy = _case(T, C, F, dtype, 6)
    nf = mhc.mhc_ffn_workspace_size(T, C, F, dtype)
    nb = mhc.mhc_ffn_backward_workspace_size(T, C, F, dtype)
    first = None
    for fill in (0, 255):
        y, gx = (torch.full((T + 2, C), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        gwg, gwu = (torch.full((F + 2, C), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        gwd = torch.full((C + 2, F), 7.0, dtype=dtype, device="cuda")
        ws = torch.full((max(nf, nb) + 256,), fill, dtype=torch.uint8, device="cuda")
        mhc.mhc_ffn(x, wg, wu, wd, out=y[1:-1], workspace=ws[:nf])
        mhc.mhc_ffn_backward(x, wg, wu, wd, gy, workspace=ws[:nb],
                             out=tuple(t[1:-1] for t in (gx, gwg, gwu, gwd)))
        for t in (y, gx, gwg, gwu, gwd):
            assert bool((t[0] == 7).all()) and bool((t[-1] == 7).all())
        assert bool((ws[max(nf, nb):] == fill).all())
        out = [t.cpu() for t in (y, gx, gwg, gwu, gwd)]
        assert first is None or all(torch.equal(a, c) for a, c in zip(first, out))
        first = out


def test_a_token_does_not_depend_on_its_batch(mhc):
    """Rows of a larger batch agree with the same rows alone, to the roundings."""
    x, wg, wu, wd, _ = _case(700, 264, 520, BF16, 8)
    whole = mhc.mhc_ffn(x, wg, wu, wd)
    for n in (1, 5, 64, 130, 256):
        _check_fwd(mhc.mhc_ffn(x[:n], wg, wu, wd), x[:n], wg, wu, wd, "silu", BF16)
        assert R.norm_rel(mhc.mhc_ffn(x[:n], wg, wu, wd), whole[:n].double()) < 2.0 ** -7


@pytest.mark.parametrize("T", [1, 200])
def test_other_stream_and_graphs_with_one_workspace(mhc, T):
    """On another stream than the current one; and two graphs that share a workspace, replayed
    one after the other on new inputs."""
    C, F = 264, 520
    x, wg, wu, wd, gy = _case(T, C, F, BF16, 10)
    want = mhc.mhc_ffn(x, wg, wu, wd), *mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (mhc.mhc_ffn(x, wg, wu, wd, stream=s),
           *mhc.mhc_ffn_backward(x, wg, wu, wd, gy, stream=s))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    n = max(mhc.mhc_ffn_workspace_size(T, C, F, BF16),
            mhc.mhc_ffn_backward_workspace_size(T, C, F, BF16))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    xs, gs = torch.zeros_like(x), torch.zeros_like(gy)
    gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gf):
        y = mhc.mhc_ffn(xs, wg, wu, wd, workspace=ws)
    with torch.cuda.graph(gb):
        grads = mhc.mhc_ffn_backward(xs, wg, wu, wd, gs, workspace=ws)
    for scale in (1.0, 0.5, 1.0):
        xs.copy_(x * scale)
        gs.copy_(gy)
        gf.replay()
        gb.replay()
        gf.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, *grads)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(mhc, act):
    """fp32: grad . d against central differences of sum(gy . y) along random d.  With h = 2^-6
    the difference's own error is h^2 times a third derivative (of order one per unit of d's
    norm, the steps being h d with |d| = 1) and the forward's rounding over h: 2^-24 * 64 * 30
    |y| |gy|.  Both stay below 2e-4 of |gy| |y|."""
    x, wg, wu, wd, gy = _case(40, 72, 136, F32, 11)
    grads = mhc.mhc_ffn_backward(x, wg, wu, wd, gy, act=act)
    args, h = (x, wg, wu, wd), 2.0 ** -6
    y = mhc.mhc_ffn(*args, act=act).double()
    for i, g in enumerate(grads):
        d = torch.randn(args[i].shape, generator=torch.Generator().manual_seed(i)).cuda()
        d /= d.norm()
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * d, args[i] - h * d
        step = (up[i].double() - dn[i].double())  # the step as rounded
        diff = (mhc.mhc_ffn(*up, act=act).double() - mhc.mhc_ffn(*dn, act=act).double())
        got = float((diff * gy.double()).sum()) / (2 * h)
        want = float((g.double() * step).sum()) / (2 * h)
        assert abs(got - want) <= 2e-4 * float(gy.norm()) * float(y.norm()), GRADS[i]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,F", [(300, 264, 520), (40, 264, 520), (1500, 1032, 2056)])
@pytest.mark.parametrize("backward", [False, True])
def test_times_out_then_recovers(mhc, T, C, F, backward, dtype):
    """A wait limit of 1 ns makes the kernels' waits give up: the status word says so, and an
    ordinary call on the same buffers and workspace is right again."""
    x, wg, wu, wd, gy = _case(T, C, F, dtype, 12)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if backward:
        ws = torch.empty(mhc.mhc_ffn_backward_workspace_size(T, C, F, dtype), dtype=torch.uint8,
                         device="cuda")
        mhc.mhc_ffn_backward(x, wg, wu, wd, gy, workspace=ws, dev_status=st, wait_ns=1)
        assert int(st.item()) == TIMEOUT
        st.zero_()
        got = mhc.mhc_ffn_backward(x, wg, wu, wd, gy, workspace=ws, dev_status=st)
        assert int(st.item()) == 0
        _check_bwd(got, x, wg, wu, wd, gy, "silu", dtype)
    else:
        ws = torch.empty(mhc.mhc_ffn_workspace_size(T, C, F, dtype), dtype=torch.uint8,
                         device="cuda")
        mhc.mhc_ffn(x, wg, wu, wd, workspace=ws, dev_status=st, wait_ns=1)
        assert int(st.item()) == TIMEOUT
        st.zero_()
        y = mhc.mhc_ffn(x, wg, wu, wd, workspace=ws, dev_status=st)
        assert int(st.item()) == 0
        _check_fwd(y, x, wg, wu, wd, "silu", dtype)


@pytest.mark.parametrize("dtype,limit", [(F32, 40000), (BF16, 40000)])
def test_the_kernel_before_is_no_wait(mhc, dtype, limit):
    """The limit is for waits inside a kernel, on copies and on other warps: microseconds.  A few
    tokens' down projection has its first weights on their way while the gate still runs, for
    hundreds of microseconds here, and does not count that."""
    x, wg, wu, wd, _ = _case(128, 7168, 14336, dtype, 19)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = mhc.mhc_ffn(x, wg, wu, wd)
    for _ in range(5):
        got = mhc.mhc_ffn(x, wg, wu, wd, dev_status=st, wait_ns=limit)
        assert int(st.item()) == 0 and torch.equal(got, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gives_up_wherever_the_limit_falls(mhc, dtype):
    """Limits from one clock to about a copy's time stop the paired products at stages that
    differ from CTA to CTA.  Each call ends well inside the half second that a wait for a copy
    which never comes would take, and leaves nothing behind for the next."""
    x, wg, wu, wd, gy = _case(1500, 1032, 2056, dtype, 17)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = mhc.mhc_ffn(x, wg, wu, wd), *mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
    for limit in (1, 50, 150, 300, 600, 1000, 2000, 4000, 8000, 20000, 1000000):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        st.zero_()
        begin.record()
        mhc.mhc_ffn(x, wg, wu, wd, dev_status=st, wait_ns=limit)
        mhc.mhc_ffn_backward(x, wg, wu, wd, gy, dev_status=st, wait_ns=limit)
        end.record()
        end.synchronize()
        assert int(st.item()) in ((TIMEOUT,) if limit == 1 else (0, TIMEOUT))
        assert begin.elapsed_time(end) < 250, limit
        got = mhc.mhc_ffn(x, wg, wu, wd), *mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
        assert all(torch.equal(a, b) for a, b in zip(want, got)), limit


@pytest.mark.parametrize("T", [3, 40, 300])
def test_powers_of_two_pass_through(mhc, T):
    """fp32: x scaled by 2^-90 and both projections by 2^90 give the very bits of the unscaled
    call (all parts of the split operands are still normal numbers)."""
    x, wg, wu, wd, gy = _case(T, 136, 200, F32, 13)
    want = mhc.mhc_ffn(x, wg, wu, wd), *mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
    s = 2.0 ** 90
    y = mhc.mhc_ffn(x / s, wg * s, wu * s, wd)
    gx, gwg, gwu, gwd = mhc.mhc_ffn_backward(x / s, wg * s, wu * s, wd, gy)
    for a, b in zip(want, (y, gx / s, gwg * s, gwu * s, gwd)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [4, 100, 300])
def test_values_near_the_type_limit(mhc, T, dtype):
    """A token of 3.3e38 with weights that bring it back: finite, and right."""
    x, wg, wu, wd, _ = _case(T, 64, 72, dtype, 14)
    x[1] = 0
    x[1, 3] = 3.3e38
    wg[:, 3] *= 1e-38
    wu[:, 3] *= 1e-38
    _check_fwd(mhc.mhc_ffn(x, wg, wu, wd), x, wg, wu, wd, "silu", dtype)


def test_calls_on_two_streams_at_once(mhc):
    """Independent calls, each with its own workspace, in flight together."""
    cases = [_case(T, 520, 1032, dt, 20 + i)
             for i, (T, dt) in enumerate([(3, BF16), (200, BF16), (700, BF16), (5, F32),
                                          (90, F32), (400, F32)])]
    want = [(mhc.mhc_ffn(*c[:4]), *mhc.mhc_ffn_backward(*c)) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append([(mhc.mhc_ffn(*c[:4], stream=streams[i % 3]),
                     *mhc.mhc_ffn_backward(*c, stream=streams[(i + 1) % 3]))
                    for i, c in enumerate(cases)])
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(want, g):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,F", [(1, 1024, 2728), (5, 1024, 2728), (48, 1024, 2728),
                                   (200, 1024, 2728), (300, 1024, 2728)])
def test_weights_written_just_before_the_call(mhc, T, C, F, dtype):
    """The later products of a call read their weights before the kernel ahead of them has ended;
    a write of the weights that the stream has ahead of the call is seen all the same, by a copy
    or by the library's own kernels, which let the next one start early."""
    a = _case(T, C, F, dtype, 40)
    sets = [a[1:4], _case(T, C, F, dtype, 41)[1:4]]
    x, gy = a[0], a[4]
    want = [(mhc.mhc_ffn(x, *w), *mhc.mhc_ffn_backward(x, *w, gy)) for w in sets]
    w = [t.clone() for t in sets[0]]
    got = []
    for i in (1, 0, 1, 1, 0, 0, 1):
        for order in ((0, 1, 2), (2, 1, 0)):
            for k in order:
                w[k].copy_(sets[i][k])
            got.append((i, (mhc.mhc_ffn(x, *w),)))
            for k in order:
                w[k].copy_(sets[1 - i][k])
            got.append((1 - i, (None, *mhc.mhc_ffn_backward(x, *w, gy))))
    torch.cuda.synchronize()
    for i, outs in got:
        for p, q in zip(want[i], outs):
            assert q is None or torch.equal(p, q)
    # w_down and w_up as rows that the norm writes, the call's input from another call
    ones = torch.ones(F, device="cuda"), torch.ones(C, device="cuda")
    down, up = mhc.mhc_layer_norm(sets[1][2], ones[0]), mhc.mhc_layer_norm(sets[1][1], ones[1])
    h = mhc.mhc_ffn(x, *sets[0])
    torch.cuda.synchronize()
    want = mhc.mhc_ffn(h, sets[0][0], up, down), *mhc.mhc_ffn_backward(h, sets[0][0], up, down, gy)
    for _ in range(5):
        h2, up2, down2 = (torch.full_like(t, float("nan")) for t in (h, up, down))
        torch.cuda.synchronize()
        mhc.mhc_ffn(x, *sets[0], out=h2)
        mhc.mhc_layer_norm(sets[1][1], ones[1], out=up2)
        mhc.mhc_layer_norm(sets[1][2], ones[0], out=down2)
        got = (mhc.mhc_ffn(h2, sets[0][0], up2, down2),
               *mhc.mhc_ffn_backward(h2, sets[0][0], up2, down2, gy))
        assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_back_to_back_calls_share_a_workspace(mhc):
    """Calls on one stream with one workspace: each starts when the one before is done with it,
    although their kernels are set up early."""
    a, b = _case(300, 520, 1032, BF16, 30), _case(130, 520, 1032, BF16, 31)
    want = [[mhc.mhc_ffn(*c[:4]), *mhc.mhc_ffn_backward(*c)] for c in (a, b)]
    n = max(mhc.mhc_ffn_backward_workspace_size(300, 520, 1032, BF16),
            mhc.mhc_ffn_workspace_size(300, 520, 1032, BF16))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        got = [[mhc.mhc_ffn(*c[:4], workspace=ws), *mhc.mhc_ffn_backward(*c, workspace=ws)]
               for c in (a, b)]
        for w, g in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(w, g))


@pytest.mark.slow
def test_largest_offsets(mhc):
    """More than 2^31 hidden values: the last tokens agree with the same tokens alone."""
    T, C, F = 70000, 64, 32768
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 50 GB")
    x, wg, wu, wd, gy = _case(T, C, F, BF16, 15)
    y = mhc.mhc_ffn(x, wg, wu, wd)
    gx, gwg, _, gwd = mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
    for sl in (slice(0, 64), slice(T - 64, T)):
        R.assert_within(y[sl], R.ffn(x[sl], wg, wu, wd, "silu"),
                        R.ffn_bound(x[sl], wg, wu, wd, "silu", BF16), "y")
        R.assert_within(gx[sl], R.ffn_grad(x[sl], wg, wu, wd, gy[sl], "silu")[0],
                        R.ffn_grad_bound(x[sl], wg, wu, wd, gy[sl], "silu", BF16)[0], "grad_x")
    del y, gx
    # the weight gradients of 32 hidden units, over all tokens
    f = slice(F - 32, F)
    ref = R.ffn_grad(x, wg[f], wu[f], wd[:, f], gy, "silu")
    assert R.norm_rel(gwg[f], ref[1]) < 2.0 ** -7 and R.norm_rel(gwd[:, f], ref[3]) < 2.0 ** -7


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,F", [(8000, 64, 64), (4001, 136, 72), (300, 72, 8200),
                                   (1030, 2056, 136), (7, 64, 6656), (258, 8, 16384)])
def test_long_sums_with_few_results(mhc, T, C, F, dtype):
    """Products whose sums are split over the machine: long in tokens, in hidden units or in
    channels against a small result; twice, for the same bits."""
    x, wg, wu, wd, gy = _case(T, C, F, dtype, 16)
    y = mhc.mhc_ffn(x, wg, wu, wd)
    _check_fwd(y, x, wg, wu, wd, "silu", dtype)
    got = mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
    _check_bwd(got, x, wg, wu, wd, gy, "silu", dtype)
    again = mhc.mhc_ffn(x, wg, wu, wd), *mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
    assert all(torch.equal(a, b) for a, b in zip((y, *got), again))


# Sums of one sign, where a tensor-core adder that cuts is off in one direction.  A step of 16
# products may cut twice, by up to 2^-23 of what is summed so far: half of k 2^-26 over a sum of
# k equal terms, k 2^-27.
def _positive(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.rand(*s, generator=g, device="cuda") * 0.5 + 0.5


def _long_gate(mhc, T, C, dtype):
    """y = a through a w_down that picks 64 hidden units, and a in fp64: the sums are over C.
    Tokens and hidden units have factors of their own (g is 4.5 to 18), so that the results do
    not all round the same way."""
    p = _positive(C)
    x, wg = (p(T, C) * 2 * p(T, 1)).to(dtype), (p(64, C) * 16 / C).to(dtype)
    wu = (p(64, C) * 2 * p(64, 1) * 16 / C).to(dtype)
    wd = torch.zeros(C, 64, dtype=dtype, device="cuda")
    wd[:64] = torch.eye(64, device="cuda")
    g = u = 0
    for k in range(0, C, 1 << 15):
        s = slice(k, k + (1 << 15))
        g, u = g + x[:, s].double() @ wg[:, s].double().T, u + x[:, s].double() @ wu[:, s].double().T
    return mhc.mhc_ffn(x, wg, wu, wd)[:, :64], R.gate(g, "silu")[0] * u


def _long_weight_grads(mhc, T, C, F, dtype):
    """grad_w_up and grad_w_down of 64 hidden units, and both in fp64: the sums are over T.  Each
    channel has a factor of its own, so that the results do not all round the same way."""
    p = _positive(T)
    x, gy = ((p(T, C) * 2 * p(1, C)).to(dtype) for _ in range(2))
    wg, wu, wd = (p(F, C) * 4 / C).to(dtype), (p(F, C) * 4 / C).to(dtype), (p(C, F) / F).to(dtype)
    _, _, gwu, gwd = mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
    ru = rd = 0
    for t in range(0, T, 1 << 13):
        s = slice(t, t + (1 << 13))
        _, _, u, d = R.ffn_grad(x[s], wg[:64], wu[:64], wd[:, :64], gy[s], "silu")
        ru, rd = ru + u, rd + d
    return (gwu[:64], ru), (gwd[:, :64], rd)


def _off(got, ref):
    """The mean of the relative differences: what all elements are off by together."""
    return abs(float(((got.double() - ref) / ref).mean()))


# fp32, k_ffn_tc: the first planes' sums leave their accumulator every 256 k, 2^-19; the others,
# below 2^-6 of them together and in five products each, every 4096: 5 2^-15 2^-6 = 2^-18.7;
# what is left out 2^-21; what is added in rounded steps does not lean to a side.
FP32_SUM = 2.0 ** -19 + 5 * 2.0 ** -21 + 2.0 ** -21


def test_long_fp32_sums_of_one_sign(mhc):
    """a = silu(g) u takes the error of g (times at most 1.1 for g above 4) and that of u."""
    for C in (4096, 65536, 131072):
        assert _off(*_long_gate(mhc, 300, C, F32)) < 2.1 * FP32_SUM, C
    for got, ref in _long_weight_grads(mhc, 131072, 1024, 2432, F32):
        # the factors of the terms are themselves products: g, u and da over at most 1024
        assert _off(got, ref) < (1 + 2.1) * FP32_SUM


def test_long_bf16_sums_of_one_sign(mhc):
    """Sums over tokens and over hidden units are added up in fp32 from parts of 65536 terms:
    65536 2^-27 (a quarter of a bf16 rounding), however long they are.  What else all elements
    are off by together: the cuts in g, u and da over 1024 or 2048 channels, and the mean of as
    many roundings to bf16 as there are elements (2^-9 over the square root of 8192)."""
    own = 2.1 * 2048 * 2.0 ** -27 + 2 * 2.0 ** -9 / 8192 ** 0.5
    for got, ref in _long_weight_grads(mhc, 262144, 1024, 2560, BF16):
        assert _off(got, ref) < 2.0 ** -11 + own
    # y over 2^18 hidden units: many row tiles, and few tokens
    C, F = 2048, 262144
    p = _positive(F)
    wg, wu = (p(F, C) * 4 / C).to(BF16), (p(F, C) * 4 / C).to(BF16)
    wd = (p(C, F) * p(C, 1) / F).to(BF16)
    for T in (1300, 40):
        x = p(T, C).to(BF16)
        y = mhc.mhc_ffn(x, wg, wu, wd)[:4]
        ref = sum(R.ffn(x[:4], wg[f:f + 4096], wu[f:f + 4096], wd[:, f:f + 4096], "silu")
                  for f in range(0, F, 4096))
        assert _off(y, ref) < 2.0 ** -11 + own, T


def test_long_bf16_gates_of_one_sign(mhc):
    """The gate's sums over channels, and those of da: 65536 2^-27 at every length, for few tokens
    (up to eight parts of 65536) and for many.  a takes that of g (1.1) and of u; dg and du take
    that of da, and of u or g.  The mean of n roundings to bf16 adds 2^-9 / sqrt(n)."""
    for T, C in ((300, 65600), (300, 262144), (300, 1048576), (40, 524288), (17, 524296)):
        assert _off(*_long_gate(mhc, T, C, BF16)) < 2.1 * 2.0 ** -11 + 2.0 ** -9 / (64 * T) ** 0.5
    for T, C in ((300, 262144), (40, 524288)):
        p = _positive(C + T)
        x, gy = ((p(T, C) * 2 * p(1, C)).to(BF16) for _ in range(2))
        wg, wu, wd = (p(64, C) * 4 / C).to(BF16), (p(64, C) * 4 / C).to(BF16), p(C, 64).to(BF16)
        got = mhc.mhc_ffn_backward(x, wg, wu, wd, gy)
        ref = R.ffn_grad(x, wg, wu, wd, gy, "silu")
        for g, r, name in zip(got, ref, GRADS):
            assert _off(g, r) < 2.2 * 2.0 ** -11 + 2.0 ** -9 / 8192 ** 0.5, (T, C, name)


@pytest.mark.parametrize("T,C,F", [(300, 65600, 72), (700, 131080, 200), (129, 524296, 64),
                                   (5, 64, 262152)])
def test_sums_of_either_sign_over_many_channels(mhc, T, C, F):
    """Beyond 65536 channels (and, for few tokens, 2^19 or 2^18 hidden units)."""
    x, wg, wu, wd, gy = _case(T, C, F, BF16, 21)
    for act in ("silu", "gelu"):
        assert R.norm_rel(mhc.mhc_ffn(x, wg, wu, wd, act=act), R.ffn(x, wg, wu, wd, act)) < 2.0 ** -7
        ref = R.ffn_grad(x, wg, wu, wd, gy, act)
        for g, r, name in zip(mhc.mhc_ffn_backward(x, wg, wu, wd, gy, act=act), ref, GRADS):
            assert R.norm_rel(g, r) < 2.0 ** -7, name


def test_few_token_fp32_sums_of_one_sign(mhc):
    """k_ffn_few32 leaves up to 2048 k in an accumulator: 2^-16."""
    for T, C in ((17, 32768), (100, 16384)):
        assert _off(*_long_gate(mhc, T, C, F32)) < 2.1 * 2.0 ** -16, (T, C)


@pytest.mark.parametrize("T,C,F", [(3, 4096, 8200), (17, 8192, 4096), (100, 4096, 8192),
                                   (300, 8192, 4096), (4500, 1024, 2432)])
def test_fp32_error_in_the_norm(mhc, T, C, F):
    """The element bound grows with k and would let a lost plane pass; in the 2-norm the
    roundings of a sum of k terms of either sign grow with its square root: 2^-19 (the adder, in
    256 k) or 2^-16 (2048 k of k_ffn_few32), less than 2^-17 in fact, and two products in a row
    with a factor each.  A lost second plane would be 2^-9."""
    x, wg, wu, wd, gy = _case(T, C, F, F32, 18)
    assert R.norm_rel(mhc.mhc_ffn(x, wg, wu, wd), R.ffn(x, wg, wu, wd, "silu")) < 2.0 ** -15
    ref = R.ffn_grad(x, wg, wu, wd, gy, "silu")
    for g, r, name in zip(mhc.mhc_ffn_backward(x, wg, wu, wd, gy), ref, GRADS):
        assert R.norm_rel(g, r) < 2.0 ** -15, name
