"""RMSNorm and LayerNorm rows and their gradients (moe_norm_forward, moe_norm_backward) against plain
64-bit forms: rows held by a warp, by a block and read again, every vector width and type."""
import threading

import pytest
import torch

from tests import ops64
from tests.test_gpu_rows import DT, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mixture_experts_softmax_b200 as m
    return m


def inputs(T, d, dt, layer, seed=0):
    g = torch.Generator().manual_seed(seed + T * 7 + d)
    x = (torch.randn((T, d), generator=g) * (0.2 + 3 * torch.rand((T, 1), generator=g))
         + torch.randn((1, d), generator=g)).to(DT[dt])
    gain = (1 + 0.3 * torch.randn(d, generator=g)).to(DT[dt])
    bias = (0.3 * torch.randn(d, generator=g)).to(DT[dt]) if layer else None
    return x, gain, bias, torch.randn((T, d), generator=g).to(DT[dt])


def cuda(t):
    return None if t is None else t.cuda()


def run_forward(m, kind, dt, x, gain, bias, eps=1e-5):
    T, d = x.shape
    y, c0 = guarded((T, d), DT[dt], 99.0)
    stats, c1 = guarded((T, 2), torch.float32, 99.0)
    m.check(m.moe_norm_forward(kind, dt, T, d, x.cuda(), cuda(gain), cuda(bias), eps, y, stats), "moe_norm_forward")
    torch.cuda.synchronize()
    c0()
    c1()
    return y.cpu(), stats.cpu()


def run_backward(m, kind, dt, x, gain, stats, dy, want_bias):
    T, d = x.shape
    dx, c0 = guarded((T, d), DT[dt], 99.0)
    dgain, c1 = guarded((d,), torch.float32, 99.0)
    dbias, c2 = guarded((d,), torch.float32, 99.0)
    ws, c3 = guarded((m.moe_norm_workspace(T, d),), torch.uint8, 255)   # nan, read as fp32
    m.check(m.moe_norm_backward(kind, dt, T, d, x.cuda(), cuda(gain), stats.cuda(), dy.cuda(), dx, dgain,
                                dbias if want_bias else None, ws), "moe_norm_backward")
    torch.cuda.synchronize()
    for c in (c0, c1, c2, c3):
        c()
    return dx.cpu(), dgain.cpu(), dbias.cpu()


# a warp a row (by 16-, 4- and 2-byte vectors, and single elements), a block a row, rows read again
SIZES = [(1, 1), (1, 6144), (3, 2), (5, 37), (9, 256), (17, 1024), (130, 1030), (33, 1537), (65, 4104), (700, 520), (700, 2560),
         (2, 8191), (3, 16384), (5, 16392), (2, 33000), (1, 40001), (2, 65536)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("kind", [0, 1])
def test_norm(m, T, d, dt, kind):
    x, gain, bias, dy = inputs(T, d, dt, kind == 1)
    y, stats = run_forward(m, kind, dt, x, gain, bias)
    ref, rstats, tol, tstats = ops64.norm(x, gain, bias, float(torch.tensor(1e-5)), kind == 1, DT[dt])
    ops64.assert_close(stats, rstats, tstats, "stats")
    ops64.assert_close(y, ref, tol, "y")
    got = run_backward(m, kind, dt, x, gain, stats, dy, kind == 1)
    want, tols = ops64.norm_grad(x, gain, stats, dy, kind == 1, DT[dt])
    ops64.assert_close(got[0], want[0], tols[0], "dx")
    ops64.assert_close(got[1], want[1], tols[1], "dgain")
    if kind == 1:
        ops64.assert_close(got[2], want[2], tols[2], "dbias")


@pytest.mark.parametrize("T,d", [(3000, 96), (2500, 8200), (4000, 19), (1300, 6144), (1000, 16400), (3001, 1537),
                                 (1999, 4100), (901, 12001), (2111, 1022), (640, 16384)])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dt", [0, 2])
def test_norm_many_rows(m, T, d, kind, dt):
    """More rows than blocks: every block sums over several, of each of the classes of rows that begin at the same
    place within 16 bytes."""
    x, gain, bias, dy = inputs(T, d, dt, kind == 1)
    y, stats = run_forward(m, kind, dt, x, gain, bias)
    ref, _, tol, _ = ops64.norm(x, gain, bias, float(torch.tensor(1e-5)), kind == 1, DT[dt])
    ops64.assert_close(y, ref, tol, "y")
    got = run_backward(m, kind, dt, x, gain, stats, dy, kind == 1)
    want, tols = ops64.norm_grad(x, gain, stats, dy, kind == 1, DT[dt])
    for a, b, t in list(zip(got, want, tols))[:2 + kind]:
        ops64.assert_close(a, b, t)


@pytest.mark.parametrize("kind", [0, 1])
def test_norm_without_gain_bias_stats(m, kind):
    x, _, _, dy = inputs(20, 384, 0, False)
    y = torch.empty((20, 384), dtype=torch.bfloat16, device="cuda")
    m.check(m.moe_norm_forward(kind, 0, 20, 384, x.cuda(), None, None, 1e-6, y, None))
    ref, rstats, tol, _ = ops64.norm(x, None, None, float(torch.tensor(1e-6)), kind == 1, DT[0])
    ops64.assert_close(y.cpu(), ref, tol)
    stats = rstats.float()
    dx = torch.empty_like(y)
    ws = torch.empty(m.moe_norm_workspace(20, 384), dtype=torch.uint8, device="cuda")
    m.check(m.moe_norm_backward(kind, 0, 20, 384, x.cuda(), None, stats.cuda(), dy.cuda(), dx, None, None, ws))
    want, tols = ops64.norm_grad(x, None, stats, dy, kind == 1, DT[0])
    ops64.assert_close(dx.cpu(), want[0], tols[0])


def test_dbias_alone_and_dgain_alone(m):
    x, gain, bias, dy = inputs(50, 200, 2, True)
    _, stats = run_forward(m, 1, 2, x, gain, bias)
    full = run_backward(m, 1, 2, x, gain, stats, dy, True)
    ws = torch.empty(m.moe_norm_workspace(50, 200), dtype=torch.uint8, device="cuda")
    for which in (1, 2):
        out = torch.empty(200, device="cuda")
        dx = torch.empty((50, 200), device="cuda")
        m.check(m.moe_norm_backward(1, 2, 50, 200, x.cuda(), gain.cuda(), stats.cuda(), dy.cuda(), dx,
                                    out if which == 1 else None, out if which == 2 else None, ws))
        assert torch.equal(out.cpu(), full[which]) and torch.equal(dx.cpu(), full[0])


def test_no_rows(m):
    g, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    m.check(m.moe_norm_forward(0, 0, 0, 64, None, None, None, 1e-5, None))
    m.check(m.moe_norm_backward(1, 0, 0, 64, None, None, None, None, None, g, b, None))
    assert (g == 0).all() and (b == 0).all()


def test_constant_and_offset_rows(m):
    """A constant row has variance 0: y = bias, whatever its size; a large mean does not cost the variance."""
    x = torch.full((4, 512), 1000.0)
    x[2:] = 4096.0 + torch.randn((2, 512), generator=torch.Generator().manual_seed(0)) * 2.0 ** -3
    gain, bias = torch.full((512,), 2.0), torch.full((512,), 0.5)
    y, stats = run_forward(m, 1, 2, x, gain, bias)
    assert (y[:2] == 0.5).all() and (stats[:2, 0] == 1000.0).all()
    ref, _, tol, _ = ops64.norm(x, gain, bias, float(torch.tensor(1e-5)), True, torch.float32)
    ops64.assert_close(y, ref, tol)
    # The bound by arithmetic: the mean may be off by 80 * 2^-24 * 4096 = 0.0195, which is 0.16 of the rows'
    # deviation of 1/8 (times the gain of 2: 0.31), and the variance by 2 * 0.0195 * mean|c| = 0.0195 / 5 of
    # 1/64, a quarter: an eighth of |y - bias| <= 7.5, 0.94.  A difference of squares would be off by
    # 2^-24 * 4096^2 = 1, 64 times the variance.
    assert tol[2:].max() < 0.31 + 0.94 + 0.25


def test_nonfinite_rows_stay_in_their_row(m):
    x, gain, bias, dy = inputs(12, 300, 0, True)
    x[3, 7] = float("nan")
    x[8, 100] = float("inf")
    y, stats = run_forward(m, 1, 0, x, gain, bias)
    ok = [t for t in range(12) if t not in (3, 8)]
    assert y[3].isnan().all() and y[8].isnan().any()
    assert y[ok].isfinite().all() and stats[ok].isfinite().all()


@pytest.mark.parametrize("layer", [False, True])
def test_gradient_against_differences(m, layer):
    """The products of the gradients with random directions against central differences of the 64-bit form."""
    T, d, eps = 6, 40, float(torch.tensor(1e-5))
    x, gain, bias, dy = inputs(T, d, 2, layer)
    _, stats = run_forward(m, int(layer), 2, x, gain, bias)
    dx, dgain, dbias = (t.double() for t in run_backward(m, int(layer), 2, x, gain, stats, dy, layer))
    g = torch.Generator().manual_seed(9)
    u, v, w = (torch.randn(s, generator=g).double() for s in ((T, d), (d,), (d,)))

    def f(h):
        b = bias.double() + h * w if layer else None
        return (ops64.norm(x.double() + h * u, gain.double() + h * v, b, eps, layer, torch.float32)[0] * dy.double()).sum()
    h = 2.0 ** -12
    diff = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
    terms = torch.cat([(dx * u).flatten(), dgain * v, (dbias * w) if layer else torch.zeros(1).double()])
    # fp32 gradients and statistics: 200 roundings on each term's size; the differences leave h^4 of the
    # fifth derivative, whose scale is (1 / sd)^5 < 2^12 here: 2^-36 of the terms
    sizes = (dy.double().abs() * stats[:, 1:].double() * u.abs()).sum() * 4 * gain.abs().max() + terms.abs().sum() \
        + (dy.double().abs() * 4).sum() * v.abs().max()
    assert abs(terms.sum() - diff) <= 200 * ops64.U * sizes


def test_offsets_pass_32_bits(m):
    """Rows beyond 2^31 elements: the last rows of 262,144 x 8,704 against the same rows alone."""
    T, d = 262144, 8704
    x = torch.ones((T, d), dtype=torch.bfloat16, device="cuda")
    tail, gain, _, dy = inputs(16, d, 0, False)
    x[-16:] = tail.cuda()
    y = torch.empty_like(x)
    stats = torch.empty((T, 2), device="cuda")
    m.check(m.moe_norm_forward(0, 0, T, d, x, gain.cuda(), None, 1e-5, y, stats))
    want, wstats = run_forward(m, 0, 0, tail, gain, None)
    assert torch.equal(y[-16:].cpu(), want) and torch.equal(stats[-16:].cpu(), wstats)
    g = torch.zeros_like(x)
    g[-16:] = dy.cuda()
    dgain = torch.empty(d, device="cuda")
    ws = torch.empty(m.moe_norm_workspace(T, d), dtype=torch.uint8, device="cuda")
    m.check(m.moe_norm_backward(0, 0, T, d, x, gain.cuda(), stats, g, y, dgain, None, ws))
    dx, dg, _ = run_backward(m, 0, 0, tail, gain, wstats, dy, False)
    assert torch.equal(y[-16:].cpu(), dx) and (y[:-16] == 0).all()
    _, tols = ops64.norm_grad(tail, gain, wstats, dy, False, DT[0])
    ops64.assert_close(dgain.cpu(), dg.double(), 2 * tols[1])


@pytest.mark.parametrize("d", [3, 37, 96, 512, 1022, 1537, 4100, 6144, 8200, 16400, 40001])
@pytest.mark.parametrize("dt", [0, 1, 2])
def test_constant_rows_of_any_width(m, d, dt):
    """Rows of one value, small to large, and of widths whose inverse is no power of two: the mean is that value and y is the
    bias, both to the bit.  The pivot is off by at most 80 U |x| (the sum's chain and the division), every difference from it is
    the same exact number e, so q and d m^2 are d e^2 but for 80 + 84 roundings: what is left is the variance's error."""
    x = torch.tensor([1000.0, -1000.1, 0.3, 30000.7, 1.0, 4096.5]).to(DT[dt])[:, None].expand(6, d).contiguous()
    gain, bias = torch.full((d,), 2.0).to(DT[dt]), torch.full((d,), 0.5).to(DT[dt])
    eps = float(torch.tensor(1e-5))
    y, stats = run_forward(m, 1, dt, x, gain, bias)
    assert torch.equal(stats[:, 0], x[:, 0].float())
    assert (y == 0.5).all()
    left = 164 * ops64.U * (80 * ops64.U * x[:, 0].double()) ** 2
    want = eps ** -0.5
    assert ((stats[:, 1].double() - want).abs() <= want * (0.5 * left / eps + 4 * ops64.U)).all()


@pytest.mark.parametrize("T,d", [(5, 96), (5, 1537), (3, 6144), (3, 8200), (3, 16400)])
def test_mean_of_offset_rows(m, T, d):
    """Rows far from 0 next to their spread, fp32: the mean is off by its own rounding and those of the differences from the
    pivot, not by those of the sum.  |x - pivot| <= |x - mean| + 80 U |mean|; each of them is rounded once, summed by a chain of
    80 and divided (4 roundings); pivot + m is rounded once."""
    g = torch.Generator().manual_seed(d)
    x = 30000 + torch.randn((T, d), generator=g) * torch.tensor([1.0, 2.0 ** -4, 8.0, 1.0, 1.0])[:T, None]
    _, stats = run_forward(m, 1, 2, x, None, None)
    x8 = x.double()
    mean = x8.mean(1)
    spread = (x8 - mean[:, None]).abs().mean(1)
    tol = ops64.U * mean.abs() + 85 * ops64.U * (spread + 80 * ops64.U * mean.abs())
    ops64.assert_close(stats[:, 0], mean, tol, "mean")


def test_host_threads_at_once(m):
    """Backward calls from four host threads, each on its own stream, of two widths that take the same kernel with different amounts
    of shared memory: no call disturbs another's launch, and the results are those of a call alone."""
    cases = []
    for d in (4096, 6144) * 2:
        x, gain, bias, dy = inputs(16, d, 2, True)
        _, stats = run_forward(m, 1, 2, x, gain, bias)
        want = run_backward(m, 1, 2, x, gain, stats, dy, True)
        ins = [t.cuda() for t in (x, gain, stats, dy)]
        outs = [torch.empty((16, d), device="cuda"), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
        ws = torch.empty(m.moe_norm_workspace(16, d), dtype=torch.uint8, device="cuda")
        cases.append((d, want, ins, outs, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    status = []

    def work(d, want, ins, outs, ws, stream):
        # addresses: the calls follow one another as closely as the host allows
        args = [t.data_ptr() for t in (*ins, *outs, ws)] + [stream.cuda_stream]
        status.append({m.moe_norm_backward(1, 2, 16, d, *args) for _ in range(20000)})
    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [{m.MOE_OK}] * 4
    for d, want, ins, outs, ws, stream in cases:
        for got, ref in zip(outs, want):
            assert torch.equal(got.cpu(), ref)


@pytest.mark.parametrize("T,d", [(12, 37), (12, 300), (12, 301), (40, 1537), (12, 8200), (12, 16401)])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dt", [0, 2])
def test_nonfinite_gradient_rows_stay_in_their_row(m, T, d, kind, dt):
    """nan and inf at both ends and inside of some rows of x and dy, next to rows that share their 16-byte vectors: the other rows'
    dx does not change by a bit, and a column's sums are nan only where a bad row is in it."""
    x, gain, bias, dy = inputs(T, d, dt, kind == 1)
    _, stats = run_forward(m, kind, dt, x, gain, bias)
    want = run_backward(m, kind, dt, x, gain, stats, dy, kind == 1)
    bad = {2: (x, float("nan")), 5: (dy, float("inf")), 8: (dy, float("nan"))}
    for row, (t, v) in bad.items():
        t[row, [0, d // 2, d - 1]] = v
    got = run_backward(m, kind, dt, x, gain, stats, dy, kind == 1)
    ok = [t for t in range(T) if t not in bad]
    assert torch.equal(got[0][ok], want[0][ok])
    for row in bad:
        assert not got[0][row].isfinite().any()
    cols = torch.ones(d, dtype=torch.bool)
    cols[[0, d // 2, d - 1]] = False
    for a, b in list(zip(got, want))[1:2 + kind]:
        assert torch.equal(a[cols], b[cols])
        assert not a[~cols].isfinite().any()


@pytest.mark.parametrize("d", [96, 1537, 6144, 8200, 16400, 40001])
def test_constant_rows_of_huge_values(m, d):
    """Values whose pivot is off by more than fp32 squares hold: the mean is still the value and y the bias."""
    x = torch.tensor([3.3e26, -1.7e30, 7.7e18])[:, None].expand(3, d).contiguous()
    gain, bias = torch.full((d,), 2.0), torch.full((d,), 0.5)
    y, stats = run_forward(m, 1, 2, x, gain, bias)
    assert torch.equal(stats[:, 0], x[:, 0])
    assert (y == 0.5).all()
