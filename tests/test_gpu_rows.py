"""Rows sorted by expert and back, and the gradients (moe_sort_rows, moe_unsort_rows,
moe_unsort_rows_backward), against plain 64-bit forms: every element type and vector width, one
launch and two, one block of the order's cluster and eight, dropped and repeated routes, empty experts."""
import pytest
import torch

from tests import ops64

pytestmark = pytest.mark.gpu

DT = {0: torch.bfloat16, 1: torch.float16, 2: torch.float32}
GUARD = 256   # elements behind every output, which must keep their value


@pytest.fixture(scope="module")
def m():
    import mixture_experts_softmax_b200 as m
    return m


def guarded(shape, dtype, fill):
    """A tensor of the shape with a guard behind it: (tensor, check())."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + GUARD,), fill, dtype=dtype, device="cuda")

    def check():
        assert (buf[n:] == fill).all(), "written behind the end"
    return buf[:n].view(shape), check


def choices(T, k, E, drop, seed, repeat=False):
    g = torch.Generator().manual_seed(seed)
    if repeat:
        idx = torch.randint(0, E, (T, k), generator=g)
    else:
        idx = torch.rand((T, E), generator=g).argsort(1)[:, :k]
        if idx.shape[1] < k:
            idx = torch.cat([idx, torch.zeros(T, k - idx.shape[1], dtype=idx.dtype)], 1)
    idx = idx.to(torch.int32).contiguous()
    lost = torch.rand((T, k), generator=g) < drop
    idx[lost] = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)[torch.randint(0, 4, (int(lost.sum()),),
                                                                                              generator=g)]
    return idx


def run_sort(m, dt, idx, E, x):
    T, k = idx.shape
    d = x.shape[1]
    offsets, c0 = guarded((E + 1,), torch.int32, -7)
    perm, c1 = guarded((T * k,), torch.int32, -7)
    slot, c2 = guarded((T, k), torch.int32, -7)
    rows, c3 = guarded((T * k, d), DT[dt], 99.0)
    m.check(m.moe_sort_rows(dt, T, k, E, d, x.cuda(), idx.cuda(), offsets, perm, slot, rows), "moe_sort_rows")
    torch.cuda.synchronize()
    for c in (c0, c1, c2, c3):
        c()
    return offsets.cpu(), perm.cpu(), slot.cpu(), rows.cpu()


def check_sort(got, idx, E, x):
    offsets, perm, slot, rows = got
    want = ops64.sort(idx, E)
    assert torch.equal(offsets, want[0])
    assert torch.equal(perm, want[1])
    assert torch.equal(slot, want[2])
    n = int(want[0][-1])
    assert torch.equal(rows[:n], x[want[1][:n].long() // idx.shape[1]])
    assert (rows[n:] == 99.0).all(), "rows behind the last one changed"


# widths: 16-, 8-, 4- and 2-byte vectors; short rows that share a warp, long ones over many units
SORT = [(1, 2, 8, 256), (1, 1, 1, 1), (8, 2, 8, 6144), (13, 3, 5, 37), (64, 2, 8, 2), (33, 8, 160, 1030), (511, 2, 8, 72),
        (512, 2, 8, 130), (513, 2, 8, 131), (1024, 4, 16, 64), (1025, 4, 16, 68), (2100, 4, 256, 33), (5000, 4, 31, 40),
        (9001, 16, 256, 8), (30000, 2, 2, 24)]


@pytest.mark.parametrize("T,k,E,d", SORT)
@pytest.mark.parametrize("dt", [0, 1, 2])
def test_sort(m, T, k, E, d, dt):
    idx = choices(T, k, E, 0.0, T + d)
    x = torch.randn((T, d), generator=torch.Generator().manual_seed(d)).to(DT[dt])
    check_sort(run_sort(m, dt, idx, E, x), idx, E, x)


@pytest.mark.parametrize("T,k,E,d,drop,repeat", [(300, 4, 8, 64, 0.3, True), (1500, 2, 3, 10, 0.5, True), (40, 2, 8, 16, 1.0, False),
                                                 (4000, 2, 8, 16, 1.0, False), (777, 16, 5, 9, 0.1, True)])
def test_sort_dropped_and_repeated(m, T, k, E, d, drop, repeat):
    idx = choices(T, k, E, drop, T, repeat)
    x = torch.randn((T, d), generator=torch.Generator().manual_seed(d)).to(torch.bfloat16)
    check_sort(run_sort(m, 0, idx, E, x), idx, E, x)


@pytest.mark.parametrize("T", [100, 6000])
def test_sort_all_to_one_expert(m, T):
    idx = torch.full((T, 2), 5, dtype=torch.int32)
    idx[:, 1] = 0
    x = torch.randn(T, 48).to(torch.float16)
    check_sort(run_sort(m, 1, idx, 8, x), idx, 8, x)


def test_sort_order_alone_and_no_tokens(m):
    for T in (50, 3000):
        idx = choices(T, 2, 8, 0.2, T)
        offsets = torch.empty(9, dtype=torch.int32, device="cuda")
        perm = torch.empty(2 * T, dtype=torch.int32, device="cuda")
        slot = torch.empty((T, 2), dtype=torch.int32, device="cuda")
        m.check(m.moe_sort_rows(0, T, 2, 8, 64, None, idx.cuda(), offsets, perm, slot, None))
        for got, want in zip((offsets, perm, slot), ops64.sort(idx, 8)):
            assert torch.equal(got.cpu(), want)
    m.check(m.moe_sort_rows(0, 0, 2, 8, 64, None, None, offsets, None, None, None))
    assert (offsets == 0).all()


def test_sort_matches_the_layer_s_own_dispatch(m):
    """On the layer's routing (8 experts, 2 picks) the order is that of moe_route_noalloc."""
    T, d = 1200, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((d, 8), generator=g, device="cuda") / 16
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, offsets, perm = torch.empty((T, 2), **i32), torch.empty(9, **i32), torch.empty(2 * T, **i32)
    gate = torch.empty((T, 2), device="cuda")
    m.check(m.moe_route_noalloc(T, d, x, w, None, idx, gate, offsets, perm))
    off2, perm2, slot2 = torch.empty(9, **i32), torch.empty(2 * T, **i32), torch.empty((T, 2), **i32)
    m.check(m.moe_sort_rows(m.MOE_BF16, T, 2, 8, d, None, idx, off2, perm2, slot2, None))
    assert torch.equal(offsets, off2) and torch.equal(perm, perm2)


BACK = [(1, 1, 1), (1, 2, 6144), (7, 3, 37), (64, 2, 256), (65, 8, 130), (30, 16, 1030), (300, 2, 4104), (500, 5, 24), (3, 6, 2051)]


def back_case(T, k, d, rd, dt, drop=0.2):
    g = torch.Generator().manual_seed(T * 31 + d)
    idx = choices(T, k, 16, drop, T + k, repeat=True)
    slot = ops64.sort(idx, 16)[2]
    rows = torch.randn((T * k, d), generator=g).to(DT[rd])
    gate = torch.rand((T, k), generator=g)
    return slot, rows, gate, torch.randn((T, d), generator=g).to(DT[dt])


@pytest.mark.parametrize("T,k,d", BACK)
@pytest.mark.parametrize("rd,dt", [(0, 0), (1, 1), (2, 2), (2, 0), (2, 1)])
@pytest.mark.parametrize("gated", [True, False])
def test_unsort(m, T, k, d, rd, dt, gated):
    slot, rows, gate, _ = back_case(T, k, d, rd, dt)
    gate = gate if gated else None
    out, check = guarded((T, d), DT[dt], 99.0)
    m.check(m.moe_unsort_rows(rd, dt, T, k, d, rows.cuda(), slot.cuda(), None if gate is None else gate.cuda(), out))
    torch.cuda.synchronize()
    check()
    ref, tol = ops64.unsort(rows, slot, gate, DT[dt])
    ops64.assert_close(out.cpu(), ref, tol, "out")


@pytest.mark.parametrize("T,k,d", BACK)
@pytest.mark.parametrize("rd,dt", [(0, 0), (1, 1), (2, 2), (2, 0), (2, 1)])
def test_unsort_gradient(m, T, k, d, rd, dt):
    slot, rows, gate, dout = back_case(T, k, d, rd, dt)
    drows, c0 = guarded((T * k, d), DT[rd], 99.0)
    dgate, c1 = guarded((T, k), torch.float32, 99.0)
    m.check(m.moe_unsort_rows_backward(rd, dt, T, k, d, dout.cuda(), rows.cuda(), slot.cuda(), gate.cuda(), drows, dgate))
    torch.cuda.synchronize()
    c0()
    c1()
    want, wgate, tol, tgate = ops64.unsort_grad(dout, rows, slot, gate, DT[rd])
    hit = ~want.isnan().any(1)
    ops64.assert_close(drows.cpu()[hit], want[hit], tol[hit], "drows")
    assert (drows.cpu()[~hit] == 99.0).all(), "a row that no route points to changed"
    ops64.assert_close(dgate.cpu(), wgate, tgate, "dgate")
    # without the gates' gradient the rows are not read, and the rows' gradient is the same
    again = torch.full_like(drows, 99.0)
    m.check(m.moe_unsort_rows_backward(rd, dt, T, k, d, dout.cuda(), None, slot.cuda(), gate.cuda(), again, None))
    assert torch.equal(again, drows)


def test_gradient_against_differences(m):
    """<dout, unsort(rows + h v, gate + h w) - unsort(rows, gate)> / h, in 64 bits, is the gradients' product
    with (v, w): the operator is linear in each, so the central difference is exact up to rounding."""
    T, k, d = 40, 3, 50
    slot, rows, gate, dout = back_case(T, k, d, 2, 2)
    drows = torch.zeros((T * k, d), device="cuda")
    dgate = torch.zeros((T, k), device="cuda")
    m.check(m.moe_unsort_rows_backward(2, 2, T, k, d, dout.cuda(), rows.cuda(), slot.cuda(), gate.cuda(), drows, dgate))
    g = torch.Generator().manual_seed(0)
    v, w = torch.randn(rows.shape, generator=g).double(), torch.randn(gate.shape, generator=g).double()
    h = 2.0 ** -10
    up, dn = (ops64.unsort(rows.double() + s * h * v, slot, gate.double() + s * h * w, torch.float32)[0] for s in (1, -1))
    diff = ((up - dn) / (2 * h) * dout.double()).sum()
    terms = torch.cat([(drows.cpu().double() * v).flatten(), (dgate.cpu().double() * w).flatten()])
    # fp32 gradients: (ceil(50 / 32) + 16) U at most on each term's sizes; 32 U of all terms covers it, and
    # dgate's own terms are sums of 50 products
    size = terms.abs().sum() + (dout.double().abs().sum(1, keepdim=True) * w.abs()).sum() * rows.abs().max()
    assert abs(terms.sum() - diff) <= 32 * ops64.U * size


def test_sort_and_its_gradient_are_adjoint(m):
    """<rows(x), r> = <x, unsort(r)> with every gate 1."""
    T, k, E, d = 700, 4, 9, 96
    idx = choices(T, k, E, 0.25, 5)
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randint(-8, 9, s, generator=g).float() for s in ((T, d), (T * k, d)))
    rows = run_sort(m, 2, idx, E, x)
    n = int(rows[0][-1])
    dx = torch.empty((T, d), device="cuda")
    m.check(m.moe_unsort_rows(2, 2, T, k, d, r.cuda(), rows[2].cuda(), None, dx))
    assert (rows[3][:n].double() * r[:n].double()).sum() == (x.double() * dx.cpu().double()).sum()   # whole numbers


def test_dropped_routes_ignore_their_gate_and_row(m):
    """nan and inf in the gate of a dropped route, and in rows that no route points to, stay out of the results."""
    T, k, d = 90, 2, 64
    idx = choices(T, k, 4, 0.4, 11)
    slot = ops64.sort(idx, 4)[2]
    n = int((slot >= 0).sum())
    g = torch.Generator().manual_seed(2)
    rows = torch.randn((T * k, d), generator=g)
    rows[n:] = float("nan")
    gate = torch.rand((T, k), generator=g)
    gate[slot < 0] = float("inf")
    out = torch.empty((T, d), device="cuda")
    m.check(m.moe_unsort_rows(2, 2, T, k, d, rows.cuda(), slot.cuda(), gate.cuda(), out))
    ref, tol = ops64.unsort(rows, slot, gate, torch.float32)
    ops64.assert_close(out.cpu(), ref, tol)
    assert (out[(slot < 0).all(1).cuda()] == 0).all()
    dgate = torch.full((T, k), 7.0, device="cuda")
    drows = torch.full((T * k, d), 5.0, device="cuda")
    dout = torch.randn((T, d), generator=g)
    m.check(m.moe_unsort_rows_backward(2, 2, T, k, d, dout.cuda(), rows.cuda(), slot.cuda(), gate.cuda(), drows, dgate))
    assert (dgate.cpu()[slot < 0] == 0).all() and dgate.isfinite().all()
    assert (drows[n:] == 5.0).all() and drows.isfinite().all()


def test_nonfinite_values_follow_the_formula(m):
    """An inf row times a positive gate is inf; inf times 0 and nan are nan; other tokens do not change."""
    slot = torch.arange(6, dtype=torch.int32).view(3, 2)
    rows = torch.ones(6, 16)
    rows[0, 3] = float("inf")
    rows[2, 5] = float("nan")
    gate = torch.tensor([[0.5, 0.5], [0.5, 0.5], [1.0, 0.25]])
    out = torch.empty((3, 16), device="cuda")
    m.check(m.moe_unsort_rows(2, 2, 3, 2, 16, rows.cuda(), slot.cuda(), gate.cuda(), out))
    out = out.cpu()
    assert out[0, 3] == float("inf") and out[1, 5].isnan() and (out[2] == 1.25).all()
    assert out[0].isfinite().sum() == 15 and out[1].isfinite().sum() == 15


def test_bad_slots_are_dropped_routes(m):
    slot = torch.tensor([[0, 8], [-5, 2 ** 31 - 1], [3, -2 ** 31], [7, 1]], dtype=torch.int32)
    rows = torch.arange(8.0)[:, None].expand(8, 8).contiguous()
    out = torch.empty((4, 8), device="cuda")
    m.check(m.moe_unsort_rows(2, 2, 4, 2, 8, rows.cuda(), slot.cuda(), None, out))
    assert out[:, 0].tolist() == [0.0, 0.0, 3.0, 8.0]


def test_sort_offsets_pass_32_bits(m):
    """Rows beyond 2^31 elements: 262,144 tokens of 8,704 values, one pick (4.6 GB a side)."""
    T, d = 262144, 8704
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.arange(T, device="cuda") % 251
    x[:, -1] = torch.arange(T, device="cuda") % 241
    idx = (1 - torch.arange(T, device="cuda") % 2).to(torch.int32).view(T, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, perm, slot = torch.empty(3, **i32), torch.empty(T, **i32), torch.empty((T, 1), **i32)
    rows = torch.empty_like(x)
    m.check(m.moe_sort_rows(0, T, 1, 2, d, x, idx, offsets, perm, slot, rows))
    assert offsets.tolist() == [0, T // 2, T]
    assert torch.equal(perm[:3].cpu(), torch.tensor([1, 3, 5], dtype=torch.int32))
    assert torch.equal(rows[:, 0], x[:, 0][perm.long()]) and torch.equal(rows[:, -1], x[:, -1][perm.long()])
    out = torch.empty_like(x)
    m.check(m.moe_unsort_rows(0, 0, T, 1, d, rows, slot, None, out))
    assert torch.equal(out, x)
    drows = torch.zeros_like(x)
    m.check(m.moe_unsort_rows_backward(0, 0, T, 1, d, x, None, slot, None, drows, None))
    assert torch.equal(drows, rows)


def test_sort_four_million_routes(m):
    """The most tokens, picks and experts: 262,144 x 16 over 256, a tenth dropped, against a stable sort by key."""
    T, k, E, d = 262144, 16, 256, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    idx[torch.rand((T, k), generator=g, device="cuda") < 0.1] = -1
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].expand(T, d).contiguous()
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, perm, slot = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty((T, k), **i32)
    rows = torch.full((T * k, d), -1.0, device="cuda")
    m.check(m.moe_sort_rows(m.MOE_F32, T, k, E, d, x, idx, offsets, perm, slot, rows))
    flat = idx.flatten().long()
    key = torch.where(flat >= 0, flat, E)
    order = key.argsort(stable=True)
    n = int((flat >= 0).sum())
    assert torch.equal(perm[:n].long(), order[:n]) and (perm[n:] == -1).all()
    assert torch.equal(offsets.long(), torch.searchsorted(key[order].contiguous(), torch.arange(E + 1, device="cuda")))
    want = torch.full((T * k,), -1, dtype=torch.int64, device="cuda")
    want[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(slot.flatten().long(), want)
    assert torch.equal(rows[:n, 0].long(), order[:n] // k) and (rows[n:] == -1).all()


@pytest.mark.parametrize("T,d", [(3000, 1024), (700, 6144), (400, 256)])
def test_sort_right_behind_the_writer_of_x(m, T, d):
    """One buffer of tokens, written anew on the device right before every sort of it, with no wait between: the rows are always
    the last tokens'."""
    g = torch.Generator(device="cuda").manual_seed(T)
    hs = [torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(5)]
    want = [torch.empty_like(h) for h in hs]
    for h, u in zip(hs, want):
        m.check(m.moe_norm_forward(m.MOE_NORM_RMS, 0, T, d, h, None, None, 1e-5, u))
    idx = torch.rand((T, 8), generator=g, device="cuda").argsort(1)[:, :2].to(torch.int32).contiguous()
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, perm, slot = torch.empty(9, **i32), torch.empty(2 * T, **i32), torch.empty((T, 2), **i32)
    x, rows = torch.empty_like(hs[0]), [torch.empty((2 * T, d), dtype=torch.bfloat16, device="cuda") for _ in range(40)]
    torch.cuda.synchronize()
    for turn, out in enumerate(rows):
        m.check(m.moe_norm_forward(m.MOE_NORM_RMS, 0, T, d, hs[turn % 5], None, None, 1e-5, x))
        m.check(m.moe_sort_rows(0, T, 2, 8, d, x, idx, offsets, perm, slot, out))
    at = perm.long() // 2
    for turn, out in enumerate(rows):
        assert torch.equal(out, want[turn % 5][at]), turn
