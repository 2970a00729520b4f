"""Few rows times 4-bit expert weights (moe_w4_pack, moe_w4_matvec) against the plain 64-bit form: both input types
and output types, all group sizes, one row to several passes, shapes that do not fill a block or a unit,
inputs split over warps and clusters, experts without rows; and the operators together as a layer."""
import math

import pytest
import torch

from tests import ops64
from tests.test_gpu_rows import DT, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mixture_experts_softmax_b200 as m
    return m


def weights(E, K, N, group, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-8, 8, (E, K, N), generator=g, dtype=torch.int8)
    s = (torch.randn((E, -(-K // group), N), generator=g) / (4 * math.sqrt(K))).to(torch.bfloat16)
    return q, s


def pack(m, q, s, group):
    E, K, N = q.shape
    p, check = guarded((m.moe_w4_packed_bytes(E, K, N, group),), torch.uint8, 77)
    m.check(m.moe_w4_pack(E, K, N, group, q.cuda(), s.cuda(), p), "moe_w4_pack")
    check()
    return p


def run(m, dt, out, x, offsets, packs, group, shape):
    E, K, N = shape
    R = x.shape[0]
    y, check = guarded((R, N), DT[out], 99.0)
    p = [pack(m, q, s, group) for q, s in packs] + [None]
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    m.check(m.moe_w4_matvec(dt, out, E, K, N, group, R, x.cuda(), off, p[0], p[1], y), "moe_w4_matvec")
    torch.cuda.synchronize()
    check()
    return y.cpu()


def check_rows(got, ref, tol):
    hit = ~ref.isnan().all(1)
    ops64.assert_close(got[hit], ref[hit], tol[hit], "y")
    assert (got[~hit] == 99.0).all(), "a row of no expert changed"


# (R, K, N): blocks and units that are not full, one unit, many splits, every operand count, several passes
SHAPES = [(1, 1, 1), (1, 128, 32), (1, 127, 31), (2, 6144, 512), (3, 333, 77), (7, 64, 4100), (8, 4096, 96), (9, 257, 64),
          (16, 1000, 200), (17, 2048, 40), (31, 130, 260), (32, 512, 128), (33, 384, 96), (70, 264, 50), (1, 20000, 33)]


@pytest.mark.parametrize("R,K,N", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt,out", [(0, 0), (1, 1), (0, 2), (1, 2)])
def test_matvec(m, R, K, N, group, dt, out):
    pk = weights(1, K, N, group, K + N)
    x = torch.randn((R, K), generator=torch.Generator().manual_seed(R)).to(DT[dt])
    ref, tol = ops64.w4(x, [0, R], [pk], group, DT[out])
    check_rows(run(m, dt, out, x, None, [pk], group, (1, K, N)), ref, tol)


@pytest.mark.parametrize("R,K,N", [(1, 128, 32), (2, 333, 77), (8, 2048, 520), (12, 130, 100), (40, 512, 64), (5, 9000, 48)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", [0, 1])
def test_gated(m, R, K, N, group, dt):
    packs = [weights(1, K, N, group, s) for s in (1, 2)]
    x = torch.randn((R, K), generator=torch.Generator().manual_seed(R)).to(DT[dt])
    ref, tol = ops64.w4(x, [0, R], packs, group, DT[dt])
    check_rows(run(m, dt, dt, x, None, packs, group, (1, K, N)), ref, tol)


OFFSETS = {"spread": [0, 2, 3, 9, 10], "empty": [0, 0, 5, 5, 10], "one": [0, 0, 0, 10, 10], "none": [0, 0, 0, 0, 0],
           "tail": [0, 1, 2, 3, 4], "behind": [2, 4, 4, 6, 8], "long": [0, 1, 34, 40, 40]}


@pytest.mark.parametrize("name", sorted(OFFSETS))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("group,K,N", [(128, 520, 72), (32, 2048, 256)])
def test_experts(m, name, gated, group, K, N):
    offsets = OFFSETS[name]
    R = max(10, offsets[-1] + (2 if name == "tail" else 0))
    packs = [weights(4, K, N, group, s) for s in range(2 if gated else 1)]
    x = torch.randn((R, K), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    ref, tol = ops64.w4(x, offsets, packs, group, torch.float32)
    check_rows(run(m, 0, 2, x, offsets, packs, group, (4, K, N)), ref, tol)


def test_offsets_are_clamped(m):
    """Row ranges outside [0, R] lose what lies outside; nothing is read or written there."""
    pk = weights(3, 256, 64, 64, 0)
    x = torch.randn((6, 256), generator=torch.Generator().manual_seed(0)).to(torch.float16)
    offsets = [-3, 2, 1, 2 ** 31 - 1]
    got = run(m, 1, 2, x, offsets, [pk], 64, (3, 256, 64))
    # row 1 lies in the ranges of experts 0 and 2: it gets either one's product, the others have one
    ref, tol = ops64.w4(x, offsets, [pk], 64, torch.float32)
    first, ftol = ops64.w4(x, [0, 2, 2, 2], [pk], 64, torch.float32)
    last = ((got[1].double() - ref[1]).abs() <= tol[1]).all()
    assert last or ((got[1].double() - first[1]).abs() <= ftol[1]).all()
    rest = [0, 2, 3, 4, 5]
    check_rows(got[rest], ref[rest], tol[rest])


def test_every_value_and_place(m):
    """Each weight of a small matrix is found again, exactly, by unit rows; values cover -8 .. 7."""
    for group, K, N in ((32, 160, 40), (64, 192, 33), (128, 129, 64)):
        q = (torch.arange(K * N).view(1, K, N) * 7 % 16 - 8).to(torch.int8)
        s = (1 + torch.arange(-(-K // group) * N).view(1, -1, N) % 128).to(torch.bfloat16)
        want = q[0].float() * s[0].float().repeat_interleave(group, 0)[:K]
        for at in range(0, K, 32):
            x = torch.zeros((min(32, K - at), K), dtype=torch.bfloat16)
            x[torch.arange(x.shape[0]), at + torch.arange(x.shape[0])] = 1
            got = run(m, 0, 2, x, None, [(q, s)], group, (1, K, N))
            assert torch.equal(got, want[at:at + 32])


def test_values_outside_the_range_are_refused(m):
    for bad in (-9, 8, 127, -128):
        q = torch.zeros((2, 40, 24), dtype=torch.int8)
        q[1, 39, 23] = bad
        s = torch.ones((2, 2, 24), dtype=torch.bfloat16)
        p = torch.empty(m.moe_w4_packed_bytes(2, 40, 24, 32), dtype=torch.uint8, device="cuda")
        assert m.moe_w4_pack(2, 40, 24, 32, q.cuda(), s.cuda(), p) == m.MOE_ERANGE
        q[1, 39, 23] = max(-8, min(7, bad))
        assert m.moe_w4_pack(2, 40, 24, 32, q.cuda(), s.cuda(), p) == m.MOE_OK


def test_nonfinite_inputs_stay_in_their_row(m):
    pk = weights(1, 300, 48, 64, 3)
    x = torch.randn((5, 300), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    clean, tol = ops64.w4(x, [0, 5], [pk], 64, torch.float32)
    x[1, 299] = float("nan")
    x[3, 0] = float("inf")
    got = run(m, 0, 2, x, None, [pk], 64, (1, 300, 48))
    keep = [0, 2, 4]
    ops64.assert_close(got[keep], clean[keep], tol[keep])
    assert got[1].isnan().all()
    # inf times a weight of 0 is nan, times any other an infinity of its sign
    w = pk[0][0, 0].double() * pk[1][0, 0].double()
    assert got[3][w == 0].isnan().all() and torch.equal(got[3][w != 0].double(), torch.sign(w[w != 0]) * math.inf)


def test_large_values(m):
    """fp16 inputs near the type's largest value: the sums are fp32."""
    pk = weights(1, 512, 64, 128, 8)
    x = torch.full((4, 512), 60000.0).to(torch.float16)
    x[::2] *= -1
    ref, tol = ops64.w4(x, [0, 4], [pk], 128, torch.float32)
    check_rows(run(m, 1, 2, x, None, [pk], 128, (1, 512, 64)), ref, tol)


def test_same_bits_every_time(m):
    pk = weights(8, 1024, 512, 64, 1)
    x = torch.randn((24, 1024), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    offsets = [0, 3, 3, 10, 11, 12, 20, 23, 24]
    a = run(m, 0, 2, x, offsets, [pk], 64, (8, 1024, 512))
    for _ in range(3):
        assert torch.equal(a, run(m, 0, 2, x, offsets, [pk], 64, (8, 1024, 512)))


def test_weights_beyond_2_gib(m):
    """Experts whose packed weights lie behind 2^31 bytes: 24 experts of 16384 x 12288 (2.4 GB)."""
    E, K, N, group = 24, 16384, 12288, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randint(-8, 8, (1, K, N), generator=g, device="cuda", dtype=torch.int8)
    p = torch.zeros(m.moe_w4_packed_bytes(E, K, N, group), dtype=torch.uint8, device="cuda")
    s = torch.full((1, K // group, N), 2.0 ** -6, dtype=torch.bfloat16, device="cuda")
    full_q = q.expand(E, K, N).contiguous()
    full_q[:E - 1] = 0
    m.check(m.moe_w4_pack(E, K, N, group, full_q, s.expand(E, -1, -1).contiguous(), p))
    del full_q
    x = torch.randint(-4, 5, (3, K), generator=g, device="cuda").to(torch.bfloat16)
    offsets = torch.tensor([0] * E + [3], dtype=torch.int32, device="cuda")
    y = torch.full((3, N), 99.0, device="cuda")
    m.check(m.moe_w4_matvec(m.MOE_BF16, m.MOE_F32, E, K, N, group, 3, x, offsets, p, None, y))
    want = (x.double() @ q[0].double()) * 2.0 ** -6    # whole numbers below 2^24: exact in fp32
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("scale", [2.0 ** 26, 2.0 ** 27, 2.0 ** 100, 2.0 ** -60, 2.0 ** -90])
@pytest.mark.parametrize("rows", [3, 20])
def test_bf16_inputs_of_any_size(m, scale, rows):
    """Inputs on both sides of the size from which on a phase takes the exact form, alone and mixed with ordinary ones
    in other places of the same rows (phases of 2048 inputs and fewer), and tiny ones."""
    K = 5000
    pk = weights(1, K, 96, 128, 21)
    x = torch.randn((rows, K), generator=torch.Generator().manual_seed(5))
    x[:, K // 3:K // 2] *= scale
    x[rows // 2] *= scale if scale < 2.0 ** 50 else 1
    x = x.to(torch.bfloat16)
    ref, tol = ops64.w4(x, [0, rows], [pk], 128, torch.float32)
    check_rows(run(m, 0, 2, x, None, [pk], 128, (1, K, 96)), ref, tol)


@pytest.mark.parametrize("power", [-98, -104, -110, -118])
@pytest.mark.parametrize("rows,group", [(3, 32), (5, 128), (20, 64)])
def test_tiny_bf16_inputs(m, power, rows, group):
    """Rows of nothing but bf16 inputs around 2^-100 and below: each group of inputs may be off by 2^-112 of its scale
    beside the usual roundings.  (A product is u x 2^-33 in steps of 2^-149: 9 additions of a group, each off by a step,
    make 9 * 2^-116.)"""
    K = 1000
    q, s = weights(1, K, 96, group, 23)
    x = (torch.randn((rows, K), generator=torch.Generator().manual_seed(6)) * 2.0 ** power).to(torch.bfloat16)
    ref, tol = ops64.w4(x, [0, rows], [(q, s)], group, torch.float32)
    tol = tol + s[0].double().abs().sum(0) * 2.0 ** -112
    check_rows(run(m, 0, 2, x, None, [(q, s)], group, (1, K, 96)), ref, tol)


def test_subnormal_inputs(m):
    """Subnormal fp16 inputs count like any others."""
    pk = weights(1, 256, 64, 32, 2)
    x = (torch.randn((4, 256), generator=torch.Generator().manual_seed(1)) * 2.0 ** -18).to(torch.float16)
    ref, tol = ops64.w4(x, [0, 4], [pk], 32, torch.float32)
    check_rows(run(m, 1, 2, x, None, [pk], 32, (1, 256, 64)), ref, tol)


@pytest.mark.parametrize("dt", [0, 1])
def test_weights_of_zero(m, dt):
    """Weights that are all 0, next to others: what is left of the inputs' sum is a rounding of it."""
    q, s = weights(1, 640, 64, 64, 2)
    q[:, :, ::2] = 0
    x = torch.randn((5, 640), generator=torch.Generator().manual_seed(1)).to(DT[dt])
    ref, tol = ops64.w4(x, [0, 5], [(q, s)], 64, torch.float32)
    assert (ref[:, ::2] == 0).all()
    check_rows(run(m, dt, 2, x, None, [(q, s)], 64, (1, 640, 64)), ref, tol)


def test_a_product_right_behind_another(m):
    """Products in a row on one stream, each reading what the one before wrote (a launch may begin before its
    predecessor has ended), give the same bits as with a wait between them."""
    d, f = 512, 2048
    up, down = pack(m, *weights(1, d, f, 64, 1), 64), pack(m, *weights(1, f, d, 64, 2), 64)
    x0 = torch.randn((6, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda() / 8

    def chain(wait):
        x, mid = x0.clone(), torch.empty((6, f), dtype=torch.bfloat16, device="cuda")
        for _ in range(8):
            for a, b, w, K, N in ((x, mid, up, d, f), (mid, x, down, f, d)):
                m.check(m.moe_w4_matvec(0, 0, 1, K, N, 64, 6, a, None, w, None, b))
                if wait:
                    torch.cuda.synchronize()
        return x
    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)


def test_few_rows_of_many_experts(m):
    """Rows at the first, some middle and the last of many experts; fewer rows than experts."""
    E, K, N = 70, 200, 96
    pk = weights(E, K, N, 64, 3)
    for at in ([0, 31, 69], [3, 32, 33], [69, 69, 69]):
        x = torch.randn((3, K), generator=torch.Generator().manual_seed(at[0])).to(torch.bfloat16)
        offsets = [sum(e < i for e in at) for i in range(E + 1)]
        ref, tol = ops64.w4(x, offsets, [pk], 64, torch.float32)
        assert not ref.isnan().any()
        check_rows(run(m, 0, 2, x, offsets, [pk], 64, (E, K, N)), ref, tol)


def test_ranges_that_overlap(m):
    """More ranges than rows: every row that lies in a range gets the product of one it lies in."""
    pk = weights(5, 96, 32, 32, 4)
    x = torch.randn((2, 96), generator=torch.Generator().manual_seed(0)).to(torch.float16)
    got = run(m, 1, 2, x, [0, 1, 0, 1, 0, 2], [pk], 32, (5, 96, 32))
    one, tol = ops64.w4(x, [0, 0, 0, 0, 0, 2], [pk], 32, torch.float32)
    ops64.assert_close(got[1:], one[1:], tol[1:])
    first = [ops64.w4(x, [0] * (e + 1) + [1] * (5 - e), [pk], 32, torch.float32) for e in (0, 2, 4)]
    assert any(((got[0].double() - r[0]).abs() <= t[0]).all() for r, t in first)


def test_most_rows_and_experts(m):
    """The largest row count, in 32-row passes over one expert; the largest expert count, a row each."""
    pk = weights(1, 160, 64, 32, 6)
    x = torch.randn((1024, 160), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    ref, tol = ops64.w4(x, [0, 1024], [pk], 32, torch.bfloat16)
    check_rows(run(m, 0, 0, x, None, [pk], 32, (1, 160, 64)), ref, tol)
    pk = weights(1024, 130, 34, 128, 7)
    ref, tol = ops64.w4(x[:, :130].contiguous(), list(range(1025)), [pk], 128, torch.float32)
    check_rows(run(m, 0, 2, x[:, :130].contiguous(), list(range(1025)), [pk], 128, (1024, 130, 34)), ref, tol)


@pytest.mark.parametrize("K,N", [(131072, 40), (40, 131072)])
def test_longest_sides(m, K, N):
    pk = weights(1, K, N, 128, 9)
    x = torch.randn((2, K), generator=torch.Generator().manual_seed(0)).to(torch.float16)
    ref, tol = ops64.w4(x, [0, 2], [pk], 128, torch.float32)
    check_rows(run(m, 1, 2, x, None, [pk], 128, (1, K, N)), ref, tol)


@pytest.mark.parametrize("offsets", [[0, 1, 0, 1, 0, 2], [0, 2, 1, 2, 0, 2], [1, 2, 0, 2, 0, 1], [-5, 1, -2 ** 31, 2 ** 31 - 1, 0, 2],
                                     [2, 0, 1, 0, 2, 2], [30, 38, 0, 40, 20, 40], [40, 3, 5, 0, 33, 1]])
@pytest.mark.parametrize("gated", [False, True])
def test_a_row_in_several_ranges_is_the_first_one_s(m, offsets, gated):
    """Offsets that go down and up again: a row that several ranges hold gets the first one's product, over all tiles of a wide
    product, and the same bits every time; a row that one range holds gets that one's."""
    E, R, K, N = 5, max(2, min(max(offsets), 40)), 500, 4100
    packs = [weights(E, K, N, 64, s) for s in (4, 5)[:1 + gated]]
    x = torch.randn((R, K), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    ref, tol = (torch.full((R, N), float("nan"), dtype=ops64.F8) for _ in range(2))
    for e in reversed(range(E)):   # the first range last
        lo, hi = max(offsets[e], 0), min(offsets[e + 1], R)
        if lo < hi:
            y, t = ops64.w4(x, [0] * e + [lo] + [hi] * (E - e), packs, 64, torch.float32)
            ref[lo:hi], tol[lo:hi] = y[lo:hi], t[lo:hi]
    got = [run(m, 0, 2, x, offsets, packs, 64, (E, K, N)) for _ in range(10)]
    check_rows(got[0], ref, tol)
    for again in got[1:]:
        assert torch.equal(again, got[0])


@pytest.mark.parametrize("power", [-90, -93, -96])
@pytest.mark.parametrize("rows,group", [(3, 32), (5, 128), (20, 64)])
def test_small_bf16_inputs_lose_nothing(m, power, rows, group):
    """Inputs between 2^-100 and some 2^power, whose products are subnormal sums in multiples of 2^-149: only the usual
    roundings.  A result of 0 would fail."""
    K = 1000
    q, s = weights(1, K, 96, group, 24)
    x = (torch.randn((rows, K), generator=torch.Generator().manual_seed(7)) * 2.0 ** power).to(torch.bfloat16)
    x = torch.where(x.abs() < 2.0 ** -100, 0, x)
    ref, tol = ops64.w4(x, [0, rows], [(q, s)], group, torch.float32)
    assert (tol < ref.abs() / 8).double().mean() > 0.9
    check_rows(run(m, 0, 2, x, None, [(q, s)], group, (1, K, 96)), ref, tol)
