"""Refusals of the stand-alone operators: bad sizes, types and pointers return their status on the host, before
any CUDA call (fake addresses are never dereferenced)."""
import pytest

A = 1 << 32   # fake, 16-byte aligned and far apart


def addr(i):
    return A * (i + 1)


@pytest.fixture(scope="module")
def m():
    import mixture_experts_softmax_b200 as m
    return m


def check_refusals(call, good, ok, einval, pointers, optional=()):
    """good: the arguments by name; einval: (name, bad value); pointers: names that must be present and aligned."""
    assert call(**good) in ok, call(**good)
    for name, bad in einval:
        assert call(**{**good, name: bad}) == -1, (name, bad)
    for name in pointers:
        if name not in optional:
            assert call(**{**good, name: None}) == -1, name
        assert call(**{**good, name: (good[name] or addr(40)) + 8}) == -1, name


@pytest.fixture(scope="module")
def ran(m):
    """What a well-formed call may say here: no device, or (on a GPU machine these fakes must not run) nothing."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the well-formed call of each test would run on the fake addresses")
    return (m.MOE_ENODEV,)


def test_sort_rows_refusals(m, ran):
    good = dict(dtype=m.MOE_BF16, T=4, k=2, E=8, d=64, x=addr(0), idx=addr(1), offsets=addr(2), perm=addr(3), slot=addr(4),
                rows=addr(5), stream=0)
    check_refusals(m.moe_sort_rows, good, ran,
                   [("dtype", 3), ("dtype", -1), ("T", -1), ("T", m.MOE_MAX_TOKENS + 1), ("k", 0), ("k", 17), ("E", 0), ("d", 0),
                    ("d", 65537), ("rows", addr(0) + 16), ("perm", addr(1)), ("slot", addr(3) + 16), ("offsets", addr(4)),
                    ("idx", addr(2) + 16), ("x", None), ("rows", None)],
                   ["x", "idx", "offsets", "perm", "slot", "rows"])
    assert m.moe_sort_rows(**{**good, "E": 257}) == m.MOE_EUNSUPPORTED
    assert m.moe_sort_rows(**{**good, "x": None, "rows": None}) in ran
    assert m.moe_sort_rows(**{**good, "T": 0, "offsets": None}) == m.MOE_EINVAL


def test_unsort_rows_refusals(m, ran):
    good = dict(rows_dtype=m.MOE_F32, dtype=m.MOE_BF16, T=4, k=2, d=64, rows=addr(0), slot=addr(1), gate=addr(2), out=addr(3),
                stream=0)
    check_refusals(m.moe_unsort_rows, good, ran,
                   [("rows_dtype", 9), ("dtype", 9), ("T", -1), ("k", 0), ("k", 17), ("d", 0), ("d", 65537), ("out", addr(0) + 16),
                    ("out", addr(1)), ("out", addr(2))],
                   ["rows", "slot", "gate", "out"], optional=("gate",))
    assert m.moe_unsort_rows(**{**good, "rows_dtype": m.MOE_F16}) == m.MOE_EUNSUPPORTED
    assert m.moe_unsort_rows(**{**good, "dtype": m.MOE_F32, "rows_dtype": m.MOE_BF16}) == m.MOE_EUNSUPPORTED
    assert m.moe_unsort_rows(**{**good, "T": 0, "rows": None}) == m.MOE_OK


def test_unsort_rows_backward_refusals(m, ran):
    good = dict(rows_dtype=m.MOE_BF16, dtype=m.MOE_BF16, T=4, k=2, d=64, dout=addr(0), rows=addr(1), slot=addr(2), gate=addr(3),
                drows=addr(4), dgate=addr(5), stream=0)
    check_refusals(m.moe_unsort_rows_backward, good, ran,
                   [("rows_dtype", 9), ("dtype", 9), ("T", -1), ("k", 17), ("d", 0), ("drows", addr(0)), ("drows", addr(1) + 16),
                    ("drows", addr(2)), ("drows", addr(3)), ("dgate", addr(3)), ("dgate", addr(0)), ("dgate", addr(4)),
                    ("rows", None)],
                   ["dout", "rows", "slot", "gate", "drows", "dgate"], optional=("gate", "dgate"))
    assert m.moe_unsort_rows_backward(**{**good, "rows": None, "dgate": None}) in ran
    assert m.moe_unsort_rows_backward(**{**good, "rows_dtype": m.MOE_F16}) == m.MOE_EUNSUPPORTED
    assert m.moe_unsort_rows_backward(**{**good, "T": 0, "dout": None}) == m.MOE_OK


def test_norm_refusals(m, ran):
    good = dict(kind=m.MOE_NORM_LAYER, dtype=m.MOE_F16, T=4, d=64, x=addr(0), gain=addr(1), bias=addr(2), eps=1e-5, y=addr(3),
                stats=addr(4), stream=0)
    check_refusals(m.moe_norm_forward, good, ran,
                   [("kind", 2), ("kind", -1), ("dtype", 5), ("T", -1), ("T", m.MOE_MAX_TOKENS + 1), ("d", 0), ("d", 65537),
                    ("eps", -1.0), ("eps", float("nan")), ("y", addr(0)), ("y", addr(1)), ("y", addr(2)), ("stats", addr(0)),
                    ("stats", addr(3)), ("stats", addr(1))],
                   ["x", "gain", "bias", "y", "stats"], optional=("gain", "bias", "stats"))
    assert m.moe_norm_forward(**{**good, "kind": m.MOE_NORM_RMS}) == m.MOE_EINVAL    # RMSNorm has no bias
    assert m.moe_norm_forward(**{**good, "kind": m.MOE_NORM_RMS, "bias": None}) in ran
    assert m.moe_norm_forward(**{**good, "T": 0, "x": None}) == m.MOE_OK


def test_norm_backward_refusals(m, ran):
    good = dict(kind=m.MOE_NORM_LAYER, dtype=m.MOE_BF16, T=4, d=64, x=addr(0), gain=addr(1), stats=addr(2), dy=addr(3), dx=addr(4),
                dgain=addr(5), dbias=addr(6), workspace=addr(7), stream=0)
    check_refusals(m.moe_norm_backward, good, ran,
                   [("kind", 2), ("dtype", 5), ("T", -1), ("d", 0), ("d", 65537), ("dx", addr(0)), ("dx", addr(3)), ("dx", addr(1)),
                    ("dx", addr(2)), ("dgain", addr(6)), ("dgain", addr(4)), ("dbias", addr(3)), ("workspace", addr(0)),
                    ("workspace", addr(5)), ("workspace", addr(4) + 16)],
                   ["x", "gain", "stats", "dy", "dx", "dgain", "dbias", "workspace"], optional=("gain", "dgain", "dbias"))
    assert m.moe_norm_backward(**{**good, "kind": m.MOE_NORM_RMS}) == m.MOE_EINVAL
    assert m.moe_norm_backward(**{**good, "dgain": None, "dbias": None}) in ran


def test_norm_workspace(m):
    assert m.moe_norm_workspace(-1, 64) == m.MOE_EINVAL
    assert m.moe_norm_workspace(4, 0) == m.MOE_EINVAL
    assert m.moe_norm_workspace(4, 65537) == m.MOE_EINVAL
    assert m.moe_norm_workspace(0, 64) == 0
    for d in (1, 64, 6144, 20000, 65536):
        sizes = [m.moe_norm_workspace(T, d) for T in (1, 8, 500, 8192, m.MOE_MAX_TOKENS)]
        assert sizes[0] >= 8 * d and sizes == sorted(sizes) and sizes[-1] <= 64 << 20


def test_tensor_arguments_are_checked(m):
    """The binding refuses tensors that the C side would misread."""
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.moe_norm_forward(m.MOE_NORM_RMS, m.MOE_BF16, 4, 64, x, None, None, 1e-5, x, None, 0)   # not on the GPU
    with pytest.raises(TypeError):
        m.moe_norm_forward(m.MOE_NORM_RMS, m.MOE_BF16, 4, 64, [1.0], None, None, 1e-5, x, None, 0)


def test_w4_refusals(m, ran):
    assert m.moe_w4_packed_bytes(0, 64, 64, 32) == m.MOE_EINVAL
    assert m.moe_w4_packed_bytes(1, 0, 64, 32) == m.MOE_EINVAL
    assert m.moe_w4_packed_bytes(1, 64, 131073, 32) == m.MOE_EINVAL
    assert m.moe_w4_packed_bytes(1, 64, 64, 48) == m.MOE_EUNSUPPORTED
    assert m.moe_w4_packed_bytes(1025, 64, 64, 32) == m.MOE_EUNSUPPORTED
    # half a byte a weight, two bytes a group's scale, and a tail
    assert m.moe_w4_packed_bytes(8, 6144, 32768, 128) - 8 * (6144 * 32768 // 2 + 48 * 32768 * 2) in range(0, 4096)
    good = dict(E=2, K=64, N=64, group=32, q=addr(0), scales=addr(1), packed=addr(2), stream=0)
    check_refusals(m.moe_w4_pack, good, ran, [("E", 0), ("K", 0), ("N", 0), ("packed", addr(0)), ("packed", addr(1) + 16)],
                   ["q", "scales", "packed"])
    assert m.moe_w4_pack(**{**good, "group": 256}) == m.MOE_EUNSUPPORTED


def test_w4_matvec_refusals(m, ran):
    good = dict(dtype=m.MOE_BF16, out_dtype=m.MOE_F32, E=2, K=64, N=64, group=32, R=3, x=addr(0), offsets=addr(1), packed=addr(2),
                packed_v=addr(3), y=addr(4), stream=0)
    check_refusals(m.moe_w4_matvec, good, ran,
                   [("dtype", 7), ("out_dtype", 7), ("E", 0), ("K", 0), ("N", 0), ("K", 131073), ("R", -1), ("y", addr(0)),
                    ("y", addr(1)), ("y", addr(2) + 16), ("y", addr(3)), ("offsets", None)],
                   ["x", "offsets", "packed", "packed_v", "y"], optional=("packed_v",))
    for name, bad in (("dtype", m.MOE_F32), ("out_dtype", m.MOE_F16), ("group", 16), ("R", 1025), ("E", 1025)):
        assert m.moe_w4_matvec(**{**good, name: bad}) == m.MOE_EUNSUPPORTED, name
    assert m.moe_w4_matvec(**{**good, "E": 1, "offsets": None, "packed_v": None}) in ran
    assert m.moe_w4_matvec(**{**good, "R": 0, "x": None}) == m.MOE_OK


def test_sort_rows_refuses_every_overlap(m, ran):
    """Each output against each input and each other output, from its first byte, from its end and from its middle."""
    good = dict(dtype=m.MOE_BF16, T=4, k=2, E=8, d=64, x=addr(0), idx=addr(1), offsets=addr(2), perm=addr(3), slot=addr(4),
                rows=addr(5), stream=0)
    size = dict(x=4 * 64 * 2, idx=4 * 2 * 4, offsets=9 * 4, perm=4 * 2 * 4, slot=4 * 2 * 4, rows=8 * 64 * 2)
    for out in ("offsets", "perm", "slot", "rows"):
        for other in set(size) - {out}:
            last = (size[other] - 1) // 16 * 16
            for at in {0, 16, last}:
                assert m.moe_sort_rows(**{**good, out: good[other] + at}) == m.MOE_EINVAL, (out, other, at)
            assert m.moe_sort_rows(**{**good, out: good[other] + (size[other] + 15) // 16 * 16}) in ran, (out, other)
    # the order alone has no rows to overlap
    assert m.moe_sort_rows(**{**good, "x": None, "rows": None, "d": 65536}) in ran


def test_norm_backward_refuses_overlaps_without_rows(m):
    """T == 0 still writes the gradients of gain and bias."""
    good = dict(kind=m.MOE_NORM_LAYER, dtype=m.MOE_BF16, T=0, d=64, x=None, gain=addr(0), stats=None, dy=None, dx=None, dgain=addr(1),
                dbias=addr(2), workspace=None, stream=0)
    for name in ("dgain", "dbias"):
        for at in (addr(0), addr(0) + 112, addr(3 - {"dgain": 1, "dbias": 2}[name]) + 240):
            assert m.moe_norm_backward(**{**good, name: at}) == m.MOE_EINVAL, (name, at)
