"""Sizes and refusals of the products grouped by expert and of the matrix-vector products with group
scales (no GPU): every argument is refused on the host, before the device is looked at."""
import ctypes
import shutil
import tempfile

import numpy as np
import pytest

from oracle import layer_oracle as lo
from oracle import q4g_oracle as qo
from tests import grouped_util as gu
from tests import test_m0_reservation as m0

mmq = pytest.importorskip("q4_q8_int8_amd")
torch = pytest.importorskip("torch")

P = 1 << 20       # a 16-byte aligned address that is never used
ODD = P + 4
BIG = 1 << 40


def test_group_bytes():
    # offsets 9 -> 12 words, order and place 6 -> 8 each; then, above 4096 pairs, chunks of 2048 x experts
    assert mmq.mmq_moe_group_bytes(3, 8, 2) == 4 * (12 + 8 + 8)
    assert mmq.mmq_moe_group_bytes(4097, 8, 1) == 4 * (12 + 2 * 4100 + 24)
    g = torch.zeros(12 + 8 + 8, dtype=torch.int32)
    g[:] = torch.arange(28)
    offsets, order, place = mmq.moe_groups(g, 3, 8, 2)
    assert offsets.tolist() == list(range(9))
    assert order.tolist() == list(range(12, 18)) and place.tolist() == list(range(20, 26))
    for bad in (g[:-1], g.float(), g[::2]):
        with pytest.raises(mmq.MMQArgumentError):
            mmq.moe_groups(bad, 3, 8, 2)


CALLS = {
    "group": lambda M, E, k: ("mmq_moe_group", M, E, k, P, P, None),
    "grouped": lambda M, E, k: ("mmq_q4K_grouped", M, E, k, 64, 256, P, 0, P, P, P, P, 0, None),
    "gated": lambda M, E, k: ("mmq_q4K_grouped_gated", M, E, k, 64, 256, P, P, P, P, P, 2, None),
    "down": lambda M, E, k: ("mmq_q4K_grouped_down", M, E, k, 64, 256, P, P, P, P, None, P, P, BIG,
                             None),
    "moe": lambda M, E, k: ("mmq_q4K_grouped_moe", M, E, k, 256, 256, P, P, 0, 1, P, 2, P, None, P, P,
                            BIG, None),
}


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("args,status", [
    ((0, 8, 2), mmq.MMQ_E_ARG), ((1, 0, 2), mmq.MMQ_E_ARG), ((1, 8, 0), mmq.MMQ_E_ARG),
    ((-1, 8, 2), mmq.MMQ_E_ARG), ((1, 8, 9), mmq.MMQ_E_SHAPE), ((1, 513, 2), mmq.MMQ_E_SHAPE),
    ((1, 512, 65), mmq.MMQ_E_SHAPE), ((1 << 21, 8, 2), mmq.MMQ_E_SHAPE),
    ((1 << 62, 8, 8), mmq.MMQ_E_SHAPE),
])
def test_group_limits(call, args, status):
    assert mmq.raw_call(*CALLS[call](*args)) == status


@pytest.mark.parametrize("call,ptrs", [("group", (4, 5)), ("grouped", (6, 8, 9, 10, 11)),
                                       ("gated", (6, 7, 8, 9, 10)), ("down", (6, 7, 8, 9, 11, 12)),
                                       ("moe", (6, 7, 10, 12, 14, 15))])
def test_pointers(call, ptrs):
    good = list(CALLS[call](100, 8, 2))
    for i in ptrs:
        for bad in (None, ODD):
            a = list(good)
            a[i] = bad
            assert mmq.raw_call(*a) == mmq.MMQ_E_ARG, i


def test_residual_must_be_aligned():
    for call, i in (("down", 10), ("moe", 13)):
        a = list(CALLS[call](100, 8, 2))
        a[i] = ODD
        assert mmq.raw_call(*a) == mmq.MMQ_E_ARG


@pytest.mark.parametrize("call", ["grouped", "gated", "down"])
@pytest.mark.parametrize("i,v,status", [
    (4, 0, mmq.MMQ_E_ARG), (5, 0, mmq.MMQ_E_ARG), (5, -256, mmq.MMQ_E_ARG),
    (5, 300, mmq.MMQ_E_SHAPE), (5, (1 << 24) + 256, mmq.MMQ_E_SHAPE),
    (4, (1 << 30) + 1, mmq.MMQ_E_SHAPE), (5, 1 << 24, mmq.MMQ_E_SHAPE)])
def test_product_sizes(call, i, v, status):
    a = list(CALLS[call](200, 8, 2))   # 200 x 2^24 values are 2^31 or more
    a[i] = v
    assert mmq.raw_call(*a) == status


def test_grids_stay_below_2_to_the_32_work_items():
    a = list(CALLS["grouped"](1 << 20, 512, 2))   # 2^16 + 512 tiles
    a[4] = 256 * 128                              # by 128 weight-tile groups
    assert mmq.raw_call(*a) == mmq.MMQ_E_SHAPE
    a = list(CALLS["down"](1 << 20, 8, 1))
    a[4] = 16 * 256                               # 2^24 workgroups of the weighted sum
    assert mmq.raw_call(*a) == mmq.MMQ_E_SHAPE


def test_every_forms_grid_stays_below_2_to_the_32_work_items():
    """At the largest products that the calls take, whatever form is chosen; workgroups come in eights."""
    tile = {"wide": (128, 256, 512), "narrow": (32, 128, 256), "split2": (32, 128, 512),
            "split4": (32, 128, 1024)}
    for P in (1, 40, 512, 5000, 100000, 1 << 21):
        for E in (1, 7, 64, 512):
            most = P // 32 + min(E, P)
            for K in (256, 4096, 1 << 18, 1 << 24):
                for share in (1, 2, 16, 300, 3000):
                    N = min(((1 << 23) - 4097) // share // most * 256, 1 << 30)
                    if N == 0:
                        continue
                    rows, cols, threads = tile[gu.grouped_form(P, E, N, K)]
                    grid = (P // rows + min(E, P)) * -(-N // cols)
                    grid = (grid + 7) // 8 * 8 + (256 if rows == 128 else 0)   # and a round more
                    assert grid * threads < 2 ** 32, (P, E, N, K)


@pytest.mark.parametrize("call,i,v", [
    ("grouped", 7, 2), ("grouped", 7, -1), ("grouped", 12, 5), ("grouped", 12, -1),
    ("gated", 11, 5), ("gated", 11, -1), ("moe", 8, 2), ("moe", 9, 2), ("moe", 11, 7)])
def test_options(call, i, v):
    a = list(CALLS[call](100, 8, 2))
    a[i] = v
    assert mmq.raw_call(*a) == mmq.MMQ_E_ARG


def test_workspaces_are_checked():
    need = mmq.mmq_grouped_down_workspace_bytes(100, 8, 2, 64, 256)
    a = list(CALLS["down"](100, 8, 2))
    a[13] = need - 1
    assert mmq.raw_call(*a) == mmq.MMQ_E_ARG and str(need) in mmq.mmq_last_error()
    need = mmq.mmq_grouped_moe_workspace_bytes(100, 8, 2, 256, 256)
    a = list(CALLS["moe"](100, 8, 2))
    a[16] = need - 1
    assert mmq.raw_call(*a) == mmq.MMQ_E_ARG and str(need) in mmq.mmq_last_error()
    # H in q8_1 and the pairs' products
    assert need > mmq.mmq_q8_1_bytes(200, 256) + 4 * 200 * 256
    for fn in ("mmq_moe_group_bytes", "mmq_grouped_down_workspace_bytes",
               "mmq_grouped_moe_workspace_bytes"):
        sizes = (100, 8, 2) if fn == "mmq_moe_group_bytes" else (100, 8, 2, 256, 256)
        assert mmq.raw_call(fn, *sizes, None) == mmq.MMQ_E_ARG


# ---------------------------------------------------------------- group scales

def fmt(group=64, scale=None, zeros=1, reserved=0):
    return mmq.mmq_q4G_format(group, mmq.MMQ_F16 if scale is None else scale, zeros, reserved)


def q4g(M=1, N=64, K=256, xt=1, x=P, w=P, f=None, yt=1, y=P, epi=None):
    f = fmt() if f is None else f
    return mmq.raw_call("mmq_q4G", M, N, K, xt, x, w, ctypes.byref(f) if f else None, yt, y, epi,
                        None)


def test_q4g_bytes():
    # 3 tiles of 16 rows by 3 records of 128 values, each with 1024 bytes of values and, per row, one
    # 16-bit scale per 32 values, per 64 or per record, and as many zeros
    for group, scales in ((32, 4), (64, 2), (96, 4), (128, 1), (160, 4), (256, 1), (288, 1),
                          (1 << 20, 1)):
        for zeros in (0, 1):
            assert mmq.mmq_q4G_repacked_bytes(35, 288, fmt(group, zeros=zeros)) == (
                9 * (1024 + 32 * scales * (1 + zeros)))


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), mmq.MMQ_E_ARG), (dict(N=0), mmq.MMQ_E_ARG), (dict(K=0), mmq.MMQ_E_ARG),
    (dict(M=17), mmq.MMQ_E_SHAPE), (dict(K=48), mmq.MMQ_E_SHAPE),
    (dict(K=(1 << 24) + 32), mmq.MMQ_E_SHAPE), (dict(N=(1 << 25) + 1), mmq.MMQ_E_SHAPE),
    (dict(N=1 << 25, K=1 << 12), mmq.MMQ_E_SHAPE),
    (dict(xt=3), mmq.MMQ_E_ARG), (dict(xt=-1), mmq.MMQ_E_ARG), (dict(yt=3), mmq.MMQ_E_ARG),
    (dict(x=None), mmq.MMQ_E_ARG), (dict(x=ODD), mmq.MMQ_E_ARG), (dict(w=None), mmq.MMQ_E_ARG),
    (dict(w=ODD), mmq.MMQ_E_ARG), (dict(y=None), mmq.MMQ_E_ARG), (dict(y=ODD), mmq.MMQ_E_ARG),
    (dict(f=False), mmq.MMQ_E_ARG), (dict(f=fmt(0)), mmq.MMQ_E_ARG),
    (dict(f=fmt(-32)), mmq.MMQ_E_ARG), (dict(f=fmt(48)), mmq.MMQ_E_SHAPE),
    (dict(f=fmt(scale=0)), mmq.MMQ_E_ARG), (dict(f=fmt(scale=3)), mmq.MMQ_E_ARG),
    (dict(f=fmt(zeros=2)), mmq.MMQ_E_ARG), (dict(f=fmt(reserved=1)), mmq.MMQ_E_ARG),
])
def test_q4g_refusals(kw, status):
    assert q4g(**kw) == status, mmq.mmq_last_error()


@pytest.mark.parametrize("e", [(ODD, None, 0, 0), (None, ODD, 0, 0), (None, None, 5, 0),
                               (None, None, -1, 0), (None, None, 0, 1)])
def test_q4g_epilogue_refusals(e):
    assert q4g(epi=ctypes.byref(mmq.mmq_q4G_epilogue(*e))) == mmq.MMQ_E_ARG


def test_repack_q4g_refusals():
    def call(w=P, s=P, z=P, N=64, K=256, f=None, rep=P):
        return mmq.raw_call("repack_q4_G", w, s, z, N, K, ctypes.byref(f or fmt()), rep, None)
    for kw in (dict(w=None), dict(w=ODD), dict(s=None), dict(s=ODD), dict(z=None), dict(z=ODD),
               dict(rep=None), dict(rep=ODD), dict(f=fmt(zeros=0)), dict(N=0)):
        assert call(**kw) == mmq.MMQ_E_ARG, kw
    assert call(K=100) == mmq.MMQ_E_SHAPE
    assert mmq.raw_call("mmq_q4G_repacked_bytes", 64, 256, ctypes.byref(fmt()),
                        None) == mmq.MMQ_E_ARG


def test_q4g_format_takes_16_bit_scales():
    assert mmq.q4G_format(64, torch.bfloat16, False).scale_type == mmq.MMQ_BF16
    for bad in (torch.float32, torch.int8, None):
        with pytest.raises(mmq.MMQArgumentError):
            mmq.q4G_format(64, bad, True)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses here are not real")
def test_well_formed_calls_reach_the_device_check():
    for call in CALLS:
        assert mmq.raw_call(*CALLS[call](1000, 8, 2)) == mmq.MMQ_E_DEVICE, call
    assert q4g(M=16, K=224, f=fmt(1000, mmq.MMQ_BF16, 0)) == mmq.MMQ_E_DEVICE
    assert q4g(xt=0, yt=2, epi=ctypes.byref(mmq.mmq_q4G_epilogue(P, P, 4, 0))) == mmq.MMQ_E_DEVICE


@pytest.mark.parametrize("fn,args", [
    ("mmq_moe_group", "M 8 2 ids groups"), ("mmq_q4K_grouped", "M 8 2 64 256 x g w C q8"),
    ("mmq_q4K_grouped_gated", "M 8 2 64 256 x g w H q8"),
    ("mmq_q4K_grouped_down", "M 8 2 64 256 H g weights w out ws"),
    ("mmq_q4K_grouped_moe", "M 8 2 256 256 x logits w w out ws")])
def test_calls_check_buffers_against_the_size_of_the_call(fn, args, monkeypatch):
    class Seen(Exception):
        pass

    def first(t, name, nbytes, *a, **kw):
        raise Seen(nbytes)

    monkeypatch.setattr(mmq, "_dev", first)

    def size(M):
        with pytest.raises(Seen) as e:
            getattr(mmq, fn)(*(M if a == "M" else int(a) if a.isdigit() else a
                               for a in args.split()))
        return e.value.args[0]

    assert size(400) > size(4) > 0
    M = torch.tensor(4)
    assert size(M) == size(np.array(4)) == size(4)
    M *= 100
    assert size(M) == size(400)


@pytest.mark.skipif(not m0.os.path.exists(m0.build.HIPCC), reason="hipcc not found")
@pytest.mark.parametrize("source", ["grouped.hip", "q4g.hip"])
def test_compiler_leaves_m0_to_the_loads_into_lds(source):
    tmp = tempfile.mkdtemp(prefix="m0_check_")
    try:
        path = m0.assembly(source, tmp)
        assert "buffer_load_dwordx4" in open(path).read()
        assert not m0.compiler_m0_uses(path)
    finally:
        shutil.rmtree(tmp, ignore_errors=True)


# ---------------------------------------------------------------- the oracle by hand

def test_groups_by_hand():
    ids = np.array([[2, 0], [2, -1], [7, 2]])       # 7 is outside E = 4
    offsets, order, place = lo.groups(ids, 4)
    assert offsets.tolist() == [0, 1, 1, 4, 4]
    assert order.tolist() == [1, 0, 2, 5, -1, -1]
    assert place.tolist() == [1, 0, 2, -1, -1, 3]


def test_q4g_by_hand():
    # one row of four values 1, 15, 0, 9 in groups of two: bytes 0xF1, 0x90
    w = np.array([[0xF1, 0x90]], np.uint8)
    assert qo.values(w).tolist() == [[1, 15, 0, 9]]
    x = np.array([[1.0, -2.0, 3.0, 0.5]])
    y, T = qo.product(x, w, np.array([[0.5, 2.0]]), np.array([[3.0, 0.5]]), 2)
    # 0.5 (1*(1-3) - 2*(15-3)) + 2 (3*(0-0.5) + 0.5*(9-0.5)) = -13 + 5.5
    assert y.tolist() == [[-7.5]]
    assert T.tolist() == [[0.5 * (4 + 36) + 2 * (1.5 + 4.75)]]
    y, _ = qo.product(x, w, np.array([[0.5, 2.0]]), None, 2)
    assert y.tolist() == [[0.5 * (-7 - 14) + 2 * (-24 + 0.5)]]
