"""The layer operators' entry points on the host (CPU only): sizes, refusals, and that a
well-formed call gets as far as the device check."""
import ctypes
import glob
import importlib
import os
import shutil
import tempfile

import numpy as np
import pytest
import torch

mmq = pytest.importorskip("q4_q8_int8_amd")
m0 = importlib.import_module("tests.test_m0_reservation")

P = 1 << 20        # a 16-byte aligned address that nothing reads: the checks end before the device
ODD = P + 4


def test_sizes():
    assert mmq.mmq_q4K_pair_bytes(1, 256) == 4608
    assert mmq.mmq_q4K_pair_bytes(16, 256) == 4608
    assert mmq.mmq_q4K_pair_bytes(17, 512) == 2 * 2 * 4608
    assert mmq.mmq_q4K_pair_bytes(11008, 4096) == 2 * mmq.mmq_q4K_repacked_bytes(11008, 4096)
    assert mmq.mmq_moe_plan_bytes(1, 64, 8) == 4 * (4 + 4 * 8 + 8)
    assert mmq.mmq_moe_plan_bytes(64, 8, 8) == 4 * (4 + 4 * 8 + 512)
    assert mmq.mmq_gated_workspace_bytes(1, 11008, 4096) == 0
    assert (mmq.mmq_gated_workspace_bytes(300, 1376, 4096)
            == mmq.mmq_workspace_bytes(300, 2752, 4096))


def test_layer_workspace_holds_its_parts():
    M, E, k, D, F = 3, 16, 4, 512, 768
    n = mmq.mmq_moe_workspace_bytes(M, E, k, D, F)
    parts = (4 * M * k * 2 + mmq.mmq_moe_plan_bytes(M, E, k) + 4 * M * k * F
             + max(mmq.mmq_q8_1_bytes(M, D), mmq.mmq_q8_1_bytes(M * k, F)))
    assert parts <= n <= parts + 6 * 256 and n % 256 == 0


def _size(fn, *args):
    n = ctypes.c_size_t()
    return mmq.raw_call(fn, *args, ctypes.byref(n))


@pytest.mark.parametrize("fn,args,status", [
    ("mmq_q4K_pair_bytes", (0, 256), mmq.MMQ_E_ARG),
    ("mmq_q4K_pair_bytes", (16, 100), mmq.MMQ_E_SHAPE),
    ("mmq_q4K_pair_bytes", ((1 << 29) + 1, 256), mmq.MMQ_E_SHAPE),
    ("mmq_gated_workspace_bytes", (4, 0, 256), mmq.MMQ_E_ARG),
    ("mmq_gated_workspace_bytes", (4, 64, 128), mmq.MMQ_E_SHAPE),
    ("mmq_moe_plan_bytes", (0, 8, 2), mmq.MMQ_E_ARG),
    ("mmq_moe_plan_bytes", (65, 8, 2), mmq.MMQ_E_SHAPE),
    ("mmq_moe_plan_bytes", (64, 64, 9), mmq.MMQ_E_SHAPE),
    ("mmq_moe_plan_bytes", (1, 513, 2), mmq.MMQ_E_SHAPE),
    ("mmq_moe_plan_bytes", (1, 4, 5), mmq.MMQ_E_SHAPE),
    ("mmq_moe_plan_bytes", (1, 128, 65), mmq.MMQ_E_SHAPE),
    ("mmq_moe_workspace_bytes", (1, 8, 2, 300, 256), mmq.MMQ_E_SHAPE),
    ("mmq_moe_workspace_bytes", (1, 8, 2, 256, 300), mmq.MMQ_E_SHAPE),
    ("mmq_moe_workspace_bytes", (1, 8, 2, 256, -256), mmq.MMQ_E_ARG),
])
def test_size_errors(fn, args, status):
    assert _size(fn, *args) == status
    assert mmq.mmq_last_error()
    assert mmq.raw_call(fn, *args, None) == mmq.MMQ_E_ARG


def _epi(bias=0, residual=0, act=0, reserved=0):
    return ctypes.byref(mmq.mmq_epilogue(bias or None, residual or None, act, reserved))


@pytest.mark.parametrize("epi,status", [
    (dict(act=5), mmq.MMQ_E_ARG), (dict(act=-1), mmq.MMQ_E_ARG),
    (dict(reserved=1), mmq.MMQ_E_ARG), (dict(bias=ODD), mmq.MMQ_E_ARG),
    (dict(residual=ODD), mmq.MMQ_E_ARG),
])
def test_bad_epilogues(epi, status):
    assert mmq.raw_call("mmq_q4K_q8_1_epilogue", 4, 64, 256, P, P, P, None, _epi(**epi),
                        None) == status
    assert mmq.raw_call("mmq_q4K_f32_epilogue", 4, 64, 256, P, P, P, None, _epi(**epi)) == status


EPI = ("mmq_q4K_q8_1_epilogue", "mmq_q4K_f32_epilogue")


@pytest.mark.parametrize("args,status", [
    ((0, 64, 256, P, P, P), mmq.MMQ_E_ARG), ((4, 64, 100, P, P, P), mmq.MMQ_E_SHAPE),
    ((4, 64, 256, 0, P, P), mmq.MMQ_E_ARG), ((4, 64, 256, P, 0, P), mmq.MMQ_E_ARG),
    ((4, 64, 256, P, P, 0), mmq.MMQ_E_ARG), ((4, 64, 256, ODD, P, P), mmq.MMQ_E_ARG),
])
def test_epilogue_calls_check_the_product(args, status):
    m, n, k, *ptrs = args
    ptrs = [p or None for p in ptrs]
    assert mmq.raw_call(EPI[0], m, n, k, *ptrs, None, _epi(act=1), None) == status
    assert mmq.raw_call(EPI[1], m, n, k, *ptrs, None, _epi(act=1)) == status
    assert mmq.raw_call("mmq_q4K_q8_1_gated", m, n, k, *ptrs, None, 2, None) == status
    assert mmq.raw_call("mmq_q4K_f32_gated", m, n, k, *ptrs, None, 2) == status


def test_f32_forms_are_for_few_tokens():
    assert mmq.raw_call(EPI[1], 129, 64, 256, P, P, P, None, None) == mmq.MMQ_E_SHAPE
    assert mmq.raw_call("mmq_q4K_f32_gated", 129, 64, 256, P, P, P, None, 2) == mmq.MMQ_E_SHAPE
    assert "mmq_q4K_f32_gated" in mmq.mmq_last_error()


@pytest.mark.parametrize("act", [-1, 5])
def test_gated_bad_act(act):
    assert mmq.raw_call("mmq_q4K_q8_1_gated", 4, 64, 256, P, P, P, None, act,
                        None) == mmq.MMQ_E_ARG
    assert mmq.raw_call("mmq_q4K_f32_gated", 4, 64, 256, P, P, P, None, act) == mmq.MMQ_E_ARG
    assert mmq.raw_call("mmq_q4K_moe_gated", 4, 8, 2, 64, 256, P, P, P, P, P, act,
                        None) == mmq.MMQ_E_ARG


def test_workspace_of_the_gated_product():
    """A split's second kernel is counted, so K is split at most where the plain product's is."""
    for M, F, K in ((77, 688, 4096), (300, 1376, 4096), (20, 1376, 4096), (512, 512, 11008)):
        assert (mmq.mmq_gated_workspace_bytes(M, F, K)
                <= mmq.mmq_workspace_bytes(M, 32 * ((F + 15) // 16), K))
    assert mmq.mmq_gated_workspace_bytes(77, 688, 4096) == 0


def test_pairs_to_tokens_by_multiplication():
    """The kernels' p / k, (p * (65535 // k + 1)) >> 16, for every pair of every plan."""
    for k in range(1, mmq.MOE_MAX_SLOTS + 1):
        m = 65535 // k + 1
        assert all((p * m) >> 16 == p // k for p in range(mmq.MOE_MAX_PAIRS)), k


def test_gated_experts_grid_limit():
    # 8 experts, ceil(F/16) = 2^20: 2^23 in all
    a = [4, 8, 2, 1 << 24, 256, P, P, P, P, P, 2, None]
    assert mmq.raw_call("mmq_q4K_moe_gated", *a) == mmq.MMQ_E_SHAPE


def test_epilogue_options_are_checked():
    o = mmq.mmq_options(99, 0, 0, None, 0, 0, 0)
    assert mmq.raw_call(EPI[0], 4, 64, 256, P, P, P, None, _epi(act=1),
                        ctypes.byref(o)) == mmq.MMQ_E_ARG
    o = mmq.mmq_options(0, 0, 0, ODD, 64, 0, 0)
    assert mmq.raw_call("mmq_q4K_q8_1_gated", 4, 64, 256, P, P, P, None, 2,
                        ctypes.byref(o)) == mmq.MMQ_E_ARG


@pytest.mark.parametrize("args,status", [
    ((0, 8, 2), mmq.MMQ_E_ARG), ((1, 0, 2), mmq.MMQ_E_ARG), ((1, 8, 0), mmq.MMQ_E_ARG),
    ((1, 8, 9), mmq.MMQ_E_SHAPE), ((1, 600, 2), mmq.MMQ_E_SHAPE), ((65, 8, 2), mmq.MMQ_E_SHAPE),
    ((60, 64, 10), mmq.MMQ_E_SHAPE),
])
def test_routing_limits(args, status):
    M, E, k = args
    assert mmq.raw_call("mmq_moe_route", M, E, k, P, 0, 1, P, P, P, None) == status
    assert mmq.raw_call("mmq_moe_plan", M, E, k, P, P, None) == status
    assert mmq.raw_call("mmq_q4K_moe_gated", M, E, k, 64, 256, P, P, P, P, P, 2, None) == status
    assert mmq.raw_call("mmq_q4K_moe_down", M, E, k, 64, 256, P, P, P, P, None, P, P,
                        None) == status
    assert mmq.raw_call("mmq_q4K_moe", M, E, k, 256, 256, P, P, 0, 1, P, 2, P, None, P, P, 1 << 40,
                        None) == status


def test_routing_pointers_and_options():
    for i in range(3):
        ptrs = [P, P, P]
        for bad in (None, ODD):
            ptrs[i] = bad
            assert mmq.raw_call("mmq_moe_route", 1, 8, 2, ptrs[0], 0, 1, ptrs[1], ptrs[2], P,
                                None) == mmq.MMQ_E_ARG
    assert mmq.raw_call("mmq_moe_route", 1, 8, 2, P, 0, 1, P, P, ODD, None) == mmq.MMQ_E_ARG
    assert mmq.raw_call("mmq_moe_route", 1, 8, 2, P, 2, 1, P, P, P, None) == mmq.MMQ_E_ARG
    assert mmq.raw_call("mmq_moe_route", 1, 8, 2, P, 0, 2, P, P, P, None) == mmq.MMQ_E_ARG
    assert mmq.raw_call("mmq_moe_plan", 1, 8, 2, None, P, None) == mmq.MMQ_E_ARG
    assert mmq.raw_call("mmq_moe_plan", 1, 8, 2, P, ODD, None) == mmq.MMQ_E_ARG


def test_expert_products_check_shapes_and_pointers():
    gated = [4, 8, 2, 64, 256, P, P, P, P, P, 2, None]
    down = [4, 8, 2, 64, 256, P, P, P, P, P, P, P, None]
    for fn, good, ptrs in (("mmq_q4K_moe_gated", gated, range(5, 10)),
                           ("mmq_q4K_moe_down", down, (5, 6, 7, 8, 10, 11))):
        for i in ptrs:
            for bad in (None, ODD):
                a = list(good)
                a[i] = bad
                assert mmq.raw_call(fn, *a) == mmq.MMQ_E_ARG
        for i, v, status in ((3, 0, mmq.MMQ_E_ARG), (4, 0, mmq.MMQ_E_ARG),
                             (4, 300, mmq.MMQ_E_SHAPE), (4, (1 << 24) + 256, mmq.MMQ_E_SHAPE),
                             (3, (1 << 30) + 1, mmq.MMQ_E_SHAPE)):
            a = list(good)
            a[i] = v
            assert mmq.raw_call(fn, *a) == status
    a = list(down)
    a[9] = ODD                                     # residual
    assert mmq.raw_call("mmq_q4K_moe_down", *a) == mmq.MMQ_E_ARG
    # 512 pairs of 2^23 values: 2^32 of them
    assert mmq.raw_call("mmq_q4K_moe_down", 64, 8, 8, 64, 1 << 23, P, P, P, P, None, P, P,
                        None) == mmq.MMQ_E_SHAPE


def test_grids_stay_below_2_to_the_32_work_items():
    assert mmq.raw_call("mmq_moe_route", (1 << 25) + 1, 1, 1, P, 0, 1, P, P, None,
                        None) == mmq.MMQ_E_SHAPE
    assert mmq.raw_call("mmq_q4K_moe_down", 1, 1, 1, (1 << 25) + 1, 256, P, P, P, P, None, P, P,
                        None) == mmq.MMQ_E_SHAPE
    # 2^24 records of 256 work-items
    assert mmq.raw_call("repack_q4_K_pair", P, P, 1 << 28, 256, P, None) == mmq.MMQ_E_SHAPE
    assert mmq.raw_call("mmq_q4K_moe_gated", 1, 1, 1, 1 << 27, 256, P, P, P, P, P, 2,
                        None) == mmq.MMQ_E_SHAPE


def test_layer_checks_its_workspace():
    need = mmq.mmq_moe_workspace_bytes(2, 8, 2, 256, 256)
    call = [2, 8, 2, 256, 256, P, P, 0, 1, P, 2, P, None, P, P, need - 1, None]
    assert mmq.raw_call("mmq_q4K_moe", *call) == mmq.MMQ_E_ARG
    assert str(need) in mmq.mmq_last_error()
    call[15] = need
    call[14] = ODD
    assert mmq.raw_call("mmq_q4K_moe", *call) == mmq.MMQ_E_ARG


@pytest.mark.skipif(mmq.torch.cuda.is_available(), reason="the addresses here are not real")
def test_well_formed_calls_reach_the_device_check():
    need = mmq.mmq_moe_workspace_bytes(2, 8, 2, 256, 256)
    for fn, *args in (
            (EPI[0], 4, 64, 256, P, P, P, None, _epi(P, P, 2), None),
            (EPI[0], 4, 64, 256, P, P, P, None, None, None),
            (EPI[1], 4, 64, 256, P, P, P, None, _epi(P, P, 2)),
            ("repack_q4_K_pair", P, P, 20, 256, P, None),
            ("mmq_q4K_q8_1_gated", 4, 20, 256, P, P, P, None, 2, None),
            ("mmq_q4K_f32_gated", 4, 20, 256, P, P, P, None, 2),
            ("mmq_moe_plan", 1, 8, 2, P, P, None),
            ("mmq_moe_route", 1 << 20, 8, 2, P, 0, 1, P, P, None, None),
            ("mmq_q4K_moe_gated", 4, 8, 2, 20, 256, P, P, P, P, P, 2, None),
            ("mmq_q4K_moe_down", 4, 8, 2, 20, 256, P, P, P, P, None, P, P, None),
            ("mmq_q4K_moe", 2, 8, 2, 256, 256, P, P, 0, 1, P, 2, P, None, P, P, need, None)):
        assert mmq.raw_call(fn, *args) == mmq.MMQ_E_DEVICE, (fn, mmq.mmq_last_error())


def test_python_names_match_the_header():
    names = set(mmq.exported_symbols())
    assert {"mmq_q4K_moe", "mmq_moe_route", "mmq_q4K_q8_1_gated", "mmq_q4K_f32_epilogue"} <= names
    for n in names - {"mmq_status_str", "mmq_last_error", "mmq_last_kernel"}:
        assert callable(getattr(mmq, n)), n
    for path in glob.glob(os.path.join(mmq.INCLUDE_DIR, "*.h")):
        assert path in mmq.HEADER_PATHS


@pytest.mark.skipif(not os.path.exists(m0.build.HIPCC), reason="hipcc not found")
def test_compiler_leaves_m0_to_the_loads_in_the_experts_products():
    tmp = tempfile.mkdtemp(prefix="m0_check_")
    try:
        path = m0.assembly("moe.hip", tmp)
        assert "buffer_load_dwordx4" in open(path).read()
        assert not m0.compiler_m0_uses(path)
    finally:
        shutil.rmtree(tmp, ignore_errors=True)


@pytest.mark.parametrize("M", [np.array(4), np.int64(4), torch.tensor(4), True, 4])
def test_sizes_of_integers_of_any_kind(M):
    """Whatever a size query takes as an integer, the wrappers take too."""
    assert mmq._sized(mmq.mmq_q8_1_bytes, M, 256) == mmq.mmq_q8_1_bytes(int(M), 256)


def test_sizes_follow_an_integer_that_changes():
    """A 0-d tensor or array that is changed in place: the buffers are checked against its value of
    the call, not of an earlier one."""
    for M in (torch.tensor(4), np.array(4)):
        assert mmq._sized(mmq.mmq_q8_1_bytes, M, 256) == mmq.mmq_q8_1_bytes(4, 256)
        M += 396
        assert mmq._sized(mmq.mmq_q8_1_bytes, M, 256) == mmq.mmq_q8_1_bytes(400, 256)


@pytest.mark.parametrize("fn,args", [
    ("quantize_q8_1", "x M 256 q8"), ("mmq_q4K_q8_1", "M 64 256 q8 w C"),
    ("mmq_q6K_q8_1", "M 64 256 q8 w C"), ("mmq_q4K_f32", "M 64 256 x w C"),
    ("mmq_q4K_q8_1_gated", "M 64 256 q8 w H"), ("mmq_q4K_f32_gated", "M 64 256 x w H"),
    ("mmq_moe_route", "M 8 2 logits ids weights"),
    ("mmq_q4K_moe_gated", "M 8 2 64 256 x plan w H q8"),
    ("mmq_q4K_moe_down", "M 8 2 64 256 H plan weights w out q8"),
    ("mmq_q4K_moe", "M 8 2 256 256 x logits w w out ws")])
def test_calls_check_buffers_against_the_size_of_the_call(fn, args, monkeypatch):
    """The first buffer of each call is checked for the number of tokens M that the call is given: an
    int, a 0-d array, and a 0-d tensor that is changed in place."""
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

    assert size(40) > size(4) > 0
    assert size(np.array(40)) == size(np.int32(40)) == size(40)
    M = torch.tensor(4)
    assert size(M) == size(4)
    M *= 10
    assert size(M) == size(40)
