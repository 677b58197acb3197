"""The Python calls check buffers against sizes taken from whole numbers (no GPU): a size that arrives as
a narrow integer, a numpy one or a 0-d tensor, is not multiplied in its own width, where the product
would wrap and let a short buffer through.
"""
import ctypes
import types

import numpy as np
import pytest

mmq = pytest.importorskip("q4_q8_int8_amd")
torch = pytest.importorskip("torch")


class Stub:
    """The library with one entry point that does nothing."""

    def __init__(self, lib, name):
        self._lib, self._name = lib, name

    def __getattr__(self, name):
        return (lambda *a: 0) if name == self._name else getattr(self._lib, name)


def needed(monkeypatch, fn, *args, **kw):
    """{buffer: bytes} that mmq.<fn>(*args) asks for."""
    seen = {}

    def dev(t, name, nbytes, *a, **k):
        seen[name] = int(nbytes)
        return 1 << 20

    with monkeypatch.context() as m:
        m.setattr(mmq, "_dev", dev)
        m.setattr(mmq, "_lib", Stub(mmq._lib, fn))
        getattr(mmq, fn)(*args, stream=0, **kw)
    return seen


T32, T16 = (types.SimpleNamespace(dtype=t) for t in (torch.float32, torch.bfloat16))
KINDS = [np.int32, lambda v: torch.tensor(v, dtype=torch.int32), lambda v: np.array(v, np.int32)]


@pytest.mark.filterwarnings("ignore:overflow encountered")
@pytest.mark.parametrize("kind", KINDS)
def test_q4g_sizes(kind, monkeypatch):
    f = mmq.q4G_format(32, torch.float16, True)
    N, K = 1 << 20, 1 << 12           # N K is 2^32
    want = needed(monkeypatch, "repack_q4_G", 0, 0, 0, N, K, f, 0)
    assert want["w"] == N * K // 2 and want["scales"] == want["zeros"] == 2 * N * K // 32
    assert needed(monkeypatch, "repack_q4_G", 0, 0, 0, kind(N), kind(K), f, 0) == want
    for y, size in ((T32, 4), (T16, 2)):
        M, N, K = 16, 1 << 25, 32     # M N is 2^29
        a = (y, 0, f, y)
        want = needed(monkeypatch, "mmq_q4G", M, N, K, *a, bias=0, residual=0)
        assert want["y"] == want["residual"] == size * M * N and want["x"] == size * M * K
        assert want["bias"] == 4 * N
        assert needed(monkeypatch, "mmq_q4G", kind(M), kind(N), kind(K), *a, bias=0,
                      residual=0) == want


# calls whose sizes are multiplied in the wrapper itself; the buffers that then need more than 2^31 bytes
OTHERS = [
    ("mmq_q4K_q8_1_epilogue", (1 << 15, 1 << 16, 256), ("residual",)),
    ("mmq_q4K_f32_epilogue", (128, 1 << 25, 256), ("residual",)),
    ("convert_f32_f16", (1 << 16, 1 << 14), ("x",)),
    ("gemm_f16", (1 << 15, 1 << 16, 256), ("C",)),
]


@pytest.mark.filterwarnings("ignore:overflow encountered")
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("fn,sizes,large", OTHERS)
def test_sizes_of_the_other_calls(fn, sizes, large, kind, monkeypatch):
    rest = {"mmq_q4K_q8_1_epilogue": 3, "mmq_q4K_f32_epilogue": 3, "convert_f32_f16": 0,
            "gemm_f16": 3}[fn]
    args = (0,) * rest
    kw = dict(bias=0, residual=0) if "epilogue" in fn else {}
    if fn == "convert_f32_f16":     # x comes before the sizes
        call = lambda t: needed(monkeypatch, fn, 0, *map(t, sizes), 0)
    else:
        call = lambda t: needed(monkeypatch, fn, *map(t, sizes), *args, **kw)
    want = call(int)
    assert all(want[b] >= 2 ** 31 for b in large), want
    assert call(kind) == want


@pytest.mark.filterwarnings("ignore:overflow encountered")
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("fn,per", [("mmq_q4K_q8_1_blockdots", 32), ("mmq_q6K_q8_1_blockdots", 16)])
def test_sizes_of_the_block_dots(fn, per, kind, monkeypatch):
    M, N, K, rows, cols = 4096, 8192, 4096, 4096, 8192
    call = lambda t: needed(monkeypatch, fn, *map(t, (M, N, K)), 0, 0, t(0), t(rows), t(0), t(cols),
                            0)
    want = call(int)
    assert want["S"] == 4 * (K // per) * rows * cols
    assert call(kind) == want


def test_size_of_a_plans_ids(monkeypatch):
    """(A plan's sizes fit any integer of 16 bits and more.)"""
    want = needed(monkeypatch, "mmq_moe_plan", 64, 512, 8, 0, 0)
    assert want["ids"] == 4 * 64 * 8
    for kind in (np.int8, np.uint8):
        assert needed(monkeypatch, "mmq_moe_plan", kind(64), 512, kind(8), 0, 0) == want


def test_sizes_are_not_multiplied_before_they_are_checked():
    """The rows of x per pair, M k, would pass 64 bits."""
    p = 1 << 20
    for per_pair in (0, 1, 2):
        for M, k in ((1 << 62, 8), (2 ** 63 - 1, 64), (-(1 << 62), 8)):
            assert mmq.raw_call("mmq_q4K_grouped", M, 64, k, 64, 256, p, per_pair, p, p, p, p, 0,
                                None) == (mmq.MMQ_E_SHAPE if M > 0 else mmq.MMQ_E_ARG)


def test_a_plans_sizes_are_not_multiplied_before_they_are_checked():
    p = 1 << 20
    for M, E, k in ((2 ** 63 - 1, 8, 8), (1 << 40, 1 << 40, 1 << 40), (1, 8, 2 ** 63 - 1)):
        sizes = (M, E, k, 256, 256)
        assert mmq.raw_call("mmq_q4K_moe_gated", *sizes, p, p, p, p, p, 2, None) == mmq.MMQ_E_SHAPE
        assert mmq.raw_call("mmq_q4K_moe_down", *sizes, p, p, p, p, None, p, p, None) == mmq.MMQ_E_SHAPE
        assert mmq.raw_call("mmq_moe_plan", M, E, k, p, p, None) == mmq.MMQ_E_SHAPE
        assert mmq.raw_call("mmq_moe_route", M, E, k, p, 0, 1, p, p, p, None) == mmq.MMQ_E_SHAPE
        assert mmq.raw_call("mmq_moe_workspace_bytes", *sizes,
                            ctypes.byref(ctypes.c_size_t())) == mmq.MMQ_E_SHAPE
