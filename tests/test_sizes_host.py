"""The Python calls check buffers against sizes taken from whole numbers (no GPU): a size that arrives as
a narrow integer, a numpy one or a 0-d tensor, is not multiplied in its own width, where the product
would wrap and let a short buffer through.
"""
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
