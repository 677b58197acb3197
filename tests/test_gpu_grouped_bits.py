"""A pair's bits in the products grouped by expert go by the sizes of the call, not by the ids: the same
row of the same expert, beside any number of other rows, in every form of the kernel.
"""
import numpy as np
import pytest

import synth
from tests import grouped_util as gu
from tests import layer_util as lu
from tests.gpu_util import say, to_dev

pytestmark = pytest.mark.gpu

mmq = pytest.importorskip("q4_q8_int8_amd")
torch = pytest.importorskip("torch")

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    yield
    torch.cuda.synchronize()


def raw(n):
    return torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")


def f32(*shape):
    return torch.full(shape, NAN, dtype=torch.float32, device="cuda")


# rows of the expert: its last tile has 1, a few, 15 to 17, 31, 32 and more, alone and behind whole tiles
ROWS = [1, 2, 15, 16, 17, 31, 32, 33, 48, 49, 64, 80, 128, 129, 145]


def ids_with(n, M, k, E, expert):
    """ids [M, k] that give `expert` n pairs, the last pair among them, and the others no expert."""
    flat = np.full(M * k, E, np.int32)
    at = np.random.default_rng(n).permutation(M * k - 1)[:n - 1]
    flat[at] = expert
    flat[-1] = expert
    return flat.reshape(M, k)


def group(ids, E):
    M, k = ids.shape
    g = torch.zeros(mmq.mmq_moe_group_bytes(M, E, k) // 4, dtype=torch.int32, device="cuda")
    mmq.mmq_moe_group(M, E, k, to_dev(ids), g)
    return g


@pytest.mark.parametrize("form,M,E,k,N,K", [
    ("narrow", 200, 8, 2, 8200, 768), ("split2", 200, 8, 2, 2050, 2048),
    ("split4", 300, 8, 2, 1290, 4352), ("wide", 4096, 4, 2, 2050, 2048)])
def test_bits_do_not_go_by_the_ids(form, M, E, k, N, K):
    """The last pair is in the last tile of its expert, whatever its size; and its bits are those of
    the plain product's row where K is not split."""
    assert gu.grouped_form(M * k, E, N, K) == form
    w = to_dev(synth.q4k_weights("random_fields", N, K, 3)[0])
    n = mmq.mmq_q4K_repacked_bytes(N, K)
    rep = raw(E * n)
    mmq.repack_q4_K(w, N, K, rep[(E - 1) * n:])
    x = to_dev(synth.activations("normal_outliers", M, K, N))
    q8 = raw(mmq.mmq_q8_1_bytes(M, K))
    rows = {}
    for r in ROWS:
        C = f32(M * k, N)
        say("grouped", form, "rows", r)
        mmq.mmq_q4K_grouped(M, E, k, N, K, x, group(ids_with(r, M, k, E, E - 1), E), rep, C, q8)
        rows[r] = C[-1].clone()
    assert bool(torch.isfinite(rows[1]).all())
    for r in ROWS:
        assert torch.equal(rows[r], rows[1]), (r, int((rows[r] != rows[1]).sum()))
    if form in ("wide", "narrow"):
        P, qp = f32(M, N), raw(mmq.mmq_q8_1_bytes(M, K))
        mmq.quantize_q8_1(x, M, K, qp)
        mmq.mmq_q4K_q8_1_ex(M, N, K, qp, rep[(E - 1) * n:], P, force_tile=mmq.MMQ_TILE_LARGE)
        assert torch.equal(rows[1], P[-1])


@pytest.mark.parametrize("form,M,E,k,F,D", [
    ("narrow", 300, 6, 2, 4100, 256), ("split2", 200, 8, 2, 1025, 2048),
    ("split4", 300, 8, 2, 645, 4352), ("wide", 2048, 2, 2, 2050, 2048)])
def test_gated_bits_do_not_go_by_the_ids(form, M, E, k, F, D):
    assert gu.grouped_form(M * k, E, -(-F // 16) * 32, D) == form
    n = mmq.mmq_q4K_pair_bytes(F, D)
    rep = raw(E * n)
    mmq.repack_q4_K_pair(to_dev(lu.weights(F, D, 1)), to_dev(lu.weights(F, D, 2)), F, D,
                         rep[(E - 1) * n:])
    x = to_dev(synth.activations("normal_outliers", M, D, F))
    q8 = raw(mmq.mmq_q8_1_bytes(M, D))
    first = None
    for r in ROWS:
        H = f32(M * k, F)
        say("grouped gated", form, "rows", r)
        mmq.mmq_q4K_grouped_gated(M, E, k, F, D, x, group(ids_with(r, M, k, E, E - 1), E), rep, H,
                                  q8, act=mmq.MMQ_ACT_GELU)
        first = H[-1].clone() if first is None else first
        assert bool(torch.isfinite(first).all()) and torch.equal(H[-1], first), r
