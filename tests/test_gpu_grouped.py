"""The products grouped by expert on the GPU: the sort of the pairs, the grouped product, its gated form
and the weighted sum against the float64 oracle, the unsplit forms of the kernel bit for bit against the
plain product of each expert's rows, the whole layer against its calls, in graphs, on two streams, and
groups of nonsense.
"""
import functools

import numpy as np
import pytest

import synth
from oracle import layer_oracle as lo
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


def f32(*shape):
    return torch.full(shape, NAN, dtype=torch.float32, device="cuda")


def raw(n):
    return torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def group(ids, E):
    M, k = ids.shape
    g = torch.full((mmq.mmq_moe_group_bytes(M, E, k) // 4,), -7, dtype=torch.int32, device="cuda")
    mmq.mmq_moe_group(M, E, k, to_dev(ids), g)
    return g


# ---------------------------------------------------------------- the sort

# one workgroup of 1, 2 and 4 pairs per work-item, and chunks; each at its border
SORTS = [(1, 1, 1), (1, 8, 8), (5, 512, 64), (100, 64, 8), (1023, 7, 1), (1024, 3, 1), (1025, 3, 1),
         (2048, 5, 1), (683, 16, 3), (2048, 8, 2), (4097, 512, 1), (2049, 300, 4), (8192, 256, 8),
         (32767, 512, 3)]


def ids_of(kind, M, E, k, seed):
    rng = np.random.default_rng(seed)
    if kind == "random":
        return rng.integers(0, E, (M, k)).astype(np.int32)
    if kind == "one":
        return np.full((M, k), E - 1, np.int32)
    if kind == "none":
        return np.full((M, k), -1, np.int32)
    ids = rng.integers(-2, E + 2, (M, k)).astype(np.int32)   # some outside
    ids[rng.random((M, k)) < 0.02] = 2 ** 31 - 1
    ids[rng.random((M, k)) < 0.02] = -2 ** 31
    return ids


@pytest.mark.parametrize("kind", ["random", "outside", "one", "none"])
@pytest.mark.parametrize("M,E,k", SORTS)
def test_group(M, E, k, kind):
    ids = ids_of(kind, M, E, k, M + E + k)
    say("group", (M, E, k), kind)
    offsets, order, place = mmq.moe_groups(group(ids, E), M, E, k)
    for got, want in zip((offsets, order, place), lo.groups(ids, E)):
        assert np.array_equal(host(got), want)


def test_group_of_the_most_pairs():
    M, E, k = 1 << 18, 200, 8
    ids = ids_of("outside", M, E, k, 3)
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    want = np.argsort(key, kind="stable")
    n = int((key < E).sum())
    say("group", (M, E, k))
    offsets, order, place = (host(t) for t in mmq.moe_groups(group(ids, E), M, E, k))
    assert np.array_equal(order[:n], want[:n]) and np.all(order[n:] == -1)
    assert np.array_equal(np.diff(offsets), np.bincount(key, minlength=E + 1)[:E])
    assert np.array_equal(place[want[:n]], np.arange(n)) and np.all(place[want[n:]] == -1)


# ---------------------------------------------------------------- the products

# rows of the experts: none, one, a part of a 32-row part, each number of parts, and several tiles
RAGGED = [0, 1, 31, 32, 33, 0, 64, 65, 96, 97, 127, 128, 129, 300, 5]


@functools.lru_cache(maxsize=8)
def experts(kind, E, N, K, seed):
    """E matrices, repacked one behind the other, and their q4_K blocks."""
    ws = [lu.weights(N, K, seed + e) for e in range(E)]
    if kind == "plain":
        n = mmq.mmq_q4K_repacked_bytes(N, K)
        rep = raw(E * n)
        for e in range(E):
            mmq.repack_q4_K(to_dev(ws[e]), N, K, rep[e * n:(e + 1) * n])
        return rep, np.stack(ws), None
    up = [lu.weights(N, K, 1000 + seed + e) for e in range(E)]
    n = mmq.mmq_q4K_pair_bytes(N, K)
    rep = raw(E * n)
    for e in range(E):
        mmq.repack_q4_K_pair(to_dev(ws[e]), to_dev(up[e]), N, K, rep[e * n:(e + 1) * n])
    return rep, np.stack(ws), np.stack(up)


def ragged_ids(counts, k, rng, none=3):
    """ids [M, k] in which expert e has counts[e] pairs, in random order, `none` and what fills the last
    token without an expert; tokens may name an expert twice."""
    flat = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [np.full(none, -1)])
    flat = np.concatenate([flat, np.full(-len(flat) % k, len(counts))])
    rng.shuffle(flat)
    return flat.reshape(-1, k).astype(np.int32)


def plain_rows(x, rep, e, n_bytes, N, K):
    """The plain product of some rows with expert e's matrix, by a tile that the unsplit grouped forms
    share their order of additions with (the decode and skinny tiles, which few rows get by default,
    have others)."""
    M = x.shape[0]
    q8, C = raw(mmq.mmq_q8_1_bytes(M, K)), f32(M, N)
    mmq.quantize_q8_1(x, M, K, q8)
    mmq.mmq_q4K_q8_1_ex(M, N, K, q8, rep[e * n_bytes:(e + 1) * n_bytes], C,
                        force_tile=mmq.MMQ_TILE_LARGE)
    return C


# one super-block, and more of them than ranges of K in each form, and than fit them evenly
@pytest.mark.parametrize("per_pair", [False, True])
@pytest.mark.parametrize("k,N,K", [(1, 64, 256), (2, 70, 512), (1, 258, 768), (3, 515, 1280),
                                   (2, 1, 256), (1, 2050, 512), (1, 130, 2816), (2, 33, 4096)])
def test_grouped(k, N, K, per_pair):
    E = len(RAGGED)
    ids = ragged_ids(RAGGED, k, np.random.default_rng(N + K))
    M = ids.shape[0]
    rows = M * k if per_pair else M
    xh = synth.activations("normal_outliers", rows, K, N)
    rep, ws, _ = experts("plain", E, N, K, 40)
    q8, C = raw(mmq.mmq_q8_1_bytes(rows, K)), f32(M * k, N)
    say("grouped", (M, E, k, N, K), "per pair" if per_pair else "per token",
        gu.grouped_form(M * k, E, N, K))
    mmq.mmq_q4K_grouped(M, E, k, N, K, to_dev(xh), group(ids, E), rep, C, q8, per_pair=per_pair)
    got = host(C)
    flat = ids.reshape(-1)
    assert np.all(np.isnan(got[(flat < 0) | (flat >= E)])), "rows without an expert were written"
    for e in range(E):
        ps = np.nonzero(flat == e)[0]
        if ps.size:
            P, T = lu.product(np.ascontiguousarray(xh[ps if per_pair else ps // k]), ws[e])
            lu.assert_close(got[ps], P, lu.BAR * T, what=f"expert {e}")


# few experts with few rows (every form in turn as the grid shrinks); the last one: many rows
FORMS = [("narrow", 200, 8, 2, 8200, 768), ("split2", 200, 8, 2, 2050, 2048),
         ("split4", 300, 8, 2, 1290, 4352), ("wide", 4096, 4, 2, 2050, 2048)]


@pytest.mark.parametrize("form,M,E,k,N,K", FORMS)
def test_every_form(form, M, E, k, N, K):
    """Each form of the kernel, on ragged experts, against the plain product of each expert's rows: bit
    for bit where K is not split and the tile is of 32-row parts, else within both products' bars."""
    assert gu.grouped_form(M * k, E, N, K) == form
    rng = np.random.default_rng(M)
    ids = np.minimum(rng.geometric(0.3, (M, k)) - 1, E).astype(np.int32)   # E: none
    x = to_dev(synth.activations("normal_outliers", M, K, N))
    blocks = synth.q4k_weights("random_fields", E * N, K, 3)[0]
    n = mmq.mmq_q4K_repacked_bytes(N, K)
    rep = raw(E * n)
    for e in range(E):
        mmq.repack_q4_K(to_dev(blocks[e * N:(e + 1) * N]), N, K, rep[e * n:(e + 1) * n])
    C, q8 = f32(M * k, N), raw(mmq.mmq_q8_1_bytes(M, K))
    say("grouped", form, (M, E, k, N, K))
    mmq.mmq_q4K_grouped(M, E, k, N, K, x, group(ids, E), rep, C, q8)
    flat = ids.reshape(-1)
    for e in range(E):
        ps = torch.from_numpy(np.nonzero(flat == e)[0]).cuda()
        if not ps.numel():
            continue
        want, got = plain_rows(x[ps // k].contiguous(), rep, e, n, N, K), C[ps]
        exact = {"wide": len(ps), "narrow": gu.rows_in_32(len(ps))}.get(form, 0)
        assert torch.equal(got[:exact], want[:exact]), e
        if exact < len(ps):
            some = np.arange(exact, min(len(ps), exact + 20))
            _, T = lu.product(np.ascontiguousarray(host(x[ps[exact:exact + 20] // k])),
                              blocks[e * N:(e + 1) * N])
            lu.assert_close(host(got)[some], host(want)[some].astype(np.float64), 2 * lu.BAR * T)
            # and every row to a looser bound of the whole: a row that is wrong is far off
            assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max())
    assert bool(torch.isnan(C[torch.from_numpy(np.nonzero(flat == E)[0]).cuda()]).all())


# tiles of an XCD (32 compute units each): 8, 28, 38, 40, 44, 52, 54, 64, 68, 75: none, a few, some and most in
# its last round, whose tiles are cut finer where they are few
@pytest.mark.parametrize("rows,N", [(100, 8192), (700, 8192), (1100, 7500), (1152, 8192), (1280, 8192),
                                    (1536, 8192), (1535, 8330), (1920, 8192), (2048, 8192), (2049, 8400)])
def test_wide_forms_last_round(rows, N):
    """One expert with most rows and a ragged one, against the plain product bit for bit."""
    E, K = 2, 2048
    counts = (rows, 45)
    assert gu.grouped_form(4096, E, N, K) == "wide"
    ids = np.full((4096, 1), -1, np.int32)
    at = np.random.default_rng(rows).permutation(4096)
    ids[at[:rows]], ids[at[rows:rows + 45]] = 0, 1
    x = to_dev(synth.activations("normal_outliers", 4096, K, N))
    blocks = to_dev(synth.q4k_weights("random_fields", E * N, K, 3)[0]).reshape(E, -1)
    n = mmq.mmq_q4K_repacked_bytes(N, K)
    rep = raw(E * n)
    for e in range(E):
        mmq.repack_q4_K(blocks[e], N, K, rep[e * n:(e + 1) * n])
    C = f32(4096, N)
    say("grouped wide", counts, N, "tiles", -(-rows // 128) + 1, "by", -(-N // 256))
    mmq.mmq_q4K_grouped(4096, E, 1, N, K, x, group(ids, E), rep, C, raw(mmq.mmq_q8_1_bytes(4096, K)))
    for e in range(E):
        ps = torch.from_numpy(np.nonzero(ids.reshape(-1) == e)[0]).cuda()
        assert len(ps) == counts[e]
        assert torch.equal(C[ps], plain_rows(x[ps].contiguous(), rep, e, n, N, K)), e
    none = torch.from_numpy(np.nonzero(ids.reshape(-1) < 0)[0]).cuda()
    assert bool(torch.isnan(C[none]).all())


def test_tokens_of_nan_and_infinity_stay_alone():
    """In every form: the other pairs' rows are bit for bit what they are without them."""
    for form, M, E, k, N, K in FORMS:
        assert gu.grouped_form(M * k, E, N, K) == form
        ids = np.random.default_rng(2).integers(0, E, (M, k)).astype(np.int32)
        x = to_dev(synth.activations("normal_outliers", M, K, N))
        n = mmq.mmq_q4K_repacked_bytes(N, K)
        rep = raw(E * n)
        blocks = synth.q4k_weights("random_fields", N, K, 3)[0]
        for e in range(E):
            mmq.repack_q4_K(to_dev(blocks), N, K, rep[e * n:(e + 1) * n])
        g, q8 = group(ids, E), raw(mmq.mmq_q8_1_bytes(M, K))
        clean, C = f32(M * k, N), f32(M * k, N)
        say("grouped with NaN", form)
        mmq.mmq_q4K_grouped(M, E, k, N, K, x, g, rep, clean, q8)
        assert bool(torch.isfinite(clean).all())
        x[3, 7], x[M - 1, K - 1], x[11, 300] = NAN, float("inf"), -float("inf")
        mmq.mmq_q4K_grouped(M, E, k, N, K, x, g, rep, C, q8)
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[[3, 11, M - 1]] = False
        keep = keep.repeat_interleave(k)
        assert torch.equal(C[keep], clean[keep]), form


@pytest.mark.parametrize("M,k", [(3, 2), (150, 2), (4000, 1)])
def test_no_pair_has_an_expert(M, k):
    E, D, F = 8, 256, 256
    ids = np.full((M, k), -1, np.int32)
    pairs, down = experts("pair", E, F, D, 700)[0], experts("plain", E, D, F, 800)[0]
    g = group(ids, E)
    x = to_dev(synth.activations("normal", M, D, 1))
    H, out = f32(M * k, F), f32(M, D)
    say("no experts", M, k)
    mmq.mmq_q4K_grouped_gated(M, E, k, F, D, x, g, pairs, H, raw(mmq.mmq_q8_1_bytes(M, D)))
    assert bool(torch.isnan(H).all())
    space = raw(mmq.mmq_grouped_down_workspace_bytes(M, E, k, D, F))
    wts = torch.ones(M, k, device="cuda")
    mmq.mmq_q4K_grouped_down(M, E, k, D, F, H, g, wts, down, out, space)
    assert not bool(out.any()) and bool(torch.isfinite(out).all())
    mmq.mmq_q4K_grouped_down(M, E, k, D, F, H, g, wts, down, out, space, residual=x)
    assert torch.equal(out, x)


@pytest.mark.parametrize("act", lo.ACTS)
def test_grouped_activation(act):
    k, N, K, E = 2, 100, 512, len(RAGGED)
    rng = np.random.default_rng(5)
    ids = ragged_ids(RAGGED, k, rng)
    M = ids.shape[0]
    xh = synth.activations("normal_outliers", M, K, 6)
    rep, ws, _ = experts("plain", E, N, K, 70)
    C, q8 = f32(M * k, N), raw(mmq.mmq_q8_1_bytes(M, K))
    say("grouped", act)
    mmq.mmq_q4K_grouped(M, E, k, N, K, to_dev(xh), group(ids, E), rep, C, q8,
                        act=mmq.ACTIVATIONS[act])
    got, flat = host(C), ids.reshape(-1)
    for e in range(E):
        ps = np.nonzero(flat == e)[0]
        if ps.size:
            P, T = lu.product(np.ascontiguousarray(xh[ps // k]), ws[e])
            lu.assert_close(got[ps], *lo.epilogue(P, T, lu.BAR, act), what=f"{act}, expert {e}")


@pytest.mark.parametrize("k,F,D", [(1, 64, 256), (2, 40, 512), (1, 129, 768), (3, 515, 1280),
                                   (2, 1, 256), (1, 1030, 256), (2, 17, 4096)])
def test_grouped_gated(k, F, D):
    E = len(RAGGED)
    ids = ragged_ids(RAGGED, k, np.random.default_rng(F + D))
    M = ids.shape[0]
    xh = synth.activations("normal_outliers", M, D, F)
    rep, gate, up = experts("pair", E, F, D, 300)
    q8, H = raw(mmq.mmq_q8_1_bytes(M, D)), f32(M * k, F)
    say("grouped gated", (M, E, k, F, D), gu.grouped_form(M * k, E, -(-F // 16) * 32, D))
    mmq.mmq_q4K_grouped_gated(M, E, k, F, D, to_dev(xh), group(ids, E), rep, H, q8,
                              act=mmq.MMQ_ACT_SILU)
    got, flat = host(H), ids.reshape(-1)
    none = (flat < 0) | (flat >= E)
    assert np.all(np.isnan(got[none])), "rows without an expert were written"
    want, err = lu.experts_gated(xh, ids, gate, up, "silu")
    lu.assert_close(got[~none], want[~none], err[~none])


def test_grouped_gated_is_the_gated_product_of_each_expert():
    """Bit for bit, in the unsplit forms and tiles of 32-row parts."""
    for form, M, E, k, F, D in (("narrow", 300, 6, 2, 4100, 256), ("wide", 2048, 2, 2, 2050, 2048)):
        assert gu.grouped_form(M * k, E, -(-F // 16) * 32, D) == form
        ids = np.random.default_rng(F).integers(0, E, (M, k)).astype(np.int32)
        x = to_dev(synth.activations("normal_outliers", M, D, F))
        n, m = mmq.mmq_q4K_pair_bytes(F, D), F * (D // 256) * 144
        blocks = to_dev(synth.q4k_weights("random_fields", 2 * E * F, D, 5)[0]).reshape(2 * E, -1)
        rep = raw(E * n)
        for e in range(E):
            mmq.repack_q4_K_pair(blocks[e], blocks[E + e], F, D, rep[e * n:(e + 1) * n])
        H = f32(M * k, F)
        say("grouped gated", form, (M, E, k, F, D))
        mmq.mmq_q4K_grouped_gated(M, E, k, F, D, x, group(ids, E), rep, H,
                                  raw(mmq.mmq_q8_1_bytes(M, D)), act=mmq.MMQ_ACT_GELU)
        for e in range(E):
            ps = torch.from_numpy(np.nonzero(ids.reshape(-1) == e)[0]).cuda()
            rows, He = x[ps // k].contiguous(), f32(ps.numel(), F)
            qe = raw(mmq.mmq_q8_1_bytes(ps.numel(), D))
            mmq.quantize_q8_1(rows, ps.numel(), D, qe)
            mmq.mmq_q4K_q8_1_gated(ps.numel(), F, D, qe, rep[e * n:(e + 1) * n], He,
                                   act=mmq.MMQ_ACT_GELU, force_tile=mmq.MMQ_TILE_LARGE)
            exact = ps.numel() if form == "wide" else gu.rows_in_32(ps.numel())
            assert exact and torch.equal(H[ps[:exact]], He[:exact]), (form, e)


# few and many rows per expert, experts that no one names, one expert that everyone names, tokens
# without any, one token, an odd width
LAYERS = [(1, 4, 2, 256, 256), (70, 8, 2, 512, 768), (200, 3, 3, 300, 512), (65, 64, 6, 256, 256),
          (333, 5, 1, 1025, 1280), (129, 1, 1, 64, 256)]


def layer_ids(M, E, k, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32)
    if M > 64:
        ids[M - 5:] = -1
        ids[7, 0] = -1
    return ids


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,E,k,D,F", LAYERS)
def test_grouped_down(M, E, k, D, F, residual):
    ids = layer_ids(M, E, k, M + D)
    rng = np.random.default_rng(F)
    Hh = synth.activations("normal_outliers", M * k, F, D + 1)
    wts = rng.random((M, k)).astype(np.float32)
    res = rng.standard_normal((M, D)).astype(np.float32) if residual else None
    rep, ws, _ = experts("plain", E, D, F, 500)
    H = to_dev(Hh)
    H[torch.from_numpy(np.nonzero(ids.reshape(-1) < 0)[0]).cuda()] = NAN   # unused rows
    out = f32(M, D) if res is None else to_dev(res)
    n = mmq.mmq_grouped_down_workspace_bytes(M, E, k, D, F)
    space = torch.full((n,), 255, dtype=torch.uint8, device="cuda")        # NaN in every float
    say("grouped down", (M, E, k, D, F))
    mmq.mmq_q4K_grouped_down(M, E, k, D, F, H, group(ids, E), to_dev(wts), rep, out, space,
                             residual=None if res is None else out)
    lu.assert_close(host(out), *lu.experts_down(Hh, ids, wts, ws, res))


def layer_inputs(M, E, k, D, F):
    x = to_dev(synth.activations("normal_outliers", M, D, 1))
    rng = np.random.default_rng(2)
    logits = rng.standard_normal((M, E)).astype(np.float32)
    if M > 64:
        logits[M - 3:] = -np.inf
    return (x, to_dev(logits), experts("pair", E, F, D, 700)[0], experts("plain", E, D, F, 800)[0],
            to_dev(rng.standard_normal((M, D)).astype(np.float32)))


@pytest.mark.parametrize("M,E,k,D,F", [(1, 4, 2, 256, 256), (100, 8, 2, 512, 768),
                                       (300, 64, 6, 256, 256)])
def test_grouped_layer_is_its_calls(M, E, k, D, F):
    x, logits, pairs, down, res = layer_inputs(M, E, k, D, F)
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    wts, H, out, whole = f32(M, k), f32(M * k, F), f32(M, D), f32(M, D)
    say("grouped layer", (M, E, k, D, F))
    mmq.mmq_moe_route(M, E, k, logits, ids, wts, score=mmq.MMQ_SCORE_SIGMOID)
    g = torch.empty(mmq.mmq_moe_group_bytes(M, E, k) // 4, dtype=torch.int32, device="cuda")
    mmq.mmq_moe_group(M, E, k, ids, g)
    mmq.mmq_q4K_grouped_gated(M, E, k, F, D, x, g, pairs, H, raw(mmq.mmq_q8_1_bytes(M, D)),
                              act=mmq.MMQ_ACT_GELU)
    mmq.mmq_q4K_grouped_down(M, E, k, D, F, H, g, wts, down, out,
                             raw(mmq.mmq_grouped_down_workspace_bytes(M, E, k, D, F)), residual=res)
    mmq.mmq_q4K_grouped_moe(M, E, k, D, F, x, logits, pairs, down, whole,
                            raw(mmq.mmq_grouped_moe_workspace_bytes(M, E, k, D, F)),
                            score=mmq.MMQ_SCORE_SIGMOID, act=mmq.MMQ_ACT_GELU, residual=res)
    assert np.array_equal(host(whole), host(out))
    masked = host(torch.isinf(logits).all(1))
    assert np.array_equal(host(whole)[masked], host(res)[masked])
    # and the few tokens' products, which take a plan, agree: both are within their bar of the same H
    if M * k <= 512 and M <= 64:
        few = f32(M, D)
        mmq.mmq_q4K_moe(M, E, k, D, F, x, logits, pairs, down, few,
                        raw(mmq.mmq_moe_workspace_bytes(M, E, k, D, F)),
                        score=mmq.MMQ_SCORE_SIGMOID, act=mmq.MMQ_ACT_GELU, residual=res)
        assert np.all(np.isfinite(host(few)))


def test_grouped_layer_in_a_graph_and_on_two_streams():
    """Captured once per stream with a workspace each, replayed together several times with other
    inputs in between: every replay gives what the eager call gives for its inputs."""
    M, E, k, D, F = 150, 8, 2, 256, 512
    x, logits, pairs, down, res = layer_inputs(M, E, k, D, F)
    n = mmq.mmq_grouped_moe_workspace_bytes(M, E, k, D, F)
    sides = []
    say("grouped layer in graphs")
    for _ in range(2):
        s = torch.cuda.Stream()
        d = dict(s=s, x=x.clone(), l=logits.clone(), out=f32(M, D), w=raw(n))

        def call(d=d):
            mmq.mmq_q4K_grouped_moe(M, E, k, D, F, d["x"], d["l"], pairs, down, d["out"], d["w"],
                                    residual=res)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            call()
        torch.cuda.synchronize()
        d["g"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(d["g"], stream=s):
            call()
        sides.append(d)
    eager, we = f32(M, D), raw(n)
    for i in range(4):
        for j, d in enumerate(sides):
            d["x"].copy_(to_dev(synth.activations("normal", M, D, 10 * i + j)))
            d["l"].copy_(torch.from_numpy(
                np.random.default_rng(10 * i + j).standard_normal((M, E)).astype(np.float32)))
            d["out"].fill_(NAN)
        torch.cuda.synchronize()
        for d in sides:
            with torch.cuda.stream(d["s"]):
                d["g"].replay()
        torch.cuda.synchronize()
        for d in sides:
            mmq.mmq_q4K_grouped_moe(M, E, k, D, F, d["x"], d["l"], pairs, down, eager, we,
                                    residual=res)
            assert np.array_equal(host(d["out"]), host(eager)), i


def test_sort_of_many_pairs_in_a_graph():
    """The sort in chunks, captured and replayed with other ids in between."""
    M, E, k = 3001, 60, 2
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    g = torch.empty(mmq.mmq_moe_group_bytes(M, E, k) // 4, dtype=torch.int32, device="cuda")
    ids.fill_(-1)
    say("sort in a graph")
    mmq.mmq_moe_group(M, E, k, ids, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmq.mmq_moe_group(M, E, k, ids, g)
    for i, kind in enumerate(("random", "outside", "one", "random")):
        h = ids_of(kind, M, E, k, i)
        ids.copy_(torch.from_numpy(h))
        graph.replay()
        for got, want in zip(mmq.moe_groups(g, M, E, k), lo.groups(h, E)):
            assert np.array_equal(host(got), want), i


def test_expert_weights_past_4_gib():
    """The last of 512 experts starts 4.3 GB into the weights; 3 and 200 rows of it."""
    E, D, F = 512, 4096, 1840
    n = mmq.mmq_q4K_pair_bytes(F, D)
    assert (E - 1) * n > 2 ** 32
    w_in = torch.empty(E * n, dtype=torch.uint8, device="cuda")   # only two experts are written
    gate = {e: lu.weights(F, D, 2 * e) for e in (0, E - 1)}
    up = {e: lu.weights(F, D, 2 * e + 1) for e in (0, E - 1)}
    for e in gate:
        mmq.repack_q4_K_pair(to_dev(gate[e]), to_dev(up[e]), F, D, w_in[e * n:(e + 1) * n])
    for M in (3, 200):
        x = synth.activations("normal", M, D, 3)
        ids = np.full((M, 1), E - 1, np.int32)
        ids[1] = 0
        H = f32(M, F)
        say("experts past 4 GiB", M)
        mmq.mmq_q4K_grouped_gated(M, E, 1, F, D, to_dev(x), group(ids, E), w_in, H,
                                  raw(mmq.mmq_q8_1_bytes(M, D)))
        got = host(H)
        for t in (0, 1, 2, M - 1):
            e = ids[t, 0]
            (G, TG), (U, TU) = lu.product(x[t:t + 1], gate[e]), lu.product(x[t:t + 1], up[e])
            lu.assert_close(got[t:t + 1], *lo.gated(G, TG, U, TU, lu.BAR, "silu"))


def test_output_past_4_gib():
    """The last pairs' rows start more than 4 GiB into the output, and into the workspace of the
    weighted sum."""
    M, E, k, N, K = 35000, 2, 2, 16400, 256
    assert (M * k - 8) * N * 4 > 2 ** 32
    rep, ws, _ = experts("plain", E, N, K, 40)
    xh = synth.activations("normal", M * k, K, 2)
    ids = np.random.default_rng(1).integers(0, E, (M, k)).astype(np.int32)
    g, x = group(ids, E), to_dev(xh)
    C = f32(M * k, N)
    say("grouped output past 4 GiB")
    mmq.mmq_q4K_grouped(M, E, k, N, K, x, g, rep, C, raw(mmq.mmq_q8_1_bytes(M * k, K)),
                        per_pair=True)
    wts = np.random.default_rng(2).random((M, k)).astype(np.float32)
    out = f32(M, N)
    mmq.mmq_q4K_grouped_down(M, E, k, N, K, x, g, to_dev(wts), rep, out,
                             raw(mmq.mmq_grouped_down_workspace_bytes(M, E, k, N, K)))
    for t in (0, 1, M - 3, M - 2, M - 1):
        ps = np.arange(t * k, t * k + k)
        for p in ps:
            P, T = lu.product(np.ascontiguousarray(xh[p:p + 1]), ws[ids.reshape(-1)[p]])
            lu.assert_close(host(C[p:p + 1]), P, lu.BAR * T)
        lu.assert_close(host(out[t:t + 1]),
                        *lu.experts_down(np.ascontiguousarray(xh[ps]), ids[t:t + 1], wts[t:t + 1],
                                         ws, None))
    assert bool(torch.isfinite(C).all())


def test_groups_of_nonsense_select_rows_of_the_product_only():
    """Every int32 in the groups: the calls return, and write nothing outside their outputs."""
    M, E, k, N, K = 200, 8, 2, 64, 256
    x = to_dev(synth.activations("normal", M, K, 1))
    rep, _, _ = experts("plain", E, N, K, 900)
    guard = torch.full((M * k + 2, N), 5.0, dtype=torch.float32, device="cuda")
    C = guard[1:-1]
    rng = np.random.default_rng(3)
    n = mmq.mmq_moe_group_bytes(M, E, k) // 4
    say("groups of nonsense")
    for i in range(4):
        g = rng.integers(-2 ** 31, 2 ** 31, n) if i < 2 else rng.integers(-3, M * k + 3, n)
        mmq.mmq_q4K_grouped(M, E, k, N, K, x, to_dev(g.astype(np.int32)), rep, C,
                            raw(mmq.mmq_q8_1_bytes(M, K)))
        got = host(guard)
        assert np.all(got[0] == 5.0) and np.all(got[-1] == 5.0) and np.all(np.isfinite(got))


def test_grouped_results_repeat_bit_for_bit():
    M, E, k, D, F = 300, 8, 3, 512, 512
    x, logits, pairs, down, res = layer_inputs(M, E, k, D, F)
    n = mmq.mmq_grouped_moe_workspace_bytes(M, E, k, D, F)
    first = None
    for _ in range(5):
        out = f32(M, D)
        mmq.mmq_q4K_grouped_moe(M, E, k, D, F, x, logits, pairs, down, out, raw(n), residual=res)
        first = host(out) if first is None else first
        assert np.array_equal(first, host(out))


def test_grouped_python_checks_tensors():
    M, E, k, N, K = 4, 2, 1, 32, 256
    x, C, q8 = f32(M, K), f32(M, N), raw(mmq.mmq_q8_1_bytes(M, K))
    g = group(np.zeros((M, k), np.int32), E)
    rep = raw(E * mmq.mmq_q4K_repacked_bytes(N, K))
    for bad in (dict(x=x.double()), dict(x=x[:3].contiguous()), dict(g=g[:-4]), dict(g=g.float()),
                dict(rep=rep[:-16]), dict(C=C[:3]), dict(C=C.t()), dict(q8=q8[:-1]),
                dict(x=x.cpu())):
        a = dict(x=x, g=g, rep=rep, C=C, q8=q8)
        a.update(bad)
        with pytest.raises(mmq.MMQArgumentError):
            mmq.mmq_q4K_grouped(M, E, k, N, K, a["x"], a["g"], a["rep"], a["C"], a["q8"])
    with pytest.raises(mmq.MMQArgumentError):
        mmq.mmq_q4K_grouped(M, E, 2, N, K, x, g, rep, C, q8, per_pair=True)
    with pytest.raises(mmq.MMQArgumentError):
        mmq.moe_groups(g[:-4], M, E, k)
