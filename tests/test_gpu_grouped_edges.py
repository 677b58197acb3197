"""The products grouped by expert where there is little or nothing sensible to do, in every form of the
kernel: no pair with an expert, groups of nonsense, experts without rows between ragged ones; and the
layer of many tokens against the one of a few.
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
# a shape for each form: M, E, k, N, K (also the down product's M, E, k, D, F, whose rows are pairs)
FORMS = {"narrow": (200, 8, 2, 8200, 768), "split2": (200, 8, 2, 2050, 2048),
         "split4": (300, 8, 2, 1290, 4352), "wide": (4096, 4, 2, 2050, 2048)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    yield
    torch.cuda.synchronize()


def raw(n):
    return torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")


def f32(*shape, value=NAN):
    return torch.full(shape, value, dtype=torch.float32, device="cuda")


def shape(form):
    M, E, k, N, K = FORMS[form]
    assert gu.grouped_form(M * k, E, N, K) == form
    return FORMS[form]


def group(ids, E):
    M, k = ids.shape
    g = torch.zeros(mmq.mmq_moe_group_bytes(M, E, k) // 4, dtype=torch.int32, device="cuda")
    mmq.mmq_moe_group(M, E, k, to_dev(ids), g)
    return g


def same_experts(E, N, K):
    """E times one matrix, repacked."""
    one = raw(mmq.mmq_q4K_repacked_bytes(N, K))
    mmq.repack_q4_K(to_dev(synth.q4k_weights("random_fields", N, K, 3)[0]), N, K, one)
    return one.repeat(E)


def same_pairs(E, F, K):
    one = raw(mmq.mmq_q4K_pair_bytes(F, K))
    mmq.repack_q4_K_pair(to_dev(lu.weights(F, K, 1)), to_dev(lu.weights(F, K, 2)), F, K, one)
    return one.repeat(E)


@pytest.mark.parametrize("form", list(FORMS))
def test_no_pair_has_an_expert(form):
    M, E, k, N, K = shape(form)
    F = N // 2
    assert gu.grouped_form(M * k, E, -(-F // 16) * 32, K) == form
    g = group(np.full((M, k), -1, np.int32), E)
    x = to_dev(synth.activations("normal", M, K, 1))
    C, H = f32(M * k, N), f32(M * k, F)
    q8 = raw(mmq.mmq_q8_1_bytes(M, K))
    rep = same_experts(E, N, K)
    say("no experts", form)
    mmq.mmq_q4K_grouped(M, E, k, N, K, x, g, rep, C, q8)
    mmq.mmq_q4K_grouped_gated(M, E, k, F, K, x, g, same_pairs(E, F, K), H, q8)
    assert bool(torch.isnan(C).all()) and bool(torch.isnan(H).all())
    residual, out, h = f32(M, N, value=2.5), f32(M, N), f32(M * k, K)
    space = torch.full((mmq.mmq_grouped_down_workspace_bytes(M, E, k, N, K),), 255,
                       dtype=torch.uint8, device="cuda")
    w = f32(M, k)
    mmq.mmq_q4K_grouped_down(M, E, k, N, K, h, g, w, rep, out, space)
    assert bool((out == 0).all())
    mmq.mmq_q4K_grouped_down(M, E, k, N, K, h, g, w, rep, out, space, residual=residual)
    assert torch.equal(out, residual)


def nonsense(P, E, n):
    """Groups of n int32 that no sort makes."""
    rng = np.random.default_rng(3)
    yield "any", rng.integers(-2 ** 31, 2 ** 31, n)
    yield "near", rng.integers(-3, P + 3, n)
    g = rng.integers(-3, P + 3, n)
    g[:E + 1] = np.arange(E + 1) % 2 * P        # every other expert has all the pairs
    yield "all", g
    g = rng.integers(0, P, n)
    g[:E + 1] = np.linspace(P, 0, E + 1)        # falling offsets
    yield "falling", g
    g[:E + 1] = 2 ** 31 - 1
    g[0] = -2 ** 31                             # the first expert has them all, the others none
    yield "extremes", g


@pytest.mark.parametrize("form", list(FORMS))
def test_groups_of_nonsense_select_rows_of_the_product_only(form):
    """The calls return, and write finite values into rows of their outputs and nothing beside them."""
    M, E, k, N, K = shape(form)
    P, F = M * k, N // 2
    x, h = (to_dev(synth.activations("normal", r, K, 1)) for r in (M, P))
    rep, pairs = same_experts(E, N, K), same_pairs(E, F, K)
    q8, w = raw(mmq.mmq_q8_1_bytes(M, K)), f32(M, k, value=0.5)
    space = raw(mmq.mmq_grouped_down_workspace_bytes(M, E, k, N, K))
    out = {"C": (P, N), "H": (P, F), "out": (M, N)}
    guard = {n: f32(r + 8, c, value=5.0) for n, (r, c) in out.items()}   # four rows on each side
    n = mmq.mmq_moe_group_bytes(M, E, k) // 4
    for kind, ints in nonsense(P, E, n):
        g = to_dev(ints.astype(np.int32))
        say("groups of nonsense", form, kind)
        mmq.mmq_q4K_grouped(M, E, k, N, K, x, g, rep, guard["C"][4:-4], q8)
        mmq.mmq_q4K_grouped_gated(M, E, k, F, K, x, g, pairs, guard["H"][4:-4], q8)
        mmq.mmq_q4K_grouped_down(M, E, k, N, K, h, g, w, rep, guard["out"][4:-4], space)
        torch.cuda.synchronize()
        for name, t in guard.items():
            assert bool((t[:4] == 5.0).all()) and bool((t[-4:] == 5.0).all()), (name, kind)
            assert bool(torch.isfinite(t).all()), (name, kind)


# rows of the experts in the wide form: none, one, part of a 32-row part, each number of parts, and
# several tiles
RAGGED = [0, 1, 31, 32, 33, 0, 64, 65, 96, 97, 127, 128, 129, 300, 5]


def ragged_ids(k):
    flat = np.concatenate([np.full(c, e) for e, c in enumerate(RAGGED)])
    flat = np.concatenate([flat, np.full(2200 - len(flat), -1)])
    np.random.default_rng(k).shuffle(flat)
    return flat.reshape(-1, k).astype(np.int32)


def rows_of(blocks, e, N, K):
    """Expert e's N rows of blocks of more of them."""
    return blocks.reshape(-1, K // 256, 144)[7 * e:7 * e + N].contiguous()


@pytest.mark.parametrize("per_pair", [False, True])
@pytest.mark.parametrize("k", [1, 2])
def test_ragged_experts_in_the_wide_form(k, per_pair):
    """Bit for bit the plain product of each expert's rows."""
    E, N, K = len(RAGGED), 2050, 1024
    ids = ragged_ids(k)
    M = ids.shape[0]
    assert gu.grouped_form(M * k, E, N, K) == "wide"
    rows = M * k if per_pair else M
    x = to_dev(synth.activations("normal_outliers", rows, K, N))
    blocks = to_dev(synth.q4k_weights("random_fields", N + 7 * E, K, 3)[0])
    n = mmq.mmq_q4K_repacked_bytes(N, K)
    rep, C = raw(E * n), f32(M * k, N)
    for e in range(E):
        mmq.repack_q4_K(rows_of(blocks, e, N, K), N, K, rep[e * n:(e + 1) * n])
    say("grouped wide, ragged", (M, E, k, N, K), per_pair)
    mmq.mmq_q4K_grouped(M, E, k, N, K, x, group(ids, E), rep, C,
                        raw(mmq.mmq_q8_1_bytes(rows, K)), per_pair=per_pair)
    flat = ids.reshape(-1)
    for e in range(E):
        ps = torch.from_numpy(np.nonzero(flat == e)[0]).cuda()
        assert len(ps) == RAGGED[e]
        if len(ps) == 0:
            continue
        xe = x[ps if per_pair else ps // k].contiguous()
        q8, want = raw(mmq.mmq_q8_1_bytes(len(ps), K)), f32(len(ps), N)
        mmq.quantize_q8_1(xe, len(ps), K, q8)
        mmq.mmq_q4K_q8_1_ex(len(ps), N, K, q8, rep[e * n:(e + 1) * n], want,
                            force_tile=mmq.MMQ_TILE_LARGE)
        assert torch.equal(C[ps], want), e
    assert bool(torch.isnan(C[torch.from_numpy(np.nonzero(flat < 0)[0]).cuda()]).all())


@pytest.mark.parametrize("k", [1, 2])
def test_ragged_experts_in_the_wide_gated_form(k):
    E, F, D = len(RAGGED), 1030, 1024
    ids = ragged_ids(k)
    M = ids.shape[0]
    assert gu.grouped_form(M * k, E, -(-F // 16) * 32, D) == "wide"
    x = to_dev(synth.activations("normal_outliers", M, D, F))
    gate, up = (to_dev(synth.q4k_weights("random_fields", F + 7 * E, D, s)[0]) for s in (3, 4))
    n = mmq.mmq_q4K_pair_bytes(F, D)
    rep, H = raw(E * n), f32(M * k, F)
    for e in range(E):
        mmq.repack_q4_K_pair(rows_of(gate, e, F, D), rows_of(up, e, F, D), F, D,
                             rep[e * n:(e + 1) * n])
    say("grouped gated wide, ragged", (M, E, k, F, D))
    mmq.mmq_q4K_grouped_gated(M, E, k, F, D, x, group(ids, E), rep, H,
                              raw(mmq.mmq_q8_1_bytes(M, D)))
    flat = ids.reshape(-1)
    for e in range(E):
        ps = torch.from_numpy(np.nonzero(flat == e)[0]).cuda()
        if len(ps) == 0:
            continue
        q8, want = raw(mmq.mmq_q8_1_bytes(len(ps), D)), f32(len(ps), F)
        mmq.quantize_q8_1(x[ps // k].contiguous(), len(ps), D, q8)
        mmq.mmq_q4K_q8_1_gated(len(ps), F, D, q8, rep[e * n:(e + 1) * n], want,
                               act=mmq.MMQ_ACT_SILU, force_tile=mmq.MMQ_TILE_LARGE)
        assert torch.equal(H[ps], want), e
    assert bool(torch.isnan(H[torch.from_numpy(np.nonzero(flat < 0)[0]).cuda()]).all())


@pytest.mark.parametrize("M,E,k,D,F", [(64, 8, 2, 512, 768), (61, 4, 3, 300, 512),
                                       (9, 16, 8, 256, 256), (1, 4, 2, 256, 512)])
def test_the_layer_of_many_tokens_against_that_of_a_few(M, E, k, D, F):
    """Both gated products within their bound of one oracle; both down products, on either's H, within
    the sum of their bounds of each other; and both layers are their own calls, bit for bit."""
    K = -(-D // 256) * 256      # the tokens' width
    gate, up = ([lu.weights(F, K, s + e) for e in range(E)] for s in (700, 900))
    ws = np.stack([lu.weights(D, F, 800 + e) for e in range(E)])
    n, m = mmq.mmq_q4K_pair_bytes(F, K), mmq.mmq_q4K_repacked_bytes(D, F)
    pairs, down = raw(E * n), raw(E * m)
    for e in range(E):
        mmq.repack_q4_K_pair(to_dev(gate[e]), to_dev(up[e]), F, K, pairs[e * n:(e + 1) * n])
        mmq.repack_q4_K(to_dev(ws[e]), D, F, down[e * m:(e + 1) * m])
    xh = synth.activations("normal_outliers", M, K, 1)
    rng = np.random.default_rng(2)
    logits = rng.standard_normal((M, E)).astype(np.float32)
    logits[M // 2] = -np.inf if M > 1 else logits[0]
    residual = rng.standard_normal((M, D)).astype(np.float32)
    x, lg, res = to_dev(xh), to_dev(logits), to_dev(residual)
    ids, w = torch.empty(M, k, dtype=torch.int32, device="cuda"), f32(M, k)
    plan = torch.zeros(mmq.mmq_moe_plan_bytes(M, E, k) // 4, dtype=torch.int32, device="cuda")
    say("layers of many and of a few", (M, E, k, D, F))
    mmq.mmq_moe_route(M, E, k, lg, ids, w, plan=plan)
    torch.cuda.synchronize()
    idh, wh = ids.cpu().numpy(), w.cpu().numpy()
    g = group(idh, E)
    H = {"few": f32(M * k, F, value=0.0), "many": f32(M * k, F, value=0.0)}
    q8 = raw(max(mmq.mmq_q8_1_bytes(M, K), mmq.mmq_q8_1_bytes(M * k, F)))
    mmq.mmq_q4K_moe_gated(M, E, k, F, K, x, plan, pairs, H["few"], q8)
    mmq.mmq_q4K_grouped_gated(M, E, k, F, K, x, g, pairs, H["many"], q8)
    want, err = lu.experts_gated(xh, idh, np.stack(gate), np.stack(up), "silu")
    used = idh.reshape(-1) >= 0
    got = {name: t.cpu().numpy() for name, t in H.items()}
    for name in H:
        lu.assert_close(got[name][used], want[used], err[used], what=name)
    lu.assert_close(got["few"][used], got["many"][used].astype(np.float64), 2 * err[used])
    space = raw(mmq.mmq_grouped_down_workspace_bytes(M, E, k, D, F))
    last = {}
    for name, h in H.items():
        few, many = f32(M, D), f32(M, D)
        mmq.mmq_q4K_moe_down(M, E, k, D, F, h, plan, w, down, few, q8, residual=res)
        mmq.mmq_q4K_grouped_down(M, E, k, D, F, h, g, w, down, many, space, residual=res)
        torch.cuda.synchronize()
        out, oerr = lu.experts_down(got[name], idh, wh, ws, residual)
        lu.assert_close(few.cpu().numpy(), out, oerr)
        lu.assert_close(many.cpu().numpy(), out, oerr)
        lu.assert_close(few.cpu().numpy(), many.double().cpu().numpy(), 2 * oerr)
        last[name] = few if name == "few" else many
    if K == D:      # the layers take one width
        few, many = f32(M, D), f32(M, D)
        mmq.mmq_q4K_moe(M, E, k, D, F, x, lg, pairs, down, few,
                        raw(mmq.mmq_moe_workspace_bytes(M, E, k, D, F)), residual=res)
        mmq.mmq_q4K_grouped_moe(M, E, k, D, F, x, lg, pairs, down, many,
                                raw(mmq.mmq_grouped_moe_workspace_bytes(M, E, k, D, F)),
                                residual=res)
        assert torch.equal(few, last["few"]) and torch.equal(many, last["many"])
