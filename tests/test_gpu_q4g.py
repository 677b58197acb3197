"""The matrix-vector products with group scales on the GPU, against the float64 oracle: every type, both
kinds of zeros and scales, group sizes that end inside a record and past K, ragged rows, 1 to 16
tokens, the epilogue, graphs and two streams.
"""
import numpy as np
import pytest

from oracle import layer_oracle as lo
from oracle import q4g_oracle as qo
from tests import layer_util as lu
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

mmq = pytest.importorskip("q4_q8_int8_amd")
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a step of each type relative to the value, and its least step's half below the normal range
HALF = {"f32": (2.0 ** -24, 2.0 ** -150), "f16": (2.0 ** -11, 2.0 ** -25),
        "bf16": (2.0 ** -8, 2.0 ** -134)}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    yield
    torch.cuda.synchronize()


def np64(t):
    torch.cuda.synchronize()
    return None if t is None else t.double().cpu().numpy()


class Matrix:
    """Random q4_G weights: the packed bytes, scales of both signs, and, with zeros, zeros that are not
    whole numbers and lie outside 0..15 too."""

    def __init__(self, N, K, group, scale="f16", zeros=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        n = -(-K // group)
        self.N, self.K, self.group = N, K, group
        self.w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
        self.s = (0.02 * torch.randn(N, n, generator=g)).to(DT[scale]).cuda()
        self.z = (8.0 + 5.0 * torch.randn(N, n, generator=g)).to(DT[scale]).cuda() if zeros else None
        self.format = mmq.q4G_format(group, DT[scale], zeros)
        self.rep = torch.full((mmq.mmq_q4G_repacked_bytes(N, K, self.format),), 255,
                              dtype=torch.uint8, device="cuda")
        mmq.repack_q4_G(self.w, self.s, self.z, N, K, self.format, self.rep)

    def product(self, x):
        # bf16 operands (those of float32 tokens too) hold 16 + v
        return qo.product(np64(x), self.w.cpu().numpy(), np64(self.s), np64(self.z), self.group,
                          0.0 if x.dtype == torch.float16 else 16.0)


def tokens(M, K, t, seed):
    g = torch.Generator().manual_seed(1000 + seed)
    x = torch.randn(M, K, generator=g)
    x[torch.rand(M, K, generator=g) < 0.01] *= 20.0
    return x.to(DT[t]).cuda()


def rounded(want, err, y):
    half, least = HALF[y]
    return err + half * (np.abs(want) + err) + least


def check(m, x, y="f32", act="none", bias=None, residual=None):
    M = x.shape[0]
    out = torch.full((M, m.N), NAN, dtype=DT[y], device="cuda")
    mmq.mmq_q4G(M, m.N, m.K, x, m.rep, m.format, out, bias=bias, residual=residual,
                act=mmq.ACTIVATIONS[act])
    P, T = m.product(x)
    z, dz = P, qo.bound(T, m.K)
    if bias is not None:
        z = P + np64(bias)
        dz = dz + lo.EPS * (np.abs(z) + dz)
    want, err = lo.act(z, act), lo.act_err(z, dz, act)
    if residual is not None:
        want = want + np64(residual)
        err = err + lo.EPS * (np.abs(want) + err)
    lu.assert_close(np64(out), want, rounded(want, err, y), what=f"{M}x{m.N}x{m.K}")
    return out


# K of one record, of less, of a short last one, of more records than wavefronts; groups of a step, of
# steps that cross records, of a record, of more, of the whole row and past it
SHAPES = [(1, 16, 32, 32), (1, 1, 128, 128), (3, 17, 96, 32), (1, 33, 160, 160), (2, 40, 512, 96),
          (5, 15, 1056, 64), (4, 100, 1280, 256), (6, 31, 2080, 128), (10, 48, 800, 4096),
          (11, 20, 2304, 32), (16, 64, 1024, 128), (1, 70, 4352, 64), (8, 130, 3104, 224)]


@pytest.mark.parametrize("x", list(DT))
@pytest.mark.parametrize("scale,zeros", [("f16", True), ("f16", False), ("bf16", True),
                                         ("bf16", False)])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_q4g(M, N, K, group, scale, zeros, x):
    m = Matrix(N, K, group, scale, zeros, seed=N + K)
    say("q4_G", (M, N, K), "group", group, scale, zeros, x)
    check(m, tokens(M, K, x, M))


@pytest.mark.parametrize("x", list(DT))
def test_every_number_of_tokens(x):
    m = Matrix(50, 672, 64)
    for M in range(1, 17):
        say("q4_G", M, "tokens", x)
        a = tokens(M, m.K, x, M)
        out = check(m, a)
        # a token's result does not depend on the tokens beside it, within a form
        if M > 1 and x != "f32":
            one = torch.empty(1, m.N, device="cuda")
            mmq.mmq_q4G(1, m.N, m.K, a[M - 1:].contiguous(), m.rep, m.format, one)
            assert np.array_equal(np64(one)[0], np64(out)[M - 1])


@pytest.mark.parametrize("x", list(DT))
@pytest.mark.parametrize("y", list(DT))
@pytest.mark.parametrize("act", lo.ACTS)
def test_epilogue(x, y, act):
    m = Matrix(75, 544, 32, seed=7)
    for M in (1, 7):
        g = torch.Generator().manual_seed(M)
        bias = torch.randn(m.N, generator=g).cuda()
        res = torch.randn(M, m.N, generator=g).to(DT[y]).cuda()
        say("q4_G epilogue", x, y, act, M)
        a = tokens(M, m.K, x, M)
        check(m, a, y, act)
        check(m, a, y, act, bias=bias)
        out = check(m, a, y, act, bias=bias, residual=res)
        stream = res.clone()                       # the residual stream, updated in place
        mmq.mmq_q4G(M, m.N, m.K, a, m.rep, m.format, stream, bias=bias, residual=stream,
                    act=mmq.ACTIVATIONS[act])
        assert torch.equal(stream, out)


def test_integers_are_exact():
    """Small integers times scale 1: every sum is exact, whatever the order."""
    for x, M in (("f32", 5), ("f16", 16), ("bf16", 3)):
        m = Matrix(40, 1120, 32, seed=3)
        m.s.fill_(1.0)
        m.z.copy_(torch.randint(0, 16, m.z.shape).to(m.z.dtype))
        mmq.repack_q4_G(m.w, m.s, m.z, m.N, m.K, m.format, m.rep)
        a = torch.randint(-8, 9, (M, m.K)).to(DT[x]).cuda()
        out = torch.empty(M, m.N, device="cuda")
        mmq.mmq_q4G(M, m.N, m.K, a, m.rep, m.format, out)
        assert np.array_equal(np64(out), m.product(a)[0]), x


@pytest.mark.parametrize("x,size", [("f16", 3e-7), ("f16", 5e-5), ("f16", 4e4), ("bf16", 1e-30),
                                    ("bf16", 1e30), ("f32", 1e-25), ("f32", 1e30)])
def test_small_and_large_activations(x, size):
    """f16 values below their normal range count in full; nothing overflows on the way."""
    m = Matrix(33, 512, 128, scale="bf16", seed=5)
    a = (torch.randn(4, m.K, generator=torch.Generator().manual_seed(1)).clamp(-1.5, 1.5)
         * size).to(DT[x]).cuda()
    check(m, a)


def test_a_token_of_nan_stays_alone():
    m = Matrix(20, 256, 64)
    for x in DT:
        a = tokens(6, m.K, x, 1)
        clean = torch.empty(6, m.N, device="cuda")
        mmq.mmq_q4G(6, m.N, m.K, a, m.rep, m.format, clean)
        a[2, 5], a[4, 100] = NAN, float("inf")
        out = torch.empty(6, m.N, device="cuda")
        mmq.mmq_q4G(6, m.N, m.K, a, m.rep, m.format, out)
        keep = [0, 1, 3, 5]
        assert np.array_equal(np64(out)[keep], np64(clean)[keep]), x


def test_wide_and_long():
    """More row tiles than a round of the compute units, and more records than are loaded ahead."""
    for (M, N, K, group, x) in ((1, 9000, 256, 128, "f16"), (2, 24, 33000 // 32 * 32, 32, "f32"),
                                (16, 4100, 512, 64, "bf16")):
        say("q4_G", (M, N, K))
        check(Matrix(N, K, group, seed=1), tokens(M, K, x, 2))


# tokens that do not fit the LDS for all records of a wavefront: one tile to a workgroup, and several;
# float32 tokens kept for several tiles; more tiles than one workgroup's sums of them fit the LDS
@pytest.mark.parametrize("M,N,K,group,x", [
    (16, 40, 8192, 128, "f16"), (13, 40, 8192, 64, "bf16"), (16, 4200, 8192, 128, "bf16"),
    (9, 4200, 4096, 32, "f32"), (3, 4200, 512, 64, "f32"), (9, 4200, 256, 128, "f32"),
    (4, 8300, 640, 64, "f32"), (4, 8300, 1152, 32, "bf16"), (16, 25000, 2048, 256, "bf16"),
    (16, 32810, 1024, 64, "f32")])
def test_many_tiles_and_many_tokens(M, N, K, group, x):
    say("q4_G", (M, N, K), "group", group, x)
    check(Matrix(N, K, group, seed=4), tokens(M, K, x, 6))


def test_weights_past_4_gib():
    """The last rows' packed values and records start more than 4 GiB into both."""
    N, K, group = (1 << 21) + 40, 4128, 128
    n = -(-K // group)
    f = mmq.q4G_format(group, torch.float16, False)
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.rand(N, n, device="cuda").half()
    rep = torch.empty(mmq.mmq_q4G_repacked_bytes(N, K, f), dtype=torch.uint8, device="cuda")
    assert (N - 64) * K // 2 > 2 ** 32
    say("q4_G past 4 GiB")
    mmq.repack_q4_G(w, s, None, N, K, f, rep)
    x, y = tokens(2, K, "bf16", 3), torch.full((2, N), NAN, device="cuda")
    mmq.mmq_q4G(2, N, K, x, rep, f, y)
    for rows in (slice(0, 20), slice(N - 50, N)):
        P, T = qo.product(np64(x), w[rows].cpu().numpy(), np64(s[rows]), None, group, 16.0)
        err = qo.bound(T, K)
        lu.assert_close(np64(y[:, rows]), P, rounded(P, err, "f32"))
    assert bool(torch.isfinite(y).all())


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,S", [(96, 4), (64, 2), (128, 1), (288, 1)])
def test_repack_layout(group, S, zeros):
    """The records as documented: dwords [c][row][m], nibbles j and j + 4 of two neighbouring values, then
    S scales and S zeros of every row."""
    N, K = 35, 288
    m = Matrix(N, K, group, zeros=zeros, seed=11)
    torch.cuda.synchronize()
    v = np.zeros((48, 384), np.int64)
    v[:N, :K] = qo.values(m.w.cpu().numpy())
    want = np.zeros((3, 3, 4, 16, 4), np.uint32)
    for e in range(8):
        part = v.reshape(3, 16, 3, 4, 4, 8)[..., e]           # tile, row, record, m, c
        want |= (part.transpose(0, 2, 4, 1, 3) << (4 * (e // 2 + 4 * (e % 2)))).astype(np.uint32)
    img = m.rep.cpu().numpy().reshape(3, 3, -1)
    assert np.array_equal(img[..., :1024].copy().view(np.uint32), want.reshape(3, 3, -1))
    at = 1024
    for t in (m.s, m.z)[:1 + zeros]:
        bits = t.cpu().view(torch.int16).numpy().view(np.uint16)
        s = np.zeros((48, 3 * S), np.uint16)
        k = np.arange(3 * S) * (128 // S)
        s[:N, k < K] = bits[:, k[k < K] // group]
        got = img[..., at:at + 32 * S].copy().view(np.uint16).reshape(3, 3, 16, S)
        assert np.array_equal(got, s.reshape(3, 16, 3, S).transpose(0, 2, 1, 3))
        at += 32 * S
    assert img.shape[2] == at


def test_decode_step_in_a_graph_and_on_two_streams():
    """Two products behind one another (up with silu, down with the residual stream), captured per
    stream and replayed together with other inputs in between."""
    up, down = Matrix(96, 256, 64, seed=1), Matrix(256, 96, 32, "bf16", False, seed=2)
    sides = []
    say("q4_G in graphs")
    for M in (1, 4):
        d = dict(s=torch.cuda.Stream(), M=M, x=tokens(M, 256, "bf16", M),
                 h=torch.empty(M, 96, dtype=torch.bfloat16, device="cuda"),
                 y=torch.empty(M, 256, dtype=torch.bfloat16, device="cuda"))

        def call(d, y, h):
            mmq.mmq_q4G(d["M"], 96, 256, d["x"], up.rep, up.format, h, act=mmq.MMQ_ACT_SILU)
            mmq.mmq_q4G(d["M"], 256, 96, h, down.rep, down.format, y, residual=d["x"])
        torch.cuda.synchronize()
        with torch.cuda.stream(d["s"]):
            call(d, d["y"], d["h"])
        torch.cuda.synchronize()
        d["g"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(d["g"], stream=d["s"]):
            call(d, d["y"], d["h"])
        sides.append(d)
    for i in range(4):
        for d in sides:
            d["x"].copy_(tokens(d["M"], 256, "bf16", 50 + i))
            d["y"].fill_(NAN)
        torch.cuda.synchronize()
        for d in sides:
            with torch.cuda.stream(d["s"]):
                d["g"].replay()
        torch.cuda.synchronize()
        for d in sides:
            y, h = torch.empty_like(d["y"]), torch.empty_like(d["h"])
            call(d, y, h)
            assert np.array_equal(np64(y), np64(d["y"])), i


def test_python_checks_tensors():
    m = Matrix(32, 256, 64)
    x, y = tokens(2, 256, "f16", 1), torch.empty(2, 32, device="cuda")
    ok = dict(x=x, rep=m.rep, y=y, bias=None, residual=None)
    for bad in (dict(x=x.double()), dict(x=x[:1]), dict(x=x.t()), dict(rep=m.rep[:-2]),
                dict(y=y[:1]), dict(y=y.int()), dict(x=x.cpu()), dict(residual=y.half()),
                dict(bias=torch.zeros(32, device="cuda").half()),
                dict(bias=torch.zeros(31, device="cuda")), dict(x=None)):
        a = {**ok, **bad}
        with pytest.raises(mmq.MMQArgumentError):
            mmq.mmq_q4G(2, 32, 256, a["x"], a["rep"], m.format, a["y"], bias=a["bias"],
                        residual=a["residual"])
    for w, s, z in ((m.w[:-1], m.s, m.z), (m.w, m.s[:-1], m.z), (m.w, m.s.bfloat16(), m.z),
                    (m.w, m.s, m.z[:, :-1].contiguous()), (m.w.int(), m.s, m.z)):
        with pytest.raises(mmq.MMQArgumentError):
            mmq.repack_q4_G(w, s, z, 32, 256, m.format, m.rep)
    with pytest.raises(mmq.MMQError):
        mmq.repack_q4_G(m.w, m.s, None, 32, 256, m.format, m.rep)
