"""Matrix-vector products with group scales where the result is known to a rounding: one value in each
token that is not 0, in every place of a record and for every number of tokens, with x on every way into
LDS; and finite tokens of any size, up to the greatest float.
"""
import numpy as np
import pytest

from oracle import q4g_oracle as qo
from tests import layer_util as lu
from tests import q4g_util as qu
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

mmq = pytest.importorskip("q4_q8_int8_amd")
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    yield
    torch.cuda.synchronize()


def np64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


class Matrix:
    """Random values with scale `s` everywhere and whole zeros in 0..15."""

    def __init__(self, N, K, group, s=1.0, scale="f16", seed=0):
        g = torch.Generator().manual_seed(seed)
        n = -(-K // group)
        self.N, self.K, self.group, self.size = N, K, group, s
        self.w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
        self.s = torch.full((N, n), s, dtype=DT[scale], device="cuda")
        self.z = torch.randint(0, 16, (N, n), generator=g).to(DT[scale]).cuda()
        self.format = mmq.q4G_format(group, DT[scale], True)
        self.rep = torch.empty(mmq.mmq_q4G_repacked_bytes(N, K, self.format), dtype=torch.uint8,
                               device="cuda")
        mmq.repack_q4_G(self.w, self.s, self.z, N, K, self.format, self.rep)
        self.v = qo.values(self.w.cpu().numpy()).astype(np.float64)
        self.zeros = np.repeat(np64(self.z), group, axis=1)[:, :K]

    def __call__(self, x):
        y = torch.full((x.shape[0], self.N), NAN, device="cuda")
        mmq.mmq_q4G(x.shape[0], self.N, self.K, x, self.rep, self.format, y)
        return np64(y)

    def product(self, x):
        return qo.product(np64(x), self.w.cpu().numpy(), np64(self.s), np64(self.z), self.group,
                          0.0 if x.dtype == torch.float16 else 16.0)


def one_value_each(values, at, K, t):
    """Tokens [len(at), K] with values[i] at at[i] and 0 elsewhere."""
    x = np.zeros((len(at), K), np.float32)
    x[np.arange(len(at)), at] = values
    return torch.from_numpy(x).to(DT[t]).cuda()


# K of two records, the second short, in tiles of one workgroup each and in more than a round of the compute
# units; and of more records than LDS holds x of, for many tokens, both ways
@pytest.mark.parametrize("x", list(DT))
@pytest.mark.parametrize("N,K,group,counts", [
    (35, 160, 32, range(1, 17)), (4200, 160, 64, (1, 2, 3, 4, 5, 8, 9, 16)),
    (35, 8192, 128, (3, 16)), (4200, 8192, 64, (4, 7, 16))])
def test_one_value_each(N, K, group, counts, x):
    m = Matrix(N, K, group, seed=N + K)
    places = np.arange(K) if K == 160 else np.random.default_rng(K).permutation(K)[:48]
    for M in counts:
        say("q4_G, one value each", (M, N, K), x)
        for i in range(0, len(places), M):
            at = np.resize(places[i:i + M], M)
            values = qu.full_mantissas(M, 100 * M + i)
            a = one_value_each(values, at, K, x)
            got, used = m(a), np64(a)[np.arange(M), at][:, None]
            v, z = m.v[:, at].T, m.zeros[:, at].T
            if x == "f32":
                assert np.array_equal(used[:, 0], values.astype(np.float64))
                lu.assert_close(got, used * (v - z), qu.one_value_bound(used, v, z), what=str(at))
            else:   # at most 11 and 4 bits
                assert np.array_equal(got, used * (v - z)), at


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", [(35, 160), (4200, 160), (35, 8192)])
def test_one_value_of_any_size(N, K, x):
    """Up to the greatest float of the type; the results, 2^-6 x (v - z), are finite."""
    m = Matrix(N, K, 32, s=2.0 ** -6, seed=3)
    greatest = torch.finfo(DT[x]).max
    for M in (1, 3, 9, 16):
        at = np.random.default_rng(M).permutation(K)[:M]
        for size in (1e35, 1e36, 1e37, 1e38, greatest):
            say("q4_G, one value of", size, (M, N, K), x)
            a = one_value_each(np.where(np.arange(M) % 2, -size, size), at, K, x)
            used = np64(a)[np.arange(M), at][:, None]
            v, z = m.v[:, at].T, m.zeros[:, at].T
            lu.assert_close(m(a), used * (v - z) / 64, qu.one_value_bound(used, v, z) / 64)


@pytest.mark.parametrize("x,size", [("f32", 1e34), ("f32", 3e38), ("bf16", 1e34), ("bf16", 3e38),
                                    ("f32", 2.0 ** -110), ("f32", 2.0 ** -124),
                                    ("bf16", 2.0 ** -110), ("bf16", 2.0 ** -124),
                                    ("f16", 6e4), ("f16", 2.0 ** -23)])
def test_tokens_of_any_size(x, size):
    """Every value of a token of this size, in groups of a record and of several. What is below 2^-126
    after the operands' factor of 2^-12 is rounded to 2^-149, a unit per sum of a piece's products
    with 16 + v (at most 31) or with 1 (taken 16 + z times, at most 31): 2^-137 each in the result,
    which is 4096 times as large."""
    for K, group in ((512, 128), (1056, 1056)):
        m = Matrix(33, K, group, s=2.0 ** -14 if size > 1 else 1.0, scale="bf16", seed=5)
        g = torch.Generator().manual_seed(K)
        for M in (2, 4, 11):
            a = ((torch.rand(M, K, generator=g) + 0.1).clamp(max=1.0) * size
                 * torch.where(torch.rand(M, K, generator=g) < 0.5, -1.0, 1.0)).to(DT[x]).cuda()
            say("q4_G, tokens of", size, x, (M, K))
            y, T = m.product(a)
            least = 0.0 if x == "f16" else 3 * (1 + 31) * K * 2.0 ** -137 * m.size
            lu.assert_close(m(a), y, qo.bound(T, K) + least + 2.0 ** -149)
