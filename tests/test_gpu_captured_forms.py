"""Every form of the grouped products and of the q4_G products captured into a graph and replayed with
other inputs between the replays, on a stream handed to the call, and called by two threads at once:
each time the bits of an eager call on the same inputs.
"""
import threading

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


def bits(t):
    return t.contiguous().view(torch.uint8)


class Grouped:
    """The sort, the grouped product, the gated one and the weighted sum of one shape, each with the
    buffers of one caller: load(seed) gives it inputs, call() runs them."""

    def __init__(self, form, M, E, k, N, K):
        assert gu.grouped_form(M * k, E, N, K) == form
        self.sizes, self.F = (M, E, k, N, K), N // 2
        one = raw(mmq.mmq_q4K_repacked_bytes(N, K))
        mmq.repack_q4_K(to_dev(synth.q4k_weights("fit", N, K, 3)[0]), N, K, one)
        pair = raw(mmq.mmq_q4K_pair_bytes(self.F, K))
        mmq.repack_q4_K_pair(to_dev(lu.weights(self.F, K, 1)), to_dev(lu.weights(self.F, K, 2)),
                             self.F, K, pair)
        self.rep, self.pairs = one.repeat(E), pair.repeat(E)

    def caller(self):
        M, E, k, N, K = self.sizes
        return dict(ids=torch.full((M, k), -1, dtype=torch.int32, device="cuda"),
                    x=torch.zeros(M, K, device="cuda"), h=torch.zeros(M * k, K, device="cuda"),
                    w=torch.zeros(M, k, device="cuda"), q8=raw(mmq.mmq_q8_1_bytes(M, K)),
                    space=raw(mmq.mmq_grouped_down_workspace_bytes(M, E, k, N, K)),
                    g=torch.zeros(mmq.mmq_moe_group_bytes(M, E, k) // 4, dtype=torch.int32,
                                  device="cuda"),
                    C=f32(M * k, N), H=f32(M * k, self.F), out=f32(M, N))

    def load(self, c, seed):
        M, E, k, N, K = self.sizes
        g = torch.Generator(device="cuda").manual_seed(seed)
        c["ids"].copy_(torch.randint(-1, E, (M, k), generator=g, device="cuda"))
        for n in ("x", "h", "w"):
            c[n].copy_(torch.randn(c[n].shape, generator=g, device="cuda"))
        for n in ("C", "H", "out"):
            c[n].fill_(NAN)

    def call(self, c, **kw):
        M, E, k, N, K = self.sizes
        mmq.mmq_moe_group(M, E, k, c["ids"], c["g"], **kw)
        mmq.mmq_q4K_grouped(M, E, k, N, K, c["x"], c["g"], self.rep, c["C"], c["q8"], **kw)
        mmq.mmq_q4K_grouped_gated(M, E, k, self.F, K, c["x"], c["g"], self.pairs, c["H"], c["q8"],
                                  **kw)
        mmq.mmq_q4K_grouped_down(M, E, k, N, K, c["h"], c["g"], c["w"], self.rep, c["out"],
                                 c["space"], **kw)

    def results(self, c):
        return [bits(c[n]) for n in ("C", "H", "out")]


class Q4G:
    def __init__(self, M, N, K, group, x):
        self.sizes, self.t = (M, N, K), x
        self.format = mmq.q4G_format(group, torch.float16, True)
        n = -(-K // group)
        g = torch.Generator(device="cuda").manual_seed(N)
        w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
        s = (0.02 * torch.randn(N, n, generator=g, device="cuda")).half()
        z = torch.randint(0, 16, (N, n), generator=g, device="cuda").half()
        self.rep = raw(mmq.mmq_q4G_repacked_bytes(N, K, self.format))
        mmq.repack_q4_G(w, s, z, N, K, self.format, self.rep)

    def caller(self):
        M, N, K = self.sizes
        return dict(x=torch.zeros(M, K, dtype=self.t, device="cuda"), y=f32(M, N))

    def load(self, c, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        c["x"].copy_(torch.randn(c["x"].shape, generator=g, device="cuda"))
        c["y"].fill_(NAN)

    def call(self, c, **kw):
        mmq.mmq_q4G(*self.sizes, c["x"], self.rep, self.format, c["y"], act=mmq.MMQ_ACT_SILU, **kw)

    def results(self, c):
        return [bits(c["y"])]


BF, F32 = torch.bfloat16, torch.float32
# x of all records in LDS or not, one tile to a workgroup or several, two workgroups to a compute unit;
# LDS below and above 64 KiB
OPS = {
    "narrow": lambda: Grouped("narrow", 200, 8, 2, 8200, 768),
    "split2": lambda: Grouped("split2", 200, 8, 2, 2050, 2048),
    "split4": lambda: Grouped("split4", 300, 8, 2, 1290, 4352),
    "wide": lambda: Grouped("wide", 4096, 4, 2, 2050, 2048),
    "q4_G 1": lambda: Q4G(1, 100, 512, 64, BF),
    "q4_G 4 of many rows": lambda: Q4G(4, 9000, 2048, 128, BF),
    "q4_G 16": lambda: Q4G(16, 4200, 2048, 64, BF),
    "q4_G 16 long": lambda: Q4G(16, 4200, 8192, 128, BF),
    "q4_G 3 float32": lambda: Q4G(3, 200, 1024, 32, F32),
    "q4_G 16 float32": lambda: Q4G(16, 4200, 1024, 32, F32),
    "q4_G 16 float32 long": lambda: Q4G(16, 4200, 8192, 128, F32),
}


def want(op, seed):
    c = op.caller()
    op.load(c, seed)
    op.call(c)
    torch.cuda.synchronize()
    return op.results(c)


def assert_same(op, c, seed, what):
    torch.cuda.synchronize()
    for a, b in zip(op.results(c), want(op, seed)):
        assert torch.equal(a, b), (what, seed)


@pytest.mark.parametrize("name", list(OPS))
def test_captured_and_replayed(name):
    op = OPS[name]()
    c = op.caller()
    op.load(c, 0)
    op.call(c)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    say("captured", name)
    with torch.cuda.graph(graph, stream=side):
        op.call(c)
    for seed in (1, 2, 3, 1):
        op.load(c, seed)
        torch.cuda.synchronize()
        graph.replay()
        assert_same(op, c, seed, name)


@pytest.mark.parametrize("name", list(OPS))
def test_on_a_stream_handed_over(name):
    """The stream as an object and as its number, with another stream current."""
    op = OPS[name]()
    side = torch.cuda.Stream()
    for seed, stream in ((4, side), (5, side.cuda_stream)):
        c = op.caller()
        with torch.cuda.stream(side):       # the inputs are made there, behind what is queued
            torch.cuda._sleep(200000)
            op.load(c, seed)
        say("on a stream", name)
        op.call(c, stream=stream)
        side.synchronize()
        assert_same(op, c, seed, name)


def test_two_threads_at_once():
    """Calls of one kernel with different LDS sizes, and of several kernels, from two threads, each on
    its own stream with its own buffers."""
    ops = [[OPS[n]() for n in names] for names in (
        ("q4_G 16", "q4_G 16 float32", "wide"), ("q4_G 16 long", "q4_G 3 float32", "split4"))]
    ops[1].append(Q4G(16, 4200, 1024, 64, BF))      # the kernel of "q4_G 16", less LDS
    sides = []
    for mine in ops:
        calls = [(op, op.caller()) for op in mine]
        for i, (op, c) in enumerate(calls):
            op.load(c, 20 + i)
        sides.append((calls, torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed = []

    def work(calls, stream):
        try:
            for _ in range(20):
                for op, c in calls:
                    op.call(c, stream=stream)
        except Exception as e:      # (shown by the assertion below)
            failed.append(repr(e))

    say("two threads")
    threads = [threading.Thread(target=work, args=s) for s in sides]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for calls, _ in sides:
        for i, (op, c) in enumerate(calls):
            assert_same(op, c, 20 + i, i)
