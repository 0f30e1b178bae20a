"""The checked entry points without a given stream: on the current stream, in a
capture, and from two threads at once (the calls let go of the interpreter's lock)."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

vit = pytest.importorskip("vision_transformer_encoder_layernorm_b200")

T, H, D = 300, 4, 72
C = H * D


@pytest.fixture(scope="module")
def ctx():
    c = vit.Context(C, H, D, 4 * C, vit.BF16)
    yield c
    c.close()


class Calls:
    """One of each entry point, chained from x to `out`."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.src = torch.randn(T, C, device="cuda", generator=g).to(torch.bfloat16)
        self.x = torch.zeros(T, C, **bf)
        self.gamma = torch.ones(C, **bf)
        self.w = torch.randn(C, C, device="cuda", generator=g).to(torch.bfloat16)
        self.pos = torch.randint(0, 50, (T, 3), device="cuda", generator=g).int()
        self.n, self.r, self.y, self.out, self.back = (torch.zeros(T, C, **bf) for _ in range(5))
        self.a = u8(T, vit.mx4_row_bytes(C)), u8(vit.mx4_scale_bytes(T, C))
        self.wq = u8(C, vit.mx4_row_bytes(C)), u8(vit.mx4_scale_bytes(C, C))
        self.m8 = u8(T, vit.mx8_row_bytes(C)), u8(vit.mx8_scale_bytes(T, C))

    def run(self, ctx, **kw):
        ctx.rmsnorm(self.x, self.gamma, self.n, **kw)
        ctx.rmsnorm_mx8(self.x, self.gamma, *self.m8, **kw)
        ctx.rope3d(self.n.view(T, H, D), self.pos, (12, 12, 12), out=self.r.view(T, H, D), **kw)
        ctx.mx4_quantize(self.r, *self.a, **kw)
        ctx.mx4_quantize(self.w, *self.wq, **kw)
        ctx.mx4_dequantize(*self.a, self.back, **kw)
        ctx.linear_mx4(self.a, self.wq, None, self.out, C, epi=vit.EPI_BIAS_RESIDUAL,
                       residual=self.back, **kw)

    def outputs(self):
        return [t.clone() for t in (self.n, self.r, self.back, self.out, *self.a, *self.m8)]

    def expected(self, ctx):
        self.x.copy_(self.src)
        self.run(ctx)
        torch.cuda.synchronize()
        want = self.outputs()
        self.x.zero_()
        self.run(ctx)
        torch.cuda.synchronize()
        return want


def same(got, want):
    return all(torch.equal(g, w) for g, w in zip(got, want))


def test_current_stream(ctx):
    c = Calls(1)
    want = c.expected(ctx)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # some ms: calls on another stream would read x before
        c.x.copy_(c.src)
        c.run(ctx)
        got = c.outputs()
    torch.cuda.synchronize()
    assert same(got, want) and ctx.device_status() == 0


def test_capture_on_the_current_stream(ctx):
    c = Calls(2)
    want = c.expected(ctx)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(ctx)
    c.x.copy_(c.src)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert same(c.outputs(), want) and ctx.device_status() == 0
    del g


@pytest.mark.parametrize("fresh", [False, True])
def test_two_threads(ctx, fresh):
    """Two threads on one context (the first checked calls of it when fresh)."""
    c = vit.Context(C, H, D, 4 * C, vit.BF16) if fresh else ctx
    jobs = [Calls(3), Calls(4)]
    want = [j.expected(ctx) for j in jobs]
    errors, start = [], threading.Barrier(2)

    def work(j):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                j.x.copy_(j.src)
                for _ in range(100):
                    j.run(c)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for j, w in zip(jobs, want):
        assert same(j.outputs(), w)
    assert c.device_status() == 0
    if fresh:
        c.close()
