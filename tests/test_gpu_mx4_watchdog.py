"""Failure detection in vit_linear_mx4's kernels without a GPU fault, as in
test_gpu_watchdog.py: stage barriers are told to expect more bytes than their
copies deliver (vit_debug_lost_tx), the bounded waits (2 s each) run out, the
kernels wind down and report VIT_ERR_TIMEOUT, and the context keeps working."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

vit = pytest.importorskip("vision_transformer_encoder_layernorm_b200")

TIMEOUT = 6  # VIT_ERR_TIMEOUT
MARK = 7.0   # what y holds before a call that gives up


class Call:
    """A vit_linear_mx4 call that takes the form named by VIT_MX4_TILE."""

    def __init__(self, M, N, K, epi):
        self.ctx = vit.Context(1152, 16, 72, 4304, vit.BF16)
        g = torch.Generator(device="cuda").manual_seed(M + N + K)
        self.K, self.epi = K, epi
        self.a, self.w = (self.quantised(n, K, g) for n in (M, N))
        self.res = torch.randn(M, N, device="cuda", generator=g).to(torch.bfloat16)
        self.y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def quantised(self, rows, K, g):
        x = torch.randn(rows, K, device="cuda", generator=g).to(torch.bfloat16)
        codes = torch.empty(rows, vit.mx4_row_bytes(K), dtype=torch.uint8, device="cuda")
        scales = torch.empty(vit.mx4_scale_bytes(rows, K), dtype=torch.uint8, device="cuda")
        self.ctx.mx4_quantize(x, codes, scales)
        return codes, scales

    def run(self):
        """The status, the host's wait for it in seconds, and y."""
        self.y.fill_(MARK)
        torch.cuda.synchronize()
        t0 = time.monotonic()
        self.ctx.linear_mx4(self.a, self.w, None, self.y, self.K, epi=self.epi,
                            residual=self.res if self.epi == vit.EPI_BIAS_RESIDUAL else None)
        status = self.ctx.device_status()  # synchronises
        return status, time.monotonic() - t0, self.y.clone()


@pytest.mark.parametrize("tile,M,N,K,epi", [
    ("1x128x2", 33, 136, 2049, vit.EPI_BIAS_RESIDUAL), ("1x128x4", 128, 264, 2305, vit.EPI_BIAS_GELU),
    ("1x128x8", 1, 1152, 4304, vit.EPI_BIAS)])
def test_split_tile_that_lost_bytes_is_not_written(monkeypatch, tile, M, N, K, epi):
    """Only the last CTA of a cluster gives up; the others must not add what it left
    in its shared memory to their own columns of the tile."""
    monkeypatch.setenv("VIT_MX4_TILE", tile)
    c = Call(M, N, K, epi)
    status, _, want = c.run()
    assert status == 0
    c.ctx.debug_lost_tx(16)
    status, waited, y = c.run()
    assert status == TIMEOUT and 1.5 <= waited <= 30.0, (status, waited)
    assert torch.all(y == MARK)
    c.ctx.debug_lost_tx(0)
    status, _, y = c.run()
    assert status == 0 and torch.equal(y, want)
    c.ctx.close()


@pytest.mark.parametrize("tile", ["1x128", "2x128", "2x192", "2x256"])
@pytest.mark.parametrize("M,N,K,epi", [
    (300, 264, 130, vit.EPI_BIAS),                # every copy is issued before a wait runs out
    (300, 392, 4304, vit.EPI_BIAS_RESIDUAL)])     # the producer waits too, residual copies in flight
def test_tiles_that_lost_bytes_time_out(monkeypatch, tile, M, N, K, epi):
    monkeypatch.setenv("VIT_MX4_TILE", tile)
    c = Call(M, N, K, epi)
    status, _, want = c.run()
    assert status == 0
    c.ctx.debug_lost_tx(16)
    status, waited, _ = c.run()
    assert status == TIMEOUT and 1.5 <= waited <= 30.0, (status, waited)
    c.ctx.debug_lost_tx(0)
    for _ in range(3):
        status, _, y = c.run()
        assert status == 0 and torch.equal(y, want)
    c.ctx.close()
