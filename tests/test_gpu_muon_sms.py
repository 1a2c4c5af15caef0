"""zero_muon on fewer SMs than the device has: the products are dealt to the blocks that can run at one time, and a tile's
result does not depend on which of them makes it, so that every comparison is bit for bit."""
import pytest
import torch
from test_gpu_muon import Muon, stream

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


# blocks of their own, pairs of them, and several matrices
@pytest.mark.parametrize("shapes", [[(300, 700)], [(64, 96), (130, 40)], [(520, 520), (700, 300), (65, 129)],
                                    [(2500, 2100)] * 3])
def test_fewer_blocks_give_the_same_bits(shapes):
    ref, mu, hyper = Muon(shapes, 2).fill(3), Muon(shapes, 2).fill(3), Z.muon_hyper(lr=0.01)
    try:
        for t, sms in enumerate((2, 3, 7, 40, 151, 1000, 0), 1):
            Z.zero_muon_set_option(mu.h, Z.ZERO_MUON_OPT_SMS, sms)
            mu.bind(-1)
            assert mu.step(hyper).t == ref.step(hyper).t == t
            assert all(torch.equal(a, b) for a, b in zip(ref.p + ref.p16 + ref.x + ref.halves, mu.p + mu.p16 + mu.x + mu.halves)), sms
        mu.guards_stand()
    finally:
        mu.close()
        ref.close()


def test_two_optimizers_share_the_device():
    """Each on half of the SMs, on streams of their own."""
    shapes, hyper = [(700, 900), (260, 1300)], Z.muon_hyper(lr=0.01)
    ref, *both = (Muon(shapes, 2).fill(5) for _ in range(3))
    try:
        for mu in both:
            Z.zero_muon_set_option(mu.h, Z.ZERO_MUON_OPT_SMS, 76)
            mu.bind(0)
        streams = [torch.cuda.Stream() for _ in both]
        torch.cuda.synchronize()
        for _ in range(4):
            ref.step(hyper)
            for mu, s in zip(both, streams):
                Z.zero_muon_step(mu.h, hyper, 1.0, s.cuda_stream)
        torch.cuda.synchronize()
        for mu in both:
            assert Z.zero_muon_read(mu.h, stream()).t == 4
            assert all(torch.equal(a, b) for a, b in zip(ref.p + ref.halves, mu.p + mu.halves))
    finally:
        for mu in (ref, *both):
            mu.close()
