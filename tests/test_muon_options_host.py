"""zero_muon_set_option's refusals (no GPU)."""
import pytest

import zero_sharded_mixed_03_gb300 as Z


def test_refusals():
    h = Z.zero_muon_create([8], [16])
    try:
        for handle, option, value in ((0, Z.ZERO_MUON_OPT_WAIT_LIMIT_NS, 1), (h, Z.ZERO_MUON_OPT_WAIT_LIMIT_NS, -1), (h, -1, 0),
                                      (h, 99, 0), (h, Z.ZERO_MUON_OPT_WAIT_LIMIT_NS, Z.ZERO_MUON_MAX_WAIT_NS + 1),
                                      (h, Z.ZERO_MUON_OPT_SMS, 1), (h, Z.ZERO_MUON_OPT_SMS, -2)):
            with pytest.raises(Z.ZeroError) as e:
                Z.zero_muon_set_option(handle, option, value)
            assert e.value.status == Z.ZERO_EINVAL
        for ns in (0, 1, 2_000_000_000, Z.ZERO_MUON_MAX_WAIT_NS):
            Z.zero_muon_set_option(h, Z.ZERO_MUON_OPT_WAIT_LIMIT_NS, ns)
        for sms in (0, 2, 152, 1 << 40):
            Z.zero_muon_set_option(h, Z.ZERO_MUON_OPT_SMS, sms)
    finally:
        Z.zero_muon_destroy(h)
