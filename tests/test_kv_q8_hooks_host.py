"""Refusals of the 8-bit attention's test hook (no GPU)."""
import pytest

import speculative_decoding_rl_b200 as sv


def test_stalled_attention_refuses_limits_and_roles():
    d = sv.SvAttnDesc(2, 5, 8, 2, 128, 16, 8, 32)
    kv = sv.SvKVQ8(0x1000000, 0x2000000, 0x3000000)
    for limit, role in ((0, 1), (999_999, 1), (2_000_000_001, 1), (5_000_000, 0), (5_000_000, 5), (5_000_000, -1)):
        with pytest.raises(sv.SvError) as e:
            sv.sv_testing_verify_attention_q8_stalled(d, 0x4000000, kv, 0x5000000, 0x6000000, None, 0x7000000, 256,
                                                      1 << 20, 0x8000000, limit, role, stream=0)
        assert e.value.status == sv.SV_ERR_INVALID_ARG
    with pytest.raises(sv.SvError):  # and what the call itself refuses
        sv.sv_testing_verify_attention_q8_stalled(sv.SvAttnDesc(2, 5, 8, 2, 96, 16, 8, 32), 0x4000000, kv, 0x5000000,
                                                  0x6000000, None, 0x7000000, 256, 1 << 20, 0x8000000, 5_000_000, 1,
                                                  stream=0)
