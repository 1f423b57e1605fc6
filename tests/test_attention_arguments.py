"""Arguments of the rotary call that the library would read as others (no GPU needed)."""
import pytest

import extended_precision_gemm_gb300 as ddg

from test_attention import Stand, binding  # noqa: F401


def test_positions_of_unsigned_32_bits_are_refused(binding):  # noqa: F811
    """From 2^31 on they would turn as negative ones; of 64 bits both are the same modulo a turn."""
    torch, calls = binding
    x, table = Stand((6, 3, 64), torch.float16), ddg.Rotary(Stand((16,), torch.int64))
    for call in (ddg.rotary, ddg.rotary_backward):
        with pytest.raises(TypeError, match="positions"):
            call(x, Stand((6,), torch.uint32), table)
        assert not calls
        for dtype in (torch.int32, torch.int64, torch.uint64):
            call(x, Stand((6,), dtype), table)
            assert calls.pop()[0] == "dd_rotary"
