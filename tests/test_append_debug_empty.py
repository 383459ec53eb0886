"""The debug mode's checks of a rotating append without tokens."""
import pytest
import torch

from paged_kv_cache_104_gb300 import binding as B
from paged_kv_cache_104_gb300 import validate as V


def test_positions_of_no_tokens():
    none = torch.zeros(0, dtype=torch.int64)
    for positions in (torch.zeros(0), torch.zeros(1, 0), torch.zeros(3, 0)):
        V.check_positions(positions.to(torch.int32), none, 7)
    with pytest.raises(V.ValidationError, match="token 1"):
        V.check_positions(torch.tensor([[0, 7]]).to(torch.int32), torch.tensor([3, 4]), 7)


@pytest.mark.parametrize("call", ["rope", "block"])
def test_rotating_appends_of_no_tokens_pass_the_debug_mode(call, monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    monkeypatch.setattr(B, "_stream_on", lambda stream, index: None)
    rope = B.Rope(torch.zeros(4, 32))
    new, slots = torch.zeros(0, 2, 64, dtype=torch.bfloat16), torch.zeros(0, dtype=torch.int64)
    pos = torch.zeros(1, 0, dtype=torch.int32)
    B.set_debug(True)
    try:
        if call == "rope":
            pool = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
            B.kv_append_rope(new.clone(), new, new, new, pool, pool.clone(), slots, pos, rope)
        else:
            pool, scale = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, dtype=torch.uint8)
            B.kv_append_fp8_block(new, new, pool, pool.clone(), scale, scale.clone(), slots, positions=pos, rope=rope)
    finally:
        B.set_debug(False)
