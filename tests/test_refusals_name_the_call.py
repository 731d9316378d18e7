"""A refusal by the binding names the call that was made, no GPU needed."""
import pytest
import torch

import elementwise_row_rmsnorm_gb300 as gbe

Q, K = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
ODD = torch.zeros(5, 64, 4).transpose(1, 2)      # [5, 4, 64] whose entries are not contiguous
ODD_K = torch.zeros(5, 64, 2).transpose(1, 2)
POS, OM, STARTS = torch.zeros(5, dtype=torch.int32), torch.zeros(32), torch.tensor([0, 5], dtype=torch.int32)


def _cache():
    c = gbe.KvCache.__new__(gbe.KvCache)  # a cache as far as its shape
    c.shape = (3, 2, 16, 64)
    return c


CALLS = {
    "kv_write": lambda: gbe.gbe_kv_write(ODD_K, ODD_K, POS, _cache()),
    "kv_read": lambda: gbe.gbe_kv_read(K, ODD_K, POS, _cache()),
    "attn_decode": lambda: gbe.gbe_attn_decode(ODD, ODD, _cache(), torch.zeros(5, 1, dtype=torch.int32), POS, 0.1),
    "attn_decode ": lambda: gbe.gbe_attn_decode(Q, ODD, _cache(), torch.zeros(5, 1, dtype=torch.int32), POS, 0.1),
    "attn_prompt": lambda: gbe.gbe_attn_prompt(ODD, K, K, Q, STARTS, 0.1),
    "attn_prompt ": lambda: gbe.gbe_attn_prompt(Q, K, ODD_K, Q, STARTS, 0.1),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_the_call_is_named(name):
    with pytest.raises(ValueError, match=f"^{name.strip()}: "):
        CALLS[name]()


@pytest.mark.parametrize("name,call", [
    ("rope_qk", lambda: gbe.gbe_rope_qk(ODD, ODD, None, None, POS, OM, 64)),
    ("qk_norm_rope", lambda: gbe.gbe_qk_norm_rope(ODD, ODD, torch.ones(64), None, None, None, 1e-5, POS, OM, 64)),
    ("rope_pair", lambda: gbe.gbe_rope_pair((ODD, ODD, OM, 64, 1.0, 0), None, POS))])
def test_the_call_is_named_past_the_check_of_the_device(name, call, monkeypatch):
    import elementwise_row_rmsnorm_gb300.binding as binding
    monkeypatch.setattr(binding, "_on_device", lambda t: True)
    with pytest.raises(ValueError, match=f"^{name}: "):
        call()
