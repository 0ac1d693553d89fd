"""Sizes whose counts would pass 32 bits are refused on the host (fake addresses, never dereferenced)."""
import pytest

from linear_attention_recurrence_kda_gb300 import binding as B
from test_abi_host import L  # noqa: F401  (fixture)
from test_attention_host import attention, cache, decode


@pytest.mark.parametrize("tokens,heads,kv,status", [
    (1 << 27, 128, 1, B.KDA_ERR_UNSUPPORTED),      # 2^34 rows of one key head
    (1 << 24, 128, 1, B.KDA_ERR_UNSUPPORTED),      # 2^31
    ((1 << 24) - 1024, 128, 1, B.KDA_ERR_WORKSPACE),  # just below: refused for its workspace alone
    (1 << 24, 128, 2, B.KDA_ERR_WORKSPACE),
])
def test_decode_rows_of_a_key_head(L, tokens, heads, kv, status):  # noqa: F811
    p = attention(num_seqs=1, total_tokens=tokens, num_heads=heads, num_kv_heads=kv, head_dim=32)
    assert decode(L, p, cache(), ws=None, q=1 << 44, lengths=1 << 43, out=1 << 45) == status
    assert (B.kda_attention_decode_workspace_bytes(p) == 0) == (status == B.KDA_ERR_UNSUPPORTED)
