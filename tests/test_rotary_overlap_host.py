"""Queries turned in place among the keys and values of one projection: what may lie where (host checks; the fake addresses are
never dereferenced)."""
from linear_attention_recurrence_kda_gb300 import binding as B
from test_abi_host import L, _addr  # noqa: F401  (fixture)
from test_attention_host import attention, cache
from test_rotary_host import append, descriptor

WIDE = dict(q_stride=512, k_stride=512, v_stride=512)  # 4 + 2 + 2 heads of 64 channels, 1024 bytes a token
INSIDE = _addr(0) + 10 * 1024 + 64


def views(**over):
    return dict(dict(k=_addr(0) + 512, v=_addr(0) + 768, q_out=_addr(0)), **over)


def test_nothing_else_lies_inside(L):  # noqa: F811
    p, c, r = attention(**WIDE), cache(), descriptor()
    assert append(L, p, c, r, **views()) != B.KDA_ERR_INVALID_ARG
    for name in ("cu", "lengths", "positions", "check"):
        at = INSIDE if name != "check" else _addr(0) + 10 * 1024
        assert append(L, p, c, r, **views(**{name: at})) == B.KDA_ERR_INVALID_ARG, name
    for name in ("block_table", "k", "v", "k_scale", "v_scale"):
        assert append(L, p, cache(**{name: INSIDE}), r, **views()) == B.KDA_ERR_INVALID_ARG, name


def test_a_projection_of_two(L):  # noqa: F811
    """q with k or with v; the third lies elsewhere, packed.  Rows that touch are refused."""
    c, r = cache(), descriptor()
    ok = append(L, attention(**WIDE), c, r, **views())
    assert ok != B.KDA_ERR_INVALID_ARG
    assert append(L, attention(q_stride=512, k_stride=512), c, r, k=_addr(0) + 512, q_out=_addr(0)) == ok
    assert append(L, attention(q_stride=512, v_stride=512), c, r, v=_addr(0) + 512, q_out=_addr(0)) == ok
    assert append(L, attention(q_stride=512, k_stride=512), c, r, k=_addr(0) + 256, q_out=_addr(0)) == B.KDA_ERR_INVALID_ARG
    assert append(L, attention(q_stride=512, v_stride=512), c, r, v=_addr(0) + 896, q_out=_addr(0)) == B.KDA_ERR_INVALID_ARG
    assert append(L, attention(q_stride=512, k_stride=256), c, r, k=_addr(0) + 512, q_out=_addr(0)) == B.KDA_ERR_INVALID_ARG
    assert append(L, attention(q_stride=512, k_stride=512), c, r, k=_addr(0) + 512) == ok  # out of place: no question
