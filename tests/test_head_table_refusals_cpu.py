"""A rotation by a table of no positions is refused on the host, by both directions."""
from tests.test_attention_refusals_cpu import P, call, ops, qk_desc  # noqa: F401


def test_a_table_without_positions(gdr, ops):  # noqa: F811
    for name, n in (("gdr_qk_norm_fwd", 10), ("gdr_qk_norm_bwd", 14)):
        assert call(gdr, name, qk_desc(ops, P=0), [P] * n) == gdr.GDR_ERR_SHAPE, name
        assert "table" in gdr.last_error()
    # without tokens nothing is looked up
    assert call(gdr, "gdr_qk_norm_fwd", qk_desc(ops, P=0, M=0), [None] * 10) == 0
