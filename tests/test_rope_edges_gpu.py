"""qk_rope and qk_rope_bwd of tokens that the tables have no row for."""
import pytest
import torch

from test_rope_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


def test_tables_shorter_than_a_sequence_are_refused(fa):
    """Without positions the tables have a row for every token of a sequence."""
    c = Case(41, 4, 2, 128, 64, P=40)
    q4, k4 = c.q[:40].unflatten(0, (2, 20)), c.k[:40].unflatten(0, (2, 20))
    for q, k, n in ((c.q, c.k, 40), (q4, k4, 19)):
        cos, sin = c.cos[:n].contiguous(), c.sin[:n].contiguous()
        with pytest.raises(ValueError):
            fa.qk_rope(q, k, cos, sin)
        with pytest.raises(ValueError):
            fa.qk_rope(q, k, cos, sin, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
        with pytest.raises(ValueError):
            fa.qk_rope_bwd(q, k, None, None, cos, sin)
    fa.qk_rope(q4, k4, c.cos[:20].contiguous(), c.sin[:20].contiguous())
    fa.qk_rope(c.q[:0], c.k[:0], c.cos[:1].contiguous(), c.sin[:1].contiguous())
    assert fa.device_status() == 0
