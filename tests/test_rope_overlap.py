"""hs_rope_append refuses outputs whose rows overlap: several tokens would write one."""
import pytest
import torch

from sparse_top_kv_gb300 import hs
from test_step_ops import ROPE


@pytest.mark.parametrize("code,kw", [
    (1, dict(q_out_stride=0)), (1, dict(q_out_stride=1016)), (1, dict(head_stride=0)),
    (1, dict(head_stride=120)), (1, dict(row_stride=0)), (1, dict(page_stride=0)),
    (0, dict(tokens=0, q_out_stride=0)), (7, dict(d=100, rot=0, q_out_stride=0))])
def test_strides(code, kw):
    assert hs.lib().hs_rope_append(*{**ROPE, **kw}.values()) == code


@pytest.mark.gpu
def test_calls():
    """One entry of a dimension may have any stride; inputs may be broadcast."""
    bf = torch.bfloat16
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(1, 4, 64, device="cuda").to(bf).expand(3, 4, 64)
    turns = hs.rope_turns(hs.rope_frequencies(64)[0])
    pos, slot = torch.zeros(3, **i32), torch.arange(3, **i32)
    cache = lambda *s: torch.zeros(*s, 64, dtype=bf, device="cuda")
    ok = dict(q=q, k=q, v=q, positions=pos, slot=slot, turns=turns, k_cache=cache(1, 16, 4),
              v_cache=cache(1, 16, 4))
    out = hs.rope_append(**ok)
    assert torch.equal(out, q) and torch.equal(ok["k_cache"][0, :3], q)
    one = dict(q=q[:1], k=q[:1, :1], v=q[:1, :1], positions=pos[:1], slot=slot[:1], turns=turns,
               k_cache=cache(1, 1, 1).expand(1, 1, 1, 64), v_cache=cache(1, 1, 1))
    hs.rope_append(**one, q_out=torch.zeros(1, 4, 64, dtype=bf, device="cuda"))
    assert torch.equal(one["k_cache"][0, 0], q[0, :1])
    for bad in (dict(q_out=torch.zeros(1, 4, 64, dtype=bf, device="cuda").expand(3, 4, 64)),
                dict(k_cache=cache(1, 16, 4).expand(2, 16, 4, 64),
                     v_cache=cache(1, 16, 4).expand(2, 16, 4, 64)),
                dict(k_cache=cache(1, 1, 4).expand(1, 16, 4, 64),
                     v_cache=cache(1, 1, 4).expand(1, 16, 4, 64)),
                dict(k_cache=cache(1, 16, 1).expand(1, 16, 4, 64),
                     v_cache=cache(1, 16, 1).expand(1, 16, 4, 64))):
        with pytest.raises(hs.HSError):
            hs.rope_append(**{**ok, **bad})
