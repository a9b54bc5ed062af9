"""BudgetedDecoder: calls that do not fit are refused before anything has
changed (a step that fails half-way would leave a token counted but not there;
tensors of one row would be spread over all requests)."""
import pytest
import torch

from sparse_top_kv_gb300.pipeline import BudgetedDecoder

SHAPE = dict(num_reqs=3, heads=8, kv_heads=2, d=64, page_size=16, budget=16, capacity=40, scale=0.1)


@pytest.mark.parametrize("bad", [dict(budget=0), dict(d=96), dict(heads=7), dict(kv_heads=0),
                                 dict(num_reqs=0), dict(page_size=0)])
def test_set_up(bad):
    with pytest.raises(ValueError):
        BudgetedDecoder(**{**SHAPE, **bad})


def state(dec):
    torch.cuda.synchronize()
    return [x.clone() for x in (dec.k_cache, dec.v_cache, dec.seq_lens, dec.next_pos,
                                dec.positions, dec.score)]


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["step", "replay"])
@pytest.mark.parametrize("bad,error", [
    (dict(q=(1, 8, 64)), ValueError), (dict(q=(3, 4, 64)), ValueError),
    (dict(k=(1, 2, 64)), ValueError), (dict(v=(3, 1, 64)), ValueError),
    (dict(v=(3, 2, 1)), ValueError), (dict(k=torch.float32), TypeError),
    (dict(q=torch.float16), TypeError), (dict(v="cpu"), ValueError),
    (dict(q="heads"), ValueError)])
def test_step(how, bad, error):
    shapes = dict(q=(3, 8, 64), k=(3, 2, 64), v=(3, 2, 64))
    dec = BudgetedDecoder(**SHAPE)
    good = [torch.ones(*s, dtype=torch.bfloat16, device="cuda") for s in shapes.values()]
    with pytest.raises(ValueError):
        dec.replay(*good)  # nothing captured yet
    dec.start(0, torch.ones(30, 2, 64), torch.ones(30, 2, 64))
    dec.start(2, torch.ones(5, 2, 64), torch.ones(5, 2, 64))
    dec.step(*good)
    dec.capture()
    before = state(dec)
    args = dict(zip("qkv", good))
    (name, what), = bad.items()
    if isinstance(what, tuple):
        args[name] = torch.ones(*what, dtype=torch.bfloat16, device="cuda")
    elif isinstance(what, torch.dtype):
        args[name] = args[name].to(what)
    elif what == "cpu":
        args[name] = args[name].cpu()
    else:
        args[name] = args[name].transpose(1, 2).contiguous().transpose(1, 2)
    if how == "replay" and not isinstance(what, tuple):
        dec.replay(*args.values())  # copied into the captured inputs, which fit
        return
    with pytest.raises(error):
        getattr(dec, how)(*args.values())
    assert all(torch.equal(a, b) for a, b in zip(before, state(dec)))


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [dict(k=(5, 1, 64)), dict(v=(4, 2, 64)), dict(v=(5, 2, 1)),
                                 dict(score=(1,)), dict(score=(6,)), dict(q=(0, 8, 64)),
                                 dict(q=(6, 8, 64)), dict(q=(2, 2, 64))])
def test_start(bad):
    dec = BudgetedDecoder(**SHAPE)
    dec.start(1, torch.ones(7, 2, 64), torch.ones(7, 2, 64))
    before = state(dec)
    args = {n: torch.ones(*s) for n, s in {**dict(k=(5, 2, 64), v=(5, 2, 64)), **bad}.items()}
    with pytest.raises(ValueError):
        dec.start(1, args.pop("k"), args.pop("v"), **args)
    assert all(torch.equal(a, b) for a, b in zip(before, state(dec)))
