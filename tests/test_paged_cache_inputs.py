"""An append whose new tokens do not fit the cache is refused before a page is taken, on the CPU (the device copies of
test_paged_cache.py in place of the kernels)."""
import pytest
import torch

from test_paged_cache import _consistent, _read, _tokens, cache  # noqa: F401


@pytest.mark.parametrize("spoil", [
    lambda k, v, ki: (k, v[:, :39], ki), lambda k, v, ki: (k, v, ki[:1]), lambda k, v, ki: (k.float(), v, ki),
    lambda k, v, ki: (k, v, ki[..., :16]), lambda k, v, ki: (k[..., 0], v, ki), lambda k, v, ki: (k[0], v[0], ki[0]),
    lambda k, v, ki: (k, v, ki.to(torch.float16)), lambda k, v, ki: (k.expand(-1, -1, 2, -1), v, ki),
    lambda k, v, ki: (torch.zeros(2, dtype=k.dtype), v, ki)],
    ids=["v-short", "idx-batch", "k-fp32", "idx-dim", "k-no-dim", "no-batch", "idx-fp16", "k-heads", "one-dim"])
def test_new_tokens_that_do_not_fit_change_nothing(cache, spoil):  # noqa: F811
    c = cache()
    a, b = c.new(), c.new()
    c.append([a], *_tokens(1, 5, [list(range(5))]))
    f = c.fork(a)  # an append to either would copy the shared page
    before = {s: c.page_list(s) for s in (a, b, f)}, c.free_pages
    with pytest.raises(ValueError):
        c.append([a, b], *spoil(*_tokens(2, 40, [[0.0] * 40] * 2)))
    assert before == ({s: c.page_list(s) for s in (a, b, f)}, c.free_pages)
    _consistent(c)
    assert _read(c, a) == _read(c, f) == list(range(5))
