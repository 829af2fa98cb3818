"""Arguments of the operators over an 8-bit paged cache at the ends of their ranges, without a GPU: what is
refused, and what no longer is."""
import pytest
import torch

from tests.test_kv8_host import CUDA, INVALID, UNSUPPORTED, _attend, lib  # noqa: F401


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls on pointers that are none")
@pytest.mark.parametrize("kw", [
    # one prompt among many decoding requests: 2^31 tiles by the bounds, a few thousand by the tokens
    dict(B=512, h=8, Hq=32, new=4096, n=4096 + 511, page=128, W=2**13, max_kv=2**20),
    dict(B=4096, h=8, Hq=64, new=1000, n=8192, page=128, W=2**13, max_kv=2**20)])
def test_attend_takes_wide_bounds_of_few_tokens(lib, kw):  # noqa: F811
    assert _attend(lib, **kw) in (CUDA, UNSUPPORTED)


@pytest.mark.parametrize("kw", [
    dict(B=512, h=8, Hq=32, new=4096, n=512 * 4096, page=128, W=2**13, max_kv=2**20),
    dict(B=4096, h=64, Hq=64, new=1, n=4096, page=128, W=2**13, max_kv=2**20)])
def test_attend_refuses_too_many_tiles(lib, kw):  # noqa: F811
    assert _attend(lib, **kw) == INVALID
    assert b"too large" in lib.star_last_error()
