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


@pytest.mark.parametrize("max_kv", [2**31 - 256, 2**31 - 128, 2**31 - 127, 2**31 - 16])
def test_attend_refuses_lengths_whose_tiles_leave_int32(lib, max_kv):  # noqa: F811
    """kv_len + 127 did not fit int32: such a request was attended over its first 128 keys only."""
    assert _attend(lib, page=16, W=2**27 - 1, max_kv=max_kv) == INVALID
    assert b"max_kv" in lib.star_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls on pointers that are none")
def test_attend_takes_the_longest_lengths(lib):  # noqa: F811
    assert _attend(lib, page=16, W=2**27 - 1, B=1, n=1, max_kv=2**31 - 257) in (CUDA, UNSUPPORTED)
