"""ula_rotate of as many heads as an int32 can count."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [2 ** 31 - 1, 2 ** 31 - 512, 2 ** 30 + 1])
def test_heads_up_to_the_range_of_their_count(heads):
    """One token's heads of two channels, turned in place: both ends and the middle equal calls of those alone."""
    import torch
    from serving_pb_lru_amd import rotate
    x = torch.empty((1, heads, 2), dtype=torch.bfloat16, device="cuda").uniform_(-1, 1)
    pos = torch.tensor([5], dtype=torch.int32, device="cuda")
    parts = [slice(0, 1000), slice(heads // 2 - 500, heads // 2 + 500), slice(heads - 1000, heads)]
    want = [rotate(x[:, p].clone(), pos) for p in parts]
    assert rotate(x, pos, out=x) is x
    for p, w in zip(parts, want):
        assert torch.equal(x[:, p], w)
