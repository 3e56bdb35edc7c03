"""Workspace sizes of the projection with per-token adapters, by number of adapters and result type:
plain host arithmetic."""
import pytest

BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def fg():
    import moe_fp8_e4m3_gb300 as lib
    return lib


@pytest.mark.parametrize("m", [1, 16, 100, 129, 2048, 65536])
@pytest.mark.parametrize("r", [8, 64, 128])
def test_size_follows_the_adapters_that_a_tile_can_use(fg, m, r):
    n, k = 4096, 4096
    size = lambda l, dtype: fg.lib.fg_lora_workspace_for(m, n, k, l, r, dtype)  # noqa: E731
    assert 0 < size(1, BF16) < size(2, BF16) <= size(8, BF16) <= size(1024, BF16) < size(1024, F32)
    assert size(1024, F32) == size(128, F32) == fg.lib.fg_lora_workspace(m, n, k, r)
    bn = 16 if m <= 16 else 32 if m <= 32 else 64 if m <= 64 else 128
    tiles, rp = -(-m // bn), max(16, r)
    per_adapter = tiles * 2 * bn * rp * 2
    assert abs(size(9, BF16) - size(1, BF16) - 8 * per_adapter) < 256


def test_a_long_prompt_with_few_adapters_needs_little(fg):
    """x @ lora_a^T of 8 adapters in two parts (16 and 32 MB), and the partial tiles (64 MB)."""
    mb = 1 << 20
    partial = 256 * 2 * 2 * 128 * 128 * 4
    assert partial == 64 * mb
    assert 80 * mb <= fg.lib.fg_lora_workspace_for(8192, 4096, 4096, 8, 64, BF16) < 81 * mb
    assert 96 * mb <= fg.lib.fg_lora_workspace_for(65536, 4096, 4096, 8, 16, BF16) < 97 * mb


@pytest.mark.parametrize("bad", [(4, 250, 256, 3, 16, 0), (4, 256, 256, 0, 16, 0), (4, 256, 256, 1025, 16, 0), (4, 256, 256, 3, 7, 0),
                                 (4, 256, 256, 3, 16, 2), (65537, 256, 256, 3, 16, 0)])
def test_bad_sizes_have_no_workspace(fg, bad):
    assert fg.lib.fg_lora_workspace_for(*bad) == -1
