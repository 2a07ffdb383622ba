"""Which kernel a call of the operators between a block's projections takes, by its sizes.  No kernel is launched."""
import pytest


@pytest.fixture(scope="module")
def rows():
    import bit_quantized_matvec_amd as m

    return m.lib().tq_paged_attn_tile_rows


def test_paged_attn_rows_of_a_workgroup(rows):
    # one token each: 16, however many
    assert rows(1, 1, 1, 24, 2, 256) == rows(64, 64, 1, 48, 4, 128) == rows(4096, 4096, 0, 1024, 64, 64) == 16
    # a prompt that fills the card: 128
    assert rows(2048, 1, 2048, 48, 4, 128) == rows(500, 1, 0, 24, 2, 256) == rows(60, 2, 40, 32, 16, 64) == 128
    # few 16-row tiles: 16.  An eighth of the places (two workgroups per compute unit, one at 256 columns) decides
    assert rows(32, 1, 32, 16, 16, 64) == 16 and rows(48, 1, 48, 16, 16, 64) == 128       # 3, 4 tiles x 16 key heads
    assert rows(48, 1, 48, 7, 7, 256) == 16 and rows(48, 1, 48, 8, 8, 256) == 128         # 4 tiles x 7, 8
    # the longest sequence has 16 rows: 16
    assert rows(900, 100, 16, 64, 64, 64) == 16 and rows(900, 100, 17, 64, 64, 64) == 128
    assert rows(0, 0, 0, 24, 2, 256) == 16


@pytest.mark.parametrize("args", [(-1, 1, 1, 24, 2, 256), (1, -1, 1, 24, 2, 256), (1, 1, -1, 24, 2, 256), (1, 1, 1, 24, 5, 256), (1, 1, 1, 24, 2, 96),
                                  (1, 0, 1, 24, 2, 256), (1 << 21, 1, 1, 24, 2, 256)])
def test_paged_attn_rows_of_refused_sizes(rows, args):
    assert rows(*args) == 0
