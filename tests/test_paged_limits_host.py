"""The sizes that gpt2.h names as the limits of the paged-cache and sampling operations:
below them a call is not refused for its sizes (it gets as far as the device), at them it
is."""
import pytest

from test_paged_host import attend, sample
from test_spec_host import kv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls' arrays do not exist")

E = 64


def paged(rows, heads, width, n_positions, kv_heads=None, **cache):
    return attend(kv(n_head=kv_heads or heads, n_positions=n_positions, head_dim=E, **cache), heads=heads, rows=rows,
                  seqs=rows, width=width, q_stride=heads * E, out_stride=heads * E)


@pytest.mark.parametrize("heads,width,n_positions,tiles", [(8, 1, 1, 1), (8, 3, 3, 2), (16, 100, 16, 200), (1, 4096, 16, 8192)])
def test_tiles_of_a_paged_attention(heads, width, n_positions, tiles):
    most = 4 * 10 ** 9 // (heads * tiles)
    assert paged(min(most - 1, (1 << 30) - 1), heads, width, n_positions) != -1
    # (fp32 rows of 128 take the most tiles: rows of 8)
    if 2 * most < 1 << 30:
        assert attend(kv(n_head=heads, n_positions=n_positions, head_dim=128), heads=heads, rows=most + 1, seqs=most + 1,
                      width=width, q_stride=heads * 128, out_stride=heads * 128) == -1


def test_other_limits_of_a_paged_attention():
    assert paged(1, 1 << 16, 1, 16, kv_heads=1) != -1
    assert paged(1, 1 << 17, 1, 16, kv_heads=1) == -1
    assert paged((1 << 30) - 1, 1, 1, 16) != -1
    assert paged(1 << 30, 1, 1, 16) == -1


def test_rows_of_a_sampling():
    assert sample(rows=(1 << 27) - 1) != -1
    assert sample(rows=1 << 27) == -1
