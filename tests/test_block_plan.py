"""What hq_launch_plan says of the products with block scales (host only)."""
import pytest

hq = pytest.importorskip("quantized_gemm_dequant_gb300")


def _plan(monkeypatch, choice, M=600, N=4096, K=2048):
    monkeypatch.setenv("HQ_TUNE", choice)
    return hq.launch_plan(hq.make_format("e4m3_block", N, K), M)


# variant 5: a CTA or a cluster of CTAs a tile; 6 and 7: CTA pairs with 256 tokens by 128 and by 256 features
@pytest.mark.parametrize("choice,variant,bt", [("kernel=1,bt=16,sk=1", 5, 16), ("kernel=1,bt=32,sk=1", 5, 32),
                                               ("kernel=1,bt=64,sk=1", 5, 64), ("kernel=1,bt=128,sk=1", 5, 128),
                                               ("kernel=0,bt=128", 6, 256), ("kernel=0,bt=256", 7, 256)])
def test_kernels_are_told_apart(monkeypatch, choice, variant, bt):
    p = _plan(monkeypatch, choice)
    assert (p["kernel"], p["variant"], p["bt"], p["sk"], p["grouped"]) == ("umma", variant, bt, 0, 0)


def test_split(monkeypatch):
    assert _plan(monkeypatch, "kernel=1,bt=128,sk=4")["sk"] == 1


def test_pairs_stop_where_their_row_index_ends(monkeypatch):
    """The CTA pairs number the packed weights' rows of 128 bytes with an int: below 2^24 blocks of 128 rows they may be
    chosen, from there on they are not."""
    K = 128 << 12
    below, at = ((1 << 12) - 1) * 128, (1 << 12) * 128
    for choice, variant in (("kernel=0,bt=128", 6), ("kernel=0,bt=256", 7)):
        assert _plan(monkeypatch, choice, N=below, K=K)["variant"] == variant
        assert _plan(monkeypatch, choice, N=at, K=K)["variant"] == 5
        assert _plan(monkeypatch, choice, N=below + 1, K=K)["variant"] == 5
