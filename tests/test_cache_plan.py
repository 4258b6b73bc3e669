"""cache_attention's plan, as its workspace tells it (no GPU)."""
import pytest

import direct_implicit_gemm_amd as L


def workspace(B, T, most, positions, hq, hk, d, dtype=L.BF16):
    return L.libconv_cache_attention_workspace(B, T, most, 16, positions // 16, hq, hk, d, dtype)


@pytest.mark.parametrize("B,T,most,hq,hk", [(1, 16, 16, 16, 4), (1, 1, 1, 64, 1), (4, 4, 1, 64, 1),
                                            (1, 100, 100, 2, 2), (1, 33, 33, 1, 1)])
def test_many_keys_of_few_sets_are_shared(B, T, most, hq, hk):
    """More than 32 rows of a key head: some workgroups for each 1024 keys, not one for all keys."""
    for positions in (2048, 8192, 131072):
        few = 2 * 512 * 32 * (64 + 1) * 4 if hq // hk <= 32 and positions >= 16 * B * hk else 0
        rest = workspace(B, T, most, positions, hq, hk, 64) - few
        sets = min(-(-most * (hq // hk) // 128) * B, T * (hq // hk) // 128 + B) * hk
        shares, left = divmod(rest, sets * 128 * (64 + 1) * 4)
        assert left == 0 and 4 <= shares <= 64
        assert shares * 2048 >= positions


@pytest.mark.parametrize("B,T,most,hq,hk", [(1, 16, 16, 16, 4), (2, 260, 130, 8, 8)])
def test_few_keys_are_not(B, T, most, hq, hk):
    assert workspace(B, T, most, 528, hq, hk, 64) == 0


@pytest.mark.parametrize("B,most,hq,hk", [(2, 64, 32, 8), (1, 16, 16, 4), (64, 40, 8, 8)])
def test_rows_of_no_entry_take_no_room(B, most, hq, hk):
    """A buffer of more rows than the entries have: a padded batch."""
    full = workspace(B, B * most, most, 131072, hq, hk, 128)
    assert full > 0
    for T in (B * most + 100, 8192, 65536, 1 << 20):
        # (as many sets as the entries have at most, and as many again where they are looked up)
        assert workspace(B, T, most, 131072, hq, hk, 128) <= 2 * full
