"""linear's choice between tiles and runs of the sums' axis, as its workspace tells it (no GPU)."""
import pytest

import direct_implicit_gemm_amd as L

size = L.libconv_linear_workspace


def runs(T, K, N, dtype):
    n = size(T, K, N, dtype)
    per = 4 * T * (-(-N // 64) * 64)
    assert n >= 0 and n % per == 0
    return n // per


@pytest.mark.parametrize("T,K,N", [(136, 3624, 3934), (367, 3848, 2691), (92, 3848, 4141)])
def test_idle_compute_units_are_given_runs(T, K, N):
    """More tiles of 64 x 64 than half of the compute units, or a few more than all."""
    tiles = -(-T // 64) * -(-N // 64)
    assert 128 < tiles < 512
    r = runs(T, K, N, L.F32)
    assert r > 1
    # on the fullest compute unit, in tiles' time
    assert -(-tiles * r // 256) / r < 0.85 * -(-tiles // 256)


@pytest.mark.parametrize("T,K,N,dtype", [(1462, 688, 188, L.BF16), (467, 368, 197, L.BF16),
                                         (8192, 4096, 8192, L.F32), (3, 64, 4096, L.F16)])
def test_no_runs_where_their_sums_take_longer(T, K, N, dtype):
    assert runs(T, K, N, dtype) == 0


def test_runs_are_no_shorter_than_their_start_and_no_more_than_16():
    for dtype, least in ((L.F32, 2), (L.BF16, 4)):
        for T in (1, 16, 100, 700, 5000, 65535):
            for K in (8, 264, 1000, 4096, 16384):
                for N in (1, 64, 1000, 4096):
                    r = runs(T, K, N, dtype)
                    assert r == 0 or 2 <= r <= 16
                    assert r * least * 128 <= K * (4 if dtype == L.F32 else 2) + 127


def test_no_more_rows_than_a_launch_has():
    assert runs(65536 + 5, 16384, 64, L.F32) == 0
