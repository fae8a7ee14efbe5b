"""idx_norm_rope_store (needs a GPU) on both sides of the sizes at which a half warp goes from one
row at a time to chunks of four and to chunks of 16 that are loaded a batch ahead, with heads and
tokens that fill neither."""
import pytest

from test_gpu_rope import DTYPES, Case, check_case

pytestmark = pytest.mark.gpu


# ceil(tokens / 16) * rows of a token: chunks of four from 608 on, of 16 from 7296 on
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,Hq,H", [(240, 32, 4), (241, 32, 4), (2912, 32, 4), (2913, 32, 4), (3001, 33, 3),
                                    (7001, 17, 1), (11001, 5, 3), (1000, 100, 9)])
def test_chunks(dtype, T, Hq, H):
    check_case(Case(T, Hq, H, dtype, seed=T + Hq))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("how", [
    dict(norm=False, rotary_dim=64), dict(norm=False, rotary_dim=0), dict(q_codes=True, values=False),
    dict(q_codes=True, interleaved=True, rotary_dim=96), dict(axes=3), dict(axes=4, interleaved=True),
    dict(rotary_dim=80, interleaved=True), dict(values=False, rotary_dim=16)])
def test_parts_of_long_chunks(dtype, how):
    check_case(Case(3003, 35, 5, dtype, seed=7, **how))


def test_no_queries_in_long_chunks():
    for T, H in ((4001, 17), (40001, 2)):
        check_case(Case(T, 0, H, "nvfp4", seed=T, outers=(0.25, 8.0)))
