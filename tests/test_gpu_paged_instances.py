"""The attention kernels at every head size they are built for (64, 96, 128,
192, 256 dims, and dims below them that are padded), with up to 8 and with 9
and more query heads a key/value head, over both cache types: rows dealt in
shares and joined (a wide table with short requests in it decides that), and
rows of one launch.  Tolerances as in test_gpu_paged.py."""
import random

import pytest

from .test_gpu_paged import attention_problem, check_attention, w  # noqa: F401  (w: the fixture)

pytestmark = pytest.mark.gpu
DIMS = [16, 48, 64, 80, 96, 112, 128, 160, 192, 224, 256]


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("group", [1, 3, 8, 9, 12, 16, 17])
@pytest.mark.parametrize("dim", DIMS)
def test_attention_shares_and_join(w, dim, group, dtype):
    # 4096 columns of 16 tokens: 4096 tiles a row are more than one launch takes (512); and
    # 5 * 65536 tokens of 256 dims are more than a cache of two rows of 8 heads may show
    lens = [0, 1, 700, 33, 1500]
    page, layout = (16, "token") if (dim + group) % 3 else (24, "head")
    q, cache, table = attention_problem(w, dim * 32 + group, lens, 2 * group if dim < 128 else group, 2 if dim < 128 else 1, dim, page, dtype, layout,
                                        columns=4096)
    check_attention(w, q, cache, table, lens)
    # a window longer than 512 tiles: nothing of these requests lies before it, or 300 tokens do
    check_attention(w, q, cache, table, lens, window=9000)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("dim,group", [(64, 9), (128, 16), (192, 12), (240, 10), (256, 16)])
def test_attention_shares_inside_a_window(w, dim, group, dtype):
    lens = [12000, 9005]
    q, cache, table = attention_problem(w, dim + group, lens, group, 1, dim, 16, dtype, "token")
    check_attention(w, q, cache, table, lens, window=8999)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_two_rows_of_eight_in_shares(w, dtype):
    # one request whose table could hold 32768 tokens of 256 dims: 16 heads as two rows, in shares
    q, cache, table = attention_problem(w, 5, [777], 16, 1, 256, 16, dtype, "token", columns=2048)
    check_attention(w, q, cache, table, [777])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("group", [9, 12, 16, 17, 31])
@pytest.mark.parametrize("dim", DIMS)
def test_attention_rows_of_sixteen_heads(w, dim, group, dtype):
    lens = [3, 0, 90, 161]
    q, cache, table = attention_problem(w, dim + group, lens, group, 1, dim, 16 if group % 2 else 24, dtype, "token")
    check_attention(w, q, cache, table, lens)


@pytest.mark.parametrize("dtype,requests", [("bf16", 1100), ("fp8", 2100)])
def test_attention_rows_of_sixteen_heads_of_256_dims(w, dtype, requests):
    # so many requests that the cache they may show is past what L2 holds, each of 8 tiles at most
    rng = random.Random(requests)
    lens = [rng.choice([0, 1, 128, rng.randrange(129)]) for _ in range(requests)]
    q, cache, table = attention_problem(w, requests, lens, 9, 1, 256, 16, dtype, "token", columns=8)
    check_attention(w, q, cache, table, lens)
