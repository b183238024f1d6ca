"""Window attention where a block of threads takes several work items, with and without padding, and both forms of the
masked steps without a window."""
import pytest
import torch

from test_gpu_window_attention import check, draw, mka, run  # noqa: F401  (mka: the fixture)

ITEMS = [
    # B, S, Hq, Hkv, dh, window, sinks: more items than SMs in the forward, dQ and (but for the third) dK/dV
    (4, 1300, 16, 4, 64, 200, 3), (3, 1500, 14, 2, 128, 1100, 130), (2, 1200, 16, 16, 128, 0, 0), (6, 700, 15, 5, 64, 0, 0),
    (5, 900, 12, 4, 128, 64, 200),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ITEMS)
@pytest.mark.parametrize("padded", [False, True])
def test_several_items_per_block(mka, case, padded):  # noqa: F811
    B, S, Hq, Hkv, dh, window, sinks = case
    x = draw(B, S, Hq, Hkv, dh, sum(case))
    lens = [S - 301 * b % S if b != 1 else b for b in range(B)] if padded else None
    if padded:
        for t in x:
            for b, n in enumerate(lens):
                t[b, n:] = float("nan")
    got = run(mka, *x, window, sinks, lens)
    check(got, *x, window, sinks, lens)
    again = run(mka, *x, window, sinks, lens)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], again[:4]))


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(1, 767, 4, 2, 64, 0, 0), (1, 768, 4, 2, 64, 0, 0), (2, 767, 3, 1, 128, 0, 0), (2, 769, 3, 1, 128, 0, 7)])
def test_without_a_window(mka, case):  # noqa: F811
    B, S, Hq, Hkv, dh, window, sinks = case
    x = draw(B, S, Hq, Hkv, dh, sum(case))
    check(run(mka, *x, window, sinks), *x, window, sinks)
