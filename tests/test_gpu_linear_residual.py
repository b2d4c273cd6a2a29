"""Products whose epilogue is a residual and a scale alone, through every form that is not the stream kernel: residual
loaded ahead of its rows, in place and not, 16 and 32 bits, columns and rows that end inside a tile; and infinities past
the end of k. Against 64 bits (bounds: linear_ref64)."""
import pytest
import torch

import linear_ref64 as ref
import mixture_experts_router_amd as moe
from test_gpu_linear import make, near, rand
from test_gpu_linear_forms import form

pytestmark = pytest.mark.gpu

# T, K, N: rows and columns that end inside a tile, also inside its last eight columns
SIZES = [(33, 520, 9002), (33, 328, 9000), (33, 2056, 3301), (1500, 72, 2002), (1500, 136, 2000), (70, 4104, 3302),
         (1237, 1096, 4010), (1333, 2056, 4000), (2001, 72, 4002), (2001, 328, 4008), (3001, 72, 2602),
         (3001, 200, 2608), (2501, 72, 5002), (2501, 328, 4992)]


def padded(T, C, dtype, fill):
    """A tensor [T, C] inside one whose rows start aligned, and the whole."""
    wide = torch.full((T, (C + 7) // 8 * 8 + 8), fill, dtype=dtype, device="cuda")
    return wide[:, :C], wide


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_residual_and_scale(T, K, N, dtype, out):
    x, w = make(T, T, K, N, dtype)
    odt = torch.float32 if out == "f32" else x.dtype
    s = rand(2, T)
    r, r_wide = padded(T, N, odt, float("nan"))
    r.copy_(rand(3, T, N))
    for res, scale in ((r, s), (r, None), (None, s)):
        want, bound, *_ = ref.forward(x, w, None, "none", res, scale, odt)
        got, wide = padded(T, N, odt, 7.0)
        assert moe.linear(x, w, residual=res, row_scale=scale, out_dtype=odt, out=got) is got
        assert not form(moe.last_plan()).startswith("linear_stream")
        near(got, want, bound, "out")
        assert bool((wide[:, N:] == 7.0).all())
        assert torch.equal(moe.linear(x, w, residual=res, row_scale=scale, out_dtype=odt), got)  # rows side by side
        if res is not None:
            mine, mine_wide = padded(T, N, odt, 7.0)
            mine.copy_(res)
            assert moe.linear(x, w, residual=mine, row_scale=scale, out_dtype=odt, out=mine) is mine
            assert torch.equal(mine, got) and bool((mine_wide[:, N:] == 7.0).all())
    # in place through views of the same rows, and of rows that are not aligned
    flat = r.contiguous().clone()
    moe.linear(x, w, residual=flat.view(T, N), row_scale=s, out_dtype=odt, out=flat)
    want, bound, *_ = ref.forward(x, w, None, "none", r, s, odt)
    near(flat, want, bound, "views")


@pytest.mark.parametrize("T,K,N", [(33, 520, 9000), (70, 4104, 3304), (777, 200, 4000), (2001, 328, 4008),
                                   (2501, 72, 4992)])
def test_infinities_past_the_end_of_k(T, K, N):
    """K is no multiple of a step: what lies behind a row's end is not read, and a row's infinity stays in it."""
    x, w = make(4, T, K, N)
    want = moe.linear(x, w)
    assert not form(moe.last_plan()).startswith("linear_stream")
    wx = torch.full((T, K + 64), float("inf"), dtype=x.dtype, device="cuda")
    ww = torch.full((N, K + 64), float("nan"), dtype=x.dtype, device="cuda")
    wx[:, :K], ww[:, :K] = x, w
    assert torch.equal(moe.linear(wx[:, :K], ww[:, :K]), want)
    x[1, K - 1], x[T - 1, 0] = float("nan"), float("inf")
    got = moe.linear(x, w)
    other = torch.ones(T, dtype=torch.bool, device="cuda")
    other[1] = other[T - 1] = False
    assert torch.equal(got[other], want[other]) and bool(got[1].isnan().all())
    assert bool((~torch.isfinite(got[T - 1])).all())
