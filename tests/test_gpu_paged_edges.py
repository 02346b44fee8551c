"""Corners of the paged-cache operators on the GPU: exact choices beside NaN pages and where an MMA's dropped
bits add up."""
import math

import pytest
import torch

import paged_ref as ref
from fp8_attention_forward_gb300 import build, fa8
from paged_ref import E4M3, Problem, e4m3, val

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa8.lib()


def ok():
    assert fa8.check() == fa8.FA8_SUCCESS


def check_choice(p, q, bnd, K, four, keep_first=0, keep_last=0):
    """The choice for one token; `four`: the same token many times over, enough of them for blocks of four."""
    p.q, b8 = q.float().to(E4M3), bnd.float().to(E4M3)
    want = ref.select(p, b8, K, True, keep_first, keep_last)[0]
    if four:
        p.q = p.q.view(torch.uint8).expand(1, 1301, -1, -1).contiguous().view(E4M3)
        p.new, p.T = [1301], 1301
    got = fa8.select_pages(p.q.cuda(), b8.cuda(), K, causal=not four, keep_first=keep_first, keep_last=keep_last,
                           **p.index_args())
    ok()
    assert (got.cpu()[0] == want).all(), (got[0, 0].tolist(), want.tolist())


# ------------------------------------------------------------------ page selection
@pytest.mark.parametrize("four", [False, True], ids=["one", "four"])
@pytest.mark.parametrize("nan_pages", [range(8), [0, 2, 4, 6, 9, 11, 13, 15], [7]])
def test_nan_pages_hide_no_other_page(nan_pages, four):
    """Pages that are NaN in every channel beside pages whose scores differ by the smallest products only."""
    p = Problem([8 * 16], [1], Hq=1, Hkv=1, D=64, DV=64, ps=8, seed=50)
    phys = p.bt[0].long()
    q = torch.full((1, 1, 1, 64), 448.0, dtype=torch.float64)
    q[..., 3] = 2.0 ** -9
    bnd = torch.full((p.k.shape[0], 1, 2, 64), 448.0, dtype=torch.float64)
    bnd[phys, 0, :, 3] = (torch.arange(16) % 8).double()[:, None] * 2.0 ** -9
    bnd[phys[list(nan_pages)]] = math.nan
    check_choice(p, q, bnd, len(nan_pages) + 1, four)


@pytest.mark.parametrize("four", [False, True], ids=["one", "four"])
@pytest.mark.parametrize("large", [448.0, -448.0])
def test_choice_where_dropped_bits_add_up(large, four):
    """One product of 448 x 448 first, then 254 equal ones just below 2^-f of it: of its sign on pages 0 to 3,
    of the other on 4 to 7, which a last product g lifts.  An MMA that drops the small products ranks 4 to 7
    first, while the real scores may have it the other way round."""
    for f in range(20, 30):
        ea = int((16 - f) / 2)
        eb = 16 - f - ea
        small = 254 * 1.125 * 2.0 ** ea * 1.75 * 2.0 ** eb
        steps = [m / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8, 16)]
        for g in [s for s in steps if s < 2 * small][-3:] + [s for s in steps if s > 2 * small][:1]:
            p = Problem([8 * 16], [1], Hq=1, Hkv=1, D=256, DV=256, ps=8, seed=51)
            q = torch.full((1, 1, 1, 256), 1.75 * 2.0 ** eb, dtype=torch.float64)
            q[..., 0], q[..., 255] = 448.0, 1.0
            page = torch.zeros((16, 256), dtype=torch.float64)
            page[:8, 0] = large
            page[:4, 1:255], page[4:8, 1:255] = 1.125 * 2.0 ** ea, -1.125 * 2.0 ** ea
            page[4:8, 255] = g
            if large < 0:  # the pages beside them, of higher scores
                page[8:, 0] = -16.0
            bnd = torch.zeros((p.k.shape[0], 1, 2, 256), dtype=torch.float64)
            bnd[p.bt[0].long(), 0] = page[:, None]
            check_choice(p, q, bnd, 4 if large > 0 else 12, four)
