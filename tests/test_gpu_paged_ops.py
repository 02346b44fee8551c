"""GPU tests of the operators around the paged cache (rotary append, page bounds, page
selection, attention over listed pages) against plain 64-bit forms."""
import math

import pytest
import torch

import paged_ref as ref
from fp8_attention_forward_gb300 import build, fa8, inputs
from paged_ref import E4M3, Problem, e4m3, val

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa8.lib()


def ok():
    assert fa8.check() == fa8.FA8_SUCCESS


# ------------------------------------------------------------------ page bounds
@pytest.mark.parametrize("D,Hkv,ps,keys", [
    (16, 1, 8, [1]), (64, 2, 8, [7, 8, 9, 100]), (96, 3, 24, [50, 0, 73]), (128, 8, 16, [1, 1000, 333]),
    (192, 4, 64, [640, 641]), (256, 1, 128, [129, 5]), (128, 2, 4096, [5000]),
])
def test_page_bounds(D, Hkv, ps, keys):
    """Minimum and maximum are E4M3 values themselves: equal, not close."""
    p = Problem(keys, [0] * len(keys), Hq=Hkv, Hkv=Hkv, D=D, DV=D, ps=ps, seed=1)
    p.poison()
    got = fa8.page_bounds(p.k.cuda(), cu_seqlens_k=p.cu_k.cuda(), block_table=p.bt.cuda(), page_size=ps)
    ok()
    assert torch.equal(val(got.cpu()), ref.bounds(p))


@pytest.mark.parametrize("new,packed", [([0, 0, 0], False), ([1, 1, 1], False), ([17, 17, 17], False),
                                        ([40, 40, 40], False), ([0, 33, 5], True), ([100, 1, 48], True)])
def test_page_bounds_update_touches_new_pages_only(new, packed):
    p = Problem([100, 33, 48], new, ps=16, packed=packed, seed=2)
    p.poison()
    before = e4m3(torch.full((p.k.shape[0], p.Hkv, 2, p.D), 3.5))
    got = before.cuda()
    kw = dict(cu_seqlens_q=p.cu_q.cuda()) if packed else dict(new_tokens=new[0])
    fa8.page_bounds(p.k.cuda(), got, cu_seqlens_k=p.cu_k.cuda(), block_table=p.bt.cuda(), page_size=16, **kw)
    ok()
    assert torch.equal(val(got.cpu()), ref.bounds(p, only_new=True, into=before))


def test_page_bounds_nan_and_extremes():
    p = Problem([40], [0], Hq=1, Hkv=1, D=64, DV=64, ps=16, seed=3)
    b = p.k.view(torch.uint8)
    pg = p.bt[0].long()
    b[pg[0], 3, 0, 5] = 0x7F
    b[pg[1], 0, 0, 6] = 0xFF
    b[pg[1], :, 0, 7] = 0x80
    b[pg[2], 7, 0, 8] = 0xFE
    got = val(fa8.page_bounds(p.k.cuda(), cu_seqlens_k=p.cu_k.cuda(), block_table=p.bt.cuda(), page_size=16).cpu())
    ok()
    torch.testing.assert_close(got, ref.bounds(p), rtol=0, atol=0, equal_nan=True)
    assert got[pg[0], 0, :, 5].isnan().all() and got[pg[1], 0, :, 6].isnan().all() and got[pg[2], 0, 0, 8] == -448


# ------------------------------------------------------------------ page selection
def run_select(p, bnd, K, **kw):
    got = fa8.select_pages(p.q.cuda(), bnd.cuda(), K, **p.index_args(), **kw)
    ok()
    return got.cpu()


SELECT = [
    dict(keys=[1], new=[1], K=1, kf=0, kl=0),
    dict(keys=[500], new=[1], K=4, kf=0, kl=0),
    dict(keys=[500], new=[1], K=4, kf=4, kl=0),
    dict(keys=[500, 3, 70], new=[3] * 3, K=3, Hq=16, Hkv=1, D=64),
    dict(keys=[900, 0, 33], new=[2, 0, 33], K=5, packed=True, tail=2, D=96, Hq=6, Hkv=2),
    dict(keys=[900, 640], new=[1, 4], K=7, packed=True, D=192, Hq=40, Hkv=2, ps=8),
    dict(keys=[2000], new=[2], K=33, D=256, Hq=3, Hkv=3, ps=8),
    dict(keys=[1000], new=[5], K=6, Hq=128, Hkv=1, causal=False),
    dict(keys=[8200], new=[1], K=64, ps=8, Hq=8, Hkv=1, width=1100),       # clusters
    dict(keys=[33000], new=[1], K=100, ps=8, Hq=16, Hkv=1, width=4200, D=64),
    dict(keys=[2, 5], new=[4, 9], K=2, packed=True),                         # more new tokens than keys
    # enough tokens for blocks of four: 1, 2, 3 and 8 q-heads per kv-head, ragged blocks, short and empty
    # requests, tokens on both sides of top_k
    dict(keys=[300, 400], new=[90] * 2, K=11, Hq=13, Hkv=13, ps=8, D=64),
    dict(keys=[300, 91], new=[91] * 2, K=4, Hq=26, Hkv=13, ps=8, D=96),
    dict(keys=[250, 0, 333, 60], new=[101, 0, 222, 60], K=5, Hq=15, Hkv=5, packed=True, tail=2),
    dict(keys=[600, 500], new=[77] * 2, K=9, Hq=64, Hkv=8, ps=16, D=192, causal=False),
    dict(keys=[200], new=[200], K=20, Hq=48, Hkv=8, ps=8, D=256, kf=2, kl=3),
]


@pytest.mark.parametrize("c", SELECT, ids=[str(i) for i in range(len(SELECT))])
def test_select_pages(c):
    c = dict(c)
    K, kf, kl, causal = c.pop("K"), c.pop("kf", 1), c.pop("kl", 1), c.pop("causal", True)
    p = Problem(seed=4, **c)
    kf, kl = min(kf, K), min(kl, K - min(kf, K))
    bnd = e4m3(ref.bounds(p))
    q = p.q.cuda()
    lists = torch.full((*p.q.shape[:-2], p.Hkv, K), -7, dtype=torch.int32, device="cuda")
    fa8.select_pages(q, bnd.cuda(), K, pages=lists, causal=causal, keep_first=kf, keep_last=kl, **p.index_args())
    ok()
    assert torch.equal(p.flat(lists.cpu()), ref.select(p, bnd, K, causal, kf, kl))
    assert (lists[p.T:] == -7).all() if p.packed else True  # rows behind the last sequence


@pytest.mark.parametrize("four", [False, True], ids=["one", "four"])
@pytest.mark.parametrize("K", [2, 37, 300])
@pytest.mark.parametrize("kind", ["all_equal", "zero_query", "few_levels", "cancel", "one_ulp", "nan_page", "nan_query",
                                  "many_ties"])
def test_select_pages_ties_and_close_scores(kind, K, four):
    """Scores that are equal, or differ only below fp32: the choice is that of exact numbers."""
    p = Problem([8 * 700], [1], Hq=8, Hkv=1, D=128, ps=8, seed=5)
    n = 700
    g = p.g
    bnd = val(e4m3(ref.bounds(p)))
    q = val(p.q)
    phys = p.bt[0].long()
    if kind == "all_equal":
        bnd[:] = bnd[0].clone()
    elif kind == "zero_query":
        q[:] = 0
    elif kind == "few_levels":
        bnd[phys] = torch.randint(-1, 2, (n, 1, 1, 1), generator=g).double().expand(n, 1, 2, 128)
    elif kind == "cancel":  # +-448 products that cancel, the order decided by the smallest values
        bnd[:] = 448.0
        q[..., :64], q[..., 64:] = 448.0, -448.0
        q[..., 0] = 2.0 ** -9
        bnd[phys, 0, :, 0] = torch.randint(0, 8, (n, 1), generator=g).double() * 2.0 ** -9
    elif kind == "one_ulp":  # page j differs from the others by one smallest product
        bnd[:] = bnd[0].clone()
        q[..., 7] = 2.0 ** -9
        bnd[phys, 0, :, 7] = (torch.randperm(n, generator=g) % 5).double()[:, None] * 2.0 ** -9
    elif kind == "nan_page":
        bnd[phys[[5, 600]], 0, :, 3] = math.nan
    elif kind == "nan_query":
        q[0, 0, 2, 9] = math.nan
    elif kind == "many_ties":  # 600 equal pages around the threshold
        bnd[phys[50:650]] = bnd[phys[50]].clone()
    p.q = q.float().to(E4M3)
    b8 = bnd.float().to(E4M3)
    want = ref.select(p, b8, K)[0]
    if four:  # the same token many times over, enough of them for blocks of four
        m = 1301
        p.q = p.q.view(torch.uint8).expand(1, m, -1, -1).contiguous().view(E4M3)
        p.new, p.T = [m], m
        got = run_select(p, b8, K, causal=False)
        assert (got == want).all()
    else:
        assert torch.equal(run_select(p, b8, K)[0, 0], want)


def test_select_pages_widest_table():
    """16384 columns, most of them used: more scores than a CTA's threads hold in registers."""
    p = Problem([8 * 15001 - 3], [1], Hq=4, Hkv=1, D=64, DV=64, ps=8, width=16384, seed=40)
    b = e4m3(torch.randn((p.k.shape[0], 1, 2, 64), generator=p.g))
    for K in (1, 500, 4096):
        got = run_select(p, b, K, keep_first=0, keep_last=1)
        q, lo, hi = val(p.q)[0, 0], val(b)[p.bt[0, :15001].long(), 0, 0], val(b)[p.bt[0, :15001].long(), 0, 1]
        s = (q.clamp_max(0) @ lo.T + q.clamp_min(0) @ hi.T).amax(0)
        s[-1] = math.inf
        want = s.sort(descending=True, stable=True).indices[:K].sort().values
        assert torch.equal(got[0, 0, 0].long(), want)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("four", [False, True], ids=["one", "four"])
def test_select_pages_keys_of_the_largest_scores(sign, four):
    """Products of the largest values over 256 channels, apart by the smallest ones, more undecided pages
    than are ranked directly: the exact scores reach their full width on either side of zero."""
    n, K = 700, 150
    p = Problem([8 * n], [1], Hq=2, Hkv=1, D=256, ps=8, seed=43)
    bnd = torch.full(p.k.shape[:1] + (1, 2, 256), 448.0 * sign, dtype=torch.float64)
    q = torch.full((1, 1, 2, 256), 448.0, dtype=torch.float64)
    q[..., 3] = 2.0 ** -9
    bnd[p.bt[0].long(), 0, :, 3] = (torch.randperm(n, generator=p.g) % 8).double()[:, None] * 2.0 ** -9
    p.q, b8 = q.float().to(E4M3), bnd.float().to(E4M3)
    want = ref.select(p, b8, K)[0]
    if four:
        m = 1301
        p.q = p.q.view(torch.uint8).expand(1, m, -1, -1).contiguous().view(E4M3)
        p.new, p.T = [m], m
        assert (run_select(p, b8, K, causal=False) == want).all()
    else:
        assert torch.equal(run_select(p, b8, K)[0, 0], want)


@pytest.mark.parametrize("n", [600, 1025, 2047])
def test_select_pages_long_lists_by_one_warp(n):
    """Blocks of four tokens over more pages than a warp holds in registers."""
    p = Problem([8 * n - 3], [60], Hq=42, Hkv=21, D=64, DV=64, ps=8, seed=44)
    bnd = e4m3(ref.bounds(p))
    got = run_select(p, bnd, 77, keep_first=0, keep_last=1)
    assert torch.equal(p.flat(got), ref.select(p, bnd, 77, True, 0, 1))


@pytest.mark.parametrize("Hkv", [2, 40])
def test_packed_rows_ahead_of_the_first_sequence_stay(Hkv):
    """cu_seqlens_q that begins past row 0, one token at a time and in blocks of four."""
    p = Problem([90, 200], [33, 70], Hq=Hkv, Hkv=Hkv, D=64, DV=64, ps=8, packed=True, tail=6, seed=41)
    shift = 5
    bnd = e4m3(ref.bounds(p))
    q = torch.roll(p.q.view(torch.uint8), shift, 0).view(E4M3).cuda()
    kw = dict(p.index_args(), cu_seqlens_q=(p.cu_q + shift).cuda())
    lists = torch.full((p.T + p.tail, Hkv, 4), -7, dtype=torch.int32, device="cuda")
    fa8.select_pages(q, bnd.cuda(), 4, pages=lists, **kw)
    out = torch.full((p.T + p.tail, Hkv, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hkv, p.T + p.tail), 7.0, device="cuda")
    fa8.fwd_pages(q, p.k.cuda(), p.v.cuda(), lists, out=out, lse=lse, **kw)
    ok()
    assert torch.equal(lists[shift:shift + p.T].cpu(), ref.select(p, bnd, 4))
    for x, keep in ((lists, -7), (out, 7.0), (lse.T, 7.0)):
        assert (x[:shift] == keep).all() and (x[shift + p.T:] == keep).all() and (x[shift:shift + p.T] != keep).any()


def test_select_pages_strided():
    p = Problem([800, 300], [2, 2], Hq=8, Hkv=2, D=64, DV=64, ps=16, seed=6)
    bnd = e4m3(ref.bounds(p))
    wide = torch.zeros((bnd.shape[0], 2, 3, 64), dtype=torch.uint8, device="cuda")
    wide[:, :, :2] = bnd.view(torch.uint8).cuda()
    bs = wide.view(E4M3)[:, :, :2]
    qs = torch.zeros((2, 2, 8, 96), dtype=torch.uint8, device="cuda")
    qs[..., :64] = p.q.view(torch.uint8).cuda()
    out = torch.full((2, 2, 2, 9), -3, dtype=torch.int32, device="cuda")
    table = torch.full((2, 99), 1 << 30, dtype=torch.int32, device="cuda")
    table[:, :p.bt.shape[1]] = p.bt.cuda()
    kw = dict(p.index_args(), block_table=table[:, :p.bt.shape[1]])
    fa8.select_pages(qs.view(E4M3)[..., :64], bs, 7, pages=out[..., 1:8], **kw)
    ok()
    assert torch.equal(p.flat(out[..., 1:8].cpu()), ref.select(p, bnd, 7))
    assert (out[..., 0] == -3).all() and (out[..., 8] == -3).all()


# ------------------------------------------------------------------ attention over listed pages
def random_lists(p, K, seed=0, causal=True, hole=0.1):
    g = torch.Generator().manual_seed(seed)
    out = torch.full((p.T, p.Hkv, K), -1, dtype=torch.int32)
    for b, i, t in p.tokens():
        n = -(-p.visible(b, i, causal) // p.ps)
        for h in range(p.Hkv):
            m = min(n, K)
            out[t, h, :m] = torch.randperm(n, generator=g)[:m].to(torch.int32)
            out[t, h][torch.rand(K, generator=g) < hole] = -1
    return out


def check_attend(p, lists, causal=True, sink=None, scale=None, out_dtype=torch.bfloat16, descales=True, got=None):
    """|O - O_ref| <= half a step of the output type + sum p|v| (2^-11: P in f16; 2^-17 reach: each
    score is off by up to D/16 <= 16 MMA steps' dropped bits, 2^-22 each, and the fp32 roundings
    of its scale, argument and exponential) + n 2^-25 max|v| (P below the f16 normals).
    |LSE - LSE_ref| <= 2^-17 reach + 2^-20 (1 + |LSE|)."""
    d = dict(dq=p.dq, dk=p.dk, dv=p.dv) if descales else {}
    o_ref, l_ref, mass, reach = ref.attend(p, lists, causal, sink, scale, **d)
    if got is None:
        shape = (p.T, p.Hkv, lists.shape[-1]) if p.packed else (p.B, p.new[0], p.Hkv, lists.shape[-1])
        pages = torch.nn.functional.pad(lists, (0, 0, 0, 0, 0, p.tail), value=0).cuda() if p.packed else lists.reshape(shape).cuda()
        kw = {f"descale_{n}": x.cuda() for n, x in zip("qkv", (p.dq, p.dk, p.dv))} if descales else {}
        out = torch.full((*p.q.shape[:-1], p.DV), 7.0, dtype=out_dtype, device="cuda")
        lse = torch.full((p.B, p.Hq, p.new[0]) if not p.packed else (p.Hq, p.T + p.tail), 7.0, device="cuda")
        fa8.fwd_pages(p.q.cuda(), p.k.cuda(), p.v.cuda(), pages, out=out, lse=lse, causal=causal,
                      sink=None if sink is None else sink.cuda(), softmax_scale=scale or 0.0, **p.index_args(), **kw)
        ok()
    else:
        out, lse = got
    o = p.flat(out.cpu()).double()
    l = (lse.cpu().T[:p.T] if p.packed else lse.cpu().transpose(1, 2).reshape(p.T, p.Hq)).double()
    if p.packed:  # rows behind the last sequence stay as they were
        assert (out[p.T:] == 7.0).all() and (lse[:, p.T:] == 7.0).all()
    n = lists.shape[-1] * p.ps
    vmax = float(val(p.v).nan_to_num(0).abs().max()) * (float(p.dv.max()) if descales else 1.0)
    step = torch.finfo(out_dtype).eps / 2
    tol = step * o_ref.abs() + (1 + step) * (mass * (2.0 ** -11 + 2.0 ** -17 * (1 + reach[..., None])) + n * 2.0 ** -25 * vmax)
    bad = ((o - o_ref).abs() > tol) | o.isnan()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((o - o_ref).abs() / tol.clamp_min(1e-30)).max()):.3g} of the bound"
    same = (l == l_ref) | ((l - l_ref).abs() <= 2.0 ** -17 * reach + 2.0 ** -20 * (1 + l_ref.abs()))
    assert same.all(), (l - l_ref).abs().max()
    return out, lse


DIMS = [(64, 64), (96, 96), (128, 128), (192, 128), (192, 192), (256, 256)]


@pytest.mark.parametrize("D,DV", DIMS)
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1), (24, 2), (20, 1)])
def test_fwd_pages_dims_and_heads(D, DV, Hq, Hkv):
    p = Problem([300, 77], [2, 2], Hq=Hq, Hkv=Hkv, D=D, DV=DV, ps=16, seed=7)
    p.poison()
    check_attend(p, random_lists(p, 9))


ATTEND = [
    dict(keys=[1], new=[1], K=1),
    dict(keys=[5, 0, 9], new=[1] * 3, K=2, ps=8),
    dict(keys=[100, 0, 64, 1], new=[7, 0, 64, 1], K=3, packed=True, tail=3),
    dict(keys=[3, 2], new=[5, 5], K=2),                                   # tokens that see no key
    dict(keys=[3, 2], new=[5, 5], K=2, sink=True),
    dict(keys=[500], new=[4], K=12, ps=24, causal=False, sink=True),
    dict(keys=[700, 650], new=[1, 1], K=5, ps=128, out=torch.float16),
    dict(keys=[900], new=[1], K=6, Hq=128, Hkv=1),
    dict(keys=[900], new=[1], K=40, Hq=12, Hkv=1, ps=8, descales=False),
    dict(keys=[1200], new=[1], K=64, Hq=8, Hkv=1, ps=16),                 # two CTAs a cluster
    dict(keys=[3000], new=[1], K=256, Hq=8, Hkv=1, ps=8, sink=True),      # four
    dict(keys=[5000], new=[1], K=300, Hq=16, Hkv=1, ps=16),               # eight, of eight warps
    dict(keys=[5000], new=[2], K=200, Hq=24, Hkv=3, ps=24, D=256, DV=256),
    dict(keys=[4200], new=[1], K=520, Hq=6, Hkv=2, ps=8, D=96, DV=96),
    dict(keys=[9000], new=[1], K=2, Hq=4, Hkv=1, ps=4096, D=64, DV=64),   # the largest page
    dict(keys=[300], new=[3], K=0),                                        # an empty list
    dict(keys=[400], new=[1], K=20, scale=2.5),                           # sharp softmax
    dict(keys=[400], new=[1], K=20, qscale=30.0),                         # large scores
]


@pytest.mark.parametrize("c", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_fwd_pages(c):
    c = dict(c)
    K, causal, out = c.pop("K"), c.pop("causal", True), c.pop("out", torch.bfloat16)
    sink, descales, scale = c.pop("sink", False), c.pop("descales", True), c.pop("scale", None)
    p = Problem(seed=8, scale=c.pop("qscale", 1.0), **c)
    p.poison()
    s = torch.randn(p.Hq, generator=p.g) if sink else None
    check_attend(p, random_lists(p, K, causal=causal), causal, s, scale, out, descales)


@pytest.mark.parametrize("order", ["up", "down", "saw"])
@pytest.mark.parametrize("span", [3.0, 8.0, 40.0, 400.0])
@pytest.mark.parametrize("Hq,D", [(4, 128), (12, 64), (8, 256)])
def test_fwd_pages_scores_that_climb(Hq, D, span, order):
    """One row's scores run through `span` binary orders over the list, chunk after chunk, up, down and in
    a saw: the maximum that P is taken against moves in small and in large steps, for some rows only."""
    n, ps = 900, 16
    p = Problem([n], [1], Hq=Hq, Hkv=1, D=D, DV=D, ps=ps, seed=45)
    levels = torch.arange(1, 127).to(torch.uint8).view(E4M3).double()  # the positive values
    j = torch.arange(n)
    at = {"up": j * 126 // n, "down": 125 - j * 126 // n, "saw": (j * 5) % n * 126 // n}[order]
    k = torch.zeros((p.k.shape[0], ps, 1, D), dtype=torch.float64)
    k[p.bt[0].long()[j // ps], j % ps, 0, 1] = levels[at]
    q = torch.zeros((1, 1, Hq, D), dtype=torch.float64)
    q[0, 0, :, 1] = torch.tensor([1.0, 0.5, -1.0, 0.125] * 4)[:Hq].double()
    p.q, p.k = q.float().to(E4M3), k.float().to(E4M3)
    lists = torch.arange(-(-n // ps), dtype=torch.int32).reshape(1, 1, -1)
    check_attend(p, lists, scale=span * math.log(2) / 448, descales=False)


def test_fwd_pages_duplicates_order_and_invisible():
    """A page listed twice counts twice; order does not matter; pages past the token add nothing."""
    p = Problem([200], [3], Hq=8, Hkv=2, ps=16, seed=9)
    p.poison()
    lists = torch.tensor([[9, 2, 2, -1, 12, 0, -5]] * 6, dtype=torch.int32).reshape(3, 2, 7)
    check_attend(p, lists)
    lists = torch.full((3, 2, 7), 12, dtype=torch.int32)  # holds the last keys only: key 197 up
    o, l = check_attend(p, lists)
    assert (l.cpu() > -math.inf).all()
    p2 = Problem([200], [60], Hq=8, Hkv=2, ps=16, seed=9)
    o, l = check_attend(p2, torch.full((60, 2, 1), 12, dtype=torch.int32))
    assert (o[0, :52] == 0).all() and (l[0, :, :52] == -math.inf).all()


def test_fwd_pages_nan_reaches_only_its_rows():
    p = Problem([64], [1], Hq=4, Hkv=2, ps=16, seed=10)
    p.k.view(torch.uint8)[int(p.bt[0, 1]), 3, 0, 5] = 0x7F  # a visible key of kv-head 0
    lists = torch.tensor([[[0, 1, 2], [0, 1, 2]]], dtype=torch.int32)
    out, lse = fa8.fwd_pages(p.q.cuda(), p.k.cuda(), p.v.cuda(), lists.cuda()[None], **p.index_args())
    ok()
    assert out[0, 0, :2].isnan().all() and lse[0, :2].isnan().all()
    assert not out[0, 0, 2:].isnan().any() and not lse[0, 2:].isnan().any()


def test_fwd_pages_strided_and_bit_stable():
    """K and V as views of one buffer, strided Q, O and LSE; twice the same bits."""
    p = Problem([600, 210], [2, 2], Hq=8, Hkv=2, D=192, DV=128, ps=16, seed=11)
    p.poison()
    pool = torch.zeros((p.k.shape[0], 16, 2, 320), dtype=torch.uint8, device="cuda")
    pool[..., :192], pool[..., 192:] = p.k.view(torch.uint8).cuda(), p.v.view(torch.uint8).cuda()
    k, v = pool.view(E4M3)[..., :192], pool.view(E4M3)[..., 192:]
    q = torch.zeros((2, 2, 8, 208), dtype=torch.uint8, device="cuda")
    q[..., :192] = p.q.view(torch.uint8).cuda()
    lists = random_lists(p, 10)
    pages = torch.zeros((2, 2, 2, 11), dtype=torch.int32, device="cuda")
    pages[..., :10] = lists.reshape(2, 2, 2, 10).cuda()
    outs = []
    for _ in range(2):
        out = torch.zeros((2, 2, 8, 136), dtype=torch.bfloat16, device="cuda")[..., :128]
        lse = torch.zeros((2, 2, 8), device="cuda").transpose(1, 2)
        fa8.fwd_pages(q.view(E4M3)[..., :192], k, v, pages[..., :10], out=out, lse=lse, descale_q=p.dq.cuda(),
                      descale_k=p.dk.cuda(), descale_v=p.dv.cuda(), **p.index_args())
        ok()
        outs.append((out.clone(), lse.clone()))
    check_attend(p, lists, got=outs[0])
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ------------------------------------------------------------------ rotary append
def check_rope(p, dtype, R, off, inter, positions=None, rot_scale=1.0, layout="paged", freq=torch.float64, base=10000.0,
               mult=1.0, descales=True):
    """Every stored value lies between the E4M3 roundings of ref - slack and ref + slack, where slack
    = 2^-20 (|x0| + |x1|) |rot_scale| / descale bounds the fp32 arithmetic: sine and cosine to 2^-22
    (their argument and CUDA's two ulps), two products and a sum, the reciprocal and its product."""
    g = p.g
    T, D, DV = p.T + p.tail, p.D, p.DV
    x = torch.randn((T, p.Hq * D + p.Hkv * (D + DV)), generator=g).mul(mult).to(dtype)
    shape = (T,) if p.packed else (p.B, p.new[0])
    dev = x.cuda().reshape(*shape, -1)
    cut = [p.Hq * D, (p.Hq + p.Hkv) * D]
    q, k, v = (t.unflatten(-1, (-1, d)) for t, d in ((dev[..., :cut[0]], D), (dev[..., cut[0]:cut[1]], D), (dev[..., cut[1]:], DV)))
    inv = (base ** -(torch.arange(0, R, 2, dtype=torch.float64) / R)).to(freq)
    d = {n: torch.rand((p.B, p.Hkv), generator=g) * 0.1 + 0.01 for n in "qkv"} if descales else {}
    if layout == "paged":
        ko, vo = p.k.cuda(), p.v.cuda()
        kw = p.index_args()
    elif layout == "varlen":
        ko, vo = (e4m3(torch.randn((sum(p.keys) + 5, p.Hkv, z), generator=g)).cuda() for z in (D, DV))
        kw = dict(p.index_args(), block_table=None, page_size=0)
    else:
        ko, vo = (e4m3(torch.randn((p.B, p.keys[0], p.Hkv, z), generator=g)).cuda() for z in (D, DV))
        kw = dict(cu_seqlens_q=p.index_args()["cu_seqlens_q"])
    k0, v0 = val(ko.cpu()).clone(), val(vo.cpu()).clone()
    q8 = torch.zeros((*shape, p.Hq, D), dtype=torch.uint8, device="cuda").view(E4M3)
    fa8.rope_append(q, k, v, inv.cuda(), k_out=ko, v_out=vo, q_out=q8, interleaved=inter, rotary_offset=off,
                    rot_scale=rot_scale, positions=None if positions is None else positions.cuda().reshape(shape),
                    **{f"descale_{n}": t.cuda() for n, t in d.items()}, **kw)
    ok()
    req = torch.tensor([b for b, _, _ in p.tokens()], dtype=torch.long)
    key = torch.tensor([p.keys[b] - p.new[b] + i for b, i, _ in p.tokens()], dtype=torch.long)
    pos = key if positions is None else positions.reshape(-1)[:p.T]
    rows = x.cpu()[:p.T].double()
    parts = {"q": rows[:, :cut[0]].unflatten(-1, (-1, D)), "k": rows[:, cut[0]:cut[1]].unflatten(-1, (-1, D)),
             "v": rows[:, cut[1]:].unflatten(-1, (-1, DV))}
    if layout == "paged":
        slot = (p.bt.long()[req, key // p.ps], key % p.ps)
    elif layout == "varlen":
        slot = (p.cu_k.long()[req] + key,)
    else:
        slot = (req, key)
    for n, out in (("q", q8), ("k", ko), ("v", vo)):
        y = parts[n]
        ds = d[n][req].double().repeat_interleave(y.shape[1] // p.Hkv, 1)[..., None] if d else torch.ones(1, 1, 1).double()
        want, slack = y, torch.zeros_like(y)
        if n != "v":
            want = ref.rope(y, pos, inv, inter, off, rot_scale)
            mag = ref.rope(y.abs(), torch.zeros_like(pos), inv, inter, off, 1.0)
            i = torch.arange(R // 2)
            a, b = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + R // 2 + i)
            slack = torch.zeros_like(y)
            slack[..., a] = slack[..., b] = (mag[..., a] + mag[..., b]) * abs(rot_scale) * 2.0 ** -20
        want, slack = want / ds, slack / ds + want.abs() / ds * 2.0 ** -22
        got = val(out.cpu())
        if n == "q":
            if p.packed:
                assert (got[p.T:] == 0).all()
            got = p.flat(got)
        else:
            rest = (k0 if n == "k" else v0).clone()
            rest[slot] = got[slot]
            assert torch.equal(got.nan_to_num(9e9), rest.nan_to_num(9e9))  # other slots as they were
            got = got[slot]
        lo, hi = val(e4m3(want - slack)), val(e4m3(want + slack))
        assert ((got >= lo) & (got <= hi)).all(), n


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,DV,R,off", [(64, 64, 64, 0), (96, 96, 48, 0), (128, 128, 128, 0), (128, 128, 16, 8),
                                        (192, 128, 64, 128), (192, 192, 192, 0), (256, 256, 64, 192), (256, 256, 256, 0)])
def test_rope_append(D, DV, R, off, dtype, inter):
    check_rope(Problem([40, 7, 300], [3] * 3, Hq=6, Hkv=2, D=D, DV=DV, seed=12), dtype, R, off, inter)


@pytest.mark.parametrize("layout", ["paged", "varlen"])
def test_rope_append_packed(layout):
    p = Problem([40, 0, 300, 9], [33, 0, 300, 1], Hq=8, Hkv=8, packed=True, tail=3, seed=13)
    check_rope(p, torch.bfloat16, 128, 0, False, layout=layout)


def test_rope_append_dense_many_tokens():
    """More tokens than a wave of one-token CTAs, not a multiple of four."""
    p = Problem([401, 401], [399, 399], Hq=2, Hkv=1, D=64, DV=64, seed=14)
    check_rope(p, torch.float16, 32, 16, True, layout="dense", descales=False)


@pytest.mark.parametrize("D,DV,R,off,Hq,Hkv,T,inter", [
    (128, 128, 128, 0, 24, 8, 1301, False), (96, 96, 32, 24, 9, 9, 1707, True), (192, 128, 64, 128, 10, 5, 1799, False),
    (256, 256, 256, 0, 7, 7, 1111, True), (64, 64, 48, 8, 8, 1, 9733, False)])
def test_rope_append_prefill(D, DV, R, off, Hq, Hkv, T, inter):
    """Token counts at which a thread walks several heads: odd numbers of them, packed, with a tail."""
    p = Problem([T - 500 + 16, 500], [T - 500, 500], Hq=Hq, Hkv=Hkv, D=D, DV=DV, packed=True, tail=2, seed=42)
    check_rope(p, torch.bfloat16, R, off, inter)


@pytest.mark.parametrize("freq", [torch.float64, torch.float32])
def test_rope_append_far_positions(freq):
    """Positions up to 2^29 and negative ones; an attention factor.  The 64-bit reference's own
    angle is off by 2^29 2^-53 = 2^-24 rad there, the kernel's 2^29 (1 / 2 pi) 2^-52 turns = 2^-23 rad."""
    p = Problem([40, 90], [20, 20], Hq=2, Hkv=1, seed=15)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (2, 20), generator=p.g, dtype=torch.int64).to(torch.int32)
    pos[0, :3] = torch.tensor([(1 << 31) - 1, -(1 << 31), 1 << 20], dtype=torch.int32)
    check_rope(p, torch.bfloat16, 128, 0, False, positions=pos // 4, rot_scale=1.37, freq=freq)


def test_rope_append_saturates_and_keeps_nan():
    p = Problem([4], [4], Hq=1, Hkv=1, D=64, DV=64, seed=16)
    check_rope(p, torch.bfloat16, 64, 0, False, mult=1e4)
    x = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0, 0], x[0, 1, 0, 0], x[0, 2, 0, 0] = math.inf, -math.inf, math.nan
    ko, vo = p.k.cuda(), p.v.cuda()
    for inter in (False, True):  # dims 16 to 47 rotated; an infinity beside them stays one
        fa8.rope_append(x, x, x, torch.ones(16, dtype=torch.float64).cuda(), k_out=ko, v_out=vo, rotary_offset=16,
                        interleaved=inter, **p.index_args())
        ok()
        for cache in (ko, vo):
            got = val(cache.cpu())[int(p.bt[0, 0]), :4, 0]
            assert got[0, 0] == 448 and got[1, 0] == -448 and got[2, 0].isnan() and got[3, 0] == 0
            assert (got[:, 1:] == 0).all()


def test_rope_inv_freq_on_device_matches_angles():
    """The stretched frequencies reach the kernel: YaRN's, at a far position."""
    inv = fa8.rope_inv_freq(64, 10000.0, scaling="yarn", factor=8.0, original_len=4096, device="cuda")
    x = torch.ones((1, 1, 1, 64), dtype=torch.float16, device="cuda")
    p = Problem([1], [1], Hq=1, Hkv=1, D=64, DV=64, seed=17)
    pos = torch.tensor([[123457]], dtype=torch.int32, device="cuda")
    q8 = fa8.rope_append(x, x, x, inv, k_out=p.k.cuda(), v_out=p.v.cuda(), positions=pos, descale_q=torch.tensor(2.0 ** -8).cuda(), **p.index_args())
    ok()
    want = ref.rope(torch.ones(1, 1, 64), torch.tensor([123457]), inv.cpu(), False, 0, 1.0) * 256
    got = val(q8.cpu()).reshape(1, 1, 64)
    lo, hi = val(e4m3(want - 2e-3)), val(e4m3(want + 2e-3))
    assert ((got >= lo) & (got <= hi)).all()


# ------------------------------------------------------------------ bad pages are reported, not followed
def test_bad_table_entries_are_reported():
    p = Problem([64], [1], Hq=2, Hkv=1, ps=16, seed=18)
    good = p.bt.clone()
    q, k, v = p.q.cuda(), p.k.cuda(), p.v.cuda()
    lists = torch.tensor([[[[0, 1, 2, 3]]]], dtype=torch.int32, device="cuda")
    x = torch.zeros((1, 1, 2, 128), dtype=torch.bfloat16, device="cuda")
    inv = torch.ones(8, dtype=torch.float64, device="cuda")
    for entry in (-1, p.k.shape[0], 1 << 30):
        bt = good.clone()
        bt[0, 3] = entry
        kw = dict(p.index_args(), block_table=bt.cuda())
        before = k.clone().view(torch.uint8), v.clone().view(torch.uint8)
        fa8.rope_append(x, x[:, :, :1], x[:, :, :1], inv, k_out=k, v_out=v, **kw)
        assert fa8.check() == fa8.FA8_ERR_DEVICE_BOUNDS
        assert torch.equal(before[0], k.view(torch.uint8)) and torch.equal(before[1], v.view(torch.uint8))
        bnd = fa8.page_bounds(k, cu_seqlens_k=kw["cu_seqlens_k"], block_table=kw["block_table"], page_size=16)
        assert fa8.check() == fa8.FA8_ERR_DEVICE_BOUNDS
        out, lse = fa8.fwd_pages(q, k, v, lists, **kw)
        assert fa8.check() == fa8.FA8_ERR_DEVICE_BOUNDS
        want, lw = fa8.fwd_pages(q, k, v, lists[..., :3].contiguous(), **p.index_args())
        ok()
        assert torch.equal(out, want) and torch.equal(lse, lw)
        got = fa8.select_pages(q, bnd, 2, keep_first=0, keep_last=0, **kw)
        assert fa8.check() == fa8.FA8_ERR_DEVICE_BOUNDS
        assert 3 not in got.flatten().tolist()
    fa8.fwd_pages(q, k, v, lists + 100, **p.index_args())  # list entries past the table
    assert fa8.check() == fa8.FA8_ERR_DEVICE_BOUNDS
    long = dict(p.index_args(), cu_seqlens_k=torch.tensor([0, 1000], dtype=torch.int32, device="cuda"))
    fa8.fwd_pages(q, k, v, lists, **long)  # more keys than the table has room for
    assert fa8.check() == fa8.FA8_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("python", [False, True])
def test_outputs_made_for_another_stream(python, monkeypatch):
    """With stream= the outputs that a call makes must not share memory with work that the current stream
    has still to run, and page_bounds' zeros must come before its kernel."""
    monkeypatch.setattr(fa8, "_entries", {})
    if python:
        monkeypatch.setattr(fa8, "_args_module", lambda: None)
    p = Problem([640], [2], Hq=8, Hkv=2, D=128, ps=16, seed=46)
    q, k, v = p.q.cuda(), p.k.cuda(), p.v.cuda()
    w = fa8.rope_inv_freq(128, device="cuda")
    x = [torch.randn((1, 2, h, 128), generator=p.g).cuda().bfloat16() for h in (8, 2, 2)]
    kw = p.index_args()
    caches = [[t.clone() for t in (k, v)] for _ in range(2)]
    side = torch.cuda.Stream()

    def calls(cache, stream):
        b = fa8.page_bounds(k, stream=stream, **{n: t for n, t in kw.items() if n != "cu_seqlens_q"})
        lists = fa8.select_pages(q, b, 5, stream=stream, **kw)
        return (b.view(torch.uint8), lists, *fa8.fwd_pages(q, k, v, lists, stream=stream, **kw),
                fa8.rope_append(*x, w, k_out=cache[0], v_out=cache[1], stream=stream, **kw).view(torch.uint8))

    want = [t.clone() for t in calls(caches[0], None)]
    sizes = [t.nbytes for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for n in sizes:  # freed blocks that the current stream writes later
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x55)
    got = calls(caches[1], side)
    side.synchronize()
    kept = [t.clone() for t in got]
    ok()
    for a, b, c in zip(got, want, kept):
        assert torch.equal(a, b) and torch.equal(c, b)


@pytest.mark.parametrize("python", [False, True])
def test_host_tensors_are_refused(python, monkeypatch):
    monkeypatch.setattr(fa8, "_entries", {})
    if python:
        monkeypatch.setattr(fa8, "_args_module", lambda: None)
    p = Problem([64], [1], Hq=2, Hkv=1, ps=16, seed=18)
    lists = torch.zeros((1, 1, 1, 2), dtype=torch.int32)
    args = (p.q.cuda(), p.k.cuda(), p.v.cuda(), lists.cuda())
    for i in range(4):
        mixed = list(args)
        mixed[i] = mixed[i].cpu()
        with pytest.raises(ValueError, match="device"):
            fa8.fwd_pages(*mixed, **p.index_args())
    with pytest.raises(ValueError, match="device"):
        fa8.fwd_pages(*args, **dict(p.index_args(), block_table=p.bt))
    with pytest.raises(ValueError, match="device"):
        fa8.page_bounds(p.k, **{n: t for n, t in p.index_args("cpu").items() if n != "cu_seqlens_q"})
    fa8.fwd_pages(*args, **p.index_args())
    ok()


# ------------------------------------------------------------------ together
def chain(q, k, v, inv, p, kc, vc, bnd, K, dev_args, ds, **kw):
    q8 = fa8.rope_append(q, k, v, inv, k_out=kc, v_out=vc, descale_q=ds, descale_k=ds, descale_v=ds, **dev_args)
    fa8.page_bounds(kc, bnd, new_tokens=p.new[0], **{n: dev_args[n] for n in ("cu_seqlens_k", "block_table", "page_size")})
    lists = fa8.select_pages(q8, bnd, K, **dev_args)
    out, lse = fa8.fwd_pages(q8, kc, vc, lists, descale_q=ds, descale_k=ds, descale_v=ds, **dev_args)
    return q8, lists, out, lse


def chain_inputs(p, seed):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn((p.B, p.new[0], h, d), generator=g).bfloat16().cuda() for h, d in ((p.Hq, p.D), (p.Hkv, p.D), (p.Hkv, p.DV))]
    return x + [fa8.rope_inv_freq(p.D, 500000.0, device="cuda")]


@pytest.mark.parametrize("D,DV,Sq", [(128, 128, 1), (192, 128, 3), (256, 256, 2)])
def test_a_step_with_all_pages_is_dense_attention(D, DV, Sq):
    """With room for every page the run of the four equals fa8_fwd on the cache that they filled."""
    from parity_util import LSE_ABS, MAX_ABS
    p = Problem([700, 150, 16], [Sq] * 3, Hq=8, Hkv=2, D=D, DV=DV, ps=16, seed=19)
    args, ds = p.index_args(), torch.full((3, 2), 1.0 / 64, device="cuda")
    kc, vc = e4m3(val(p.k).float() * 16).cuda(), e4m3(val(p.v).float() * 16).cuda()
    bnd = fa8.page_bounds(kc, **{n: args[n] for n in ("cu_seqlens_k", "block_table", "page_size")})
    q8, lists, out, lse = chain(*chain_inputs(p, 20), p, kc, vc, bnd, 64, args, ds)
    dense, dlse = fa8.fwd(q8, kc, vc, descale_q=ds, descale_k=ds, descale_v=ds, causal=True, **args)
    ok()
    vs = float((vc.float() / 64).square().mean().sqrt())
    assert (out.float() - dense.float()).abs().max() <= 2 * MAX_ABS * vs
    assert (lse - dlse).abs().max() <= 2 * LSE_ABS
    # and the 64-bit form on the same cache, with its own choice of pages
    p.q, p.k, p.v = q8.cpu(), kc.cpu(), vc.cpu()
    p.dq = p.dk = p.dv = ds.cpu()
    check_attend(p, p.flat(lists.cpu()), got=(out, lse))


def test_a_step_chooses_what_the_plain_forms_choose_and_replays():
    """Captured into a graph and replayed on new inputs: the same bits as eager calls, on a stream
    that is not the default one."""
    p = Problem([900, 1300], [2, 2], Hq=8, Hkv=2, ps=16, seed=21)
    args, ds = p.index_args(), torch.full((2, 2), 1.0 / 64, device="cuda")
    kc, vc = e4m3(val(p.k).float() * 16).cuda(), e4m3(val(p.v).float() * 16).cuda()
    bnd = fa8.page_bounds(kc, **{n: args[n] for n in ("cu_seqlens_k", "block_table", "page_size")})
    x = chain_inputs(p, 22)
    start = [t.view(torch.uint8).clone() for t in (kc, vc, bnd)]

    def reset():
        for t, s in zip((kc, vc, bnd), start):
            t.view(torch.uint8).copy_(s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(*x, p, kc, vc, bnd, 10, args, ds)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = chain(*x, p, kc, vc, bnd, 10, args, ds)
    torch.cuda.synchronize()
    for seed in (23, 24):
        for a, b in zip(x, chain_inputs(p, seed)):
            a.copy_(b)
        reset()
        want = [t.clone() for t in chain(*x, p, kc, vc, bnd, 10, args, ds)]
        ends = [t.view(torch.uint8).clone() for t in (kc, vc, bnd)]
        reset()
        graph.replay()
        torch.cuda.synchronize()
        ok()
        for a, b in zip(held, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        for a, b in zip((kc, vc, bnd), ends):
            assert torch.equal(a.view(torch.uint8), b)
        p.q, p.k, p.v = held[0].cpu(), kc.cpu(), vc.cpu()
        p.dq = p.dk = p.dv = ds.cpu()
        assert torch.equal(val(bnd.cpu()), ref.bounds(p, into=start[2].view(E4M3).reshape(bnd.shape).cpu()))
        assert torch.equal(p.flat(held[1].cpu()), ref.select(p, bnd.cpu(), 10))
        check_attend(p, p.flat(held[1].cpu()), got=held[2:])


def test_offsets_past_32_bits():
    """A pool whose last pages lie beyond 2^32 bytes."""
    ps, Hkv, D, pages = 64, 8, 256, 36000  # 4.7 GB of K, as much of V
    p = Problem([150], [2], Hq=8, Hkv=Hkv, D=D, DV=D, ps=ps, extra=0, seed=25)
    k = torch.zeros((pages, ps, Hkv, D), dtype=torch.uint8, device="cuda").view(E4M3)
    v = torch.zeros((pages, ps, Hkv, D), dtype=torch.uint8, device="cuda").view(E4M3)
    far = torch.tensor([35999, 35990, 35997])
    k.view(torch.uint8)[far.cuda()] = p.k.view(torch.uint8)[p.bt[0].long()].cuda()
    v.view(torch.uint8)[far.cuda()] = p.v.view(torch.uint8)[p.bt[0].long()].cuda()
    kw = dict(p.index_args(), block_table=far.to(torch.int32)[None].cuda())
    x = torch.randn((1, 2, Hkv, D), generator=p.g).half().cuda()
    inv = fa8.rope_inv_freq(D, device="cuda")
    fa8.rope_append(x, x, x, inv, k_out=k, v_out=v, **kw)
    bnd = fa8.page_bounds(k, cu_seqlens_k=kw["cu_seqlens_k"], block_table=kw["block_table"], page_size=ps)
    lists = fa8.select_pages(p.q.cuda(), bnd, 2, **kw)
    out, lse = fa8.fwd_pages(p.q.cuda(), k, v, lists, **kw)
    ok()
    near = [t.view(torch.uint8)[far.cuda()].view(E4M3) for t in (k, v)]
    kw2 = dict(p.index_args(), block_table=torch.arange(3, dtype=torch.int32, device="cuda")[None])
    b2 = fa8.page_bounds(near[0], cu_seqlens_k=kw2["cu_seqlens_k"], block_table=kw2["block_table"], page_size=ps)
    l2 = fa8.select_pages(p.q.cuda(), b2, 2, **kw2)
    o2, s2 = fa8.fwd_pages(p.q.cuda(), near[0], near[1], l2, **kw2)
    ok()
    assert torch.equal(lists, l2) and torch.equal(out, o2) and torch.equal(lse, s2)
    p.k, p.v, p.bt = near[0].cpu(), near[1].cpu(), kw2["block_table"].cpu()
    check_attend(p, p.flat(lists.cpu()), descales=False, got=(out, lse))
    want = ref.rope(x.cpu()[0], torch.tensor([148, 149]), inv.cpu(), False, 0, 1.0)
    got = val(p.k)[2, 20:22]
    assert ((got >= val(e4m3(want - 1e-4))) & (got <= val(e4m3(want + 1e-4)))).all()
