"""Corners of the paged-cache operators on the GPU: exact choices beside NaN pages and where an MMA's dropped
bits add up, quotients halfway between two E4M3 values, small weights, the largest scores and vanishing
scales, and padded slots of a batch."""
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


# ------------------------------------------------------------------ rotary append
def append(x, ds, dev="cuda", **kw):
    """E4M3 (Q, K, V) of the same rows x (tokens, D) divided by ds; D = DV = 64, dims 0 to 15 rotated at position 0."""
    T = x.shape[0]
    p = Problem([T], [T], Hq=1, Hkv=1, D=64, DV=64, ps=16, seed=52)
    rows = x.to(dev)[None, :, None]
    d = torch.as_tensor(ds, dtype=torch.float32).reshape(1, 1).to(dev)
    ko, vo = p.k.to(dev), p.v.to(dev)
    q8 = fa8.rope_append(rows, rows, rows, torch.ones(8, dtype=torch.float64, device=dev), k_out=ko, v_out=vo, descale_q=d,
                         descale_k=d, descale_v=d, positions=torch.zeros((1, T), dtype=torch.int32, device=dev),
                         **p.index_args(dev), **kw)
    ok()
    page, row = p.bt[0].long()[torch.arange(T) // 16], torch.arange(T) % 16
    return val(q8.cpu())[0, :, 0], val(ko.cpu())[page, row, 0], val(vo.cpu())[page, row, 0]


def check_append(x, d, **kw):
    """Q and K are rotated first: by cos 0 = 1 and sin 0 = 0, which leaves what is finite, and makes a NaN of an
    infinity's partner."""
    x, d = x.cpu(), torch.as_tensor(d, dtype=torch.float32)
    turned = ref.rope(x[:, None], torch.zeros(len(x)), torch.ones(8), kw.get("interleaved", False), 0, 1.0)[:, 0]
    for got, y in zip(append(x, d, **kw), (turned, turned, x.double())):
        y = y / d.double()
        want = torch.where(y.isnan(), y, val(e4m3(y.nan_to_num(0.0, 1e9, -1e9))))
        same = (got == want) | (got.isnan() & want.isnan())
        assert same.all(), [(float(x[i]), float(got[i]), float(want[i])) for i in (~same).nonzero()[:4].unbind(1)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quotients_halfway_between_two_values(dtype, inter):
    """x / descale halfway between neighbours of E4M3 goes to the even one, whatever the descale's reciprocal
    rounds to: x = (odd five-bit number) times a three-bit descale, exact in both types."""
    odd = torch.arange(17, 32, 2, dtype=torch.float64)
    t = torch.cat([odd * 2.0 ** e for e in range(-10, 5)] + [torch.arange(1, 16, 2) * 2.0 ** -10])
    t = torch.cat([t, -t])
    t = torch.nn.functional.pad(t, (0, -len(t) % 64)).reshape(-1, 64)
    for d in (3.0, 5.0, 7.0, 3 / 64, 5 / 128, 7 / 32, 7 * 2.0 ** 10):
        x = (t * d).to(dtype)
        assert torch.equal(x.double(), t * d) or dtype is torch.float16  # fp16 has fewer exponents
        check_append(x, d, interleaved=inter)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quotients_are_those_of_fp32_division(dtype):
    g = torch.Generator().manual_seed(53)
    for k in range(20):
        x = (torch.randn((40, 64), generator=g) * 2.0 ** (k - 10)).to(dtype)
        d = torch.rand((), generator=g) * 2.0 ** (k - 10) + 2.0 ** (k - 11)
        check_append(x, d)


@pytest.mark.parametrize("d", [2.0 ** -126, 1.5 * 2.0 ** -126, 2.0 ** -64, 1.0, 1e30, 1.75 * 2.0 ** 126, 3e38])
def test_quotients_at_the_ends_of_the_range(d):
    """Zeros, infinities, NaN and the largest and smallest values by the smallest and largest normal descales."""
    v = [0.0, -0.0, math.inf, -math.inf, math.nan, 3e38, -3e38, 2.0 ** -133, 2.0 ** -126, 1.0, 1e30, 1e10, d, -448.0 * d, 18.0 * d, 1e5 * d]
    if d < 2.0 ** 100:  # halfway between two values
        v += [2.0 ** -10 * d, 3 * 2.0 ** -10 * d, 17.0 * d, -464.0 * d]
    x = torch.zeros((len(v), 64), dtype=torch.bfloat16)
    x[:, 20] = torch.tensor(v, dtype=torch.float64).bfloat16()  # a dim that passes through, in a row of zeros
    check_append(x, d)


# ------------------------------------------------------------------ attention over listed pages
@pytest.mark.parametrize("Hq,D", [(1, 64), (4, 128), (12, 128), (8, 256)])
@pytest.mark.parametrize("tokens", [1, 600])
def test_many_small_weights_add_up(tokens, Hq, D):
    """Keys of weight 2^-x beside one of weight 1 and value 0 in every 32: all that O holds are the small ones.
    P is taken in units of 2^-31 of the maximum or less, so each weight is off by at most 2^-32 (of a sum of
    about n / 32, in n keys of value 448), or by 2^-11 of itself; then O's rounding, and 2^-15 for the fp32 steps
    (an exponent of 30 in 2^-23, twice)."""
    n, ps = 2048, 16
    p = Problem([n + tokens], [tokens], Hq=Hq, Hkv=1, D=D, DV=D, ps=ps, seed=54)
    phys = p.bt[0].long()
    j = torch.arange(n)
    small = j % 32 != 5
    p.q = torch.zeros((1, tokens, Hq, D)).to(E4M3)
    q = val(p.q)
    q[..., 1] = 1.0
    p.q = q.float().to(E4M3)
    lists = torch.arange(n // ps, dtype=torch.int32).expand(1, tokens, 1, n // ps).contiguous().cuda()
    for x in (20.0, 24.0, 28.0, 30.0):
        k, v = torch.zeros(p.k.shape, dtype=torch.float64), torch.zeros(p.v.shape, dtype=torch.float64)
        k[phys[j // ps], j % ps, 0, 1] = torch.where(small, -x, 0.0).double()
        v[phys[j // ps], j % ps, 0] = torch.where(small, 448.0, 0.0).double()[:, None]
        out, lse = fa8.fwd_pages(p.q.cuda(), k.float().to(E4M3).cuda(), v.float().to(E4M3).cuda(), lists,
                                 softmax_scale=math.log(2), **p.index_args())
        ok()
        count = int(small.sum())
        total = (n - count) + count * 2.0 ** -x
        want = count * 2.0 ** -x * 448 / total
        tol = want * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15) + count * 2.0 ** -32 * 448 / total
        assert (out.double().cpu() - want).abs().max() <= tol, (x, out.flatten()[:4], want)
        assert (lse.double().cpu() - math.log(total)).abs().max() <= 2.0 ** -18


@pytest.mark.parametrize("scale", [1.0, 2.0])
@pytest.mark.parametrize("climb", [0.0, 0.125, 1.0])
def test_largest_scores_leave_no_nan(climb, scale):
    """Scores of 448 x 448 over all channels, above 2^24 in log2 units, equal or climbing slowly over the list: V is
    1 everywhere, so O is 1 but for the weights that saturate (by two at most) and bf16's rounding."""
    n, ps = 1000, 16
    p = Problem([n], [1], Hq=2, Hkv=1, D=64, DV=64, ps=ps, seed=55)
    j = torch.arange(n)
    q, k = torch.full((1, 1, 2, 64), 448.0), torch.full(p.k.shape, 448.0)
    q[..., 1] = climb
    k[p.bt[0].long()[j // ps], j % ps, 0, 1] = (j // 40).float().to(E4M3).float()
    v = torch.ones(p.v.shape).to(E4M3)
    lists = torch.arange(-(-n // ps), dtype=torch.int32).reshape(1, 1, 1, -1).cuda()
    out, lse = fa8.fwd_pages(q.to(E4M3).cuda(), k.to(E4M3).cuda(), v.cuda(), lists, softmax_scale=scale, **p.index_args())
    ok()
    assert (out >= 0.5).all() and (out <= 1.0 + 2.0 ** -8).all(), out.flatten()[:4]
    z = (q.to(E4M3).double()[0, 0, 0] * k.to(E4M3).double()[p.bt[0].long()[j // ps], j % ps, 0]).sum(-1) * scale
    assert ((lse.double().cpu() - torch.logsumexp(z, 0)).abs() <= 2.0 ** -21 * z.max()).all()


@pytest.mark.parametrize("scale,descale", [(1e-30, 1e-10), (1e-38, 1e-30), (1e-20, 1.0)])
def test_vanishing_scales_weigh_keys_alike(scale, descale):
    """A scale whose product with the descales is below fp32: every visible key has one weight, and the keys behind
    them have none.  O is V's mean to bf16's rounding, LSE the logarithm of the number of keys."""
    n, ps = 77, 16
    p = Problem([n], [1], Hq=4, Hkv=2, D=64, DV=64, ps=ps, seed=56)
    p.poison()
    lists = torch.arange(-(-n // ps), dtype=torch.int32).expand(1, 1, 2, -1).contiguous().cuda()
    d = torch.tensor(descale).cuda()
    out, lse = fa8.fwd_pages(p.q.cuda(), p.k.cuda(), p.v.cuda(), lists, softmax_scale=scale, descale_q=d, descale_k=d,
                             **p.index_args())
    ok()
    j = torch.arange(n)
    v = val(p.v)[p.bt[0].long()[j // ps], j % ps]
    want, mass = v.mean(0).repeat_interleave(2, 0), v.abs().mean(0).repeat_interleave(2, 0)
    assert ((out.double().cpu()[0, 0] - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * mass).all(), out.flatten()[:4]
    assert ((lse.double().cpu() - math.log(n)).abs() <= 2.0 ** -20).all(), lse


@pytest.mark.parametrize("layout", ["paged", "varlen", "dense"])
def test_padded_slots_append_nothing(layout):
    """Requests without keys, or with fewer than new tokens, in a batch: the other requests' keys are appended, the
    rest of the cache stays, Q is stored for all, and nothing is reported; keys that cu_seqlens_k takes back are."""
    keys = [20, 20, 20] if layout == "dense" else [70, 0, 2]
    Sq = 33 if layout == "dense" else 3
    p = Problem(keys, [Sq] * 3, Hq=2, Hkv=1, D=64, DV=64, ps=16, seed=57)
    x = torch.randn((3, Sq, 2, 64), generator=p.g).bfloat16().cuda()
    w = torch.ones(16, dtype=torch.float64, device="cuda")
    args = p.index_args()
    kw = {"paged": args, "varlen": dict(args, block_table=None, page_size=0), "dense": {}}[layout]
    if layout == "paged":
        ko, vo = p.k.cuda(), p.v.cuda()
    else:
        shape = (3, 20, 1, 64) if layout == "dense" else (72, 1, 64)
        ko, vo = (e4m3(torch.randn(shape, generator=p.g)).cuda() for _ in range(2))
    before = [t.clone().view(torch.uint8) for t in (ko, vo)]

    def run(**change):
        q8 = fa8.rope_append(x, x[:, :, :1], x[:, :, :1], w, k_out=ko, v_out=vo, rotary_offset=16, **dict(kw, **change))
        return q8, fa8.check()

    q8, status = run()
    assert status == fa8.FA8_SUCCESS
    assert torch.equal(val(q8.cpu())[..., :16], val(e4m3(x.cpu()))[..., :16])  # dims that pass through
    written = torch.zeros(before[0].shape[:-2], dtype=torch.bool)
    for b, i, _ in p.tokens():
        j = p.keys[b] - Sq + i
        if j >= 0:
            at = {"paged": lambda: (int(p.bt[b, j // 16]), j % 16), "varlen": lambda: (int(p.cu_k[b]) + j,),
                  "dense": lambda: (b, j)}[layout]()
            written[at] = True
            for out in (ko, vo):
                assert torch.equal(val(out[at].cpu())[0, :16], val(e4m3(x[b, i, 0].cpu()))[:16])
    for out, b in zip((ko, vo), before):
        assert torch.equal(out.view(torch.uint8)[~written.cuda()], b[~written.cuda()])
    if layout != "dense":
        cu = torch.tensor([0, 70, 65, 67], dtype=torch.int32, device="cuda")
        assert run(cu_seqlens_k=cu)[1] == fa8.FA8_ERR_DEVICE_BOUNDS


# ------------------------------------------------------------------ the binding
@pytest.mark.parametrize("python", [False, True])
def test_outputs_that_do_not_fit_raise_as_torch_does(python, monkeypatch):
    """Outputs of petabytes (of an expanded q): torch's OutOfMemoryError, which callers catch to free memory."""
    monkeypatch.setattr(fa8, "_entries", {})
    if python:
        monkeypatch.setattr(fa8, "_args_module", lambda: None)
    q = torch.zeros((1, 1, 8, 128), dtype=torch.uint8, device="cuda").view(E4M3).expand(1 << 20, 1 << 20, 8, 128)
    p = Problem([16], [1], Hq=8, Hkv=8, seed=58)
    k, v = p.k.cuda(), p.v.cuda()
    bnd = torch.zeros((p.k.shape[0], 8, 2, 128), dtype=torch.uint8, device="cuda").view(E4M3)
    pages = torch.zeros((1, 1, 1, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: fa8.select_pages(q, bnd, 64, **p.index_args()), lambda: fa8.fwd_pages(q, k, v, pages, **p.index_args()),
                 lambda: fa8.fwd_pages(q, k, v, pages, out=k, **p.index_args())):
        with pytest.raises(torch.OutOfMemoryError):
            call()
    ok()
