"""Attention with changed scores and of drafted trees where it can go wrong quietly: rows of a unit that do not exist, windows
at the end of 32 bits, caps far above the scores, NaN values that cost time, slots and tokens past the drafted ones."""
import math

import pytest
import torch

from fp8_attention_forward_gb300 import fa8

import scored_ref as R

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
B16 = HALF[torch.bfloat16]


@pytest.fixture(autouse=True)
def no_errors():
    fa8.check()
    yield
    assert fa8.check() == fa8.FA8_SUCCESS


def slopes_of(n):
    return (2.0 ** (-8.0 * torch.arange(1, n + 1) / n)).float()


def call(p, **kw):
    kw = {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    return fa8.fwd_scored(p.q.cuda(), p.k.cuda(), p.v.cuda(), **p.kw(), **kw)


def same_bits(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


# ------------------------------------------------------------------ rows that do not exist
def leave_in_shared_memory(byte, D, DV):
    """A call whose queries, all of this byte, fill every unit's 128 rows on every SM."""
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    q = torch.full((1, 32 * blocks, 4, D), byte, dtype=torch.uint8, device="cuda").view(R.E4M3)
    k = torch.zeros((1, 64, 1, D), dtype=torch.uint8, device="cuda").view(R.E4M3)
    v = torch.zeros((1, 64, 1, DV), dtype=torch.uint8, device="cuda").view(R.E4M3)
    fa8.fwd_scored(q, k, v)


@pytest.mark.parametrize("G", [3, 5, 12])
@pytest.mark.parametrize("D,DV", [(128, 128), (64, 64), (256, 256)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
def test_equal_bits_whatever_shared_memory_held(G, D, DV, cap, bias):
    """Heads that do not divide a unit's 128 rows leave some without a query: what is made of them changes nothing."""
    for keys, m in (([900, 333], 200), ([5000], 60)):
        p = R.Problem(keys, [m] * len(keys), Hq=2 * G, Hkv=2, D=D, DV=DV, seed=G)
        got = []
        for byte in (0x00, 0x7E, 0xFE, 0x7F):  # zeros, the largest, the smallest, NaN
            leave_in_shared_memory(byte, D, DV)
            got.append(call(p, softcap=cap, slopes=slopes_of(2 * G) if bias else None, causal=True))
        assert all(same_bits(got[0], x) for x in got[1:])


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
def test_a_packed_request_does_not_depend_on_the_next(cap, bias):
    """The last rows of a packed request share a unit with queries of the next one, and those are not its own."""
    p = R.Problem([700, 900], [37, 70], Hq=8, Hkv=2, packed=True, seed=1)
    kw = dict(softcap=cap, slopes=slopes_of(8) if bias else None, causal=True)
    got = []
    for byte in (0x00, 0x7E, 0xFE, 0x7F):
        p.q.view(torch.uint8)[37:] = byte
        out, lse = call(p, **kw)
        got.append((out[:37], lse[:, :37]))
    assert all(same_bits(got[0], x) for x in got[1:])


# ------------------------------------------------------------------ windows at the end of 32 bits
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 31 - 100, 2 ** 30])
@pytest.mark.parametrize("m,packed", [(4, False), (150, False), (150, True)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_window_without_end_and_more_tokens_than_keys(window, m, packed, causal):
    """Positions below zero less such a window pass 32 bits; the tokens see what they see without a window."""
    p = R.Problem([m - 2, 1, 40, 0], [m] * 4, Hq=4, Hkv=1, seed=m, packed=packed)
    for cap, slopes in ((3.0, None), (0.0, slopes_of(4))):
        want = R.attend(p, cap=cap, slopes=slopes, causal=causal, window=window)
        R.check(p, call(p, softcap=cap, slopes=slopes, causal=causal, window_left=window), want, B16)


# ------------------------------------------------------------------ the forward's window
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
@pytest.mark.parametrize("D,m", [(128, 2), (128, 150), (192, 150)])
@pytest.mark.parametrize("layout,packed", [("dense", False), ("paged", False), ("varlen", True)])
def test_the_forward_under_a_window_without_end(window, D, m, layout, packed):
    """fa8_fwd likewise: the same bits as without a window."""
    keys = [max(1, m - 60)] * 3 if layout == "dense" else [max(0, m - 60), 1, 40]
    p = R.Problem(keys, [m] * 3, Hq=4, Hkv=1, D=D, DV=D, layout=layout, packed=packed, seed=m)
    q, k, v, kw = p.q.cuda(), p.k.cuda(), p.v.cuda(), p.kw()
    for causal in (True, False):
        a, b = (fa8.fwd(q, k, v, causal=causal, window_left=w, **kw) for w in (window, -1))
        assert same_bits(a, b)


# ------------------------------------------------------------------ large caps
@pytest.mark.parametrize("cap", [30.0, 128.0, 129.0, 1e3, 1e4, 1e6, 1e8, 1e12, 1e30])
@pytest.mark.parametrize("m", [1, 3, 40, 150])
@pytest.mark.parametrize("scale", [0.0, 1.0, 8.0])
@pytest.mark.parametrize("bias", [False, True])
def test_caps_far_above_the_scores(cap, m, scale, bias):
    """A cap of more than 128 costs a score 2^-20 of itself at the most, whatever the cap is; smaller ones 2^-20 of the cap:
    a reciprocal and an exponential of 2^-22 each, the second weighed by at most a quarter, and six products and sums of
    2^-24 of at most twice the value."""
    p = R.Problem([300, 40], [m] * 2, Hq=4, Hkv=1, D=128, DV=128, seed=3)
    slopes = slopes_of(4) if bias else None
    o, lse, mag, _ = R.attend(p, cap=cap, slopes=slopes, scale=scale, causal=True)
    err = R.attend(p, slopes=slopes, scale=scale, causal=True)[3]
    for b in range(2):
        f = (p.dq[b, 0] * p.dk[b, 0]).double() * (scale or 1.0 / math.sqrt(p.D))
        z = (torch.einsum("ihd,jd->hij", p.q[b].double(), p.kl[b][:, 0].double()) * f).abs().amax(-1)
        err[b] += 2.0 ** -20 * (z.clamp(max=cap) if cap > 128 else cap)
    R.check(p, call(p, softcap=cap, slopes=slopes, softmax_scale=scale, causal=True), (o, lse, mag, err), B16)


@pytest.mark.parametrize("D,DV", [(64, 64), (96, 96), (128, 128), (192, 128), (192, 192), (256, 256)])
@pytest.mark.parametrize("m,Hq", [(1, 6), (70, 6), (70, 8)])
@pytest.mark.parametrize("bias", [False, True])
def test_large_caps_at_every_head_dim(D, DV, m, Hq, bias):
    """With ranges, NaN values, negative descales and trees; the error of a score as above, which stays far under 2^-20 of the cap."""
    p = R.Problem([300, 700], [m] * 2, Hq=Hq, Hkv=2, D=D, DV=DV, seed=D + m, scale=2.0, fill=0x7F)
    p.vl[1].view(torch.uint8)[650, 1, 7] = 0x7F
    p.dq[0, 0] = -2.0
    p.lay_out()
    slopes = slopes_of(Hq) if bias else None
    ranges = torch.tensor([[[3 * i, n - 40 + i] if i % 7 else [n, n] for i in range(m)] for n in p.keys], dtype=torch.int32)
    for kw in (dict(causal=True), dict(ranges=ranges), dict(causal=True, window=90)):
        o, lse, mag, _ = R.attend(p, cap=1000.0, slopes=slopes, **kw)
        err = R.attend(p, slopes=slopes, **kw)[3]
        for b in range(2):
            k = p.kl[b].double().repeat_interleave(p.G, 1)
            f = (p.dq[b] * p.dk[b]).double().repeat_interleave(p.G)[:, None] / math.sqrt(D)
            err[b] += 2.0 ** -20 * torch.einsum("ihd,jhd->hij", p.q[b].double(), k).abs().amax(-1) * f.abs()
        kw["window_left"] = kw.pop("window", -1)
        R.check(p, call(p, softcap=1000.0, slopes=slopes, **kw), (o, lse, mag, err), B16)
    if not bias:
        rows = [R.tree_rows(R.tree(m, b))[0] for b in range(2)]
        masks = torch.stack([R.pack(r, -(-m // 32)) for r in rows])
        got = fa8.fwd_tree(p.q.cuda(), p.k.cuda(), p.v.cuda(), masks.cuda(), softcap=1e6, **p.kw())
        o, lse, mag, _ = R.attend(p, cap=1e6, rows=rows)
        R.check(p, got, (o, lse, mag, err), B16)


# ------------------------------------------------------------------ tiny caps
@pytest.mark.parametrize("m", [1, 40])
def test_a_tiny_cap_under_a_huge_scale(m):
    """scale / cap past fp32: scores of zero stay zero, the others are the cap."""
    p = R.Problem([300, 40], [m] * 2, Hq=4, Hkv=1, D=64, DV=64, seed=3)
    p.q.view(torch.uint8)[:, :, 1] = 0
    R.check(p, call(p, softcap=1e-30, softmax_scale=1e12, causal=True), R.attend(p, cap=1e-30, scale=1e12, causal=True), B16)


# ------------------------------------------------------------------ NaN values that some tokens see
def nan_problem(keys, m, D, DV, seed, at, **kw):
    p = R.Problem([keys], [m], Hq=4, Hkv=1, D=D, DV=DV, seed=seed, **kw)
    for j, c in at:
        p.vl[0].view(torch.uint8)[j, 0, c] = 0x7F if c % 2 else 0xFF
    p.lay_out()
    return p


@pytest.mark.parametrize("D,DV", [(64, 64), (96, 96), (128, 128), (192, 128), (192, 192), (256, 256)])
@pytest.mark.parametrize("m,packed", [(1, False), (4, False), (60, False), (60, True), (300, False)])
def test_nan_values_reach_those_that_see_them(D, DV, m, packed):
    """In one tile and in several, alone and many, in gaps that no token sees, in every 16 channels."""
    n = 2600
    at = [(2, 0), (70, 1), (71, DV - 1), (700, 17), (1300, 33), (2590, 5)] + [(1400 + j, j % DV) for j in range(90)] + [(1900, c) for c in range(DV)]
    p = nan_problem(n, m, D, DV, m, at, packed=packed)
    r = torch.tensor([[(37 * i) % 1500, n - (53 * i) % 1500] if i % 5 else [0, 72 * (i % 2)] for i in range(m)], dtype=torch.int32)
    for kw in (dict(ranges=r if packed else r[None]), dict(ranges=(r + 60) if packed else (r + 60)[None], causal=True), dict(causal=True, window=800)):
        want = R.attend(p, cap=4.0, **kw)
        kw["window_left"] = kw.pop("window", -1)
        R.check(p, call(p, softcap=4.0, **kw), want, B16)
    rows = torch.rand((m, m), generator=p.g) < 0.3
    p.vl[0].view(torch.uint8)[n - m + m // 2, 0, 9] = 0x7F
    p.lay_out()
    words = -(-m // 32)
    masks = R.pack(rows, words) if packed else R.pack(rows, words)[None]
    R.check(p, fa8.fwd_tree(p.q.cuda(), p.k.cuda(), p.v.cuda(), masks.cuda(), **p.kw()), R.attend(p, rows=[rows]), B16)


def time_of(f):
    f()
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return sorted(times)[2]


@pytest.mark.parametrize("m,packed", [(1, False), (4, False), (60, False), (60, True)])
def test_a_nan_value_in_a_long_request_costs_little(m, packed):
    """One NaN among the values of a request whose keys some tokens see and others do not."""
    n, D = 60000, 256
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn((m, 4, D) if packed else (1, m, 4, D), generator=g, device="cuda").to(R.E4M3)
    k, v = (torch.randn((n, 1, D), generator=g, device="cuda").to(R.E4M3) for _ in range(2))
    ranges = torch.tensor([[0, n] if i % 2 else [n // 3, n // 3 + 7] for i in range(m)], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kw = dict(ranges=ranges if packed else ranges[None], cu_seqlens_k=cu_k)
    if packed:
        kw["cu_seqlens_q"] = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    clean = time_of(lambda: fa8.fwd_scored(q, k, v, **kw))
    for j in (n // 3 + 3, n // 2):
        v.view(torch.uint8)[j, 0, 100] = 0x7F
    with_nan = time_of(lambda: fa8.fwd_scored(q, k, v, **kw))
    out = fa8.fwd_scored(q, k, v, **kw)[0].view(m, 4, D)
    assert bool(out[..., 100].isnan().all()) and not bool(out[..., :100].isnan().any()) and not bool(out[..., 101:].isnan().any())
    assert with_nan < 3 * clean + 0.1, f"{clean:.3f} ms, with a NaN {with_nan:.3f} ms"


# ------------------------------------------------------------------ slots past the drafted tokens
@pytest.mark.parametrize("layout", ["paged", "varlen", "dense"])
def test_a_kept_slot_past_the_drafted_tokens_is_reported(layout):
    """Even one that would keep its own."""
    p = R.Problem([40, 40], [4, 4], Hq=2, Hkv=2, D=64, DV=64, layout=layout, seed=3)
    k, v = p.k.cuda(), p.v.cuda()
    kw = {n: x for n, x in p.kw().items() if not n.startswith("descale")}
    kept = torch.tensor([[0, 1, 2, 3], [0, 1, -1, 3]], dtype=torch.int32, device="cuda")
    fa8.keep_tokens(k, v, kept, new_tokens=4, **kw)
    assert fa8.check() == fa8.FA8_SUCCESS
    kept = torch.tensor([[0, 1, 2, 3, -1], [0, 1, -1, 3, 4]], dtype=torch.int32, device="cuda")
    fa8.keep_tokens(k, v, kept, new_tokens=4, **kw)
    assert fa8.check() == fa8.FA8_ERR_DEVICE_BOUNDS
    assert torch.equal(k.view(torch.uint8).cpu(), p.k.view(torch.uint8)) and torch.equal(v.view(torch.uint8).cpu(), p.v.view(torch.uint8))


# ------------------------------------------------------------------ lengths near 2^31
def test_a_length_near_2_31_is_reported():
    """A packed request that claims more tokens than there are, by so much that its blocks of rows pass 32 bits."""
    p = R.Problem([300], [20], Hq=4, Hkv=1, packed=True, seed=2)
    kw = dict(p.kw(), cu_seqlens_q=torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    out = torch.full((20, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    fa8.fwd_scored(p.q.cuda(), p.k.cuda(), p.v.cuda(), out=out, **kw)
    assert fa8.check() == fa8.FA8_ERR_DEVICE_BOUNDS
    assert bool((out == 7.0).all())


# ------------------------------------------------------------------ outputs that do not fit
def test_outputs_that_do_not_fit_raise_torchs_error():
    """Outputs of petabytes (of an expanded q): torch's OutOfMemoryError, which callers catch to free memory."""
    q = torch.zeros((1, 1, 1, 64), dtype=torch.uint8, device="cuda").view(R.E4M3).expand(1 << 20, 1 << 20, 128, 64)
    k = torch.zeros((1, 64, 1, 64), dtype=torch.uint8, device="cuda").view(R.E4M3)
    parents = torch.zeros((1, 1), dtype=torch.int32, device="cuda").expand(1 << 24, 1 << 14)
    for f in (lambda: fa8.fwd_scored(q, k, k), lambda: fa8.fwd_tree(q, k, k, parents), lambda: fa8.tree_masks(parents)):
        with pytest.raises(torch.OutOfMemoryError):
            f()


# ------------------------------------------------------------------ far keys
@pytest.mark.parametrize("m", [1, 4, 60])
@pytest.mark.parametrize("packed", [False, True])
def test_ranges_a_million_keys_before_the_token(m, packed):
    """Only the distances of a range's keys from one another weigh: O is that of the same keys near the token, the LSE less by the
    slope times the positions between."""
    n, small, ps = 1_000_000, 300, 64
    p = R.Problem([small], [m], Hq=4, Hkv=1, D=64, DV=64, ps=ps, packed=packed, seed=5)
    slopes, r = torch.tensor([1.0, 8.0, 0.3, 0.0]), torch.tensor([[100, 230]] * m, dtype=torch.int32)
    r = r if packed else r[None]
    o, lse, mag, err = want = R.attend(p, slopes=slopes, ranges=r)
    kw = p.kw()
    used = -(-small // ps)
    table = torch.full((1, -(-n // ps)), int(p.bt[0, 0]), dtype=torch.int32)  # the pages behind the range are one and the same
    table[0, :used] = p.bt[0, :used]
    kw.update(block_table=table.cuda(), cu_seqlens_k=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    got = fa8.fwd_scored(p.q.cuda(), p.k.cuda(), p.v.cuda(), slopes=slopes.cuda(), ranges=r.cuda(), **kw)
    R.check(p, (got[0], lse), want, B16)
    away = (slopes.double() * (n - small)).view(*([-1, 1] if packed else [1, -1, 1]))
    # a product and a sum of fp32, and the LSE's own rounding
    assert ((got[1].double().cpu() - (lse - away)).abs() <= err + 2.0 ** -20 + away * 2.0 ** -22).all()


@pytest.mark.parametrize("D,DV", [(64, 64), (128, 128), (256, 256)])
@pytest.mark.parametrize("new,keys", [([1, 1, 1], [9000, 130, 4097]), ([1, 5, 200, 0, 16], [5000, 8200, 700, 40, 3001])])
def test_packed_requests_over_longer_keys(D, DV, new, keys):
    """Decode steps, chunks and trees of unequal size in one batch."""
    p = R.Problem(keys, new, Hq=8, Hkv=2, D=D, DV=DV, packed=True, tail=2, seed=D)
    for cap, slopes, kw in ((4.0, None, dict(causal=True)), (0.0, slopes_of(8), dict(causal=True, window=3000))):
        want = R.attend(p, cap=cap, slopes=slopes, **kw)
        R.check(p, call(p, softcap=cap, slopes=slopes, causal=True, window_left=kw.get("window", -1)), want, B16)
    rows = [R.tree_rows(R.tree(m, m))[0] for m in new]
    masks = torch.cat([R.pack(r, 7) for r in rows] + [torch.full((2, 7), -1, dtype=torch.int32)])
    R.check(p, fa8.fwd_tree(p.q.cuda(), p.k.cuda(), p.v.cuda(), masks.cuda(), **p.kw()), R.attend(p, rows=rows), B16)
