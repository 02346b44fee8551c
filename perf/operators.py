"""The operators around the FP8 paged cache, measured: filling it (rotary positions, E4M3
rounding, append), summarising it (page bounds), choosing pages of it for each query, and
attention over the chosen pages.

``run`` computes each in a plain form (elementary torch operations, 32 bits, 64 for angles
and page scores), or, where ``own`` is true, through the library's entry points.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
OUT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------ the cases
# Common keys: op; B requests with Sq new tokens each (Sq = 0: packed sequences whose new
# tokens are all their keys); key counts evenly spread over lo..hi (their order follows the
# seed); heads Hq/Hkv; head dims D/DV; page = page size (0: contiguous K/V); dtype of the
# 16-bit side.
def listed():
    gqa = dict(Hq=32, Hkv=8, D=128, DV=128)
    return [
        # one request's decode step: a single token, where latency is all
        dict(gqa, name="rope decode 1x1", op="rope", B=1, Sq=1, lo=4096, hi=4096, page=16, dtype="bf16",
             rot=128, off=0, inter=False, far=0),
        # packed prefill of 16 sequences, 64 rotated dims behind 128 plain ones, pairs side by side
        dict(name="rope varlen d192 part", op="rope", B=16, Sq=0, lo=256, hi=8192, page=0, dtype="fp16", Hq=16,
             Hkv=4, D=192, DV=128, rot=64, off=128, inter=True, far=0),
        # a prefill step into 64-token pages, positions of a long context
        dict(gqa, name="rope prefill 2x4096", op="rope", B=2, Sq=4096, lo=4096, hi=12288, page=64, dtype="bf16",
             rot=128, off=0, inter=False, far=500000),
        # decode: only the page that the new token fell into
        dict(name="bounds step 64x1", op="bounds", B=64, Sq=1, lo=1024, hi=32768, page=16, dtype="bf16", Hq=64,
             Hkv=8, D=128, DV=128),
        # after a long prefill: all pages of the requests
        dict(gqa, name="bounds build 4x32k", op="bounds", B=4, Sq=0, lo=32000, hi=32768, page=64, dtype="bf16"),
        # one long request, one token: few (token, kv-head) pairs, many pages
        dict(name="select 1x1 131072 d256", op="select", B=1, Sq=1, lo=131072, hi=131072, page=64, dtype="bf16",
             Hq=8, Hkv=1, D=256, DV=256, K=64),
        # a ragged decode batch with small pages: the most pages to score
        dict(name="select 64x1 ragged", op="select", B=64, Sq=1, lo=1024, hi=32768, page=16, dtype="bf16", Hq=64,
             Hkv=8, D=128, DV=128, K=128),
        # a chunk of new tokens, each with its own choice
        dict(gqa, name="select chunk 512 of 32k", op="select", B=1, Sq=512, lo=32768, hi=32768, page=64,
             dtype="bf16", K=32),
        # one request's decode step over 2048 chosen keys
        dict(gqa, name="attend 1x1", op="attend", B=1, Sq=1, lo=32768, hi=32768, page=16, dtype="bf16", K=128),
        # the ragged decode batch over 2048 chosen keys each
        dict(name="attend 64x1 ragged", op="attend", B=64, Sq=1, lo=1024, hi=32768, page=16, dtype="bf16", Hq=64,
             Hkv=8, D=128, DV=128, K=128),
        # wide heads, several long requests
        dict(name="attend 8x1 d256", op="attend", B=8, Sq=1, lo=20001, hi=131072, page=64, dtype="fp16", Hq=8,
             Hkv=1, D=256, DV=256, K=64),
        # a chunk of new tokens, each over its own pages
        dict(gqa, name="attend chunk 512 of 32k", op="attend", B=1, Sq=512, lo=32768, hi=32768, page=64,
             dtype="bf16", K=32),
    ]


DIMS = [(64, 64), (96, 96), (128, 128), (128, 128), (192, 128), (192, 192), (256, 256)]
HEADS = [(32, 8), (64, 8), (16, 2), (32, 4), (8, 1), (16, 4), (3, 3), (24, 8), (20, 4), (16, 1)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the ranges above, cut (requests first, then new tokens) to the largest listed one's bytes."""
    c = _any(rng)
    most = 8e8 if c["op"] in ("rope", "bounds") else 2.6e8
    while work(c)["bytes"] > most or work(c)["flops"] > 1.7e10:
        if c["B"] > 1:
            c["B"] //= 2
        elif c["Sq"] > 1:
            c["Sq"] //= 2
        else:
            c["hi"] //= 2
            c["lo"] = min(c["lo"], c["hi"])
    return c


def _any(rng):
    Hq, Hkv = rng.choice(HEADS)
    D, DV = rng.choice(DIMS)
    c = dict(op=rng.choice(["rope", "bounds", "select", "attend"]), Hq=Hq, Hkv=Hkv, D=D, DV=DV,
             page=rng.choice([8, 16, 16, 32, 64, 64, 128]), dtype=rng.choice(["bf16", "fp16"]))
    c["hi"] = _log(rng, 64, 65536)
    c["lo"] = _log(rng, max(1, c["hi"] // 32), c["hi"])
    if c["op"] == "rope":
        packed = rng.random() < 0.3
        c["hi"] = min(c["hi"], 8192)
        c["lo"] = min(c["lo"], c["hi"])
        c["B"] = min(_log(rng, 1, 8 if packed else 128), (1 << 19) // c["hi"])
        c["Sq"] = 0 if packed else rng.choice([1, 1, 2, 4, _log(rng, 1, max(1, min(c["lo"], 16384 // c["B"])))])
        c["Sq"] = min(c["Sq"], c["lo"])
        c["rot"], c["off"] = rng.choice([(D, 0), (D // 2 // 16 * 16, 0), (32, D - 32)])
        c["inter"], c["far"] = rng.random() < 0.5, rng.choice([0, 0, rng.randrange(1, 1 << 20)])
        if packed and rng.random() < 0.5:
            c["page"] = 0
        return c
    c["B"] = min(_log(rng, 1, 128), max(1, (1 << 20) // c["hi"]))
    if c["op"] == "bounds":
        c["Sq"] = min(c["lo"], rng.choice([0, 1, 4, _log(rng, 1, 4096)]))
        return c
    c["Sq"] = min(c["lo"], rng.choice([1, 1, 1, 2, 4, 5, _log(rng, 1, 256)]))
    c["B"] = max(1, min(c["B"], 256 // c["Sq"]))
    c["K"] = min(_log(rng, 2, 512), max(2, 4096 // c["page"]))
    return c


# ------------------------------------------------------------------------------ the inputs
def _lengths(c):
    n = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, n - 1) if n > 1 else c["hi"] for i in range(n)]


def _cu(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(E4M3)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    lens = _lengths(c)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=h).tolist()]
    B, Hq, Hkv, D, DV, ps = (c[k] for k in ("B", "Hq", "Hkv", "D", "DV", "page"))
    new = [c["Sq"] or n for n in lens]
    total = sum(new)
    batched = c["Sq"] > 0
    s = dict(c=c, lens=lens, batched=batched, total=total)
    s["cu_k"] = torch.tensor(_cu(lens), dtype=torch.int32, device=dev)
    s["cu_q"] = None if batched else torch.tensor(_cu(new), dtype=torch.int32, device=dev)
    # for every new token: its request, its key index and how many keys it sees
    s["req"] = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(dev)
    s["key"] = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).to(dev)

    # the pool of pages in a shuffled order, trailing entries of the table unused
    if ps:
        used = [-(-n // ps) for n in lens]
        perm = torch.randperm(sum(used), generator=h).to(torch.int32)
        bt = torch.full((B, max(used)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            bt[b, :n] = perm[at:at + n]
            at += n
        s["bt"], rows, kv = bt.to(dev), (sum(used), ps), "paged"
    else:
        s["bt"], rows, kv = None, (sum(lens),), "packed"
    if c["op"] == "rope":
        dt = OUT[c["dtype"]]
        shape = (B, c["Sq"]) if batched else (total,)
        qkv = randn(*shape, Hq * D + Hkv * (D + DV)).to(dt)  # the projection's output, split into views
        s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = qkv[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        s["v"] = qkv[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, DV))
        s["inv_freq"] = (500000.0 ** -(torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).to(dev)
        s["pos"] = (s["key"] + c["far"]).to(torch.int32).reshape(shape) if c["far"] else None
        for n in "qkv":
            s["d" + n] = (torch.rand((B, Hkv), generator=g, device=dev) * 0.03 + 0.005).float()
        s["k_cache"] = _e4m3(randn(*rows, Hkv, D))
        s["v_cache"] = _e4m3(randn(*rows, Hkv, DV))
        s["slot"] = s["key"] if kv == "paged" else s["cu_k"].long()[s["req"]] + s["key"]
        return s
    s["k_cache"] = _e4m3(randn(*rows, Hkv, D))
    if c["op"] == "bounds":
        # rows that no update touches keep what they hold
        s["bounds"] = torch.zeros((rows[0], Hkv, 2, D), dtype=torch.uint8, device=dev).view(E4M3)
        return s
    shape = (B, c["Sq"], Hq, D)
    s["q"] = _e4m3(randn(*shape))
    if c["op"] == "select":
        kf = s["k_cache"].float()
        s["bounds"] = torch.stack([kf.amin(1), kf.amax(1)], 2).to(E4M3).contiguous()
        s["k_cache"] = None
        return s
    s["v_cache"] = _e4m3(randn(*rows, Hkv, DV) + 0.5)
    for n in "qkv":
        s["d" + n] = (torch.rand((B, Hkv), generator=g, device=dev) * 1.5 + 0.5).float()
    # each (token, kv-head) has its own pages: a random choice, the token's own page always among it
    vis = -(-(s["key"] + 1) // ps)  # pages that hold a visible key
    n = int(vis.max())
    r = torch.rand((total, Hkv, n), generator=g, device=dev)
    idx = torch.arange(n, device=dev)
    r = r.masked_fill(idx >= vis[:, None, None], -1.0).masked_fill(idx == vis[:, None, None] - 1, 2.0)
    k = min(c["K"], n)
    top = r.topk(k, -1)
    pages = top.indices.masked_fill(top.values < 0, n).sort(-1).values
    pages = torch.where(pages < n, pages, -1)
    s["pages"] = torch.nn.functional.pad(pages, (0, c["K"] - k), value=-1).to(torch.int32).reshape(
        B, c["Sq"], Hkv, c["K"]).contiguous()
    return s


# ------------------------------------------------------------------------------ the operators
def run(s):
    return {"rope": _rope, "bounds": _bounds, "select": _select, "attend": _attend}[s["c"]["op"]](s)


def _per_token(s, d):
    """(B, Hkv) descales for every token."""
    return d[s["req"]][:, :, None]


def _rope(s):
    c = s["c"]
    kw = dict(positions=s["pos"], interleaved=c["inter"], rotary_offset=c["off"], descale_q=s["dq"],
              descale_k=s["dk"], descale_v=s["dv"], k_out=s["k_cache"], v_out=s["v_cache"],
              cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"], block_table=s["bt"], page_size=c["page"])
    if own:
        from fp8_attention_forward_gb300 import fa8
        q8 = fa8.rope_append(s["q"], s["k"], s["v"], s["inv_freq"], **kw)
        return q8, s["k_cache"], s["v_cache"]
    R, off, G, T = c["rot"], c["off"], c["Hq"] // c["Hkv"], s["total"]
    pos = s["key"] if s["pos"] is None else s["pos"].reshape(-1)
    ang = pos.double()[:, None] * s["inv_freq"]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def rotate(x):
        x = x.reshape(T, -1, c["D"]).float()
        r = x[..., off:off + R]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :R // 2], r[..., R // 2:])
        y, z = a * cos - b * sin, a * sin + b * cos
        r = torch.stack([y, z], -1).flatten(-2) if c["inter"] else torch.cat([y, z], -1)
        return torch.cat([x[..., :off], r, x[..., off + R:]], -1)

    q8 = _e4m3(rotate(s["q"]) / _per_token(s, s["dq"]).repeat_interleave(G, 1)).view_as(s["q"])
    for x, d, cache in ((rotate(s["k"]), "dk", "k_cache"),
                        (s["v"].reshape(T, c["Hkv"], c["DV"]).float(), "dv", "v_cache")):
        y = _e4m3(x / _per_token(s, s[d])).view(torch.uint8)
        to = s[cache].view(torch.uint8)
        if c["page"]:
            page = s["bt"].long()[s["req"], s["slot"] // c["page"]]
            to[page, s["slot"] % c["page"]] = y
        else:
            to[s["slot"]] = y
    return q8, s["k_cache"], s["v_cache"]


def _touched(s):
    """(request, page) pairs that hold one of the new keys, and the key counts of the requests."""
    ps = s["c"]["page"]
    Lk = (s["cu_k"][1:] - s["cu_k"][:-1]).long()
    new = torch.full_like(Lk, s["c"]["Sq"]) if s["batched"] else Lk
    page = torch.arange(s["bt"].shape[1], device=Lk.device)
    at = (page >= ((Lk - new) // ps)[:, None]) & (page * ps < Lk[:, None])
    return at.nonzero(), Lk


def _bounds(s):
    c = s["c"]
    if own:
        from fp8_attention_forward_gb300 import fa8
        return fa8.page_bounds(s["k_cache"], s["bounds"], cu_seqlens_k=s["cu_k"], block_table=s["bt"],
                               page_size=c["page"], new_tokens=c["Sq"] if s["batched"] else -1)
    at, Lk = _touched(s)
    req, page = at[:, 0], at[:, 1]
    phys = s["bt"].long()[req, page]
    k = s["k_cache"].view(torch.uint8)[phys].view(E4M3).float()
    key = page[:, None] * c["page"] + torch.arange(c["page"], device=k.device)
    out = (key >= Lk[req][:, None])[:, :, None, None]
    lo, hi = k.masked_fill(out, math.inf).amin(1), k.masked_fill(out, -math.inf).amax(1)
    s["bounds"].view(torch.uint8)[phys] = torch.stack([lo, hi], 2).to(E4M3).view(torch.uint8)
    return s["bounds"]


def _select(s):
    c = s["c"]
    B, Sq, Hq, Hkv, D, ps, K = (c[k] for k in ("B", "Sq", "Hq", "Hkv", "D", "page", "K"))
    if own:
        from fp8_attention_forward_gb300 import fa8
        return fa8.select_pages(s["q"], s["bounds"], K, cu_seqlens_k=s["cu_k"], block_table=s["bt"],
                                page_size=ps, causal=True, keep_first=1, keep_last=1)
    # sums of products of E4M3 values are exact in 64 bits, so the order of pages is too
    b = s["bounds"].view(torch.uint8)[s["bt"].long().clamp_min(0)].view(E4M3).double()  # (B, n, Hkv, 2, D)
    n = b.shape[1]
    b = b.permute(0, 2, 3, 4, 1).reshape(B, Hkv, 2 * D, n)
    q = s["q"].double().reshape(B, Sq, Hkv, Hq // Hkv, D).transpose(1, 2)
    q = torch.cat([q.clamp_max(0), q.clamp_min(0)], -1).flatten(2, 3)
    score = (q @ b).view(B, Hkv, Sq, -1, n).amax(3).transpose(1, 2)  # (B, Sq, Hkv, n)
    vis = (-(-(s["key"] + 1) // ps)).view(B, Sq, 1, 1)
    page = torch.arange(n, device=b.device)
    score = score.masked_fill((page < 1) | (page >= vis - 1), math.inf).masked_fill(page >= vis, -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    best = torch.where(best < vis, best, n).sort(-1).values
    best = torch.where(best < n, best, -1)
    return torch.nn.functional.pad(best, (0, K - best.shape[-1]), value=-1).to(torch.int32)


def _attend(s):
    c = s["c"]
    B, Sq, Hq, Hkv, D, DV, ps, K = (c[k] for k in ("B", "Sq", "Hq", "Hkv", "D", "DV", "page", "K"))
    if own:
        from fp8_attention_forward_gb300 import fa8
        return fa8.fwd_pages(s["q"], s["k_cache"], s["v_cache"], s["pages"], descale_q=s["dq"], descale_k=s["dk"],
                             descale_v=s["dv"], cu_seqlens_k=s["cu_k"], block_table=s["bt"], page_size=ps,
                             causal=True, out_dtype=OUT[c["dtype"]])
    T, G = s["total"], Hq // Hkv
    pages = s["pages"].long().view(T, Hkv, K)
    phys = s["bt"].long()[s["req"][:, None, None], pages.clamp_min(0)].clamp_min(0)
    head = torch.arange(Hkv, device=phys.device)[None, :, None, None]
    row = torch.arange(ps, device=phys.device)
    key = pages[..., None] * ps + row
    off = ((pages[..., None] < 0) | (key > s["key"][:, None, None, None])).flatten(2)  # (T, Hkv, n)

    def rows(cache):
        return cache.view(torch.uint8)[phys[..., None], row, head].flatten(2, 3).view(E4M3).float()

    q = s["q"].float().view(T, Hkv, G, D)
    k = rows(s["k_cache"])
    scale = (_per_token(s, s["dq"] * s["dk"]) / math.sqrt(D))[..., None]
    sc = (q @ k.transpose(2, 3) * scale).masked_fill(off[:, :, None], -math.inf)
    del k
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp()
    l = p.sum(-1, keepdim=True)
    v = rows(s["v_cache"]).masked_fill(off[..., None], 0.0)
    o = p @ v / l * _per_token(s, s["dv"])[..., None]
    lse = (m + l.log()).view(B, Sq, Hq).transpose(1, 2)
    return o.view(B, Sq, Hq, DV).to(OUT[c["dtype"]]), lse.contiguous()


# ------------------------------------------------------------------------------ what each needs
def work(case):
    c = case
    lens = _lengths(c)
    B, Hq, Hkv, D, DV, ps = (c[k] for k in ("B", "Hq", "Hkv", "D", "DV", "page"))
    T = sum(c["Sq"] or n for n in lens)
    if c["op"] == "rope":
        each = Hq * D + Hkv * (D + DV)
        return {"bytes": 3 * T * each + 8 * (c["rot"] // 2), "flops": T * (3 * (Hq + Hkv) * c["rot"] + each)}
    if c["op"] == "bounds":
        first = [(n - (c["Sq"] or n)) // ps for n in lens]
        keys = sum(n - f * ps for n, f in zip(lens, first))
        pages = sum(-(-n // ps) - f for n, f in zip(lens, first))
        return {"bytes": Hkv * D * (keys + 2 * pages), "flops": 2 * Hkv * D * keys}
    if c["op"] == "select":
        n = sum(-(-x // ps) for x in lens)
        return {"bytes": n * (Hkv * 2 * D + 4) + T * (Hq * D + 4 * Hkv * c["K"]),
                "flops": c["Sq"] * n * Hq * 4 * D}
    read = sum(min(x, c["Sq"] * c["K"] * ps) for x in lens)  # keys of one kv-head, each once
    seen = c["Sq"] * sum(min(x, c["K"] * ps) for x in lens)
    return {"bytes": Hkv * read * (D + DV) + T * (Hq * (D + 2 * DV + 4) + 4 * Hkv * c["K"]),
            "flops": 2 * seen * Hq * (D + DV)}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """What ``run`` returns before its last rounding, from the definition, request by request."""
    s = prepare(case, seed)
    return {"rope": _exact_rope, "bounds": _exact_bounds, "select": lambda s: None,
            "attend": _exact_attend}[case["op"]](s)


def _requests(s):
    """(request, first new token, new tokens, keys) of each request."""
    at = 0
    for b, n in enumerate(s["lens"]):
        m = s["c"]["Sq"] or n
        yield b, at, m, n
        at += m


def _exact_rope(s):
    c = s["c"]
    R, off, D, DV, Hq, Hkv, ps = (c[k] for k in ("rot", "off", "D", "DV", "Hq", "Hkv", "page"))
    q, k, v = (s[n].double().reshape(s["total"], -1, s[n].shape[-1]) for n in "qkv")
    i = torch.arange(R // 2, device=q.device)
    first, second = (off + 2 * i, off + 2 * i + 1) if c["inter"] else (off + i, off + R // 2 + i)
    caches = {"k": s["k_cache"].double(), "v": s["v_cache"].double()}
    q_out = torch.empty_like(q)
    for b, at, m, n in _requests(s):
        pos = torch.arange(n - m, n, device=q.device).double() + c["far"]
        turn = torch.exp(1j * (pos[:, None] * s["inv_freq"]))[:, None]
        for x, d, name in ((q, s["dq"], "q"), (k, s["dk"], "k"), (v, s["dv"], "v")):
            y = x[at:at + m].clone()
            if name != "v":
                z = torch.complex(y[..., first], y[..., second]) * turn
                y[..., first], y[..., second] = z.real, z.imag
            y /= d[b].double().repeat_interleave(y.shape[1] // Hkv)[:, None]
            y = y.clamp(-448, 448)
            if name == "q":
                q_out[at:at + m] = y
            elif ps:
                j = torch.arange(n - m, n, device=q.device)
                caches[name][s["bt"][b].long()[j // ps], j % ps] = y
            else:
                start = int(s["cu_k"][b])
                caches[name][start + n - m:start + n] = y
    return q_out.view(s["q"].shape), caches["k"], caches["v"]


def _exact_bounds(s):
    ps = s["c"]["page"]
    out = s["bounds"].double()
    for b, _, m, n in _requests(s):
        k = s["k_cache"].view(torch.uint8)[s["bt"][b].long().clamp_min(0)].view(E4M3).double()
        first, last, full = (n - m) // ps, -(-n // ps), n // ps
        phys = s["bt"][b].long()
        if full > first:
            out[phys[first:full], :, 0] = k[first:full].min(1).values
            out[phys[first:full], :, 1] = k[first:full].max(1).values
        if last > full:
            out[phys[full], :, 0] = k[full, :n - full * ps].min(0).values
            out[phys[full], :, 1] = k[full, :n - full * ps].max(0).values
    return out


def _exact_attend(s):
    c = s["c"]
    Sq, Hq, Hkv, D, DV, ps = (c[k] for k in ("Sq", "Hq", "Hkv", "D", "DV", "page"))
    G = Hq // Hkv
    out = torch.zeros((c["B"], Sq, Hq, DV), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    k8, v8 = s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)
    heads = torch.arange(Hkv, device="cuda")[:, None]
    for b, at, m, n in _requests(s):
        f = (s["dq"][b].double() * s["dk"][b].double() / math.sqrt(D))[:, None, None]
        for i in range(m):
            lst = s["pages"][b, i].long()  # (Hkv, K)
            key = (lst[..., None] * ps + torch.arange(ps, device="cuda")).flatten(1)
            seen = (lst[..., None] >= 0).expand(-1, -1, ps).flatten(1) & (key < n - m + i + 1)
            key = key.clamp_min(0)
            page = s["bt"][b].long()[(key // ps).clamp_max(s["bt"].shape[1] - 1)].clamp_min(0)
            kk = k8[page, key % ps, heads].view(E4M3).double()
            vv = v8[page, key % ps, heads].view(E4M3).double()
            qq = s["q"][b, i].double().view(Hkv, G, D)
            z = (torch.einsum("hgd,hnd->hgn", qq, kk) * f).masked_fill(~seen[:, None], -math.inf)
            e = torch.logsumexp(z, -1)
            w = torch.exp(z - e[..., None])
            y = torch.einsum("hgn,hnd->hgd", w, vv.masked_fill(~seen[..., None], 0.0))
            out[b, i] = (y * s["dv"][b].double()[:, None, None]).reshape(Hq, DV)
            lse[b, :, i] = e.reshape(Hq)
    return out, lse
