"""Plain 64-bit forms of the paged-cache operators on CPU tensors, written from their
definitions, and a builder of small problems.  Test infrastructure only."""
import math

import torch

E4M3 = torch.float8_e4m3fn


def e4m3(x):
    return x.float().clamp(-448.0, 448.0).to(E4M3)


def val(x):
    """E4M3 -> fp64 (float8 tensors cannot be indexed everywhere: index the result)."""
    return x.to(torch.float64)


class Problem:
    """B requests with new[b] new tokens and keys[b] keys over a shuffled page pool."""

    def __init__(self, keys, new, Hq=8, Hkv=2, D=128, DV=128, ps=16, packed=False, tail=0, extra=3, width=0, seed=0,
                 scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.keys, self.new, self.ps = g, list(keys), list(new), ps
        self.B, self.Hq, self.Hkv, self.D, self.DV, self.G = len(keys), Hq, Hkv, D, DV, Hq // Hkv
        self.packed, self.tail = packed, tail
        if not packed:
            assert len(set(new)) == 1 and tail == 0
        self.T = sum(new)
        shape = (self.T + tail, Hq, D) if packed else (self.B, new[0], Hq, D)
        self.q = e4m3(torch.randn(shape, generator=g) * scale)
        used = [-(-n // ps) for n in keys]
        pool = sum(used) + extra
        perm = torch.randperm(pool, generator=g).to(torch.int32)
        self.bt = torch.full((self.B, max(used + [1, width])), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            self.bt[b, :n] = perm[at:at + n]
            at += n
        self.k = e4m3(torch.randn((pool, ps, Hkv, D), generator=g) * scale)
        self.v = e4m3(torch.randn((pool, ps, Hkv, DV), generator=g) + 0.5)
        self.cu_k = torch.tensor([0] + list(torch.tensor(self.keys).cumsum(0)), dtype=torch.int32)
        self.cu_q = torch.tensor([0] + list(torch.tensor(self.new).cumsum(0)), dtype=torch.int32) if packed else None
        self.dq, self.dk, self.dv = (torch.rand((self.B, Hkv), generator=g) * 1.5 + 0.5 for _ in range(3))

    def tokens(self):
        """(request, index among its new tokens, flat token) of every new token."""
        t = 0
        for b, m in enumerate(self.new):
            for i in range(m):
                yield b, i, t
                t += 1

    def visible(self, b, i, causal=True):
        return max(0, min(self.keys[b], self.keys[b] - self.new[b] + i + 1)) if causal else self.keys[b]

    def flat(self, x):
        """(T, ...) rows of a per-token tensor, without the rows behind the last sequence."""
        return x[:self.T] if self.packed else x.reshape(self.T, *x.shape[2:])

    def poison(self):
        """NaN in every row of the pool that no request owns."""
        own = torch.zeros(self.k.shape[:2], dtype=torch.bool)
        for b, n in enumerate(self.keys):
            j = torch.arange(n)
            own[self.bt[b].long()[j // self.ps], j % self.ps] = True
        for x in (self.k, self.v):
            x.view(torch.uint8)[~own] = 0x7F

    def index_args(self, dev="cuda"):
        return dict(cu_seqlens_k=self.cu_k.to(dev), block_table=self.bt.to(dev), page_size=self.ps,
                    cu_seqlens_q=self.cu_q.to(dev) if self.packed else None)


def bounds(p, only_new=False, into=None):
    """(num_pages, Hkv, 2, D) fp64; pages that hold no key of any request stay as in `into` (0)."""
    out = torch.zeros((p.k.shape[0], p.Hkv, 2, p.D), dtype=torch.float64) if into is None else val(into).clone()
    k = val(p.k)
    for b, n in enumerate(p.keys):
        if only_new and p.new[b] == 0:
            continue
        first = max(0, n - p.new[b]) // p.ps if only_new else 0
        for pi in range(first, -(-n // p.ps)):
            rows = k[int(p.bt[b, pi]), :min(p.ps, n - pi * p.ps)]
            nan = rows.isnan().any(0)
            out[int(p.bt[b, pi]), :, 0] = torch.where(nan, math.nan, rows.nan_to_num(math.inf, math.inf, -math.inf).amin(0))
            out[int(p.bt[b, pi]), :, 1] = torch.where(nan, math.nan, rows.nan_to_num(-math.inf, math.inf, -math.inf).amax(0))
    return out


def select(p, bnd, K, causal=True, keep_first=1, keep_last=1):
    """(T, Hkv, K) page lists; scores are sums of products of E4M3 values, exact in 64 bits."""
    out = torch.full((p.T, p.Hkv, K), -1, dtype=torch.int32)
    q, bnd = val(p.flat(p.q)), val(bnd) if bnd.dtype == E4M3 else bnd
    for b, i, t in p.tokens():
        vis = p.visible(b, i, causal)
        n = -(-vis // p.ps)
        phys = p.bt[b, :n].long()
        for h in range(p.Hkv):
            qq = q[t, h * p.G:(h + 1) * p.G]  # (G, D)
            lo, hi = bnd[phys, h, 0], bnd[phys, h, 1]  # (n, D)
            s = (torch.where(qq < 0, qq, 0.0 * qq) @ lo.T + torch.where(qq < 0, 0.0 * qq, qq) @ hi.T)
            s = torch.where(s.isnan().any(0), math.inf, s.nan_to_num(-math.inf, math.inf, -math.inf).amax(0))
            idx = torch.arange(n)
            force = (idx < keep_first) | (idx >= n - keep_last)
            order = sorted(range(n), key=lambda j: (not bool(force[j]), -float(s[j]), j))
            chosen = sorted(order[:K])
            out[t, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return out


def attend(p, lists, causal=True, sink=None, scale=None, dq=None, dk=None, dv=None):
    """fp64 (T, Hq, DV) output, (T, Hq) LSE, and what error bounds need: (T, Hq) sums of
    p |v| dv per channel's maximum and the largest sum of |q k| in units of the scaled score."""
    scale = 1.0 / math.sqrt(p.D) if scale is None else scale
    q, k, v = val(p.flat(p.q)), val(p.k), val(p.v)
    o = torch.zeros((p.T, p.Hq, p.DV), dtype=torch.float64)
    mass = torch.zeros((p.T, p.Hq, p.DV), dtype=torch.float64)
    lse = torch.full((p.T, p.Hq), -math.inf, dtype=torch.float64)
    reach = torch.zeros((p.T, p.Hq), dtype=torch.float64)
    for b, i, t in p.tokens():
        vis = p.visible(b, i, causal)
        for h in range(p.Hkv):
            js = [pg * p.ps + r for pg in lists[t, h].tolist() if pg >= 0 for r in range(p.ps) if pg * p.ps + r < vis]
            j = torch.tensor(js, dtype=torch.long)
            page = p.bt[b].long()[j // p.ps]
            kk, vv = k[page, j % p.ps, h], v[page, j % p.ps, h]
            f = scale * float(dq[b, h] if dq is not None else 1) * float(dk[b, h] if dk is not None else 1)
            dvv = float(dv[b, h]) if dv is not None else 1.0
            for hq in range(h * p.G, (h + 1) * p.G):
                z = kk @ q[t, hq] * f
                extra = [float(sink[hq])] if sink is not None else []
                allz = torch.cat([z, torch.tensor(extra, dtype=torch.float64)])
                if len(allz) == 0:
                    continue
                e = torch.logsumexp(allz, 0)
                lse[t, hq] = e
                w = torch.exp(z - e)
                o[t, hq] = w @ vv * dvv
                mass[t, hq] = w @ vv.abs() * dvv
                if len(js):
                    reach[t, hq] = (kk.abs() @ q[t, hq].abs() * f).max()
    return o, lse, mass, reach


def rope(x, pos, inv_freq, interleaved, off, scale):
    """fp64 rotation of (T, H, D) rows at positions pos (T)."""
    R = 2 * len(inv_freq)
    i = torch.arange(R // 2)
    a, b = (off + 2 * i, off + 2 * i + 1) if interleaved else (off + i, off + R // 2 + i)
    x = x.double().clone()
    ang = (pos.double()[:, None] * inv_freq.double())[:, None]
    c, s = ang.cos() * scale, ang.sin() * scale
    y0, y1 = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    x[..., a], x[..., b] = y0, y1
    return x
