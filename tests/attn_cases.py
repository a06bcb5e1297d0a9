"""Inputs and 64-bit references of the tests of gdn_attn.h.

Every slot of a cache that no token of a call lies in holds NaN, so a kernel
that lets one in is seen.  Page tables are in no order and padded with -1.
"""
import math

import torch

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = 2.0 ** -8  # half a step of bf16, relative to the value


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Paged:
    """Sequences of `counts` tokens in a cache: k and v hold what the cache stands for, [B][tokens][H][d] as lists."""

    def __init__(self, counts, H, d, page=16, dtype=BF16, seed=0, layout="rows", spare=3, extra_pages=0):
        gen, cpu = generator(seed), torch.Generator().manual_seed(seed)
        pages = [-(-n // page) for n in counts]
        pool = sum(pages) + spare
        perm = torch.randperm(pool, generator=cpu).to(torch.int32)
        width = max(max(pages, default=0), 1) + extra_pages
        table = torch.full((len(counts), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table, self.counts, self.page = table.cuda(), list(counts), page
        shape = {"rows": (pool, page, H, d), "heads": (pool, H, page, d), "wide": (pool, page, H, 2 * d),
                 "both": (pool, 2, page, H, d)}[layout]
        nan = torch.full(shape, float("nan"), device="cuda").to(dtype)
        if layout == "both":
            self.k, self.v = nan[:, 0], nan[:, 1]
        else:
            self.k, self.v = nan, nan.clone()
            if layout == "heads":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
            elif layout == "wide":
                self.k, self.v = self.k[..., d:], self.v[..., :d]
        self.k_scale = self.v_scale = None
        if dtype == E4M3:
            self.k_scale, self.v_scale = (x * torch.linspace(0.7, 1.3, H, device="cuda") for x in (0.02, 0.04))
        self.real = {"k": [], "v": []}
        for b, n in enumerate(counts):
            for name, pool_t, scale in (("k", self.k, self.k_scale), ("v", self.v, self.v_scale)):
                x = randn(gen, n, H, d)
                x = x.to(BF16) if dtype == BF16 else (x / scale[:, None]).to(E4M3)
                self.put(pool_t, b, torch.arange(n), x)
                self.real[name].append(x.double() if scale is None else x.double() * scale.double()[:, None])

    def slots(self, b, tokens):
        tokens = tokens.cuda()
        return self.table[b][tokens // self.page].long() * self.page + tokens % self.page

    def put(self, pool, b, tokens, x):
        slot = self.slots(b, tokens)
        raw = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
        raw[slot // self.page, slot % self.page] = x.view(torch.uint8) if x.dtype == E4M3 else x

    def get(self, pool, b, tokens):
        slot = self.slots(b, tokens)
        raw = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
        return raw[slot // self.page, slot % self.page].view(pool.dtype)

    def cache(self):
        import gated_deltanet_tree_gdn_amd as gdn
        return gdn.GdnKvCache(self.k, self.v, self.k_scale, self.v_scale)


def attend(q, k, v, mask, scale, gate=None):
    """(o, average of |v| under the weights, largest sum of |q k| scale of a visible pair) in 64 bits: q [n][H_q][d],
    k and v [keys][H_kv][d], mask [n][keys].  Rows that see nothing are zero."""
    n, H_q, d = q.shape
    group = H_q // k.shape[1]
    o, avg = (torch.zeros(n, H_q, d, dtype=torch.double, device=q.device) for _ in range(2))
    largest = torch.zeros(n, H_q, 1, dtype=torch.double, device=q.device)
    if k.shape[0]:
        some = mask.any(1)
        for h in range(H_q):
            kh, vh = k[:, h // group], v[:, h // group]
            s = (q[:, h].double() @ kh.t().contiguous() * scale).masked_fill(~mask, -math.inf)
            w = torch.softmax(s[some], 1)
            o[some, h], avg[some, h] = w @ vh, w @ vh.abs()
            both = (q[:, h].double().abs() @ kh.abs().t().contiguous() * scale).masked_fill(~mask, 0.0)
            largest[:, h, 0] = both.amax(1)
    if gate is not None:
        g = torch.sigmoid(gate.double())
        o, avg = o * g, avg * g
    return o, avg, largest


def tolerance(o, avg, largest, d, weights):
    """What a bf16 output may be off by.  Its rounding: half a step.  `weights`: what a weight may be off by when it is
    rounded for the product (bf16: half a step; two bf16: half a step of each, so its square), which moves the
    average by that much of |v| at most.  fp32: a score is a sum of d products (d 2^-24 of the sum of their
    magnitudes), its factor and difference to the maximum are three more roundings, and the powers, their sum and the
    gate some 64 units more; the sum of the weights is off as the weights are, hence twice."""
    rel = weights + 2.0 ** -24 * (2 * (d + 3) * largest + 64)
    return (HALF * o.abs() + rel * avg) * 1.01 + 1e-30


def close(got, o, tol, what=""):
    assert not got.isnan().any(), f"{what}: NaN"
    far = ((got.double() - o).abs() - tol).max().item() if got.numel() else 0.0
    worst = ((got.double() - o).abs() / tol).max().item() if got.numel() else 0.0
    assert far <= 0, f"{what}: {worst:.2f} times the tolerance"
    return worst


def ancestors(parent):
    """Bits [N][ceil(N / 32)] int32 and the mask [N][N] of a tree."""
    N = len(parent)
    mask = torch.zeros(N, N, dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            mask[i] = mask[p]
        mask[i, i] = True
    return bits_of(mask), mask


def bits_of(mask):
    N = mask.shape[0]
    W = max((N + 31) // 32, 1)
    padded = torch.zeros(N, 32 * W, dtype=torch.int64)
    padded[:, :N] = mask
    words = (padded.view(N, W, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def random_tree(N, seed):
    g = torch.Generator().manual_seed(seed)
    return [-1] + [int(torch.randint(-1, i, (1,), generator=g)) for i in range(1, N)]
