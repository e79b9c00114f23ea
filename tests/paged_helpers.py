"""Inputs and comparisons of the tests of the paged key-value cache."""
from __future__ import annotations

import torch

import paged_reference as ref

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
# half a step of each type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BEHIND = 2 ** 31 - 1  # in table entries that must not be read


class Cache:
    """A cache on the GPU and the fp64 values that it holds, on the CPU.

    `layout`: "phtd" is contiguous [P, H, page_size, d]; "pthd" has the heads
    inside the tokens; "kv" has K and V of each page side by side."""

    def __init__(self, pages, heads, page_size, d, kind, layout="phtd", seed=0, spread=0):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.page_size, self.heads, self.d = kind, page_size, heads, d
        shape = (pages, heads, page_size, d)
        self.values, tensors, self.scales = [], [], [None, None]
        for i in range(2):
            x = torch.randn(shape, generator=g, dtype=torch.float64)
            if spread:  # rows of very unlike magnitude
                x = x * 2.0 ** torch.randint(-spread, spread + 1, shape[:3] + (1,), generator=g)
            if kind == "e4m3":
                code = x / x.abs().amax(-1, keepdim=True).clamp(min=1e-300) * 300
                code = code.float().to(torch.float8_e4m3fn)
                e = torch.randint(110, 122, shape[:3], generator=g, dtype=torch.int32)
                if spread:
                    e = e + torch.randint(-spread, spread + 1, shape[:3], generator=g)
                tensors.append(code)
                self.scales[i] = e.to(torch.uint8).cuda()
                self.values.append(code.double() * 2.0 ** (e - 127.0)[..., None])
            else:
                tensors.append(x.to(TYPES[kind]))
                self.values.append(tensors[-1].double())
        if layout == "kv":
            raw = torch.uint8 if kind == "e4m3" else tensors[0].dtype
            both = torch.stack([t.view(raw) for t in tensors], 1).cuda().view(tensors[0].dtype)
            self.k, self.v = both[:, 0], both[:, 1]
        elif layout == "pthd":
            self.k, self.v = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
                              for t in tensors)
        else:
            self.k, self.v = (t.cuda() for t in tensors)
        self.k_values, self.v_values = self.values

    @property
    def scale_args(self):
        return {"k_scale": self.scales[0], "v_scale": self.scales[1]}

    def held(self):
        """The fp64 values that the GPU's tensors hold now."""
        out = []
        for t, s in zip((self.k, self.v), self.scales):
            x = t.contiguous().cpu().double()
            if s is not None:
                e = s.cpu().double()
                x = x * torch.where(e == 255, torch.nan, 2.0 ** (e - 127.0))[..., None]
            out.append(x)
        return out


def make_table(lens, page_size, pages, seed=0, width=None, behind=BEHIND):
    """A table of distinct pages in a shuffled order; entries behind a sequence are `behind`."""
    g = torch.Generator().manual_seed(seed + 77)
    counts = [-(-n // page_size) for n in lens]
    assert sum(counts) <= pages
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width or max(1, max(counts))), behind, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table


def pages_for(lens, page_size, spare=3):
    return sum(-(-n // page_size) for n in lens) + spare


def check_attention(o, lse, want_o, want_lse, magnitude, what="", kind=""):
    """o against the 64-bit result: half a step of its type for the rounding, and 2^-12 of
    sum_j p_j |v_j| for the weights.  A score is a sum of d <= 128 products in fp32, off by at
    most d 2^-24 of the sum of their magnitudes: for inputs near N(0, 1) and scale 1/sqrt(d)
    that sum is below 12, so a weight and the total are each off by less than 128 * 2^-24 * 12
    = 9.2e-5, together 1.9e-4 < 2^-12 = 2.4e-4.  The LSE: the same 9.2e-5, and 2^-21 of its
    value for the logarithm.  With an e4m3 cache and bf16 queries each weight is also rounded
    to fp16, by at most half a step, 2^-11 of the weight: 2^-11 of sum_j p_j |v_j| more."""
    half = HALF[o.dtype]
    weight = 2.0 ** -12
    if kind == "e4m3" and o.dtype is torch.bfloat16:
        weight += 2.0 ** -11
    o, lse = o.cpu().double(), lse.cpu().double()
    assert torch.equal(torch.isnan(o), torch.isnan(want_o)), what
    assert torch.equal(torch.isnan(lse), torch.isnan(want_lse)), what
    inf = torch.isinf(want_o)
    assert torch.equal(o[inf], want_o[inf]), what
    fine = torch.isfinite(want_o)
    least = 2.0 ** -25 if half == HALF[torch.float16] else 0.0  # half of fp16's least step
    off = (o - want_o).abs()[fine]
    allowed = (half * want_o.abs() + weight * magnitude + least)[fine] + 1e-30
    worst = (off / allowed).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: o off by {worst:.3g} of what rounding allows"
    inf = torch.isinf(want_lse)
    assert torch.equal(lse[inf], want_lse[inf]), what
    fine = torch.isfinite(want_lse)
    off = ((lse - want_lse).abs() - 2.0 ** -21 * want_lse.abs())[fine]
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 1e-4, f"{what}: lse off by {worst:.3g}"


def queries(B, Hq, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 5)
    return torch.randn((B, Hq, d), generator=g).to(TYPES[dtype])


__all__ = ["Cache", "make_table", "pages_for", "check_attention", "queries", "ref", "TYPES"]
