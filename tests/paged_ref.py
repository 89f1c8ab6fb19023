"""The paged-cache operators in 64 bits, from their definitions, on the CPU: what the GPU tests
compare with, and the builders of their inputs.

A cache is built from dense per-request keys and values: ``PagedCase`` places them in randomly
ordered pages of a pool whose every other element is NaN, so that a kernel that reads a position
it should not shows it.
"""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def local_len(seq: int, shard: int, num_shards: int, interleave: int) -> int:
    """Positions p < seq with (p // interleave) % num_shards == shard, by counting."""
    return sum(1 for p in range(max(0, seq)) if (p // interleave) % num_shards == shard)


def owned(seq: int, shard: int, num_shards: int, interleave: int) -> list[int]:
    return [p for p in range(max(0, seq)) if (p // interleave) % num_shards == shard]


@dataclasses.dataclass
class PagedCase:
    """A pool with the local positions of requests of the given lengths.

    layout: "slots" [pages, page, heads, D]; "heads" [pages, heads, page, D] permuted;
    "mixed" one [pages, 2, page, heads, D + pad] pool for keys and values (strided rows)."""
    lens: list[int]
    heads: int
    D: int
    page: int
    dtype: str = "bf16"
    layout: str = "slots"
    width: int | None = None
    seed: int = 0
    spare: int = 3
    std: float = 1.0

    def __post_init__(self):
        g = torch.Generator().manual_seed(self.seed)
        dt = DTYPES[self.dtype]
        B, page = len(self.lens), self.page
        used = [-(-max(0, n) // page) for n in self.lens]
        self.width = self.width if self.width is not None else max(1, max(used, default=1))
        used = [min(u, self.width) for u in used]
        pages = sum(used) + self.spare
        order = torch.randperm(pages, generator=g)
        nan = float("nan")
        if self.layout == "slots":
            k = torch.full((pages, page, self.heads, self.D), nan, dtype=dt)
            v = torch.full_like(k, nan)
        elif self.layout == "heads":
            k = torch.full((pages, self.heads, page, self.D), nan, dtype=dt).permute(0, 2, 1, 3)
            v = torch.full((pages, self.heads, page, self.D), nan, dtype=dt).permute(0, 2, 1, 3)
        else:
            pad = 16 // torch.empty(0, dtype=dt).element_size()
            pool = torch.full((pages, 2, page, self.heads, self.D + pad), nan, dtype=dt)
            k, v = pool[:, 0, :, :, :self.D], pool[:, 1, :, :, :self.D]
        # entries past a request's length name no page
        table = torch.full((B, self.width), 2 ** 30, dtype=torch.int32)
        self.keys, self.values = [], []
        at = 0
        for b, n in enumerate(self.lens):
            n = min(max(0, n), self.width * page)
            kk = torch.randn(n, self.heads, self.D, generator=g).mul_(self.std).to(dt)
            vv = torch.randn(n, self.heads, self.D, generator=g).to(dt)
            for j in range(used[b]):
                table[b, j] = order[at + j]
                part = slice(j * page, min(n, (j + 1) * page))
                m = part.stop - part.start
                k[order[at + j], :m] = kk[part]
                v[order[at + j], :m] = vv[part]
            at += used[b]
            self.keys.append(kk)
            self.values.append(vv)
        self.k, self.v, self.table, self.pages = k, v, table, pages

    def gpu(self):
        """(k, v, table) on the device with the same strides."""
        if self.layout == "mixed":
            pool = self.k._base.cuda()
            return pool[:, 0, :, :, :self.D], pool[:, 1, :, :, :self.D], self.table.cuda()
        if self.layout == "heads":
            return (self.k.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3),
                    self.v.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3), self.table.cuda())
        return self.k.cuda(), self.v.cuda(), self.table.cuda()


def attention(q: torch.Tensor, keys, values, scale: float, held=None):
    """Per request b: softmax attention of q[b] over keys[b], values[b] [n, heads, D] in 64 bits.
    held[b]: positions that count (default all).  Returns (out, lse, logits list, spread) where
    spread[b, h] = sum p |v| / sum p per element and xabs[b][h] = scale * sum |q k| per position."""
    B, H, D = q.shape
    out, lse = np.zeros((B, H, D)), np.full((B, H), -np.inf)
    spread, logits, xabs = np.zeros((B, H, D)), [], []
    for b in range(B):
        kk, vv = keys[b].double().numpy(), values[b].double().numpy()
        n, heads = kk.shape[0], kk.shape[1]
        G = H // heads
        lo, la = np.full((H, n), -np.inf), np.zeros((H, n))
        keep = np.arange(n) if held is None else np.asarray(held[b], dtype=np.int64)
        for h in range(H):
            qq = q[b, h].double().numpy()
            x = scale * (kk[keep, h // G] @ qq)
            la[h, keep] = abs(scale) * (np.abs(kk[keep, h // G]) @ np.abs(qq))
            lo[h, keep] = x
            if len(keep):
                m = x.max()
                p = np.exp(x - m)
                out[b, h] = p @ vv[keep, h // G] / p.sum()
                spread[b, h] = p @ np.abs(vv[keep, h // G]) / p.sum()
                lse[b, h] = np.log(p.sum()) + m
        logits.append(lo)
        xabs.append(la)
    return out, lse, logits, spread, xabs


# Rounding of a carried probability: two bf16 parts 2^-8 * 2^-8, two fp16 parts 2^-11 * 2^-11
# (counted as 2^-20), fp32 products as tf32 parts whose dropped terms are below 2^-20.
PART = {"bf16": 2.0 ** -16, "fp16": 2.0 ** -20, "fp32": 2.0 ** -20}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}


def logit_bound(xabs: np.ndarray, D: int, dtype: str) -> np.ndarray:
    """|error| of a logit: D products of 16-bit values are exact in fp32 and their sums lose at
    most 2^-23 of the running absolute sum per addition (the scale: two more roundings); fp32
    operands add PART per product."""
    return xabs * ((D + 2) * 2.0 ** -23 + (PART["fp32"] if dtype == "fp32" else 0.0)) + 2.0 ** -120


def assert_attention(out, lse, ref, n_max: int, dtype: str, base_e: bool = True, what: str = "") -> None:
    """out [B, H, D], lse [B, H] (tensors) against attention()'s values within the bound that
    follows from the arithmetic:
      - a logit error e changes p by a factor exp(+-e), the ratio of sums by at most 2 e spread;
      - exp itself and its argument's rounding: 2^-21 + 2^-23 * |x - m| (|x - m| < 128 counts);
      - p in two parts (PART), sums of n terms in fp32: (n + 64) 2^-23;
      - one rounding of the result (HALF) or a subnormal step (TINY)."""
    o_ref, l_ref, _, spread, xabs = ref
    D = out.shape[2]
    got = out.detach().cpu().double().numpy()
    gl = lse.detach().cpu().double().numpy()
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    e = np.array([[float(logit_bound(x[h], D, dtype).max(initial=0.0)) for h in range(x.shape[0])] for x in xabs])
    rel = 2 * (e + 2.0 ** -21 + 128 * 2.0 ** -23 + (n_max + 64) * 2.0 ** -23 + PART[dtype])
    bound = rel[:, :, None] * spread + HALF[dtype] * np.abs(o_ref) * (1 + 2.0 ** -6) + TINY[dtype]
    err = np.abs(got - o_ref)
    assert (err <= bound).all(), f"{what}: {(err > bound).sum()} outputs beyond the bound, worst ratio " \
                                 f"{(err / np.maximum(bound, 1e-300)).max():.3g}"
    l_ref = l_ref if base_e else l_ref / math.log(2.0)
    empty = np.isinf(l_ref)
    assert np.array_equal(gl[empty], l_ref[empty]), f"{what}: the LSE of an empty row is -inf"
    lb = (e + (n_max + 64) * 2.0 ** -23 + 2.0 ** -20) * (1 if base_e else 1 / math.log(2.0))
    lb = lb + 4 * 2.0 ** -23 * np.abs(np.where(empty, 0, l_ref)) + 2 * 2.0 ** -23 * np.array(
        [[float(x[h].max(initial=0.0)) for h in range(x.shape[0])] for x in xabs])
    err = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, l_ref))
    assert np.isfinite(gl[~empty]).all() and (err <= lb).all(), f"{what}: LSE off by {err.max():.3g}"


def weights(logits: np.ndarray, lse: np.ndarray, w: np.ndarray, lens, base_e: bool) -> np.ndarray:
    """w [B, heads, cap] plus the group sums of exp(logits - lse) at p < lens[b], in 64 bits."""
    B, H, _ = logits.shape
    heads = w.shape[1]
    nat = lse.astype(np.float64) * (1.0 if base_e else math.log(2.0))
    out = w.astype(np.float64).copy()
    for b in range(B):
        for h in range(H):
            if np.isfinite(nat[b, h]):
                n = lens[b]
                out[b, h // (H // heads), :n] += np.exp(logits[b, h, :n].astype(np.float64) - nat[b, h])
    return out


def select(w: np.ndarray, keep: int, recent: int) -> list[int]:
    """The kept positions of one request and key head with weights w [n], increasing."""
    n = len(w)
    if n <= keep:
        return list(range(n))
    rank = [-math.inf if math.isnan(x) else float(x) for x in w]
    # NaN below -inf: a second sort key
    order = sorted(range(n - recent), key=lambda p: (-rank[p], math.isnan(w[p]), p))
    return sorted(order[:keep - recent]) + list(range(n - recent, n))
