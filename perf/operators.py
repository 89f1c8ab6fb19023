"""The paged-cache operators of decode context parallelism, as they are measured.

Four operators work on one rank's shard of a paged key-value cache:

  attend   attention of one new token per request over the shard, with its LSE, as [B, H, D] +
           [B, H] or written straight into the packed send buffer (``pack`` ranks); on request
           (``logits``) the scaled logits too
  append   the rows of new tokens written into the pages of the shard that owns their positions
  weigh    each cached position's accumulated attention weight, from the logits and the LSE over
           all shards
  evict    the ``keep`` positions of largest accumulated weight (the last ``recent`` ones always
           among them) moved into new pages

``own`` is False: ``run`` computes the plain form with elementary torch operations in 32 bits;
True: ``run`` makes the library's calls.  Request lengths are a function of the case alone, all
other inputs of the seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- cases -----------------------------------------------------------------------------------
def _attend(B, H, Hkv, D, page, lo, hi, dtype="bf16", pack=0, logits=False, shards=1, interleave=1, base_e=True):
    return dict(op="attend", dtype=dtype, B=B, H=H, Hkv=Hkv, D=D, page=page, lo=lo, hi=hi, pack=pack, logits=logits,
                shards=shards, interleave=interleave, base_e=base_e)


def _append(R, q, Hkv, D, page, lo, hi, dtype="bf16", shards=1, interleave=1):
    return dict(op="append", dtype=dtype, R=R, q=q, Hkv=Hkv, D=D, page=page, lo=lo, hi=hi, shards=shards,
                interleave=interleave)


def _weigh(B, H, Hkv, lo, hi, shards=1, interleave=1, base_e=True):
    return dict(op="weigh", B=B, H=H, Hkv=Hkv, lo=lo, hi=hi, shards=shards, interleave=interleave, base_e=base_e)


def _evict(B, Hkv, D, page, lo, hi, keep, recent, dtype="bf16"):
    return dict(op="evict", dtype=dtype, B=B, Hkv=Hkv, D=D, page=page, lo=lo, hi=hi, keep=keep, recent=recent)


def listed():
    return [
        # one user's chat turn on one rank: launch latency and the join over a short cache
        dict(_attend(1, 32, 8, 128, 16, 777, 777), name="attend_one_short"),
        # a full decode batch of mixed lengths (empty to 8192 positions), small pages
        dict(_attend(64, 64, 8, 128, 16, 0, 8192), name="attend_ragged"),
        # few users with long documents: the cache's length is split over the whole GPU
        dict(_attend(3, 64, 4, 128, 64, 100000, 131072, dtype="fp16"), name="attend_long"),
        # the largest batch: the bandwidth of the cache alone
        dict(_attend(128, 128, 8, 128, 32, 2048, 8192), name="attend_large"),
        # fp32 cache with an odd page and small heads, base-2 LSE
        dict(_attend(24, 12, 4, 64, 24, 1, 3001, dtype="fp32", base_e=False), name="attend_fp32"),
        # one of 4 ranks of a GQA group: interleaved shard, logits kept for the weights, output
        # written as the packed send buffer of the exchange
        dict(_attend(32, 32, 8, 128, 16, 500, 20000, pack=4, logits=True, shards=4, interleave=16),
             name="attend_pack_logits"),
        # every request of a decode batch appends its token
        dict(_append(256, 1, 8, 128, 16, 1, 1024), name="append_decode"),
        # prompts of a few thousand tokens written to one of 2 ranks
        dict(_append(6, 2731, 8, 128, 16, 2731, 9000, shards=2), name="append_prompt"),
        # a small batch after one step
        dict(_weigh(4, 32, 8, 1, 1500), name="weigh_small"),
        # a full batch after one step, base-2 LSE
        dict(_weigh(64, 64, 8, 2048, 8192, base_e=False), name="weigh_batch"),
        # a few requests reach their budget
        dict(_evict(3, 8, 128, 16, 300, 2000, keep=512, recent=64), name="evict_small"),
        # long contexts cut to an eighth
        dict(_evict(32, 8, 128, 16, 20000, 32768, keep=4096, recent=256), name="evict_long"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for k in ("bytes", "flops"):
            most[c["op"], k] = max(most.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(["attend", "attend", "attend", "append", "weigh", "evict"])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 3, 4, 6, 8, 16])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        page = rng.choice([8, 16, 16, 24, 32, 64, 128])
        shards = rng.choice([1, 1, 2, 4, 8])
        interleave = rng.choice([1, 16, 64]) if shards > 1 else 1
        B = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, 131072)
        lo = rng.choice([0, 1, hi // 3, hi])
        if op == "attend":
            H = Hkv * G
            pack = rng.choice([0] + [n for n in (2, 4, 8) if H % n == 0])
            c = _attend(B, H, Hkv, D, page, lo, hi * shards, dtype, pack, rng.random() < 0.3, shards, interleave,
                        rng.random() < 0.7)
        elif op == "append":
            q = _log_int(rng, 1, 4096)
            c = _append(B, q, Hkv, D, page, q, max(q, min(16384, hi)), dtype, shards, interleave)
        elif op == "weigh":
            c = _weigh(B, Hkv * G, Hkv, lo, hi * shards, shards, interleave, rng.random() < 0.7)
        else:
            keep = _log_int(rng, 8, max(8, hi // 2))
            c = _evict(B, Hkv, D, page, lo, hi, keep, rng.choice([0, keep // 8, keep // 2]), dtype)
        w = work(c)
        cap = B * Hkv * hi * (D if op in ("attend", "evict") else G)  # what the plain form lays out
        if all(w[k] <= most[op, k] for k in w) and cap <= 1 << 30 and max(_lens(c)) > 0:
            return c


def _lens(case):
    """The requests' lengths over all shards: a function of the case alone."""
    n = case["R"] if case["op"] == "append" else case["B"]
    rng = random.Random(n * 1000003 + case["hi"])
    return [rng.randint(case["lo"], case["hi"]) for _ in range(n)]


def _local(length, case, shard=0):
    """Positions of a request of `length` that shard `shard` holds (blocks dealt round-robin)."""
    n, s = case.get("shards", 1), case.get("interleave", 1)
    full, rest = divmod(length, n * s)
    return full * s + max(0, min(s, rest - shard * s))


def work(case):
    op = case["op"]
    if op == "weigh":
        n = sum(_local(x, case) for x in _lens(case))
        return {"bytes": n * (case["H"] + 2 * case["Hkv"]) * 4 + 4 * case["B"] * case["H"], "flops": 3 * n * case["H"]}
    row = case["Hkv"] * case["D"] * _ES[case["dtype"]]
    if op == "attend":
        n = sum(_local(x, case) for x in _lens(case))
        q = case["B"] * case["H"] * case["D"] * _ES[case["dtype"]]
        return {"bytes": 2 * n * row + 2 * q + 4 * case["B"] * case["H"] + (4 * n * case["H"] if case["logits"] else 0),
                "flops": 4 * n * case["H"] * case["D"]}
    if op == "append":
        n = sum(_local(x, case) - _local(x - case["q"], case) for x in _lens(case))
        return {"bytes": 4 * n * row, "flops": 0}
    kept = sum(min(x, case["keep"]) for x in _lens(case))
    # weights read and rewritten, kept indices written, kept rows of K and V read and written
    return {"bytes": case["Hkv"] * (8 * sum(_lens(case)) + 4 * case["B"] * case["keep"]) + 4 * kept * row, "flops": 0}


# ---- inputs ----------------------------------------------------------------------------------
def _paged(need, page, gen, width):
    """Block table [n, width] of int32 page numbers (pages in random order, 0 where unused) and
    the pool's page count; the pool's last page is in no table."""
    used = [-(-x // page) for x in need]
    total = max(1, sum(used))
    order = torch.randperm(total, generator=gen, dtype=torch.int64)
    table, at = torch.zeros(len(need), width, dtype=torch.int32), 0
    for r, u in enumerate(used):
        table[r, :u] = order[at:at + u].to(torch.int32)
        at += u
    return table.cuda(), total + 1


def prepare(case, seed):
    op = case["op"]
    gen, cpu = torch.Generator("cuda").manual_seed(seed), torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, dtype=None):
        return torch.empty(shape, dtype=dtype or torch.float32, device="cuda").normal_(0.0, std, generator=gen)

    lens = _lens(case)
    s = {"case": case, "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    local = [_local(x, case) for x in lens]
    if op == "weigh":
        B, H, Hkv, cap = case["B"], case["H"], case["Hkv"], max(1, max(local))
        s["logits"] = normal(B, H, cap, std=2.0)
        # the LSE of all shards: that of about `length` logits of this spread
        tot = torch.tensor(lens, dtype=torch.float32, device="cuda").clamp(min=1)
        s["lse"] = (tot.log() + 2.0)[:, None] + 0.1 * normal(B, H)
        if not case["base_e"]:
            s["lse"] = s["lse"] * (1.0 / math.log(2.0))
        s["weights"] = normal(B, Hkv, cap, std=0.01).abs_()
        return s
    dt, Hkv, D, page = _DTYPES[case["dtype"]], case["Hkv"], case["D"], case["page"]
    table, pages = _paged(local, page, cpu, max(1, -(-max(local) // page)))
    s["table"] = table
    # one pool per tensor, [pages, page, heads, D]
    s["k"] = normal(pages, page, Hkv, D, dtype=dt)
    s["v"] = normal(pages, page, Hkv, D, dtype=dt)
    if op == "attend":
        # logits of standard deviation 2.5: attention that prefers some positions
        s["q"] = normal(case["B"], case["H"], D, std=2.5, dtype=dt)
        if case["logits"]:
            s["logits"] = torch.zeros(case["B"], case["H"], max(1, max(local)), device="cuda")
    elif op == "append":
        T = case["R"] * case["q"]
        s["k_new"], s["v_new"] = normal(T, Hkv, D, dtype=dt), normal(T, Hkv, D, dtype=dt)
        s["starts"] = torch.arange(0, T + 1, case["q"], dtype=torch.int32, device="cuda")
    else:
        B, cap, keep = case["B"], max(1, max(lens)), case["keep"]
        # accumulated weights spread over some decades, as many steps leave them
        s["weights"] = normal(B, Hkv, cap, std=1.5).exp_().mul_(1e-3)
        kept = [min(x, keep) for x in lens]
        s["new_table"], new_pages = _paged(kept, page, cpu, max(1, -(-keep // page)))
        s["k_out"] = torch.zeros(new_pages, page, Hkv, D, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    return s


# ---- one pass --------------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import decode_context_attention_dcp_b200 as dcp
    c = s["case"]
    if c["op"] == "weigh":
        dcp.dcp_kv_weights(s["logits"], s["lse"], s["seq_lens"], s["weights"], num_shards=c["shards"],
                           interleave=c["interleave"], is_lse_base_on_e=c["base_e"])
        return {"weights": s["weights"]}
    if c["op"] == "attend":
        args = dict(num_shards=c["shards"], interleave=c["interleave"], is_lse_base_on_e=c["base_e"],
                    logits=s.get("logits"))
        if c["pack"]:
            send = dcp.paged_attention_pack(s["q"], s["k"], s["v"], s["table"], s["seq_lens"], c["pack"], **args)
            out = {"out": send[..., :c["D"]], "lse": send.view(torch.float32)[..., -1]}
        else:
            o, lse = dcp.paged_attention(s["q"], s["k"], s["v"], s["table"], s["seq_lens"], **args)
            out = {"out": o, "lse": lse}
        return dict(out, logits=s["logits"]) if c["logits"] else out
    if c["op"] == "append":
        dcp.dcp_kv_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["seq_lens"], s["starts"],
                          num_shards=c["shards"], interleave=c["interleave"])
        return {"k": s["k"][:-1], "v": s["v"][:-1]}
    kept, new_lens, new_weights = dcp.kv_evict(s["weights"], s["k"], s["v"], s["table"], s["seq_lens"],
                                               s["new_table"], c["keep"], c["recent"], k_out=s["k_out"],
                                               v_out=s["v_out"])
    return {"kept": kept, "new_lens": new_lens, "weights": new_weights, "k": s["k_out"][:-1], "v": s["v_out"][:-1]}


def _local_lens(seq_lens, c, shard=0):
    n, i = c["shards"], c["interleave"]
    return seq_lens // (n * i) * i + (seq_lens % (n * i) - shard * i).clamp(0, i)


def _run_plain(s):
    return {"weigh": _plain_weigh, "attend": _plain_attend, "append": _plain_append,
            "evict": _plain_evict}[s["case"]["op"]](s)


def _plain_attend(s):
    c = s["case"]
    B, H, Hkv, D, page = c["B"], c["H"], c["Hkv"], c["D"], c["page"]
    k = s["k"][s["table"]].reshape(B, -1, Hkv, D).float()
    v = s["v"][s["table"]].reshape(B, -1, Hkv, D).float()
    cap = k.shape[1]
    held = torch.arange(cap, device="cuda") < _local_lens(s["seq_lens"], c)[:, None]
    q = s["q"].float().reshape(B, Hkv, H // Hkv, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    x = torch.where(held[:, None, None, :], x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(held[:, :, None, None], v, 0.0).permute(0, 2, 1, 3))
    o = torch.where(total > 0, o / total, 0.0).reshape(B, H, D).to(s["q"].dtype)
    lse = (total.log() + m).reshape(B, H)
    if not c["base_e"]:
        lse = lse * (1.0 / math.log(2.0))
    if c["pack"]:
        n = c["pack"]
        rows = o.reshape(B, n, H // n, D).transpose(0, 1)
        tail = lse.reshape(B, n, H // n, 1).transpose(0, 1).contiguous().view(o.dtype)
        send = torch.cat([rows, tail], dim=-1)
        out = {"out": send[..., :D], "lse": send.view(torch.float32)[..., -1]}
    else:
        out = {"out": o, "lse": lse}
    if c["logits"]:
        w = s["logits"].shape[2]
        s["logits"].copy_(torch.where(held[:, None, :w], x.reshape(B, H, cap)[:, :, :w], s["logits"]))
        out["logits"] = s["logits"]
    return out


def _plain_append(s):
    c = s["case"]
    T, n, i, page = s["k_new"].shape[0], c["shards"], c["interleave"], c["page"]
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(s["starts"], t, right=True) - 1
    pos = s["seq_lens"][r] - (s["starts"][r + 1] - t)
    mine = pos // i % n == 0
    at = pos // (i * n) * i + pos % i
    width = s["table"].shape[1]
    where = s["table"][r, (at // page).clamp(max=width - 1)].long() * page + at % page
    spare = (s["k"].shape[0] - 1) * page  # rows of other shards go to the page that is in no table
    where = torch.where(mine, where, spare)
    s["k"].flatten(0, 1).index_copy_(0, where, s["k_new"])
    s["v"].flatten(0, 1).index_copy_(0, where, s["v_new"])
    return {"k": s["k"][:-1], "v": s["v"][:-1]}


def _plain_weigh(s):
    c = s["case"]
    B, H, cap = s["logits"].shape
    x = s["logits"] if c["base_e"] else s["logits"] * (1.0 / math.log(2.0))
    x = x - s["lse"][:, :, None]
    w = (torch.exp(x) if c["base_e"] else torch.exp2(x)).reshape(B, c["Hkv"], H // c["Hkv"], cap).sum(2)
    held = torch.arange(cap, device="cuda") < _local_lens(s["seq_lens"], c)[:, None]
    s["weights"].add_(torch.where(held[:, None, :], w, 0.0))
    return {"weights": s["weights"]}


def _plain_evict(s):
    c = s["case"]
    B, Hkv, cap = s["weights"].shape
    D, page, keep = c["D"], c["page"], c["keep"]
    n = s["seq_lens"][:, None, None]
    pos = torch.arange(cap, device="cuda")
    held = pos < n
    last = held & (pos >= n - c["recent"])
    key = torch.where(held, s["weights"], float("-inf"))
    key = torch.where(last, float("inf"), key)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    order = torch.where(torch.arange(order.shape[-1], device="cuda") < n, order, cap)
    kept = torch.full((B, Hkv, keep), cap, device="cuda")
    kept[..., :order.shape[-1]] = torch.sort(order, dim=-1).values
    new_lens = s["seq_lens"].clamp(max=keep)
    valid = kept < cap
    src = kept.clamp(max=cap - 1)
    rows = torch.arange(B, device="cuda")[:, None, None]
    width = s["table"].shape[1]
    frm = s["table"][rows, (src // page).clamp(max=width - 1)].long() * page + src % page
    j = torch.arange(keep, device="cuda")
    spare = (s["k_out"].shape[0] - 1) * page
    to = torch.where(valid, (s["new_table"][:, j // page].long() * page + j % page)[:, None, :], spare)
    heads = torch.arange(Hkv, device="cuda")[None, :, None].expand_as(to)
    for name in ("k", "v"):
        s[name + "_out"].flatten(0, 1)[to, heads] = s[name].flatten(0, 1)[frm, heads]
    new_weights = torch.zeros_like(s["weights"])
    m = min(cap, keep)
    new_weights[..., :m] = torch.where(valid, torch.gather(s["weights"], 2, src), 0.0)[..., :m]
    return {"kept": torch.where(valid, kept, -1).int(), "new_lens": new_lens, "weights": new_weights,
            "k": s["k_out"][:-1], "v": s["v_out"][:-1]}


# ---- the definitions in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":  # rows are copied as they are
        pools = {"k": s["k"].double(), "v": s["v"].double()}
        n, i, q, page = case["shards"], case["interleave"], case["q"], case["page"]
        for r, length in enumerate(_lens(case)):
            mine = [p for p in range(length - q, length) if (p // i) % n == 0]
            if not mine:
                continue
            tok = torch.tensor([r * q + p - (length - q) for p in mine], device="cuda")
            at = torch.tensor([_local(p, case) for p in mine], device="cuda")  # held before position p
            pages = s["table"][r, at // page].long()
            for x in pools:
                pools[x][pages, at % page] = s[x + "_new"][tok].double()
        return {x: pools[x][:-1] for x in pools}
    if case["op"] == "weigh":
        w = s["weights"].double()
        G = case["H"] // case["Hkv"]
        base = math.e if case["base_e"] else 2.0
        for b, length in enumerate(_lens(case)):
            n = _local(length, case)
            for h in range(case["H"]):
                nat = s["lse"][b, h].double() * math.log(base)
                w[b, h // G, :n] += torch.exp(s["logits"][b, h, :n].double() - nat)
        return {"weights": w}
    if case["op"] == "evict":  # rows and weights are copied as they are
        out = {"weights": torch.zeros_like(s["weights"]).double(), "k": s["k_out"].double(), "v": s["v_out"].double()}
        page, keep, recent = case["page"], case["keep"], case["recent"]
        for b, n in enumerate(_lens(case)):
            m = min(n, keep)
            last = min(recent, m)
            new_slots = torch.arange(m, device="cuda")
            to = s["new_table"][b, new_slots // page].long(), new_slots % page
            for h in range(case["Hkv"]):
                w = s["weights"][b, h, :n].double()
                # largest first, ties by position
                best = torch.argsort(-w[:n - last], stable=True)[:m - last]
                kept = torch.cat([best.sort().values, torch.arange(n - last, n, device="cuda")])
                out["weights"][b, h, :m] = w[kept]
                frm = s["table"][b, kept // page].long(), kept % page
                for x in ("k", "v"):
                    out[x][to[0], to[1], h] = s[x][frm[0], frm[1], h].double()
        return {"kept": None, "new_lens": None, "weights": out["weights"], "k": out["k"][:-1], "v": out["v"][:-1]}
    B, H, Hkv, D, page = (case[x] for x in ("B", "H", "Hkv", "D", "page"))
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), float("-inf"), dtype=torch.float64, device="cuda")
    logits = s["logits"].double() if case["logits"] else None
    G = H // Hkv
    for b, length in enumerate(_lens(case)):
        n = _local(length, case)
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        for j in range(Hkv):
            keys = s["k"][pages, :, j].reshape(-1, D)[:n].double()
            vals = s["v"][pages, :, j].reshape(-1, D)[:n].double()
            x = s["q"][b, j * G:(j + 1) * G].double() @ keys.t() / math.sqrt(D)
            z = torch.logsumexp(x, 1)
            out[b, j * G:(j + 1) * G] = torch.softmax(x, 1) @ vals
            lse[b, j * G:(j + 1) * G] = z
            if logits is not None:
                logits[b, j * G:(j + 1) * G, :n] = x
    if not case["base_e"]:
        lse = lse / math.log(2.0)
    if case["pack"]:
        n = case["pack"]
        out = out.reshape(B, n, H // n, D).permute(1, 0, 2, 3).contiguous()
        lse = lse.reshape(B, n, H // n).permute(1, 0, 2).contiguous()
    r = {"out": out, "lse": lse}
    return dict(r, logits=logits) if case["logits"] else r
