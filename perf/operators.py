"""What the serving-step operators are measured on: the query/key norm and rotation with the cache
write (kind "rope"), the step's page tables and slot maps ("tables"), and attention of one new token
per sequence over a 16-bit paged cache ("attention").

With `own` false, run() computes an operator in elementary torch operations; with `own` true it makes
the library's calls.  Heads have 128 channels throughout; pages hold [heads][page_size][128].
"""
import math
import random

import torch

own = False

D = 128
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------
def listed():
    return [
        # one user's decode step: three or four rows, pure latency
        _rope("rope_decode_3", tokens=3, hq=32, hkv=8, norm=True, page=128),
        # a batch of decode steps, rows cut out of one fused projection
        _rope("rope_step_256", tokens=256, hq=32, hkv=8, norm=True, page=16, fused=True),
        # a large prefill chunk
        _rope("rope_prefill_16k", tokens=16384, hq=32, hkv=8, norm=True, page=128, fused=True),
        # odd chunk, no norm, part of the head rotated in the interleaved layout, fp16
        _rope("rope_partial_interleaved_5003", tokens=5003, hq=40, hkv=10, x="fp16", page=64, rot=64,
              interleaved=True, far=True),
        # projections left in fp32, as the block pseudo-decode has them
        _rope("rope_fp32_in_2000", tokens=2000, hq=32, hkv=8, x="fp32", norm=True, page=128),
        # a decode step of a serving batch: every sequence one token, few new pages
        _tables("tables_decode_64", batch=64, max_new=1, page=128, hkv=8, max_len=32768),
        # a mixed step: most rows decode, some prefill, some finish and hand their pages back
        _tables("tables_mixed_1000", batch=1000, max_new=700, page=16, hkv=0, max_len=4096, finish=True),
        # a single user at a moderate context: latency of the split and the join
        _attention("attention_b1_4k", batch=1, hq=32, hkv=8, max_len=4096, page=128),
        # the decode shape the packed cache is measured on
        _attention("attention_b16_32k", batch=16, hq=32, hkv=8, max_len=32768, page=128),
        # ragged long contexts, 40 query heads over 10
        _attention("attention_b4_ragged_128k", batch=4, hq=40, hkv=10, min_len=65536, max_len=131072, page=64),
        # many short conversations, small pages, capped scores
        _attention("attention_b256_short", batch=256, hq=64, hkv=8, x="fp16", min_len=1, max_len=900, page=16,
                   softcap=30.0, out="fp16"),
        # one kv head per query head, distance bias and a sliding window over ragged contexts
        _attention("attention_b32_window", batch=32, hq=32, hkv=32, min_len=50, max_len=9000, page=32,
                   window=2000, slopes=True, out="bf16"),
    ]


def _rope(name, tokens, hq, hkv, x="bf16", norm=False, page=128, rot=128, interleaved=False, fused=False, far=False):
    return {"name": name, "kind": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "x": x,
            "cache": "fp16" if x == "fp16" else "bf16", "norm": norm, "page": page, "rot": rot,
            "interleaved": interleaved, "fused": fused, "far": far}


def _tables(name, batch, max_new, page, hkv, max_len, finish=False):
    return {"name": name, "kind": "tables", "batch": batch, "max_new": max_new, "page": page, "hkv": hkv,
            "max_len": max_len, "finish": finish}


def _attention(name, batch, hq, hkv, max_len, page, min_len=None, x="bf16", softcap=0.0, window=0, slopes=False,
               starts=False, out="fp32"):
    return {"name": name, "kind": "attention", "batch": batch, "hq": hq, "hkv": hkv, "x": x,
            "min_len": max_len if min_len is None else min_len, "max_len": max_len, "page": page,
            "softcap": softcap, "window": window, "slopes": slopes, "starts": starts, "out": out}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (40, 10), (8, 1), (64, 8), (28, 4), (16, 16), (5, 5), (71, 1), (32, 32), (12, 2)]


def draw(rng):
    kind = rng.choice(["rope", "rope", "tables", "attention", "attention", "attention"])
    if kind == "rope":
        hq, hkv = rng.choice(HEADS)
        x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 16384 * 48 // (hq + 2 * hkv) // (2 if x == "fp32" else 1)
        c = _rope("", tokens=_log_int(rng, 1, most), hq=hq, hkv=hkv, x=x, norm=rng.random() < 0.6,
                  page=rng.choice([16, 32, 64, 128, 48, 1]), rot=rng.choice([128, 128, 64, 32, 96]),
                  interleaved=rng.random() < 0.4, fused=rng.random() < 0.5, far=rng.random() < 0.3)
    elif kind == "tables":
        batch = _log_int(rng, 1, 2048)
        c = _tables("", batch=batch, max_new=_log_int(rng, 1, max(1, min(4000, 350000 // batch))),
                    page=rng.choice([16, 32, 64, 128, 48]), hkv=rng.choice([0, 0, 1, 8, 10]),
                    max_len=_log_int(rng, 500, max(600, 4000000 // batch)), finish=rng.random() < 0.5)
    else:
        hq, hkv = rng.choice(HEADS)
        batch = _log_int(rng, 1, 256)
        max_len = _log_int(rng, 1, max(1, min(131072, 4194304 // (batch * hkv))))
        c = _attention("", batch=batch, hq=hq, hkv=hkv, max_len=max_len,
                       min_len=rng.choice([None, 1, max(1, max_len // 2)]), page=rng.choice([16, 32, 64, 128, 48]),
                       x=rng.choice(["bf16", "bf16", "fp16"]), softcap=rng.choice([0.0, 0.0, 50.0]),
                       window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), slopes=rng.random() < 0.25,
                       starts=rng.random() < 0.25, out=rng.choice(["fp32", "fp32", "16"]))
        if c["out"] == "16":
            c["out"] = c["x"]
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------------------------
def _lens(case, seed):
    r = random.Random(seed)
    return [r.randint(case["min_len"], case["max_len"]) for _ in range(case["batch"])]


def _starts(case, seed, lens):
    """First visible key of each sequence: another document's tokens come before it in its pages."""
    r = random.Random(seed + 7)
    return [r.randint(0, n // 2) for n in lens]


def _rope_frequencies(rot):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return 500000.0 ** (-2.0 * i / rot)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": dict(case)}
    if case["kind"] == "rope":
        _prepare_rope(case, g, st)
    elif case["kind"] == "tables":
        _prepare_tables(case, seed, g, st)
    else:
        _prepare_attention(case, seed, g, st)
    return st


def _prepare_rope(case, g, st):
    T, hq, hkv, P = case["tokens"], case["hq"], case["hkv"], case["page"]
    xt, ct = DT[case["x"]], DT[case["cache"]]
    chan = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))

    def rows(h):
        return (torch.randn(T, h, D, generator=g, device="cuda") * chan).to(xt)

    if case["fused"]:  # q, k and v are columns of one projection's rows
        qkv = rows(hq + 2 * hkv)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        st["q"], st["k"], st["v"] = rows(hq), rows(hkv), rows(hkv)
    most = 1000000 if case["far"] else 32768
    # runs of neighbouring positions, as chunks of prompts have
    first = torch.randint(0, most - 700, (T // 500 + 1,), generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    st["positions"] = (first[t // 500] + t % 500).to(torch.int32)
    n_pages = -(-T // P) + 3
    slots = torch.randperm(n_pages, generator=g, device="cuda")[t // P] * P + t % P
    st["slots"] = slots.to(torch.int32)
    st["k_cache"] = torch.randn(n_pages, hkv, P, D, generator=g, device="cuda").to(ct)
    st["v_cache"] = torch.randn(n_pages, hkv, P, D, generator=g, device="cuda").to(ct)
    st["q_out"] = torch.empty(T, hq, D, dtype=ct, device="cuda")
    st["freqs"] = _rope_frequencies(case["rot"])
    st["scale"] = 1.1 if case["far"] else 1.0
    st["qw"] = st["kw"] = None
    if case["norm"]:
        st["qw"] = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
        st["kw"] = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")


def _prepare_tables(case, seed, g, st):
    B, P, hkv = case["batch"], case["page"], case["hkv"]
    # the same mix of requests for every seed, in another order: the step's row count stays
    r = random.Random(B * 1000003 + case["max_new"] * 1009 + case["max_len"])
    mix = [(r.randint(0, case["max_len"]), 1 if r.random() < 0.8 else r.randint(1, case["max_new"]))
           for _ in range(B)]
    if case["finish"]:
        mix = [(a, -1 if r.random() < 0.1 else n) for a, n in mix]
    random.Random(seed).shuffle(mix)
    lens, new = [a for a, _ in mix], [n for _, n in mix]
    counts = [-(-n // P) for n in lens]
    need = [0 if n < 0 else max(0, -(-(a + n) // P) - c) for a, n, c in zip(lens, new, counts)]
    width = -(-(case["max_len"] + case["max_new"]) // P)
    held, total = sum(counts), sum(counts) + sum(need)
    pool = torch.randperm(total + 5, generator=g, device="cuda").to(torch.int32)
    i = torch.arange(width, device="cuda")
    cnt = torch.tensor(counts, device="cuda")
    at = torch.cumsum(cnt, 0) - cnt
    owned = i[None] < cnt[:, None]
    table = torch.where(owned, pool[(at[:, None] + i[None]).clamp(max=total)], -1).to(torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")
    st["lens"], st["new"] = torch.tensor(lens, **i32), torch.tensor(new, **i32)
    st["counts"], st["table"] = cnt.to(torch.int32), table.contiguous()
    st["free"] = torch.full((total + 5,), -1, **i32)
    st["free"][:total + 5 - held] = pool[held:]
    st["n_free"] = torch.tensor([total + 5 - held], **i32)
    st["kv_lens"], st["counts_out"] = torch.empty(B, **i32), torch.empty(B, **i32)
    st["n_free_out"], st["status"] = torch.empty(1, **i32), torch.empty(1, **i32)
    T = sum(max(0, n) for n in new)
    T += T // 50  # room for a few more rows than this step has
    st["cu"] = torch.empty(B + 1, **i32)
    st["positions"], st["slots"] = torch.empty(T, **i32), torch.empty(T, **i32)
    st["blocks"] = None
    if hkv:
        h = torch.arange(hkv, device="cuda", dtype=torch.int32)
        st["blocks"] = torch.where(owned[:, None], table[:, None] * hkv + h[None, :, None], -1).to(torch.int32).contiguous()


def _prepare_attention(case, seed, g, st):
    B, hq, hkv, P = case["batch"], case["hq"], case["hkv"], case["page"]
    xt = DT[case["x"]]
    lens = _lens(case, seed)
    width = -(-max(lens) // P) + 1
    used = [-(-n // P) for n in lens]
    n_pages = sum(used) + 2
    pool = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    cnt = torch.tensor(used, device="cuda")
    at = torch.cumsum(cnt, 0) - cnt
    i = torch.arange(width, device="cuda")
    st["table"] = torch.where(i[None] < cnt[:, None], pool[(at[:, None] + i[None]).clamp(max=n_pages - 1)], 0).to(torch.int32)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["k_cache"] = torch.randn(n_pages, hkv, P, D, dtype=xt, generator=g, device="cuda")
    st["k_cache"] *= torch.exp(0.5 * torch.randn(hkv, 1, D, generator=g, device="cuda")).to(xt)
    st["v_cache"] = torch.randn(n_pages, hkv, P, D, dtype=xt, generator=g, device="cuda")
    st["q"] = torch.randn(B, hq, D, dtype=xt, generator=g, device="cuda")
    st["out"] = torch.empty(B, hq, D, dtype=DT[case["out"]], device="cuda")
    st["lse"] = torch.empty(B, hq, device="cuda")
    st["slopes"] = None
    if case["slopes"]:
        st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq)
    st["starts"] = None
    if case["starts"]:
        st["starts"] = torch.tensor(_starts(case, seed, lens), dtype=torch.int32, device="cuda")
    st["longest"] = max(lens)


# ---- one pass --------------------------------------------------------------------------------------
def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"rope": _own_rope, "tables": _own_tables, "attention": _own_attention}[kind](state)
    return {"rope": _plain_rope, "tables": _plain_tables, "attention": _plain_attention}[kind](state)


def _own_rope(s):
    import bit_kv_cache_kvarn_gb300 as kv

    c = s["case"]
    kv.kvarn_rope_qkv(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["q_out"], s["k_cache"], s["v_cache"],
                      slot_map=s["slots"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, rope_scale=s["scale"],
                      interleaved=c["interleaved"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_tables(s):
    import bit_kv_cache_kvarn_gb300 as kv

    kv.kvarn_step_tables(s["lens"], s["new"], s["counts"], s["table"], s["free"], s["n_free"], s["case"]["page"],
                         s["kv_lens"], s["counts_out"], s["n_free_out"], s["cu"], s["positions"], s["slots"],
                         s["status"], block_table=s["blocks"])
    return _tables_out(s)


def _own_attention(s):
    import bit_kv_cache_kvarn_gb300 as kv

    c = s["case"]
    if "workspace" not in s:  # a user's program allocates it once
        n = kv.kvarn_paged_attention_workspace_size(c["batch"], c["hq"], c["hkv"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    kv.kvarn_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"], 1 / math.sqrt(D),
                             s["workspace"], softcap=c["softcap"], slopes=s["slopes"], window=c["window"],
                             kv_starts=s["starts"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _rotate(x, w, cos, sin, case):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(torch.mean(x * x, dim=-1, keepdim=True) + 1e-6) * w
    R = case["rot"]
    r, rest = x[..., :R], x[..., R:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _plain_rope(s):
    c = s["case"]
    ang = s["positions"].double()[:, None] * s["freqs"][None]
    cos = (torch.cos(ang) * s["scale"]).float()[:, None]
    sin = (torch.sin(ang) * s["scale"]).float()[:, None]
    s["q_out"].copy_(_rotate(s["q"], s["qw"], cos, sin, c))
    page, off = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    s["k_cache"][page, :, off] = _rotate(s["k"], s["kw"], cos, sin, c).to(s["k_cache"].dtype)
    s["v_cache"][page, :, off] = s["v"].to(s["v_cache"].dtype)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _tables_out(s):
    out = {k: s[k] for k in ("kv_lens", "counts_out", "n_free_out", "cu", "positions", "slots", "status", "table", "free")}
    if s["blocks"] is not None:
        out["blocks"] = s["blocks"]
    return out


def _plain_tables(s):
    P = s["case"]["page"]
    lens, counts, table = s["lens"].long(), s["counts"].long(), s["table"]
    width, T = table.shape[1], s["positions"].numel()
    rel = s["new"] < 0
    add = s["new"].long().clamp(min=0)
    kv = torch.where(rel, 0, lens + add)
    held = torch.where(rel, 0, torch.maximum(counts, (kv + P - 1) // P))
    fresh = torch.where(rel, 0, held - counts)
    given = torch.where(rel, counts, 0)
    cu = torch.cumsum(add, 0)
    n_free = s["n_free"].long()
    left = n_free + given.sum() - fresh.sum()
    ok = (left >= 0) & (held.max() <= width) & (cu[-1] <= T)
    i = torch.arange(width, device=table.device)
    # the page stack with the finished sequences' pages pushed, in order, on top
    back = (rel[:, None] & (i[None] < counts[:, None])).flatten()
    nth = torch.cumsum(back, 0) - 1
    size = s["free"].numel()
    stack = torch.cat([s["free"], s["free"].new_zeros(1)])
    stack[torch.where(back, (n_free + nth).clamp(max=size), size)] = table.flatten()
    top = n_free + given.sum()
    j = torch.arange(size, device=table.device)
    write = ok & (j >= n_free) & (j < left)
    # and the new pages popped, in order
    take = ((i[None] >= counts[:, None]) & (i[None] < held[:, None])).flatten() & ok
    kth = torch.cumsum(take, 0) - 1
    page = stack[(top - 1 - kth).clamp(min=0, max=size)]
    take, page = take.view(table.shape), page.view(table.shape)
    new_table = torch.where(take, page, table)
    # one row for each token of the step
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(cu, t, right=True).clamp(max=cu.numel() - 1)
    live = ok & (t < cu[-1])
    pos = lens[b] + t - (cu - add)[b]
    slot = new_table[b, (pos // P).clamp(min=0, max=width - 1)].long() * P + pos % P
    s["positions"].copy_(torch.where(live, pos, -1))
    s["slots"].copy_(torch.where(live, slot, -1))
    s["cu"].copy_(torch.cat([cu.new_zeros(1), torch.where(ok, cu, 0)]))
    s["kv_lens"].copy_(torch.where(ok, kv, lens))
    s["counts_out"].copy_(torch.where(ok, held, counts))
    s["n_free_out"].copy_(torch.where(ok, left, n_free))
    s["status"].copy_(torch.where(left < 0, 1, 0) + torch.where(held.max() > width, 2, 0) + torch.where(cu[-1] > T, 4, 0))
    s["free"].copy_(torch.where(write, stack[:-1], s["free"]))
    if s["blocks"] is not None:
        hkv = s["blocks"].shape[1]
        h = torch.arange(hkv, device=table.device)
        s["blocks"].copy_(torch.where(take[:, None], page[:, None] * hkv + h[None, :, None], s["blocks"]))
    table.copy_(new_table)
    return _tables_out(s)


def _plain_attention(s):
    c = s["case"]
    B, hq, hkv, P = c["batch"], c["hq"], c["hkv"], c["page"]
    g, L = hq // hkv, s["longest"]
    pos = torch.arange(L, device="cuda")
    lens = s["lens"].long()
    seen = pos[None] < lens[:, None]
    if c["window"]:
        seen &= pos[None] >= lens[:, None] - c["window"]
    if s["starts"] is not None:
        seen &= pos[None] >= s["starts"][:, None]
    page, off = s["table"].long()[:, pos // P], (pos % P)[None].expand(B, L)
    k = s["k_cache"][page, :, off].permute(0, 2, 3, 1).float()  # [B, hkv, 128, L]
    x = torch.matmul(s["q"].view(B, hkv, g, D).float(), k)
    del k
    x = x * (1 / math.sqrt(D))
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    if s["slopes"] is not None:
        x = x + s["slopes"].view(1, hkv, g, 1) * (pos[None] - (lens[:, None] - 1)).float()[:, None, None]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    v = s["v_cache"][page, :, off].permute(0, 2, 1, 3).float()  # [B, hkv, L, 128]
    v = v.masked_fill(~seen[:, None, :, None], 0)
    o = torch.matmul(p, v)
    del v
    o = torch.where(z > 0, o / z, 0)
    s["out"].copy_(o.view(B, hq, D))
    s["lse"].copy_((m + torch.log(z)).view(B, hq))
    return {"out": s["out"], "lse": s["lse"]}


# ---- what a pass cannot do without -----------------------------------------------------------------
def work(case):
    if case["kind"] == "rope":
        T, h = case["tokens"], case["hq"] + 2 * case["hkv"]
        size = 4 if case["x"] == "fp32" else 2
        turned = T * (case["hq"] + case["hkv"])
        return {"bytes": T * h * D * (size + 2) + 8 * T,
                "flops": turned * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    if case["kind"] == "tables":
        B, new = case["batch"], 0.8 + 0.2 * (1 + case["max_new"]) / 2
        new *= 0.9 if case["finish"] else 1.0
        pages = B * new / case["page"] + (0.1 * B * case["max_len"] / 2 / case["page"] if case["finish"] else 0)
        return {"bytes": 4 * (6 * B + 2 * B * new + pages * (2 + case["hkv"])), "flops": 0}
    seen = (case["min_len"] + case["max_len"]) / 2
    if case["window"]:
        seen = _mean_seen(case)
    elif case["starts"]:
        seen *= 0.75
    size = 4 if case["out"] == "fp32" else 2
    head_tokens = case["batch"] * seen * case["hkv"]
    rows = case["batch"] * case["hq"]
    return {"bytes": head_tokens * 4 * D + rows * (D * (2 + size) + 4) + case["batch"] * (4 + 4 * seen / case["page"]),
            "flops": case["batch"] * seen * case["hq"] * 4 * D}


def _mean_seen(case):
    """Mean of min(length, window) over uniform lengths (a start before the window hides a little more)."""
    lo, hi, w = case["min_len"], case["max_len"], case["window"]
    if w >= hi:
        return (lo + hi) / 2
    if w <= lo:
        return w
    return ((w - lo) * (lo + w) / 2 + (hi - w) * w) / (hi - lo)


# ---- the same in 64 bits -----------------------------------------------------------------------------
def exact(case, seed):
    if case["kind"] == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    return (_exact_rope if case["kind"] == "rope" else _exact_attention)(case, seed, s)


def _exact_rope(case, seed, s):
    R, P, T = case["rot"], case["page"], case["tokens"]
    i = torch.arange(R // 2, device="cuda")
    a = 2 * i if case["interleaved"] else i
    b = 2 * i + 1 if case["interleaved"] else i + R // 2
    turn = torch.polar(torch.full((T, 1, R // 2), s["scale"], dtype=torch.float64, device="cuda"),
                       (s["positions"].double()[:, None] * s["freqs"][None])[:, None])
    made = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        y = s[name].double()
        if w is not None:
            y = y / (y.square().sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn
        y = y.clone()
        y[..., a], y[..., b] = z.real, z.imag
        made[name] = y
    k, v = s["k_cache"].double(), s["v_cache"].double()
    at = s["slots"].long()
    k.transpose(1, 2)[at // P, at % P] = made["k"]
    v.transpose(1, 2)[at // P, at % P] = s["v"].double()
    return {"q": made["q"], "k_cache": k, "v_cache": v}


def _exact_attention(case, seed, s):
    hq, hkv, P = case["hq"], case["hkv"], case["page"]
    lens = _lens(case, seed)
    starts = _starts(case, seed, lens) if case["starts"] else [0] * len(lens)
    out = torch.zeros(len(lens), hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens), hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        lo = max(starts[b], n - case["window"] if case["window"] else 0)
        if lo >= n:
            continue
        pages = s["table"][b, :-(-n // P)].long()
        k = s["k_cache"][pages].transpose(0, 1).reshape(hkv, -1, D)[:, lo:n].double()
        v = s["v_cache"][pages].transpose(0, 1).reshape(hkv, -1, D)[:, lo:n].double()
        q = s["q"][b].double().view(hkv, hq // hkv, D)
        x = q @ k.transpose(1, 2) / math.sqrt(D)
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        if s["slopes"] is not None:
            back = torch.arange(lo - n + 1, 1, dtype=torch.float64, device="cuda")
            x = x + s["slopes"].double().view(hkv, -1, 1) * back
        lse[b] = torch.logsumexp(x, -1).view(hq)
        out[b] = (torch.softmax(x, -1) @ v).view(hq, D)
    return {"out": out, "lse": lse}
