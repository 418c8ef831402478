"""What the operators beside a decode step are measured on: attention of many new tokens per sequence over
16-bit pages (kind "prompt"), attention of a batch over a prefix that its sequences share (kind "prefix"),
the write of keys and values into 8-bit pages (kind "quantize") and attention of one new token per sequence
over them (kind "q8").

With `own` false, run() computes an operator in elementary torch operations; with `own` true it makes the
library's calls.  Heads have 128 channels throughout; pages hold [heads][page_size][128].
"""
import math
import random

import torch

own = False

D = 128
SCALE = 1 / math.sqrt(D)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------
def listed():
    return [
        # drafts of a few tokens checked against their conversations: latency
        _prompt("prompt_drafts_b8", batch=8, new=(4, 6), ctx=(100, 2000), hq=32, hkv=8, page=16),
        # an ordinary batch of prompts, packed, of any lengths; the step's row buffer is longer than they are
        _prompt("prompt_packed_b24", batch=24, new=(1, 2000), ctx=(0, 0), hq=32, hkv=8, page=16, spare=100),
        # a chunk of a long document behind what is in the cache already
        _prompt("prompt_chunk_2000_behind_60k", batch=1, new=(2000, 2000), ctx=(60001, 60001), hq=32, hkv=8, page=128),
        # one long prompt
        _prompt("prompt_long_16k", batch=1, new=(16384, 16384), ctx=(0, 0), hq=32, hkv=8, page=128),
        # a kv head for each query head, capped scores, sliding window, some documents behind others
        _prompt("prompt_window_b3", batch=3, new=(1500, 5000), ctx=(0, 2500), hq=16, hkv=16, page=48, x="fp16",
                softcap=50.0, window=1000, starts=True),
        # a few answers to one prompt, sampled together: latency
        _prefix("prefix_b4_700", batch=4, groups=1, prefix=(700, 700), tail=(1, 60), hq=32, hkv=8, page=16),
        # a large batch behind one long system prompt
        _prefix("prefix_b128_32k", batch=128, groups=1, prefix=(32768, 32768), tail=(1, 500), hq=32, hkv=8, page=128),
        # several prompts at once, each with its own batch
        _prefix("prefix_groups_b90", batch=90, groups=5, prefix=(900, 12000), tail=(1, 1500), hq=40, hkv=10, page=64,
                x="fp16", softcap=30.0),
        # a decode step's new rows
        _quantize("quantize_step_64", tokens=64, hkv=8, page=16, holes=True),
        # a prompt's rows, cut out of one fused projection
        _quantize("quantize_prompt_16k", tokens=16384, hkv=8, page=128, fused=True),
        # decode over short conversations, small pages
        _q8("q8_b200_short", batch=200, min_len=1, max_len=1200, hq=64, hkv=8, page=16, x="fp16", out="fp16"),
        # decode over long ones
        _q8("q8_b16_32k", batch=16, min_len=32768, max_len=32768, hq=32, hkv=8, page=128),
    ]


def _prompt(name, batch, new, ctx, hq, hkv, page, x="bf16", softcap=0.0, window=0, slopes=False, starts=False,
            causal=True, spare=0):
    return {"name": name, "kind": "prompt", "batch": batch, "min_new": new[0], "max_new": new[1], "min_ctx": ctx[0],
            "max_ctx": ctx[1], "hq": hq, "hkv": hkv, "page": page, "x": x, "softcap": softcap, "window": window,
            "slopes": slopes, "starts": starts, "causal": causal, "spare": spare}


def _prefix(name, batch, groups, prefix, tail, hq, hkv, page, x="bf16", softcap=0.0):
    return {"name": name, "kind": "prefix", "batch": batch, "groups": groups, "min_prefix": prefix[0],
            "max_prefix": prefix[1], "min_tail": tail[0], "max_tail": tail[1], "hq": hq, "hkv": hkv, "page": page, "x": x,
            "softcap": softcap}


def _quantize(name, tokens, hkv, page, x="bf16", fused=False, holes=False):
    return {"name": name, "kind": "quantize", "tokens": tokens, "hkv": hkv, "page": page, "x": x, "fused": fused,
            "holes": holes}


def _q8(name, batch, min_len, max_len, hq, hkv, page, x="bf16", softcap=0.0, window=0, slopes=False, starts=False,
        out="fp32"):
    return {"name": name, "kind": "q8", "batch": batch, "min_len": min_len, "max_len": max_len, "hq": hq, "hkv": hkv,
            "page": page, "x": x, "softcap": softcap, "window": window, "slopes": slopes, "starts": starts, "out": out}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (40, 10), (8, 1), (64, 8), (28, 4), (16, 16), (5, 5), (71, 1), (32, 32), (12, 2)]
PAGES = [16, 32, 64, 128, 48, 256]


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "prompt", "prefix", "prefix", "quantize", "q8", "q8"])
    hq, hkv = rng.choice(HEADS)
    page, x, softcap = rng.choice(PAGES), rng.choice(["bf16", "bf16", "fp16"]), rng.choice([0.0, 0.0, 0.0, 50.0])
    if kind == "prompt":
        batch = _log_int(rng, 1, 64)
        causal = rng.random() < 0.85
        new = _log_int(rng, 1, 8000)
        room = 16384 * 16384 * 32 // (batch * hq * new)  # keys a sequence, at the cost of the largest listed case
        while room < new:  # that many rows leave no room for their own keys
            new = max(1, new // 2)
            room = 16384 * 16384 * 32 // (batch * hq * new)
        ctx = rng.choice([0, 0, _log_int(rng, 1, max(1, min(100000, room - new, 2000000 // (batch * hkv))))])
        ctx = min(ctx, room - new)
        c = _prompt("", batch=batch, new=(rng.choice([new, 1, max(1, new // 2)]), new), ctx=(rng.choice([0, ctx]), ctx),
                    hq=hq, hkv=hkv, page=page, x=x, softcap=softcap,
                    window=rng.choice([0, 0, _log_int(rng, 1, 4096)]) if causal else 0, slopes=causal and rng.random() < 0.2,
                    starts=rng.random() < 0.25, causal=causal, spare=rng.choice([0, 0, rng.randint(1, 40)]))
    elif kind == "prefix":
        batch = _log_int(rng, 1, 192)
        groups = min(batch, rng.choice([1, 1, 2, _log_int(rng, 1, 16)]))
        most = max(1, min(40000, 2000000 // (hkv * groups)))
        prefix = _log_int(rng, min(16, most), most)
        tail = _log_int(rng, 1, min(2000, max(1, 1500000 // (batch * hkv))))
        c = _prefix("", batch=batch, groups=groups, prefix=(rng.choice([prefix, 1, max(1, prefix // 2)]), prefix),
                    tail=(rng.choice([0, 1, tail]), tail), hq=hq, hkv=hkv, page=page, x=x, softcap=softcap)
    elif kind == "quantize":
        c = _quantize("", tokens=_log_int(rng, 1, 131072 // hkv), hkv=hkv, page=rng.choice(PAGES + [1]),
                      x=rng.choice(["bf16", "bf16", "fp16", "fp32"]), fused=rng.random() < 0.5, holes=rng.random() < 0.4)
    else:
        batch = _log_int(rng, 1, 256)
        max_len = _log_int(rng, 1, max(1, min(131072, 4194304 // (batch * hkv))))
        c = _q8("", batch=batch, min_len=rng.choice([max_len, 0, 1, max(1, max_len // 2)]), max_len=max_len, hq=hq, hkv=hkv,
                page=page, x=x, softcap=softcap, window=rng.choice([0, 0, _log_int(rng, 1, 4096)]),
                slopes=rng.random() < 0.25, starts=rng.random() < 0.25, out=rng.choice(["fp32", "fp32", x]))
    del c["name"]
    return c


def _mix(case, lo, hi, n, salt):
    """n whole numbers of lo..hi, the same ones for every seed."""
    r = random.Random("%d %s" % (salt, sorted((k, v) for k, v in case.items() if k != "name")))
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case, seed):
    """(new tokens, context) of a prompt's sequences, (prefix of each group, own tokens, group sizes) of a
    prefix case, lengths of a q8 case: one mix of requests, in an order that the seed gives."""
    r = random.Random(seed)
    if case["kind"] == "prompt":
        both = list(zip(_mix(case, case["min_new"], case["max_new"], case["batch"], 1),
                        _mix(case, case["min_ctx"], case["max_ctx"], case["batch"], 2)))
        r.shuffle(both)
        return [n for n, _ in both], [c for _, c in both]
    if case["kind"] == "prefix":
        G, B = case["groups"], case["batch"]
        # sizes of the groups: B cut at G - 1 places
        cuts = sorted(random.Random(B * 1009 + G).sample(range(1, B), G - 1))
        groups = list(zip([b - a for a, b in zip([0] + cuts, cuts + [B])],
                          _mix(case, case["min_prefix"], case["max_prefix"], G, 3)))
        r.shuffle(groups)
        tails = _mix(case, case["min_tail"], case["max_tail"], B, 4)
        r.shuffle(tails)
        return [p for _, p in groups], tails, [n for n, _ in groups]
    lens = _mix(case, case["min_len"], case["max_len"], case["batch"], 5)
    r.shuffle(lens)
    return lens


def _starts(case, seed, lens):
    """First visible key of each sequence: another document's tokens come before it in its pages."""
    r = random.Random(seed + 7)
    return [r.randint(0, n // 2) for n in lens]


# ---- inputs --------------------------------------------------------------------------------------
def _tables(lens, page, g, extra=1):
    """A page table for sequences of these lengths with pages scattered over a pool, and the pool's size."""
    used = [-(-n // page) for n in lens]
    width, total = max(used) + extra, sum(used) + 2
    pool = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    cnt = torch.tensor(used, device="cuda")
    at = torch.cumsum(cnt, 0) - cnt
    i = torch.arange(width, device="cuda")
    table = torch.where(i[None] < cnt[:, None], pool[(at[:, None] + i[None]).clamp(max=total - 1)], 0)
    return table.to(torch.int32).contiguous(), total


def _kv(n_pages, case, g, dt):
    """Keys with channels of different sizes, as projections give them, and values."""
    shape = (n_pages, case["hkv"], case["page"], D)
    k = torch.randn(shape, dtype=dt, generator=g, device="cuda")
    k *= torch.exp(0.5 * torch.randn(case["hkv"], 1, D, generator=g, device="cuda")).to(dt)
    return k, torch.randn(shape, dtype=dt, generator=g, device="cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _slopes(hq):
    return 2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": dict(case)}
    {"prompt": _prepare_prompt, "prefix": _prepare_prefix, "quantize": _prepare_quantize,
     "q8": _prepare_q8}[case["kind"]](case, seed, g, st)
    return st


def _prepare_prompt(case, seed, g, st):
    new, ctx = _lens(case, seed)
    lens = [n + c for n, c in zip(new, ctx)]
    xt, hq = DT[case["x"]], case["hq"]
    st["table"], n_pages = _tables(lens, case["page"], g)
    st["k_cache"], st["v_cache"] = _kv(n_pages, case, g, xt)
    rows = sum(new) + case["spare"]
    st["q"] = torch.randn(rows, hq, D, dtype=xt, generator=g, device="cuda")
    st["cu"] = torch.nn.functional.pad(torch.cumsum(_i32(new), 0), (1, 0)).to(torch.int32)
    st["lens"] = _i32(lens)
    # rows behind the last sequence are left as they were
    st["out"] = torch.full((rows, hq, D), 0.5, dtype=xt, device="cuda")
    st["lse"] = torch.full((rows, hq), 0.5, device="cuda")
    st["slopes"] = _slopes(hq) if case["slopes"] else None
    st["starts"] = _i32(_starts(case, seed, lens)) if case["starts"] else None
    st["most_new"], st["longest"] = max(new), max(lens)


def _prepare_prefix(case, seed, g, st):
    prefix, tails, sizes = _lens(case, seed)
    xt, B, hq = DT[case["x"]], case["batch"], case["hq"]
    table, n_pages = _tables(prefix + tails, case["page"], g)
    G = len(prefix)
    st["prefix_table"], st["table"] = table[:G].contiguous(), table[G:].contiguous()
    st["k_cache"], st["v_cache"] = _kv(n_pages, case, g, xt)
    st["q"] = torch.randn(B, hq, D, dtype=xt, generator=g, device="cuda")
    st["cu"] = torch.nn.functional.pad(torch.cumsum(_i32(sizes), 0), (1, 0)).to(torch.int32)
    st["prefix_lens"], st["lens"] = _i32(prefix), _i32(tails)
    st["out"] = torch.empty(B, hq, D, dtype=xt, device="cuda")
    st["lse"] = torch.empty(B, hq, device="cuda")
    st["most_seqs"], st["most_prefix"], st["most_tail"] = max(sizes), max(prefix), max(tails)


def _prepare_quantize(case, seed, g, st):
    T, hkv, P = case["tokens"], case["hkv"], case["page"]
    chan = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    size = torch.exp(0.5 * torch.randn(T, 1, 1, generator=g, device="cuda"))

    def rows(h):
        return (torch.randn(T, h, D, generator=g, device="cuda") * chan * size).to(DT[case["x"]])

    if case["fused"]:  # keys and values are columns of one projection's rows, with the queries before them
        kv = rows(3 * hkv)
        st["k"], st["v"] = kv[:, hkv:2 * hkv], kv[:, 2 * hkv:]
    else:
        st["k"], st["v"] = rows(hkv), rows(hkv)
    n_pages = -(-T // P) + 3
    t = torch.arange(T, device="cuda")
    slots = torch.randperm(n_pages, generator=g, device="cuda")[t // P] * P + t % P
    if case["holes"]:  # rows of a padded batch
        slots = torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, -1, slots)
    st["slots"] = slots.to(torch.int32)
    # what earlier steps wrote
    for name in ("k", "v"):
        old = torch.randn(n_pages, hkv, P, D, generator=g, device="cuda")
        st[name + "_cache"], st[name + "_exp"] = _to_8bit(old)


def _prepare_q8(case, seed, g, st):
    lens = _lens(case, seed)
    xt, B, hq = DT[case["x"]], case["batch"], case["hq"]
    st["table"], n_pages = _tables(lens, case["page"], g)
    k, v = _kv(n_pages, case, g, xt)
    v *= torch.exp(0.5 * torch.randn(n_pages, case["hkv"], case["page"], 1, generator=g, device="cuda")).to(xt)
    st["k_cache"], st["k_exp"] = _to_8bit(k)
    st["v_cache"], st["v_exp"] = _to_8bit(v)
    st["lens"] = _i32(lens)
    st["q"] = torch.randn(B, hq, D, dtype=xt, generator=g, device="cuda")
    st["out"] = torch.empty(B, hq, D, dtype=DT[case["out"]], device="cuda")
    st["lse"] = torch.empty(B, hq, device="cuda")
    st["slopes"] = _slopes(hq) if case["slopes"] else None
    st["starts"] = _i32(_starts(case, seed, lens)) if case["starts"] else None
    st["longest"] = max(1, max(lens))


# ---- the 8-bit format: E4M3 values times a power of two for each token and head ----------------------
def _to_8bit(x):
    """x ~ code * 2^e; e is the smallest exponent with max |x| <= 448 * 2^e, -127 for a row of zeros."""
    x = x.float()
    f, e = torch.frexp(x.abs().amax(-1))  # max = f 2^e, f in [1/2, 1): 448 = 0.875 * 2^9
    e = torch.where(f > 0, e - 9 + (f > 0.875).int(), -127).clamp(min=-127)
    return (x * _power(-e)[..., None]).to(torch.float8_e4m3fn), e.to(torch.int8)


def _from_8bit(code, e):
    return code.float() * _power(e)[..., None]


def _power(e):
    """2^e for whole e of -127..127, exactly: the exponent's bits, and the one number below the normal ones."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).view(torch.float32)


# ---- one pass --------------------------------------------------------------------------------------
def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"prompt": _own_prompt, "prefix": _own_prefix, "quantize": _own_quantize, "q8": _own_q8}[kind](state)
    return {"prompt": _plain_prompt, "prefix": _plain_prefix, "quantize": _plain_quantize, "q8": _plain_q8}[kind](state)


def _own_prompt(s):
    import bit_kv_cache_kvarn_gb300 as kv

    c = s["case"]
    if "workspace" not in s:  # a user's program allocates it once
        n = kv.kvarn_prompt_attention_workspace_size(s["q"].shape[0], c["hq"], c["hkv"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    kv.kvarn_prompt_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["lens"], s["out"], SCALE,
                              s["workspace"], causal=c["causal"], softcap=c["softcap"], slopes=s["slopes"],
                              window=c["window"], kv_starts=s["starts"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_prefix(s):
    import bit_kv_cache_kvarn_gb300 as kv

    c = s["case"]
    if "workspace" not in s:
        n = kv.kvarn_prefix_attention_workspace_size(c["batch"], c["hq"], c["hkv"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    kv.kvarn_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_lens"], s["cu"], s["table"],
                              s["lens"], s["out"], SCALE, s["workspace"], softcap=c["softcap"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_quantize(s):
    import bit_kv_cache_kvarn_gb300 as kv

    kv.kvarn_quantize_kv(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], slot_map=s["slots"])
    return {k: s[k] for k in ("k_cache", "v_cache", "k_exp", "v_exp")}


def _own_q8(s):
    import bit_kv_cache_kvarn_gb300 as kv

    c = s["case"]
    if "workspace" not in s:
        n = kv.kvarn_paged_attention_workspace_size(c["batch"], c["hq"], c["hkv"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    kv.kvarn_paged_attention_q8(s["q"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], s["table"], s["lens"], s["out"],
                                SCALE, s["workspace"], softcap=c["softcap"], slopes=s["slopes"], window=c["window"],
                                kv_starts=s["starts"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _scores(x, c):
    x = x.mul_(SCALE)
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    return x


def _softmax(x):
    """exp(x - its maximum) in x's place, the sum, and the log of the unshifted sum; rows of -inf: 0, 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    return p, z, m + torch.log(z)


def _gather(cache, table, P, n):
    """[rows of the table, heads, n tokens, 128] of a paged cache."""
    pos = torch.arange(n, device="cuda")
    page, off = table.long()[:, pos // P], (pos % P)[None].expand(table.shape[0], n)
    return cache[page, :, off].transpose(1, 2)


def _plain_prompt(s):
    c = s["case"]
    hq, hkv, P, N, L = c["hq"], c["hkv"], c["page"], s["most_new"], s["longest"]
    B, g, T = c["batch"], hq // hkv, s["q"].shape[0]
    cu, lens = s["cu"].long(), s["lens"].long()
    i = torch.arange(N, device="cuda")
    new = cu[1:] - cu[:-1]
    live = i[None] < new[:, None]
    at = (cu[:-1, None] + i[None]).clamp(max=T - 1)
    q = s["q"][at].float().view(B, N, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * g, D)
    x = _scores(torch.matmul(q, _gather(s["k_cache"], s["table"], P, L).float().transpose(2, 3)), c).view(B, hkv, N, g, L)
    j = torch.arange(L, device="cuda")
    pos = (lens - new)[:, None] + i[None]  # [B, N]
    seen = (j[None] < lens[:, None])[:, None].expand(B, N, L)
    if s["starts"] is not None:
        seen = seen & (j[None] >= s["starts"][:, None])[:, None]
    if c["causal"]:
        seen = seen & (j <= pos[:, :, None])
    if c["window"]:
        seen = seen & (j > pos[:, :, None] - c["window"])
    if s["slopes"] is not None:
        x += s["slopes"].view(1, hkv, 1, g, 1) * (j - pos[:, :, None]).float()[:, None, :, None]
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    p, z, lse = _softmax(x)
    v = _gather(s["v_cache"], s["table"], P, L).float()
    v = v.masked_fill(~(j[None] < lens[:, None])[:, None, :, None], 0)
    o = torch.matmul(p.view(B, hkv, N * g, L), v).view(B, hkv, N, g, D)
    o = torch.where(z > 0, o / z, 0).permute(0, 2, 1, 3, 4).reshape(B, N, hq, D)
    s["out"][at[live]] = o[live].to(s["out"].dtype)
    s["lse"][at[live]] = lse.permute(0, 2, 1, 3, 4).reshape(B, N, hq)[live]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_prefix(s):
    c = s["case"]
    hq, hkv, P, M, L, own_L = c["hq"], c["hkv"], c["page"], s["most_seqs"], s["most_prefix"], max(1, s["most_tail"])
    B, G, g = c["batch"], c["groups"], hq // hkv
    cu, lens = s["cu"].long(), s["lens"].long()
    i = torch.arange(M, device="cuda")
    live = i[None] < (cu[1:] - cu[:-1])[:, None]  # [G, M]
    at = (cu[:-1, None] + i[None]).clamp(max=B - 1)
    q = s["q"].float().view(B, hkv, g, D)
    # the prefix: every group's queries against its keys at once
    k = _gather(s["k_cache"], s["prefix_table"], P, L).float()
    x = torch.matmul(q[at].transpose(1, 2).reshape(G, hkv, M * g, D), k.transpose(2, 3))
    x = x.view(G, hkv, M, g, L).transpose(1, 2)[live]  # [B, hkv, g, L]
    j = torch.arange(L, device="cuda")
    group = torch.arange(G, device="cuda")[:, None].expand(G, M)[live]
    hidden = j[None] >= s["prefix_lens"].long()[group][:, None]
    x = _scores(x, c).masked_fill_(hidden[:, None, None], -math.inf)
    # each sequence's own tokens
    t = torch.arange(own_L, device="cuda")
    past = t[None] >= lens[:, None]
    y = torch.matmul(q, _gather(s["k_cache"], s["table"], P, own_L).float().transpose(2, 3))
    y = _scores(y, c).masked_fill_(past[:, None, None], -math.inf)
    p, z, lse = _softmax(torch.cat([x, y], -1))
    pad = torch.zeros(G, M, hkv, g, L, device="cuda")
    pad[live] = p[..., :L]
    v = _gather(s["v_cache"], s["prefix_table"], P, L).float()
    v = v.masked_fill((j[None] >= s["prefix_lens"].long()[:, None])[:, None, :, None], 0)
    o = torch.matmul(pad.transpose(1, 2).reshape(G, hkv, M * g, L), v).view(G, hkv, M, g, D).transpose(1, 2)[live]
    v = _gather(s["v_cache"], s["table"], P, own_L).float().masked_fill(past[:, None, :, None], 0)
    o += torch.matmul(p[..., L:], v)
    s["out"].copy_(torch.where(z > 0, o / z, 0).view(B, hq, D))
    s["lse"].copy_(lse.view(B, hq))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_quantize(s):
    P = s["case"]["page"]
    slots = s["slots"].long()
    rows = (slots >= 0).nonzero()[:, 0]
    page, off = slots[rows] // P, slots[rows] % P
    code, e = _to_8bit(s["k"][rows])
    s["k_cache"].view(torch.uint8)[page, :, off] = code.view(torch.uint8)
    s["k_exp"][page, :, off] = e
    code, e = _to_8bit(s["v"][rows])
    s["v_cache"].view(torch.uint8)[page, :, off] = code.view(torch.uint8)
    s["v_exp"][page, :, off] = e
    return {k: s[k] for k in ("k_cache", "v_cache", "k_exp", "v_exp")}


def _plain_q8(s):
    c = s["case"]
    B, hq, hkv, P = c["batch"], c["hq"], c["hkv"], c["page"]
    g, L = hq // hkv, s["longest"]
    pos, lens = torch.arange(L, device="cuda"), s["lens"].long()
    seen = pos[None] < lens[:, None]
    if c["window"]:
        seen &= pos[None] >= lens[:, None] - c["window"]
    if s["starts"] is not None:
        seen &= pos[None] >= s["starts"][:, None]

    def rows(name):
        code = _gather(s[name + "_cache"].view(torch.uint8), s["table"], P, L)
        e = _gather(s[name + "_exp"], s["table"], P, L)
        return _from_8bit(code.contiguous().view(torch.float8_e4m3fn), e)

    x = _scores(torch.matmul(s["q"].view(B, hkv, g, D).float(), rows("k").transpose(2, 3)), c)
    if s["slopes"] is not None:
        x = x + s["slopes"].view(1, hkv, g, 1) * (pos[None] - (lens[:, None] - 1)).float()[:, None, None]
    p, z, lse = _softmax(x.masked_fill_(~seen[:, None, None], -math.inf))
    o = torch.matmul(p, rows("v").masked_fill_(~seen[:, None, :, None], 0))
    s["out"].copy_(torch.where(z > 0, o / z, 0).view(B, hq, D))
    s["lse"].copy_(lse.view(B, hq))
    return {"out": s["out"], "lse": s["lse"]}


# ---- what a pass cannot do without -----------------------------------------------------------------
def _triangle(first, last, window):
    """Sum over the positions first .. last of the keys that a causal row sees, and the first key that any does."""
    if not window:
        return (first + last + 2) * (last - first + 1) // 2, 0
    ramp = max(0, min(last + 1, window) - first)  # rows that see fewer than the window's keys or just that many
    return ramp * (2 * first + ramp + 1) // 2 + (last - first + 1 - ramp) * window, max(0, first + 1 - window)


def work(case):
    hkv = case["hkv"]
    if case["kind"] == "quantize":
        T = case["tokens"] * (0.8 if case["holes"] else 1)
        return {"bytes": 2 * T * hkv * (D * ((4 if case["x"] == "fp32" else 2) + 1) + 1) + 4 * case["tokens"],
                "flops": 2 * T * hkv * D * 2}
    hq, P = case["hq"], case["page"]
    if case["kind"] == "prompt":
        new, ctx = _lens(case, 0)
        starts = _starts(case, 0, [n + c for n, c in zip(new, ctx)]) if case["starts"] else [0] * len(new)
        pairs = keys = 0
        for n, c, s in zip(new, ctx, starts):
            if case["causal"]:
                f = max(0, c - s)  # rows before the first visible key see nothing
                if c + n > s:
                    seen, first = _triangle(f, c + n - 1 - s, case["window"])
                    pairs, keys = pairs + seen, keys + c + n - s - first
            else:
                pairs, keys = pairs + n * (c + n - s), keys + c + n - s
        rows = sum(new) * hq
        return {"bytes": keys * hkv * 4 * D + rows * (4 * D + 4) + len(new) * 8 + 4 * keys / P, "flops": pairs * hq * 4 * D}
    if case["kind"] == "prefix":
        prefix, tails, sizes = _lens(case, 0)
        rows = case["batch"] * hq
        return {"bytes": (sum(prefix) + sum(tails)) * (hkv * 4 * D + 4 / P) + rows * (4 * D + 4) + 4 * (case["batch"] + 2 * len(sizes)),
                "flops": (sum(a * b for a, b in zip(prefix, sizes)) + sum(tails)) * hq * 4 * D}
    lens = _lens(case, 0)
    starts = _starts(case, 0, lens) if case["starts"] else [0] * len(lens)
    seen = sum(n - min(n, max(s, n - case["window"] if case["window"] else 0)) for n, s in zip(lens, starts))
    rows = case["batch"] * hq
    return {"bytes": seen * hkv * 2 * (D + 1) + rows * (D * (2 + (4 if case["out"] == "fp32" else 2)) + 4) + 4 * case["batch"] + 4 * seen / P,
            "flops": seen * hq * 4 * D}


# ---- the same in 64 bits -----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "prefix": _exact_prefix, "quantize": _exact_quantize, "q8": _exact_q8}[case["kind"]](case, seed, s)


def _attend(q, k, v, cap, bias=None):
    """Rows q [heads, rows, 128] over keys [heads, n, 128] in 64 bits; bias broadcasts over [heads, rows, n]."""
    x = (q @ k.transpose(1, 2)) / math.sqrt(D)
    if cap:
        x = cap * torch.tanh(x / cap)
    if bias is not None:
        x = x + bias
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[..., None]) @ v, lse


def _dense(cache, row, lo, n, P):
    """Tokens lo .. n of one sequence: [heads, n - lo, 128] in 64 bits."""
    pages = row[:-(-n // P)].long()
    return cache[pages].transpose(0, 1).reshape(cache.shape[1], -1, D)[:, lo:n].double()


def _exact_prompt(case, seed, s):
    new, ctx = _lens(case, seed)
    hq, hkv, P, w = case["hq"], case["hkv"], case["page"], case["window"]
    g = hq // hkv
    starts = _starts(case, seed, [n + c for n, c in zip(new, ctx)]) if case["starts"] else [0] * len(new)
    out, lse, row = s["out"].double(), s["lse"].double(), 0
    out[:sum(new)], lse[:sum(new)] = 0, -math.inf
    for b, (n, c, s0) in enumerate(zip(new, ctx, starts)):
        k, v = (_dense(s[x], s["table"][b], s0, c + n, P) for x in ("k_cache", "v_cache"))
        for i in range(0, n, 512):
            e = min(n, i + 512)
            pos = torch.arange(c + i, c + e, device="cuda")
            lo = max(s0, c + i + 1 - w) if w else s0
            hi = c + e if case["causal"] else c + n
            if lo >= hi:
                continue
            q = s["q"][row + i:row + e].double().view(e - i, hkv, g, D).permute(1, 0, 2, 3).reshape(hkv, -1, D)
            ahead = torch.arange(lo, hi, device="cuda") - pos[:, None]  # key - query
            bias = torch.zeros(1, 1, *ahead.shape, dtype=torch.float64, device="cuda")
            if s["slopes"] is not None:
                bias = s["slopes"].double().view(hkv, g, 1, 1) * ahead
            bad = (ahead > 0) & case["causal"]
            if w:
                bad = bad | (ahead <= -w)
            bias = bias.masked_fill(bad, -math.inf).transpose(1, 2)  # [hkv or 1, rows, g or 1, keys]
            bias = bias.expand(-1, -1, g, -1).reshape(bias.shape[0], -1, hi - lo)
            o, z = _attend(q, k[:, lo - s0:hi - s0], v[:, lo - s0:hi - s0], case["softcap"], bias)
            out[row + i:row + e] = o.view(hkv, e - i, g, D).transpose(0, 1).reshape(e - i, hq, D)
            lse[row + i:row + e] = z.view(hkv, e - i, g).transpose(0, 1).reshape(e - i, hq)
        row += n
    return {"out": out, "lse": lse}


def _exact_prefix(case, seed, s):
    prefix, tails, sizes = _lens(case, seed)
    hq, hkv, P = case["hq"], case["hkv"], case["page"]
    out = torch.zeros(len(tails), hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(len(tails), hq, dtype=torch.float64, device="cuda")
    b = 0
    for i, (n, m) in enumerate(zip(prefix, sizes)):
        k, v = (_dense(s[x], s["prefix_table"][i], 0, n, P) for x in ("k_cache", "v_cache"))
        for _ in range(m):
            t = tails[b]
            k1, v1 = (torch.cat([a, _dense(s[x], s["table"][b], 0, t, P)], 1) for a, x in ((k, "k_cache"), (v, "v_cache")))
            o, z = _attend(s["q"][b].double().view(hkv, hq // hkv, D), k1, v1, case["softcap"])
            out[b], lse[b] = o.reshape(hq, D), z.reshape(hq)
            b += 1
    return {"out": out, "lse": lse}


def _exact_quantize(case, seed, s):
    P, slots = case["page"], s["slots"].long()
    powers = torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device="cuda")

    def two(e):  # a computed power may be off by a last digit, which would move ties
        return powers[e.long() + 160]

    made = {}
    for name in ("k", "v"):
        x = s[name].double()
        top = x.abs().amax(-1)
        e = torch.ceil(torch.log2(top / 448)).clamp(min=-127)
        e = e + (top > 448 * two(e)).int()  # so may the logarithm
        e = e - ((top <= 448 * two(e - 1)) & (e > -127)).int()
        y = x / two(e)[..., None]
        near = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
        near = near - (two(near) > y.abs().clamp(min=2.0 ** -6)).int()
        near = near + (two(near + 1) <= y.abs()).int()
        step = two(near - 3)
        y = torch.round(y / step) * step
        cache, exps = s[name + "_cache"].double(), s[name + "_exp"].clone()
        keep = slots >= 0
        at = slots[keep]
        cache.transpose(1, 2)[at // P, at % P] = y[keep]
        exps.transpose(1, 2)[at // P, at % P] = e[keep].to(torch.int8)
        made[name + "_cache"], made[name + "_exp"] = cache, exps
    return made


def _exact_q8(case, seed, s):
    lens = _lens(case, seed)
    hq, hkv, P = case["hq"], case["hkv"], case["page"]
    starts = _starts(case, seed, lens) if case["starts"] else [0] * len(lens)
    out = torch.zeros(len(lens), hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens), hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        lo = max(starts[b], n - case["window"] if case["window"] else 0)
        if lo >= n:
            continue
        pages = s["table"][b, :-(-n // P)].long()
        kv = []
        for name in ("k", "v"):
            code = s[name + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
            x = code * 2.0 ** s[name + "_exp"][pages].double()[..., None]
            kv.append(x.transpose(0, 1).reshape(hkv, -1, D)[:, lo:n])
        bias = None
        if s["slopes"] is not None:
            bias = s["slopes"].double().view(hkv, -1, 1) * torch.arange(lo - n + 1, 1, dtype=torch.float64, device="cuda")
        o, z = _attend(s["q"][b].double().view(hkv, hq // hkv, D), *kv, case["softcap"], bias)
        out[b], lse[b] = o.reshape(hq, D), z.reshape(hq)
    return {"out": out, "lse": lse}
