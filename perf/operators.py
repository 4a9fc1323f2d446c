"""The paged-cache operators of a serving step, as a benchmark and a check see them.

A step of a server that keeps its requests' keys and values in 64-token pages
(64 query heads that share one K and one V head of dimension 256) runs

    reserve   pages for the tokens that arrive, the slot of every token
    append    the tokens' K and V rows, scattered to their slots
    prefix    decode attention in which the sequences of a group share a
              prefix, whose pages are read once for the whole group
    release   the pages of the requests that ended

`run` computes each of them either by elementary torch operations (`own` is
false) or by the calls of the library (`own` is true), on the same inputs.
"""
import math

import numpy as np
import torch

own = False

HEADS, DIM, PAGE = 64, 256, 64
SCALE = 1.0 / 16.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of requests behind one system prompt, a few tokens into their answers: latency counts
        dict(name="prefix_small", op="prefix", kv="bf16", sizes="4", pages="16", lo=1, hi=70, empty=0, short=0, seed=1),
        # one long instruction shared by an ordinary decode batch
        dict(name="prefix_one", op="prefix", kv="bf16", sizes="32", pages="128", lo=1, hi=512, empty=0, short=0, seed=2),
        # several system prompts in one batch, odd group sizes, requests of their own (no shared pages), padded slots
        dict(name="prefix_groups", op="prefix", kv="bf16", sizes="7,1,19,12,2", pages="72,40,130,0,17", lo=1, hi=1500,
             empty=2, short=1, seed=3),
        # many samples of one long document
        dict(name="prefix_large", op="prefix", kv="bf16", sizes="128", pages="512", lo=256, hi=2048, empty=0, short=0, seed=4),
        # two long prompts on an 8-bit cache
        dict(name="prefix_fp8", op="prefix", kv="fp8", sizes="39,25", pages="256,97", lo=1, hi=1024, empty=1, short=0, seed=5),
        # one new token for each request of a decode batch: latency counts
        dict(name="append_decode", op="append", kv="bf16", rows=128, pad=0, fused=True, pages=4096, seed=7),
        # the prompts of a prefill step, K and V beside each other in the projection's rows, padded to a fixed row count
        dict(name="append_prefill", op="append", kv="bf16", rows=16200, pad=184, fused=True, pages=4096, seed=8),
        # a large prefill step into an 8-bit cache
        dict(name="append_fp8", op="append", kv="fp8", rows=65000, pad=536, fused=False, pages=2048, seed=9),
        # tables and slots of a decode step: one new token each
        dict(name="reserve_decode", op="reserve", batch=128, max_pages=512, held=16384, new=1, pad=0, seed=10),
        # tables and slots of a step that mixes decode with long prompts
        dict(name="reserve_prefill", op="reserve", batch=1000, max_pages=512, held=8000, new=500, pad=1000, seed=11),
        # a sixteenth of a large batch has ended
        dict(name="release", op="release", batch=1000, max_pages=512, held=30000, share=0.0625, keep=16, seed=12),
        # half of a small batch has ended
        dict(name="release_half", op="release", batch=64, max_pages=128, held=8000, share=0.5, keep=5, seed=13),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prefix", "append", "reserve", "release"])
    seed = rng.randrange(1 << 30)
    if op == "prefix":
        groups = rng.choice([1, 1, 2, 3, 5])
        sizes = [_log(rng, 1, 128 // groups) for _ in range(groups)]
        pages = [0 if groups > 1 and rng.random() < 0.15 else _log(rng, 4, 512 // groups) for _ in range(groups)]
        hi = _log(rng, 1, 2048)
        return dict(op=op, kv=rng.choice(["bf16", "fp8"]), sizes=",".join(map(str, sizes)), pages=",".join(map(str, pages)),
                    lo=rng.randint(1, hi), hi=hi, empty=rng.choice([0, 0, 1]), short=rng.choice([0, 0, 1]), seed=seed)
    if op == "append":
        rows = _log(rng, 1, 60000)
        return dict(op=op, kv=rng.choice(["bf16", "fp8"]), rows=rows, pad=rng.choice([0, rng.randint(1, 200)]),
                    fused=rng.random() < 0.5, pages=_log(rng, rows // PAGE + 8, 4096), seed=seed)
    if op == "reserve":
        return dict(op=op, batch=_log(rng, 1, 1000), max_pages=512, held=_log(rng, 1, 16000),
                    new=rng.choice([1, _log(rng, 2, 900)]), pad=rng.randint(0, 500), seed=seed)
    return dict(op=op, batch=_log(rng, 2, 1000), max_pages=512, held=_log(rng, 64, 30000), share=rng.choice([0.05, 0.2, 0.5]),
                keep=rng.choice([0, 3, 16]), seed=seed)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _layout(case):
    """What the host of a server knows of its step: lengths, tables, counts. From the case alone."""
    rng = np.random.default_rng(case["seed"])
    if case["op"] == "prefix":
        sizes, pages = _ints(case["sizes"]), _ints(case["pages"])
        batch = sum(sizes)
        group = np.repeat(np.arange(len(sizes)), sizes)
        shared = np.array(pages)[group]
        suffix = rng.integers(case["lo"], case["hi"] + 1, batch)
        lens = shared * PAGE + suffix
        pick = rng.permutation(batch)
        for b in pick[:case["short"]]:  # a request that ends inside its group's prefix
            lens[b] = rng.integers(1, max(2, shared[b] * PAGE))
        for b in pick[case["short"]:case["short"] + case["empty"]]:  # a padded slot of the batch
            lens[b] = 0
        own_pages = np.maximum(0, -(-lens // PAGE) - shared)
        total = int(sum(pages) + own_pages.sum()) + 7
        order = rng.permutation(total)
        table = np.zeros((batch, int((shared + own_pages).max()) + 1), np.int32)
        at = int(sum(pages))
        first = np.concatenate([[0], np.cumsum(pages)])
        for b in range(batch):
            g = group[b]
            table[b, :shared[b]] = order[first[g]:first[g] + shared[b]]
            table[b, shared[b]:shared[b] + own_pages[b]] = order[at:at + own_pages[b]]
            at += int(own_pages[b])
        starts = np.concatenate([[0], np.cumsum(sizes)])
        return dict(batch=batch, lens=lens, table=table, total=total, starts=starts, shared=shared, group=group)
    if case["op"] == "append":
        slots = np.full(case["rows"] + case["pad"], -1, np.int64)
        slots[:case["rows"]] = rng.permutation(case["pages"] * PAGE)[:case["rows"]]
        return dict(slots=slots)
    batch, cap = case["batch"], case["max_pages"]
    lens = rng.integers(0, min(case["held"], cap * PAGE - 1) + 1, batch)
    if case["op"] == "reserve":
        lens = np.minimum(lens, cap * PAGE - case["new"])
        new = rng.integers(0, case["new"] + 1, batch) if case["new"] > 1 else np.ones(batch, np.int64)
        used = -(-lens // PAGE)
        need = -(-(lens + new) // PAGE) - used
        spare = int(need.sum()) + 64
        out = dict(new=new, extra=spare)
    else:
        ended = rng.random(batch) < case["share"]
        ended[int(rng.integers(batch))] = True
        used = -(-lens // PAGE)
        out = dict(ended=ended, keep=np.minimum(case["keep"], rng.integers(0, case["keep"] + 1, batch)), extra=64)
    total = int(used.sum()) + out["extra"]
    order = rng.permutation(total)
    table = np.full((batch, cap), -1, np.int32)
    ends = np.cumsum(used)
    for b in range(batch):
        table[b, :used[b]] = order[ends[b] - used[b]:ends[b]]
    free = np.zeros(total, np.int32)
    free[:out["extra"]] = order[ends[-1]:]
    return dict(out, lens=lens, table=table, free=free, total=total)


def work(case):
    at = _layout(case)
    if case["op"] == "prefix":
        pages = _ints(case["pages"])
        # positions of the prefixes that some request of the group attends to, each once, and every suffix
        seen = sum(int(min(p * PAGE, at["lens"][at["group"] == g].max())) for g, p in enumerate(pages))
        keys = seen + int(np.maximum(0, at["lens"] - at["shared"] * PAGE).sum())
        row = 2 * DIM * 2 if case["kv"] == "bf16" else 2 * DIM + 8
        rows = at["batch"] * HEADS
        return {"bytes": keys * row + 2 * rows * DIM * 2 + rows * 4, "flops": 4 * HEADS * DIM * int(at["lens"].sum())}
    if case["op"] == "append":
        out = 2 * DIM * 2 if case["kv"] == "bf16" else 2 * DIM + 8
        return {"bytes": case["rows"] * (2 * DIM * 2 + out) + 8 * (case["rows"] + case["pad"]), "flops": 0}
    if case["op"] == "reserve":
        batch, tokens = case["batch"], int(at["new"].sum())
        touched = int((-(-(at["lens"] + at["new"]) // PAGE) - at["lens"] // PAGE).sum())
        return {"bytes": 16 * batch + 8 * (tokens + case["pad"]) + 8 * touched, "flops": 0}
    moved = int(np.maximum(0, -(-at["lens"] // PAGE) - at["keep"])[at["ended"]].sum())
    return {"bytes": 16 * case["batch"] + 8 * moved, "flops": 0}


# ------------------------------------------------------------------ inputs
def _rows(shape, gen):
    """K or V rows as projections give them: a few strong channels, token norms that vary."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x[..., :4] *= 3.0
    return (x * torch.exp(0.3 * torch.randn(shape[:-1], generator=gen, device="cuda")).unsqueeze(-1)).bfloat16()


def _quantised(x):
    x = x.float()
    top = x.abs().amax(-1)
    s = torch.where(top > 0, top / torch.full_like(top, 448.0), torch.ones_like(top))  # by a tensor: a true division
    return (x / s.unsqueeze(-1)).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    at = _layout(case)
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    ints = lambda a, t=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
    st = dict(case=case)
    if case["op"] == "prefix":
        batch = at["batch"]
        st.update(batch=batch, host=at, q=torch.randn((batch, HEADS, DIM), generator=gen, device="cuda").bfloat16(),
                  table=ints(at["table"]), lens=ints(at["lens"]), starts=ints(at["starts"]),
                  pages=ints(_ints(case["pages"])), out=torch.zeros((batch, HEADS, DIM), dtype=torch.bfloat16, device="cuda"),
                  lse=torch.zeros((batch, HEADS), device="cuda"))
        st["kc"], st["vc"] = (_rows((at["total"], PAGE, DIM), gen) for _ in range(2))
        if case["kv"] == "fp8":
            (st["kc"], st["ks"]), (st["vc"], st["vs"]) = _quantised(st["kc"]), _quantised(st["vc"])
        st["hint"] = (max(_ints(case["pages"])) * PAGE, int(max(1, case["hi"])))
    elif case["op"] == "append":
        n, pool = case["rows"] + case["pad"], case["pages"]
        if case["fused"]:  # one projection's output, K beside V
            kv = _rows((n, 2, DIM), gen)
            st.update(k=kv[:, 0], v=kv[:, 1])
        else:
            st.update(k=_rows((n, DIM), gen), v=_rows((n, DIM), gen))
        st["slots"] = ints(at["slots"], torch.int64)
        if case["kv"] == "bf16":
            st["kc"], st["vc"] = (torch.zeros((pool, PAGE, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        else:
            st["kc"], st["vc"] = (torch.zeros((pool, PAGE, DIM), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
            st["ks"], st["vs"] = (torch.ones((pool, PAGE), device="cuda") for _ in range(2))
    else:
        # the pages of another seed are other pages
        names = torch.randperm(at["total"], generator=gen, device="cuda").int()
        table, free = ints(at["table"]), ints(at["free"])
        st.update(total=at["total"], table=torch.where(table >= 0, names[table.clamp(min=0).long()], table),
                  free=names[free.long()], lens=ints(at["lens"]), nfree=ints([at["extra"]]),
                  lens_out=torch.zeros(case["batch"], dtype=torch.int32, device="cuda"),
                  nfree_out=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if case["op"] == "reserve":
            most = int(at["new"].sum()) + case["pad"]
            st.update(new=ints(at["new"]), most=most, slots=torch.zeros(most, dtype=torch.int64, device="cuda"),
                      starts=torch.zeros(case["batch"] + 1, dtype=torch.int32, device="cuda"))
        else:
            st.update(ended=ints(at["ended"]), keep=ints(at["keep"]))
    if own:
        from decode_attention_mfa_gb300 import capi
        need = 256
        if case["op"] == "prefix":
            need = capi.mfa_decode_prefix_workspace_bytes(st["batch"], len(at["starts"]) - 1, *st["hint"])
        st["ws_bytes"], st["ws"] = need, torch.empty(need, dtype=torch.uint8, device="cuda")
        capi.mfa_workspace_init(st["ws"], need)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _part(q, k, v, seen):
    """exp-sum attention of rows q [.., r, d] over keys k, v [.., t, d], of which `seen` [.., r or 1, t] count: O, maximum, sum."""
    s = q @ k.transpose(-1, -2) * SCALE
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    return p @ v, m, p.sum(-1, keepdim=True)


def _rows_of(st, pages):
    """K and V rows of a table of pages, in 32 bits."""
    pages = pages.long()
    if "ks" in st:
        k, v = (st[c].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() for c in ("kc", "vc"))
        k, v = k * st["ks"][pages].unsqueeze(-1), v * st["vs"][pages].unsqueeze(-1)
    else:
        k, v = st["kc"][pages].float(), st["vc"][pages].float()
    return k.flatten(-3, -2), v.flatten(-3, -2)


def _plain_group(st, b0, b1, pages):
    n = b1 - b0
    q = st["q"][b0:b1].float()
    lens = st["lens"][b0:b1].long()
    longest = max(1, int(st["host"]["lens"][b0:b1].max()) - pages * PAGE)
    k, v = _rows_of(st, st["table"][b0:b1, pages:pages - (-longest // PAGE)])
    left = (lens - pages * PAGE).view(n, 1, 1)
    o, m, l = _part(q, k, v, torch.arange(k.shape[1], device="cuda") < left)
    if pages:  # the shared pages: one product for all of the group's rows
        k, v = _rows_of(st, st["table"][b0, :pages])
        seen = torch.arange(pages * PAGE, device="cuda") < lens.repeat_interleave(HEADS, output_size=n * HEADS).unsqueeze(-1)
        o2, m2, l2 = (x.view(n, HEADS, -1) for x in _part(q.reshape(n * HEADS, DIM), k, v, seen))
        top = torch.maximum(m, m2)
        base = torch.where(top > -math.inf, top, torch.zeros_like(top))
        w, w2 = torch.exp(m - base), torch.exp(m2 - base)
        o, l, m = o * w + o2 * w2, l * w + l2 * w2, top
    some = l > 0
    out = torch.where(some, o / torch.where(some, l, torch.ones_like(l)), torch.zeros_like(o))
    lse = torch.where(some, m + torch.log(torch.where(some, l, torch.ones_like(l))), m)
    return out.bfloat16(), lse.squeeze(-1)


def _plain_prefix(st):
    starts, pages = st["host"]["starts"].tolist(), _ints(st["case"]["pages"])
    parts = [_plain_group(st, b0, b1, p) for b0, b1, p in zip(starts, starts[1:], pages)]
    return {"out": torch.cat([o for o, _ in parts]), "lse": torch.cat([x for _, x in parts])}


def _own_prefix(st):
    from decode_attention_mfa_gb300 import capi
    args = [st["table"], st["lens"], st["starts"], st["pages"], len(st["pages"]), st["out"], st["lse"], SCALE, st["batch"],
            st["table"].shape[1], st["kc"].shape[0], *st["hint"], st["ws"], st["ws_bytes"]]
    if "ks" in st:
        capi.mfa_decode_attention_prefix_fp8(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], *args)
    else:
        capi.mfa_decode_attention_prefix(st["q"], st["kc"], st["vc"], *args)
    return {"out": st["out"], "lse": st["lse"]}


def _plain_append(st):
    rows = st["slots"] >= 0
    at = st["slots"][rows]
    new = {}
    if "ks" in st:
        for x, c, s in (("k", "kc", "ks"), ("v", "vc", "vs")):
            codes, scale = _quantised(st[x][rows])
            st[c].view(torch.uint8).view(-1, DIM)[at] = codes.view(torch.uint8)
            st[s].view(-1)[at] = scale
            new[s] = st[s]
    else:
        st["kc"].view(-1, DIM)[at] = st["k"][rows]
        st["vc"].view(-1, DIM)[at] = st["v"][rows]
    return {"k": st["kc"], "v": st["vc"], **new}


def _own_append(st):
    from decode_attention_mfa_gb300 import capi
    k, v = st["k"], st["v"]
    if "ks" in st:
        capi.mfa_kv_append_slots_fp8(k, v, k.stride(0), v.stride(0), st["slots"], len(k), st["kc"], st["vc"], st["ks"],
                                     st["vs"], st["kc"].shape[0], st["ws"])
        return {"k": st["kc"], "v": st["vc"], "ks": st["ks"], "vs": st["vs"]}
    capi.mfa_kv_append_slots(k, v, k.stride(0), v.stride(0), st["slots"], len(k), st["kc"], st["vc"], st["kc"].shape[0],
                             st["ws"])
    return {"k": st["kc"], "v": st["vc"]}


def _plain_reserve(st):
    lens, new, table = st["lens"].long(), st["new"].long(), st["table"]
    held, after = (lens + PAGE - 1) // PAGE, (lens + new + PAGE - 1) // PAGE
    need = torch.cumsum(after - held, 0)
    starts = torch.cat([torch.zeros_like(need[:1]), torch.cumsum(new, 0)])
    j = torch.arange(table.shape[1], device="cuda")
    take = st["nfree"] - 1 - ((need - (after - held) - held).unsqueeze(1) + j)  # from the top of the stack
    fresh = (j >= held.unsqueeze(1)) & (j < after.unsqueeze(1))
    table.copy_(torch.where(fresh, st["free"][take.clamp(0, st["free"].numel() - 1)], table))
    i = torch.arange(st["most"], device="cuda")
    b = torch.searchsorted(starts[1:], i, right=True).clamp(max=len(lens) - 1)
    pos = lens[b] + i - starts[b]
    slots = table[b, (pos // PAGE).clamp(max=table.shape[1] - 1)].long() * PAGE + pos % PAGE
    return {"table": table, "slots": torch.where(i < starts[-1], slots, torch.full_like(slots, -1)), "starts": starts.int(),
            "lens": (lens + new).int(), "nfree": (st["nfree"] - need[-1:]).int()}


def _own_reserve(st):
    from decode_attention_mfa_gb300 import capi
    capi.mfa_reserve_pages(st["new"], st["lens"], st["table"], st["free"], st["nfree"], st["case"]["batch"],
                           st["table"].shape[1], st["total"], st["most"], st["starts"], st["slots"], st["lens_out"],
                           st["nfree_out"], st["ws"])
    return {"table": st["table"], "slots": st["slots"], "starts": st["starts"], "lens": st["lens_out"],
            "nfree": st["nfree_out"]}


def _plain_release(st):
    lens, table, free = st["lens"].long(), st["table"], st["free"]
    held = (lens + PAGE - 1) // PAGE
    kept = torch.minimum(st["keep"].long(), held)
    count = torch.where(st["ended"] != 0, held - kept, torch.zeros_like(held))
    upto = torch.cumsum(count, 0)
    j = torch.arange(table.shape[1], device="cuda")
    gone = (j >= kept.unsqueeze(1)) & (j < (kept + count).unsqueeze(1))
    at = st["nfree"] + (upto - count - kept).unsqueeze(1) + j
    free[at[gone]] = table[gone]
    left = torch.where(st["ended"] != 0, torch.minimum(lens, kept * PAGE), lens)
    return {"free": free, "lens": left.int(), "nfree": (st["nfree"] + upto[-1:]).int()}


def _own_release(st):
    from decode_attention_mfa_gb300 import capi
    capi.mfa_release_pages(st["ended"], st["keep"], st["lens"], st["table"], st["free"], st["nfree"], st["case"]["batch"],
                           st["table"].shape[1], st["total"], st["lens_out"], st["nfree_out"], st["ws"])
    return {"free": st["free"], "lens": st["lens_out"], "nfree": st["nfree_out"]}


_plain = dict(prefix=_plain_prefix, append=_plain_append, reserve=_plain_reserve, release=_plain_release)
_own = dict(prefix=_own_prefix, append=_own_append, reserve=_own_reserve, release=_own_release)


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    st, at = prepare(case, seed), _layout(case)
    if case["op"] == "prefix":
        outs, lses = [], []
        for b in range(at["batch"]):
            n = int(at["lens"][b])
            if n == 0:  # nothing to attend to
                outs.append(torch.zeros((HEADS, DIM), dtype=torch.float64, device="cuda"))
                lses.append(torch.full((HEADS,), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            ids = st["table"][b, :-(-n // PAGE)].long()
            k, v = (st[c].view(torch.int16 if case["kv"] == "bf16" else torch.uint8)[ids].view(st[c].dtype).double()
                    .reshape(-1, DIM)[:n] for c in ("kc", "vc"))
            if "ks" in st:
                k = k * st["ks"][ids].double().reshape(-1, 1)[:n]
                v = v * st["vs"][ids].double().reshape(-1, 1)[:n]
            logits = torch.einsum("hd,td->ht", st["q"][b].double(), k) * SCALE
            lse = torch.logsumexp(logits, 1)
            outs.append(torch.exp(logits - lse[:, None]) @ v)
            lses.append(lse)
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    if case["op"] == "append":
        got = {"k": torch.zeros((case["pages"] * PAGE, DIM), dtype=torch.float64, device="cuda")}
        got["v"] = torch.zeros_like(got["k"])
        if case["kv"] == "fp8":
            got.update(ks=torch.ones(case["pages"] * PAGE, dtype=torch.float64, device="cuda"),
                       vs=torch.ones(case["pages"] * PAGE, dtype=torch.float64, device="cuda"))
        at = st["slots"][:case["rows"]]
        for x in "kv":
            y = st[x][:case["rows"]].double()
            if case["kv"] == "fp8":
                top = y.abs().max(1).values
                s = torch.where(top > 0, top / 448.0, torch.ones_like(top)).float().double()  # the scale is held in 32 bits
                z = (y / s[:, None]).float().double()  # the quotient as well
                # the nearest E4M3 value: 3 bits behind the leading one, steps of 2^-9 below 2^-6
                step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
                y = (torch.round(z / step) * step).clamp(-448.0, 448.0)
                got[x + "s"][at] = s
            got[x][at] = y
        shape = lambda t: t.view(case["pages"], PAGE, *t.shape[1:])  # noqa: E731
        return {name: shape(t) for name, t in got.items()}
    return None  # whole numbers only
