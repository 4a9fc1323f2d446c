"""Prompts in chunks over a paged cache, and a 4-bit cache written and read back, as a benchmark and a check see them.

A server that takes prompts in chunks, between the decode steps of its other requests, runs per layer (64 query heads
that share one K and one V head of dimension 256, 64-token pages)

    chunk   attention of every sequence's new tokens over all that its pages hold, causal among the new ones
    write   the new tokens' K and V rows to 4 bits at their slots, and the values that the cache now holds, read back
            (what goes on to a server that decodes, or into another cache)
    read    a range of positions of each sequence out of a paged cache, as bf16 rows

`run` computes each of them either by elementary torch operations (`own` is false) or by the calls of the library (`own`
is true), on the same inputs.
"""
import math

import numpy as np
import torch

own = False

HEADS, DIM, PAGE = 64, 256, 64
SCALE = 1.0 / 16.0
CODE_BYTES = {"bf16": 2 * DIM, "fp8": DIM, "fp4": DIM // 2}  # of a K or V row


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the end of a short question behind a system prompt, nothing else in the step: latency counts
        dict(name="chunk_small", op="chunk", kv="bf16", new="23", held="900", ones=0, reach=0, idle=0, pad=0, seed=1),
        # a step that mixes one chunk of a prompt with the decode tokens of other requests, rows padded to a fixed count
        dict(name="chunk_mixed", op="chunk", kv="bf16", new="961", held="2500", ones=63, reach=9000, idle=2, pad=30, seed=2),
        # whole prompts of odd lengths, nothing cached before them
        dict(name="chunk_prompts", op="chunk", kv="bf16", new="7001,1189,300,2047,517", held="0,0,0,0,0", ones=0, reach=0, idle=0,
             pad=0, seed=3),
        # one chunk of a document of 64K tokens: the largest
        dict(name="chunk_long", op="chunk", kv="bf16", new="2048", held="63488", ones=0, reach=0, idle=0, pad=0, seed=4),
        # an 8-bit cache: further turns of two conversations, and decode tokens
        dict(name="chunk_fp8", op="chunk", kv="fp8", new="1500,811", held="16100,5005", ones=17, reach=6000, idle=1, pad=12, seed=5),
        # a 4-bit cache: the same kind of step at half the bytes
        dict(name="chunk_fp4", op="chunk", kv="fp4", new="1021,640", held="24000,0", ones=9, reach=4000, idle=0, pad=0, seed=6),
        # one new token of each request of a decode batch into a 4-bit cache: latency counts
        dict(name="write_decode", op="write", kv="fp4", new="", held="", ones=128, reach=4096, idle=0, pad=0, seed=7),
        # a large prefill step into a 4-bit cache, K and V beside each other in the projection's rows
        dict(name="write_prompts", op="write", kv="fp4", new="30001,20011,14000", held="0,777,64", ones=0, reach=0, idle=0,
             pad=536, seed=8),
        # the last tokens of some requests, out of a bf16 cache: latency counts
        dict(name="read_tail", op="read", kv="bf16", new="64,7,130", held="500,3,0", ones=0, reach=0, idle=1, pad=3, seed=9),
        # prompts on an 8-bit cache, for a server that decodes them
        dict(name="read_fp8", op="read", kv="fp8", new="32000,9001,17777", held="0,0,100", ones=0, reach=0, idle=0, pad=0, seed=10),
        # one long prompt out of a 4-bit cache
        dict(name="read_fp4", op="read", kv="fp4", new="65111", held="33", ones=0, reach=0, idle=0, pad=0, seed=11),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op, seed = rng.choice(["chunk", "chunk", "chunk", "write", "read"]), rng.randrange(1 << 30)
    ones = rng.choice([0, 0, _log(rng, 1, 128)])
    prompts = rng.choice([1, 1, 2, 3, 6] if ones == 0 else [0, 1, 1, 2, 4])
    most_new, most_held = (4096, 60000) if op == "chunk" else (30000, 30000)
    most_new //= max(1, prompts)
    new = [_log(rng, 1, most_new) for _ in range(prompts)]
    # what a chunk stands behind: nothing, or so much that all of them cost no more than the largest listed case
    room = [max(1, min(most_held, int(1.2e8 / max(1, prompts) / n) - n)) for n in new]
    held = [0 if rng.random() < 0.3 else _log(rng, 1, r) for r in room]
    return dict(op=op, kv="fp4" if op == "write" else rng.choice(["bf16", "fp8", "fp4"]), new=",".join(map(str, new)),
                held=",".join(map(str, held)), ones=ones, reach=_log(rng, 1, 9000), idle=rng.choice([0, 0, 1, 3]),
                pad=rng.choice([0, rng.randint(1, 200)]), seed=seed)


def _ints(text):
    return [int(x) for x in text.split(",") if x]


def _layout(case):
    """What the host of a server knows of its step: tables, lengths before and after, rows. From the case alone."""
    rng = np.random.default_rng(case["seed"])
    new = np.array(_ints(case["new"]) + [1] * case["ones"] + [0] * case["idle"], np.int64)
    held = np.concatenate([np.array(_ints(case["held"]), np.int64),
                           rng.integers(0, case["reach"] + 1, case["ones"] + case["idle"])])
    mix = rng.permutation(len(new))  # decode requests and prompts in any order
    new, held = new[mix], held[mix]
    after = held + new
    pages = -(-after // PAGE)
    total = int(pages.sum()) + 5
    order, ends = rng.permutation(total), np.cumsum(pages)
    table = np.zeros((len(new), max(1, int(pages.max()))), np.int32)
    for b in range(len(new)):
        table[b, :pages[b]] = order[ends[b] - pages[b]:ends[b]]
    starts = np.concatenate([[0], np.cumsum(new)])
    seq = np.repeat(np.arange(len(new)), new)
    pos = held[seq] + np.arange(starts[-1]) - starts[seq]
    slots = np.full(int(starts[-1]) + case["pad"], -1, np.int64)
    slots[:starts[-1]] = table[seq, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
    return dict(new=new, held=held, after=after, table=table, starts=starts, slots=slots, total=total)


def work(case):
    at = _layout(case)
    rows = int(at["starts"][-1])
    row = 2 * CODE_BYTES[case["kv"]] + (0 if case["kv"] == "bf16" else 8)  # K and V of a token in the cache
    ids = 4 * int((-(-at["after"] // PAGE)).sum())
    if case["op"] == "chunk":
        attended = int((at["new"] * at["held"] + at["new"] * (at["new"] + 1) // 2).sum())
        keys = int(at["after"][at["new"] > 0].sum())
        return {"bytes": keys * row + ids + rows * HEADS * (2 * 2 * DIM + 4), "flops": 4 * HEADS * DIM * attended}
    if case["op"] == "write":  # bf16 rows in, codes out, codes in again, bf16 rows out
        return {"bytes": rows * (2 * 2 * 2 * DIM + 2 * row + 8) + ids, "flops": 0}
    return {"bytes": rows * (row + 2 * 2 * DIM) + ids, "flops": 0}


# ------------------------------------------------------------------ inputs
def _rows(shape, gen):
    """K or V rows as projections give them: a few strong channels, token norms that vary."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x[..., :4] *= 3.0
    return (x * torch.exp(0.3 * torch.randn(shape[:-1], generator=gen, device="cuda")).unsqueeze(-1)).bfloat16()


def _scaled(x, most):
    x = x.float()
    top = x.abs().amax(-1)
    s = torch.where(top > 0, top / torch.full_like(top, most), torch.ones_like(top))  # by a tensor: a true division
    return x / s.unsqueeze(-1), s


def _to_fp8(x):
    q, s = _scaled(x, 448.0)
    return q.to(torch.float8_e4m3fn), s


def _to_fp4(x):
    """Packed E2M1 codes (element 2 k in the low half of byte k) and scales; ties to the even code."""
    q, s = _scaled(x, 6.0)
    m = q.abs()
    code = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
            + 8 * torch.signbit(q).byte())
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def prepare(case, seed):
    at = _layout(case)
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    ints = lambda a, t=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
    n, kv = int(at["starts"][-1]) + case["pad"], case["kv"]
    st = dict(case=case, host=at, batch=len(at["new"]), rows=n, total=at["total"], table=ints(at["table"]),
              lens=ints(at["after"]), first=ints(at["held"]), starts=ints(at["starts"]))
    pool = (at["total"], PAGE)
    if case["op"] == "write":
        both = _rows((n, 2, DIM), gen)  # one projection's output, K beside V
        st.update(k=both[:, 0], v=both[:, 1], slots=ints(at["slots"], torch.int64))
        st["kc"], st["vc"] = (torch.zeros((*pool, DIM // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
        st["ks"], st["vs"] = (torch.ones(pool, device="cuda") for _ in range(2))
    else:
        st["kc"], st["vc"] = (_rows((*pool, DIM), gen) for _ in range(2))
        if kv != "bf16":
            to = _to_fp8 if kv == "fp8" else _to_fp4
            (st["kc"], st["ks"]), (st["vc"], st["vs"]) = to(st["kc"]), to(st["vc"])
    need = 256
    if case["op"] == "chunk":
        st["q"] = torch.randn((n, HEADS, DIM), generator=gen, device="cuda").bfloat16()
        st["out"] = torch.zeros((n, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros((n, HEADS), device="cuda")
    else:
        st["k_out"], st["v_out"] = (torch.zeros((n, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        from decode_attention_mfa_gb300 import capi
        if case["op"] == "chunk":
            need = capi.mfa_chunk_workspace_bytes(st["batch"], n)
        st["ws_bytes"], st["ws"] = need, torch.empty(need, dtype=torch.uint8, device="cuda")
        capi.mfa_workspace_init(st["ws"], need)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _values(st, c, s, at):
    """Rows of a cache at flat slots `at`, in 32 bits."""
    kv = st["case"]["kv"]
    x = st[c].flatten(0, 1)
    if kv == "bf16":
        return x[at].float()
    if kv == "fp8":
        x = x.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    else:
        x = x[at]
        code = torch.stack([x & 15, x >> 4], -1).flatten(-2)
        m = (code & 7).float()
        m = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, 2 * m - 8))  # 0 .5 1 1.5 2 3 4 6
        x = torch.where(code > 7, -m, m)
    return x * st[s].flatten()[at].unsqueeze(-1)


def _slots(st, b, pos):
    return st["table"][b, pos // PAGE].long() * PAGE + pos % PAGE


def _block(q, k, v, limits):
    """Rows q [n, 64, d] over keys of which row i sees the first limits[i]: the output and the LSE."""
    s = q.flatten(0, 1) @ k.T * SCALE
    seen = torch.arange(k.shape[0], device=k.device) < limits.repeat_interleave(HEADS).unsqueeze(-1)
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return (p @ v / total).bfloat16().view_as(q), (m + torch.log(total)).view(-1, HEADS)


def _plain_chunk(st):
    at, step = st["host"], 256  # tokens at a time: what the logits of more take is the card's memory

    def sequence(b):
        held, after, r0 = int(at["held"][b]), int(at["after"][b]), int(at["starts"][b])
        every = _slots(st, b, torch.arange(after, device="cuda"))
        k, v = _values(st, "kc", "ks", every), _values(st, "vc", "vs", every)
        ends = [(t, min(after, t + step)) for t in range(held, after, step)]
        return [_block(st["q"][r0 + t - held:r0 + e - held].float(), k[:e], v[:e], torch.arange(t + 1, e + 1, device="cuda"))
                for t, e in ends]

    parts = [x for b in range(st["batch"]) for x in sequence(b)]
    n = int(at["starts"][-1])
    return {"out": torch.cat([o for o, _ in parts] + [st["out"][n:]]), "lse": torch.cat([x for _, x in parts] + [st["lse"][n:]])}


def _own_chunk(st):
    from decode_attention_mfa_gb300 import capi
    args = [st["table"], st["lens"], st["starts"], st["out"], st["lse"], SCALE, st["batch"], st["rows"], st["table"].shape[1],
            st["total"], st["ws"], st["ws_bytes"]]
    if st["case"]["kv"] == "bf16":
        capi.mfa_chunk_attention(st["q"], st["kc"], st["vc"], *args)
    else:
        call = capi.mfa_chunk_attention_fp8 if st["case"]["kv"] == "fp8" else capi.mfa_chunk_attention_fp4
        call(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], *args)
    return {"out": st["out"], "lse": st["lse"]}


def _plain_read(st):
    n = int(st["host"]["starts"][-1])
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(st["starts"][1:].long(), i, right=True)
    at = _slots(st, b, st["first"].long()[b] + i - st["starts"].long()[b])
    return {"k": torch.cat([_values(st, "kc", "ks", at).bfloat16(), st["k_out"][n:]]),
            "v": torch.cat([_values(st, "vc", "vs", at).bfloat16(), st["v_out"][n:]])}


def _own_read(st):
    from decode_attention_mfa_gb300 import capi
    args = [st["table"], st["first"], st["starts"], st["k_out"], st["v_out"], DIM, DIM, st["batch"], st["rows"],
            st["table"].shape[1], st["total"], st["ws"]]
    if st["case"]["kv"] == "bf16":
        capi.mfa_kv_read(st["kc"], st["vc"], *args)
    else:
        call = capi.mfa_kv_read_fp8 if st["case"]["kv"] == "fp8" else capi.mfa_kv_read_fp4
        call(st["kc"], st["vc"], st["ks"], st["vs"], *args)
    return {"k": st["k_out"], "v": st["v_out"]}


def _plain_write(st):
    rows = st["slots"] >= 0
    at = st["slots"][rows]
    (st["kc"].view(-1, DIM // 2)[at], st["ks"].view(-1)[at]) = _to_fp4(st["k"][rows])
    (st["vc"].view(-1, DIM // 2)[at], st["vs"].view(-1)[at]) = _to_fp4(st["v"][rows])
    return {**_plain_read(st), "ks": st["ks"], "vs": st["vs"]}


def _own_write(st):
    from decode_attention_mfa_gb300 import capi
    k, v = st["k"], st["v"]
    capi.mfa_kv_append_slots_fp4(k, v, k.stride(0), v.stride(0), st["slots"], len(k), st["kc"], st["vc"], st["ks"], st["vs"],
                                 st["total"], st["ws"])
    return {**_own_read(st), "ks": st["ks"], "vs": st["vs"]}


_plain = dict(chunk=_plain_chunk, write=_plain_write, read=_plain_read)
_own = dict(chunk=_own_chunk, write=_own_write, read=_own_read)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _held(st, c, s, ids, tokens):
    """The first `tokens` rows that pages `ids` hold, by value."""
    kv = st["case"]["kv"]
    if kv == "bf16":
        return st[c][ids].double().reshape(-1, DIM)[:tokens]
    if kv == "fp8":
        rows = st[c].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
    else:
        worth = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
        packed = st[c][ids].long()
        rows = torch.empty((*packed.shape[:-1], DIM), dtype=torch.float64, device="cuda")
        rows[..., 0::2], rows[..., 1::2] = worth[packed % 16], worth[packed // 16]
    return (rows * st[s][ids].double()[..., None]).reshape(-1, DIM)[:tokens]


def exact(case, seed):
    if case["op"] == "chunk" and work(case)["flops"] > 5e12:
        return None
    st, at = prepare(case, seed), _layout(case)
    n = int(at["starts"][-1])
    if case["op"] == "chunk":
        out = torch.zeros((st["rows"], HEADS, DIM), dtype=torch.float64, device="cuda")
        lse = torch.zeros((st["rows"], HEADS), dtype=torch.float64, device="cuda")
        for b in range(st["batch"]):
            held, total = int(at["held"][b]), int(at["after"][b])
            ids = st["table"][b, :-(-total // PAGE)].long()
            k, v = _held(st, "kc", "ks", ids, total), _held(st, "vc", "vs", ids, total)
            for t0 in range(0, total - held, 64):
                t1 = min(total - held, t0 + 64)
                r = int(at["starts"][b]) + t0
                q = st["q"][r:r + t1 - t0].double()
                logits = torch.einsum("thd,jd->htj", q, k[:held + t1]) * SCALE
                future = torch.ones((t1 - t0, held + t1), device="cuda").triu(held + t0 + 1).bool()
                logits.masked_fill_(future, -math.inf)
                z = torch.logsumexp(logits, -1)
                lse[r:r + t1 - t0] = z.T
                out[r:r + t1 - t0] = torch.einsum("htj,jd->thd", torch.exp(logits - z[..., None]), v[:held + t1])
        return {"out": out, "lse": lse}
    got = {name: torch.zeros((st["rows"], DIM), dtype=torch.float64, device="cuda") for name in "kv"}
    if case["op"] == "read":
        for b in range(st["batch"]):
            total, r0, r1 = int(at["after"][b]), int(at["starts"][b]), int(at["starts"][b + 1])
            ids = st["table"][b, :-(-total // PAGE)].long()
            for x in "kv":
                got[x][r0:r1] = _held(st, x + "c", x + "s", ids, total)[int(at["held"][b]):]
        return got
    for x in "kv":
        y = st[x][:n].double()
        top = y.abs().max(1).values
        s = torch.where(top > 0, top / 6.0, torch.ones_like(top)).float().double()  # the scale is held in 32 bits
        z = (y / s[:, None]).float().double()  # the quotient as well
        # the nearest E2M1 value: one bit behind the leading one, steps of a half below 1
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=1.0))) - 1)
        got[x][:n] = (torch.round(z / step) * step).clamp(-6.0, 6.0) * s[:, None]
        scales = torch.ones(at["total"] * PAGE, dtype=torch.float64, device="cuda")
        scales[st["slots"][:n]] = s
        got[x + "s"] = scales.view(at["total"], PAGE)
    return got
