"""A paged cache written by slot in 4 bits, and read back in every format (mfa_kv_append_slots_fp4, mfa_kv_read*); serving
steps that take prompts in chunks.

Written codes and scales are compared for equality with mfa_kv_append_fp4's and the oracle's, bf16 rows read back bit for
bit. A value read from codes is decode(code) * scale rounded to fp32 (off by at most 2^-24 of itself) and then to bf16 (at
most 2^-8): 1.001 * 2^-8 of it, and half a step of the smallest bf16 numbers, 2^-134, where it is one of those."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi
from test_gpu_chunk import E2M1, Step, values

pytestmark = pytest.mark.gpu
PAGE, HEADS, DIM = 64, 64, 256
KV = pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
READ = {"bf16": capi.mfa_kv_read, "fp8": capi.mfa_kv_read_fp8, "fp4": capi.mfa_kv_read_fp4}
APPEND = {"bf16": capi.mfa_kv_append_slots, "fp8": capi.mfa_kv_append_slots_fp8, "fp4": capi.mfa_kv_append_slots_fp4}


def workspace():
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    capi.mfa_workspace_init(ws, 256)
    return ws


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a)).int().cuda()


# ---------------------------------------------------------------- written
def special_rows():
    """Zeros of both signs, one large value among small ones, every tie of the format, tiny and huge rows, no numbers."""
    gen = torch.Generator().manual_seed(1)
    rows = torch.randn((300, DIM), generator=gen).bfloat16()
    rows[0], rows[1] = 0.0, -0.0
    rows[2] *= 1e-4
    rows[2, 5] = 3.0
    rows[3] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 32)
    rows[4] = -rows[3]
    rows[5] = (rows[5].float() * 1e38).bfloat16()
    rows[6] = (rows[6].float() * 1e-38).bfloat16()  # below the range of the quick quotients, some of it subnormal
    rows[7] = 9.2e-41
    rows[8, ::2] = float("nan")
    rows[9] = float("nan")
    rows[10, 3] = float("inf")
    rows[11, 3] = -float("inf")
    rows[12] = rows[3] * 1.5 * 2.0 ** -60  # a scale on either side of the quick quotients' range
    rows[13] = rows[3] * 2.0 ** -60
    rows[14] = rows[3] * 2.0 ** 61
    return rows


@pytest.mark.parametrize("n", [1, 127, 300, 9001])
def test_append_slots_fp4(oracle_mod, n):
    rows = special_rows() if n == 300 else torch.randn((n, DIM), generator=torch.Generator().manual_seed(n)).bfloat16()
    pages = -(-n // PAGE) + 2
    rng = np.random.default_rng(n)
    slots = rng.permutation(pages * PAGE)[:n]
    skipped = rng.random(n) < 0.1
    both = torch.stack([rows, rows.flip(0)], 1).cuda()  # K beside V
    k, v = both[:, 0], both[:, 1]
    kc, vc = (torch.full((pages, PAGE, DIM // 2), 0x77, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, PAGE), -3.0, device="cuda") for _ in range(2))
    ws = workspace()
    d_slots = torch.from_numpy(np.where(skipped, -1, slots)).cuda()
    capi.mfa_kv_append_slots_fp4(k, v, k.stride(0), v.stride(0), d_slots, n, kc, vc, ks, vs, pages, ws)
    capi.mfa_check_device_errors(ws)
    for x, c, s in ((rows, kc, ks), (rows.flip(0), vc, vs)):
        bits = x.view(torch.int16).numpy().view(np.uint16)
        codes, scale = oracle_mod.quantize_tokens_e2m1(bits)
        odd = ~np.isfinite(x.float().numpy()).all(1)  # the oracle says nothing of these: compared with the other append below
        want = np.full((pages * PAGE, DIM // 2), 0x77, np.uint8)
        want_s = np.full(pages * PAGE, -3.0, np.float32)
        keep = ~skipped
        want[slots[keep]], want_s[slots[keep]] = codes[keep], scale[keep]
        same = np.ones(pages * PAGE, bool)
        same[slots[odd]] = False
        assert np.array_equal(c.cpu().numpy().reshape(-1, DIM // 2)[same], want[same])
        assert np.array_equal(s.cpu().numpy().reshape(-1)[same], want_s[same])
    # the same as the other append, row by row, whatever the values
    one = torch.empty((pages, PAGE, DIM // 2), dtype=torch.uint8, device="cuda")
    two, s1, s2 = torch.empty_like(one), torch.empty((pages, PAGE), device="cuda"), torch.empty((pages, PAGE), device="cuda")
    lens, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.arange(pages, dtype=torch.int32, device="cuda")
    capi.mfa_kv_append_fp4(k.contiguous(), v.contiguous(), n, one, two, s1, s2, table, lens, 1, pages, pages, ws)
    at = torch.from_numpy(slots[~skipped]).cuda()
    kept = torch.from_numpy(~skipped).cuda()
    for a, b, width in ((one, kc, DIM // 2), (two, vc, DIM // 2), (s1, ks, 1), (s2, vs, 1)):
        assert torch.equal(a.reshape(-1, width)[:n][kept].view(torch.uint8), b.reshape(-1, width)[at].view(torch.uint8))


def test_append_slots_fp4_bad_slot():
    rows = torch.randn((3, DIM), device="cuda").bfloat16()
    kc, vc = (torch.full((2, PAGE, DIM // 2), 5, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((2, PAGE), device="cuda") for _ in range(2))
    ws = workspace()
    capi.mfa_kv_append_slots_fp4(rows, rows, DIM, DIM, torch.tensor([0, 2 * PAGE, 2 ** 40], device="cuda"), 3, kc, vc, ks, vs, 2, ws)
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(ws)
    assert e.value.status == 5
    assert (kc.view(-1, DIM // 2)[1:] == 5).all() and (vc.view(-1, DIM // 2)[1:] == 5).all()


@pytest.mark.parametrize("n", [2047, 2048, 6081, 16383, 16384, 18239, 18241, 30000])  # all ways, with whole and ragged loops
@pytest.mark.parametrize("kv", ["fp8", "fp4"])
def test_append_slots_many_rows(kv, n):
    """Codes and scales of rows of every kind, in a shuffled pool and beside skipped and bad slots, are those of the other append."""
    rows = torch.randn((n, DIM), generator=torch.Generator().manual_seed(n)).bfloat16()
    odd = special_rows()[:15]
    rows[: 15 * 130: 130], rows[-15:] = odd, odd
    both = torch.stack([rows, rows.flip(0)], 1).cuda()
    k, v = both[:, 0], both[:, 1]
    pages, width = -(-n // PAGE) + 2, DIM if kv == "fp8" else DIM // 2
    rng = np.random.default_rng(n)
    slots = rng.permutation(pages * PAGE)[:n]
    given = np.where(rng.random(n) < 0.1, -1, slots)
    given[n - 7] = pages * PAGE  # one that the pool does not have
    pools = lambda: ([torch.full((pages, PAGE, width), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]  # noqa: E731
                     + [torch.full((pages, PAGE), -3.0, device="cuda") for _ in range(2)])
    got, want = pools(), pools()
    ws = workspace()
    call = capi.mfa_kv_append_slots_fp8 if kv == "fp8" else capi.mfa_kv_append_slots_fp4
    call(k, v, k.stride(0), v.stride(0), torch.from_numpy(given).cuda(), n, *got, pages, ws)
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(ws)
    assert e.value.status == 5
    lens, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.arange(pages, dtype=torch.int32, device="cuda")
    other = capi.mfa_kv_append_fp8 if kv == "fp8" else capi.mfa_kv_append_fp4
    other(k.contiguous(), v.contiguous(), n, *want, table, lens, 1, pages, pages, ws)
    written = (given >= 0) & (given < pages * PAGE)
    at, kept = torch.from_numpy(slots[written]).cuda(), torch.from_numpy(written).cuda()
    rest = torch.ones(pages * PAGE, dtype=torch.bool, device="cuda")
    rest[at] = False
    for a, b in zip(got, want):
        a, b = a.reshape(pages * PAGE, -1), b.reshape(pages * PAGE, -1)
        assert torch.equal(a[at].view(torch.uint8), b[:n][kept].view(torch.uint8))
        assert (a[rest] == (0x55 if a.dtype == torch.uint8 else -3.0)).all()


# ---------------------------------------------------------------- read back
def read_plain(s, first, starts, i):
    """(values in 64 bits, flat slots) of the rows of cache i."""
    slots = np.concatenate([np.asarray([s.row(b, int(first[b]) + j) for j in range(starts[b + 1] - starts[b])], np.int64)
                            for b in range(s.B)])
    at = torch.from_numpy(slots).cuda()
    c = s.cache[i].reshape(s.num_pages * PAGE, -1)[at]
    return values(c, s.scales[i].view(-1)[at] if s.scales else None, s.kv), at


@KV
@pytest.mark.parametrize("lens,first,rows,pad,stride", [
    ([1], [0], [1], 0, 256), ([64], [0], [64], 0, 256), ([65, 130], [64, 3], [1, 127], 2, 512), ([500], [17], [400], 0, 264),
    ([70, 5, 200, 0, 3], [69, 5, 0, 0, 0], [1, 0, 200, 0, 3], 11, 1024), ([9000, 4000], [0, 111], [8999, 3889], 70, 256),
])
def test_read(kv, lens, first, rows, pad, stride):
    s = Step([0] * len(lens), None, kv, seed=len(lens), lens=lens)
    starts = np.concatenate([[0], np.cumsum(rows)])
    n = int(starts[-1]) + pad
    space = torch.full((2, n, stride), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace()

    def read(first):
        READ[kv](*s.cache, *s.scales, s.d_table, first, i32(starts), space[0], space[1], stride, stride, s.B, n,
                 s.table.shape[1], s.num_pages, ws)
        capi.mfa_check_device_errors(ws)

    read(i32(first))
    for i in range(2):
        got, want = space[i, :n - pad, :DIM], read_plain(s, first, starts, i)[0]
        assert torch.isfinite(got).all()
        assert ((got.double() - want).abs() <= (0 if kv == "bf16" else 1.001 * 2 ** -8 * want.abs() + 2 ** -134)).all()
        assert (space[i, n - pad:] == 3).all() and (space[i, :, DIM:] == 3).all()
    if all(r <= m for r, m in zip(rows, lens)):
        space.fill_(3)
        read(None)  # from the first position on
        assert (space[0, :n - pad, :DIM].double() - read_plain(s, [0] * s.B, starts, 0)[0]).abs().max() <= 0.2


@KV
def test_read_is_exact_where_bf16_holds_the_product(kv):
    """Scales that are powers of two: codes have four bits, so that nothing is rounded."""
    s = Step([0], None, kv, lens=[300])
    for x in s.scales:
        x.copy_(torch.exp2(torch.randint(-120, 100, x.shape, device="cuda").float()))
    out = torch.zeros((2, 300, DIM), dtype=torch.bfloat16, device="cuda")
    ws = workspace()
    READ[kv](*s.cache, *s.scales, s.d_table, None, i32([0, 300]), out[0], out[1], DIM, DIM, 1, 300, s.table.shape[1], s.num_pages, ws)
    for i in range(2):
        assert torch.equal(out[i].double(), read_plain(s, [0], [0, 300], i)[0])


def test_every_code():
    """All codes of both formats, NaN and signed zeros among them."""
    ws = workspace()
    table, starts = i32([[0]]), i32([0, 1])
    for kv, codes in (("fp8", torch.arange(256)), ("fp4", torch.arange(128) * 2 % 256)):
        cache = codes.to(torch.uint8).cuda().expand(1, PAGE, -1).contiguous()
        scale = torch.full((1, PAGE), 0.5, device="cuda")
        out = torch.zeros((2, 1, DIM), dtype=torch.bfloat16, device="cuda")
        READ[kv](cache, cache, scale, scale, table, None, starts, out[0], out[1], DIM, DIM, 1, 1, 1, 1, ws)
        want = values(cache[0, 0], scale[0, :1], kv).view(-1).bfloat16()
        for i in range(2):
            assert torch.equal(out[i, 0].view(torch.int16)[~torch.isnan(want)], want.view(torch.int16)[~torch.isnan(want)])
            assert torch.equal(torch.isnan(out[i, 0]), torch.isnan(want))
    assert len(E2M1) == 16


@KV
def test_read_out_of_range(kv):
    """Bad positions and pages leave their rows as they were; the others are read."""
    s = Step([0, 0, 0], None, kv, lens=[100, 100, 100])
    cap = s.table.shape[1] * PAGE
    starts, first = [0, 10, 20, 30], [cap - 4, 0, -3]
    s.d_table[0, -1] = int(s.table[0, 0])
    s.d_table[1, 0] = s.num_pages
    out = torch.full((2, 40, DIM), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace()

    def read(starts, rows=40):
        READ[kv](*s.cache, *s.scales, s.d_table, i32(first), i32(starts), out[0], out[1], DIM, DIM, 3, rows, s.table.shape[1],
                 s.num_pages, ws)

    def error():
        with pytest.raises(capi.MFAError) as e:
            capi.mfa_check_device_errors(ws)
        return e.value.status

    read(starts)
    assert error() == 5
    assert (out[:, 4:23] == 3).all() and (out[:, 30:] == 3).all()
    assert torch.isfinite(out[:, 23:30]).all() and not (out[:, 23:30] == 3).any(-1).all()
    s.d_table[1, 0] = int(s.table[1, 0])
    read(starts)
    assert error() == 6
    out.fill_(3)
    read([0, 10, 20, 90])  # past the rows: these are read, no others
    assert error() == 6
    for bad in ([5, 3, 20, 30], [-7, 10, 20, 30], [0, 10, 20, 2 ** 31 - 1]):
        read(bad)
        assert error() == 6


@KV
def test_read_many_sequences(kv):
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 40, 1024)
    s = Step([0] * 1024, None, kv, seed=3, lens=lens)
    first = (lens * rng.random(1024)).astype(int)
    starts = np.concatenate([[0], np.cumsum(lens - first)])
    out = torch.zeros((2, starts[-1], DIM), dtype=torch.bfloat16, device="cuda")
    ws = workspace()
    READ[kv](*s.cache, *s.scales, s.d_table, i32(first), i32(starts), out[0], out[1], DIM, DIM, 1024, int(starts[-1]),
             s.table.shape[1], s.num_pages, ws)
    capi.mfa_check_device_errors(ws)
    for i in range(2):
        want = read_plain(s, first, starts, i)[0]
        assert ((out[i].double() - want).abs() <= 1.001 * 2 ** -8 * want.abs()).all()


def test_read_past_four_gigabytes():
    """Slots whose byte offsets pass 32 bits."""
    pages = (1 << 32) // (PAGE * DIM * 2) + 5
    cache = torch.empty((pages, PAGE, DIM), dtype=torch.bfloat16, device="cuda")
    cache[-3:] = torch.randn((3, PAGE, DIM), device="cuda").bfloat16()
    out = torch.zeros((2, 192, DIM), dtype=torch.bfloat16, device="cuda")
    ws = workspace()
    capi.mfa_kv_read(cache, cache, i32([[pages - 1, pages - 3, pages - 2]]), None, i32([0, 192]), out[0], out[1], DIM, DIM, 1, 192, 3,
                     pages, ws)
    for i in range(2):
        assert torch.equal(out[i].view(3, PAGE, DIM), cache[[pages - 1, pages - 3, pages - 2]])
    q = torch.randn((5, HEADS, DIM), device="cuda").bfloat16()
    o, lse = torch.zeros_like(q), torch.zeros((5, HEADS), device="cuda")
    need = capi.mfa_chunk_workspace_bytes(1, 5)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    capi.mfa_workspace_init(ws, need)
    capi.mfa_chunk_attention(q, cache, cache, i32([[pages - 1, pages - 3, pages - 2]]), i32([192]), i32([0, 5]), o, lse, 1 / 16, 1, 5, 3,
                             pages, ws, need)
    k = cache[[pages - 1, pages - 3, pages - 2]].double().view(-1, DIM)
    s = torch.einsum("thd,jd->thj", q.double(), k) / 16
    s.masked_fill_(torch.ones((5, 1, 192), device="cuda").triu(0).cumsum(-1) > 188 + torch.arange(5, device="cuda").view(5, 1, 1), -torch.inf)
    want = torch.softmax(s, -1) @ k
    assert (o.double() - want).abs().max() <= 2 ** -8 * 2 * k.abs().max()


# ---------------------------------------------------------------- steps of a server
@KV
@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_with_chunked_prompts(kv, captured):
    """Five requests whose prompts arrive in chunks of different lengths beside decode tokens: each step reserves pages, appends
    by slot, attends and reads its own rows back, with nothing of it on the host; captured, one graph for every step."""
    torch.manual_seed(4)
    B, cap, pages, most = 5, 12, 64, 200
    steps = [[100, 0, 63, 0, 1], [64, 30, 1, 0, 1], [1, 129, 1, 64, 1], [1, 1, 1, 65, 0], [1, 1, 60, 1, 1]]
    width = {"bf16": DIM, "fp8": DIM, "fp4": DIM // 2}[kv]
    kind = torch.bfloat16 if kv == "bf16" else torch.uint8
    cache = [torch.zeros((pages, PAGE, width), dtype=kind, device="cuda") for _ in range(2)]
    scales = [] if kv == "bf16" else [torch.zeros((pages, PAGE), device="cuda") for _ in range(2)]
    need = capi.mfa_chunk_workspace_bytes(B, most)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    capi.mfa_workspace_init(ws, need)
    table, lens, held = i32(np.full((B, cap), -1)), i32([0] * B), i32([0] * B)
    free, n_free = torch.randperm(pages, device="cuda").int(), i32([pages])
    n_new, starts, slots = i32([0] * B), i32([0] * (B + 1)), torch.zeros(most, dtype=torch.int64, device="cuda")
    kv_rows = torch.zeros((most, 2, DIM), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((most, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((most, HEADS), device="cuda")
    back = torch.zeros((2, most, DIM), dtype=torch.bfloat16, device="cuda")

    def step():
        k, v = kv_rows[:, 0], kv_rows[:, 1]
        held.copy_(lens)
        capi.mfa_reserve_pages(n_new, lens, table, free, n_free, B, cap, pages, most, starts, slots, lens, n_free, ws)
        APPEND[kv](k, v, k.stride(0), v.stride(0), slots, most, *cache, *scales, pages, ws)
        from test_gpu_chunk import CALL
        CALL[kv](q, *cache, *scales, table, lens, starts, out, lse, 1 / 16, B, most, cap, pages, ws, need)
        READ[kv](*cache, *scales, table, held, starts, back[0], back[1], DIM, DIM, B, most, cap, pages, ws)

    graph = None
    if captured:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()  # no tokens: nothing changes
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    said = [[torch.zeros((0, DIM), dtype=torch.float64, device="cuda") for _ in range(2)] for _ in range(B)]
    for new in steps:
        total = sum(new)
        n_new.copy_(torch.tensor(new))
        q.copy_(torch.randn(q.shape, device="cuda"))
        kv_rows.copy_(torch.randn(kv_rows.shape, device="cuda"))
        out.fill_(7)
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        capi.mfa_check_device_errors(ws)
        r = 0
        for b, n in enumerate(new):
            for i in range(2):
                rows = back[i, r:r + n].double()
                if kv == "bf16":
                    assert torch.equal(back[i, r:r + n], kv_rows[r:r + n, i])
                else:  # half a step of the format: of the scale, 16 for codes of 448, 1 for codes of 6; and of bf16
                    x = kv_rows[r:r + n, i].double()
                    top = x.abs().amax(-1, keepdim=True)
                    half = top * (16 / 448 if kv == "fp8" else 1 / 6)
                    assert ((rows - x).abs() <= half * 1.001 + 1.001 * 2 ** -8 * x.abs() + 2 ** -8 * half).all()
                said[b][i] = torch.cat([said[b][i], rows])
            if n:
                k, v = said[b]
                s = torch.einsum("thd,jd->thj", q[r:r + n].double(), k) / 16
                limit = len(k) - n + 1 + torch.arange(n, device="cuda").view(n, 1, 1)
                s = torch.where(torch.arange(len(k), device="cuda") >= limit, torch.full_like(s, -torch.inf), s)
                want = torch.softmax(s, -1) @ v
                # the rows read back are themselves off by a bf16 rounding, 2^-8 of a value: so is a mean of V; K's, each of
                # 256 terms of a logit, moves it by at most 2^-8 / 16 * sum |q k|, below 2^-8 * 14 (sum |q| |k| < 220), a weight
                # by 14 * 2^-8 of itself, and an output by twice that of the largest |v|
                loose = 0 if kv == "bf16" else 2 ** -8 * 29
                assert ((out[r:r + n].double() - want).abs() <= 2 ** -8 * (2 * v.abs().max() + want.abs()) + loose * v.abs().max()).all()
            r += n
        assert (out[total:] == 7).all()
