"""Attention of chunks of new tokens (mfa_chunk_attention*) against the definition in 64 bits.

Tolerances, from the roundings on the way (a rounding to bf16 is off by at most 2^-8 of the value, to f16 2^-11): each
weight enters the second product as bf16, and O is divided by the sum of what entered, so an output is off by at most 2^-8
of the weighted mean of |v - out|, which is below the largest |v| that the token sees; the output is rounded to bf16, off
by at most 2^-8 of itself; the fp32 sums of 256 products and the exponentials add less than 2^-12 of either. On E4M3 and
E2M1 caches the weights and the scaled values are f16 (2^-11 each, and 2^-11 for the scale) and the queries are held to
2^-18.8 of the row's largest: together no more than another 2^-8 of the largest |v|. The LSE is off by the logits' fp32
sums, 2^-15 of scale * sum |q k| (about 10 here), below 1e-3."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi

pytestmark = pytest.mark.gpu
PAGE, HEADS, DIM = 64, 64, 256
SCALE = 1.0 / 16.0
LSE_ABS = 1e-3
KV = pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
CALL = {"bf16": capi.mfa_chunk_attention, "fp8": capi.mfa_chunk_attention_fp8, "fp4": capi.mfa_chunk_attention_fp4}
E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def to_codes(x, kv):
    """Rows as codes and scales of a quantised cache (any rounding will do: the reference reads the codes)."""
    x = x.float()
    s = x.abs().amax(-1) / (448.0 if kv == "fp8" else 6.0)
    y = x / s.unsqueeze(-1)
    if kv == "fp8":
        return y.to(torch.float8_e4m3fn).view(torch.uint8), s
    m = y.abs()
    code = sum((m > t).to(torch.uint8) for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)) + 8 * (y < 0).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def values(codes, scale, kv):
    if kv == "bf16":
        return codes.double()
    if kv == "fp8":
        return codes.view(torch.float8_e4m3fn).double() * scale.double().unsqueeze(-1)
    worth = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return worth[both] * scale.double().unsqueeze(-1)


class Step:
    """Sequences of `held` positions and `new` tokens behind them, in pages in random order, on the device."""

    def __init__(self, new, held, kv="bf16", seed=0, lens=None, pad=0, lead=0, spare_cols=1, q_scale=1.0, spread=0.5):
        rng = np.random.default_rng(seed)
        self.kv, self.B = kv, len(new)
        self.new = np.asarray(new)
        self.lens = np.asarray(lens) if lens is not None else np.asarray(held) + self.new
        self.starts = lead + np.concatenate([[0], np.cumsum(self.new)])
        self.rows = int(self.starts[-1]) + pad
        pages = -(-self.lens // PAGE)
        self.num_pages = int(pages.sum()) + 3
        order, ends = rng.permutation(self.num_pages), np.cumsum(pages)
        self.table = np.full((self.B, int(pages.max()) + spare_cols), -1, np.int32)
        used = np.zeros((self.num_pages, PAGE), bool)
        for b in range(self.B):
            self.table[b, :pages[b]] = order[ends[b] - pages[b]:ends[b]]
            for j in range(pages[b]):
                used[self.table[b, j], :min(PAGE, self.lens[b] - j * PAGE)] = True
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.q = (q_scale * torch.randn((self.rows, HEADS, DIM), generator=gen, device="cuda")).bfloat16()
        for a, e in ((0, lead), (int(self.starts[-1]), self.rows)):  # rows of no sequence are neither read nor written
            self.q[a:e] = float("nan")
        unused = torch.from_numpy(~used).cuda()
        self.cache, self.scales = [], []
        for _ in range(2):
            x = torch.randn((self.num_pages, PAGE, DIM), generator=gen, device="cuda")
            if kv == "bf16":
                x = x.bfloat16()
                x[unused] = float("nan")  # a stale row is never read
            else:
                x, s = to_codes(x * torch.exp(spread * torch.randn((self.num_pages, PAGE, 1), generator=gen, device="cuda")), kv)
                x[unused] = 0x7F if kv == "fp8" else 0x77
                s[unused] = float("nan")
                self.scales.append(s)
            self.cache.append(x)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()  # noqa: E731
        self.d_table, self.d_lens, self.d_starts = i32(self.table), i32(self.lens), i32(self.starts)
        self.out = torch.full((self.rows, HEADS, DIM), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.rows, HEADS), 7.0, device="cuda")
        n = capi.mfa_chunk_workspace_bytes(self.B, self.rows)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        capi.mfa_workspace_init(self.ws, n)
        self.ws[256:] = 0xFF  # what the scratch holds between calls is not used: NaN floats, counts of -1
        torch.cuda.synchronize()

    def call(self, scale=SCALE, stream=None):
        CALL[self.kv](self.q, *self.cache, *self.scales, self.d_table, self.d_lens, self.d_starts, self.out, self.lse, scale,
                      self.B, self.rows, self.table.shape[1], self.num_pages, self.ws, self.ws.numel(), stream)

    def row(self, b, j):
        """Flat slot of position j of sequence b."""
        return int(self.table[b, j // PAGE]) * PAGE + j % PAGE

    def reference(self, b, scale=SCALE):
        n, t = int(self.lens[b]), int(self.new[b])
        ids = torch.from_numpy(self.table[b, :-(-n // PAGE)]).long().cuda()
        k, v = (values(c[ids], self.scales[i][ids] if self.scales else None, self.kv).reshape(-1, DIM)[:n]
                for i, c in enumerate(self.cache))
        logits = torch.einsum("thd,jd->thj", self.q[self.starts[b]:self.starts[b + 1]].double(), k) * scale
        limit = n - t + 1 + torch.arange(t, device="cuda")
        hidden = torch.arange(n, device="cuda") >= limit.view(t, 1, 1)
        logits = torch.where(hidden, torch.full_like(logits, -torch.inf), logits)
        lse = torch.logsumexp(logits, -1)
        p = torch.where(hidden, torch.zeros_like(logits), torch.exp(logits - lse.unsqueeze(-1)))
        seen = torch.cummax(v.abs().amax(-1), 0).values if n else torch.zeros(1, dtype=torch.float64, device="cuda")
        top = seen[(limit - 1).clamp(0, max(0, n - 1))].view(t, 1, 1)
        return torch.einsum("thj,jd->thd", p, v), lse, top, limit

    def check(self, scale=SCALE, which=None):
        capi.mfa_check_device_errors(self.ws)
        wide = 2 if self.kv != "bf16" else 1
        for b in range(self.B) if which is None else which:
            if self.new[b] == 0:
                continue
            out, lse, top, limit = self.reference(b, scale)
            got, got_lse = (x[self.starts[b]:self.starts[b + 1]].double() for x in (self.out, self.lse))
            none = limit <= 0  # tokens that see no position
            assert (got[none] == 0).all() and torch.isneginf(got_lse[none]).all(), b
            out, lse, top, got, got_lse = (x[~none] for x in (out, lse, top, got, got_lse))
            bound = 2 ** -8 * (wide * top + out.abs()) + 2 ** -12 * top
            assert torch.isfinite(got).all(), b
            assert ((got - out).abs() <= bound).all(), (b, float((got - out).abs().max()), float(bound.min()))
            if out.numel():
                assert float((got - out).norm() / out.norm()) <= 5e-3 * wide, b
                assert float((got_lse - lse).abs().max()) <= LSE_ABS, b
        for a, e in ((0, int(self.starts[0])), (int(self.starts[-1]), self.rows)):
            assert (self.out[a:e] == 7).all() and (self.lse[a:e] == 7).all()

    def run(self, **kw):
        self.call(**kw)
        self.check(kw.get("scale", SCALE))
        return self


# ---------------------------------------------------------------- lengths
@KV
@pytest.mark.parametrize("held", [0, 1, 60, 61, 63, 64, 124, 125, 127, 128, 129, 190, 255, 700])
@pytest.mark.parametrize("new", [1, 2, 3, 4, 5, 8, 13])
def test_one_chunk(new, held, kv):
    Step([new], [held], kv, seed=new * 1000 + held).run()


@KV
@pytest.mark.parametrize("new", [64, 127, 128, 129, 300, 513, 1025])
def test_whole_prompt(new, kv):
    Step([new], [0], kv, seed=new).run()


@KV
@pytest.mark.parametrize("new,held", [(1, 30000), (3, 20001), (40, 16384), (130, 9999)])
def test_long_context(new, held, kv):
    Step([new], [held], kv, seed=held).run()


@KV
def test_more_pages_than_l2_holds(kv):
    """Sequences of many, few and single tiles whose pages are more than L2 holds: pairs leave a tile's rest for last."""
    s = Step([9, 1, 30, 61, 4, 17, 2, 9, 40, 0, 5, 12, 3, 700], [30000 + 777 * (i % 5) for i in range(13)] + [9000], kv, seed=8, pad=2)
    s.run()
    out, lse = s.out.clone(), s.lse.clone()
    s.call()
    assert torch.equal(out, s.out) and torch.equal(lse, s.lse)


@KV
def test_ragged_batch(kv):
    rng = np.random.default_rng(5)
    new = np.where(rng.random(70) < 0.5, 1, rng.integers(0, 90, 70))
    Step(new, rng.integers(0, 1500, 70), kv, seed=6, pad=9, lead=5).run()


@KV
def test_decode_tokens_only(kv):
    rng = np.random.default_rng(7)
    Step(np.ones(100, int), rng.integers(0, 3000, 100), kv, seed=8).run()


@pytest.mark.parametrize("B", [31, 32, 33, 64, 513, 1024])
def test_batch_sizes(B):
    rng = np.random.default_rng(B)
    Step(rng.integers(0, 6, B), rng.integers(0, 200, B), seed=B).run()


@KV
def test_more_tokens_than_positions(kv):
    """Tokens before the first position see nothing; sequences without tokens, without positions, without either."""
    Step([5, 0, 9, 3, 0, 70, 1], None, kv, seed=3, lens=[5, 40, 2, 0, 0, 69, 0], pad=4).run()


def test_nothing_to_do():
    s = Step([0, 0, 0], [5, 0, 70], pad=6)
    s.run()


# ---------------------------------------------------------------- values
@KV
@pytest.mark.parametrize("scale", [0.0, -0.0625, 1e-3, 0.5])
def test_scales(kv, scale):
    Step([70, 9], [100, 333], kv, seed=11).run(scale=scale)


@KV
def test_peaked_rows(kv):
    """Logits of tens of units: the reference moves within a tile, and again behind its first unit."""
    s = Step([33, 6], [500, 1200], kv, seed=12)
    s.q[::3] *= 8
    s.call()
    capi.mfa_check_device_errors(s.ws)
    for b in range(2):
        out, lse, top, _ = s.reference(b)
        got, got_lse = (x[s.starts[b]:s.starts[b + 1]].double() for x in (s.out, s.lse))
        # the logits' fp32 sums are off by 2^-15 of scale * sum |q k|, about 80 here: 2.4e-3 in the exponent, and the
        # queries' terms on a quantised cache by 2^-18.8 of the largest |q| (32) times sum |k| (200 .. 900) / 16: 4e-3
        assert ((got - out).abs() <= 2 ** -8 * (2 * top + out.abs()) + 1.3e-2 * top).all(), b
        assert float((got_lse - lse).abs().max()) <= 1e-2, b


@KV
def test_rising_and_falling_logits(kv):
    """Keys whose logits rise along the sequence, and ones that fall."""
    for seed, sign in ((13, 1.0), (14, -1.0)):
        s = Step([40], [1500], kv, seed=seed)
        n = int(s.lens[0])
        ramp = 0.2 + 1.6 * torch.arange(n, device="cuda") / n
        ramp = ramp if sign > 0 else ramp.flip(0)
        slots = torch.tensor([s.row(0, j) for j in range(n)], device="cuda")
        if kv == "bf16":
            flat = s.cache[0].view(-1, DIM)
            flat[slots] = (flat[slots].float() * ramp.unsqueeze(1)).bfloat16()
        else:
            s.scales[0].view(-1)[slots] *= ramp
        s.run()


def _with_logits(s, b, logits, values_of=None):
    """Keys of sequence b that give every head the logits (to what the cache holds of them); values_of: their value rows."""
    s.q[:] = 0.0
    s.q[..., 0] = 16.0
    for i, x in enumerate((logits, values_of)):
        if x is None:
            continue
        rows = torch.zeros((len(x), DIM), device="cuda")
        rows[:, 0 if i == 0 else slice(None)] = x if i == 0 else x.unsqueeze(1)
        at = torch.tensor([s.row(b, j) for j in range(len(x))], device="cuda")
        if s.kv == "bf16":
            s.cache[i].view(-1, DIM)[at] = rows.bfloat16()
        else:
            code, scale = to_codes(rows, s.kv)
            s.cache[i].view(-1, code.shape[1])[at] = torch.where((scale > 0).unsqueeze(1), code, torch.zeros_like(code))
            s.scales[i].view(-1)[at] = torch.where(scale > 0, scale, torch.ones_like(scale))


@KV
@pytest.mark.parametrize("step", [-30.0, -3.0, 2.0, 5.0, 9.0, 11.0, 16.0, 18.0, 25.0, 60.0])
def test_logits_by_steps(step, kv):
    """Every 128 positions the logits rise or fall by `step`: references move within all ranges that weights have, or not at all."""
    s = Step([9], [1000], kv, seed=21)
    n = int(s.lens[0])
    noise = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    _with_logits(s, 0, noise + step * (torch.arange(n, device="cuda") // 128))
    s.run()


@KV
@pytest.mark.parametrize("below", [9.0, 13.5, 15.45, 16.2])
def test_one_key_and_many_equal_ones_far_below(below, kv):
    """One key of weight 1 and 40000 of weight 2^-below, all rounded the same way."""
    s = Step([1], [40000], kv, seed=22)
    n = int(s.lens[0])
    logits = torch.full((n,), -below * np.log(2.0), device="cuda")
    logits[100] = 0.0
    v = torch.ones(n, device="cuda")
    v[100] = -1.0
    _with_logits(s, 0, logits, v)
    s.run()
    out, _, _, _ = s.reference(0)
    # the output's half step; weights, and values on a quantised cache, by half a step each (bf16 2^-8, f16 2^-11) of a mean of
    # values of 1, below 2^-14 by 2^-25 each instead; a sum of 1 at least
    half = 2 ** -8 if kv == "bf16" else 2 ** -11
    assert float((s.out[int(s.starts[0])].double() - out[0]).abs().max()) <= 2 ** -8 * float(out.abs().max()) + 2 * half + 2 * n * 2 ** -25


@pytest.mark.parametrize("kv", ["fp8", "fp4"])
def test_value_scales_far_apart(kv):
    """V scales from 2^-40 to 2^20 beside each other: large values without weight, small ones with all of it."""
    s = Step([21, 2], [300, 90], kv, seed=15)
    exponent = torch.randint(-40, 21, s.scales[1].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    s.scales[1].copy_(torch.where(torch.isfinite(s.scales[1]), torch.exp2(exponent.float()), s.scales[1]))
    s.run()


def _poison(s, i, b, j, what):
    """Position j of sequence b of cache i becomes `what`."""
    if s.kv == "bf16":
        s.cache[i].view(-1, DIM)[s.row(b, j)] = what
    elif s.kv == "fp8" and what != what:
        s.cache[i].view(-1, DIM)[s.row(b, j)] = 0x7F
    else:
        s.scales[i].view(-1)[s.row(b, j)] = what


@KV
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("new,held,at", [(8, 60, 62), (8, 60, 67), (7, 121, 127), (6, 125, 128), (4, 0, 1), (131, 40, 100)])
def test_a_later_position_never_reaches_an_earlier_token(new, held, at, what, kv):
    """K and V of one of the new positions are no numbers: the tokens before it come out as without it, bit for bit."""
    s = Step([new, 3], [held, 77], kv, seed=16)
    s.call()
    clean, clean_lse = s.out.clone(), s.lse.clone()
    for i in range(2):
        _poison(s, i, 0, at, what)
    s.call()
    capi.mfa_check_device_errors(s.ws)
    free = [r for r in range(new) if held + r < at] + [new, new + 1, new + 2]
    assert torch.equal(s.out[free], clean[free]) and torch.equal(s.lse[free], clean_lse[free])
    assert torch.isfinite(s.out[free]).all()
    if what != what:  # and those that see it do see it
        assert torch.isnan(s.out[at - held:new]).all()


@KV
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("new,held,at", [(6, 125, 128), (7, 121, 125), (3, 0, 2), (2000, 37, 1900)])
def test_a_value_that_is_no_number_reaches_every_token_that_sees_it(new, held, at, what, kv):
    s = Step([new], [held], kv, seed=17)
    _poison(s, 1, 0, at, what)
    s.call()
    seeing = s.out[at - held:]
    assert torch.isfinite(s.out[:at - held]).all()
    if what != what or kv != "bf16":  # (an infinite scale times codes of zero gives NaN as well)
        assert (~torch.isfinite(seeing)).all()
    else:
        assert (seeing == what).all()
    assert torch.isfinite(s.lse).all()


@KV
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_query_rows_do_not_meet(kv, what):
    """A query that is no number makes its own rows so and no others."""
    s = Step([9], [100], kv, seed=18)
    s.q[4, 7, 3] = what
    s.call()
    bad = torch.zeros((9, HEADS), dtype=torch.bool, device="cuda")
    bad[4, 7] = True
    assert torch.isnan(s.out[bad]).all() and torch.isfinite(s.out[~bad]).all()
    assert torch.isnan(s.lse[bad]).all() and torch.isfinite(s.lse[~bad]).all()


@KV
@pytest.mark.parametrize("power", [-133, -126, -110, -60, -9, 9, 40, 100])
def test_query_norms(kv, power):
    """Queries from the smallest bf16 numbers to the largest, the scale undoing their power where fp32 holds it: 100 elements of a
    row are 2^-10 of the others, so that both terms of a quantised cache's queries count."""
    s = Step([6], [300], kv, seed=28, pad=0)
    s.q[:, :, :100] *= 2.0 ** -10
    s.q.copy_((s.q.double() * 2.0 ** power).bfloat16())
    s.run(scale=SCALE * 2.0 ** min(max(-power, -100), 120))


@KV
def test_same_as_single_tokens(kv):
    """A chunk's tokens, one call each: the same to within both calls' roundings."""
    s = Step([11], [250], kv, seed=19).run()
    whole = s.out.double()
    for t in range(11):
        s.d_lens.fill_(251 + t)
        s.d_starts.copy_(torch.tensor([t, t + 1]))
        s.call()
        top = float(values(s.cache[1], s.scales[1] if s.scales else None, kv).nan_to_num().abs().max())
        assert (s.out[t].double() - whole[t]).abs().max() <= 2 * (2 ** -8 * 2 * top + 2 ** -12 * top)


# ---------------------------------------------------------------- how it is called
@KV
def test_repeated_calls_give_the_same_bits(kv):
    s = Step([37, 1, 200, 5], [900, 4000, 11, 64], kv, seed=20).run()
    first, first_lse = s.out.clone(), s.lse.clone()
    for _ in range(20):
        s.out.fill_(7)
        s.call()
        assert torch.equal(s.out, first) and torch.equal(s.lse, first_lse)


@KV
def test_captured_and_replayed_with_other_lengths(kv):
    """A graph reads lengths, starts and tables when it is replayed."""
    s = Step([60, 1, 9], [300, 500, 0], kv, seed=21, pad=0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.call()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.call()
    for new, lens in (([60, 1, 9], [360, 501, 9]), ([20, 1, 40], [200, 333, 9]), ([0, 70, 0], [0, 501, 9]), ([1, 1, 1], [1, 2, 3])):
        s.new, s.lens = np.array(new), np.array(lens)
        s.starts = np.concatenate([[0], np.cumsum(new)])
        s.d_lens.copy_(torch.from_numpy(s.lens))
        s.d_starts.copy_(torch.from_numpy(s.starts))
        s.out.fill_(7)
        s.lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        s.check()


@KV
def test_two_calls_at_once(kv):
    """On streams of their own, each with its workspace."""
    steps = [Step([150, 3], [1000, 20], kv, seed=22), Step([1] * 30, [800] * 30, kv, seed=23)]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s, st in zip(steps, streams):
            s.call(stream=st)
    torch.cuda.synchronize()
    for s in steps:
        s.check()


def test_formats_one_after_the_other_in_one_workspace():
    steps = [Step([90, 2], [700, 31], kv, seed=24) for kv in ("bf16", "fp8", "fp4")]
    for s in steps:
        s.ws = steps[0].ws
    for s in steps * 2:
        s.call()
    for s in steps:
        s.check()


# ---------------------------------------------------------------- what only the device sees
@KV
def test_bad_pages_and_lengths(kv):
    s = Step([10, 10, 10], [200, 150, 90], kv, seed=25)
    s.d_table[0, 1] = s.num_pages
    s.d_table[0, 2] = -5
    s.call()
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(s.ws)
    assert e.value.status == 5
    s.check(which=[1, 2])
    s.d_table[0, 1:3] = torch.from_numpy(s.table[0, 1:3])
    s.d_lens[1] = s.table.shape[1] * PAGE + 1
    s.d_table[1, 3:] = int(s.table[1, 0])
    s.call()
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(s.ws)
    assert e.value.status == 6
    s.check(which=[0, 2])
    s.d_lens[1] = -3
    s.call()
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(s.ws)
    assert e.value.status == 6
    assert (s.out[10:20] == 0).all()
    s.check(which=[0, 2])


@pytest.mark.parametrize("B", [3, 50])
def test_bad_starts(B):
    """Starts that fall are raised to the largest before them, ones past the rows lowered to their number."""
    s = Step([6] * B, [100] * B, seed=26)
    bad = s.starts.copy()
    bad[2] = -4
    bad[B] = s.rows + 100
    s.d_starts.copy_(torch.from_numpy(bad))
    s.call()
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(s.ws)
    assert e.value.status == 6
    s.check(which=[0] + list(range(3, B)))


@KV
def test_waits_without_a_budget_give_up_and_the_next_call_is_whole(kv):
    """Ten calls whose waits have no budget: a call is right or reports a wait that gave up, at least one of them does report
    it (a copy takes longer than two looks at its barrier), and a call with the usual budget behind each is whole."""
    s = Step([300, 5], [2000, 70], kv, seed=27)
    gave_up = 0
    try:
        for _ in range(10):
            capi.mfa_set_wait_budget_ns(0)
            s.call()
            torch.cuda.synchronize()
            capi.mfa_set_wait_budget_ns(2_000_000_000)
            try:
                s.check()
            except capi.MFAError as e:
                assert e.status == 7
                gave_up += 1
            s.out.fill_(7.0)
            s.run()
    finally:
        capi.mfa_set_wait_budget_ns(2_000_000_000)
    assert gave_up >= 1
