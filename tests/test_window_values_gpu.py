"""Values at the ends of the range for the windowed attention calls: small and
large numbers, weights far below the largest, tokens that are not finite, and
buffers that grow with the visible tokens.  The reference is a softmax in 64
bits over what the cache holds, read back in fp32 (a record's value in fp32 is
within a few 2^-24 of itself).

Tolerances, of each output row's norm.  fp32 output: a row and its weight are
two BF16 numbers each, off by at most half a step of the second, 2^-18: at
random signs over 128 products and over the tokens that is a few 1e-6 of the
logits and of the row, and the tensor cores' sums leave up to 3.5e-6: 2e-5.
BF16 output: half a step, 2^-9, of each element, of each weight and of each V; a
rounding's root mean square is 2^-9 / sqrt(3) at most, so all three, at random
signs, make 2^-9: 2^-8.
"""
import numpy as np
import pytest
import torch

import decode_attention_14_b200 as rq
import synth

import rqharness as H

pytestmark = pytest.mark.gpu
TOL = {torch.float32: 2e-5, torch.bfloat16: 2.0 ** -8}


def make(B=1, heads=2, Hq=2, Lg=4, max_tokens=512, tail=256, fmt=rq.RQ_FMT_RESIDUAL, **kw):
    return H.guarded_cache(rq.make_config(num_layers=1, num_loops=Lg, loops_per_group=Lg, batch=B, max_tokens=max_tokens,
                                          max_tail_tokens=tail if fmt == rq.RQ_FMT_RESIDUAL else 0, num_kv_heads=heads,
                                          num_q_heads=Hq, format=fmt, seed=0xA11CE, **kw))


def normal(seed, *shape):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


def reference(k, v, q, window, sinks, scale=128 ** -0.5):
    """k, v [B][P][H][d], q [B][n][Hq][d] -> [B][n][Hq][d] in 64 bits; tokens that no row sees may hold anything."""
    k, v, q = k.double(), v.double(), q.double()
    P, n, G = k.shape[1], q.shape[1], q.shape[2] // k.shape[2]
    pos = torch.arange(P - n, P, device="cuda")[:, None]
    t = torch.arange(P, device="cuda")[None, :]
    seen = (t <= pos) & ((t > pos - window) | (t < sinks)) if window else t <= pos
    k, v = (torch.where(seen.any(0)[None, :, None, None], x, 0.0).repeat_interleave(G, 2) for x in (k, v))
    z = torch.einsum("bihd,bjhd->bhij", q, k) * scale
    return torch.einsum("bhij,bjhd->bihd", torch.softmax(z.masked_fill(~seen, -float("inf")), -1), v)


def close(got, ref, tol):
    """Every row within tol of its norm."""
    far = (got.double() - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert bool((far <= tol).all()), far.max().item()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("size", [3e3, 1.0, 1e-2, 1e-4, 1e-6, 1e-12])
def test_chunks_over_values_of_any_size(size, dtype):
    """Tail rows of one size after committed ones of about 1: windows that see the tail alone, and both."""
    cache = make(B=2, heads=2, Hq=4)
    for j in range(4):
        cache.append(0, j, normal(j, 2, 100, 2, 128).bfloat16(), normal(9 + j, 2, 100, 2, 128).bfloat16())
    k, v = (normal(s, 2, 60, 2, 128) * size for s in (20, 21))
    cache.append(0, 1, (k if size < 10 else k / size).bfloat16(), v.bfloat16())     # (a large K leaves one token of a row)
    kr, vr = cache.read(0, 1, dtype=torch.float32)
    q = normal(22, 2, 40, 4, 128).bfloat16()
    for window, sinks in ((8, 0), (20, 0), (64, 0), (20, 5), (0, 0)):
        close(cache.prefill_window(0, 1, q, window, sinks, dtype=dtype), reference(kr, vr, q, window, sinks), TOL[dtype])
    cache.check()
    cache.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("size", [1e-3, 1e-2, 1.0, 30.0])
def test_chunks_over_records_of_any_size(size, dtype):
    """Committed rows, anchor and residual loops (FP8 scales reach down to 2^-9)."""
    cache = make(heads=2, Hq=4, max_tokens=400)
    for t in (0, 200):
        for j in range(4):
            cache.append(0, j, (normal(t + j, 1, 200, 2, 128) * min(size, 1.0)).bfloat16(),
                         (normal(t + 9 + j, 1, 200, 2, 128) * size).bfloat16())
    q = normal(23, 1, 50, 4, 128).bfloat16()
    for loop in (0, 3):
        kr, vr = cache.read(0, loop, dtype=torch.float32)
        for window, sinks in ((30, 0), (150, 4), (0, 0)):
            ref = reference(kr, vr, q, window, sinks)
            got = cache.prefill_window(0, loop, q, window, sinks, dtype=dtype)
            far = (got.double() - ref).norm() / ref.norm()      # (rows of records that are all zero have no norm)
            assert far <= TOL[dtype], far.item()
    cache.check()
    cache.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_chunk_queries_of_any_size(dtype):
    """q and the scale moved by powers of two against one another: the same logits, so the same bits."""
    cache = make(heads=2, Hq=4)
    for j in range(4):
        cache.append(0, j, normal(j, 1, 150, 2, 128).bfloat16(), normal(9 + j, 1, 150, 2, 128).bfloat16())
    q = normal(24, 1, 40, 4, 128).bfloat16()
    first = cache.prefill_window(0, 1, q, 70, 3, dtype=dtype, scale=2.0 ** -4)
    for e in (-40, -20, 15, 30):
        assert torch.equal(cache.prefill_window(0, 1, q * 2.0 ** e, 70, 3, dtype=dtype, scale=2.0 ** (-4 - e)), first), e
    cache.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("at", [0, 4000])
@pytest.mark.parametrize("below", [12.0, 17.5, 30.0])
def test_weights_far_below_the_largest(below, at, dtype):
    """One token's logit is `below` above all others', and its V is zero: the row is what the others' small weights make
    of theirs."""
    T, n = 8192, 40
    cache = make(heads=1, Hq=1, Lg=1, max_tokens=T)
    k, v = torch.zeros((1, T, 1, 128), device="cuda"), normal(31, 1, T, 1, 128) + 1.0
    u = torch.sign(normal(32, 128))
    k[0, at, 0], v[0, at, 0] = u, 0.0
    cache.append(0, 0, k.bfloat16(), v.bfloat16())
    kr, vr = cache.read(0, 0, dtype=torch.float32)
    q = (u * below / 128 ** 0.5).expand(1, n, 1, 128).bfloat16().contiguous()
    ref = reference(kr, vr, q, 0, 0)
    far = (ref.norm(dim=-1) * np.exp(below) / T).min().item()
    assert 1.0 < far, far                                   # the dominant token leaves the others e^-below each
    close(cache.prefill_window(0, 0, q, 0, dtype=dtype), ref, TOL[dtype])
    cache.check()
    cache.close()


def test_masked_tokens_between_the_runs_of_one_split():
    """Nearly the whole of the longest cache is visible: the sequence is dealt out as one, and whole tiles inside a split
    are masked.  What they hold does not show."""
    T, sinks, window = 262144, 1088, 260480
    cache = make(heads=1, Hq=1, Lg=1, max_tokens=T)
    clean = make(heads=1, Hq=1, Lg=1, max_tokens=T)
    for t in range(0, T, 1 << 16):
        k, v = (normal(t + i, 1, 1 << 16, 1, 128).bfloat16() for i in (1, 2))
        clean.append(0, 0, k, v)
        if t == 0:
            k[:, sinks:T - window], v[:, sinks:T - window] = float("nan"), float("nan")
        cache.append(0, 0, k, v)
    q = normal(33, 1, 1, 128).bfloat16()
    k, v = clean.read(0, 0, dtype=torch.float32)
    ref = reference(k, v, q[:, None], window, sinks)[:, 0]
    for dtype in TOL:
        close(clean.decode_window(0, 0, q, window, sinks, dtype=dtype), ref, TOL[dtype])
        close(cache.decode_window(0, 0, q, window, sinks, dtype=dtype), ref, TOL[dtype])
    cache.check()
    cache.close()
    clean.close()


@pytest.mark.parametrize("fmt,Hq", [(rq.RQ_FMT_RESIDUAL, 2), (rq.RQ_FMT_BF16, 2), (rq.RQ_FMT_BF16, 8)])
def test_rows_off_their_alignment_are_refused(fmt, Hq):
    """q or out at an odd element or 8 bytes on, contiguous all the same: refused before any launch, out as it was."""
    cache = make(heads=2, Hq=Hq, Lg=1, fmt=fmt)
    cache.append(0, 0, normal(61, 1, 50, 2, 128).bfloat16(), normal(62, 1, 50, 2, 128).bfloat16())
    rows = normal(63, 9 * Hq * 128).bfloat16()
    for n, call in ((1, cache.decode_window), (7, cache.prefill_window)):
        shape = (1, Hq, 128) if n == 1 else (1, n, Hq, 128)
        size = n * Hq * 128
        for dtype in TOL:
            space = torch.full((size + 16,), 7.0, dtype=dtype, device="cuda")
            for qo, oo in ((1, 0), (4, 0), (0, 1), (0, 2), (3, 1)):
                q, out = rows[qo:qo + size].view(shape), space[oo:oo + size].view(shape)
                with pytest.raises(ValueError, match="aligned"):
                    call(0, 0, q, 4, out=out)
                args = (cache.h, 0, 0, q) + ((n,) if n > 1 else ()) + (out, rq._out_type(dtype), 0.0, 4, 0)
                raw = rq.rq_decode_attn_window if n == 1 else rq.rq_prefill_attn_window
                assert raw(*args) == rq.RQ_ERR_INVALID
            torch.cuda.synchronize()
            assert (space == 7.0).all()
    cache.check()
    cache.close()


def test_appended_rows_off_their_alignment_are_refused():
    """k, v of an append (also the fused one) and q, out of rq_prefill_attn: refused before any launch, nothing appended."""
    cache = make(heads=2, Hq=2)
    bf = make(heads=2, Hq=2, Lg=1, fmt=rq.RQ_FMT_BF16)
    for j in range(4):
        cache.append(0, j, normal(j, 1, 20, 2, 128).bfloat16(), normal(9 + j, 1, 20, 2, 128).bfloat16())
    rows = normal(64, 9 * 2 * 128).bfloat16()
    at = lambda o, n=3: rows[o:o + n * 256].view(1, n, 2, 128)      # noqa: E731
    q, out = at(0, 1)[:, 0], torch.full((1, 2, 128), 7.0, device="cuda")
    for off in (1, 2, 4):
        for k, v in ((at(off), at(0)), (at(0), at(off))):
            assert rq.rq_append(bf.h, 0, 0, k, v, 3) == rq.RQ_ERR_INVALID
            assert rq.rq_append(cache.h, 0, 1, k, v, 3) == rq.RQ_ERR_INVALID
            assert rq.rq_append_decode_attn(cache.h, 0, 1, k, v, 3, q, out) == rq.RQ_ERR_INVALID
    assert bf.length(0, 0) == 0 and cache.tail_length(0, 1) == 0
    space = torch.full((3 * 256 + 8,), 7.0, device="cuda")
    for qo, oo in ((1, 0), (2, 0), (0, 1), (0, 2)):
        assert rq.rq_prefill_attn(cache.h, 0, 3, at(qo), 3, space[oo:oo + 768], 0.0) == rq.RQ_ERR_INVALID
    torch.cuda.synchronize()
    assert (space == 7.0).all() and (out == 7.0).all()
    for j in range(3):
        cache.append(0, j, at(0), at(0))
    for k, v in ((at(1), at(0)), (at(0), at(2))):
        assert rq.rq_append(cache.h, 0, 3, k, v, 3) == rq.RQ_ERR_INVALID
    assert rq.rq_append(cache.h, 0, 3, at(4), at(8), 3) == rq.RQ_OK      # 8 bytes do at the anchor loop
    k, v = cache.read(0, 3, t0=20, dtype=torch.float32)
    assert (k - at(4).float()).abs().max() <= 0.4 and (v - at(8).float()).abs().max() <= 0.4
    cache.check()
    cache.close()
    bf.close()


@pytest.mark.parametrize("captured", [False, True])
def test_buffers_of_a_growing_prompt(captured):
    """A prompt in chunks of 64, each of which sees all before it: the buffers that the cache keeps (after a captured call
    also those outgrown) take a small multiple of the largest call's, and few calls allocate."""
    heads, chunk, T = 8, 64, 8192
    cache = make(heads=heads, Hq=heads, Lg=1, max_tokens=T)
    k, v, q = (normal(s, 1, chunk, heads, 128).bfloat16() for s in (41, 42, 43))
    out = torch.empty((1, chunk, heads, 128), device="cuda")
    torch.cuda.synchronize()
    free = start = torch.cuda.mem_get_info()[0]
    steps = 0
    for t in range(0, T, chunk):
        cache.append(0, 0, k, v)
        cache.prefill_window(0, 0, q, 0, out=out)
        if t == 0 and captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                cache.prefill_window(0, 0, q, 0, out=out)
        now = torch.cuda.mem_get_info()[0]
        steps += now != free
        free = now
    need = heads * (T + 143) * 1024 + heads * chunk * 256 * 132 * 4     # rebuilt rows, and the most that partials take
    assert start - free <= 4 * need + (64 << 20), (start - free, need)
    assert steps <= 24, steps
    cache.check()
    cache.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("fmt,Hq", [(rq.RQ_FMT_RESIDUAL, 2), (rq.RQ_FMT_RESIDUAL, 8), (rq.RQ_FMT_BF16, 2), (rq.RQ_FMT_BF16, 8)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_visible_nan_shows(what, fmt, Hq, dtype):
    """A NaN in a visible token's K or V makes its kv head's rows NaN, in the single-token call as in a chunk, also where it
    is the only token seen; the other sequences' and heads' rows are as they were."""
    cache = make(B=3, heads=2, Hq=Hq, Lg=1, max_tokens=400, fmt=fmt)
    k, v = (normal(s, 3, 300, 2, 128).bfloat16() for s in (51, 52))
    (k if what == "k" else v)[1, 260:262, 1] = float("nan")
    cache.append(0, 0, k, v)
    cache.truncate_seq(0, 0, 1, 261)
    kr, vr = cache.read(0, 0, dtype=torch.float32)
    q = normal(53, 3, 1, Hq, 128).bfloat16()
    for window in (100, 1, 0):
        got = cache.decode_window(0, 0, q[:, 0].contiguous(), window, dtype=dtype)
        assert torch.isnan(got[1, Hq // 2:]).all(), window
        for b, heads in ((0, slice(0, Hq)), (1, slice(0, Hq // 2)), (2, slice(0, Hq))):
            P = 261 if b == 1 else 300
            kb, vb = (x[b:b + 1, :P].nan_to_num(0.0) for x in (kr, vr))
            ref = reference(kb, vb, q[b:b + 1], window, 0)[0, 0]
            close(got[b, heads], ref[heads], TOL[dtype])
    chunk = cache.prefill_window(0, 0, normal(54, 3, 9, Hq, 128).bfloat16(), 100, dtype=dtype)
    assert torch.isnan(chunk[1, -1, Hq // 2:]).all() and torch.isfinite(chunk[1, :-1]).all() and torch.isfinite(chunk[0]).all()
    cache.check()
    cache.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_a_nan_of_the_tail_shows(dtype):
    """The same for tail tokens, with committed ones before them and without."""
    for T in (0, 90):
        cache = make(heads=2, Hq=4)
        for j in range(4 if T else 0):
            cache.append(0, j, normal(j, 1, T, 2, 128).bfloat16(), normal(9 + j, 1, T, 2, 128).bfloat16())
        k, v = (normal(s, 1, 6, 2, 128).bfloat16() for s in (55, 56))
        k[0, 3, 1], v[0, 1, 0, 7] = float("nan"), float("nan")
        cache.append(0, 1, k, v)
        q = normal(57, 1, 4, 128).bfloat16()
        for window, sinks in ((6, 0), (4, 0), (2, 0), (3, 4) if T else (1, 4), (0, 0)):
            seen = lambda t: window == 0 or t >= 6 - window or T + t < sinks      # noqa: E731
            got = cache.decode_window(0, 1, q, window, sinks, dtype=dtype)
            assert torch.isnan(got[0, 2:]).all() == seen(3) and torch.isfinite(got[0, 2:]).all() == (not seen(3)), (T, window)
            assert torch.isnan(got[0, :2, 7]).all() == seen(1) and torch.isfinite(got[0, :2, :7]).all(), (T, window)
        cache.check()
        cache.close()


@pytest.mark.parametrize("Hkv,Hq,T", [(32, 32, 4200), (16, 16, 2100), (32, 128, 2100), (16, 128, 4200)])
def test_chunks_on_either_side_of_the_rule_for_few_tokens(Hkv, Hq, T):
    """One to seven tokens over many, one head per kv head and groups, an anchor and a residual loop, both output types: the
    rows agree with the formula wherever the rule sends them.

    BF16 output of a chunk has three roundings of at most half a step, 2^-9: the output's, d_o o, and in the sum those of each
    weight and of each V, sum_t p_t v_t (d_p + d_v).  Values here are independent with mean zero, so the norm of the sum is
    that of its terms, |o|^2 = sum_t p_t^2 |v_t|^2, and |sum_t p_t v_t d| <= 2^-9 |o| for roundings of either kind at random
    signs (their root mean square is smaller by sqrt(3) at least).  Together 3 2^-9, against a most likely 2.9e-3 = 1.5 2^-9."""
    tol = {torch.float32: TOL[torch.float32], torch.bfloat16: 3 * 2.0 ** -9}
    cache = make(B=2, heads=Hkv, Hq=Hq, Lg=2, max_tokens=T, tail=T)
    for j in range(2):
        cache.append(0, j, normal(70 + j, 2, T, Hkv, 128).bfloat16(), normal(72 + j, 2, T, Hkv, 128).bfloat16())
    for loop in (0, 1):
        kr, vr = cache.read(0, loop, dtype=torch.float32)
        for n in (1, 2, 3, 5, 6, 7):
            q = normal(80 + n, 2, n, Hq, 128).bfloat16()
            ref = torch.cat([reference(kr[b:b + 1], vr[b:b + 1], q[b:b + 1], 0, 0) for b in range(2)])
            for dtype in TOL:
                close(cache.prefill_window(0, loop, q, 0, dtype=dtype), ref, tol[dtype])
    cache.check()
    cache.close()


@pytest.mark.parametrize("handle", [False, True])
def test_new_outputs_on_another_stream_than_the_current_one(handle):
    """The current stream is busy for some milliseconds: rows that a call on a side stream writes into its own new tensors
    are not overwritten by their zeroing, and new tensors do not take memory that the current stream still works on."""
    cache = make(B=2, heads=2, Hq=4, Lg=1)
    cache.append(0, 0, normal(91, 2, 300, 2, 128).bfloat16(), normal(92, 2, 300, 2, 128).bfloat16())
    q1, qn = normal(93, 2, 4, 128).bfloat16(), normal(94, 2, 30, 4, 128).bfloat16()
    calls = [lambda **kw: cache.read(0, 0, **kw)[0], lambda **kw: cache.read(0, 0, dtype=torch.float32, **kw)[1],
             lambda **kw: cache.decode_window(0, 0, q1, 50, **kw), lambda **kw: cache.prefill_window(0, 0, qn, 50, **kw),
             lambda **kw: cache.decode(0, 0, q1, **kw), lambda **kw: cache.prefill(0, 0, qn, **kw)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for call, w in zip(calls, want):
        busy = torch.full(w.shape, 3.0, dtype=w.dtype, device="cuda")
        torch.cuda._sleep(20_000_000)                       # about 10 ms
        kept = busy * 2.0                                   # still to run when busy's memory is free again
        del busy
        got = call(stream=side.cuda_stream if handle else side)
        torch.cuda.synchronize()
        assert torch.equal(got, w) and (kept == 6.0).all()
        del got, kept
    cache.check()
    cache.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_a_chunk_whose_heads_go_in_groups(dtype):
    """More rebuilt rows than 4 GiB hold, and more tokens than run one by one: the last token's rows of every head against
    the single-token call (whose own error is 1e-6).

    The tensor cores cut their sums off: 24 accumulations per 128 tokens (three products of 8 steps), each by less than 2^-23
    of the sum.  40 row blocks are cut into 4 splits or more, of 40 000 tokens: 24 * 313 * 2^-23 = 9e-4, so 1e-3 for fp32
    output (2.4e-5 is what they come to).  BF16 output: three roundings of half a step at random signs beside it."""
    B, Hk, T, n = 8, 5, 160000, 7
    cache = make(B=B, heads=Hk, Hq=Hk, Lg=1, max_tokens=T)
    for t in range(0, T, 20000):
        cache.append(0, 0, normal(t, B, 20000, Hk, 128).bfloat16(), normal(t + 1, B, 20000, Hk, 128).bfloat16())
    q = normal(95, B, n, Hk, 128).bfloat16()
    ref = cache.decode_window(0, 0, q[:, -1].contiguous(), 0).double()
    got = cache.prefill_window(0, 0, q, 0, dtype=dtype)
    assert torch.isfinite(got).all()
    close(got[:, -1], ref, 1e-3 + (3 * 2.0 ** -9 if dtype == torch.bfloat16 else 0.0))
    cache.check()
    cache.close()
