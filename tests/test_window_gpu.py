"""Sliding-window attention with sinks (rq_decode_attn_window,
rq_prefill_attn_window) against a plain fp64 softmax over the keys and values
that the cache holds (rq_cache_export through the oracle's reconstruction, or
the stored BF16 values, then the BF16 tail).

Tolerances, fp32 output.  Decode of the compressed cache: value weights in 31
bits and q in 23 bits (and a sign) of fixed point relative to their largest, sums
in integers.  The logit error is at most 2^-23 max|q| times |k|_1: with |k|_1
below 128 * 3 (10 in 4 channels) and max|q| about 4, scaled by 1/sqrt(128), about
2e-5 at the very worst, and the output moves by at most twice that times the
values' spread: 2e-4 max abs and 2e-5 relative L2 leave a margin for fp32 sums.
The chunk kernel splits probabilities, keys and values into pairs of FP16 numbers
(compressed caches) or probabilities into BF16 pairs (2^-17): the contract's
1e-3 / 2e-3.  BF16 caches, decode: fp32 products and sums.  BF16 output adds half
a step, 2^-8 |x|; a chunk's weights are then one BF16 number (2^-9 of each), or
weights, keys and values one FP16 number (2^-12): at most 2 * 2^-9 max|v| with
|v| < 45, and 2^-8 of the row's norm at random signs.
"""
import numpy as np
import pytest
import torch

import decode_attention_14_b200 as rq
import synth
from oracle import oracle as orc

import rqharness as H

pytestmark = pytest.mark.gpu
BIG = 1 << 30


def keys_values(bt, layer, loop, lens):
    """Per sequence [2][H][len + n_tail][d] fp64: what (layer, loop) sees."""
    cfg = bt.cfg
    Lg, B, Hk = cfg.loops_per_group, cfg.batch, cfg.num_kv_heads
    if cfg.format == rq.RQ_FMT_BF16:
        X = bt.inputs[(layer, loop // Lg)]
        x = [orc.bf16_bits_to_f64(synth.bf16_to_u16(X[kv][loop % Lg])) for kv in range(2)]
        return [np.stack([x[kv][b, :lens[b]].transpose(1, 0, 2) for kv in range(2)]) for b in range(B)]
    grp, j = loop // Lg, loop % Lg
    rec = [H.reconstruct_gpu(bt, layer, grp, kv).reshape(Lg, B, Hk, -1, 128)[j] for kv in range(2)]
    out = [np.stack([rec[kv][b, :, :lens[b]] for kv in range(2)]) for b in range(B)]
    if j != Lg - 1 and bt.n_tail:
        X = bt.inputs[(layer, grp)]
        for b in range(B):
            tail = np.stack([orc.bf16_bits_to_f64(synth.bf16_to_u16(X[kv][j][b:b + 1, bt.T:]))[0].transpose(1, 0, 2)
                             for kv in range(2)])
            out[b] = np.concatenate([out[b], tail], 2)
    return out


def reference(kv, q, window, sinks):
    """q [B][n][Hq][d] -> the same in fp64; each of the last n positions sees its window and the sinks."""
    qf = q.double().cpu().numpy()
    B, n, Hq, _ = qf.shape
    out = np.zeros_like(qf)
    for b in range(B):
        k, v = kv[b]
        Hk, P = k.shape[0], k.shape[1]
        if P == 0:
            continue
        pos = np.arange(P - n, P)[:, None]
        t = np.arange(P)[None, :]
        seen = (t <= pos) & ((t > pos - window) | (t < sinks)) if window else t <= pos
        for h in range(Hq):
            z = qf[b, :, h] @ k[h * Hk // Hq].T / np.sqrt(128.0)
            z = np.where(seen, z, -np.inf)
            p = np.exp(z - z.max(1, keepdims=True))
            vv = np.where(seen.any(0)[:, None], v[h * Hk // Hq], 0.0)
            out[b, :, h] = (p / p.sum(1, keepdims=True)) @ vv
    return out


def check(out, ref, rel, mx):
    g = out.double().cpu().numpy().reshape(ref.shape)
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0
    far = np.maximum(np.abs(g - ref) - half * np.abs(ref), 0.0)
    assert np.isfinite(g).all()
    assert np.linalg.norm(far) <= rel * max(np.linalg.norm(ref), 1e-300) and far.max() <= mx, (
        np.linalg.norm(far) / max(np.linalg.norm(ref), 1e-300), far.max())


def queries(seed, *shape):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).bfloat16()


WINDOWS = [(1, 0), (1, 1), (2, 0), (63, 4), (64, 4), (65, 0), (100, 70), (128, 64), (150, 200), (0, 0), (0, 9),
           (BIG, 0), (BIG, 5)]


@pytest.mark.parametrize("T,n_tail", [(1, 0), (1, 1), (64, 1), (65, 3), (200, 0), (333, 2), (1000, 5)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_decode_windows(T, n_tail, out):
    bt = H.build(T=T, n_tail=n_tail, H=2, Hq=4, seed=0x5EEDBB01)
    q = queries(1, 1, 4, 128)
    for loop in (0, 3):
        kv = keys_values(bt, 0, loop, [T])
        for window, sinks in WINDOWS:
            ref = reference(kv, q[:, None], window, sinks)[:, 0]
            check(bt.cache.decode_window(0, loop, q, window, sinks, dtype=out), ref, 2e-5, 2e-4)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("kw", [
    dict(g=32), dict(ba=2), dict(br=4, g=32), dict(ba=2, br=4), dict(rotate=False), dict(Hq=2), dict(Hq=8), dict(Hq=16),
    dict(loops=2, Lg=1), dict(anchor_mode=rq.ANCHOR_CHAINED), dict(layers=2, rotation_per_layer=True),
    dict(B=3, block_tokens=128, num_blocks=24, prepare=lambda c: c.shuffle_free_blocks(5)),
    dict(B=3, block_tokens=256, num_blocks=12, prepare=lambda c: c.shuffle_free_blocks(5), Hq=8),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items() if k != "prepare"))
def test_decode_window_variants(kw):
    bt = H.build(**{"T": 700, "n_tail": 2, "H": 2, "Hq": 4, "seed": 0x5EEDBB02, **kw})
    cfg = bt.cfg
    q = queries(2, cfg.batch, cfg.num_q_heads, 128)
    layer = cfg.num_layers - 1
    for loop in range(cfg.num_loops):
        kv = keys_values(bt, layer, loop, [700] * cfg.batch)
        for window, sinks in ((300, 4), (64, 130), (257, 0)):
            ref = reference(kv, q[:, None], window, sinks)[:, 0]
            check(bt.cache.decode_window(layer, loop, q, window, sinks), ref, 2e-5, 2e-4)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("paged", [False, True])
def test_decode_windows_of_ragged_sequences(paged):
    """Sequences of different lengths, one empty: each has a window of its own; with no token at all the output is zero."""
    kw = dict(block_tokens=128, num_blocks=48, prepare=lambda c: c.shuffle_free_blocks(3)) if paged else {}
    bt = H.build(B=5, T=1100, H=2, Hq=2, seed=0x5EEDBB03, **kw)
    lens = [1100, 64, 0, 130, 129]
    for b in range(5):
        bt.cache.truncate_seq(0, 0, b, lens[b])
    K, V = bt.inputs[(0, 0)]
    q = queries(3, 5, 2, 128)

    def sweep(loop):
        kv = keys_values(bt, 0, loop, lens)
        for window, sinks in ((1, 0), (2, 1), (3, 0), (64, 4), (66, 200), (500, 64), (1030, 64), (1024, 0)):
            ref = reference(kv, q[:, None], window, sinks)[:, 0]
            check(bt.cache.decode_window(0, loop, q, window, sinks), ref, 2e-5, 2e-4)

    sweep(3)
    sweep(1)
    tail = torch.randn((2, 5, 3, 2, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    bt.cache.append(0, 1, tail[0].contiguous(), tail[1].contiguous())
    bt.inputs[(0, 0)] = tuple([torch.cat((X[j], tail[i]), 1) for j in range(4)] for i, X in ((0, K), (1, V)))
    bt.n_tail = 3
    sweep(1)
    bt.cache.check()
    bt.cache.close()


def test_decode_window_of_an_empty_cache():
    """Nothing committed: the tail alone, windows shorter than it; and nothing at all."""
    bt = H.build(T=0, n_tail=6, B=2, H=2, Hq=4, max_tokens=64, seed=0x5EEDBB04)
    q = queries(4, 2, 4, 128)
    for dtype in (torch.float32, torch.bfloat16):
        for window, sinks in ((1, 0), (2, 1), (3, 2), (6, 0), (0, 0), (4, 9)):
            kv = [
                np.stack([orc.bf16_bits_to_f64(synth.bf16_to_u16(bt.inputs[(0, 0)][i][0][b:b + 1]))[0].transpose(1, 0, 2)
                          for i in range(2)]) for b in range(2)]
            ref = reference(kv, q[:, None], window, sinks)[:, 0]
            check(bt.cache.decode_window(0, 0, q, window, sinks, dtype=dtype), ref, 2e-5, 2e-4)
        assert (bt.cache.decode_window(0, 3, q, 5, 1, dtype=dtype) == 0).all()
    bt.cache.close()


@pytest.mark.parametrize("Hq", [2, 4, 16])
def test_decode_windows_of_a_bf16_cache(Hq):
    bt = H.build(loops=1, Lg=1, B=3, T=1300, H=2, Hq=Hq, fmt=rq.RQ_FMT_BF16, seed=0x5EEDBB05)
    lens = [1300, 77, 0]
    for b in range(3):
        bt.cache.truncate_seq(0, 0, b, lens[b])
    q = queries(5, 3, Hq, 128)
    kv = keys_values(bt, 0, 0, lens)
    for dtype in (torch.float32, torch.bfloat16):
        for window, sinks in WINDOWS + [(1234, 64), (700, 600)]:
            ref = reference(kv, q[:, None], window, sinks)[:, 0]
            check(bt.cache.decode_window(0, 0, q, window, sinks, dtype=dtype), ref, 4e-6, 4e-5)
    bt.cache.check()
    bt.cache.close()


def _poison(bt, layer, loop, where, value, chunk=64):
    """The group's K and V with `value` in whole rows of the tokens `where`, appended again."""
    K, V = ([x.clone() for x in X] for X in bt.inputs[(layer, 0)])
    for X in (K, V):
        for x in X:
            x[:, where] = value
    bt.cache.truncate(layer, 0, 0)
    bt.recon.clear()
    H.fill_group(bt, layer, 0, K, V, chunk)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("fmt", [rq.RQ_FMT_RESIDUAL, rq.RQ_FMT_BF16])
def test_decode_does_not_see_what_masked_tokens_hold(fmt, value):
    """NaN, infinities and the largest numbers in every token outside the window and the sinks, in K and V."""
    Lg = 4 if fmt == rq.RQ_FMT_RESIDUAL else 1
    bt = H.build(loops=Lg, Lg=Lg, T=300, H=2, Hq=4, fmt=fmt, seed=0x5EEDBB06, max_tokens=320)
    q = queries(6, 1, 4, 128)
    window, sinks = 100, 5
    ref = {loop: reference(keys_values(bt, 0, loop, [300]), q[:, None], window, sinks)[:, 0] for loop in range(Lg)}
    _poison(bt, 0, 0, slice(5, 200), value)
    for loop in range(Lg):
        check(bt.cache.decode_window(0, loop, q, window, sinks), ref[loop], 2e-5, 2e-4)
    bt.cache.close()


def test_decode_window_equals_itself_in_any_order_of_calls():
    """Bit-equal on repetition, on a side stream, in a replayed graph and between other calls on the cache; a window
    longer than the sequence agrees with rq_decode_attn to that call's precision."""
    bt = H.build(B=2, T=900, H=2, Hq=4, n_tail=1, seed=0x5EEDBB07)
    q = queries(7, 2, 4, 128)
    first = bt.cache.decode_window(0, 1, q, 333, 4)
    full = bt.cache.decode_window(0, 1, q, 0)
    ref = reference(keys_values(bt, 0, 1, [900, 900]), q[:, None], 0, 0)[:, 0]
    rel = lambda x: np.linalg.norm(x.double().cpu().numpy() - ref) / np.linalg.norm(ref)   # noqa: E731
    assert rel(full) <= 2e-5 and rel(bt.cache.decode(0, 1, q)) <= 1e-3
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    bt.cache.decode_window(0, 1, q, 333, 4, out=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    out2 = torch.zeros_like(first)
    with torch.cuda.graph(g):
        bt.cache.decode_window(0, 2, q, 50, 0)
        bt.cache.decode_window(0, 1, q, 333, 4, out=out2)
    for _ in range(3):
        out2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, first)
        bt.cache.decode(0, 1, q)
        assert torch.equal(bt.cache.decode_window(0, 1, q, 333, 4), first)
    bt.cache.check()
    bt.cache.close()


def test_a_decode_loop_with_a_window():
    """Token by token, as a serving loop runs: append, then decode with a window, every loop of the group."""
    bt = H.build(T=130, H=2, Hq=2, seed=0x5EEDBB08, max_tokens=200)
    K, V = synth.group_kv(99, 0, 0, 4, (0.1, 0.2, 0.3), 1, 140, 2, device="cuda")
    bt.cache.truncate(0, 0, 0)
    bt.T, bt.recon = 130, {}
    for t0 in range(0, 130, 64):
        for j in range(4):
            bt.cache.append(0, j, K[j][:, t0:min(130, t0 + 64)].contiguous(), V[j][:, t0:min(130, t0 + 64)].contiguous())
    for t in range(130, 136):
        for j in range(4):
            q = queries(1000 + 4 * t + j, 1, 2, 128)
            bt.cache.append(0, j, K[j][:, t:t + 1].contiguous(), V[j][:, t:t + 1].contiguous())
            got = bt.cache.decode_window(0, j, q, 70, 3)
            bt.T, bt.n_tail, bt.recon = (t if j < 3 else t + 1), (1 if j < 3 else 0), {}
            bt.inputs[(0, 0)] = ([k[:, :t + 1] for k in K], [v[:, :t + 1] for v in V])
            ref = reference(keys_values(bt, 0, j, [bt.T]), q[:, None], 70, 3)[:, 0]
            check(got, ref, 2e-5, 2e-4)
    bt.cache.close()


def test_window_refusals():
    bt = H.build(T=20, H=2, Hq=2, seed=0x5EEDBB09)
    q, out = queries(8, 1, 2, 128), torch.zeros((1, 2, 128), device="cuda")

    def call(layer=0, loop=0, qq=q, oo=out, kind=rq.RQ_OUT_FP32, window=4, sinks=1):
        return rq.rq_decode_attn_window(bt.cache.h, layer, loop, qq, oo, kind, 0.0, window, sinks)

    assert call() == rq.RQ_OK
    for kw in (dict(layer=1), dict(layer=-1), dict(loop=4), dict(loop=-1), dict(qq=None), dict(oo=None), dict(kind=2),
               dict(kind=-1), dict(window=-1), dict(sinks=-1)):
        assert call(**kw) == rq.RQ_ERR_INVALID, kw
    for bad in (q.float(), q[:, :1], q[..., ::2]):
        with pytest.raises(ValueError):
            bt.cache.decode_window(0, 0, bad, 4)
    with pytest.raises(ValueError):
        bt.cache.decode_window(0, 0, q, 4, out=out, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bt.cache.decode_window(0, 0, q, 4, dtype=torch.float16)
    with pytest.raises(rq.RQError):
        bt.cache.decode_window(0, 0, q, -4)
    bt.cache.close()


# ------------------------------------------------------------------ several tokens
def chunk_check(bt, loop, lens, n, window, sinks, dtype=torch.float32, seed=11, rel=None, mx=None):
    rel = rel or (1e-3 if dtype == torch.float32 else 2.0 ** -8)
    mx = mx or (2e-3 if dtype == torch.float32 else 0.18)
    q = queries(seed, bt.cfg.batch, n, bt.cfg.num_q_heads, 128)
    ref = reference(keys_values(bt, 0, loop, lens), q, window, sinks)
    check(bt.cache.prefill_window(0, loop, q, window, sinks, dtype=dtype), ref, rel, mx)


@pytest.mark.parametrize("T,n", [(1, 1), (40, 7), (64, 64), (65, 33), (200, 130), (700, 1), (700, 65), (1000, 300)])
@pytest.mark.parametrize("Hq", [2, 8])
def test_prefill_windows(T, n, Hq):
    """A committed chunk (the anchor loop) and one in the tail (a residual loop), T - n tokens before it."""
    bt = H.build(T=T, H=2, Hq=Hq, seed=0x5EEDCC01, n_tail=n, max_tokens=T + 1)
    for window, sinks in ((1, 0), (5, 2), (32, 0), (64, 4), (100, 70), (257, 3), (0, 0), (BIG, 0), (640, 700)):
        chunk_check(bt, 3, [T], n, window, sinks)
        chunk_check(bt, 1, [T], n, window, sinks, torch.bfloat16)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("kw", [
    dict(g=32), dict(ba=2), dict(br=4, g=32), dict(rotate=False), dict(Hq=16), dict(loops=2, Lg=1),
    dict(B=3, block_tokens=128, num_blocks=24, prepare=lambda c: c.shuffle_free_blocks(5)),
    dict(B=2, block_tokens=256, num_blocks=8, prepare=lambda c: c.shuffle_free_blocks(6), Hq=8),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items() if k != "prepare"))
def test_prefill_window_variants(kw):
    bt = H.build(**{"T": 700, "n_tail": 70, "H": 2, "Hq": 4, "seed": 0x5EEDCC02, **kw})
    for loop in range(bt.cfg.num_loops):
        for window, sinks in ((300, 4), (64, 130), (33, 0)):
            n = 150 if loop % bt.cfg.loops_per_group == bt.cfg.loops_per_group - 1 else 70
            chunk_check(bt, loop, [700] * bt.cfg.batch, n, window, sinks)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("paged", [False, True])
def test_prefill_windows_of_ragged_sequences(paged):
    kw = dict(block_tokens=128, num_blocks=48, prepare=lambda c: c.shuffle_free_blocks(3)) if paged else {}
    bt = H.build(B=5, T=1100, H=2, Hq=4, seed=0x5EEDCC03, **kw)
    lens = [1100, 64, 40, 130, 129]
    for b in range(5):
        bt.cache.truncate_seq(0, 0, b, lens[b])
    for window, sinks in ((1, 0), (3, 1), (64, 4), (66, 200), (500, 64), (0, 0)):
        chunk_check(bt, 3, lens, 40, window, sinks)
    bt.cache.truncate_seq(0, 0, 2, 0)
    lens[2] = 0
    K, V = bt.inputs[(0, 0)]
    tail = torch.randn((2, 5, 90, 2, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    bt.cache.append(0, 1, tail[0].contiguous(), tail[1].contiguous())
    bt.inputs[(0, 0)] = tuple([torch.cat((X[j], tail[i]), 1) for j in range(4)] for i, X in ((0, K), (1, V)))
    bt.n_tail = 90
    for n in (1, 33, 90):                    # all of the tail, and its last part
        for window, sinks in ((1, 0), (3, 1), (64, 4), (66, 200), (500, 64), (30, 1200), (0, 0)):
            chunk_check(bt, 1, lens, n, window, sinks)
    bt.cache.check()
    bt.cache.close()


def test_prefill_window_of_a_cache_without_committed_tokens():
    """The first chunk of a prompt at a residual loop: everything is in the tail."""
    bt = H.build(T=0, n_tail=500, B=2, H=2, Hq=4, max_tokens=64, seed=0x5EEDCC04)
    for n in (1, 200, 500):
        for window, sinks in ((1, 0), (64, 4), (100, 450), (0, 0)):
            q = queries(12, 2, n, 4, 128)
            kv = [np.stack([orc.bf16_bits_to_f64(synth.bf16_to_u16(bt.inputs[(0, 0)][i][0][b:b + 1]))[0].transpose(1, 0, 2)
                            for i in range(2)]) for b in range(2)]
            check(bt.cache.prefill_window(0, 0, q, window, sinks), reference(kv, q, window, sinks), 1e-3, 2e-3)
    bt.cache.check()
    bt.cache.close()


def test_a_chunk_longer_than_its_window():
    """Row blocks that see neither the chunk's beginning nor its end, one split each; window and sinks apart."""
    bt = H.build(T=600, n_tail=1500, H=16, Hq=16, seed=0x5EEDCC05, chunk=300, max_tokens=2200)
    chunk_check(bt, 0, [600], 1500, 200, 10)
    chunk_check(bt, 0, [600], 1500, 700, 0, torch.bfloat16)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("where", ["committed", "tail"])
def test_prefill_does_not_see_what_masked_tokens_hold(where, value):
    """One poisoned token, in K and V: rows that do not see it are as if it held zeros; rows that do may be anything."""
    T, n = 300, 80
    bt = H.build(T=T, H=2, Hq=4, seed=0x5EEDCC06, n_tail=n, max_tokens=512)
    K, V = ([x.clone() for x in X] for X in bt.inputs[(0, 0)])
    at = 250 if where == "committed" else T + 30
    for X in (K, V):
        for x in X:
            x[:, at] = value
    ref_in = tuple([x.clone() for x in X] for X in bt.inputs[(0, 0)])
    kv0 = {loop: keys_values(bt, 0, loop, [T]) for loop in (0, 3)}
    bt.cache.append(0, 3, *[x[3][:, T:].contiguous() for x in ref_in])     # commits the tails, so that it can be emptied
    bt.cache.truncate(0, 0, 0)
    bt.recon.clear()
    H.fill_group(bt, 0, 0, K, V, 64)
    bt.inputs[(0, 0)] = ref_in
    window, sinks = 40, 5
    for loop in (0, 3):
        P = T + (n if loop == 0 else 0)
        m = n if loop == 0 else 120
        q = queries(13, 1, m, 4, 128)
        ref = reference(kv0[loop], q, window, sinks)
        got = bt.cache.prefill_window(0, loop, q, window, sinks).double().cpu().numpy()
        pos = np.arange(P - m, P)
        blind = (at > pos) | ((at <= pos - window) & (at >= sinks))
        assert blind.any()
        assert np.isfinite(got[:, blind]).all()
        far = np.abs(got[:, blind] - ref[:, blind])
        assert far.max() <= 2e-3 and np.linalg.norm(far) <= 1e-3 * np.linalg.norm(ref[:, blind])
        if np.isnan(value) and (~blind).any():
            assert np.isnan(got[:, ~blind]).all()      # where it is seen, it shows
    bt.cache.close()


def test_prefill_window_equals_itself_in_any_order_of_calls():
    bt = H.build(B=2, T=900, H=2, Hq=4, n_tail=40, seed=0x5EEDCC07)
    q = queries(14, 2, 40, 4, 128)
    first = bt.cache.prefill_window(0, 1, q, 333, 4)
    # window 0 is rq_prefill_attn; one token is the single-token call
    check(bt.cache.prefill_window(0, 1, q, 0), bt.cache.prefill(0, 1, q).double().cpu().numpy(), 1e-4, 1e-3)
    one = bt.cache.prefill_window(0, 1, q[:, -1:].contiguous(), 333, 4)
    check(one, bt.cache.decode_window(0, 1, q[:, -1].contiguous(), 333, 4)[:, None].double().cpu().numpy(), 1e-4, 1e-3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    bt.cache.prefill_window(0, 1, q, 333, 4, out=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    out2 = torch.zeros_like(first)
    with torch.cuda.graph(g):
        bt.cache.prefill_window(0, 2, q, 50, 0)
        bt.cache.prefill_window(0, 1, q, 333, 4, out=out2)
    for _ in range(3):
        out2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, first)
        bt.cache.prefill(0, 1, q)
        assert torch.equal(bt.cache.prefill_window(0, 1, q, 333, 4), first)
    bt.cache.check()
    bt.cache.close()


def test_prefill_window_refusals():
    bt = H.build(T=20, n_tail=4, H=2, Hq=2, seed=0x5EEDCC09)
    q, out = queries(8, 1, 4, 2, 128), torch.zeros((1, 4, 2, 128), device="cuda")

    def call(layer=0, loop=0, qq=q, n=4, oo=out, kind=rq.RQ_OUT_FP32, window=4, sinks=1):
        return rq.rq_prefill_attn_window(bt.cache.h, layer, loop, qq, n, oo, kind, 0.0, window, sinks)

    assert call() == rq.RQ_OK
    for kw in (dict(layer=1), dict(layer=-1), dict(loop=4), dict(loop=-1), dict(qq=None), dict(oo=None), dict(kind=2),
               dict(n=0), dict(n=-1), dict(window=-1), dict(sinks=-1)):
        assert call(**kw) == rq.RQ_ERR_INVALID, kw
    assert call(n=25) == rq.RQ_ERR_STATE and call(loop=3, n=21) == rq.RQ_ERR_STATE
    with pytest.raises(ValueError):
        bt.cache.prefill_window(0, 0, q[:, :, :1], 4)
    with pytest.raises(ValueError):
        bt.cache.prefill_window(0, 0, q, 4, out=out, dtype=torch.bfloat16)
    for kw in (dict(ba=2, br=4), dict(anchor_mode=rq.ANCHOR_CHAINED)):
        other = H.build(T=20, H=2, Hq=2, seed=0x5EEDCC0A, **kw)
        with pytest.raises(rq.RQError) as e:
            other.cache.prefill_window(0, 3, q, 4)
        assert e.value.status == rq.RQ_ERR_UNSUPPORTED
        other.cache.close()
    bt.cache.close()


# ------------------------------------------------------------------ several tokens over a BF16 cache
def _bf16(T, B=1, H_=2, Hq=2, lens=None, seed=0x5EEDDD01):
    bt = H.build(loops=1, Lg=1, B=B, T=T, H=H_, Hq=Hq, fmt=rq.RQ_FMT_BF16, seed=seed, max_tokens=T + 3)
    for b, n in enumerate(lens or []):
        bt.cache.truncate_seq(0, 0, b, n)
    return bt, lens or [T] * B


# fp32 output: weights to 2^-17 relative (BF16 pairs), 2^-22 exponentials, fp32 sums: 1e-5 of the row; BF16 output:
# weights to half a BF16 step, 2^-9 (at random over the tokens: of the row's norm; at most 2^-9 max|v|, |v| < 45), on top of
# the output's own half step
@pytest.mark.parametrize("T,n", [(1, 1), (5, 5), (127, 3), (128, 128), (129, 129), (257, 130), (640, 65), (1000, 700)])
@pytest.mark.parametrize("Hq", [2, 8, 16])
def test_prefill_windows_of_a_bf16_cache(T, n, Hq):
    bt, lens = _bf16(T, Hq=Hq)
    for window, sinks in ((0, 0), (1, 0), (5, 2), (64, 4), (128, 0), (200, 150), (BIG, 3)):
        chunk_check(bt, 0, lens, n, window, sinks, torch.float32, rel=1e-5, mx=2e-4)
        chunk_check(bt, 0, lens, n, window, sinks, torch.bfloat16, rel=2.0 ** -9, mx=9e-2)
    bt.cache.check()
    bt.cache.close()


def test_prefill_windows_of_ragged_bf16_sequences():
    bt, lens = _bf16(1500, B=4, Hq=4, lens=[1500, 70, 300, 129])
    for n in (1, 33, 70):
        for window, sinks in ((0, 0), (1, 1), (64, 4), (257, 130), (1000, 0)):
            chunk_check(bt, 0, lens, n, window, sinks, rel=1e-5, mx=2e-4)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_prefill_of_a_long_bf16_chunk(dtype):
    """Enough rows for two row tiles a CTA: the whole prompt, and a window with sinks."""
    bt, lens = _bf16(2300, B=1, H_=16, Hq=32)
    tol = dict(rel=1e-5, mx=2e-4) if dtype == torch.float32 else dict(rel=2.0 ** -9, mx=9e-2)
    chunk_check(bt, 0, lens, 2300, 0, 0, dtype, **tol)
    chunk_check(bt, 0, lens, 2201, 300, 20, dtype, **tol)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [80, 600])
def test_bf16_prefill_does_not_see_what_masked_tokens_hold(value, n):
    T, at = 700, 650
    bt, lens = _bf16(T, H_=16, Hq=16 if n == 80 else 32)
    K, V = bt.inputs[(0, 0)]
    kv0 = keys_values(bt, 0, 0, lens)
    bt.cache.truncate(0, 0, 0)
    K, V = ([X[0].clone()] for X in (K, V))
    for X in (K, V):
        X[0][:, at] = value
        X[0][:, 3:40] = value                # beside the sinks, far outside every window
    bt.cache.append(0, 0, K[0].contiguous(), V[0].contiguous())
    q = queries(15, 1, n, bt.cfg.num_q_heads, 128)
    window, sinks = 40, 3
    ref = reference(kv0, q, window, sinks)
    pos = np.arange(T - n, T)
    blind = (at > pos) | (at <= pos - window)
    for dtype, tol in ((torch.float32, 1e-5), (torch.bfloat16, 2.0 ** -8)):
        got = bt.cache.prefill_window(0, 0, q, window, sinks, dtype=dtype).double().cpu().numpy()
        rows = blind & (pos >= 40 + window)      # those that also see none of 3 .. 39
        assert rows.any() and np.isfinite(got[:, rows]).all()
        assert np.linalg.norm(got[:, rows] - ref[:, rows]) <= tol * np.linalg.norm(ref[:, rows])
        if np.isnan(value):
            assert np.isnan(got[:, ~blind]).all()
    bt.cache.check()
    bt.cache.close()


def test_bf16_prefill_repeats_itself():
    bt, lens = _bf16(1500, B=2, Hq=4, lens=[1500, 900])
    q = queries(16, 2, 33, 4, 128)
    first = bt.cache.prefill_window(0, 0, q, 700, 4)
    one = bt.cache.prefill_window(0, 0, q[:, -1:].contiguous(), 700, 4)
    check(one, bt.cache.decode_window(0, 0, q[:, -1].contiguous(), 700, 4)[:, None].double().cpu().numpy(), 1e-5, 2e-4)
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(rq.RQError) as e:           # more splits than any call so far: no room, and none while capturing
            bt.cache.prefill_window(0, 0, q, 0)
        assert e.value.status == rq.RQ_ERR_NOMEM
        bt.cache.prefill_window(0, 0, q, 700, 4, out=out)
    g.replay()
    assert torch.equal(out, first)
    bt.cache.prefill_window(0, 0, q, 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bt.cache.prefill_window(0, 0, q, 0)
        bt.cache.prefill_window(0, 0, q, 700, 4, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, first)
        assert torch.equal(bt.cache.prefill_window(0, 0, q, 700, 4), first)
    with pytest.raises(rq.RQError) as e:
        bt.cache.prefill(0, 0, q)
    assert e.value.status == rq.RQ_ERR_STATE
    bt.cache.check()
    bt.cache.close()


def test_prefill_window_beyond_one_workspace():
    """More rebuilt rows than the workspace holds at once (4 GiB): the kv heads go in groups.  8 sequences of 160 000
    tokens at an anchor loop; the last of five tokens' rows against the single-token call, for every head."""
    B, Hk, T = 8, 4, 160000
    cfg = rq.make_config(num_layers=1, num_loops=1, loops_per_group=1, batch=B, max_tokens=T, max_tail_tokens=0,
                         num_kv_heads=Hk, num_q_heads=Hk)
    cache = H.guarded_cache(cfg)
    g = torch.Generator("cuda").manual_seed(3)
    for t in range(0, T, 20000):
        k, v = (torch.randn((B, 20000, Hk, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
        cache.append(0, 0, k, v)
    q = queries(17, B, 5, Hk, 128)
    got = cache.prefill_window(0, 0, q, 0)
    ref = cache.decode_window(0, 0, q[:, -1].contiguous(), 0).double().cpu().numpy()
    for h in range(Hk):
        g_h, r_h = got[:, -1, h].double().cpu().numpy(), ref[:, h]
        assert np.linalg.norm(g_h - r_h) <= 1e-3 * np.linalg.norm(r_h) and np.abs(g_h - r_h).max() <= 2e-3, h
    cache.check()
    cache.close()


@pytest.mark.parametrize("Hq,paged", [(64, False), (32, True)])
def test_a_few_tokens_over_many(Hq, paged):
    """Chunks short enough to run token by token: committed, in the tail, and partly in each; one longer."""
    kw = dict(block_tokens=128, num_blocks=70, prepare=lambda c: c.shuffle_free_blocks(3)) if paged else {}
    bt = H.build(loops=2, Lg=2, B=2, T=4200, H=32, Hq=Hq, seed=0x5EEDEE04, **kw)
    lens = [4200, 4137]
    bt.cache.truncate_seq(0, 0, 1, lens[1])
    K, V = bt.inputs[(0, 0)]
    tail = torch.randn((2, 2, 2, 32, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    bt.cache.append(0, 0, tail[0].contiguous(), tail[1].contiguous())
    bt.inputs[(0, 0)] = tuple([torch.cat((X[j], tail[i]), 1) for j in range(2)] for i, X in ((0, K), (1, V)))
    bt.n_tail = 2
    for loop in (0, 1):
        kv = keys_values(bt, 0, loop, lens)
        for n in (1, 2, 3, 4, 5):
            q = queries(20 + n, 2, n, Hq, 128)
            for window, sinks, dtype in ((0, 0, torch.float32), (4150, 4, torch.bfloat16), (1100, 30, torch.float32)):
                few = n <= (4 if window != 1100 else 2)
                tol = (2e-5, 2e-4) if few else (1e-3, 2e-3) if dtype == torch.float32 else (2.0 ** -8, 0.18)
                check(bt.cache.prefill_window(0, loop, q, window, sinks, dtype=dtype), reference(kv, q, window, sinks), *tol)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("Hq", [8, 16])
def test_decode_of_grouped_heads_over_a_bf16_cache(Hq):
    """One pass over K and V for 4 or 8 heads (no sequence is empty); tolerances as for a chunk over such a cache.  Captured
    as the cache's first call too, and with an empty sequence, the same rows to the two paths' tolerances."""
    bt, lens = _bf16(1300, B=3, Hq=Hq, lens=[1300, 77, 1])
    q = queries(26, 3, Hq, 128)
    out, g = torch.zeros((3, Hq, 128), device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bt.cache.decode_window(0, 0, q, 700, 4, out=out)
    kv = keys_values(bt, 0, 0, lens)
    for window, sinks in WINDOWS + [(1234, 64), (700, 600)]:
        ref = reference(kv, q[:, None], window, sinks)[:, 0]
        check(bt.cache.decode_window(0, 0, q, window, sinks), ref, 1e-5, 2e-4)
        check(bt.cache.decode_window(0, 0, q, window, sinks, dtype=torch.bfloat16), ref, 2.0 ** -9, 9e-2)
    g.replay()
    assert torch.equal(out, bt.cache.decode_window(0, 0, q, 700, 4))
    bt.cache.truncate_seq(0, 0, 2, 0)
    with_empty = bt.cache.decode_window(0, 0, q, 700, 4)
    assert (with_empty[2] == 0).all()
    check(with_empty[:2], out[:2].double().cpu().numpy(), 1.4e-5, 2.4e-4)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("fmt", [rq.RQ_FMT_RESIDUAL, rq.RQ_FMT_BF16])
def test_a_captured_call_outlives_a_larger_one(fmt):
    """The buffers that a captured graph uses stay when a later, larger call outgrows them; so do rq_prefill_attn's."""
    Lg = 4 if fmt == rq.RQ_FMT_RESIDUAL else 1
    bt = H.build(loops=Lg, Lg=Lg, T=3000, H=2, Hq=4, fmt=fmt, seed=0x5EEDEE01)
    q = queries(18, 1, 300, 4, 128)
    small, out, loop = q[:, -2:].contiguous(), torch.zeros((1, 2, 4, 128), device="cuda"), Lg - 1
    plain = [torch.zeros_like(out)] if Lg == 4 else []
    first = bt.cache.prefill_window(0, loop, small, 600, 4)
    ref = [bt.cache.prefill(0, loop, small) for _ in plain]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bt.cache.prefill_window(0, loop, small, 600, 4, out=out)
        for p in plain:
            bt.cache.prefill(0, loop, small, out=p)
    big = bt.cache.prefill_window(0, loop, q, 0)                 # more splits, more rebuilt rows
    if plain:
        bt.cache.prefill(0, loop, q)
    junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(32)]     # would land in freed buffers
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(out, first) and all(torch.equal(p, r) for p, r in zip(plain, ref))
    assert torch.equal(bt.cache.prefill_window(0, loop, q, 0), big)
    del junk, g
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("fmt", [rq.RQ_FMT_RESIDUAL, rq.RQ_FMT_BF16])
def test_a_prompt_then_tokens_then_the_cache_read_back(fmt):
    """The operators as a serving loop uses them: a prompt in chunks (append, then the chunk's attention at every loop),
    then single tokens, all with one window and sinks; what is read back in the end is what the attention saw."""
    Lg, B, Hk, Hq, window, sinks = (4 if fmt == rq.RQ_FMT_RESIDUAL else 1), 2, 2, 4, 150, 6
    cfg = rq.make_config(num_layers=1, num_loops=Lg, loops_per_group=Lg, batch=B, max_tokens=512, max_tail_tokens=200,
                         num_kv_heads=Hk, num_q_heads=Hq, format=fmt)
    cache = H.guarded_cache(cfg)
    K, V = synth.group_kv(7, 0, 0, Lg, (0.1, 0.2, 0.3)[:max(Lg - 1, 1)], B, 400, Hk, device="cuda")
    done = 0
    for n in (130, 200, 1, 33, 1, 1):
        for j in range(Lg):
            cache.append(0, j, K[j][:, done:done + n].contiguous(), V[j][:, done:done + n].contiguous())
            q = queries(100 * done + j, B, n, Hq, 128)
            if n > 1:
                got = cache.prefill_window(0, j, q, window, sinks)
            else:
                got = cache.decode_window(0, j, q[:, 0].contiguous(), window, sinks)[:, None]
            k, v = (x.double().cpu().numpy().transpose(0, 2, 1, 3) for x in cache.read(0, j, dtype=torch.float32))
            assert k.shape[2] == done + n
            if j < Lg - 1:
                assert np.array_equal(k[:, :, done:], K[j][:, done:done + n].double().cpu().numpy().transpose(0, 2, 1, 3))
            check(got, reference([np.stack([k[b], v[b]]) for b in range(B)], q, window, sinks), 1e-3, 2e-3)
        done += n
    cache.check()
    cache.close()
