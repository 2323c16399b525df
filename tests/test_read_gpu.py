"""Reading the cache back (rq_cache_read) against the oracle's fp64
reconstruction of the exported records.

Tolerance.  A value is x = s a + R^T y with |R^T y| <= |y|_2.  fp32 makes one
rounding per record value, seven per butterfly, one for 1/sqrt(d) and one per
step of the chain: at most 12 of 2^-24 relative to |y|_2 + |s a|_2, and
|y|_2 <= |x|_2 + |s a|_2 with |s a|_2 at most the norm of the loop it is
fitted to (plus quantization, well below it): 12 * 2^-24 * 3 times the norms
of the rows on the chain.  A BF16 output adds half a step, 2^-8 |x|.
"""
import numpy as np
import pytest
import torch

import decode_attention_14_b200 as rq
import synth
from oracle import oracle as orc

import rqharness as H

pytestmark = pytest.mark.gpu


def _expected(bt, layer, loop, lens):
    """[2][B][H][T + n_tail][d] fp64 and the rows' bound on rounding, [2][B][H][T + n_tail]: sequence b's tokens are
    the first lens[b] committed ones and then the tail."""
    cfg = bt.cfg
    Lg, B, Hk = cfg.loops_per_group, cfg.batch, cfg.num_kv_heads
    grp, j = loop // Lg, loop % Lg
    n_tail = bt.n_tail if j != Lg - 1 else 0
    val = np.full((2, B, Hk, bt.T + n_tail, 128), np.nan)
    tol = np.zeros((2, B, Hk, bt.T + n_tail))
    for kv in range(2):
        rec = H.reconstruct_gpu(bt, layer, grp, kv).reshape(Lg, B, Hk, -1, 128)
        X = bt.inputs[(layer, grp)][kv]
        norms = np.sqrt((rec ** 2).sum(-1)).sum(0)
        for b in range(B):
            n = lens[b]
            val[kv, b, :, :n] = rec[j, b, :, :n]
            tol[kv, b, :, :n] = 36 * 2.0 ** -24 * norms[b, :, :n]
            if n_tail:
                tail = orc.bf16_bits_to_f64(synth.bf16_to_u16(X[j][:, bt.T:]))
                val[kv, b, :, n:n + n_tail] = tail[b].transpose(1, 0, 2)
    return val, tol


def _check(k, v, val, tol, lens, n_tail, t0, fill):
    """k, v [B][n][H][d] against tokens t0 .. of val; rows past a sequence's end still hold `fill`."""
    n = k.shape[1]
    half = 2.0 ** -8 if k.dtype == torch.bfloat16 else 0.0
    for kv, x in ((0, k), (1, v)):
        got = x.double().cpu().numpy()
        for b, length in enumerate(lens):
            end = max(0, min(n, length + n_tail - t0))
            want = val[kv, b, :, t0:t0 + end].transpose(1, 0, 2)
            far = np.abs(got[b, :end] - want)
            assert (far <= half * np.abs(want) + tol[kv, b, :, t0:t0 + end].T[..., None]).all(), (kv, b, far.max())
            assert (got[b, end:] == fill).all(), (kv, b)


def _filled(shape, dtype, fill):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


@pytest.mark.parametrize("kw", [
    dict(T=1), dict(T=15, n_tail=1), dict(T=16), dict(T=17, n_tail=3), dict(T=200, B=2, n_tail=2, Hq=4),
    dict(T=70, g=32), dict(T=70, ba=2), dict(T=70, br=4, g=32), dict(T=70, ba=2, br=4), dict(T=70, rotate=False),
    dict(T=40, loops=2, Lg=1), dict(T=33, loops=6, Lg=6, sigma=(0.1, 0.2, 0.3, 0.3, 0.3), n_tail=2),
    dict(T=33, anchor_mode=rq.ANCHOR_CHAINED, n_tail=2),
    dict(T=33, loops=6, Lg=6, sigma=(0.1, 0.2, 0.3, 0.3, 0.3), anchor_mode=rq.ANCHOR_CHAINED, rotate=False),
    dict(T=300, B=3, block_tokens=128, num_blocks=12, n_tail=1, prepare=lambda c: c.shuffle_free_blocks(7)),
    dict(T=40, layers=2, rotation_per_layer=True, scale_mode=rq.SCALE_NORM_RATIO),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items() if k not in ("prepare", "sigma")))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_read_matches_the_reconstruction(kw, dtype):
    bt = H.build(**{"seed": 0x5EEDAA01, **kw})
    lens = [bt.T] * bt.cfg.batch
    for loop in range(bt.cfg.num_loops):
        layer = bt.cfg.num_layers - 1
        n_tail = bt.n_tail if (loop % bt.cfg.loops_per_group) != bt.cfg.loops_per_group - 1 else 0
        val, tol = _expected(bt, layer, loop, lens)
        k, v = bt.cache.read(layer, loop, dtype=dtype)
        assert k.shape == (bt.cfg.batch, bt.T + n_tail, bt.cfg.num_kv_heads, 128) and k.dtype == dtype
        _check(k, v, val, tol, lens, n_tail, 0, 0.0)
    bt.cache.check()
    bt.cache.close()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("t0,n", [(0, 1), (3, 2), (15, 17), (16, 16), (63, 66), (120, 40), (151, 9), (159, 1), (160, 5), (4000, 3)])
def test_read_ranges_of_ragged_sequences(paged, t0, n):
    """Any piece, also past the shorter sequences' ends (one of them empty); rows there stay as they were."""
    kw = dict(block_tokens=128, num_blocks=16, prepare=lambda c: c.shuffle_free_blocks(3)) if paged else {}
    bt = H.build(B=4, T=157, H=2, Hq=2, seed=0x5EEDAA02, **kw)
    lens = [157, 64, 0, 130]
    for b in range(4):
        bt.cache.truncate_seq(0, 0, b, lens[b])
    K, V = bt.inputs[(0, 0)]
    tail = torch.randn((2, 4, 3, 2, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    bt.cache.append(0, 1, tail[0].contiguous(), tail[1].contiguous())
    bt.inputs[(0, 0)] = tuple([torch.cat((X[j], tail[kv]), 1) for j in range(4)] for kv, X in ((0, K), (1, V)))
    bt.n_tail = 3
    for loop, n_tail in ((1, 3), (3, 0)):
        val, tol = _expected(bt, 0, loop, lens)
        k, v = _filled((4, n, 2, 128), torch.bfloat16, 7.0), _filled((4, n, 2, 128), torch.bfloat16, 7.0)
        bt.cache.read(0, loop, t0, k=k, v=v)
        _check(k, v, val, tol, lens, n_tail, t0, 7.0)
    bt.cache.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_read_into_strided_rows(dtype):
    """Rows inside wider buffers, heads before tokens, guard bands around them: nothing but the rows changes."""
    bt = H.build(B=2, T=50, H=3, Hq=3, n_tail=2, seed=0x5EEDAA03)
    val, tol = _expected(bt, 0, 0, [50, 50])
    size = 2 if dtype == torch.bfloat16 else 4
    for order, pad in (((0, 2, 1), 0), ((2, 1, 0), 8), ((1, 0, 2), 136)):
        ext = (2, 52, 3)
        shape = tuple(ext[o] for o in order) + (128 + pad,)
        bufs = []
        for _ in range(2):
            big = H.guarded_buffer(int(np.prod(shape)) * size).view(dtype).view(shape)
            big.fill_(9.0)
            bufs.append(big)
        inv = tuple(order.index(d) for d in range(3))
        k, v = (x[..., :128].permute(*inv, 3) for x in bufs)
        bt.cache.read(0, 0, k=k, v=v)
        _check(k, v, val, tol, [50, 50], 2, 0, 9.0)
        assert all((x[..., 128:] == 9.0).all() for x in bufs)
    bt.cache.close()


def test_read_of_a_bf16_cache_is_the_stored_values():
    bt = H.build(loops=2, Lg=1, B=2, T=77, H=3, Hq=3, fmt=rq.RQ_FMT_BF16, seed=0x5EEDAA04)
    bt.cache.truncate_seq(0, 1, 1, 20)
    for loop, lens in ((0, (77, 77)), (1, (77, 20))):
        K, V = bt.inputs[(0, loop)]
        for dtype in (torch.bfloat16, torch.float32):
            k, v = bt.cache.read(0, loop, 5, 70, dtype=dtype)
            for b, n in enumerate(lens):
                assert torch.equal(k[b, :n - 5], K[0][b, 5:n][:70].to(dtype)) and torch.equal(v[b, :n - 5], V[0][b, 5:n][:70].to(dtype))
                assert (k[b, max(0, n - 5):] == 0).all()
    bt.cache.close()


def test_read_appended_again_keeps_the_anchor():
    """Reading an anchor loop back and quantizing it again gives values within half a code step and the FP8 rounding of
    the group's range: |x| small against the row (a use that re-encodes a prefix)."""
    bt = H.build(loops=1, Lg=1, T=64, H=2, Hq=2, seed=0x5EEDAA05)
    k, v = bt.cache.read(0, 0)
    again = H.build_from([k], [v], Hq=2, T=64)
    k2, _ = again.cache.read(0, 0, dtype=torch.float32)
    k1, _ = bt.cache.read(0, 0, dtype=torch.float32)
    span = k1.unflatten(-1, (8, 16))
    span = (span.amax(-1) - span.amin(-1)).repeat_interleave(16, -1)
    # scale off by 2^-4 relative over 15 codes, the minimum by 2^-4 |min|, half a step of 1/15, the BF16 read
    assert ((k2 - k1).abs() <= span * (2 ** -4 + 1 / 30 * (1 + 2 ** -4)) + k1.unflatten(-1, (8, 16)).abs().amax(-1).repeat_interleave(16, -1) * (2 ** -4 + 2 ** -8)).all()
    bt.cache.close()
    again.cache.close()


def test_read_on_a_side_stream_and_in_a_graph():
    bt = H.build(B=2, T=130, n_tail=1, seed=0x5EEDAA06)
    k0, v0 = bt.cache.read(0, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k1, v1 = torch.zeros_like(k0), torch.zeros_like(v0)
    bt.cache.read(0, 2, k=k1, v=v1, stream=s)
    k2, v2 = torch.zeros_like(k0), torch.zeros_like(v0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bt.cache.read(0, 2, k=k2, v=v2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(k0, k1) and torch.equal(v0, v1) and torch.equal(k0, k2) and torch.equal(v0, v2)
    bt.cache.check()
    bt.cache.close()


def test_read_of_nothing():
    bt = H.build(T=10, seed=0x5EEDAA07)
    bt.cache.truncate(0, 0, 0)
    k, v = _filled((1, 4, 4, 128), torch.float32, 3.0), _filled((1, 4, 4, 128), torch.float32, 3.0)
    bt.cache.read(0, 0, k=k, v=v)
    assert (k == 3.0).all() and (v == 3.0).all()
    with pytest.raises(ValueError):
        bt.cache.read(0, 0)
    bt.cache.close()


def test_read_refusals():
    bt = H.build(B=2, T=20, H=2, Hq=2, seed=0x5EEDAA08)
    h = bt.cache.h
    k = torch.zeros((2, 8, 2, 136), dtype=torch.float32, device="cuda")
    v = torch.zeros_like(k)

    def call(layer=0, loop=0, t0=0, n=8, kind=rq.RQ_OUT_FP32, kk=k, vv=v, sb=8 * 2 * 136, st=2 * 136, sh=136):
        return rq.rq_cache_read(h, layer, loop, t0, n, kind, kk, vv, sb, st, sh)

    assert call() == rq.RQ_OK
    bad = [dict(layer=1), dict(layer=-1), dict(loop=4), dict(loop=-1), dict(t0=-1), dict(n=0), dict(n=-3), dict(kind=2),
           dict(kk=None), dict(vv=None), dict(vv=k), dict(kk=k[..., 1:]), dict(vv=v[..., 2:]),
           dict(sh=130), dict(sh=64), dict(sh=0), dict(st=136), dict(sb=0), dict(sb=-2176), dict(st=1 << 62),
           dict(kind=rq.RQ_OUT_BF16, sh=132)]
    for kw in bad:
        assert call(**kw) == rq.RQ_ERR_INVALID, kw
    assert call(n=1, st=0) == rq.RQ_OK            # the stride of a single token does not matter
    with pytest.raises(ValueError):
        bt.cache.read(0, 0, k=k[..., :128], v=None)
    with pytest.raises(ValueError):
        bt.cache.read(0, 0, k=k[..., :128].half(), v=v[..., :128].half())
    with pytest.raises(ValueError):
        bt.cache.read(0, 0, k=k[..., :128], v=v[..., :128].bfloat16())
    with pytest.raises(ValueError):
        bt.cache.read(0, 0, k=k[..., :128], v=v[..., :128].contiguous())
    with pytest.raises(ValueError):
        bt.cache.read(0, 0, k=k[:, :, :1, :128], v=v[:, :, :1, :128])
    bt.cache.close()
