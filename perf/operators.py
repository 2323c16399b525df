"""Cases of the operators that read a looped Transformer's KV cache through a window, or hand it back:

* ``read``: the tokens [t0, t0 + n) of one (layer, loop), rebuilt from their records as K and V rows;
* ``decode``: single-token attention that sees the last `window` tokens and the first `sinks` tokens;
* ``prefill``: the same for a chunk of new tokens, each of which sees its own window.

They run over both cache formats: ``rq`` (INT anchor + INT residuals, contiguous or in pages) and ``bf16``.
A cache here is what a serving loop holds after its appends: per sequence `len` committed tokens, then (at a
loop that is not its group's anchor) the BF16 tail of tokens in flight.

The plain forms work on the records as they lie in memory: arrays [2 (K, V)][blocks][H][tokens per block][bytes]
behind a block table (one block per sequence where a cache is contiguous).
"""
import math

import numpy as np
import torch

own = False

D = 128
SEED = 0xA11CE                 # rotation seed
LOOPS = 4                      # loops of a group; the last is the anchor


# ------------------------------------------------------------------ cases
def _case(name, op, fmt="rq", **kw):
    c = dict(name=name, op=op, fmt=fmt, B=1, H=16, G=1, T=1024, tail=0, loop=0, abits=4, rbits=2, group=16, rotate=True,
             paged=0, ragged=False, n=1, t0=0, window=0, sinks=0, dtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # a few tokens handed to another kernel: latency
        _case("read_few_tokens", "read", T=200, tail=1, loop=1, t0=170, n=31),
        # a whole residual loop of the 24-layer, 4-loop benchmark shape (8k, 4 sequences) rebuilt as BF16
        _case("read_8k_b4_residual", "read", B=4, T=8192, loop=0, n=8192),
        # an anchor loop of a paged, ragged cache in fp32, an odd piece from inside it
        _case("read_paged_anchor_fp32", "read", B=3, H=8, T=5000, loop=3, paged=128, ragged=True, t0=77, n=4801, dtype="fp32"),
        # one sequence, a short window: the smallest serving call
        _case("decode_short_window", "decode", T=1000, tail=1, loop=1, window=256, sinks=4, dtype="fp32"),
        # the benchmark shape with a window of half its context
        _case("decode_8k_b4_window4k", "decode", B=4, T=8191, tail=1, loop=0, window=4096, sinks=4, dtype="fp32"),
        # long context, paged, grouped heads, ragged sequences, the anchor loop
        _case("decode_64k_paged_gqa", "decode", B=2, H=8, G=4, T=65536, loop=3, paged=256, ragged=True, window=32768, sinks=64),
        # the uncompressed cache of the same benchmark shape
        _case("decode_bf16_8k_b4", "decode", "bf16", B=4, T=8192, window=4096, sinks=4, dtype="fp32"),
        # sixteen drafted tokens on the benchmark shape
        _case("prefill_16_tokens_8k_b4", "prefill", B=4, T=8192, tail=16, loop=0, n=16, window=1024, sinks=4),
        # a committed chunk on a paged, ragged cache with grouped heads
        _case("prefill_500_paged_gqa", "prefill", B=2, H=4, G=4, T=5001, loop=3, paged=128, ragged=True, n=500, window=2000, sinks=16),
        # a long chunk in flight at a residual loop of one sequence
        _case("prefill_2048_residual", "prefill", T=4096, tail=2048, loop=0, n=2048, window=1024, sinks=64),
        # an odd chunk over the uncompressed cache, grouped heads
        _case("prefill_bf16_511_gqa", "prefill", "bf16", B=2, H=4, G=4, T=4133, n=511, window=1024, sinks=4, dtype="fp32"),
        # a whole prompt over the uncompressed cache: every token sees all before it
        _case("prefill_bf16_8k_prompt", "prefill", "bf16", T=8192, n=8192, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["read", "decode", "prefill"])
    fmt = "rq" if op == "read" else rng.choice(["rq", "rq", "bf16"])
    c = _case("", op, fmt)
    del c["name"]
    c["H"] = rng.choice([2, 4, 8, 16])
    c["B"] = rng.randint(1, 4)
    c["G"] = 1 if op == "read" else rng.choice([1, 2, 4, 8])
    c["window"], c["sinks"] = _log(rng, 1, 16384), rng.choice([0, 1, 4, 17, 64, 300])
    if fmt == "rq":
        c["loop"] = rng.randrange(LOOPS)
        c["abits"], c["rbits"] = rng.choice([(4, 2), (4, 2), (4, 4), (2, 2)])
        c["group"], c["rotate"] = rng.choice([16, 16, 32]), rng.random() < 0.8
        c["paged"], c["ragged"] = rng.choice([0, 0, 128, 256]), rng.random() < 0.4
        c["tail"] = 0 if c["loop"] == LOOPS - 1 else rng.randint(0, 8)
    most = (1 << 19) // (c["B"] * c["H"])        # tokens of a sequence, so that no drawn cache is larger than the listed ones
    # the type of the rows that come back; a chunk over the compressed cache goes on into a BF16 model
    c["dtype"] = "bf16" if op == "prefill" and fmt == "rq" else rng.choice(["bf16", "fp32"])
    if op == "read":
        c["T"] = _log(rng, 1, most)
        c["t0"] = rng.randrange(c["T"])
        c["n"] = rng.randint(1, c["T"] + c["tail"] - c["t0"])
    elif op == "decode":
        c["T"] = _log(rng, 1, min(most, 65536))
    else:
        c["T"] = _log(rng, 2, min(most, 8192))
        pairs = c["B"] * c["H"] * c["G"] * 2 * c["T"]              # no more than the whole prompt's
        c["n"] = _log(rng, 1, min(2048, c["T"], (1 << 29) // pairs))
        if fmt == "rq":
            c["ragged"] = False if c["n"] > c["T"] // 2 else c["ragged"]
            if c["loop"] != LOOPS - 1:
                c["tail"] = c["n"]
        if fmt == "bf16" and rng.random() < 0.3:
            c["window"] = 0
    return c


# ------------------------------------------------------------------ inputs
def _lens(c):
    """Committed tokens of each sequence: where ragged, the first has all T and the others fewer."""
    if not c["ragged"]:
        return [c["T"]] * c["B"]
    return [c["T"] - (b * c["T"]) // (3 * c["B"]) for b in range(c["B"])]


def _inputs(c, seed):
    """What the model produced: K and V of the loop and of its group's anchor (committed tokens), the loop's tail, q.
    Values as K/V states have them: N(0, 1) with a few channels ten times larger per head; a loop is near its anchor."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62))
    B, T, H, dev = c["B"], c["T"], c["H"], "cuda"

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    hot = torch.rand((2, 1, 1, H, D), generator=g, device=dev).argsort(-1) < 4
    scale = torch.where(hot, 10.0, 1.0)
    anchor = normal(2, B, T, H, D) * scale
    x = {"anchor": anchor.bfloat16(), "loop": None, "tail": None, "q": None}
    if c["fmt"] == "rq" and c["loop"] != LOOPS - 1:
        near = 0.8 + 0.4 * torch.rand((2, B, T, H, 1), generator=g, device=dev)
        x["loop"] = (near * anchor + 0.1 * (LOOPS - 1 - c["loop"]) * normal(2, B, T, H, D)).bfloat16()
        if c["tail"]:
            x["tail"] = (normal(2, B, c["tail"], H, D) * scale).bfloat16()
    rows = (c["n"],) if c["op"] == "prefill" else ()
    if c["op"] != "read":
        x["q"] = normal(B, *rows, H * c["G"], D).bfloat16()
    return x


def _sigma():
    """The rotation's signs: -1 where the top bit of splitmix64(seed + j) is set."""
    m = (1 << 64) - 1

    def mix(v):
        z = (v + 0x9E3779B97F4A7C15) & m
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        return z ^ (z >> 31)

    return [-1.0 if mix(SEED + j) >> 63 else 1.0 for j in range(D)]


def _hadamard(dtype):
    """H / sqrt(d) with the signs: row i, column j of R; the parity of the bits that i and j share gives H's sign."""
    i = np.arange(D)
    odd = np.array([[bin(a & b).count("1") & 1 for b in i] for a in i])
    r = (1.0 - 2.0 * odd) * np.array(_sigma())[None, :] / math.sqrt(D)
    return torch.from_numpy(r).to("cuda", dtype)


def _round_to(v, bits, low):
    """v (64 bits) to `bits` significant bits, nearest with ties to even; `low`: the exponent of the smallest normal number."""
    _, e = torch.frexp(v)
    step = (torch.clamp(e.long() - 1, min=low) - (bits - 1) + 1023 << 52).view(torch.float64)   # 2^(exponent - bits + 1)
    return torch.round(v / step) * step


def _e4m3(v):
    return torch.clamp(_round_to(v, 4, -6), -448.0, 448.0)


def _quantize(v, bits, group):
    """Codes, scale and minimum of each group of v (64 bits), and the values that they stand for."""
    w = v.unflatten(-1, (D // group, group))
    lo, hi = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
    top = (1 << bits) - 1
    sc, mn = _e4m3((hi - lo) / top), _e4m3(lo) + 0.0
    code = torch.where(sc > 0, torch.clamp(torch.round((w - mn) / torch.where(sc > 0, sc, 1.0)), 0, top), 0.0)
    meta = torch.cat((sc, mn), -1).flatten(-2).float().to(torch.float8_e4m3fn).view(torch.uint8)
    code, back = code.flatten(-2).to(torch.uint8), (mn + code * sc).flatten(-2)
    per = 8 // bits
    shift = torch.arange(per, device=v.device, dtype=torch.int32) * bits
    packed = (code.unflatten(-1, (D // per, per)).int() << shift).sum(-1).to(torch.uint8)
    return packed, meta, back


def _encode(c, x):
    """The records of the committed tokens, [2][B][H][T][bytes], as the cache format defines them, worked out in 64 bits."""
    a = x["anchor"].double().transpose(2, 3)
    out = dict(zip(("ac", "am"), (p := _quantize(a, c["abits"], c["group"]))[:2]))
    if x["loop"] is not None:
        v, ref = x["loop"].double().transpose(2, 3), p[2]
        den = (ref * ref).sum(-1, keepdim=True)
        s = torch.where(den > 0, (v * ref).sum(-1, keepdim=True) / torch.where(den > 0, den, 1.0), 0.0)
        s = _round_to(s, 8, -126)
        r = v - s * ref
        if c["rotate"]:
            r = (r @ (_hadamard(torch.float64) * math.sqrt(D)).round().T) * (1 / math.sqrt(D))
        out["rc"], out["rm"], _ = _quantize(r, c["rbits"], c["group"])
        out["rf"] = s.squeeze(-1).to(torch.bfloat16)
    return out


def _paged(c, lens, seed):
    """A block table (a shuffled pool; one block per sequence where the cache is contiguous) and the pool's size."""
    bt = c["paged"] or c["T"]
    mb = -(-c["T"] // bt)
    order = np.random.RandomState(int(seed) % (1 << 31)).permutation(c["B"] * mb)
    return bt, torch.from_numpy(order.reshape(c["B"], mb)).to("cuda")


def _pool(records, bt, table):
    """Records [2][B][H][T][...] laid out as the pool [2][blocks][H][bt][...]."""
    two, B, H, T = records.shape[:4]
    mb = table.shape[1]
    pad = torch.zeros((two, B, H, mb * bt) + records.shape[4:], dtype=records.dtype, device=records.device)
    pad[:, :, :, :T] = records
    blocks = pad.unflatten(3, (mb, bt)).movedim(3, 2)
    pool = torch.empty_like(blocks.flatten(1, 2))
    pool[:, table.flatten()] = blocks.flatten(1, 2)
    return pool


def prepare(case, seed):
    c = dict(case)
    x, lens = _inputs(c, seed), _lens(c)
    s = {"c": c, "q": x["q"]}
    s["kind"] = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    if c["op"] == "read":
        s["k"], s["v"] = (torch.zeros((c["B"], c["n"], c["H"], D), dtype=s["kind"], device="cuda") for _ in range(2))
    if own:
        import decode_attention_14_b200 as rq

        chunk = min(c["T"], 4096)
        blocks = c["B"] * -(-c["T"] // c["paged"]) if c["paged"] else 0
        cfg = rq.make_config(
            num_layers=1, num_loops=LOOPS if c["fmt"] == "rq" else 1, loops_per_group=LOOPS if c["fmt"] == "rq" else 1,
            batch=c["B"], max_tokens=c["T"], max_tail_tokens=max(chunk, c["tail"]) if c["fmt"] == "rq" else 0,
            num_kv_heads=c["H"], num_q_heads=c["H"] * c["G"], group_size=c["group"], anchor_bits=c["abits"],
            resid_bits=c["rbits"], rotate=c["rotate"], seed=SEED, block_tokens=c["paged"], num_blocks=blocks,
            format=rq.RQ_FMT_RESIDUAL if c["fmt"] == "rq" else rq.RQ_FMT_BF16)
        cache = s["cache"] = rq.Cache(cfg)
        if c["paged"]:
            cache.shuffle_free_blocks(int(seed) & 0xFFFFFFFF)
        for t in range(0, c["T"], chunk):
            kv = {k: [y.contiguous() for y in x[k][:, :, t:t + chunk]] for k in ("anchor", "loop") if x[k] is not None}
            for loop in range(cfg.num_loops):
                cache.append(0, loop, *kv["loop" if "loop" in kv and loop == c["loop"] else "anchor"])
        for b, n in enumerate(lens):
            if n < c["T"]:
                cache.truncate_seq(0, 0, b, n)
        if x["tail"] is not None:
            cache.append(0, c["loop"], x["tail"][0].contiguous(), x["tail"][1].contiguous())
        torch.cuda.synchronize()
        return s
    bt, table = _paged(c, lens, seed)
    s["table"], s["bt"], s["lens"] = table, bt, torch.tensor(lens, device="cuda")
    records = _encode(c, x) if c["fmt"] == "rq" else {"kv": x["anchor"].transpose(2, 3)}
    s["records"] = {k: _pool(v, bt, table) for k, v in records.items()}
    s["tail"] = None if x["tail"] is None else x["tail"].transpose(2, 3).contiguous()
    s["R"] = _hadamard(torch.float32) if c["rotate"] else None
    return s


# ------------------------------------------------------------------ the plain forms
def _unpack(codes, meta, bits, group):
    shift = torch.arange(8 // bits, device=codes.device, dtype=torch.int32) * bits
    code = (codes.unsqueeze(-1).int() >> shift) & ((1 << bits) - 1)
    sm = meta.view(torch.float8_e4m3fn).float().unflatten(-1, (D // group, 2))
    code = code.flatten(-2).unflatten(-1, (D // group, group)).float()
    return (code * sm[..., :1] + sm[..., 1:]).flatten(-2)


def _rows(s, at):
    """K and V, [2][B][H][N][d] in 32 bits, of the committed tokens at positions `at` [B][N]."""
    c, bt = s["c"], s["bt"]
    block, off = s["table"].gather(1, at // bt), at % bt
    take = {k: v[:, block, :, off].movedim(2, 0).transpose(2, 3) for k, v in s["records"].items()}
    if c["fmt"] == "bf16":
        return take["kv"].float()
    x = _unpack(take["ac"], take["am"], c["abits"], c["group"])
    if "rc" in take:
        y = _unpack(take["rc"], take["rm"], c["rbits"], c["group"])
        x = take["rf"].float().unsqueeze(-1) * x + (y @ s["R"] if c["rotate"] else y)
    return x


def _read(s):
    c, lens = s["c"], s["lens"]
    at = c["t0"] + torch.arange(c["n"], device="cuda").expand(c["B"], -1)
    x = _rows(s, at.clamp(max=c["T"] - 1))
    there = at < lens[:, None]
    if s["tail"] is not None:
        j = (at - lens[:, None]).clamp(0, c["tail"] - 1)[None, :, None, :, None].expand(2, -1, c["H"], -1, D)
        x = torch.where(there[None, :, None, :, None], x, s["tail"].gather(3, j).float())
        there = at < lens[:, None] + c["tail"]
    x = x.transpose(2, 3)
    m = there[:, :, None, None]
    s["k"].copy_(torch.where(m, x[0], s["k"].float()))
    s["v"].copy_(torch.where(m, x[1], s["v"].float()))
    return s["k"], s["v"]


def _attend(s):
    """Attention of the n last tokens of each sequence: token at position p sees p' <= p with p' > p - window or p' < sinks."""
    c, lens = s["c"], s["lens"]
    B, H, G, n, dev = c["B"], c["H"], c["G"], c["n"], "cuda"
    window, sinks = (c["window"], c["sinks"]) if c["window"] else (1 << 40, 0)
    end = lens[:, None] + c["tail"]                                      # tokens of each sequence
    mine = end - n + torch.arange(n, device=dev)                         # [B][n] positions of the queries
    # the committed positions that any query sees: the sinks, then from the first query's window on
    first = (end - n - window + 1).clamp(min=0)
    span = min(c["T"], window + n)
    head = torch.arange(min(sinks, c["T"]), device=dev).expand(B, -1)
    run = first + torch.arange(span, device=dev)
    at = torch.cat((head, run), 1)
    there = torch.cat((head < lens[:, None], (run < lens[:, None]) & (run >= sinks)), 1)
    kv = _rows(s, at.clamp(max=c["T"] - 1))
    if s["tail"] is not None:
        kv = torch.cat((kv, s["tail"].float()), 3)
        at = torch.cat((at, lens[:, None] + torch.arange(c["tail"], device=dev)), 1)
        there = torch.cat((there, there.new_ones(B, c["tail"])), 1)
    a, p = at[:, None, :], mine[:, :, None]
    seen = there[:, None, :] & (a <= p) & ((a > p - window) | (a < sinks))          # [B][n][keys]
    q = s["q"].float().view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    z = (q @ kv[0].transpose(-1, -2)).mul_(1 / math.sqrt(D)).view(B, H, n, G, -1)
    z.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    w = z.sub_(z.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.flatten(2, 3) @ kv[1]).view(B, H, n, G, D)
    o = torch.where(total > 0, o / total.clamp(min=1e-38), 0.0).permute(0, 2, 1, 3, 4).reshape(B, n, H * G, D).to(s["kind"])
    return o if c["op"] == "prefill" else o[:, 0]


def run(state):
    c = state["c"]
    if own:
        cache = state["cache"]
        if c["op"] == "read":
            return cache.read(0, c["loop"], c["t0"], k=state["k"], v=state["v"])
        call = cache.decode_window if c["op"] == "decode" else cache.prefill_window
        return call(0, c["loop"], state["q"], c["window"], c["sinks"], dtype=state["kind"])
    return _read(state) if c["op"] == "read" else _attend(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _token_bytes(c):
    """Bytes of one token of one kv head, K and V."""
    if c["fmt"] == "bf16":
        return 2 * 2 * D
    meta = 2 * D // c["group"]
    b = D * c["abits"] // 8 + meta
    if c["loop"] != LOOPS - 1:
        b += D * c["rbits"] // 8 + meta + 2
    return 2 * b


def work(case):
    c = dict(case)
    H, G, n, tail = c["H"], c["G"], c["n"], c["tail"]
    size = flops = 0
    for length in _lens(c):
        end = length + tail
        if c["op"] == "read":
            lo, hi = c["t0"], min(c["t0"] + n, end)
            got = max(0, min(hi, length) - lo)
            late = max(0, hi - max(lo, length))
            size += H * (got * _token_bytes(c) + late * 4 * D + (got + late) * 2 * D * (2 if c["dtype"] == "bf16" else 4))
            flops += H * got * 2 * D * (4 if c["loop"] == LOOPS - 1 else 4 + 2 * 7 + 2)
            continue
        window, sinks = (c["window"], c["sinks"]) if c["window"] else (end, 0)
        # pairs: what each query sees of its window, and of the sinks before it
        p = np.arange(end - n, end, dtype=np.int64)
        low = np.maximum(0, p + 1 - window)
        pairs = int((p + 1 - low).sum() + np.minimum(sinks, low).sum())
        first = max(0, end - n + 1 - window)
        seen = min(sinks, first) + max(0, length - first)
        size += H * (seen * _token_bytes(c) + min(tail, end - first) * 4 * D + n * G * D * (2 + (2 if c["dtype"] == "bf16" else 4)))
        flops += H * G * pairs * 4 * D
    return {"bytes": size, "flops": max(flops, 1)}


# ------------------------------------------------------------------ from the definition, in 64 bits
def exact(case, seed):
    c = dict(case)
    x, lens = _inputs(c, seed), _lens(c)
    n, H, G = c["n"], c["H"], c["G"]

    def values(codes, meta, bits):
        i = torch.arange(D, device="cuda")
        byte = codes.index_select(-1, i * bits // 8).int()
        code = torch.bitwise_and(torch.bitwise_right_shift(byte, (i * bits % 8).int()), 2 ** bits - 1).double()
        m = meta.view(torch.float8_e4m3fn).double()
        return code * m.index_select(-1, 2 * (i // c["group"])) + m.index_select(-1, 2 * (i // c["group"]) + 1)

    def unrotated(y):
        """R^T y by the recursion H_2m = [[H_m, H_m], [H_m, -H_m]]."""
        for m in (1, 2, 4, 8, 16, 32, 64):
            u = y.unflatten(-1, (-1, 2, m))
            y = torch.stack((u[..., 0, :] + u[..., 1, :], u[..., 0, :] - u[..., 1, :]), -2).flatten(-3)
        return y * torch.tensor(_sigma(), device="cuda", dtype=torch.float64) / math.sqrt(D)

    if c["fmt"] == "bf16":
        kv = x["anchor"].double().transpose(2, 3)
    else:
        rec = _encode(c, x)
        kv = values(rec["ac"], rec["am"], c["abits"])
        if "rc" in rec:
            y = values(rec["rc"], rec["rm"], c["rbits"])
            kv = rec["rf"].double()[..., None] * kv + (unrotated(y) if c["rotate"] else y)
    out = []
    for b, length in enumerate(lens):
        keys = kv[:, b, :, :length]
        if x["tail"] is not None:
            keys = torch.cat((keys, x["tail"][:, b].double().transpose(1, 2)), 2)          # [2][H][tokens][d]
        end = keys.shape[2]
        if c["op"] == "read":
            piece = keys[:, :, c["t0"]:c["t0"] + n].transpose(1, 2)
            out.append(torch.nn.functional.pad(piece, (0, 0, 0, 0, 0, n - piece.shape[1])))
            continue
        p = torch.arange(end - n, end, device="cuda")[:, None]
        t = torch.arange(end, device="cuda")[None, :]
        blind = t > p
        if c["window"]:
            blind = blind | ((p - t >= c["window"]) & (t >= c["sinks"]))
        q = x["q"].double().view(c["B"], n, H * G, D)[b]
        o = torch.empty((n, H * G, D), dtype=torch.float64, device="cuda")
        for h in range(H * G):
            z = q[:, h] @ keys[0, h // G].T / math.sqrt(D)
            o[:, h] = torch.softmax(z.masked_fill_(blind, -math.inf), -1) @ keys[1, h // G]
        out.append(o)
    out = torch.stack(out)
    return (out[:, 0], out[:, 1]) if c["op"] == "read" else out if c["op"] == "prefill" else out[:, 0]
