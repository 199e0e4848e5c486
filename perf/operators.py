"""The decode-serving operators around the packed cache, as cases that can be measured.

A decode step of a model that serves from a packed cache prepares the new token (norm of
the query and key heads, position rotation, append), attends over a sliding window of the
cache with a few first tokens that stay visible, and keeps the cache's blocks in order
(forking a sequence, freeing the blocks a window has left behind, compacting the arenas).
Each case is one such call at one size:

  window   attention over the packed cache, sliding window and first tokens (sinks)
  rope     norm and rotation of a prompt's queries and keys, values laid out beside them
  append   norm, rotation and append of one new token per sequence
  fork     sequences that continue as copies of others
  free     blocks of every sequence given up
  compact  the live records of a cache moved to the front of another one

`own` false: the operators in elementary torch operations, 32-bit arithmetic, one rounding.
`own` true: this repository's calls.  `exact`: the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128      # head_dim
BT = 128     # tokens of a block
DEV = "cuda"
FREED = -1   # offset of a freed index entry (0xFFFFFFFF as a signed integer)
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one request of a grouped-query layer at its smallest: latency is what counts
        dict(name="window one sequence", op="window", batch=1, kv_heads=8, group=4, queries=1, bits=4, tokens=2000,
             spread=0, window=512, sinks=4, structured=False, shape=1),
        # a full batch of multi-head attention, the largest window call
        dict(name="window batch of heads", op="window", batch=16, kv_heads=32, group=1, queries=1, bits=3,
             tokens=8192, spread=0, window=4096, sinks=4, structured=False, shape=2),
        # speculative positions: four queries a step, each with its own mask, ragged lengths
        dict(name="window four positions", op="window", batch=4, kv_heads=8, group=4, queries=4, bits=4,
             tokens=9000, spread=4000, window=2048, sinks=64, structured=False, shape=3),
        # compressible inputs (packed records) and sequences shorter than the window
        dict(name="window packed ragged", op="window", batch=8, kv_heads=8, group=2, queries=1, bits=2, tokens=2600,
             spread=2599, window=1000, sinks=0, structured=True, shape=4),
        # a prompt's chunk, from the token-major projections to the encoder's layout
        dict(name="rope prompt", op="rope", batch=4, tokens=4096, q_heads=32, kv_heads=8, dtype="bfloat16",
             norm=True, layout="half", rot_dim=128, scaling="parts", far=False, first=0),
        # odd sizes, part of the head, explicit far positions
        dict(name="rope odd far", op="rope", batch=3, tokens=257, q_heads=14, kv_heads=2, dtype="float32",
             norm=False, layout="interleaved", rot_dim=64, scaling="linear", far=True, first=0),
        # one decode step of a batch
        dict(name="append batch", op="append", batch=64, q_heads=32, kv_heads=8, dtype="bfloat16", norm=True,
             layout="half", rot_dim=128, scaling="none", ragged=False, tail=50),
        # a ragged batch in which some sequences pause
        dict(name="append ragged", op="append", batch=7, q_heads=6, kv_heads=6, dtype="float16", norm=True,
             layout="interleaved", rot_dim=96, scaling="base", ragged=True, tail=90),
        # half of a batch continues as copies of the other half (parallel samples of one prompt)
        dict(name="fork half the batch", op="fork", batch=64, kv_heads=8, blocks=64, bits=4, pairs=32, shape=9),
        # the blocks a window has left, in every sequence
        dict(name="free behind a window", op="free", batch=64, kv_heads=8, blocks=256, bits=4, shape=10),
        # a small cache, a few hundred records
        dict(name="compact small", op="compact", batch=4, kv_heads=4, blocks=24, bits=2, dead=0.4, forks=1,
             packed=True, shape=11),
        # a whole layer's cache of a batch
        dict(name="compact layer", op="compact", batch=16, kv_heads=32, blocks=64, bits=4, dead=0.4, forks=2,
             packed=False, shape=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "rope", "append", "fork", "free", "compact"])
    shape = rng.randrange(1 << 30)
    if op == "window":
        group, queries = rng.choice([(1, 1), (1, 2), (2, 1), (4, 1), (2, 2), (4, 2), (8, 1), (4, 4), (1, 8), (8, 4)])
        heads = rng.choice([1, 2, 3, 5, 8, 12, 16, 32])
        tokens = _log(rng, 1, 16000)
        window = _log(rng, 1, 8192)
        batch = _log(rng, 1, 16)
        while batch > 1 and batch * heads * min(tokens, window + 256) > 1_600_000:
            batch -= 1
        while batch > 1 and batch * heads * tokens > 4_000_000:
            batch -= 1
        return dict(op=op, batch=batch, kv_heads=heads, group=group, queries=queries, bits=rng.choice([2, 3, 4]),
                    tokens=tokens, spread=rng.choice([0, tokens // 2, max(tokens - 1, 0)]), window=window,
                    sinks=rng.choice([0, 1, 4, 128, 300]), structured=rng.random() < 0.4, shape=shape)
    if op == "rope":
        batch = _log(rng, 1, 8)
        return dict(op=op, batch=batch, tokens=_log(rng, 1, 16384 // batch), q_heads=rng.choice([1, 4, 7, 16, 32]),
                    kv_heads=rng.choice([1, 2, 4, 8]), dtype=rng.choice(["float16", "bfloat16", "float32"]),
                    norm=rng.random() < 0.5, layout=rng.choice(["half", "interleaved"]),
                    rot_dim=2 * rng.randrange(1, 65), scaling=rng.choice(["none", "linear", "base", "parts"]),
                    far=rng.random() < 0.4, first=rng.choice([0, 1, rng.randrange(1 << 20)]))
    if op == "append":
        kv = rng.choice([1, 2, 5, 8, 16])
        return dict(op=op, batch=_log(rng, 1, 256), q_heads=kv * rng.choice([1, 2, 4, 7]), kv_heads=kv,
                    dtype=rng.choice(["float16", "bfloat16", "float32"]), norm=rng.random() < 0.5,
                    layout=rng.choice(["half", "interleaved"]), rot_dim=2 * rng.randrange(1, 65),
                    scaling=rng.choice(["none", "linear", "base", "parts"]), ragged=rng.random() < 0.5,
                    tail=rng.randrange(1, 127))
    batch, heads, blocks = _log(rng, 2, 64), rng.choice([1, 2, 3, 8, 16]), _log(rng, 1, 200)
    while batch > 2 and batch * heads * blocks > 20000:
        batch -= 1
    if op == "fork":
        return dict(op=op, batch=batch, kv_heads=heads, blocks=blocks, bits=rng.choice([2, 3, 4]),
                    pairs=rng.randrange(1, batch // 2 + 1), shape=shape)
    if op == "free":
        return dict(op=op, batch=batch, kv_heads=heads, blocks=blocks, bits=rng.choice([2, 3, 4]), shape=shape)
    return dict(op=op, batch=batch, kv_heads=heads, blocks=blocks, bits=rng.choice([2, 3, 4]),
                dead=rng.uniform(0.05, 0.8), forks=rng.randrange(0, batch // 2 + 1), packed=rng.random() < 0.5,
                shape=shape)


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lengths(case):
    """Tokens of every sequence: `tokens`, less a random part of `spread` behind the first."""
    r = random.Random(case["shape"])
    return [case["tokens"]] + [case["tokens"] - (r.randrange(case["spread"] + 1) if case["spread"] else 0)
                               for _ in range(case["batch"] - 1)]


def _hold(z, gen):
    """Every channel takes a few levels, each held for a while (compressible codes)."""
    tokens = z.shape[-2]
    levels = torch.randint(1, 17, z.shape[:-2] + (1, D), generator=gen, device=DEV)
    every = torch.randint(1, 48, z.shape[:-2] + (1, D), generator=gen, device=DEV)
    at = torch.arange(tokens, device=DEV)[:, None].expand(z.shape)
    pick = torch.randint(0, 1 << 30, z.shape, generator=gen, device=DEV) % levels
    return (torch.gather(pick, -2, at - at % every).float() - levels / 2.0) / 4.0


def _window_inputs(case, seed):
    """k, v fp16 [B, H, T, 128] (T: the longest sequence), q fp16 [B, H*S*G, 128]."""
    gen = _gen(seed)
    B, H, T = case["batch"], case["kv_heads"], case["tokens"]
    mu = torch.randn(B, H, 1, D, generator=gen, device=DEV)
    sigma = torch.rand(B, H, 1, D, generator=gen, device=DEV) * 1.5 + 0.5
    wide = torch.rand(B, H, 1, D, generator=gen, device=DEV).argsort(-1) < 4  # four outlier channels
    sigma = torch.where(wide, 10 * sigma, sigma)
    k = torch.empty(B, H, T, D, dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    for b in range(B):  # a sequence at a time: the fp32 draws are the largest tensors here
        zk = torch.randn(H, T, D, generator=gen, device=DEV)
        zv = torch.randn(H, T, D, generator=gen, device=DEV)
        if case["structured"]:
            zk, zv = _hold(zk, gen), _hold(zv, gen)
        k[b] = (mu[b] + sigma[b] * zk).half()
        v[b] = zv.half()
    rows = H * case["queries"] * case["group"]
    q = torch.randn(B, rows, D, generator=gen, device=DEV).half()
    return k, v, q


def _head_inputs(case, seed, tokens):
    """Projections of one layer, token-major: q, k, v are slices of one [B, T, (Hq + 2 Hkv) * 128] tensor."""
    gen = _gen(seed)
    B, hq, hkv = case["batch"], case["q_heads"], case["kv_heads"]
    x = (1.5 * torch.randn(B, tokens, hq + 2 * hkv, D, generator=gen, device=DEV)).to(getattr(torch, case["dtype"]))
    wq = wk = None
    if case["norm"]:
        wq = 1 + 0.2 * torch.randn(D, generator=gen, device=DEV)
        wk = 1 + 0.2 * torch.randn(D, generator=gen, device=DEV)
    return x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], wq, wk


def _far_positions(case, seed):
    """Positions up to a million, in no order, as int32 [B, T]."""
    return torch.randint(0, 1 << 20, (case["batch"], case["tokens"]), generator=_gen(seed + 7), device=DEV).int()


def _rope_parameters(case):
    """theta, scaling factor, trained length, band borders, factor on cos and sin."""
    kind = case["scaling"]
    return dict(theta=500000.0 if kind == "parts" else 10000.0, factor=1.0 if kind == "none" else 8.0,
                original=8192, low=1.0, high=32.0,
                amplitude=0.1 * math.log(8.0) + 1.0 if kind == "parts" else 1.0)


EPS = 1e-6


def _index_inputs(case, seed):
    """Index entries and arenas of a cache whose records lie in order with dead ones between:
    int32 [B, H, blocks, 2] for K and V, uint8 arenas, the permutations, tails and lengths."""
    gen = _gen(seed)
    B, H, nb = case["batch"], case["kv_heads"], case["blocks"]
    raw = (528 + 2048 * case["bits"]) // 16
    r = random.Random(case["shape"])
    blocks = [nb] + [r.randrange(1, nb + 1) for _ in range(B - 1)]
    tails = [r.randrange(0, BT) for _ in range(B)]
    count = torch.tensor(blocks, device=DEV)
    live = torch.arange(nb, device=DEV)[None, None, :] < count[:, None, None]
    index, arenas = [], []
    for _ in range(2):
        length = torch.full((B, H, nb), raw, device=DEV)
        if case.get("packed", True):
            length = torch.randint(65 + raw // 4, raw + 1, (B, H, nb), generator=gen, device=DEV)
        offset = (length.flatten().cumsum(0) - length.flatten()).reshape(B, H, nb)
        index.append(torch.where(live[..., None], torch.stack([offset, length], -1), 0).int())
        units = B * H * nb * raw
        if case["op"] == "compact":
            arenas.append(torch.randint(-1 << 62, 1 << 62, (units, 2), generator=gen, device=DEV))
    dead = None
    if case["op"] == "compact":
        dead = (torch.rand(B, 1, nb, generator=gen, device=DEV) < case["dead"]) & live
        for i in index:
            for f in range(case["forks"]):  # sequence 2f + 1 holds what 2f holds, as far as both go
                n = min(blocks[2 * f], blocks[2 * f + 1])
                i[2 * f + 1, :, :n] = i[2 * f, :, :n]
            gone = dead[..., None].expand(i.shape)
            i[..., 0] = torch.where(gone[..., 0], FREED, i[..., 0])
            i[..., 1] = torch.where(gone[..., 1], 0, i[..., 1])
    perm = torch.rand(B, H, nb, BT, generator=gen, device=DEV).argsort(-1).to(torch.uint8)
    kt = torch.randn(B, H, BT, D, generator=gen, device=DEV).half()
    vt = torch.randn(B, H, BT, D, generator=gen, device=DEV).half()
    return index, arenas, perm, kt, vt, blocks, tails


def _restored(pk, case, index, arenas, perm, kt, vt, blocks, tails):
    """A cache of this repository with the given contents."""
    units = arenas[0].shape[0] if arenas else 1 << 10
    cache = pk.PackKVCache(case["batch"], case["kv_heads"], case["blocks"], case["bits"], arena_bytes=units * 16,
                           keep_perm=True, ragged=True)
    cache.k_index.copy_(index[0])
    cache.v_index.copy_(index[1])
    if arenas:
        cache.k_arena.copy_(arenas[0].view(torch.uint8).flatten())
        cache.v_arena.copy_(arenas[1].view(torch.uint8).flatten())
        cache.ctrl[:2] = units
    cache.perm.copy_(perm)
    cache.k_tail.copy_(kt)
    cache.v_tail.copy_(vt)
    cache.set_lengths(blocks, tails)
    return cache


# ------------------------------------------------------------------------------- prepare
def prepare(case, seed):
    return {"window": _prepare_window, "rope": _prepare_rope, "append": _prepare_append, "fork": _prepare_blocks,
            "free": _prepare_blocks, "compact": _prepare_blocks}[case["op"]](case, seed)


def _quantize(x, bits, dim):
    """Codes (uint8), minimum and scale (fp16 values, as fp32) of rows of 128 along `dim`:
    scale = range / (2^b - 1) rounded up to fp16, code = rint((x - min) / scale)."""
    x = x.float()
    mn = x.amin(dim, keepdim=True)
    most = torch.full((1,), 2.0 ** bits - 1, device=x.device)  # a tensor: division by a number multiplies by 1/number
    step = (x.amax(dim, keepdim=True) - mn) / most
    scale = step.half()
    scale = torch.where(scale.float() < step, (scale.view(torch.int16) + 1).view(torch.float16), scale).float()
    code = torch.where(scale > 0, (x - mn) / torch.where(scale > 0, scale, 1.0), 0.0)
    return code.round().clamp(0, 2 ** bits - 1).to(torch.uint8), mn, scale


def _prepare_window(case, seed):
    k, v, q = _window_inputs(case, seed)
    tokens = _lengths(case)
    B, H, bits = case["batch"], case["kv_heads"], case["bits"]
    blocks, tails = [t // BT for t in tokens], [t % BT for t in tokens]
    nb = max(blocks)
    if own:
        from decode_gemv_packkv_b200 import packkv as pk
        cache = pk.PackKVCache(B, H, max(nb, 1), bits, keep_perm=True, ragged=True)
        if nb:
            pk.packkv_encode_block(cache, k[:, :, :nb * BT].contiguous(), v[:, :, :nb * BT].contiguous(), nb)
        cache.set_lengths(blocks, [0] * B)
        seq = torch.arange(B, device=DEV)
        base = torch.tensor(blocks, device=DEV) * BT
        for t in range(max(tails)):
            at = (base + t).clamp(max=case["tokens"] - 1)
            pk.packkv_append_token_masked(cache, k[seq, :, at].contiguous(), v[seq, :, at].contiguous(),
                                          [t < n for n in tails])
        out = torch.empty(q.shape, dtype=torch.float32, device=DEV)
        return dict(case=case, pk=pk, cache=cache, q=q, out=out)
    ck = torch.empty(B, H, nb, BT, D, dtype=torch.uint8, device=DEV)
    cv = torch.empty_like(ck)
    kmn, vmn = torch.empty(B, H, nb, 1, D, device=DEV), torch.empty(B, H, nb, BT, 1, device=DEV)
    ksc, vsc = torch.empty_like(kmn), torch.empty_like(vmn)
    kt = torch.zeros(B, H, BT, D, dtype=torch.float16, device=DEV)
    vt = torch.zeros_like(kt)
    for b in range(B):
        if nb:
            ck[b], kmn[b], ksc[b] = _quantize(k[b, :, :nb * BT].reshape(H, nb, BT, D), bits, -2)
            cv[b], vmn[b], vsc[b] = _quantize(v[b, :, :nb * BT].reshape(H, nb, BT, D), bits, -1)
        kt[b, :, :tails[b]] = k[b, :, blocks[b] * BT:tokens[b]]
        vt[b, :, :tails[b]] = v[b, :, blocks[b] * BT:tokens[b]]
    return dict(case=case, q=q, ck=ck, cv=cv, kmn=kmn, ksc=ksc, vmn=vmn, vsc=vsc, kt=kt, vt=vt,
                tokens=torch.tensor(tokens, device=DEV))


def _prepare_rope(case, seed):
    q, k, v, wq, wk = _head_inputs(case, seed, case["tokens"])
    pos = _far_positions(case, seed) if case["far"] else None
    s = dict(case=case, q=q, k=k, v=v, wq=wq, wk=wk, pos=pos)
    if own:
        B, T = case["batch"], case["tokens"]
        for name, heads in (("q_out", case["q_heads"]), ("k_out", case["kv_heads"]), ("v_out", case["kv_heads"])):
            s[name] = torch.empty(B, heads, T, D, dtype=torch.float16, device=DEV)
        s["pk"], s["rope"] = _own_rope(case)
    return s


def _own_rope(case):
    from decode_gemv_packkv_b200 import packkv as pk
    p = _rope_parameters(case)
    layout = {"half": pk.ROPE_HALF, "interleaved": pk.ROPE_INTERLEAVED}[case["layout"]]
    scaling = {"none": pk.ROPE_SCALE_NONE, "linear": pk.ROPE_SCALE_LINEAR, "base": pk.ROPE_SCALE_BASE,
               "parts": pk.ROPE_SCALE_PARTS}[case["scaling"]]
    return pk, pk.Rope(case["rot_dim"], layout, p["theta"], scaling=scaling, factor=p["factor"],
                       original_tokens=p["original"], low=p["low"], high=p["high"], amplitude=p["amplitude"])


def _append_lengths(case):
    """Tail tokens of every sequence before the step and which sequences take a token."""
    r = random.Random(case["tail"] * 1000 + case["batch"])
    if not case["ragged"]:
        return [case["tail"]] * case["batch"], [True] * case["batch"]
    return ([r.randrange(0, case["tail"] + 1) for _ in range(case["batch"])],
            [b == 0 or r.random() < 0.75 for b in range(case["batch"])])


def _prepare_append(case, seed):
    q, k, v, wq, wk = _head_inputs(case, seed, 1)
    q, k, v = q[:, 0], k[:, 0], v[:, 0]
    tails, active = _append_lengths(case)
    shape = (case["batch"], case["kv_heads"], BT, D)
    s = dict(case=case, q=q, k=k, v=v, wq=wq, wk=wk, tails=tails, active=active,
             q_out=torch.zeros(case["batch"], case["q_heads"], D, dtype=torch.float16, device=DEV))
    if own:
        s["pk"], s["rope"] = _own_rope(case)
        s["cache"] = s["pk"].PackKVCache(case["batch"], case["kv_heads"], 2, 4, ragged=case["ragged"])
    else:
        s["k_tail"] = torch.zeros(shape, dtype=torch.float16, device=DEV)
        s["v_tail"] = torch.zeros(shape, dtype=torch.float16, device=DEV)
        s["at"] = torch.tensor(tails, device=DEV)
        s["on"] = torch.tensor(active, device=DEV)
    return s


def _ranges(case, blocks):
    """Per sequence the first block given up and how many."""
    r = random.Random(case["shape"] + 1)
    first = [r.randrange(0, min(n, 2)) for n in blocks]
    count = [r.randrange(0, n - f + 1) for n, f in zip(blocks, first)]
    return first, [min(count[0], blocks[0] - first[0] - 1)] + count[1:]


def _pairs(case):
    """Sequence src[i] continues as dst[i] too."""
    order = list(range(case["batch"]))
    random.Random(case["shape"] + 2).shuffle(order)
    n = case["pairs"]
    keep = max(1, min(n, case["batch"] - n))
    return [order[n + i % keep] for i in range(n)], order[:n]


def _prepare_blocks(case, seed):
    index, arenas, perm, kt, vt, blocks, tails = _index_inputs(case, seed)
    s = dict(case=case, blocks=blocks, tails=tails)
    if case["op"] == "free":
        s["first"], s["count"] = _ranges(case, blocks)
    if case["op"] == "fork":
        s["src"], s["dst"] = _pairs(case)
    if own:
        from decode_gemv_packkv_b200 import packkv as pk
        s["pk"] = pk
        s["cache"] = _restored(pk, case, index, arenas, perm, kt, vt, blocks, tails)
        if case["op"] == "compact":
            s["to"] = pk.PackKVCache(case["batch"], case["kv_heads"], case["blocks"], case["bits"],
                                     arena_bytes=arenas[0].shape[0] * 16, keep_perm=True, ragged=True)
            for x in (s["to"].k_arena, s["to"].v_arena):
                x.zero_()
        return s
    s.update(k_index=index[0], v_index=index[1], arenas=arenas, perm=perm, k_tail=kt, v_tail=vt,
             n=torch.tensor(blocks, device=DEV), t=torch.tensor(tails, device=DEV))
    for name in ("first", "count", "src", "dst"):
        if name in s:
            s[name] = torch.tensor(s[name], device=DEV)
    return s


# ------------------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_window(s):
    c = s["case"]
    s["pk"].packkv_attention_window(s["cache"], s["q"], SCALE, s["out"], c["window"], sinks=c["sinks"],
                                    queries=c["queries"])
    return s["out"]


def _plain_window(s):
    c = s["case"]
    W, N0, S, G = c["window"], c["sinks"], c["queries"], c["group"]
    B, H, nb = s["ck"].shape[:3]
    tokens = s["tokens"]
    # blocks that any query may see: the first ones, and those back from each sequence's last
    back = min(nb, (W + S + BT - 1) // BT + 1)
    front = min(nb, -(-N0 // BT))
    last = tokens // BT
    sel = torch.cat([torch.arange(front, device=DEV).expand(B, front),
                     last[:, None] - 1 - torch.arange(back, device=DEV)], 1)
    there = (sel >= 0) & (sel < last[:, None])
    there[:, front:] &= sel[:, front:] >= front
    idx = sel.clamp(0, max(nb - 1, 0))
    row = torch.arange(B, device=DEV)[:, None]

    def values(code, mn, scale, tail):  # [B, H, N, 128] in fp32
        x = mn[row, :, idx] + scale[row, :, idx] * code[row, :, idx].float()  # [B, n, H, 128, 128]
        return torch.cat([x.transpose(1, 2).reshape(B, H, -1, D), tail.float()], 2)

    at = torch.arange(BT, device=DEV)
    pos = torch.cat([(sel[..., None] * BT + at).reshape(B, -1), last[:, None] * BT + at], 1)
    real = torch.cat([there[..., None].expand(B, sel.shape[1], BT).reshape(B, -1),
                      at < (tokens - last * BT)[:, None]], 1)
    here = tokens[:, None] - S + torch.arange(S, device=DEV)  # the queries' positions [B, S]
    see = (pos[:, None] <= here[..., None]) & ((pos[:, None] > here[..., None] - W) | (pos[:, None] < N0))
    see = (see & real[:, None])[:, None, :, None]  # [B, 1, S, 1, N]
    q = s["q"].float().reshape(B, H, S * G, D)
    score = (q @ values(s["ck"], s["kmn"], s["ksc"], s["kt"]).transpose(2, 3)) * SCALE
    score = torch.where(see, score.reshape(B, H, S, G, -1), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(see, torch.exp(score - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True).reshape(B, H, S * G, 1)
    out = p.reshape(B, H, S * G, -1) @ values(s["cv"], s["vmn"], s["vsc"], s["vt"])
    return torch.where(total > 0, out / torch.where(total > 0, total, 1.0), 0.0).reshape(B, H * S * G, D)


def _frequencies(c):
    """Angle per position of every rotated pair, fp64."""
    p, r = _rope_parameters(c), c["rot_dim"]
    theta, kind = p["theta"], c["scaling"]
    if kind == "base" and r > 2:
        theta *= p["factor"] ** (r / (r - 2))
    f = theta ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device=DEV) / r)
    if kind == "linear":
        f = f / p["factor"]
    if kind == "parts":  # turns within the trained length: few -> interpolated, many -> kept
        keep = ((p["original"] * f / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = keep * f + (1 - keep) * f / p["factor"]
    return f, p["amplitude"]


def _plain_head(x, w, c, f, amplitude, pos):
    """Norm and rotation of heads x [B, T, H, 128] at positions pos [B, T], fp32."""
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    angle = pos.double()[..., None] * f
    cos = (angle.cos() * amplitude).float()[:, :, None]
    sin = (angle.sin() * amplitude).float()[:, :, None]
    r = c["rot_dim"]
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(s):
    c = s["case"]
    f, amplitude = _frequencies(c)
    pos = s["pos"]
    if pos is None:
        pos = (c["first"] + torch.arange(c["tokens"], device=DEV)).expand(c["batch"], c["tokens"])
    q = _plain_head(s["q"], s["wq"], c, f, amplitude, pos)
    k = _plain_head(s["k"], s["wk"], c, f, amplitude, pos)
    return [x.transpose(1, 2).contiguous().half() for x in (q, k, s["v"].float())]


def _own_rope_run(s):
    c = s["case"]
    s["pk"].packkv_norm_rope(s["rope"], s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["v_out"],
                             q_weight=s["wq"], k_weight=s["wk"], eps=EPS if c["norm"] else None,
                             positions=s["pos"], first=c["first"])
    return [s["q_out"], s["k_out"], s["v_out"]]


def _plain_append(s):
    c = s["case"]
    f, amplitude = _frequencies(c)
    pos = s["at"][:, None]
    q = _plain_head(s["q"][:, None], s["wq"], c, f, amplitude, pos)[:, 0].half()
    k = _plain_head(s["k"][:, None], s["wk"], c, f, amplitude, pos)[:, 0].half()
    on = s["on"][:, None, None]
    row = torch.arange(c["batch"], device=DEV)
    q_out = torch.where(on, q, s["q_out"])
    s["k_tail"][row, :, s["at"]] = torch.where(on, k, s["k_tail"][row, :, s["at"]])
    s["v_tail"][row, :, s["at"]] = torch.where(on, s["v"].half(), s["v_tail"][row, :, s["at"]])
    return [q_out, s["k_tail"], s["v_tail"]]


def _own_append(s):
    c, cache = s["case"], s["cache"]
    # the step's token takes the place of the last one, as after a rejected draft
    cache.set_lengths([0] * c["batch"] if c["ragged"] else 0, s["tails"] if c["ragged"] else c["tail"])
    s["pk"].packkv_append_norm_rope(cache, s["rope"], s["q"], s["k"], s["v"], s["q_out"], q_weight=s["wq"],
                                    k_weight=s["wk"], eps=EPS if c["norm"] else None,
                                    active=s["active"] if c["ragged"] else None)
    return [s["q_out"], cache.k_tail, cache.v_tail]


def _plain_fork(s):
    src, dst = s["src"], s["dst"]
    n = s["n"][src]
    has = (torch.arange(s["k_index"].shape[2], device=DEV) < n[:, None])[:, None, :, None]
    for x in (s["k_index"], s["v_index"], s["perm"]):
        x[dst] = torch.where(has, x[src], x[dst])
    held = (torch.arange(BT, device=DEV) < s["t"][src][:, None])[:, None, :, None]
    for x in (s["k_tail"], s["v_tail"]):
        x[dst] = torch.where(held, x[src], x[dst])
    n_new, t_new = s["n"].clone(), s["t"].clone()
    n_new[dst], t_new[dst] = n, s["t"][src]
    return [s["k_index"], s["v_index"], s["perm"], s["k_tail"], s["v_tail"], n_new, t_new]


def _own_fork(s):
    cache = s["cache"]
    s["pk"].packkv_fork_sequences(cache, s["src"], s["dst"])
    return [cache.k_index, cache.v_index, cache.perm, cache.k_tail, cache.v_tail,
            np.array(cache.seq_blocks, np.int64), np.array(cache.seq_tail, np.int64)]


def _plain_free(s):
    at = torch.arange(s["k_index"].shape[2], device=DEV)
    gone = ((at >= s["first"][:, None]) & (at < (s["first"] + s["count"])[:, None]))[:, None, :]
    for x in (s["k_index"], s["v_index"]):
        x[..., 0] = torch.where(gone, FREED, x[..., 0])
        x[..., 1] = torch.where(gone, 0, x[..., 1])
    return [s["k_index"], s["v_index"]]


def _own_free(s):
    s["pk"].packkv_free_blocks(s["cache"], s["first"], s["count"])
    return [s["cache"].k_index, s["cache"].v_index]


def _plain_compact_one(index, arena, live):
    """Live records in the order of their first entry; entries that shared one still do."""
    held = live & (index[..., 0] != FREED)
    off = torch.where(held, index[..., 0], arena.shape[0]).flatten().long()
    length = torch.where(held, index[..., 1], 0).flatten().long()
    order = torch.argsort(off, stable=True)  # entries of one record side by side, the first one first
    lead = torch.ones_like(off, dtype=torch.bool)
    lead[1:] = off[order][1:] != off[order][:-1]
    owner = torch.empty_like(off)
    owner[order] = order[torch.cummax(torch.where(lead, torch.arange(off.numel(), device=DEV), 0), 0).values]
    mine = (owner == torch.arange(off.numel(), device=DEV)) & held.flatten()
    size = torch.where(mine, length, 0)
    start = size.cumsum(0) - size
    new = start[owner]
    total = int(size.sum())
    out = torch.zeros_like(arena)
    shift = torch.repeat_interleave(off - start, size)
    out[:total] = arena[torch.arange(total, device=DEV) + shift]
    entry = torch.stack([torch.where(held, new.reshape(held.shape), FREED), length.reshape(held.shape)], -1)
    return torch.where(live[..., None], entry, 0).int(), out, total


def _plain_compact(s):
    live = (torch.arange(s["k_index"].shape[2], device=DEV) < s["n"][:, None])[:, None].expand(s["k_index"].shape[:3])
    ki, ka, kn = _plain_compact_one(s["k_index"], s["arenas"][0], live)
    vi, va, vn = _plain_compact_one(s["v_index"], s["arenas"][1], live)
    perm = torch.where(live[..., None], s["perm"], 0)
    held = (torch.arange(BT, device=DEV) < s["t"][:, None])[:, None, :, None]
    kt, vt = torch.where(held, s["k_tail"], 0), torch.where(held, s["v_tail"], 0)
    ends = torch.tensor([kn, vn], device=DEV)
    return [ki, vi, ka.view(torch.uint8).flatten(), va.view(torch.uint8).flatten(), ends, perm, kt, vt]


def _own_compact(s):
    to = s["to"]
    s["pk"].packkv_compact(to, s["cache"])
    return [to.k_index, to.v_index, to.k_arena, to.v_arena, to.ctrl[:2], to.perm, to.k_tail, to.v_tail]


_PLAIN = dict(window=_plain_window, rope=_plain_rope, append=_plain_append, fork=_plain_fork, free=_plain_free,
              compact=_plain_compact)
_OWN = dict(window=_own_window, rope=_own_rope_run, append=_own_append, fork=_own_fork, free=_own_free,
            compact=_own_compact)


# ------------------------------------------------------------------------------- work
def _seen_blocks(case, tokens):
    """Whole blocks any query of a sequence sees, and its tail tokens."""
    W, N0, S = case["window"], case["sinks"], case["queries"]
    nb = tokens // BT
    lo = max(0, tokens - S - W + 1) // BT
    front = min(-(-N0 // BT), nb)
    return max(0, nb - max(lo, front)) + front, tokens % BT


def work(case):
    op = case["op"]
    if op == "window":
        B, H, rows = case["batch"], case["kv_heads"], case["queries"] * case["group"]
        # packed records of these compressible inputs take about three quarters of a raw one
        record = (528 + 2048 * case["bits"]) * (0.75 if case["structured"] else 1.0)
        seen = [_seen_blocks(case, t) for t in _lengths(case)]
        nbytes = sum(n * (record + 8) * 2 + t * D * 4 for n, t in seen) * H + B * H * rows * D * 6
        return dict(bytes=nbytes, flops=4.0 * D * H * rows * sum(n * BT + t for n, t in seen))
    if op in ("rope", "append"):
        n = case["batch"] * case.get("tokens", 1)
        size = 4 if case["dtype"] == "float32" else 2
        heads = case["q_heads"] + 2 * case["kv_heads"]
        if op == "append":
            n = sum(_append_lengths(case)[1])
        return dict(bytes=n * heads * D * (size + 2), flops=n * heads * D * 8.0)
    r = random.Random(case["shape"])
    nb, H = case["blocks"], case["kv_heads"]
    blocks = [nb] + [r.randrange(1, nb + 1) for _ in range(case["batch"] - 1)]
    tails = [r.randrange(0, BT) for _ in range(case["batch"])]
    if op == "fork":
        src, _ = _pairs(case)
        return dict(bytes=sum(2 * H * (blocks[b] * (16 + BT) + tails[b] * D * 4) for b in src), flops=0)
    if op == "free":
        return dict(bytes=sum(_ranges(case, blocks)[1]) * H * 16, flops=0)
    raw = 528 + 2048 * case["bits"]
    mean = (16 * (65 + raw // 64) + raw) / 2 if case["packed"] else raw
    shared = sum(min(blocks[2 * f], blocks[2 * f + 1]) for f in range(case["forks"]))
    own_records = (sum(blocks) - shared) * H * (1 - case["dead"])
    return dict(bytes=2 * (2 * own_records * mean + sum(blocks) * H * (16 + BT) + sum(tails) * H * D * 4), flops=0)


# ------------------------------------------------------------------------------- exact
def exact(case, seed):
    if case["op"] == "window":
        return _exact_window(case, seed)
    if case["op"] in ("rope", "append"):
        return _exact_heads(case, seed)
    return None  # nothing is computed: entries and bytes are moved


def _exact_values(x, bits, axis):
    """What the codes of x [.., 128, 128] stand for, quantized along `axis`, fp64."""
    lo = x.double().amin(axis, keepdim=True)
    span = x.double().amax(axis, keepdim=True) - lo
    # fp64 quotients of fp32 values round to the fp32 quotient (53 >= 2*24 + 2 bits)
    s32 = (span.float().double() / torch.full((1,), 2 ** bits - 1, dtype=torch.float64, device=x.device)).float()
    h = s32.half()
    h = (h.view(torch.int16) + (h.float() < s32).short()).view(torch.float16).double()
    diff = (x.double() - lo).float().double()
    code = torch.zeros_like(diff)
    some = (h > 0).expand_as(diff)
    code[some] = torch.round((diff / h)[some].float()).double().clamp(0, 2 ** bits - 1)
    return lo + h * code


def _exact_window(case, seed):
    k, v, q = _window_inputs(case, seed)
    H, S, G, bits = case["kv_heads"], case["queries"], case["group"], case["bits"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for b, t in enumerate(_lengths(case)):
        packed = t // BT * BT
        first = max(0, t - S - case["window"] + 1)
        want = sorted(set(range(0, min(case["sinks"], t))) | set(range(first, t)))
        need = sorted({p // BT for p in want if p < packed})
        ks, vs = k[b, :, packed:t].double(), v[b, :, packed:t].double()
        at = torch.arange(packed, t, device=DEV)
        if need:
            rows = torch.tensor(need, device=DEV)
            kb = k[b, :, :packed].reshape(H, -1, BT, D)[:, rows]
            vb = v[b, :, :packed].reshape(H, -1, BT, D)[:, rows]
            ks = torch.cat([_exact_values(kb, bits, -2).reshape(H, -1, D), ks], 1)
            vs = torch.cat([_exact_values(vb, bits, -1).reshape(H, -1, D), vs], 1)
            at = torch.cat([(rows[:, None] * BT + torch.arange(BT, device=DEV)).flatten(), at])
        for s in range(S):
            p = t - S + s
            seen = ((at <= p) & ((at > p - case["window"]) | (at < case["sinks"]))).nonzero().flatten()
            if p < 0 or not len(seen):
                continue
            rows = (torch.arange(H, device=DEV)[:, None] * S * G + s * G + torch.arange(G, device=DEV)).flatten()
            qs = q[b, rows].double().reshape(H, G, D)
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", qs, ks[:, seen]) * SCALE, -1)
            out[b, rows] = torch.einsum("hgn,hnd->hgd", w, vs[:, seen]).reshape(H * G, D)
    return out


def _exact_heads(case, seed):
    tokens = case.get("tokens", 1)
    q, k, v, wq, wk = _head_inputs(case, seed, tokens)
    B, r = case["batch"], case["rot_dim"]
    par = _rope_parameters(case)
    tails, active = _append_lengths(case) if case["op"] == "append" else (None, None)
    if case["op"] == "append":
        pos = np.array(tails, np.float64)[:, None]
    elif case["far"]:
        pos = _far_positions(case, seed).cpu().numpy().astype(np.float64)
    else:
        pos = np.tile(case["first"] + np.arange(tokens, dtype=np.float64), (B, 1))
    turn = np.zeros((B, tokens, D // 2))
    for i in range(r // 2):
        base = par["theta"] * (par["factor"] ** (r / (r - 2.0)) if case["scaling"] == "base" and r > 2 else 1.0)
        f = base ** (-2.0 * i / r)
        if case["scaling"] == "linear":
            f /= par["factor"]
        if case["scaling"] == "parts":
            keep = min(1.0, max(0.0, (par["original"] * f / (2 * math.pi) - par["low"]) / (par["high"] - par["low"])))
            f = keep * f + (1.0 - keep) * f / par["factor"]
        turn[:, :, i] = pos * f
    z = torch.from_numpy(np.cos(turn) + 1j * np.sin(turn)).to(DEV)[:, :, None] * par["amplitude"]

    def head(x, w):
        x = x.double()
        if case["norm"]:
            x = x / ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        pair = [(i, i + r // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1) for i in range(r // 2)]
        a, b = [p[0] for p in pair], [p[1] for p in pair]
        turned = torch.complex(x[..., a], x[..., b]) * z[..., :r // 2]
        y = x.clone()
        y[..., a], y[..., b] = turned.real, turned.imag
        return y

    if case["op"] == "rope":
        return [x.transpose(1, 2).contiguous() for x in (head(q, wq), head(k, wk), v.double())]
    qo = torch.zeros(B, case["q_heads"], D, dtype=torch.float64, device=DEV)
    kt = torch.zeros(B, case["kv_heads"], BT, D, dtype=torch.float64, device=DEV)
    vt = torch.zeros_like(kt)
    qh, kh = head(q, wq)[:, 0], head(k, wk)[:, 0]
    for b in range(B):
        if active[b]:
            qo[b], kt[b, :, tails[b]], vt[b, :, tails[b]] = qh[b], kh[b], v[b, 0].double()
    return [qo, kt, vt]
