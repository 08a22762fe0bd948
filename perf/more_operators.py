"""The cases in which the framework's step builder, cross attention and linear attention
are timed, with a plain form of each in elementary torch operations.

Three operators of one serving step whose layers are not all causal attention over
their own cache:
  build   the step's metadata made on the GPU from request lengths, with blocks taken from
          and given back to a free list (pa_build_step)
  cross   attention of the step's rows to an encoder's states in the paged pool
          (pa_cross_attention)
  linear  linear attention with a decay per head over a pool of states
          (pa_linear_attention)
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
CHUNK = 64  # the plain form's chunk of tokens

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _build(name, block_size, width, prompts, prompt_lo, prompt_hi, decodes, specs, released, idle,
           ctx_lo, ctx_hi, padding):
    return {"name": name, "op": "build", "block_size": block_size, "width": width,
            "prompts": prompts, "prompt_lo": prompt_lo, "prompt_hi": prompt_hi,
            "decodes": decodes, "specs": specs, "released": released, "idle": idle,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "padding": padding}


def _cross(name, q_heads, kv_heads, head_dim, block_size, kv, chunks, chunk_len, decodes, specs,
           len_lo, len_hi):
    return {"name": name, "op": "cross", "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "block_size": block_size, "kv": kv, "chunks": chunks,
            "chunk_len": chunk_len, "decodes": decodes, "specs": specs, "len_lo": len_lo,
            "len_hi": len_hi}


def _linear(name, q_heads, kv_heads, head_dim, decay, chunks, chunk_len, decodes, specs, fresh):
    return {"name": name, "op": "linear", "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "decay": decay, "chunks": chunks, "chunk_len": chunk_len,
            "decodes": decodes, "specs": specs, "fresh": fresh}


def listed():
    return [
        # a decode step of a small batch: latency
        _build("build_decode", 16, 640, 0, 0, 0, 64, 0, 0, 0, 256, 8192, 0),
        # a continuous-batching step: prompt chunks, decode rows and verify rows, some rows done
        _build("build_mixed", 16, 1024, 8, 512, 512, 192, 32, 12, 12, 0, 8192, 100),
        # many prompts at once, ragged, among finished rows
        _build("build_prompts", 32, 512, 512, 33, 511, 128, 0, 64, 320, 0, 16000, 0),
        # one stream of a small encoder-decoder model: latency
        _cross("cross_one_stream", 4, 2, 64, 16, "bf16", 0, 0, 1, 0, 700, 700),
        # a decode batch, each row with its own encoder states
        _cross("cross_decode", 32, 8, 128, 16, "bf16", 0, 0, 64, 0, 512, 4096),
        # a large decode batch over a quantised pool
        _cross("cross_decode_e4m3", 32, 8, 128, 16, "e4m3", 0, 0, 256, 0, 256, 4096),
        # prompts of the decoder among decode and verify rows
        _cross("cross_mixed", 32, 8, 128, 16, "bf16", 8, 512, 192, 32, 256, 4096),
        # one token of a small model: latency
        _linear("linear_one_stream", 4, 2, 64, "head", 0, 0, 1, 0, 0),
        # a large decode batch: every request's states read and written
        _linear("linear_decode", 32, 8, 128, "head", 0, 0, 256, 0, 0),
        # speculative verification, odd numbers of rows, a decay for each token
        _linear("linear_verify", 8, 2, 64, "token", 0, 0, 0, 24, 0),
        # a continuous-batching step: prompt chunks, decode rows and verify rows
        _linear("linear_mixed", 32, 8, 128, "token", 8, 512, 192, 32, 3),
        # long prompts, a key and a value head for each query head
        _linear("linear_prompt", 32, 32, 128, "head", 2, 8192, 0, 0, 2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(4, 2), (8, 2), (32, 8), (16, 1), (14, 2), (6, 6), (12, 4), (32, 8)]


def draw(rng):
    op = rng.choice(["build", "cross", "cross", "linear", "linear", "linear"])
    shape = rng.choice(["decode", "verify", "mixed", "prefill"])
    chunks = decodes = specs = chunk_len = 0
    if shape == "decode":
        decodes = _log(rng, 1, 256)
    elif shape == "verify":
        specs = _log(rng, 1, 64)
    elif shape == "mixed":
        chunks, chunk_len = rng.randint(1, 6), _log(rng, 17, 700)
        decodes, specs = _log(rng, 1, 128), _log(rng, 1, 32)
    else:
        chunks, chunk_len = rng.randint(1, 3), _log(rng, 65, 4096)
    if op == "build":
        block_size = rng.choice([16, 16, 32, 64])
        hi = _log(rng, 64, 16384)
        longest = hi + max(chunk_len, 8)
        case = _build("", block_size, -(-longest // block_size) + rng.randint(0, 9), chunks,
                      max(1, chunk_len // 3), max(1, chunk_len), decodes, specs,
                      rng.choice([0, rng.randint(1, 40)]), rng.choice([0, _log(rng, 1, 400)]),
                      rng.choice([0, hi // 2]), hi, rng.choice([0, rng.randint(1, 500)]))
    elif op == "cross":
        kv = rng.choice(["bf16", "bf16", "e4m3"])
        head_dim = 128 if kv == "e4m3" else rng.choice([64, 128, 128])
        q_heads, kv_heads = rng.choice(HEADS)
        lo = _log(rng, 1, 1000)
        case = _cross("", q_heads, kv_heads, head_dim, rng.choice([16, 16, 32, 64]), kv, chunks,
                      min(chunk_len, 1024), decodes, specs, lo, lo + _log(rng, 1, 2000))
    else:
        q_heads, kv_heads = rng.choice(HEADS + [(16, 16)])
        n = chunks + decodes + specs
        case = _linear("", q_heads, kv_heads, rng.choice([64, 128, 128]),
                       rng.choice(["head", "token"]), chunks, chunk_len, decodes, specs,
                       rng.choice([0, n, rng.randint(0, n)]))
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _spread(i):
    """The i-th of numbers spread over [0, 1), the same for every seed."""
    return (0.381966 * (i + 1) * (i + 1)) % 1.0


def _rows(case):
    """New tokens of every request."""
    return [case["chunk_len"]] * case["chunks"] + [1] * case["decodes"] + [5] * case["specs"]


def _build_rows(case):
    """(new tokens, cached tokens) of every row of the persistent batch; new tokens -1:
    the row is done.  Rows of every kind alternate."""
    kinds = (["prompt"] * case["prompts"] + ["decode"] * case["decodes"] + ["spec"] * case["specs"]
             + ["done"] * case["released"] + ["idle"] * case["idle"])
    order = sorted(range(len(kinds)), key=lambda i: _spread(i + 7))
    span, rows = case["ctx_hi"] - case["ctx_lo"], []
    for at, i in enumerate(order):
        c = case["ctx_lo"] + int(span * _spread(at))
        n = {"decode": 1, "spec": 5, "done": -1, "idle": 0}.get(kinds[i])
        if n is None:
            n = case["prompt_lo"] + int((case["prompt_hi"] - case["prompt_lo"] + 1) * _spread(at + 3))
            c = c if at % 2 else 0  # a first chunk, or a later one
        rows.append((n, 0 if kinds[i] == "idle" and at % 3 else c))
    return rows


def _prepare_build(case, gen, dev):
    rows, bs, width = _build_rows(case), case["block_size"], case["width"]
    have = [-(-c // bs) for _, c in rows]
    need = sum(-(-(c + n) // bs) - h for (n, c), h in zip(rows, have) if n > 0)
    used = sum(have)
    num_blocks = used + need + need // 4 + 16
    perm = torch.randperm(num_blocks, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(rows), width), -1, dtype=torch.int32, device=dev)
    cols = torch.arange(width, device=dev)
    owned = cols < torch.tensor(have, device=dev)[:, None]
    table[owned] = perm[:used]
    head = int(torch.randint(0, num_blocks, (1,), generator=gen, device=dev))
    ring = torch.full((num_blocks,), -1, dtype=torch.int32, device=dev)
    free = num_blocks - used
    ring[(head + torch.arange(free, device=dev)) % num_blocks] = perm[used:]
    total = sum(max(n, 0) for n, _ in rows)
    tokens = total + case["padding"]
    i32 = dict(dtype=torch.int32, device=dev)
    b = len(rows)
    return {"case": case, "num_blocks": num_blocks,
            "query_lens": torch.tensor([n for n, _ in rows], **i32),
            "cached": torch.tensor([c for _, c in rows], **i32), "table": table, "ring": ring,
            "state": torch.tensor([head, free, 0, 0], **i32),
            "state_out": torch.zeros(4, **i32), "qsl": torch.zeros(b + 1, **i32),
            "ctx": torch.zeros(b, **i32), "seq": torch.zeros(b, **i32),
            "slots": torch.zeros(tokens, dtype=torch.int64, device=dev),
            "positions": torch.zeros(tokens, **i32)}


def _pool(gen, shape, kv, dev):
    """One cache array: normal bf16 values, or e4m3 codes of normal values of
    deviation 16 (no NaN codes)."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32
                    if math.prod(shape) < (1 << 28) else torch.bfloat16)
    if kv == "bf16":
        return x.to(torch.bfloat16)
    return (x.float() * 16).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scales(gen, heads, dev):
    return 0.03 + 0.04 * torch.rand(heads, generator=gen, device=dev)


def _cross_requests(case):
    """(encoder states, new tokens) of every request."""
    span = case["len_hi"] - case["len_lo"]
    return [(case["len_lo"] + int(span * _spread(i)), n) for i, n in enumerate(_rows(case))]


def _starts(n):
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    return starts


def _prepare_cross(case, gen, dev):
    reqs = _cross_requests(case)
    bs, hkv, hq, d = case["block_size"], case["kv_heads"], case["q_heads"], case["head_dim"]
    blocks = [-(-length // bs) for length, _ in reqs]
    used = sum(blocks)
    num_blocks = used + used // 10 + 1
    perm = torch.randperm(num_blocks, generator=gen, device=dev)[:used].to(torch.int32)
    table = torch.full((len(reqs), max(blocks)), -1, dtype=torch.int32, device=dev)
    table[torch.arange(max(blocks), device=dev) < torch.tensor(blocks, device=dev)[:, None]] = perm
    starts = _starts(n for _, n in reqs)
    total = starts[-1]
    i32 = dict(dtype=torch.int32, device=dev)
    shape = (num_blocks, hkv, bs, d)
    fp8 = case["kv"] == "e4m3"
    st = {"case": case, "scale": 1.0 / math.sqrt(d), "table": table,
          "qsl": torch.tensor(starts, **i32), "lens": torch.tensor([x for x, _ in reqs], **i32),
          "q": torch.randn((total, hq, d), generator=gen, device=dev).to(torch.bfloat16),
          "k": _pool(gen, shape, case["kv"], dev), "v": _pool(gen, shape, case["kv"], dev),
          "k_scale": _scales(gen, hkv, dev) if fp8 else None,
          "v_scale": _scales(gen, hkv, dev) if fp8 else None,
          "out": torch.zeros((total, hq, d), dtype=torch.bfloat16, device=dev),
          "lse": torch.zeros((total, hq), device=dev), "workspace": None,
          # blocks of requests with more than 64 query rows per kv head (a quantised
          # pool's bf16 staging room)
          "staging": sum(x for x, (_, n) in zip(blocks, reqs) if n * hq // hkv > 64) if fp8 else 0}
    # The plain form's tiles: `tile` consecutive query tokens of one request
    tile = min(128 if not case["decodes"] + case["specs"] else 16, max(n for _, n in reqs))
    tiles = [(b, i) for b, (_, n) in enumerate(reqs) for i in range(0, n, tile)]
    st["tile"] = tile
    st["tile_req"] = torch.tensor([b for b, _ in tiles], device=dev)
    st["tile_first"] = torch.tensor([i for _, i in tiles], device=dev)
    return st


def _prepare_linear(case, gen, dev):
    n = _rows(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    starts = _starts(n)
    total, reqs = starts[-1], len(n)
    # rows of the fused projection: q, k and v of a token next to each other
    qkv = torch.randn((total, (hq + 2 * hkv) * d), generator=gen, device=dev).to(torch.bfloat16)
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
    if case["decay"] == "head":  # half-lives from 20 to 700 tokens
        decay = torch.log1p(-2.0 ** (-5 - 5 * torch.arange(hkv, device=dev) / hkv))
    else:  # most tokens keep nearly everything, some little
        decay = -torch.exp(torch.randn((total, hkv), generator=gen, device=dev) * 1.5 - 3.5)
    i32 = dict(dtype=torch.int32, device=dev)
    # every request reads one slot and writes another (a program that may take steps
    # back); the last slot is not a user's: it takes the plain form's unused writes
    whole = torch.randn((2 * reqs + 1, hkv, d, d), generator=gen, device=dev)
    slots = torch.randperm(reqs, generator=gen, device=dev).to(torch.int32)
    state_in = slots.clone()
    state_in[:case["fresh"]] = -1
    # the plain form's groups of requests of like length
    groups = []
    for members in ([b for b in range(reqs) if n[b] <= 8], [b for b in range(reqs) if n[b] > 8]):
        if members:
            step = max(n[b] for b in members)
            step = step if step <= 8 else -(-step // CHUNK) * CHUNK
            i = torch.arange(step, device=dev)
            first = torch.tensor([starts[b] for b in members], device=dev)[:, None]
            length = torch.tensor([n[b] for b in members], device=dev)[:, None]
            groups.append((torch.tensor(members, device=dev),
                           torch.where(i < length, first + i, total)))
    return {"case": case, "scale": 1.0 / math.sqrt(d), "q": q.view(total, hq, d),
            "k": k.view(total, hkv, d), "v": v.view(total, hkv, d), "decay": decay.float(),
            "qsl": torch.tensor(starts, **i32), "whole": whole, "state": whole[:-1],
            "state_in": state_in, "state_out": slots + reqs, "groups": groups,
            "out": torch.zeros((total, hq, d), dtype=torch.bfloat16, device=dev),
            "workspace": None}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    return {"build": _prepare_build, "cross": _prepare_cross,
            "linear": _prepare_linear}[case["op"]](case, gen, dev)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _built(st):
    return {x: st[x] for x in ("qsl", "ctx", "seq", "slots", "positions", "table", "ring",
                               "state_out")}


def _run_build(st):
    bs, table, ring = st["case"]["block_size"], st["table"], st["ring"]
    rows, width = table.shape
    cap, tokens = ring.numel(), st["slots"].numel()
    dev = table.device
    q, cached = st["query_lens"].long(), st["cached"].long()
    head, count = st["state"][0].long(), st["state"][1].long()
    done, n = q < 0, q.clamp(min=0)
    have, want = (cached + bs - 1) // bs, (cached + n + bs - 1) // bs
    need = want - have
    missing = (need.sum() - count).clamp(min=0)
    good = (missing == 0) & (n.sum() <= tokens) & (want <= width).all()
    n, need = n * good, need * good
    released = done & good
    ctx = torch.where(released, 0, cached)
    cols = torch.arange(width, device=dev)
    # the last table entries of every row from the head of the free list
    fresh = (cols >= have[:, None]) & (cols < (have + need)[:, None])
    at = head + (need.cumsum(0) - need - have)[:, None] + cols
    old = torch.where(released[:, None] & (cols < have[:, None]), table, -1).flatten()
    table.copy_(torch.where(fresh, ring[at % cap].clamp(0, st["num_blocks"] - 1), table))
    # the blocks of finished rows to its tail
    given = old >= 0
    place = torch.where(given, (head + count + given.cumsum(0) - 1) % cap, cap)
    longer = torch.cat([ring, ring[:1]])
    longer[place] = old
    ring.copy_(longer[:cap])
    ends = n.cumsum(0)
    st["qsl"][1:] = ends
    st["ctx"].copy_(ctx)
    st["seq"].copy_(ctx + n)
    taken = need.sum()
    st["state_out"].copy_(torch.stack([(head + taken) % cap, count - taken + given.sum(), missing,
                                       torch.zeros_like(head)]))
    t = torch.arange(tokens, device=dev)
    b = torch.searchsorted(ends, t, right=True).clamp(max=rows - 1)
    pos = ctx[b] + t - (ends - n)[b]
    live = t < ends[-1]
    block = table[b, torch.where(live, pos // bs, 0)].long()
    st["slots"].copy_(torch.where(live, block * bs + pos % bs, -1))
    st["positions"].copy_(torch.where(live, pos, 0))
    return _built(st)


def _gather(pool, blocks, offsets, scale):
    """Rows (block, offset) of every kv head in 32 bits: [tiles, kv heads, keys, d]."""
    raw = pool if scale is None else pool.view(torch.uint8)
    x = raw[blocks, :, offsets]
    x = x.float() if scale is None else x.view(torch.float8_e4m3fn).float() * scale[:, None]
    return x.transpose(1, 2)


def _run_cross(st):
    case, q = st["case"], st["q"]
    bs, hkv = case["block_size"], case["kv_heads"]
    dev, (total, hq, d) = q.device, q.shape
    group, tile = hq // hkv, st["tile"]
    req, first = st["tile_req"], st["tile_first"]
    lens, start, end = st["lens"][req].long(), st["qsl"][req].long(), st["qsl"][req + 1].long()
    token = (start + first)[:, None] + torch.arange(tile, device=dev)
    token = torch.where(token < end[:, None], token, total)
    keys = torch.arange(st["table"].shape[1] * bs, device=dev)
    blocks = st["table"][req].clamp(min=0).long().repeat_interleave(bs, dim=1)
    offsets = (keys % bs).expand(blocks.shape)
    k = _gather(st["k"], blocks, offsets, st["k_scale"])
    v = _gather(st["v"], blocks, offsets, st["v_scale"])
    qt = q[token.clamp(max=total - 1)].float().view(-1, tile, hkv, group, d)
    qt = qt.permute(0, 2, 1, 3, 4).reshape(-1, hkv, tile * group, d)
    s = (qt @ k.transpose(2, 3)) * st["scale"]
    s.masked_fill_((keys >= lens[:, None])[:, None, None, :], float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    e = (s - m).exp_()
    z = e.sum(dim=-1, keepdim=True)
    o = ((e @ v) / z).view(-1, hkv, tile, group, d)
    lse = (m + z.log()).view(-1, hkv, tile, group)
    out = q.new_empty((total + 1, hq, d))
    out[token] = o.permute(0, 2, 1, 3, 4).reshape(-1, tile, hq, d).to(torch.bfloat16)
    out_lse = lse.new_empty((total + 1, hq))
    out_lse[token] = lse.permute(0, 2, 1, 3).reshape(-1, tile, hq)
    return {"out": out[:total], "lse": out_lse[:total]}


def _recurrent(q, k, v, g, s):
    """q [R, T, Hkv, group, d], k and v [R, T, Hkv, d], g [R, T, Hkv], s [R, Hkv, d, d]."""
    outs = []
    for t in range(k.shape[1]):
        s = g[:, t, :, None, None].exp() * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        outs.append(q[:, t] @ s)
    return torch.stack(outs, dim=1), s


def _chunked(q, k, v, g, s):
    """The same, a chunk of tokens at a time."""
    r, t, hkv, group, d = q.shape
    n = t // CHUNK
    q = q.view(r, n, CHUNK, hkv, group, d).permute(0, 3, 1, 4, 2, 5)        # [R, H, n, g, C, d]
    k, v = (x.view(r, n, CHUNK, hkv, d).permute(0, 3, 1, 2, 4) for x in (k, v))
    # the decay summed over a chunk in 64 bits: its differences lose nothing
    a = g.double().view(r, n, CHUNK, hkv).permute(0, 3, 1, 2).cumsum(dim=-1)  # [R, H, n, C]
    lower = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=q.device).tril()
    weight = (a[..., :, None] - a[..., None, :]).float().masked_fill_(~lower, float("-inf")).exp_()
    last = (a[..., -1:] - a).float().exp()
    from_chunk = (k * last[..., None]).transpose(-1, -2) @ v                # [R, H, n, d, d]
    whole = a[..., -1].float().exp()[..., None, None]
    before = []
    for i in range(n):
        before.append(s)
        s = whole[:, :, i] * s + from_chunk[:, :, i]
    before = torch.stack(before, dim=2)[:, :, :, None]
    inside = (q @ k[:, :, :, None].transpose(-1, -2)) * weight[:, :, :, None]
    o = inside @ v[:, :, :, None] + (q @ before) * a.float().exp()[:, :, :, None, :, None]
    return o.permute(0, 2, 4, 1, 3, 5).reshape(r, t, hkv, group, d), s


def _run_linear(st):
    q, k, v = st["q"], st["k"], st["v"]
    total, hq, d = q.shape
    hkv = k.shape[1]
    out = q.new_empty((total + 1, hq, d))
    decay = st["decay"] if st["decay"].dim() == 2 else st["decay"].expand(total, -1)
    state, unused = st["whole"], st["whole"].shape[0] - 1
    for members, token in st["groups"]:
        live = (token < total)
        at = token.clamp(max=total - 1)
        qf = q[at].float().view(*at.shape, hkv, hq // hkv, d)
        kf, vf, g = k[at].float() * live[..., None, None], v[at].float(), decay[at] * live[..., None]
        src = st["state_in"][members].long()
        s = state[src.clamp(min=0)] * (src >= 0)[:, None, None, None]
        o, s = (_recurrent if token.shape[1] <= 8 else _chunked)(qf, kf, vf, g, s)
        out[token] = (o * st["scale"]).view(*at.shape, hq, d).to(torch.bfloat16)
        dst = st["state_out"][members].long()
        state[torch.where(dst < 0, unused, dst)] = s
    return {"out": out[:total], "state": st["state"]}


def _own_build(st):
    import paged_kv_cache_284_gb300 as pk
    pk.pa_build_step(st["query_lens"], st["cached"], st["table"], st["ring"], st["state"],
                     st["num_blocks"], st["case"]["block_size"], st["qsl"], st["ctx"], st["seq"],
                     st["slots"], st["positions"], free_state_out=st["state_out"])
    return _built(st)


def _own_cross(st):
    import paged_kv_cache_284_gb300 as pk
    st["workspace"] = pk.pa_cross_attention(
        st["q"], st["k"], st["v"], st["table"], st["qsl"], st["lens"], st["scale"], st["out"],
        st["lse"], workspace=st["workspace"], k_scale=st["k_scale"], v_scale=st["v_scale"],
        staging_blocks=st["staging"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_linear(st):
    import paged_kv_cache_284_gb300 as pk
    st["workspace"] = pk.pa_linear_attention(
        st["q"], st["k"], st["v"], st["qsl"], st["decay"], st["state"], st["state_in"],
        st["state_out"], st["scale"], st["out"], workspace=st["workspace"])
    return {"out": st["out"], "state": st["state"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"build": _own_build, "cross": _own_cross, "linear": _own_linear}[op](state)
    return {"build": _run_build, "cross": _run_cross, "linear": _run_linear}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "build":
        rows, bs = _build_rows(case), case["block_size"]
        total = sum(max(n, 0) for n, _ in rows)
        fresh = sum(-(-(c + n) // bs) - -(-c // bs) for n, c in rows if n > 0)
        given = sum(-(-c // bs) for n, c in rows if n < 0)
        open_block = sum(n > 0 and c % bs != 0 for n, c in rows)
        return {"bytes": 20 * len(rows) + 4 + 12 * (total + case["padding"])
                + 8 * (fresh + given) + 4 * open_block + 32, "flops": 0}
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "cross":
        elem = 2 if case["kv"] == "bf16" else 1
        reqs = _cross_requests(case)
        keys, tokens = sum(x for x, _ in reqs), sum(n for _, n in reqs)
        entries = sum(-(-x // case["block_size"]) for x, _ in reqs)
        return {"bytes": 2 * keys * hkv * d * elem + tokens * hq * (4 * d + 4) + 4 * entries,
                "flops": 4 * sum(x * n for x, n in reqs) * hq * d}
    n = _rows(case)
    decay = 4 * hkv * (sum(n) if case["decay"] == "token" else 1)
    return {"bytes": sum(n) * d * 4 * (hq + hkv) + decay
            + 4 * hkv * d * d * (2 * len(n) - case["fresh"]),
            "flops": 2 * d * d * (hq + hkv) * sum(n)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_build(case, st):
    """Row after row, as a scheduler on the host would."""
    bs = case["block_size"]
    table, ring = st["table"].cpu().numpy().copy(), st["ring"].cpu().numpy().copy()
    head, count = (int(x) for x in st["state"][:2].cpu())
    taken, given = 0, []
    qsl, ctx, seq, slots, positions = [0], [], [], [], []
    for b, (n, c) in enumerate(zip(st["query_lens"].tolist(), st["cached"].tolist())):
        if n < 0:
            given += [x for x in table[b, :-(-c // bs)] if x >= 0]
            n = c = 0
        for col in range(-(-c // bs), -(-(c + n) // bs)):
            table[b, col] = ring[(head + taken) % len(ring)]
            taken += 1
        p = np.arange(c, c + n)
        slots.append(table[b, p // bs].astype(np.int64) * bs + p % bs)
        positions.append(p)
        qsl.append(qsl[-1] + n)
        ctx.append(c)
        seq.append(c + n)
    for i, x in enumerate(given):
        ring[(head + count + i) % len(ring)] = x
    pad = st["slots"].numel() - qsl[-1]
    slots.append(np.full(pad, -1))
    positions.append(np.zeros(pad, np.int64))
    found = {"qsl": qsl, "ctx": ctx, "seq": seq, "slots": np.concatenate(slots),
             "positions": np.concatenate(positions), "table": table, "ring": ring,
             "state_out": [(head + taken) % len(ring), count - taken + len(given), 0, 0]}
    return {x: torch.as_tensor(np.asarray(y)).to(st[x].dtype).to(st[x].device)
            for x, y in found.items()}


def _exact_cross(case, st):
    total, hq, d = st["q"].shape
    hkv, bs = case["kv_heads"], case["block_size"]
    group = hq // hkv
    dev = st["q"].device
    out = torch.zeros((total, hq, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((total, hq), dtype=torch.float64, device=dev)
    at = 0
    for b, (length, n) in enumerate(_cross_requests(case)):
        rows = st["table"][b, :-(-length // bs)].long()
        fp8 = st["k_scale"] is not None
        k, v = (st[x].view(torch.uint8 if fp8 else torch.bfloat16)[rows] for x in ("k", "v"))
        if fp8:
            k, v = (x.view(torch.float8_e4m3fn).double() * st[s].double()[:, None, None]
                    for x, s in ((k, "k_scale"), (v, "v_scale")))
        k, v = (x.double().transpose(0, 1).reshape(hkv, -1, d)[:, :length] for x in (k, v))
        x = st["q"][at:at + n].double().view(n, hkv, group, d)
        s = torch.einsum("thgd,hkd->htgk", x, k) * st["scale"]
        z = torch.logsumexp(s, dim=-1)
        lse[at:at + n] = z.transpose(0, 1).reshape(n, hq)
        o = torch.einsum("htgk,hkd->thgd", (s - z[..., None]).exp_(), v)
        out[at:at + n] = o.reshape(n, hq, d)
        at += n
    return {"out": out, "lse": lse}


def _exact_linear(case, st):
    """Token after token, the requests side by side, the longest first."""
    n = _rows(case)
    order = sorted(range(len(n)), key=lambda b: -n[b])
    total, hq, d = st["q"].shape
    hkv = case["kv_heads"]
    dev = st["q"].device
    starts = _starts(n)
    first = torch.tensor([starts[b] for b in order], device=dev)
    pick = torch.tensor(order, device=dev)
    src = st["state_in"][pick].long()
    s = st["state"][src.clamp(min=0)].double()
    s[src < 0] = 0
    out = torch.zeros((total, hq, d), dtype=torch.float64, device=dev)
    lengths = [n[b] for b in order]
    live = len(order)
    for t in range(lengths[0]):
        while lengths[live - 1] <= t:
            live -= 1
        at, now = first[:live] + t, s[:live]
        g = st["decay"].double()
        now.mul_((g[at] if g.dim() == 2 else g.expand(live, -1)).exp()[..., None, None])
        now.add_(st["k"][at].double()[..., :, None] * st["v"][at].double()[..., None, :])
        o = st["q"][at].double().view(live, hkv, hq // hkv, d) @ now
        out[at] = o.view(live, hq, d) * st["scale"]
    state = st["state"].double()
    dst = st["state_out"][pick].long()
    state[dst[dst >= 0]] = s[dst >= 0]
    return {"out": out, "state": state}


def exact(case, seed):
    st = prepare(case, seed)
    return {"build": _exact_build, "cross": _exact_cross,
            "linear": _exact_linear}[case["op"]](case, st)
