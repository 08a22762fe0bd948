"""The cases in which the framework's windowed attention, rotary cache write and
block copies are timed, with a plain form of each in elementary torch operations.

Three operators of one serving step over a paged KV cache:
  window  attention with a sliding window and sink tokens (pa_window_attention)
  rope    rotary positions with several axes on q and k, written to the pool
          together with v (pa_rope_write_kv)
  copy    copies of physical blocks over all layers (pa_copy_blocks)
"""
import math

import torch

own = False

E4M3_MAX = 448.0

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _window(name, q_heads, kv_heads, head_dim, block_size, kv, chunks, chunk_len, decodes, specs,
            ctx_lo, ctx_hi, window, sinks):
    return {"name": name, "op": "window", "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "block_size": block_size, "kv": kv, "chunks": chunks,
            "chunk_len": chunk_len, "decodes": decodes, "specs": specs, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "window": window, "sinks": sinks}


def _rope(name, tokens, q_heads, kv_heads, head_dim, rot_dim, block_size, kv, axes, assign,
          adjacent, max_pos, padded):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "rot_dim": rot_dim,
            "block_size": block_size, "kv": kv, "axes": axes, "assign": assign,
            "adjacent": adjacent, "max_pos": max_pos, "padded": padded}


def _copy(name, layers, kv_heads, block_size, head_dim, kv, pairs, repeat, padded):
    return {"name": name, "op": "copy", "layers": layers, "kv_heads": kv_heads,
            "block_size": block_size, "head_dim": head_dim, "kv": kv, "pairs": pairs,
            "repeat": repeat, "padded": padded}


def listed():
    return [
        # one stream of a small model: nothing but latency
        _window("window_one_stream", 4, 2, 64, 16, "bf16", 0, 0, 1, 0, 700, 700, 128, 4),
        # a batch of long-lived streams, one new token each, contexts far past the window
        _window("window_decode", 32, 8, 128, 16, "bf16", 0, 0, 64, 0, 2048, 32768, 1024, 4),
        # a large decode batch on a quantised pool, many contexts shorter than the window
        _window("window_decode_e4m3", 32, 8, 128, 16, "e4m3", 0, 0, 256, 0, 512, 8192, 4096, 64),
        # speculative verification, odd window and sinks, 64-wide heads
        _window("window_verify", 8, 2, 64, 32, "bf16", 0, 0, 0, 24, 100, 1500, 333, 7),
        # a continuous-batching step: prompt chunks, decode rows and verify rows together
        _window("window_mixed", 32, 8, 128, 16, "bf16", 8, 512, 192, 32, 0, 8192, 1024, 4),
        # long prompts in large chunks
        _window("window_prefill", 32, 8, 128, 16, "bf16", 2, 4096, 0, 0, 0, 28672, 4096, 16),
        # a small decode step: latency
        _rope("rope_decode", 8, 32, 8, 128, 128, 16, "bf16", 1, "blocks", False, 8192, 0),
        # a prompt chunk of text and images, three axes
        _rope("rope_image", 4096, 32, 8, 128, 128, 16, "bf16", 3, "blocks", False, 32768, 17),
        # video prompts into a quantised pool, half of each head rotated, axes taken in turn
        _rope("rope_video_e4m3", 16384, 32, 8, 128, 64, 16, "e4m3", 3, "cycle", True, 131072, 0),
        # copy-on-write of a few forked requests in one layer
        _copy("copy_fork", 1, 8, 16, 128, "bf16", 4, False, 0),
        # beams forked in every layer, several copies of one block among them
        _copy("copy_beams", 32, 8, 16, 128, "bf16", 61, True, 3),
        # compaction of a pool: thousands of blocks to its lower end
        _copy("copy_compact", 8, 8, 32, 128, "e4m3", 2048, False, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "rope", "copy"])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    head_dim = 128 if kv == "e4m3" else rng.choice([64, 128, 128])
    block_size = rng.choice([16, 16, 32, 64])
    if op == "window":
        q_heads, kv_heads = rng.choice([(4, 2), (8, 2), (32, 8), (16, 1), (14, 2), (6, 6), (32, 8)])
        shape = rng.choice(["decode", "verify", "mixed", "prefill"])
        chunks = decodes = specs = chunk_len = 0
        if shape == "decode":
            decodes = _log(rng, 1, 256)
        elif shape == "verify":
            specs = _log(rng, 1, 64)
        elif shape == "mixed":
            chunks, chunk_len = rng.randint(1, 4), _log(rng, 17, 1024)
            decodes, specs = _log(rng, 1, 128), _log(rng, 1, 32)
        else:
            chunks, chunk_len = rng.randint(1, 3), _log(rng, 100, 2048)
        lo = _log(rng, 1, 4096)
        case = _window("", q_heads, kv_heads, head_dim, block_size, kv, chunks, chunk_len, decodes,
                       specs, lo, lo + _log(rng, 1, 16384), _log(rng, 1, 4096),
                       rng.choice([0, 1, 4, _log(rng, 1, 256)]))
    elif op == "rope":
        q_heads, kv_heads = rng.choice([(4, 2), (8, 2), (32, 8), (16, 1), (14, 2), (6, 6)])
        rot_dim = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4, 48])
        tokens = _log(rng, 1, 12000)
        case = _rope("", tokens, q_heads, kv_heads, head_dim, rot_dim, block_size, kv,
                     rng.choice([1, 2, 3, 3]), rng.choice(["blocks", "cycle"]),
                     rng.choice([False, True]), _log(rng, 64, 1 << 20),
                     rng.choice([0, tokens // 7]))
    else:
        pairs = _log(rng, 1, 512)
        case = _copy("", _log(rng, 1, 40), rng.choice([1, 2, 6, 8]), block_size, head_dim, kv,
                     pairs, rng.choice([False, True]), rng.choice([0, pairs // 5]))
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _requests(case):
    """(context length, new tokens) of every request; the lengths are spread over
    [ctx_lo, ctx_hi] the same way for every seed."""
    n = ([case["chunk_len"]] * case["chunks"] + [1] * case["decodes"] + [5] * case["specs"])
    span = case["ctx_hi"] - case["ctx_lo"]
    return [(case["ctx_lo"] + int(span * ((0.381966 * (i + 1) * (i + 1)) % 1.0)), k)
            for i, k in enumerate(n)]


def _visible_blocks(case, ctx, n):
    """Logical blocks of a request that some row of it sees: those of the sinks, and
    those from the first row's window on."""
    bs = case["block_size"]
    end = -(-(ctx + n) // bs)
    first = max(0, ctx - case["window"] + 1) // bs
    sink = min(end, -(-case["sinks"] // bs))
    return list(range(min(sink, first))) + list(range(first, end))


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


def _prepare_window(case, gen, dev):
    reqs = _requests(case)
    bs, hkv, hq, d = case["block_size"], case["kv_heads"], case["q_heads"], case["head_dim"]
    group = hq // hkv
    lists = [_visible_blocks(case, c, n) for c, n in reqs]
    used = sum(len(x) for x in lists)
    num_blocks = used + used // 10 + 1
    perm = torch.randperm(num_blocks, generator=gen, device=dev)[:used].to(torch.int32)
    width = max(-(-(c + n) // bs) for c, n in reqs)
    # blocks that fell out of every window have been given back: -1 in the table
    table = torch.full((len(reqs), width), -1, dtype=torch.int32, device=dev)
    rows = torch.tensor([b for b, x in enumerate(lists) for _ in x], device=dev)
    cols = torch.tensor([j for x in lists for j in x], device=dev)
    table[rows, cols] = perm
    starts = [0]
    for _, n in reqs:
        starts.append(starts[-1] + n)
    total = starts[-1]
    i32 = dict(dtype=torch.int32, device=dev)
    shape = (num_blocks, hkv, bs, d)
    fp8 = case["kv"] == "e4m3"
    st = {"case": case, "scale": 1.0 / math.sqrt(d), "table": table,
          "qsl": torch.tensor(starts, **i32), "ctx": torch.tensor([c for c, _ in reqs], **i32),
          "seq": torch.tensor([c + n for c, n in reqs], **i32),
          "q": torch.randn((total, hq, d), generator=gen, device=dev).to(torch.bfloat16),
          "k": _pool(gen, shape, case["kv"], dev), "v": _pool(gen, shape, case["kv"], dev),
          "k_scale": _scales(gen, hkv, dev) if fp8 else None,
          "v_scale": _scales(gen, hkv, dev) if fp8 else None,
          "out": torch.zeros((total, hq, d), dtype=torch.bfloat16, device=dev),
          "lse": torch.zeros((total, hq), device=dev), "workspace": None,
          # blocks of requests with more than 64 query rows per kv head (a quantised
          # pool's bf16 staging room)
          "staging": sum(len(x) for x, (_, n) in zip(lists, reqs) if n * group > 64) if fp8 else 0}
    # The plain form's tiles: `tile` consecutive query tokens of one request
    tile = min(128 if not case["decodes"] + case["specs"] else 16, max(n for _, n in reqs))
    tiles = [(b, i) for b, (_, n) in enumerate(reqs) for i in range(0, n, tile)]
    st["tile"] = tile
    st["tile_req"] = torch.tensor([b for b, _ in tiles], device=dev)
    st["tile_first"] = torch.tensor([i for _, i in tiles], device=dev)
    return st


def _axis_of(case, dev):
    """Which axis each frequency takes its position from: consecutive runs, or the
    axes in turn."""
    half, axes = case["rot_dim"] // 2, case["axes"]
    i = torch.arange(half, device=dev)
    if case["assign"] == "cycle":
        return (i % axes).to(torch.int32)
    return torch.clamp(i * axes // half, max=axes - 1).to(torch.int32)


def _prepare_rope(case, gen, dev):
    t, hq, hkv, d, bs = (case[x] for x in ("tokens", "q_heads", "kv_heads", "head_dim",
                                           "block_size"))
    num_blocks = -(-t // bs) + 2 + t // (8 * bs)
    fp8 = case["kv"] == "e4m3"
    # rows of the fused projection: q, k and v of a token next to each other
    qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=gen, device=dev).to(torch.bfloat16)
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
    slots = torch.randperm(num_blocks * bs, generator=gen, device=dev)[:t]
    if case["padded"]:
        slots[t - case["padded"]:] = -1
    base = torch.randint(0, case["max_pos"], (1,), generator=gen, device=dev)
    i = torch.arange(t, device=dev)
    if case["axes"] == 1:
        pos = (base + i)[None]
    else:  # frames of 16 rows of 24 patches each
        pos = torch.stack([base + i // 384, base + i // 24 % 16, base + i % 24][-case["axes"]:])
    shape = (num_blocks + 1, hkv, bs, d)  # the last block takes the plain form's padding rows
    half = case["rot_dim"] // 2
    kc, vc = _pool(gen, shape, case["kv"], dev), _pool(gen, shape, case["kv"], dev)
    return {"case": case, "q": q.view(t, hq, d), "k": k.view(t, hkv, d), "v": v.view(t, hkv, d),
            "pos": pos.to(torch.int32).contiguous(), "axis": _axis_of(case, dev), "slots": slots,
            "inv_freq": 1e4 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half),
            "whole": (kc, vc), "kc": kc[:num_blocks], "vc": vc[:num_blocks],
            "k_scale": _scales(gen, hkv, dev) if fp8 else None,
            "v_scale": _scales(gen, hkv, dev) if fp8 else None,
            "q_out": torch.zeros((t, hq, d), dtype=torch.bfloat16, device=dev)}


def _prepare_copy(case, gen, dev):
    pairs = case["pairs"]
    num_blocks = 2 * pairs + pairs // 4 + 2
    perm = torch.randperm(num_blocks - 1, generator=gen, device=dev)
    src = perm[:pairs].clone()
    if case["repeat"]:
        src = src[torch.randint(0, pairs, (pairs,), generator=gen, device=dev)]
    both = torch.stack([src, perm[pairs:2 * pairs]], dim=1).to(torch.int32)
    if case["padded"]:
        both[pairs - case["padded"]:] = -1
    shape = (case["layers"], num_blocks, case["kv_heads"], case["block_size"], case["head_dim"])
    # the pool's last block is not a user's: it takes the plain form's padding pairs
    return {"case": case, "pairs": both.contiguous(), "k": _pool(gen, shape, case["kv"], dev),
            "v": _pool(gen, shape, case["kv"], dev), "layers": None}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    return {"window": _prepare_window, "rope": _prepare_rope,
            "copy": _prepare_copy}[case["op"]](case, gen, dev)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _gather(pool, blocks, offsets, scale):
    """Rows (block, offset) of every kv head in 32 bits: [tiles, kv heads, keys, d]."""
    raw = pool if scale is None else pool.view(torch.uint8)
    x = raw[blocks, :, offsets]
    x = x.float() if scale is None else x.view(torch.float8_e4m3fn).float() * scale[:, None]
    return x.transpose(1, 2)


def _run_window(st):
    case, q = st["case"], st["q"]
    bs, hkv, window, sinks = (case[x] for x in ("block_size", "kv_heads", "window", "sinks"))
    dev, (total, hq, d) = q.device, q.shape
    group, tile = hq // hkv, st["tile"]
    req, first = st["tile_req"], st["tile_first"]
    ctx, seq, start = st["ctx"][req].long(), st["seq"][req].long(), st["qsl"][req].long()
    i = first[:, None] + torch.arange(tile, device=dev)          # token within the request
    pos = ctx[:, None] + i
    valid = pos < seq[:, None]
    token = torch.where(valid, start[:, None] + i, total)
    # keys of a tile: the sinks, then the union of its rows' windows
    width = st["table"].shape[1] * bs
    span = min(window + tile - 1, width)
    lo = (ctx + first - window + 1).clamp(min=0)
    sink_keys = torch.arange(min(sinks, width), device=dev).expand(req.numel(), -1)
    win_keys = lo[:, None] + torch.arange(span, device=dev)
    keys = torch.cat([sink_keys, win_keys], dim=1)
    once = torch.cat([sink_keys < seq[:, None], win_keys >= sinks], dim=1)
    p, j = pos[:, :, None], keys[:, None, :]
    seen = (j <= p) & ((j > p - window) | (j < sinks)) & (once & (keys < seq[:, None]))[:, None, :]
    col = (keys // bs).clamp(max=st["table"].shape[1] - 1)
    blocks = st["table"][req[:, None], col].clamp(min=0).long()
    k = _gather(st["k"], blocks, keys % bs, st["k_scale"])
    v = _gather(st["v"], blocks, keys % bs, st["v_scale"])
    qt = q[token.clamp(max=total - 1)].float().view(-1, tile, hkv, group, d)
    qt = qt.permute(0, 2, 1, 3, 4).reshape(-1, hkv, tile * group, d)
    s = (qt @ k.transpose(2, 3)).view(-1, hkv, tile, group, keys.shape[1]) * st["scale"]
    s = s.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    m = s.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    e = (s - m).exp_()
    z = e.sum(dim=-1, keepdim=True).clamp(min=1e-37)
    o = (e.view(-1, hkv, tile * group, keys.shape[1]) @ v).view(-1, hkv, tile, group, d) / z
    lse = (m + z.log()).squeeze(-1)
    out = q.new_empty((total + 1, hq, d))
    out[token] = o.permute(0, 2, 1, 3, 4).reshape(-1, tile, hq, d).to(torch.bfloat16)
    out_lse = lse.new_empty((total + 1, hq))
    out_lse[token] = lse.permute(0, 2, 1, 3).reshape(-1, tile, hq)
    return {"out": out[:total], "lse": out_lse[:total]}


def _rotate(x, cos, sin, rot_dim, adjacent):
    x = x.float()
    r = x[..., :rot_dim]
    if adjacent:
        a, b = r[..., 0::2], r[..., 1::2]
    else:
        a, b = r[..., :rot_dim // 2], r[..., rot_dim // 2:]
    pair = [a * cos - b * sin, b * cos + a * sin]
    r = torch.stack(pair, dim=-1).flatten(-2) if adjacent else torch.cat(pair, dim=-1)
    return torch.cat([r, x[..., rot_dim:]], dim=-1)


def _store(cache, rows, slots, scale):
    bs = cache.shape[2]
    blocks = torch.where(slots < 0, cache.shape[0] - 1, slots // bs)
    if scale is None:
        cache[blocks, :, slots % bs] = rows.to(torch.bfloat16)
    else:
        codes = (rows / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        cache.view(torch.uint8)[blocks, :, slots % bs] = codes.view(torch.uint8)


def _run_rope(st):
    case = st["case"]
    # far positions: the angle in 64 bits
    angle = st["pos"][st["axis"].long()].double().T * st["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    how = (cos, sin, case["rot_dim"], case["adjacent"])
    st["q_out"].copy_(_rotate(st["q"], *how))
    _store(st["whole"][0], _rotate(st["k"], *how), st["slots"], st["k_scale"])
    _store(st["whole"][1], st["v"].float(), st["slots"], st["v_scale"])
    return {"q": st["q_out"], "k": st["kc"], "v": st["vc"]}


def _run_copy(st):
    pairs = st["pairs"].long() % st["k"].shape[1]  # a padding pair copies the last block to itself
    src, dst = pairs[:, 0], pairs[:, 1]
    k, v = (x if st["case"]["kv"] == "bf16" else x.view(torch.uint8) for x in (st["k"], st["v"]))
    k[:, dst] = k[:, src]
    v[:, dst] = v[:, src]
    return {"k": st["k"], "v": st["v"]}


def _own_window(st):
    import paged_kv_cache_284_gb300 as pk
    st["workspace"] = pk.pa_window_attention(
        st["q"], st["k"], st["v"], st["table"], st["qsl"], st["ctx"], st["seq"], st["scale"],
        st["case"]["window"], st["case"]["sinks"], st["out"], st["lse"],
        workspace=st["workspace"], k_scale=st["k_scale"], v_scale=st["v_scale"],
        staging_blocks=st["staging"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_rope(st):
    import paged_kv_cache_284_gb300 as pk
    pk.pa_rope_write_kv(st["q"], st["k"], st["v"], st["pos"], st["inv_freq"], st["axis"],
                        st["slots"], st["kc"], st["vc"], st["q_out"],
                        adjacent=st["case"]["adjacent"], k_scale=st["k_scale"],
                        v_scale=st["v_scale"])
    return {"q": st["q_out"], "k": st["kc"], "v": st["vc"]}


def _own_copy(st):
    import paged_kv_cache_284_gb300 as pk
    if st["layers"] is None:
        st["layers"] = pk.kv_layers(list(st["k"]), list(st["v"]))
    pk.pa_copy_blocks(st["layers"], st["pairs"])
    return {"k": st["k"], "v": st["v"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"window": _own_window, "rope": _own_rope, "copy": _own_copy}[op](state)
    return {"window": _run_window, "rope": _run_rope, "copy": _run_copy}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    hkv, d = case["kv_heads"], case["head_dim"]
    elem = 2 if case["kv"] == "bf16" else 1
    if case["op"] == "window":
        hq, window, sinks = case["q_heads"], case["window"], case["sinks"]
        keys = pairs = tokens = entries = 0
        for c, n in _requests(case):
            first = max(0, c - window + 1)  # the first row's window
            keys += c + n - first + min(sinks, first)
            entries += len(_visible_blocks(case, c, n))
            tokens += n
            for i in range(n):
                f = max(0, c + i - window + 1)
                pairs += c + i + 1 - f + min(sinks, f)
        return {"bytes": 2 * keys * hkv * d * elem + tokens * hq * (4 * d + 4) + 4 * entries,
                "flops": 4 * pairs * hq * d}
    if case["op"] == "rope":
        t, hq, stored = case["tokens"], case["q_heads"], case["tokens"] - case["padded"]
        return {"bytes": t * hq * d * 4 + stored * 2 * hkv * d * (2 + elem)
                + t * (8 + 4 * case["axes"]),
                "flops": 3 * case["rot_dim"] * (t * hq + stored * hkv)}
    block = hkv * case["block_size"] * d * elem
    return {"bytes": 4 * block * case["layers"] * (case["pairs"] - case["padded"])
            + 8 * case["pairs"], "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_window(case, st):
    total, hq, d = st["q"].shape
    hkv, bs = case["kv_heads"], case["block_size"]
    group = hq // hkv
    dev = st["q"].device
    out = torch.zeros((total, hq, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((total, hq), dtype=torch.float64, device=dev)
    at = 0
    for b, (c, n) in enumerate(_requests(case)):
        j = torch.arange(c + n, device=dev)
        j = j[(j < case["sinks"]) | (j >= c - case["window"] + 1)]
        rows = st["table"][b].long()[j // bs]
        k, v = (st[x].view(torch.uint8 if st["k_scale"] is not None else torch.bfloat16)
                [rows, :, j % bs] for x in ("k", "v"))
        if st["k_scale"] is not None:
            k, v = (x.view(torch.float8_e4m3fn).double() * st[s].double()[:, None]
                    for x, s in ((k, "k_scale"), (v, "v_scale")))
        k, v = k.double().permute(1, 0, 2), v.double().permute(1, 0, 2)      # [hkv, keys, d]
        for r in range(0, n, 1024):
            m = min(1024, n - r)
            p = c + torch.arange(r, r + m, device=dev)[:, None]
            hidden = (j > p) | ((j <= p - case["window"]) & (j >= case["sinks"]))
            for h in range(hkv):
                x = st["q"][at + r:at + r + m, h * group:(h + 1) * group].double()
                s = torch.einsum("tgd,kd->gtk", x, k[h]) * st["scale"]
                s[:, hidden] = float("-inf")
                z = torch.logsumexp(s, dim=-1)
                lse[at + r:at + r + m, h * group:(h + 1) * group] = z.T
                out[at + r:at + r + m, h * group:(h + 1) * group] = torch.einsum(
                    "gtk,kd->tgd", (s - z[..., None]).exp_(), v[h])
        at += n
    return {"out": out, "lse": lse}


def _exact_rope(case, st):
    rd = case["rot_dim"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=st["q"].device),
                       st["inv_freq"] * st["pos"].double().T[:, st["axis"].long()])[:, None]

    def rotated(x):
        x = x.double()
        r = x[..., :rd]
        pairs = (r.unflatten(-1, (rd // 2, 2)) if case["adjacent"]
                 else r.unflatten(-1, (2, rd // 2)).transpose(-1, -2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        x[..., :rd] = (z if case["adjacent"] else z.transpose(-1, -2)).flatten(-2)
        return x

    live = st["slots"] >= 0
    slots, caches = st["slots"][live], []
    for cache, rows, scale in ((st["kc"], rotated(st["k"]), st["k_scale"]),
                               (st["vc"], st["v"].double(), st["v_scale"])):
        whole = cache.double()
        if scale is not None:
            rows = (rows / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        whole[slots // case["block_size"], :, slots % case["block_size"]] = rows[live]
        caches.append(whole)
    return {"q": rotated(st["q"]), "k": caches[0], "v": caches[1]}


def _exact_copy(case, st):
    found = {}
    live = st["pairs"][st["pairs"][:, 0] >= 0].long()
    for name in ("k", "v"):
        old = st[name]
        new = old.double()
        for layer in range(case["layers"]):
            new[layer].index_copy_(0, live[:, 1], old[layer].double().index_select(0, live[:, 0]))
        found[name] = new
    return found


def exact(case, seed):
    st = prepare(case, seed)
    return {"window": _exact_window, "rope": _exact_rope, "copy": _exact_copy}[case["op"]](case, st)
