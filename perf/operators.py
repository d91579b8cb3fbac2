"""Cases of the positional, cache-appending and shared-prefix operators, with their plain forms.

Three operators of one decode step over a paged cache:

  rope    rotary positions on a [T, H, d] tensor
  append  new keys (rotated on the way) and values into a paged cache, queries rotated beside them
  prefix  selective decode over a paged cache whose first keys all rows share

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits (angles in 64), rounded once at the end; with ``own`` true it makes the
calls of ``head_sparse_decode_b200``.
"""
import math

import torch

own = False

DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one sequence, one token: the latency of a single rotation (LLaMA-2-7B-shaped heads)
        dict(name="rope_token", op="rope", T=1, H=32, d=128, rotary=128, interleaved=False,
             dtype="fp16", base=10000.0, scaling="none", max_pos=4096, fused=False),
        # a prefill chunk of queries inside a fused projection (LLaMA-3.1-70B-shaped heads, 128K positions)
        dict(name="rope_chunk", op="rope", T=8192, H=64, d=128, rotary=128, interleaved=False,
             dtype="bf16", base=500000.0, scaling="bands", max_pos=131072, fused=True),
        # an odd ragged chunk, part of each head rotated, neighbouring pairs
        dict(name="rope_partial", op="rope", T=1001, H=9, d=64, rotary=24, interleaved=True,
             dtype="fp16", base=10000.0, scaling="linear", max_pos=16384, fused=True),
        # one sequence's decode step: one token appended
        dict(name="append_token", op="append", B=1, T=1, H_q=32, H_kv=32, d=128, rotary=128,
             interleaved=False, dtype="fp16", base=10000.0, scaling="none", page_size=16, ctx=2048),
        # a decode batch: one token for each of 32 sequences (LLaMA-3.1-70B-shaped heads)
        dict(name="append_batch", op="append", B=32, T=32, H_q=64, H_kv=8, d=128, rotary=128,
             interleaved=False, dtype="bf16", base=500000.0, scaling="bands", page_size=16,
             ctx=4096),
        # a chunk of ragged prompts behind what their rows already hold
        dict(name="append_prompts", op="append", B=5, T=6001, H_q=64, H_kv=8, d=128, rotary=128,
             interleaved=False, dtype="bf16", base=500000.0, scaling="yarn", page_size=64,
             ctx=4096),
        # two rows behind a short shared prompt: the smallest call
        dict(name="prefix_small", op="prefix", B=2, H_q=4, H_kv=4, d=64, top_k=2, prefix=100,
             suffix=28, page_size=8, dtype="fp16", index="perm"),
        # odd everything: groups of three, a prefix that ends inside a page and a tile
        dict(name="prefix_odd", op="prefix", B=7, H_q=24, H_kv=8, d=64, top_k=5, prefix=1333,
             suffix=77, page_size=16, dtype="bf16", index="perm"),
        # grouped queries, a system prompt of 4K tokens before each row's own turn
        dict(name="prefix_groups", op="prefix", B=32, H_q=64, H_kv=8, d=128, top_k=5, prefix=4096,
             suffix=512, page_size=16, dtype="bf16", index="perm"),
        # many samples over one long document: the tensor cores' case
        dict(name="prefix_document", op="prefix", B=64, H_q=64, H_kv=8, d=128, top_k=5,
             prefix=16384, suffix=1024, page_size=64, dtype="bf16", index="perm"),
        # multi-head decode at 30 % of the heads (OPT-66B-shaped), a few-shot prompt shared
        dict(name="prefix_heads", op="prefix", B=64, H_q=72, H_kv=72, d=128, top_k=22, prefix=1920,
             suffix=256, page_size=16, dtype="fp16", index="perm"),
        # popular heads taken by most rows, others by few (LLaMA-2-7B-shaped)
        dict(name="prefix_popular", op="prefix", B=128, H_q=32, H_kv=32, d=128, top_k=16,
             prefix=2048, suffix=200, page_size=128, dtype="fp16", index="zipf"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "prefix", "prefix"])
    dtype = rng.choice(["fp16", "bf16"])
    while True:
        if op == "rope":
            d = rng.choice([64, 128])
            rotary = rng.choice([d, d, d // 2, 24, 2 * rng.randint(1, d // 2)])
            case = dict(op="rope", T=_log_int(rng, 1, 8192), H=_log_int(rng, 1, 72), d=d,
                        rotary=rotary, interleaved=rng.random() < 0.5, dtype=dtype,
                        base=rng.choice([10000.0, 500000.0]),
                        scaling=rng.choice(["none", "linear", "bands", "yarn"]),
                        max_pos=_log_int(rng, 512, 1 << 20), fused=rng.random() < 0.5)
            most = _work_rope(listed()[1])
        elif op == "append":
            H_q, H_kv, d = rng.choice([(32, 32, 128), (64, 8, 128), (72, 72, 128), (24, 8, 64),
                                       (4, 4, 64)])
            B = _log_int(rng, 1, 64)
            ctx = _log_int(rng, 64, 4096)
            T = B if rng.random() < 0.5 else _log_int(rng, 1, 6000)
            case = dict(op="append", B=B, T=min(T, B * ctx // 2) if T != B else B, H_q=H_q,
                        H_kv=H_kv, d=d, rotary=rng.choice([d, d, d // 2]),
                        interleaved=rng.random() < 0.5, dtype=dtype,
                        base=rng.choice([10000.0, 500000.0]),
                        scaling=rng.choice(["none", "linear", "bands", "yarn"]),
                        page_size=rng.choice([1, 8, 16, 24, 64, 128]), ctx=ctx)
            if case["B"] * ctx * H_kv * d > 1 << 27:      # the pool stays under 256 MiB a side
                continue
            most = _work_append(listed()[5])
        else:
            H_q, H_kv, d, top_k = rng.choice([(72, 72, 128, 22), (32, 32, 128, 16),
                                              (64, 8, 128, 5), (24, 8, 64, 5), (4, 4, 64, 2),
                                              (32, 4, 64, 3), (32, 2, 128, 1)])
            case = dict(op="prefix", B=_log_int(rng, 1, 128), H_q=H_q, H_kv=H_kv, d=d, top_k=top_k,
                        prefix=_log_int(rng, 1, 16384), suffix=_log_int(rng, 1, 1024),
                        page_size=rng.choice([8, 16, 32, 64, 128, 256]), dtype=dtype,
                        index=rng.choice(["perm", "zipf"]))
            tokens = case["prefix"] + case["B"] * case["suffix"]
            if tokens * H_kv * d > 1 << 29 or \
                    case["B"] * H_q * (case["prefix"] + case["suffix"]) > 1 << 29:
                continue
            most = _work_prefix(listed()[9])
        mine = work(case)
        if mine["bytes"] <= most["bytes"] and mine["flops"] <= most["flops"]:
            return case


# ---------------------------------------------------------------- work

def _work_rope(c):
    elems = c["T"] * c["H"] * c["d"]
    return {"bytes": 4 * elems + 4 * c["T"] + 4 * c["rotary"],
            "flops": 3 * c["T"] * c["H"] * c["rotary"]}


def _work_append(c):
    heads = c["H_q"] + 2 * c["H_kv"]
    return {"bytes": 4 * c["T"] * heads * c["d"] + 12 * c["T"] + 4 * c["rotary"],
            "flops": 3 * c["T"] * (c["H_q"] + c["H_kv"]) * c["rotary"]}


def _suffix_lengths(c):
    """Own keys of each row: fixed by the case, from 0 to suffix, the last row full."""
    B, S = c["B"], c["suffix"]
    return [S if b == B - 1 else (b * 7919 + 31) % (S + 1) for b in range(B)]


def _work_prefix(c):
    G = c["H_q"] // c["H_kv"]
    units = c["B"] * c["top_k"]
    own_keys = sum(_suffix_lengths(c)) * c["top_k"]
    heads = min(c["H_kv"], units)             # heads that any row selects, at most
    return {"bytes": 4 * c["d"] * (heads * c["prefix"] + own_keys) + 4 * units * G * c["d"]
            + 4 * units,
            "flops": 4 * G * c["d"] * (units * c["prefix"] + own_keys)}


def work(case):
    return {"rope": _work_rope, "append": _work_append, "prefix": _work_prefix}[case["op"]](case)


# ---------------------------------------------------------------- inputs

def _frequencies(c):
    """Radians per position of each pair (64 bits) and the factor on cos and sin."""
    r, base = c["rotary"], c["base"]
    freq = torch.tensor([base ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64)
    if c["scaling"] == "linear":
        return freq / 4.0, 1.0
    if c["scaling"] == "bands":
        # long wavelengths stretched by 8, short ones kept, a ramp between, for a trained length of 8192
        turns = 8192.0 * freq / (2.0 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return freq * keep + freq / 8.0 * (1.0 - keep), 1.0
    if c["scaling"] == "yarn":
        turns = 4096.0 * freq / (2.0 * math.pi)
        pair = lambda n: r * math.log(4096.0 / (n * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), r - 1)
        ramp = ((torch.arange(len(turns), dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return freq * (1.0 - ramp) + freq / 4.0 * ramp, 0.1 * math.log(4.0) + 1.0
    return freq, 1.0


def _gpu_generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _prepare_rope(c, seed):
    g = _gpu_generator(seed)
    heads = c["H"] + 8 if c["fused"] else c["H"]           # queries inside a fused projection's rows
    x = _randn((c["T"], heads, c["d"]), g, DTYPE[c["dtype"]])[:, :c["H"]]
    pos = torch.randint(0, c["max_pos"], (c["T"],), generator=g, device="cuda", dtype=torch.int32)
    freq, mscale = _frequencies(c)
    return dict(case=c, x=x, pos=pos, freq=freq.cuda(), mscale=mscale)


def _prepare_append(c, seed):
    g, dt = _gpu_generator(seed), DTYPE[c["dtype"]]
    B, T, ps = c["B"], c["T"], c["page_size"]
    pages = -(-c["ctx"] // ps)
    qkv = _randn((T, c["H_q"] + 2 * c["H_kv"], c["d"]), g, dt)
    q, k, v = qkv.split([c["H_q"], c["H_kv"], c["H_kv"]], dim=1)
    k_pages = _randn((B * pages, c["H_kv"], ps, c["d"]), g, dt)
    v_pages = _randn((B * pages, c["H_kv"], ps, c["d"]), g, dt)
    gc = torch.Generator().manual_seed(seed)
    table = torch.randperm(B * pages, generator=gc).reshape(B, pages).to(torch.int32).cuda()
    if T == B:                                             # a decode step: one token a row
        rows = None
        pos = torch.randint(0, c["ctx"], (B,), generator=gc, dtype=torch.int32)
    else:                                                  # prompts: T tokens over the rows, behind a past
        share = [T // B + (1 if b < T % B else 0) for b in range(B)]
        past = [int(torch.randint(0, c["ctx"] - n + 1, (1,), generator=gc)) for n in share]
        rows = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(share)]).cuda()
        pos = torch.cat([torch.arange(p, p + n, dtype=torch.int32) for p, n in zip(past, share)])
    freq, mscale = _frequencies(c)
    return dict(case=c, q=q, k=k, v=v, k_pages=k_pages, v_pages=v_pages, table=table, rows=rows,
                pos=pos.cuda(), freq=freq.cuda(), mscale=mscale)


def _index(c, gc):
    B, H, k = c["B"], c["H_kv"], c["top_k"]
    if c["index"] == "zipf":
        weights = (1.0 / torch.arange(1, H + 1, dtype=torch.float64))[torch.randperm(H, generator=gc)]
        return torch.multinomial(weights.expand(B, H), k, generator=gc).to(torch.int32)
    return torch.rand((B, H), generator=gc).argsort(dim=1)[:, :k].to(torch.int32).contiguous()


def _prepare_prefix(c, seed):
    g, dt = _gpu_generator(seed), DTYPE[c["dtype"]]
    gc = torch.Generator().manual_seed(seed)
    B, P, ps, d = c["B"], c["prefix"], c["page_size"], c["d"]
    first = P // ps                                        # each row's own pages begin here
    shared = -(-P // ps)
    mine = -(-(P + c["suffix"]) // ps) - first
    n = shared + B * mine
    k_pages = _randn((n, c["H_kv"], ps, d), g, dt)
    v_pages = _randn((n, c["H_kv"], ps, d), g, dt)
    perm = torch.randperm(n, generator=gc).to(torch.int32)
    prefix_table = perm[:shared].contiguous()
    table = torch.cat([prefix_table[:first].expand(B, first), perm[shared:].reshape(B, mine)], dim=1)
    lens = torch.tensor([P + s for s in _suffix_lengths(c)], dtype=torch.int32)
    q = _randn((B, c["H_q"], d), g, dt)
    return dict(case=c, q=q, k_pages=k_pages, v_pages=v_pages, idx=_index(c, gc).cuda(),
                lens=lens.cuda(), table=table.contiguous().cuda(),
                prefix_table=prefix_table.cuda(), out=torch.zeros_like(q),
                scale=1.0 / math.sqrt(d))


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append,
            "prefix": _prepare_prefix}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms (32 bits, angles in 64)

def _rotate(x, pos, freq, mscale, interleaved):
    r = 2 * freq.numel()
    angle = pos.double()[:, None] * freq
    cos = (angle.cos() * mscale).float()[:, None]
    sin = (angle.sin() * mscale).float()[:, None]
    x32 = x.float()
    a, b = (x32[..., 0:r:2], x32[..., 1:r:2]) if interleaved \
        else (x32[..., :r // 2], x32[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack([y, z], dim=-1).flatten(-2) if interleaved else torch.cat([y, z], dim=-1)
    return torch.cat([rot, x32[..., r:]], dim=-1).to(x.dtype)


def _plain_append(s):
    c = s["case"]
    pos = s["pos"].long()
    rows = s["rows"].long() if s["rows"] is not None else torch.arange(c["T"], device=pos.device)
    page = s["table"][rows, pos // c["page_size"]].long()
    off = pos % c["page_size"]
    s["k_pages"][page, :, off] = _rotate(s["k"], s["pos"], s["freq"], s["mscale"], c["interleaved"])
    s["v_pages"][page, :, off] = s["v"]
    return _rotate(s["q"], s["pos"], s["freq"], s["mscale"], c["interleaved"]), s["k_pages"], \
        s["v_pages"]


def _gather(pages, table, start, count):
    """Keys start .. start+count-1 of each row of the table, [rows, H_kv, count, d] in 32 bits."""
    ps = pages.shape[2]
    keys = torch.arange(start, start + count, device=pages.device)
    page = table[:, (keys // ps).clamp(max=table.shape[1] - 1)].long()
    return pages[page, :, (keys % ps)].permute(0, 2, 1, 3).float()


def _plain_prefix(s):
    c = s["case"]
    B, H_kv, d, P, S = c["B"], c["H_kv"], c["d"], c["prefix"], c["suffix"]
    G = c["H_q"] // H_kv
    q = s["q"].float().reshape(B, H_kv, G, d)
    kp = _gather(s["k_pages"], s["prefix_table"][None], 0, P)[0]
    vp = _gather(s["v_pages"], s["prefix_table"][None], 0, P)[0]
    ks = _gather(s["k_pages"], s["table"], P, S)
    vs = _gather(s["v_pages"], s["table"], P, S)
    by_head = q.permute(1, 0, 2, 3).reshape(H_kv, B * G, d)
    shared = (by_head @ kp.transpose(1, 2)).reshape(H_kv, B, G, P).permute(1, 0, 2, 3)
    mine = q @ ks.transpose(2, 3)
    beyond = torch.arange(P, P + S, device=q.device) >= s["lens"][:, None]
    mine = mine.masked_fill(beyond[:, None, None], -math.inf)
    top = torch.maximum(shared.amax(-1), mine.amax(-1))[..., None] * s["scale"]
    shared = torch.exp(shared * s["scale"] - top)
    mine = torch.exp(mine * s["scale"] - top)
    total = shared.sum(-1, keepdim=True) + mine.sum(-1, keepdim=True)
    flat = shared.permute(1, 0, 2, 3).reshape(H_kv, B * G, P)
    o = (flat @ vp).reshape(H_kv, B, G, d).permute(1, 0, 2, 3) + mine @ vs
    o = (o / total).to(s["q"].dtype)
    rows = torch.arange(B, device=q.device)[:, None]
    idx = s["idx"].long()
    s["out"].view(B, H_kv, G, d)[rows, idx] = o[rows, idx]
    return s["out"]


def _own(s):
    import head_sparse_decode_b200 as sha
    c = s["case"]
    if c["op"] == "rope":
        return sha.sha_rope(s["x"], s["pos"], s["freq"], interleaved=c["interleaved"],
                            mscale=s["mscale"])
    if c["op"] == "append":
        q = sha.sha_append_paged(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["pos"],
                                 rows=s["rows"], inv_freq=s["freq"], interleaved=c["interleaved"],
                                 mscale=s["mscale"], q=s["q"])
        return q, s["k_pages"], s["v_pages"]
    return sha.sha_decode_prefix(s["q"], s["k_pages"], s["v_pages"], s["idx"], s["lens"],
                                 s["table"], c["prefix"], s["prefix_table"], s["scale"], s["out"])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "rope":
        return _rotate(state["x"], state["pos"], state["freq"], state["mscale"], c["interleaved"])
    if c["op"] == "append":
        return _plain_append(state)
    return _plain_prefix(state)


# ---------------------------------------------------------------- in 64 bits, by the definitions

def _exact_rotation(x, pos, freq, mscale, interleaved):
    """Pairs as complex numbers, turned by exp(i * position * frequency)."""
    r = 2 * freq.numel()
    x64 = x.double()
    turn = torch.polar(torch.full((pos.numel(), freq.numel()), float(mscale), dtype=torch.float64,
                                  device=x.device), torch.outer(pos.double(), freq))
    if interleaved:
        z = torch.view_as_complex(x64[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous())
    else:
        z = torch.complex(x64[..., :r // 2].contiguous(), x64[..., r // 2:r].contiguous())
    z = torch.view_as_real(z * turn[:, None])
    y = x64.clone()
    y[..., :r] = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        return _exact_rotation(s["x"], s["pos"], s["freq"], s["mscale"], c["interleaved"])
    if c["op"] == "append":
        H_kv, ps = c["H_kv"], c["page_size"]
        rows = s["rows"].long() if s["rows"] is not None else torch.arange(c["T"]).cuda()
        pos = s["pos"].long()
        slot = s["table"][rows, torch.div(pos, ps, rounding_mode="floor")].long() * H_kv
        # flat row of [page, head, offset] for every token and head
        at = ((slot[:, None] + torch.arange(H_kv).cuda()) * ps + (pos % ps)[:, None]).reshape(-1)
        turned = _exact_rotation(s["k"], s["pos"], s["freq"], s["mscale"], c["interleaved"])
        pools = []
        for pool, new in ((s["k_pages"], turned), (s["v_pages"], s["v"].double())):
            flat = pool.double().reshape(-1, c["d"])
            pools.append(flat.index_copy(0, at, new.reshape(-1, c["d"])).reshape(pool.shape))
        return (_exact_rotation(s["q"], s["pos"], s["freq"], s["mscale"], c["interleaved"]),
                *pools)
    # every (row, selected head) by the definition, its keys walked through the tables
    G, ps = c["H_q"] // c["H_kv"], c["page_size"]
    P = c["prefix"]
    lens, idx = s["lens"].tolist(), s["idx"].tolist()
    n_shared = -(-P // ps)
    shared = s["prefix_table"].long()
    kp = s["k_pages"][shared].double().transpose(0, 1).reshape(c["H_kv"], n_shared * ps, -1)[:, :P]
    vp = s["v_pages"][shared].double().transpose(0, 1).reshape(c["H_kv"], n_shared * ps, -1)[:, :P]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        heads = torch.tensor(idx[b]).cuda()
        first = P // ps
        pages = s["table"][b, first:].long()
        ks, vs = (p[pages][:, heads].double().transpose(0, 1).reshape(len(heads), -1, c["d"])
                  [:, P - first * ps:lens[b] - first * ps] for p in (s["k_pages"], s["v_pages"]))
        k, v = torch.cat([kp[heads], ks], dim=1), torch.cat([vp[heads], vs], dim=1)
        q = s["q"][b].double().reshape(c["H_kv"], G, -1)[heads]
        w = torch.softmax(torch.bmm(q, k.transpose(1, 2)) * s["scale"], dim=-1)
        out[b].view(c["H_kv"], G, -1)[heads] = torch.bmm(w, v)
    return out
