"""The operators of an attention layer around the 8-bit paged cache: what is measured, in plain torch and through the library.

All take the tokens of a step one behind the other: token i of [n, heads, D] belongs to sequence b where
starts[b] <= i < starts[b + 1], and to slot lengths[b] + i - starts[b] of it (lengths: slots in use before the step).

  norm_rope   queries and keys are normed by head and rotated by their positions (one axis or several);
  append      keys and values are written to their slots in 8 bits, with a power of two for each 16 slots of a head;
  read        the values that a run of slots stands for;
  attend      the step's queries over the cache, each up to its own slot, within a window and the first slots if asked.
"""
import functools
import math

import numpy as np
import torch

own = False

BLOCK = 16                    # slots that share an exponent
LOWEST, HIGHEST = -120, 121   # exponents: code u stands for (u - 127.5) * 2^e
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One user, one token: the whole call is latency.
        dict(name="norm_rope_step_1", op="norm_rope", n=1, Hq=32, Hk=8, D=128, rot=128, axes=1, paired=False, weights=True, dtype="bf16"),
        # A prompt of a video, read from the layer's joint projection of queries, keys and values: positions in time, height and width.
        dict(name="norm_rope_video_8191", op="norm_rope", n=8191, Hq=32, Hk=8, D=128, rot=128, axes=3, paired=False, weights=True, dtype="bf16"),
        # One decode step of 64 conversations: each block may have to be shifted for its new row.
        dict(name="append_step_64", op="append", B=64, H=8, D=128, tokens=1, length=2049, page=64, dtype="bf16"),
        # A prompt of one sequence.
        dict(name="append_prompt_8192", op="append", B=1, H=8, D=128, tokens=8192, length=0, page=64, dtype="bf16"),
        # A short prefix on its way to another cache.
        dict(name="read_one_1021", op="read", B=1, H=8, D=128, tokens=1021, length=0, page=16, dtype="bf16"),
        # Odd stretches of several sequences, from the middle of a block on, in fp32.
        dict(name="read_f32_3x5001", op="read", B=3, H=8, D=128, tokens=5001, length=1021, page=64, dtype="f32"),
        # One user in the middle of a chat.
        dict(name="attend_one_1021", op="attend", B=1, H=8, G=4, D=128, tokens=1, length=1021, ragged=False, window=0, sinks=0, page=16, dtype="bf16"),
        # One long document: 8 heads have to fill the machine.
        dict(name="attend_long_131072", op="attend", B=1, H=8, G=4, D=128, tokens=1, length=131072, ragged=False, window=0, sinks=0, page=128, dtype="bf16"),
        # A full server.
        dict(name="attend_server_32x32768", op="attend", B=32, H=8, G=8, D=128, tokens=1, length=32768, ragged=False, window=0, sinks=0, page=64, dtype="bf16"),
        # Up to 5 drafted tokens of 16 sequences of all lengths, each token within a window and the first 4 slots.
        dict(name="attend_drafts_window_12345", op="attend", B=16, H=8, G=4, D=128, tokens=5, length=12345, ragged=True, window=4096, sinks=4, page=32, dtype="bf16"),
        # A piece of a long prompt, each token up to its own slot.
        dict(name="attend_prompt_1021_of_8192", op="attend", B=1, H=8, G=4, D=128, tokens=1021, length=8192, ragged=False, window=0, sinks=0, page=64, dtype="bf16"),
        # No grouping, fp32, narrow heads, ragged lengths.
        dict(name="attend_mha_f32_2049", op="attend", B=8, H=32, G=1, D=64, tokens=1, length=2049, ragged=True, window=0, sinks=0, page=16, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "read", "attend", "attend"))
    D, dtype = rng.choice((64, 128, 128)), rng.choice(("bf16", "bf16", "f32"))
    if op == "norm_rope":
        Hk = rng.choice((1, 2, 4, 8))
        Hq = Hk * rng.randint(1, 8)
        longest = 8192 * 40 * 128 * 2 // ((Hq + Hk) * D * (2 if dtype == "bf16" else 4))
        return dict(op=op, n=_log(rng, 1, min(16384, longest)), Hq=Hq, Hk=Hk, D=D, rot=rng.choice((D, D, D // 2)), axes=rng.choice((1, 1, 2, 3)),
                    paired=rng.random() < 0.4, weights=rng.random() < 0.8, dtype=dtype)
    B, H = _log(rng, 1, 64), rng.choice((1, 2, 4, 8, 16))
    common = dict(op=op, B=B, H=H, D=D, page=rng.choice((16, 32, 64, 128, 256)), dtype=dtype)
    if op != "attend":
        return dict(common, tokens=_log(rng, 1, max(1, 8192 * 8 // (B * H))), length=rng.choice((0, _log(rng, 1, 4097))))
    G = rng.randint(1, 8)
    length = _log(rng, 1, min(131072, 4194304 // (B * H)))
    # one token, a few drafted ones, or a piece of a prompt
    most = 32 * 1021 * 8192 * 128 // (B * H * G * length * D)
    tokens = max(1, min(rng.choice((1, 1, rng.randint(2, 9), _log(rng, 10, 1024))), length, most))
    window = rng.choice((0, 0, _log(rng, 1, length)))
    return dict(common, G=G, tokens=tokens, length=length, ragged=rng.random() < 0.6, window=window,
                sinks=rng.choice((0, rng.randint(1, 64))) if window else 0)


def _counts(case):
    """Tokens of each sequence in this step, and slots in use before it."""
    B, T, L = case["B"], case["tokens"], case["length"]
    if case["op"] != "attend":
        # odd places in a block, another one for each sequence
        return [T] * B, [L + 5 * b if L else 0 for b in range(B)]
    if not case["ragged"]:
        return [T] * B, [L - T] * B
    count = [1 + 7919 * b % T for b in range(B)]
    return count, [(L - T) * (b + 1) // B for b in range(B)]     # from a few slots to the longest


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    D = case["D"]
    if case["op"] == "norm_rope":
        rows = case["n"] * (case["Hq"] + case["Hk"])
        return {"bytes": rows * 2 * D * e + 4 * case["n"] * case["axes"], "flops": rows * (4 * D + 3 * case["rot"])}
    H = case["H"]
    count, before = _counts(case)
    if case["op"] != "attend":
        rows = sum(count) * H * 2
        return {"bytes": rows * (D * (e + 1) + 1 / BLOCK), "flops": 3 * rows * D}
    slots = pairs = 0
    for c, n in zip(count, before):
        far = [max(0, n + t + 1 - case["window"]) if case["window"] else 0 for t in range(c)]
        slots += n + c - max(0, far[0] - case["sinks"])
        pairs += sum(n + t + 1 - max(0, far[t] - case["sinks"]) for t in range(c))
    return {"bytes": H * (slots * 2 * (D + 1 / BLOCK) + 2 * sum(count) * case["G"] * D * e), "flops": 4 * pairs * H * case["G"] * D}


# ---------------------------------------------------------------- inputs

def _inv_freq(case):
    """Radians a position of each pair of coordinates, and the axis that turns it (blocks of pairs: time, height, width)."""
    pairs = case["rot"] // 2
    freq = 10000.0 ** (-np.arange(pairs, dtype=np.float64) / pairs)
    return freq, (np.arange(pairs) * case["axes"] // pairs).astype(np.int64)


def _exponents(most):
    """The least e with every |x| <= most below 2^(e + 7)."""
    e = torch.frexp(most.float())[1].to(torch.int32) - 7
    return torch.where(most > 0, e, torch.full_like(e, LOWEST)).clamp(LOWEST, HIGHEST)


@functools.lru_cache(maxsize=2)
def _pool(seed, D, dev):
    """Blocks of quantised rows: keys have a few large channels, values are of one scale."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    x = torch.randn(2, 2048, BLOCK, D, generator=gen, device=dev)
    x[0, :, :, [3, 17, D - 5]] *= 8.0
    x[1] *= torch.exp(0.4 * torch.randn(2048, 1, 1, generator=gen, device=dev))
    e = _exponents(x.abs().amax((-1, -2)))
    u = (torch.floor(x / torch.exp2(e.float())[..., None, None]) + 128).clamp(0, 255)
    return u.to(torch.uint8), e.to(torch.int8)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rs = np.random.default_rng(seed)
    dtype, D = DTYPES[case["dtype"]], case["D"]
    s = dict(op=case["op"])
    if case["op"] == "norm_rope":
        n, Hq, Hk = case["n"], case["Hq"], case["Hk"]
        x = torch.randn(n, (Hq + 2 * Hk) * D, generator=gen, device=dev) * torch.exp(torch.randn(n, 1, generator=gen, device=dev))
        x = x.to(dtype).view(n, Hq + 2 * Hk, D)
        s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hk]      # views of the joint projection
        freq, axis = _inv_freq(case)
        first = int(rs.integers(0, 131072))
        at = first + np.arange(n)
        pos = at[:, None] if case["axes"] == 1 else np.stack([at // 64, at // 8 % 8, at % 8][:case["axes"]], 1)
        s["positions"] = torch.from_numpy(np.ascontiguousarray(pos.astype(np.int32))).to(dev)
        s["freq"], s["axis"] = torch.from_numpy(freq).to(dev), torch.from_numpy(axis).to(dev)
        s["rot"], s["paired"] = case["rot"], case["paired"]
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(dtype) if case["weights"] else None for _ in range(2))
        if own:
            from compressed_kv_cache_gb300 import tq
            s["rotary"] = tq.Rotary(freq, dev, axis=axis, paired=case["paired"])      # a model's table, made once
        return s
    B, H, page = case["B"], case["H"], case["page"]
    count, before = _counts(case)
    order = rs.permutation(B)
    count, before = [count[i] for i in order], [before[i] for i in order]
    M = max(-(-(c + n) // page) for c, n in zip(count, before))
    N = sum(-(-(c + n) // page) for c, n in zip(count, before)) + 3
    table, ids, at = np.full((B, M), -1, dtype=np.int32), rs.permutation(N), 0      # entries behind a last page are never used
    for b in range(B):
        used = -(-(count[b] + before[b]) // page)
        table[b, :used] = ids[at:at + used]
        at += used
    pool, exps = _pool(seed, D, dev)
    pick = torch.randint(0, 2048, (2, N * H * (page // BLOCK)), generator=gen, device=dev)
    s["kc"], s["vc"] = (pool[i][pick[i]].view(N, H, page, D) for i in range(2))
    s["ex"] = torch.stack([exps[i][pick[i]] for i in range(2)], -1).view(N, H, page // BLOCK, 2).contiguous()
    n = sum(count)
    s["table"] = torch.from_numpy(table).to(dev)
    s["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(count)]).astype(np.int32)).to(dev)
    s["lengths"] = torch.tensor(before, dtype=torch.int32, device=dev)
    s["n"], s["most"], s["dtype"] = n, max(count), dtype
    if case["op"] == "append":
        w = torch.ones(D, device=dev)
        w[[3, 17, D - 5]] = 8.0
        s["K"] = (torch.randn(n, H, D, generator=gen, device=dev) * w * torch.exp(0.5 * torch.randn(n, 1, 1, generator=gen, device=dev))).to(dtype)
        joint = torch.randn(n, 2 * H, D, generator=gen, device=dev).to(dtype)
        s["V"] = joint[:, H:]      # the values' part of a joint projection
    elif case["op"] == "attend":
        s["Q"] = torch.randn(n, H * case["G"], D, generator=gen, device=dev).mul_(1.5).to(dtype)
        s["window"], s["sinks"] = case["window"], case["sinks"]
    if own:
        from compressed_kv_cache_gb300 import tq
        s["cache"] = tq.Int8Cache(s["kc"], s["vc"], s["ex"])      # a layer's handle, made once
        if case["op"] == "attend":      # scratch that a server keeps from step to step
            s["workspace"] = torch.empty(tq.attend_int8_workspace_bytes(n, B, H, case["G"], D), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"norm_rope": _norm_rope, "append": _append, "read": _read, "attend": _attend}[s["op"]](s)


def _norm_rope(s):
    if own:
        from compressed_kv_cache_gb300 import tq
        return tq.norm_rope(s["q"], s["k"], s["positions"], s["rotary"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS)
    angle = s["positions"].double()[:, s["axis"]] * s["freq"]      # far positions need the 64 bits
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    return _turned(s, s["q"], s["wq"], cos, sin), _turned(s, s["k"], s["wk"], cos, sin)


def _turned(s, x, w, cos, sin):
    y, rot = x.float(), s["rot"]
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    out = y.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if s["paired"] else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., first] = y[..., first] * cos - y[..., second] * sin
    out[..., second] = y[..., second] * cos + y[..., first] * sin
    return out.to(x.dtype)


def _power(e):
    """2^e in fp32, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _slots(s):
    """Sequence and slot of each token."""
    i = torch.arange(s["n"], device=s["table"].device)
    seq = torch.searchsorted(s["starts"].long(), i, right=True) - 1
    return seq, s["lengths"].long()[seq] + i - s["starts"].long()[seq]


def _append(s):
    if own:
        from compressed_kv_cache_gb300 import tq
        tq.append_int8(s["K"], s["V"], s["starts"], s["cache"], s["table"], s["lengths"])
    else:
        seq, slot = _slots(s)
        page, per, H = s["kc"].shape[2], s["ex"].shape[2], s["kc"].shape[1]
        table, lengths, head = s["table"].long(), s["lengths"].long(), torch.arange(H, device=seq.device)
        # the block that each sequence goes on with, and where it holds rows already
        live, last = lengths % BLOCK, torch.clamp(lengths // page, max=table.shape[1] - 1)
        tail = table.gather(1, last.unsqueeze(1)).clamp(min=0)
        goes_on = (live > 0) & (s["starts"][1:] > s["starts"][:-1])
        block = lambda pages, at: (pages * H + head) * per + at % page // BLOCK  # noqa: E731
        tails = block(tail, lengths.unsqueeze(1))
        blocks = block(table[seq, slot // page].unsqueeze(1), slot.unsqueeze(1))
        for x, codes, of in ((s["K"], s["kc"], 0), (s["V"], s["vc"], 1)):
            ex, flat = s["ex"].view(-1, 2)[:, of], codes.view(-1, BLOCK, codes.shape[-1])
            new = torch.full(ex.shape, LOWEST, dtype=torch.int32, device=ex.device)
            new.scatter_reduce_(0, blocks.view(-1), _exponents(x.float().abs().amax(-1)).view(-1), "amax")
            at = tails[goes_on].view(-1)
            old = ex[at].int()
            new[at] = torch.maximum(new[at], old)
            shift = (new[at] - old).clamp(max=31).view(-1, 1, 1)
            rows = torch.arange(BLOCK, device=ex.device) < live[goes_on].repeat_interleave(H).unsqueeze(1)
            was = flat[at]
            flat[at] = torch.where(rows.unsqueeze(-1), ((was.int() - 128 >> shift) + 128).to(torch.uint8), was)
            y = torch.floor(x.double() * _power(-new[blocks]).double().unsqueeze(-1)) + 128
            flat[blocks, slot.unsqueeze(1) % BLOCK] = y.clamp(0, 255).to(torch.uint8)
            ex[blocks.view(-1)] = new[blocks.view(-1)].to(torch.int8)
    # whole numbers: a code that differs is an error
    return {"kc": s["kc"], "vc": s["vc"], "ex": s["ex"]}


def _read(s):
    if own:
        from compressed_kv_cache_gb300 import tq
        return tq.read_int8(s["cache"], s["table"], s["starts"], s["lengths"], s["n"], s["dtype"])
    seq, slot = _slots(s)
    page = s["kc"].shape[2]
    pages = s["table"].long()[seq, slot // page]
    e = _power(s["ex"][pages, :, slot % page // BLOCK]).unsqueeze(-1)
    return tuple(((x[pages, :, slot % page].float() - 127.5) * e[:, :, i]).to(s["dtype"]) for i, x in enumerate((s["kc"], s["vc"])))


def _dense(s, codes, of):
    """Values of all slots, [B, H, M * page, D] fp32 (those of any page where there is none)."""
    pages = s["table"].clamp(min=0).long()
    e = _power(s["ex"][pages][..., of])                                    # [B, M, H, blocks]
    x = codes[pages]
    x = (x.view(*e.shape, BLOCK, x.shape[-1]).float() - 127.5) * e[..., None, None]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _attend(s):
    if own:
        from compressed_kv_cache_gb300 import tq
        return tq.attend_int8(s["Q"], s["starts"], s["cache"], s["table"], s["lengths"], window=s["window"] or None, sinks=s["sinks"], workspace=s["workspace"])
    Q, H, B, T = s["Q"], s["kc"].shape[1], s["table"].shape[0], s["most"]
    D, G = Q.shape[-1], Q.shape[1] // H
    t = torch.arange(T, device=Q.device)
    starts = s["starts"].long()
    token = starts[:-1].unsqueeze(1) + t
    there = token < starts[1:].unsqueeze(1)
    token = token.clamp(max=s["n"] - 1)
    q = Q.float()[token].view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    z = torch.matmul(q, _dense(s, s["kc"], 0).transpose(-1, -2)) / math.sqrt(D)
    slot = torch.arange(z.shape[-1], device=z.device)
    at = (s["lengths"].long().unsqueeze(1) + t).unsqueeze(-1)              # [B, T, 1]
    seen = slot <= at
    if s["window"]:
        seen = seen & ((slot > at - s["window"]) | (slot < s["sinks"]))
    z = z.view(B, H, T, G, -1).masked_fill_(~seen.view(B, 1, T, 1, -1), -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, H, T * G, -1)
    out = torch.matmul(p, _dense(s, s["vc"], 1)).view(B, H, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, H * G, D)
    return out[there].to(Q.dtype)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        turn = torch.polar(torch.ones_like(s["positions"][:, :1].double() * s["freq"]), s["positions"].double()[:, s["axis"]] * s["freq"])
        got = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            y = x.double()
            if w is not None:
                y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / case["D"] + EPS) * w.double()
            r = y[..., :case["rot"]].unflatten(-1, (-1, 2) if case["paired"] else (2, -1))
            dim = -1 if case["paired"] else -2
            a, b = r.unbind(dim)
            z = torch.complex(a, b) * turn.unsqueeze(1)
            r = torch.stack([z.real, z.imag], dim).flatten(-2)
            got.append(torch.cat([r, y[..., case["rot"]:]], -1))
        return tuple(got)
    table, lengths, starts = (s[x].cpu().numpy().astype(np.int64) for x in ("table", "lengths", "starts"))
    page, D, H, B = case["page"], case["D"], case["H"], case["B"]
    if case["op"] == "append":
        # block by block: the least power of two that holds the old rows and the new ones, the old codes shifted to it
        if s["n"] * H > 70000:
            return None
        kc, vc, ex = s["kc"].cpu().numpy(), s["vc"].cpu().numpy(), s["ex"].cpu().numpy()
        new = [x.double().cpu().numpy() for x in (s["K"], s["V"])]
        for b in range(B):
            first, stop = lengths[b], lengths[b] + starts[b + 1] - starts[b]
            for lo in range(first // BLOCK * BLOCK, stop, BLOCK):
                pg, r = table[b, lo // page], lo % page
                a, z = max(lo, first), min(lo + BLOCK, stop)
                for i, codes in enumerate((kc, vc)):
                    x = new[i][starts[b] + a - first:starts[b] + z - first]                    # [rows, H, D]
                    most = np.abs(x).max((0, 2))
                    e = np.where(most > 0, np.floor(np.log2(np.where(most > 0, most, 1.0))) - 6, LOWEST)
                    old = codes[pg, :, r:r + a - lo].astype(np.int64) - 128                    # [H, rows, D]
                    if a > lo:
                        was = ex[pg, :, r // BLOCK, i].astype(np.int64)
                        e = np.maximum(e, was)
                        codes[pg, :, r:r + a - lo] = np.floor_divide(old, 2 ** (e - was).astype(np.int64)[:, None, None]) + 128
                    codes[pg, :, r + a - lo:r + z - lo] = np.floor(x.transpose(1, 0, 2) / 2.0 ** e[:, None, None]) + 128
                    ex[pg, :, r // BLOCK, i] = e
        return {"kc": kc, "vc": vc, "ex": ex}
    kc, vc, ex = s["kc"], s["vc"], s["ex"].double()

    def values(codes, of, b, lo, hi):
        """Slots lo to hi of sequence b, [H, hi - lo, D]."""
        at = np.arange(lo, hi)
        pg, r = (torch.from_numpy(x).to(codes.device) for x in (table[b, at // page], at % page))
        x = codes[pg, :, r].double() - 127.5
        return (x * torch.exp2(ex[pg, :, r // BLOCK, of]).unsqueeze(-1)).transpose(0, 1)

    if case["op"] == "read":
        return tuple(torch.cat([values(x, i, b, lengths[b], lengths[b] + starts[b + 1] - starts[b]).transpose(0, 1) for b in range(B)]) for i, x in enumerate((kc, vc)))
    out = torch.zeros(s["Q"].shape, dtype=torch.float64, device=s["Q"].device)
    for b in range(B):
        n = int(lengths[b] + starts[b + 1] - starts[b])
        k, v = values(kc, 0, b, 0, n), values(vc, 1, b, 0, n)
        for i in range(starts[b], starts[b + 1]):
            at = int(lengths[b] + i - starts[b])
            seen = torch.arange(at + 1, device=k.device)
            if case["window"]:
                seen = seen[(seen >= at + 1 - case["window"]) | (seen < case["sinks"])]
            q = s["Q"][i].double().view(H, case["G"], D)
            w = torch.softmax(torch.einsum("hgd,hsd->hgs", q, k[:, seen]) * D ** -0.5, -1)
            out[i] = torch.einsum("hgs,hsd->hgd", w, v[:, seen]).reshape(-1, D)
    return out
