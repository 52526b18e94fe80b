"""Measured cases of the serving operators: rotary positions, the quantised
K/V cache (write and read back) and attention of drafted tokens over it.

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits, angles in 64), or, where ``own`` is true, by the calls that a
user makes of the package.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3_MAX = 448.0
AMAX_MIN = 448.0 * 2.0 ** -126   # below this a row's descale would leave the normal range


def listed():
    return [
        # one decoding step of a batch: every sequence adds one token far into its context
        dict(name="rope_decode", op="rope", B=32, Hq=32, Hk=8, N=1, d=128, rot=128,
             interleaved=False, dtype="bf16", max_pos=131072, token_major=False, stretch=8.0),
        # the prompt of the mid-context workload, rotated as it comes out of its projection
        dict(name="rope_prompt", op="rope", B=2, Hq=32, Hk=32, N=8192, d=128, rot=128,
             interleaved=True, dtype="bf16", max_pos=8192, token_major=True, stretch=1.0),
        # gradients of the padded batch, rotary on half of the head
        dict(name="rope_backward_part", op="rope_backward", B=8, Hq=16, Hk=16, N=4099, d=128, rot=64,
             interleaved=False, dtype="fp16", max_pos=32768, token_major=True, stretch=4.0),
        # gradients of the short training shape
        dict(name="rope_backward_short", op="rope_backward", B=4, Hq=16, Hk=4, N=1024, d=64, rot=64,
             interleaved=True, dtype="bf16", max_pos=1024, token_major=False, stretch=1.0),
        # one new token of each sequence of a batch goes into its page
        dict(name="cache_write_step", op="cache_write", B=64, Hk=8, N=1, d=128, page=16,
             dtype="bf16", e4m3=True, ragged=0.0, at=1000),
        # the prompts of a padded batch, each as long as it is
        dict(name="cache_write_prompt", op="cache_write", B=8, Hk=16, N=4099, d=128, page=64,
             dtype="bf16", e4m3=True, ragged=0.9, at=0),
        # the cached prefixes of a batch back in 16 bits, for the dense kernels
        dict(name="cache_read_prefix", op="cache_read", B=8, Hk=16, N=4099, d=64, page=32,
             dtype="fp16", e4m3=True, ragged=0.9, at=0),
        # one long context back in 16 bits
        dict(name="cache_read_long", op="cache_read", B=1, Hk=32, N=32768, d=128, page=128,
             dtype="bf16", e4m3=True, ragged=0.0, at=0),
        # one token of one short sequence: latency
        dict(name="tree_one", op="tree", B=1, Hq=32, Hk=8, T=1, ctx=1000, d=128, page=16,
             dtype="bf16", e4m3=True, ragged=0.0),
        # a decoding step of a batch whose sequences have all lengths
        dict(name="tree_decode", op="tree", B=64, Hq=32, Hk=8, T=1, ctx=8192, d=128, page=64,
             dtype="bf16", e4m3=True, ragged=0.9),
        # trees of drafted tokens of a batch
        dict(name="tree_draft", op="tree", B=16, Hq=32, Hk=8, T=32, ctx=8192, d=128, page=32,
             dtype="fp16", e4m3=True, ragged=0.9),
        # a few drafted tokens over very long contexts kept in 16 bits
        dict(name="tree_long", op="tree", B=2, Hq=32, Hk=8, T=8, ctx=131072, d=128, page=256,
             dtype="bf16", e4m3=False, ragged=0.2),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_backward", "cache_write", "cache_read", "tree", "tree", "tree"])
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8, 16, 32])
    most = max(work(c)["bytes"] for c in listed())
    flops = max(work(c)["flops"] for c in listed())
    while True:
        B = _spread(rng, 1, 64)
        if op.startswith("rope"):
            case = dict(op=op, B=B, Hq=Hk * rng.choice([1, 2, 4, 8]), Hk=Hk, N=_spread(rng, 1, 8192), d=d,
                        rot=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.5, dtype=dtype,
                        max_pos=rng.choice([8192, 131072, 1000000]), token_major=rng.random() < 0.5,
                        stretch=rng.choice([1.0, 4.0, 8.0]))
        elif op.startswith("cache"):
            case = dict(op=op, B=B, Hk=Hk, N=_spread(rng, 1, 32768), d=d,
                        page=rng.choice([16, 32, 48, 64, 128, 256]), dtype=dtype,
                        e4m3=rng.random() < 0.75, ragged=rng.choice([0.0, 0.5, 0.9]),
                        at=rng.choice([0, rng.randint(1, 2000)]))
        else:
            T = rng.choice([1, 1, _spread(rng, 2, 64)])
            case = dict(op=op, B=B, Hq=Hk * rng.choice([1, 2, 4, 8]), Hk=Hk, T=T, ctx=_spread(rng, 1, 131072),
                        d=d, page=rng.choice([16, 32, 48, 64, 128, 256]), dtype=dtype,
                        e4m3=rng.random() < 0.75, ragged=rng.choice([0.0, 0.5, 0.9]))
        w = work(case)
        if w["bytes"] <= most / 2 and w["flops"] <= flops:
            return case


def _lengths(B, most, ragged):
    """Lengths of B sequences, from (1 - ragged) * most to most, evenly mixed."""
    return [max(1, int(round(most * (1.0 - ragged * ((b * 0.6180339887) % 1.0))))) for b in range(B)]


def work(case):
    c = case
    if c["op"].startswith("rope"):
        n = c["B"] * c["N"] * (c["Hq"] + c["Hk"]) * c["d"]
        return {"bytes": 4 * n + 4 * c["B"] * c["N"], "flops": 3 * n * c["rot"] / c["d"]}
    size = 1 if c["e4m3"] else 2
    per_row = size * c["d"] + (4 if c["e4m3"] else 0)
    if c["op"].startswith("cache"):
        rows = 2 * c["Hk"] * sum(_lengths(c["B"], c["N"], c["ragged"]))
        return {"bytes": rows * (2 * c["d"] + per_row), "flops": 2 * rows * c["d"]}
    keys = sum(_lengths(c["B"], c["ctx"], c["ragged"])) + c["B"] * c["T"]
    q = c["B"] * c["Hq"] * c["T"]
    return {"bytes": 2 * keys * c["Hk"] * per_row + q * (4 * c["d"] + 4) + c["B"] * c["T"] ** 2,
            "flops": 4 * keys * c["Hq"] * c["T"] * c["d"]}


def _frequencies(case, device):
    """Rotary frequencies in 64 bits, all positions stretched by a factor."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=device)
    return torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=device), -2.0 * i / case["rot"]) / case["stretch"]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    s = {"case": c}
    B, d, Hk = c["B"], c["d"], c["Hk"]
    if c["op"].startswith("rope"):
        if c["token_major"]:
            s["q"], s["k"] = (normal(B, c["N"], H, d).transpose(1, 2) for H in (c["Hq"], Hk))
        else:
            s["q"], s["k"] = (normal(B, H, c["N"], d) for H in (c["Hq"], Hk))
        first = torch.randint(0, max(1, c["max_pos"] - c["N"] + 1), (B, 1), generator=g, device=dev)
        s["positions"] = (first + torch.arange(c["N"], device=dev)).to(torch.int32)
        s["inv_freq"] = _frequencies(c, dev)
        return s

    # a pool of pages in random order, enough for the longest sequence of each row of the table
    page = c["page"]
    most = c["ctx"] + c["T"] if c["op"] == "tree" else c["at"] + c["N"]
    per_seq = (most + page - 1) // page
    pages = B * per_seq + 3
    order = torch.randperm(pages, generator=g, device=dev)
    s["table"] = order[:B * per_seq].reshape(B, per_seq).to(torch.int32)
    shuffle = torch.randperm(B, generator=g, device=dev)
    lens = torch.tensor(_lengths(B, c["ctx"] if c["op"] == "tree" else c["N"], c["ragged"]),
                        dtype=torch.int32, device=dev)[shuffle].contiguous()
    shape = (pages, Hk, page, d)
    s["k_scale"] = s["v_scale"] = None
    if c["op"] == "cache_write":
        for n in ("k", "v"):
            s[n] = normal(B, c["N"], Hk, d).transpose(1, 2)
            if c["e4m3"]:
                s[n + "_cache"] = torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
                s[n + "_scale"] = torch.ones(shape[:3], device=dev)
            else:
                s[n + "_cache"] = torch.zeros(shape, dtype=dt, device=dev)
        s["start"] = torch.full((B,), c["at"], dtype=torch.int32, device=dev)
        s["lens"] = lens
        return s
    for n in ("k", "v"):
        if c["e4m3"]:
            codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
            scale = torch.empty(shape[:3], device=dev)
            flat, flat_scale = codes.view(-1, d), scale.view(-1)
            for r in range(0, flat.shape[0], 1 << 20):   # what the rows of a model's cache hold
                x = torch.randn(min(1 << 20, flat.shape[0] - r), d, generator=g, device=dev)
                flat[r:r + x.shape[0]], flat_scale[r:r + x.shape[0]] = _quantise(x.to(dt))
            s[n + "_cache"], s[n + "_scale"] = codes, scale
        else:
            s[n + "_cache"] = torch.empty(shape, dtype=dt, device=dev)
            flat = s[n + "_cache"].view(-1, d)
            for r in range(0, flat.shape[0], 1 << 20):
                flat[r:r + (1 << 20)] = torch.randn(min(1 << 20, flat.shape[0] - r), d, generator=g, device=dev).to(dt)
    if c["op"] == "cache_read":
        s["start"] = torch.full((B,), c["at"], dtype=torch.int32, device=dev)
        s["lens"] = lens
        for n in ("k_out", "v_out"):
            s[n] = torch.zeros((B, Hk, c["N"], d), dtype=dt, device=dev)
        return s
    T = c["T"]
    s["q"] = normal(B, c["Hq"], T, d)
    s["ctx_lens"] = lens
    s["out"] = torch.zeros((B, c["Hq"], T, d), dtype=dt, device=dev)
    s["lse"] = torch.zeros((B, c["Hq"], T), device=dev)
    # random trees: token t hangs below one of the tokens before it
    host = torch.Generator().manual_seed(seed)
    mask = torch.eye(T, dtype=torch.bool).repeat(B, 1, 1)
    every = torch.arange(B)
    for t in range(1, T):
        parent = torch.randint(0, t, (B,), generator=host)
        mask[:, t] |= mask[every, parent]
    s["tree_mask"] = mask.to(torch.uint8).to(dev)
    return s


def _quantise(x):
    """Rows of x as e4m3 codes and one descale each."""
    x = x.float()
    amax = x.abs().amax(-1)
    top = amax.clamp_min(AMAX_MIN)
    codes = (x * (E4M3_MAX / top).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, torch.where(amax > 0, top / E4M3_MAX, torch.ones_like(top))


def _rotate(x, positions, inv_freq, interleaved, sign):
    angle = positions.to(torch.float64).unsqueeze(-1) * inv_freq
    cos = angle.cos().float().unsqueeze(1)
    sin = sign * angle.sin().float().unsqueeze(1)
    rot = 2 * inv_freq.numel()
    y = x.float()
    a, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        x1, x2 = a[..., 0::2], a[..., 1::2]
        a = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    else:
        x1, x2 = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    return torch.cat((a, rest), -1).to(x.dtype).contiguous()


def _slots(table, position, page):
    """Pages and rows of positions [B, n]; positions past the table go to its last page."""
    at = (position // page).clamp_max(table.shape[1] - 1)
    return torch.gather(table.long(), 1, at), position % page


def _gather(cache, scale, pages, rows):
    """[B, n, Hk, d] values in 32 bits."""
    if scale is None:
        return cache[pages, :, rows].float()
    return cache.view(torch.uint8)[pages, :, rows].view(torch.float8_e4m3fn).float() * scale[pages, :, rows].unsqueeze(-1)


def _plain_write(s, x, cache, scale):
    c = s["case"]
    n = torch.arange(c["N"], device=x.device)
    valid = n < s["lens"].unsqueeze(1)
    pages, rows = _slots(s["table"], s["start"].long().unsqueeze(1) + n, c["page"])
    pages, rows = pages[valid], rows[valid]
    new = x.transpose(1, 2)[valid]
    if scale is None:
        cache[pages, :, rows] = new
    else:
        codes, new_scale = _quantise(new)
        cache.view(torch.uint8)[pages, :, rows] = codes.view(torch.uint8)
        scale[pages, :, rows] = new_scale


def _plain_read(s, cache, scale, out):
    c = s["case"]
    n = torch.arange(c["N"], device=out.device)
    pages, rows = _slots(s["table"], s["start"].long().unsqueeze(1) + n, c["page"])
    x = _gather(cache, scale, pages, rows).to(out.dtype).transpose(1, 2)
    keep = (n < s["lens"].unsqueeze(1)).view(c["B"], 1, c["N"], 1)
    out.copy_(torch.where(keep, x, out))


def _plain_tree(s):
    c = s["case"]
    B, Hq, Hk, T, d = c["B"], c["Hq"], c["Hk"], c["T"], c["d"]
    ctx = s["ctx_lens"].long()
    j = torch.arange(c["ctx"] + T, device=ctx.device)
    pages, rows = _slots(s["table"], j.expand(B, -1), c["page"])
    k = _gather(s["k_cache"], s["k_scale"], pages, rows).transpose(1, 2)
    v = _gather(s["v_cache"], s["v_scale"], pages, rows).transpose(1, 2)
    u = j - ctx.unsqueeze(1)                                      # [B, keys], negative in the context
    draft = torch.gather(s["tree_mask"].bool(), 2, u.clamp(0, T - 1).unsqueeze(1).expand(B, T, -1))
    seen = (u < 0).unsqueeze(1) | ((u >= 0) & (u < T)).unsqueeze(1) & draft
    q = s["q"].float().view(B, Hk, Hq // Hk * T, d)
    scores = (q @ k.transpose(-1, -2)) / math.sqrt(d)
    scores = scores.view(B, Hq, T, -1).masked_fill(~seen.unsqueeze(1), -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, Hk, Hq // Hk * T, -1) @ v
    s["out"].copy_((o.view(B, Hq, T, d) / total).to(s["q"].dtype))
    s["lse"].copy_((top + total.log()).squeeze(-1))
    return {"o": s["out"], "lse": s["lse"]}


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        return _run_own(s)
    if op.startswith("rope"):
        sign = 1.0 if op == "rope" else -1.0
        return {n: _rotate(s[n], s["positions"], s["inv_freq"], c["interleaved"], sign) for n in ("q", "k")}
    if op == "cache_write":
        _plain_write(s, s["k"], s["k_cache"], s["k_scale"])
        _plain_write(s, s["v"], s["v_cache"], s["v_scale"])
        return _cache_of(s)
    if op == "cache_read":
        _plain_read(s, s["k_cache"], s["k_scale"], s["k_out"])
        _plain_read(s, s["v_cache"], s["v_scale"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    return _plain_tree(s)


def _cache_of(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if s[n] is not None}


def _run_own(s):
    import exact_io_aware_47_b200 as fa
    c = s["case"]
    op = c["op"]
    if op.startswith("rope"):
        call = fa.rope if op == "rope" else fa.rope_backward
        q, k = call(s["q"], s["k"], s["inv_freq"], positions=s["positions"], interleaved=c["interleaved"])
        return {"q": q, "k": k}
    if op == "cache_write":
        fa.cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["start"], lens=s["lens"],
                       block_table=s["table"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return _cache_of(s)
    if op == "cache_read":
        k, v = fa.cache_read(s["k_cache"], s["v_cache"], s["start"], c["N"], lens=s["lens"],
                             block_table=s["table"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                             k_out=s["k_out"], v_out=s["v_out"])
        return {"k": k, "v": v}
    o, lse = fa.forward_tree(s["q"], s["k_cache"], s["v_cache"], s["ctx_lens"], tree_mask=s["tree_mask"],
                             block_table=s["table"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                             out=s["out"], lse=s["lse"])
    return {"o": o, "lse": lse}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and row by row."""
    c = case
    s = prepare(case, seed)
    op = c["op"]
    f64 = torch.float64
    if op.startswith("rope"):
        half = c["rot"] // 2
        got = {}
        for n in ("q", "k"):
            y = s[n].to(f64).contiguous()
            out = y.clone()
            for i in range(half):
                lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
                theta = s["positions"].to(f64) * 10000.0 ** (-2.0 * i / c["rot"]) / c["stretch"]
                theta = theta.unsqueeze(1) if op == "rope" else -theta.unsqueeze(1)
                out[..., lo] = y[..., lo] * theta.cos() - y[..., hi] * theta.sin()
                out[..., hi] = y[..., lo] * theta.sin() + y[..., hi] * theta.cos()
            got[n] = out
        return got

    table = s["table"].cpu().tolist()
    page = c["page"]

    def place(b, start, count):
        at = torch.arange(start, start + count, device=s["table"].device)
        pages = torch.tensor(table[b], device=at.device)
        return pages[at // page], at % page

    if op == "cache_write":
        got = _cache_of(s)
        got = {n: (x.float() if n.endswith("cache") else x).to(f64) for n, x in got.items()}
        for b in range(c["B"]):
            count = int(s["lens"][b])
            pages, rows = place(b, c["at"], count)
            for n in ("k", "v"):
                x = s[n][b, :, :count].transpose(0, 1).to(f64)
                if c["e4m3"]:
                    amax = x.abs().amax(-1, keepdim=True)
                    y = x * (E4M3_MAX / amax.clamp_min(AMAX_MIN))
                    # e4m3 holds 3 bits below the leading one, and steps of 2^-9 below 2^-6
                    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
                    got[n + "_cache"][pages, :, rows] = torch.round(y / step) * step
                    unit = torch.where(amax > 0, amax.clamp_min(AMAX_MIN) / E4M3_MAX, torch.ones_like(amax))
                    got[n + "_scale"][pages, :, rows] = unit.squeeze(-1)
                else:
                    got[n + "_cache"][pages, :, rows] = x
        return got

    def values(n, b, start, count):
        pages, rows = place(b, start, count)
        if not c["e4m3"]:
            return s[n + "_cache"][pages, :, rows].transpose(0, 1).to(f64)
        codes = s[n + "_cache"].view(torch.uint8)[pages, :, rows].view(torch.float8_e4m3fn)
        return (codes.to(f64) * s[n + "_scale"][pages, :, rows].to(f64).unsqueeze(-1)).transpose(0, 1)

    if op == "cache_read":
        got = {n: s[n + "_out"].to(f64) for n in ("k", "v")}
        for b in range(c["B"]):
            count = int(s["lens"][b])
            for n in ("k", "v"):
                got[n][b, :, :count] = values(n, b, c["at"], count)
        return got

    T, group = c["T"], c["Hq"] // c["Hk"]
    o = torch.zeros(s["q"].shape, dtype=f64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=f64, device=s["q"].device)
    for b in range(c["B"]):
        C = int(s["ctx_lens"][b])
        k, v = values("k", b, 0, C + T), values("v", b, 0, C + T)
        for h in range(c["Hq"]):
            x = s["q"][b, h].to(f64) @ k[h // group].T * c["d"] ** -0.5
            x[:, C:][s["tree_mask"][b] == 0] = -math.inf
            lse[b, h] = torch.logsumexp(x, -1)
            o[b, h] = torch.exp(x - lse[b, h].unsqueeze(-1)) @ v[h // group]
    return {"o": o, "lse": lse}
