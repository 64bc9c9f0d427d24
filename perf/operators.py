"""Cases of the serving operators around the KV cache, for timing and for comparison.

Four operators, each in a plain form (elementary torch operations, 32 bits or more
throughout, rounded once at the end) and as the framework's own call:

* norm_rope -- RMS norm of every query and key head with a weight per column, then the
  position rotation (adjacent pairs or half pairs, on part of the head, with frequencies
  scaled for long contexts);
* append    -- the same on the new rows of a packed ragged batch, the keys and values
  written to the paged pool on the way;
* shared    -- one decode step of a batch whose sequences share long prefixes, against
  the paged pool;
* cross     -- attention of decoder rows to an encoder's keys and values of another
  length, every row seeing all of its sequence's keys.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of each of 64 sequences: a decode step's projections, before the cache
        dict(name="norm_rope decode", op="norm_rope", dtype="bf16", B=64, T=1, H=32, Hkv=8, d=128, rot=128, layout="half",
             theta=1e6, scaling="none", factor=1.0, first=1000, norm=True),
        # the prompt of the causal prefill workload (14 heads of 64 columns, 2048 rows)
        dict(name="norm_rope prompt", op="norm_rope", dtype="bf16", B=1, T=2048, H=14, Hkv=2, d=64, rot=64, layout="interleaved",
             theta=1e6, scaling="turns", factor=4.0, first=0, norm=True),
        # long prompts far beyond the trained context: half of each head rotated, frequencies scaled
        dict(name="norm_rope long", op="norm_rope", dtype="bf16", B=2, T=8192, H=32, Hkv=8, d=128, rot=64, layout="half",
             theta=1e6, scaling="index", factor=8.0, first=100000, norm=True),
        # a decode step of 256 sequences, one new row each
        dict(name="append decode", op="append", dtype="bf16", B=256, rows_lo=1, rows_hi=1, pad=0, hist=256, H=32, Hkv=8, d=128,
             bs=16, rot=128, layout="half", theta=1e6, scaling="none", factor=1.0, norm=True),
        # a mixed batch: chunks of prompts beside single rows and idle sequences, rows of padding behind them
        dict(name="append ragged", op="append", dtype="bf16", B=24, rows_lo=0, rows_hi=301, pad=37, hist=1000, H=14, Hkv=2, d=64,
             bs=16, rot=64, layout="interleaved", theta=1e6, scaling="none", factor=1.0, norm=False),
        # 2048-row chunks of four prompts (the chunked prefill workload's rows at 32 heads of 128)
        dict(name="append chunks", op="append", dtype="bf16", B=4, rows_lo=2048, rows_hi=2048, pad=0, hist=6144, H=32, Hkv=8, d=128,
             bs=16, rot=128, layout="half", theta=1e6, scaling="turns", factor=8.0, norm=True),
        # a few requests behind one short system prompt
        dict(name="shared small", op="shared", dtype="bf16", B=4, groups=1, prefix=512, own_hi=64, H=14, Hkv=2, d=64, bs=16),
        # a batch of requests behind one long document
        dict(name="shared document", op="shared", dtype="bf16", B=64, groups=1, prefix=8192, own_hi=512, H=32, Hkv=8, d=128, bs=16),
        # a full server: four long prefixes, 256 requests
        dict(name="shared prefixes", op="shared", dtype="bf16", B=256, groups=4, prefix=16384, own_hi=1024, H=32, Hkv=8, d=128, bs=16),
        # a decode step against encoder states, group size 1, some slots without a source
        dict(name="cross decode", op="cross", dtype="bf16", B=64, S=1, L=1500, len_lo=0, H=16, Hkv=16, d=64),
        # a short fp32 call
        dict(name="cross small", op="cross", dtype="f32", B=2, S=37, L=201, len_lo=60, H=8, Hkv=2, d=64),
        # text rows against long encoder sequences
        dict(name="cross long", op="cross", dtype="bf16", B=8, S=1024, L=4096, len_lo=2048, H=32, Hkv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, d):
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    return G * Hkv, Hkv


def _rope_fields(rng, d):
    rot = rng.choice([d, d, d // 2, d // 4, d - 16])
    scaling = rng.choice(["none", "linear", "turns", "index"])
    return dict(rot=rot, layout=rng.choice(["half", "interleaved"]), theta=rng.choice([1e4, 5e5, 1e6]), scaling=scaling,
                factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "shared", "cross"])
    if op == "norm_rope":
        d = rng.choice([32, 64, 96, 128, 256])
        H, Hkv = _heads(rng, d)
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, min(8192, (1 << 26) // (B * (H + Hkv) * d))))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, T=T, H=H, Hkv=Hkv, d=d,
                    first=rng.choice([0, 77, 4095, 131072, 1000003]), norm=rng.random() < 0.7, **_rope_fields(rng, d))
    if op == "append":
        d = rng.choice([32, 64, 128, 256])
        H, Hkv = _heads(rng, d)
        B = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, max(1, min(2048, (1 << 25) // (B * (H + Hkv) * d))))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, rows_lo=rng.choice([0, 1, hi]), rows_hi=hi,
                    pad=rng.choice([0, 1, 29]), hist=_log_int(rng, 1, max(2, min(4000, (1 << 25) // (B * Hkv * d)))), H=H, Hkv=Hkv, d=d,
                    bs=rng.choice([8, 16, 32, 64, 128]), norm=rng.random() < 0.7, **_rope_fields(rng, d))
    if op == "shared":
        d = rng.choice([64, 128])
        H, Hkv = _heads(rng, d)
        B = _log_int(rng, 2, 256)
        room = (1 << 32) // (B * H * d)  # query-key products against the prefix
        prefix = _log_int(rng, 128, max(256, min(16384, room)))
        return dict(op=op, dtype="bf16", B=B, groups=rng.choice([1, 2, min(B, 5)]), prefix=prefix, own_hi=_log_int(rng, 1, 700),
                    H=H, Hkv=Hkv, d=d, bs=rng.choice([8, 16, 32, 64, 128]))
    d = rng.choice([64, 128])
    H, Hkv = _heads(rng, d)
    f32 = rng.random() < 0.2
    B = _log_int(rng, 1, 64)
    S = rng.choice([1, 1, _log_int(rng, 2, 32), _log_int(rng, 33, 1024)])
    room = (1 << (30 if f32 else 34)) // (B * S * H * d)
    L = _log_int(rng, 16, max(32, min(4096, room)))
    return dict(op=op, dtype="f32" if f32 else "bf16", B=B, S=S, L=L, len_lo=rng.choice([0, 1, L // 2, L]), H=H, Hkv=Hkv, d=d)


# ---------------------------------------------------------------------------- inputs
def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _frequencies(c):
    """Radians a position for each rotated pair, in 64 bits on the host, and the factor on cos and sin."""
    rot, theta, f, orig = c["rot"], c["theta"], c["factor"], 4096
    w = torch.tensor([theta ** (-2.0 * t / rot) for t in range(rot // 2)], dtype=torch.float64)
    if c["scaling"] == "linear":
        return w / f, 1.0
    if c["scaling"] == "turns":  # by how often the pair turns within the trained context
        keep = ((orig * w / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return w / f * (1 - keep) + w * keep, 1.0
    if c["scaling"] == "index":  # by the pair's place between those that turn 32 times and once
        def place(turns):
            return rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(theta))
        lo, hi = max(0.0, float(math.floor(place(32.0)))), min(rot - 1.0, float(math.ceil(place(1.0))))
        away = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return w / f * away + w * (1 - away), 0.1 * math.log(f) + 1.0
    return w, 1.0


def _rope_state(c, s):
    """What a program sets up once for its model: the frequencies, or the framework's own handle of them."""
    freq, s["magnitude"] = _frequencies(c)
    s["freq"] = freq.cuda()
    if own:
        import causal_gqa_attention_row_gb300 as g
        s["rope"] = g.rope_init(c["rot"], c["theta"], layout=c["layout"], scaling=c["scaling"], factor=c["factor"],
                                original_max=4096, low=1.0, high=32.0 if c["scaling"] == "index" else 4.0)


def _tables(gen, need, num_blocks, mbps):
    """Tables over disjoint blocks of a permuted pool, -1 behind each sequence's last block."""
    perm = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    start = torch.cumsum(need, 0) - need
    col = torch.arange(mbps, device="cuda")
    at = (start[:, None] + col[None, :]).clamp(max=num_blocks - 1)
    return torch.where(col[None, :] < need[:, None], perm[at], torch.full_like(perm[at], -1))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    dt = DTYPES[c["dtype"]]
    s = dict(c)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["op"] in ("norm_rope", "append"):
        _rope_state(c, s)
        s["wq"] = _randn(g, (d,), torch.float32, 0.2).add(1.0).to(dt) if c["norm"] else None
        s["wk"] = _randn(g, (d,), torch.float32, 0.2).add(1.0).to(dt) if c["norm"] else None
    if c["op"] == "norm_rope":
        B, T = c["B"], c["T"]
        # the fused projection's output: q, k and v of a token side by side
        qkv = _randn(g, (B, T, (H + 2 * Hkv) * d), dt, 1.3)
        s["q"] = qkv[..., :H * d].unflatten(-1, (H, d))
        s["k"] = qkv[..., H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d))
        at = torch.randint(0, 500, (B, 1), generator=g, device="cuda") + c["first"]
        s["positions"] = (at + torch.arange(T, device="cuda")).to(torch.int32)
        s["q_out"] = torch.empty(B, T, H, d, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(B, Hkv, T, d, dtype=dt, device="cuda")  # head-major, as the prefill takes the keys
    elif c["op"] == "append":
        B, bs = c["B"], c["bs"]
        rows = torch.randint(c["rows_lo"], c["rows_hi"] + 1, (B,), generator=g, device="cuda")
        hist = torch.randint(0, c["hist"] + 1, (B,), generator=g, device="cuda")
        mbps = (c["hist"] + c["rows_hi"] + bs - 1) // bs
        num_blocks = B * mbps + 3
        N = B * c["rows_hi"] + c["pad"]  # the packed buffer's rows: those behind the last sequence are padding
        s["tables"] = _tables(g, (hist + rows + bs - 1) // bs, num_blocks, mbps)
        s["row_starts"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(rows, 0)]).to(torch.int32)
        s["lens_in"] = hist.to(torch.int32)
        s["lens_out"] = torch.empty_like(s["lens_in"])
        qkv = _randn(g, (N, (H + 2 * Hkv) * d), dt, 1.3)
        s["q"] = qkv[:, :H * d].unflatten(-1, (H, d))
        s["k"] = qkv[:, H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d))
        s["v"] = qkv[:, (H + Hkv) * d:].unflatten(-1, (Hkv, d))
        s["q_out"] = torch.zeros(N, H, d, dtype=dt, device="cuda")
        s["k_pool"] = _randn(g, (num_blocks, Hkv, bs, d), dt)
        s["v_pool"] = _randn(g, (num_blocks, Hkv, bs, d), dt)
    elif c["op"] == "shared":
        B, bs, groups = c["B"], c["bs"], c["groups"]
        per = c["prefix"] // bs  # whole blocks of each prefix
        lens = torch.randint(1, c["own_hi"] + 1, (B,), generator=g, device="cuda")
        own_blocks = (c["own_hi"] + bs - 1) // bs
        num_blocks = groups * per + B * own_blocks + 3
        cut = torch.sort(torch.randperm(B - 1, generator=g, device="cuda")[:groups - 1] + 1).values if groups > 1 else lens[:0]
        s["group_starts"] = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), B)]).to(torch.int32)
        s["shared_blocks"] = torch.full((groups,), per, dtype=torch.int32, device="cuda")
        perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
        group = torch.bucketize(torch.arange(B, device="cuda"), s["group_starts"][1:], right=True)
        prefix = perm[:groups * per].view(groups, per)[group]
        tail = perm[groups * per:groups * per + B * own_blocks].view(B, own_blocks)
        tail = torch.where(torch.arange(own_blocks, device="cuda")[None] < ((lens + bs - 1) // bs)[:, None], tail, torch.full_like(tail, -1))
        s["tables"] = torch.cat([prefix, tail], 1).contiguous()
        s["lens"] = (lens + per * bs).to(torch.int32)
        s["q"] = _randn(g, (B, H, d), dt, 1.5)
        s["k_pool"] = _randn(g, (num_blocks, Hkv, bs, d), dt)
        s["v_pool"] = _randn(g, (num_blocks, Hkv, bs, d), dt)
        s["out"] = torch.empty(B, H, d, dtype=dt, device="cuda")
        if own:
            import causal_gqa_attention_row_gb300 as fw
            s["workspace"] = fw.shared_prefix_workspace(B, H, Hkv, d, s["tables"].shape[1] * bs, groups)
    else:
        B, S, L = c["B"], c["S"], c["L"]
        s["q"] = _randn(g, (B, S, H, d), dt, 1.5)
        s["k"] = _randn(g, (B, Hkv, L, d), dt)
        s["v"] = _randn(g, (B, Hkv, L, d), dt)
        s["lens"] = torch.randint(c["len_lo"], L + 1, (B,), generator=g, device="cuda").to(torch.int32)
        s["out"] = torch.empty(B, S, H, d, dtype=dt, device="cuda")
        if own:
            import causal_gqa_attention_row_gb300 as fw
            s["workspace"] = fw.cross_workspace(B, S, H, Hkv, d, d, L, dt)
    return s


# ---------------------------------------------------------------------------- plain forms
def _norm_rotate(s, x, w, positions):
    """x [..., heads, d] with positions of x's leading shape: norm with weight w, rotation; 32 bits."""
    y = x.float()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    angle = positions.double()[..., None, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()
    rot = s["rot"]
    if s["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_norm_rope(s):
    s["q_out"].copy_(_norm_rotate(s, s["q"], s["wq"], s["positions"]))
    s["k_out"].copy_(_norm_rotate(s, s["k"], s["wk"], s["positions"]).transpose(1, 2))
    return s["q_out"], s["k_out"]


def _plain_append(s):
    starts, bs = s["row_starts"].long(), s["bs"]
    n = s["q"].shape[0]
    token = torch.arange(n, device="cuda")
    b = torch.bucketize(token, starts[1:], right=True)
    real = token < starts[-1]
    b = b.clamp(max=s["B"] - 1)
    pos = s["lens_in"].long()[b] + token - starts[b]
    q, k = _norm_rotate(s, s["q"], s["wq"], pos), _norm_rotate(s, s["k"], s["wk"], pos)
    s["q_out"].copy_(torch.where(real[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    # rows of padding have no slot
    block = s["tables"].long()[b, (pos // bs).clamp(max=s["tables"].shape[1] - 1)]
    at, slot = block[real], (pos % bs)[real]
    s["k_pool"][at, :, slot] = k[real].to(s["k_pool"].dtype)
    s["v_pool"][at, :, slot] = s["v"][real]
    s["lens_out"].copy_(s["lens_in"] + (starts[1:] - starts[:-1]).to(torch.int32))
    return s["q_out"], s["k_pool"], s["v_pool"], s["lens_out"]


def _attend(q, k, v, lens, scale):
    """q [B, S, H, d], k and v [B, Hkv, L, d]: softmax over each sequence's first lens keys, in 32 bits; no keys give zeros."""
    B, S, H, d = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    rows = q.float().view(B, S, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    score = rows @ k.float().transpose(-1, -2) * scale
    seen = (torch.arange(L, device="cuda")[None, :] < lens[:, None])[:, None, None, :]
    score.masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top)), torch.zeros_like(score))
    total = p.sum(-1, keepdim=True)
    out = (p @ v.float()) / torch.where(total > 0, total, torch.ones_like(total))
    return out.view(B, Hkv, H // Hkv, S, d).permute(0, 3, 1, 2, 4).reshape(B, S, H, d)


def _plain_shared(s):
    t = s["tables"].long().clamp(min=0)
    k = s["k_pool"][t].transpose(1, 2).flatten(2, 3)
    v = s["v_pool"][t].transpose(1, 2).flatten(2, 3)
    s["out"].copy_(_attend(s["q"][:, None], k, v, s["lens"], 1.0 / math.sqrt(s["d"]))[:, 0])
    return s["out"]


def _plain_cross(s):
    s["out"].copy_(_attend(s["q"], s["k"], s["v"], s["lens"], 1.0 / math.sqrt(s["d"])))
    return s["out"]


# ---------------------------------------------------------------------------- the framework's calls
def _own_run(s):
    import causal_gqa_attention_row_gb300 as g
    if s["op"] == "norm_rope":
        g.attn_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"].transpose(1, 2), s["positions"], s["rope"],
                            q_weight=s["wq"], k_weight=s["wk"], eps=1e-6)
        return s["q_out"], s["k_out"]
    if s["op"] == "append":
        g.kv_append_paged_rows(s["q"], s["k"], s["v"], s["q_out"], s["k_pool"], s["v_pool"], s["tables"], s["row_starts"],
                               s["lens_in"], s["lens_out"], rope=s["rope"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6)
        return s["q_out"], s["k_pool"], s["v_pool"], s["lens_out"]
    if s["op"] == "shared":
        g.attn_decode_shared_prefix(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["group_starts"], s["shared_blocks"],
                                    s["out"], 1.0 / math.sqrt(s["d"]), workspace=s["workspace"])
        return s["out"]
    g.attn_cross(s["q"], s["k"], s["v"], s["out"], 1.0 / math.sqrt(s["d"]), kv_lens=s["lens"], workspace=s["workspace"])
    return s["out"]


def run(state):
    if own:
        return _own_run(state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "shared": _plain_shared, "cross": _plain_cross}[state["op"]](state)


# ---------------------------------------------------------------------------- work
def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["op"] == "norm_rope":
        n = c["B"] * c["T"]
        return {"bytes": 2 * n * (H + Hkv) * d * es + 4 * n, "flops": n * (H + Hkv) * (4 * d * c["norm"] + 3 * c["rot"])}
    if c["op"] == "append":
        n = c["B"] * (c["rows_lo"] + c["rows_hi"]) / 2
        return {"bytes": 2 * n * (H + 2 * Hkv) * d * es + 12 * c["B"], "flops": n * (H + Hkv) * (4 * d * c["norm"] + 3 * c["rot"])}
    if c["op"] == "shared":
        per = c["prefix"] // c["bs"] * c["bs"]
        mine = c["B"] * (1 + c["own_hi"]) / 2
        return {"bytes": (c["groups"] * per + mine) * Hkv * d * 2 * es + 2 * c["B"] * H * d * es,
                "flops": 4 * (c["B"] * per + mine) * H * d}
    keys = c["B"] * (c["len_lo"] + c["L"]) / 2
    return {"bytes": keys * Hkv * d * 2 * es + 2 * c["B"] * c["S"] * H * d * es, "flops": 4 * keys * c["S"] * H * d}


# ---------------------------------------------------------------------------- 64 bits
def _exact_rows(c, x, w, positions, freq, magnitude):
    """The definition, in 64 bits, by complex numbers: each pair is one number, turned by e^(i angle)."""
    y = x.double()
    if w is not None:
        y = y * w.double() * torch.rsqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + 1e-6)
    rot = c["rot"]
    first = torch.arange(rot // 2, device="cuda") * (1 if c["layout"] == "half" else 2)
    second = first + (rot // 2 if c["layout"] == "half" else 1)
    turn = torch.polar(torch.full_like(freq, magnitude), torch.zeros_like(freq)) * torch.exp(1j * (positions.double().unsqueeze(-1) * freq)).unsqueeze(-2)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_attend(q, k, v, scale):
    """q [S, H, d], k and v [Hkv, n, d] of one sequence, in 64 bits."""
    S, H, d = q.shape
    if k.shape[1] == 0:
        return torch.zeros(S, H, v.shape[-1], dtype=torch.float64, device="cuda")
    out = torch.empty(S, H, v.shape[-1], dtype=torch.float64, device="cuda")
    for h in range(k.shape[0]):
        of = slice(h * (H // k.shape[0]), (h + 1) * (H // k.shape[0]))
        weight = torch.softmax(torch.matmul(q[:, of].double(), k[h].double().T) * scale, -1)
        out[:, of] = torch.matmul(weight, v[h].double())
    return out


def exact(case, seed):
    global own
    c, kept = case, own
    own = False  # the inputs are the same on both sides; no handle of the framework is wanted here
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    scale = 1.0 / math.sqrt(c["d"])
    if c["op"] == "norm_rope":
        q = _exact_rows(c, s["q"], s["wq"], s["positions"], s["freq"], s["magnitude"])
        k = _exact_rows(c, s["k"], s["wk"], s["positions"], s["freq"], s["magnitude"])
        return q, k.transpose(1, 2)
    if c["op"] == "append":
        q_out, kp, vp = s["q_out"].double(), s["k_pool"].double(), s["v_pool"].double()
        starts, hist = s["row_starts"].tolist(), s["lens_in"].tolist()
        for b in range(c["B"]):
            rows = slice(starts[b], starts[b + 1])
            pos = torch.arange(hist[b], hist[b] + starts[b + 1] - starts[b], device="cuda")
            q_out[rows] = _exact_rows(c, s["q"][rows], s["wq"], pos, s["freq"], s["magnitude"])
            block = s["tables"][b].long()[pos // c["bs"]]
            kp[block, :, pos % c["bs"]] = _exact_rows(c, s["k"][rows], s["wk"], pos, s["freq"], s["magnitude"])
            vp[block, :, pos % c["bs"]] = s["v"][rows].double()
        return q_out, kp, vp, s["lens_in"] + torch.diff(s["row_starts"])
    if c["op"] == "shared":
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            block = s["tables"][b, :-(-n // c["bs"])].long()
            k = s["k_pool"][block].transpose(0, 1).reshape(c["Hkv"], -1, c["d"])[:, :n]
            v = s["v_pool"][block].transpose(0, 1).reshape(c["Hkv"], -1, c["d"])[:, :n]
            out[b] = _exact_attend(s["q"][b:b + 1], k, v, scale)[0]
        return out
    return torch.stack([_exact_attend(s["q"][b], s["k"][b, :, :n], s["v"][b, :, :n], scale) for b, n in enumerate(s["lens"].tolist())])
