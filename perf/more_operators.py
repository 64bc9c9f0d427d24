"""Cases of a decoding step that verifies drafted tokens, for timing and for comparison.

Each sequence brings a tree of drafted tokens behind its history: row i of the tree hangs on
row parents[i] (-1: on the history), is stored behind the history in the order of the rows,
stands at the position of its depth, and sees the history, its ancestors and itself. Four
operators, each in a plain form (elementary torch operations, 32 bits or more throughout,
rounded once at the end) and as the framework's own call:

* plan   -- from the requests' lengths: block tables that grow from, and give back to, a list
  of free blocks, the rows' starts, positions and slots, and the trees' masks;
* slots  -- norm and rotation of the new rows, keys and values written to given slots;
* tree   -- attention of the drafted rows over the paged cache;
* commit -- the rows of the accepted path moved together behind the history, in all layers.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a plain decode step of a full server: one row each, a block now and then
        dict(name="plan decode", op="plan", B=256, rows_lo=1, rows_hi=1, hist=4096, bs=16, tree=False, finished=0.05, pool=1.0, pad=0),
        # trees of up to 64 drafted rows, some requests over, some with blocks to spare after a rejection
        dict(name="plan trees", op="plan", B=128, rows_lo=1, rows_hi=64, hist=8192, bs=16, tree=True, finished=0.1, pool=1.0, pad=19),
        # prompts that come in chunks of up to 2048 rows, more than the pool has blocks for
        dict(name="plan prompts", op="plan", B=48, rows_lo=0, rows_hi=2048, hist=6144, bs=16, tree=False, finished=0.2, pool=0.7, pad=0),
        # the drafted rows' projections into the cache, 32 sequences of up to 16 rows
        dict(name="slots trees", op="slots", dtype="bf16", B=32, rows_lo=8, rows_hi=16, hist=2048, H=32, Hkv=8, d=128, bs=16,
             rot=128, layout="half", theta=1e6, norm=True, pad=5),
        # prompts of the causal prefill workload's heads, in fp32
        dict(name="slots prompts", op="slots", dtype="f32", B=6, rows_lo=1, rows_hi=2048, hist=500, H=14, Hkv=2, d=64, bs=16,
             rot=64, layout="interleaved", theta=1e6, norm=False, pad=0),
        # a few requests, short histories, small trees: latency
        dict(name="tree small", op="tree", dtype="bf16", B=4, rows_lo=4, rows_hi=8, hist_lo=100, hist=600, H=14, Hkv=2, d=64, bs=16, pad=0),
        # a single token each, as a step without a draft
        dict(name="tree of one", op="tree", dtype="bf16", B=32, rows_lo=1, rows_hi=1, hist_lo=500, hist=4096, H=32, Hkv=8, d=128, bs=16, pad=0),
        # a server's batch: trees of up to 32 rows, some sequences idle
        dict(name="tree server", op="tree", dtype="bf16", B=64, rows_lo=0, rows_hi=32, hist_lo=0, hist=8192, H=32, Hkv=8, d=128, bs=16, pad=11),
        # long histories with wide trees
        dict(name="tree long", op="tree", dtype="bf16", B=8, rows_lo=48, rows_hi=64, hist_lo=16384, hist=32768, H=32, Hkv=8, d=128, bs=64, pad=0),
        # fp32
        dict(name="tree f32", op="tree", dtype="f32", B=6, rows_lo=3, rows_hi=24, hist_lo=0, hist=1500, H=8, Hkv=2, d=64, bs=16, pad=2),
        # one request's accepted rows in one layer
        dict(name="commit one", op="commit", dtype="bf16", B=1, layers=1, rows=16, most=5, hist=900, Hkv=2, d=64, bs=16),
        # a batch's, in all layers of a model
        dict(name="commit layers", op="commit", dtype="bf16", B=64, layers=28, rows=64, most=8, hist=300, Hkv=8, d=128, bs=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 3, 4, 8])
    return rng.choice([1, 2, 3, 4, 5, 7, 8]) * Hkv, Hkv


def draw(rng):
    op = rng.choice(["plan", "slots", "tree", "tree", "commit"])
    bs = rng.choice([8, 16, 32, 64, 128])
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        tree = rng.random() < 0.5
        hi = _log_int(rng, 1, min(200 if tree else 2048, max(2, (1 << 16) // B)))
        return dict(op=op, B=B, rows_lo=rng.choice([0, 1, hi]), rows_hi=hi, hist=_log_int(rng, 1, 8192), bs=bs, tree=tree,
                    finished=rng.choice([0.0, 0.1, 0.5]), pool=rng.choice([0.3, 0.8, 1.0, 1.0]), pad=rng.choice([0, 1, 23]))
    if op == "slots":
        d = rng.choice([32, 64, 96, 128, 256])
        H, Hkv = _heads(rng)
        B = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(1, min(2048, (1 << 23) // (B * (H + Hkv) * d))))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, rows_lo=rng.choice([0, 1, hi]), rows_hi=hi,
                    hist=_log_int(rng, 1, max(2, min(4000, (1 << 24) // (B * Hkv * d)))), H=H, Hkv=Hkv, d=d, bs=bs,
                    rot=rng.choice([d, d, d // 2, d - 16]), layout=rng.choice(["half", "interleaved"]),
                    theta=rng.choice([1e4, 1e6]), norm=rng.random() < 0.6, pad=rng.choice([0, 1, 29]))
    if op == "tree":
        f32 = rng.random() < 0.25
        d = rng.choice([16, 32, 64, 128]) if f32 else rng.choice([64, 64, 128, 128, 128, 32, 256])
        slow = f32 or d not in (64, 128)  # no tensor cores for these
        H, Hkv = _heads(rng)
        B = _log_int(rng, 1, 96)
        hi = _log_int(rng, 1, 130)
        room = (1 << (27 if slow else 31)) // (B * hi * H * max(d, 64))
        hist = _log_int(rng, 1, max(2, min(32768, room * 16, (1 << 28) // (B * Hkv * d))))
        return dict(op=op, dtype="f32" if f32 else "bf16", B=B, rows_lo=rng.choice([0, 1, hi]), rows_hi=hi,
                    hist_lo=rng.choice([0, hist // 2, hist]), hist=hist, H=H, Hkv=Hkv, d=d, bs=bs, pad=rng.choice([0, 3]))
    d = rng.choice([32, 64, 128, 256])
    B = _log_int(rng, 1, 64)
    Hkv = rng.choice([1, 2, 4, 8])
    rows = _log_int(rng, 2, 100)
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, layers=_log_int(rng, 1, max(1, min(40, (1 << 26) // (B * 400 * Hkv * d)))),
                rows=rows, most=rng.randint(1, max(1, min(rows // 2, 10))), hist=_log_int(rng, 1, 300), Hkv=Hkv, d=d, bs=bs)


# ---------------------------------------------------------------------------- inputs
def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _randint(g, lo, hi, n):
    """n numbers of lo..hi."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")


def _starts(rows):
    return torch.cat([rows.new_zeros(1), torch.cumsum(rows, 0)]).to(torch.int32)


def _tables(gen, need, num_blocks, mbps):
    """Tables over disjoint blocks of a permuted pool, -1 behind each sequence's last block; and the blocks left over."""
    perm = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(mbps, device="cuda")
    at = ((torch.cumsum(need, 0) - need)[:, None] + col[None, :]).clamp(max=num_blocks - 1)
    return torch.where(col[None, :] < need[:, None], perm[at], torch.full_like(perm[at], -1)), perm[int(need.sum()):]


def _parents(g, rows, n):
    """A tree of rows[b] rows for each sequence, packed in n rows (-1 in the padding): a row hangs on any earlier one."""
    starts = _starts(rows).long()
    token = torch.arange(n, device="cuda")
    b = torch.bucketize(token, starts[1:], right=True)
    i = token - starts[b.clamp(max=rows.numel() - 1)]
    hang = (torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * i).long()
    return torch.where((b < rows.numel()) & (i > 0), hang, torch.full_like(hang, -1)).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    s = dict(c)
    B, bs = c["B"], c["bs"]
    if c["op"] == "plan":
        lens, new = _randint(g, 0, c["hist"], B), _randint(g, c["rows_lo"], c["rows_hi"], B)
        # blocks from the step before: what the rows need, and more where drafted rows were rejected
        held = (lens + _randint(g, 0, 64, B) * (torch.rand(B, generator=g, device="cuda") < 0.3) + bs - 1) // bs
        over = torch.rand(B, generator=g, device="cuda") < c["finished"]
        lens, new = lens.masked_fill(over, 0), new.masked_fill(over, 0)
        need = (lens + new + bs - 1) // bs
        mbps = (c["hist"] + max(c["rows_hi"], 64) + bs - 1) // bs
        num_blocks = B * mbps + 1  # some of them with other holders: of those that are free a share is listed
        s["tables"], left = _tables(g, held, num_blocks, mbps)
        spare = min(left.numel(), int(((need - held).clamp(min=0).sum() * c["pool"]).item()) + int(B * (c["pool"] >= 1.0)))
        s["free_list"] = torch.cat([left[:spare], left.new_full((num_blocks - spare,), -1)])
        s["free_in"] = torch.tensor([spare], dtype=torch.int32, device="cuda")
        s["lens"], s["new_rows"], s["held_in"] = lens.to(torch.int32), new.to(torch.int32), held.to(torch.int32)
        n = max(1, B * c["rows_hi"]) + c["pad"]
        s["parents"] = _parents(g, new, n) if c["tree"] else None
        s["mask"] = torch.zeros(n, (c["rows_hi"] + 63) // 64, dtype=torch.int64, device="cuda") if c["tree"] else None
        s["held_out"], s["free_out"] = torch.empty_like(s["held_in"]), torch.empty(2, dtype=torch.int32, device="cuda")
        s["row_starts"] = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        s["positions"] = torch.empty(n, dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(n, dtype=torch.int64, device="cuda")
        return s
    dt, Hkv, d = DTYPES[c["dtype"]], c["Hkv"], c["d"]
    if c["op"] == "slots":
        H = c["H"]
        rows, hist = _randint(g, c["rows_lo"], c["rows_hi"], B), _randint(g, 0, c["hist"], B)
        mbps = (c["hist"] + c["rows_hi"] + bs - 1) // bs
        num_blocks = B * mbps + 3
        n = B * c["rows_hi"] + c["pad"]
        tables, _ = _tables(g, (hist + rows + bs - 1) // bs, num_blocks, mbps)
        starts = _starts(rows).long()
        token = torch.arange(n, device="cuda")
        b = torch.bucketize(token, starts[1:], right=True).clamp(max=B - 1)
        at = hist[b] + token - starts[b]
        real = token < starts[-1]
        block = tables.long()[b, (at // bs).clamp(max=mbps - 1)]
        s["slots"] = torch.where(real, block * bs + at % bs, torch.full_like(at, -1))
        # a drafted row stands at the position of its depth, not at that of its slot
        s["positions"] = torch.where(real, hist[b] + (token - starts[b]) // 2, torch.zeros_like(at)).to(torch.int32)
        s["freq"] = torch.tensor([c["theta"] ** (-2.0 * t / c["rot"]) for t in range(c["rot"] // 2)], dtype=torch.float64).cuda()
        if own:
            import causal_gqa_attention_row_gb300 as fw
            s["rope"] = fw.rope_init(c["rot"], c["theta"], layout=c["layout"])
        s["wq"] = _randn(g, (d,), torch.float32, 0.2).add(1.0).to(dt) if c["norm"] else None
        s["wk"] = _randn(g, (d,), torch.float32, 0.2).add(1.0).to(dt) if c["norm"] else None
        qkv = _randn(g, (n, (H + 2 * Hkv) * d), dt, 1.3)
        s["q"] = qkv[:, :H * d].unflatten(-1, (H, d))
        s["k"] = qkv[:, H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d))
        s["v"] = qkv[:, (H + Hkv) * d:].unflatten(-1, (Hkv, d))
        s["q_out"] = torch.zeros(n, H, d, dtype=dt, device="cuda")
        s["k_pool"] = _randn(g, (num_blocks, Hkv, bs, d), dt)
        s["v_pool"] = _randn(g, (num_blocks, Hkv, bs, d), dt)
        return s
    if c["op"] == "tree":
        H = c["H"]
        rows, hist = _randint(g, c["rows_lo"], c["rows_hi"], B), _randint(g, c["hist_lo"], c["hist"], B)
        mbps = (c["hist"] + c["rows_hi"] + bs - 1) // bs
        num_blocks = int(((hist + rows + bs - 1) // bs).sum()) + 3
        n = B * c["rows_hi"] + c["pad"]
        s["tables"], _ = _tables(g, (hist + rows + bs - 1) // bs, num_blocks, mbps)
        s["row_starts"], s["lens"] = _starts(rows), hist.to(torch.int32)
        s["mask"] = _masks(_parents(g, rows, n), s["row_starts"], (c["rows_hi"] + 63) // 64)
        s["q"] = _randn(g, (n, H, d), dt, 1.5)
        s["k_pool"] = _randn(g, (num_blocks, Hkv, bs, d), dt)
        s["v_pool"] = _randn(g, (num_blocks, Hkv, bs, d), dt)
        s["out"] = torch.zeros(n, H, d, dtype=dt, device="cuda")
        if own:
            import causal_gqa_attention_row_gb300 as fw
            s["workspace"] = fw.tree_workspace(n, B, c["rows_hi"], H, Hkv, d, d, mbps * bs, dt)
        return s
    # commit: paths of accepted rows; those that move come from behind the accepted ones, so
    # that the same call on its own result changes nothing (a pass can be repeated)
    rows, most = c["rows"], c["most"]
    hist, n_path = _randint(g, 0, c["hist"], B), _randint(g, 0, most, B)
    mbps = (c["hist"] + rows + bs - 1) // bs
    num_blocks = B * mbps + 1
    s["tables"], _ = _tables(g, (hist + rows + bs - 1) // bs, num_blocks, mbps)
    j = torch.arange(most, device="cuda")[None, :]
    stay = (torch.rand(B, generator=g, device="cuda") * (n_path + 1)).long()  # so many lie where they belong
    luck = torch.rand(B, rows, generator=g, device="cuda")
    pick = torch.argsort(luck.masked_fill(torch.arange(rows, device="cuda")[None, :] < n_path[:, None], 2.0), 1)[:, :most]
    pick = torch.sort(pick.masked_fill(j >= (n_path - stay)[:, None], rows), 1).values
    path = torch.where(j < stay[:, None], j, torch.gather(pick, 1, (j - stay[:, None]).clamp(min=0)))
    s["path"] = torch.where(j < n_path[:, None], path, torch.full_like(path, -1)).to(torch.int32)
    s["n_path"], s["lens_in"] = n_path.to(torch.int32), hist.to(torch.int32)
    s["row_starts"] = torch.arange(0, (B + 1) * rows, rows, dtype=torch.int32, device="cuda")
    s["lens_out"] = torch.empty_like(s["lens_in"])
    s["k_pools"] = _randn(g, (c["layers"], num_blocks, Hkv, bs, d), dt)
    s["v_pools"] = _randn(g, (c["layers"], num_blocks, Hkv, bs, d), dt)
    return s


# ---------------------------------------------------------------------------- plain forms
def _masks(parents, row_starts, words):
    """Bit j of a row's mask: row j of its sequence is the row itself or an ancestor. Ancestors by doubling: after
    step i a row knows those up to 2^i above it, and `up` is the next one above those (the row `n`: none)."""
    n, starts = parents.numel(), row_starts.long()
    token = torch.arange(n, device="cuda")
    b = torch.bucketize(token, starts[1:], right=True)
    real = b < starts.numel() - 1
    first = starts[b.clamp(max=starts.numel() - 2)]
    i = token - first
    bit = torch.where(real, torch.ones_like(i), torch.zeros_like(i)) << (i % 64)
    mask = torch.zeros(n + 1, words, dtype=torch.int64, device="cuda")
    mask[:-1].scatter_(1, (i // 64).clamp(min=0, max=words - 1)[:, None], bit[:, None])
    up = torch.full((n + 1,), n, device="cuda")
    up[:-1] = torch.where(real & (parents >= 0), first + parents, torch.full_like(i, n))
    for _ in range((64 * words - 1).bit_length()):
        mask = mask | mask[up]
        up = up[up]
    return mask[:-1]


def _depths(mask):
    """How many bits are set in a row's words, less the row's own."""
    return ((mask[:, :, None] >> torch.arange(64, device="cuda")) & 1).sum((1, 2)) - 1


def _plain_plan(s):
    B, bs, n = s["B"], s["bs"], s["positions"].numel()
    lens, new, held = s["lens"].long(), s["new_rows"].long(), s["held_in"].long()
    free, stack, tables = s["free_in"].long()[0], s["free_list"], s["tables"]
    need = (lens + new + bs - 1) // bs
    give, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    served = (take == 0) | (torch.cumsum(take, 0) <= free + give.sum())
    missing = (take * ~served).sum()
    take = take * served
    have = torch.where(served, need, held)
    # blocks given back go onto the list, blocks taken come off its end
    col = torch.arange(tables.shape[1], device="cuda")[None, :]
    back = tables[(col >= need[:, None]) & (col < held[:, None])]  # sequence by sequence, entries ascending
    taken = take.sum()
    given, left = back.numel(), free + back.numel() - taken
    grown = (col >= held[:, None]) & (col < have[:, None])
    at = free + given - 1 - torch.arange(tables.numel(), device="cuda")  # of the t-th block taken
    both = torch.cat([stack, stack.new_zeros(1), back])  # (the list's own blocks, then those given back)
    at = torch.where(at >= free, at - free + stack.numel() + 1, at.clamp(min=0))
    order = (torch.cumsum(grown.flatten(), 0) - 1).clamp(min=0)
    tables.copy_(torch.where(grown, both[at[order]].view_as(tables), tables))
    where = torch.arange(stack.numel(), device="cuda")
    kept = both[(where - free + stack.numel() + 1).clamp(min=0, max=both.numel() - 1)]
    stack.copy_(torch.where((where >= free) & (where < left), kept, stack))
    s["held_out"].copy_(have)
    s["free_out"].copy_(torch.stack([left, missing]))
    s["row_starts"][0] = 0
    s["row_starts"][1:] = torch.cumsum(new, 0)
    starts = s["row_starts"].long()
    token = torch.arange(n, device="cuda")
    b = torch.bucketize(token, starts[1:], right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = lens[b] + token - starts[b]
    block = tables.long()[b, (pos // bs).clamp(min=0, max=tables.shape[1] - 1)]
    s["slots"].copy_(torch.where(real & served[b], block * bs + pos % bs, torch.full_like(pos, -1)))
    if s["parents"] is not None:
        s["mask"].copy_(_masks(s["parents"], s["row_starts"], s["mask"].shape[1]))
        pos = lens[b] + _depths(s["mask"])
    s["positions"].copy_(torch.where(real, pos, torch.zeros_like(pos)))


def _plan_outputs(s):
    # (behind held_out a table's entries, behind free_out the list's, are whatever was there)
    out = dict(tables=s["tables"], held=s["held_out"], free_list=s["free_list"], free=s["free_out"], row_starts=s["row_starts"],
               positions=s["positions"], slots=s["slots"])
    return out if s["mask"] is None else dict(out, mask=s["mask"])


def _norm_rotate(s, x, w):
    """x [N, heads, d]: norm with weight w, rotation; 32 bits."""
    y = x.float()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    angle = s["positions"].double()[:, None, None] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    rot = s["rot"]
    if s["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_slots(s):
    real = s["slots"] >= 0
    q, k = _norm_rotate(s, s["q"], s["wq"]), _norm_rotate(s, s["k"], s["wk"])
    s["q_out"].copy_(torch.where(real[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    block, row = s["slots"][real] // s["bs"], s["slots"][real] % s["bs"]
    s["k_pool"][block, :, row] = k[real].to(s["k_pool"].dtype)
    s["v_pool"][block, :, row] = s["v"][real]


def _plain_tree(s):
    B, H, Hkv, d, T = s["B"], s["H"], s["Hkv"], s["d"], s["rows_hi"]
    starts, hist = s["row_starts"].long(), s["lens"].long()
    t = s["tables"].long().clamp(min=0)
    k = s["k_pool"][t].transpose(1, 2).flatten(2, 3).float()  # [B, Hkv, L, d]
    v = s["v_pool"][t].transpose(1, 2).flatten(2, 3).float()
    L = k.shape[2]
    i = torch.arange(T, device="cuda")
    real = i[None, :] < (starts[1:] - starts[:-1])[:, None]  # [B, T]
    row = torch.where(real, starts[:-1, None] + i, torch.zeros_like(starts[:-1, None] + i))
    q = s["q"][row].float().view(B, T, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    score = (q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))).view(B, H, T, L)
    key = torch.arange(L, device="cuda")[None, :] - hist[:, None]  # [B, L]: the drafted row of a key, if not below 0
    word = (key // 64).clamp(min=0, max=s["mask"].shape[1] - 1)
    bits = torch.gather(s["mask"][row], 2, word[:, None, :].expand(B, T, L)) >> (key % 64)[:, None, :]
    seen = (key < 0)[:, None, :] | ((key < 64 * s["mask"].shape[1])[:, None, :] & ((bits & 1) != 0))  # [B, T, L]
    score.masked_fill_(~seen[:, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total > 0, total, torch.ones_like(total))).view(B, Hkv, -1, L)
    # keys behind a sequence's last weigh zero, whatever the slots hold
    out = (p @ v.masked_fill_((key >= (starts[1:] - starts[:-1])[:, None])[:, None, :, None], 0.0)).view(B, H, T, d).transpose(1, 2)
    s["out"][row[real]] = out[real].to(s["out"].dtype)


def _plain_commit(s):
    hist, path, bs = s["lens_in"].long(), s["path"].long(), s["bs"]
    moved = torch.arange(path.shape[1], device="cuda")[None, :] < s["n_path"].long()[:, None]
    b = torch.arange(s["B"], device="cuda")[:, None].expand_as(path)[moved]
    to = (hist[:, None] + torch.arange(path.shape[1], device="cuda"))[moved]
    of = (hist[:, None] + path)[moved]
    t = s["tables"].long()
    for pools in (s["k_pools"], s["v_pools"]):
        pools[:, t[b, to // bs], :, to % bs] = pools[:, t[b, of // bs], :, of % bs]
    s["lens_out"].copy_(s["lens_in"] + s["n_path"])


# ---------------------------------------------------------------------------- the framework's calls
def _own_run(s):
    import causal_gqa_attention_row_gb300 as g
    if s["op"] == "plan":
        g.kv_plan_rows(s["lens"], s["new_rows"], s["tables"], s["held_in"], s["held_out"], s["free_list"], s["free_in"], s["free_out"],
                       s["row_starts"], s["positions"], s["slots"], s["bs"], parents=s["parents"], tree_mask=s["mask"])
    elif s["op"] == "slots":
        g.kv_append_slots(s["q"], s["k"], s["v"], s["q_out"], s["k_pool"], s["v_pool"], s["slots"], s["positions"], rope=s["rope"],
                          q_weight=s["wq"], k_weight=s["wk"], eps=1e-6)
    elif s["op"] == "tree":
        g.attn_tree_paged(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["row_starts"], s["mask"], s["out"],
                          1.0 / math.sqrt(s["d"]), s["rows_hi"], workspace=s["workspace"])
    else:
        g.kv_commit_rows(s["k_pools"].unbind(0), s["v_pools"].unbind(0), s["tables"], s["lens_in"], s["row_starts"], s["path"],
                         s["n_path"], s["lens_out"])


def _outputs(s):
    if s["op"] == "plan":
        return _plan_outputs(s)
    if s["op"] == "slots":
        return s["q_out"], s["k_pool"], s["v_pool"]
    if s["op"] == "tree":
        return s["out"]
    return s["k_pools"], s["v_pools"], s["lens_out"]


def run(state):
    if own:
        _own_run(state)
    else:
        {"plan": _plain_plan, "slots": _plain_slots, "tree": _plain_tree, "commit": _plain_commit}[state["op"]](state)
    return _outputs(state)


# ---------------------------------------------------------------------------- work
def work(case):
    c = case
    B = c["B"]
    if c["op"] == "plan":
        n = B * (c["rows_lo"] + c["rows_hi"]) / 2
        blocks = n / c["bs"] + B * c["finished"] * c["hist"] / 2 / c["bs"]
        words = (c["rows_hi"] + 63) // 64
        return {"bytes": 20 * B + 8 * blocks + n * (12 + c["tree"] * (4 + 8 * words)), "flops": 0}
    es = 2 if c["dtype"] == "bf16" else 4
    Hkv, d = c["Hkv"], c["d"]
    if c["op"] == "slots":
        n, H = B * (c["rows_lo"] + c["rows_hi"]) / 2, c["H"]
        return {"bytes": 2 * n * (H + 2 * Hkv) * d * es + 12 * n, "flops": n * (H + Hkv) * (4 * d * c["norm"] + 3 * c["rot"])}
    if c["op"] == "tree":
        H, n, hist = c["H"], B * (c["rows_lo"] + c["rows_hi"]) / 2, (c["hist_lo"] + c["hist"]) / 2
        keys = B * hist + n
        depth = math.log(max(2, c["rows_hi"]))  # rows of the tree that a row sees
        return {"bytes": keys * Hkv * d * 2 * es + 2 * n * H * d * es + 8 * n * ((c["rows_hi"] + 63) // 64),
                "flops": 4 * n * (hist + depth) * H * d}
    return {"bytes": 2 * B * c["most"] / 2 * c["layers"] * Hkv * d * 2 * es / 2 + 8 * B, "flops": 0}


# ---------------------------------------------------------------------------- 64 bits
def _exact_rows(c, x, w, positions, freq):
    """The definition, in 64 bits, by complex numbers: each pair is one number, turned by e^(i angle)."""
    y = x.double()
    if w is not None:
        y = y * w.double() * torch.rsqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + 1e-6)
    rot = c["rot"]
    first = torch.arange(rot // 2, device="cuda") * (1 if c["layout"] == "half" else 2)
    second = first + (rot // 2 if c["layout"] == "half" else 1)
    z = torch.complex(y[..., first], y[..., second]) * torch.exp(1j * (positions.double().unsqueeze(-1) * freq)).unsqueeze(-2)
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    global own
    c, kept = case, own
    if c["op"] == "plan":
        return None  # whole numbers
    own = False  # the inputs are the same on both sides; no handle of the framework is wanted here
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if c["op"] == "slots":
        q_out, kp, vp = s["q_out"].double(), s["k_pool"].double(), s["v_pool"].double()
        real = torch.nonzero(s["slots"] >= 0)[:, 0]
        block, row = s["slots"][real] // c["bs"], s["slots"][real] % c["bs"]
        q_out[real] = _exact_rows(c, s["q"][real], s["wq"], s["positions"][real], s["freq"])
        kp[block, :, row] = _exact_rows(c, s["k"][real], s["wk"], s["positions"][real], s["freq"])
        vp[block, :, row] = s["v"][real].double()
        return q_out, kp, vp
    if c["op"] == "tree":
        out, G = s["out"].double(), c["H"] // c["Hkv"]
        starts, words = s["row_starts"].tolist(), s["mask"].cpu().tolist()
        for b, hist in enumerate(s["lens"].tolist()):
            n = starts[b + 1] - starts[b]
            if n == 0:
                continue
            block = s["tables"][b, :-(-(hist + n) // c["bs"])].long()
            seen = torch.ones(n, hist + n, dtype=torch.bool)
            for i in range(n):
                bits = sum((w % (1 << 64)) << (64 * x) for x, w in enumerate(words[starts[b] + i]))
                seen[i, hist:] = torch.tensor([bits >> j & 1 for j in range(n)], dtype=torch.bool)
            seen = seen.cuda()
            for h in range(c["Hkv"]):
                k = s["k_pool"][block, h].reshape(-1, c["d"])[:hist + n].double()
                v = s["v_pool"][block, h].reshape(-1, c["d"])[:hist + n].double()
                q = s["q"][starts[b]:starts[b + 1], h * G:(h + 1) * G].double()
                score = torch.einsum("ngd,kd->ngk", q, k) / math.sqrt(c["d"])
                weight = torch.softmax(score.masked_fill(~seen[:, None], float("-inf")), -1)
                out[starts[b]:starts[b + 1], h * G:(h + 1) * G] = torch.einsum("ngk,kd->ngd", weight, v)
        return out
    k, v = s["k_pools"].double(), s["v_pools"].double()
    path, n_path, tables = s["path"].tolist(), s["n_path"].tolist(), s["tables"].tolist()
    for b, hist in enumerate(s["lens_in"].tolist()):
        for j in range(n_path[b]):
            to, of = hist + j, hist + path[b][j]
            for pools in (k, v):
                pools[:, tables[b][to // c["bs"]], :, to % c["bs"]] = pools[:, tables[b][of // c["bs"]], :, of % c["bs"]].clone()
    return k, v, s["lens_in"] + s["n_path"]
