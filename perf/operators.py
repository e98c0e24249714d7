"""Cases, plain forms and 64-bit values of the long-context operators over an MLA latent KV pool.

Five operators are measured, two families that read and write the same page_size=1 pool and slot tables
as verify attention (rows of 576 bf16 values: 512 latent + 64 rope dims, one KV head):

  keeping a cache small
    weight    accumulated attention weight of every prefix key over (accepted) tree nodes
    evict     keep each request's heaviest positions, rewrite its slot table, list the freed slots
  reading a long cache sparsely
    summary   8-bit means of consecutive blocks of prefix rows
    select    per tree node, the blocks of the best cheap score (integer dot products)
    blocks    tree attention over each node's selected blocks, its ancestors and itself

`run` computes an operator in elementary torch operations where `own` is false, and calls the framework
where it is true.
"""
import math

import torch

own = False

D_QK, D_V = 576, 512
SM_SCALE = 1.0 / math.sqrt(192.0)


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: one short request, all nodes of a 9-node tree
        dict(name="weight_short", op="weight", batch=1, min_len=256, max_len=256, nodes=9, heads=16, chosen=0,
             pool=4096, slots="perm", decay=0.0),
        # one long conversation after a verify step: the 5 accepted nodes of a chain of 9 add their weights
        dict(name="weight_accepted_185k", op="weight", batch=1, min_len=185000, max_len=185000, nodes=9, heads=16,
             chosen=5, pool=1 << 20, slots="perm", decay=0.9),
        # every node of a wide tree with 128 heads: the most arithmetic
        dict(name="weight_tree_65k", op="weight", batch=1, min_len=65536, max_len=65536, nodes=65, heads=128,
             chosen=0, pool=1 << 18, slots="runs", decay=0.0),
        # one long request cut to a budget
        dict(name="evict_185k", op="evict", batch=1, min_len=185000, max_len=185000, keep=0.25, sink=4, recent=512),
        # a serving batch of mixed lengths cut at once
        dict(name="evict_batch", op="evict", batch=64, min_len=4096, max_len=131072, keep=0.5, sink=4, recent=256),
        # after prefill: every block of one long request
        dict(name="summary_185k", op="summary", batch=1, min_len=185000, max_len=185000, block=64, fresh=0,
             pool=1 << 20, slots="perm"),
        # after a decode step: only the blocks that the last accepted tokens touch
        dict(name="summary_step", op="summary", batch=64, min_len=1000, max_len=32768, block=64, fresh=5,
             pool=1 << 21, slots="runs"),
        # a batch of trees picks 32 blocks of 64 positions for each node
        dict(name="select_batch", op="select", batch=8, min_len=4096, max_len=131072, nodes=33, heads=16, block=64,
             topk=32, first=1, last=2),
        # one long request with small blocks
        dict(name="select_185k", op="select", batch=1, min_len=185000, max_len=185000, nodes=9, heads=16, block=16,
             topk=128, first=1, last=4),
        # plain decoding, one token a request, few blocks: latency counts
        dict(name="blocks_decode", op="blocks", batch=16, min_len=2000, max_len=32768, nodes=1, heads=16, block=32,
             topk=32, pool=1 << 19, slots="runs"),
        # a batch of trees, 2048 positions a node out of up to 131072
        dict(name="blocks_batch", op="blocks", batch=8, min_len=4096, max_len=131072, nodes=33, heads=16, block=64,
             topk=32, pool=1 << 20, slots="runs"),
        # a wide tree with 128 heads
        dict(name="blocks_heads128", op="blocks", batch=1, min_len=65536, max_len=65536, nodes=65, heads=128,
             block=64, topk=32, pool=1 << 18, slots="perm"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weight", "evict", "summary", "select", "blocks"])
    slots = rng.choice(["perm", "runs"])
    if op == "weight":
        while True:
            batch, hi, nodes, heads = rng.randint(1, 8), _log_int(rng, 64, 131072), rng.randint(1, 65), rng.choice(
                [1, 8, 16, 24, 64, 128])
            if batch * hi * nodes * heads <= 65536 * 65 * 128 // 2 and batch * hi <= 400000:
                break
        return dict(op=op, batch=batch, min_len=max(1, hi // rng.randint(1, 8)), max_len=hi, nodes=nodes, heads=heads,
                    chosen=rng.choice([0, rng.randint(1, nodes)]), pool=batch * hi + 4096, slots=slots,
                    decay=rng.choice([0.0, 0.5, 1.0]))
    if op == "evict":
        hi = _log_int(rng, 64, 131072)
        return dict(op=op, batch=rng.randint(1, 64), min_len=max(1, hi // rng.randint(1, 32)), max_len=hi,
                    keep=rng.uniform(0.05, 1.05), sink=rng.randint(0, 16), recent=rng.randint(0, 512))
    block = rng.choice([16, 32, 64, 128])
    if op == "summary":
        batch, hi = rng.randint(1, 32), _log_int(rng, 64, 131072)
        batch = max(1, min(batch, 400000 // hi))
        return dict(op=op, batch=batch, min_len=max(1, hi // rng.randint(1, 8)), max_len=hi, block=block,
                    fresh=rng.choice([0, rng.randint(1, 200)]), pool=batch * hi + 4096, slots=slots)
    batch, nodes, heads = rng.randint(1, 16), rng.randint(1, 65), rng.choice([1, 8, 16, 24, 64, 128])
    hi, topk = _log_int(rng, 64, 131072), _log_int(rng, 2, 2048 // block)
    if op == "select":
        batch = max(1, min(batch, int(4e8) // max(1, nodes * heads * (hi // block + 1))))
        return dict(op=op, batch=batch, min_len=max(1, hi // rng.randint(1, 8)), max_len=hi, nodes=nodes, heads=heads,
                    block=block, topk=topk, first=rng.randint(0, 2), last=rng.randint(0, 2))
    batch = max(1, min(batch, 400000 // hi, 600 // nodes, 12000 // (nodes * heads)))
    return dict(op=op, batch=batch, min_len=max(1, hi // rng.randint(1, 8)), max_len=hi, nodes=nodes, heads=heads,
                block=block, topk=topk, pool=batch * hi + batch * nodes + 4096, slots=slots)


def _lengths(case, gen):
    lo, hi, n = case["min_len"], case["max_len"], case["batch"]
    lens = torch.randint(lo, hi + 1, (n,), generator=gen)
    lens[0] = hi
    return lens.to(torch.int32)


# ----------------------------------------------------------------------------- inputs

def _slot_order(pool, kind, gen):
    """An order of the pool's slots 1.. : scattered ("perm"), or runs of about 64 consecutive slots ("runs")."""
    if kind == "perm":
        return torch.randperm(pool - 1, generator=gen, device="cuda") + 1
    run = (torch.rand(pool - 1, generator=gen, device="cuda") < 1.0 / 64).cumsum(0)
    key = torch.rand(pool, generator=gen, device="cuda")[run]
    return torch.argsort(key, stable=True) + 1


def _pool_inputs(case, gen, lens, nodes):
    """Pool, slot table and tree slots of one batch; every row N(0, 1) in bf16."""
    batch, stride, pool = case["batch"], case["max_len"], case["pool"]
    order = _slot_order(pool, case["slots"], gen).to(torch.int32)
    start = torch.cumsum(lens, 0) - lens
    pos = torch.arange(stride)
    at = (start[:, None] + pos[None, :]).clamp_(max=pool - 2)
    slot_idx = order[at.cuda()]
    slot_idx[(pos[None, :] >= lens[:, None]).cuda()] = 0
    used = int(lens.sum())
    tree_slots = order[used:used + batch * nodes].reshape(batch, nodes) if nodes else None
    kv = torch.randn(pool, D_QK, dtype=torch.bfloat16, device="cuda", generator=gen)
    return kv, slot_idx.contiguous(), tree_slots


def _tree(batch, nodes, host):
    """Random parents in topological order, at most four children each."""
    parent = torch.full((batch, nodes), -1, dtype=torch.int32)
    for b in range(batch):
        kids = [0] * nodes
        for i in range(1, nodes):
            p = int(torch.randint(0, i, (1,), generator=host))
            while kids[p] >= 4:
                p = (p + 1) % i
            kids[p] += 1
            parent[b, i] = p
    return parent


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed + 1)
    lens = _lengths(case, host)
    op, batch, stride = case["op"], case["batch"], case["max_len"]
    s = dict(case=case, prefix_len=lens.cuda())
    if op in ("weight", "select", "blocks"):
        nodes, heads = case["nodes"], case["heads"]
        s["q"] = torch.randn(batch, nodes, heads, D_QK, dtype=torch.bfloat16, device="cuda", generator=gen)
    if op in ("weight", "summary", "blocks"):
        s["kv"], s["slot_idx"], s["tree_slots"] = _pool_inputs(case, gen, lens, case.get("nodes", 0))
    if op == "weight":
        # the log-sum-exp that a verify call left, and the weights of the steps before
        k = s["kv"][s["slot_idx"].long()].float()
        qf = s["q"].float().reshape(batch, nodes * heads, D_QK)
        sc = torch.baddbmm(torch.zeros((), device="cuda"), qf, k.transpose(1, 2), beta=0, alpha=SM_SCALE)
        live = torch.arange(stride, device="cuda")[None, :] < s["prefix_len"][:, None]
        sc.masked_fill_(~live[:, None, :], -math.inf)
        s["lse"] = (torch.logsumexp(sc, -1) + 0.05).reshape(batch, nodes, heads).contiguous()
        del sc, k
        s["old"] = torch.rand(batch, stride, device="cuda", generator=gen).pow_(8)
        s["out"] = torch.zeros(batch, stride, device="cuda")
        s["chosen"] = None
        if case["chosen"]:
            pick = torch.stack([torch.randperm(nodes, generator=host)[:case["chosen"]] for _ in range(batch)])
            s["chosen"] = pick.sort(-1).values.to(torch.int32).cuda()
    elif op == "evict":
        # accumulated weights have a heavy tail
        s["weight"] = torch.rand(batch, stride, device="cuda", generator=gen).pow_(8)
        s["slot_idx"] = torch.randint(1, 1 << 22, (batch, stride), generator=gen, device="cuda", dtype=torch.int32)
        s["keep"] = (lens.double() * case["keep"]).to(torch.int32).cuda()
        for name, like in (("slots_out", s["slot_idx"]), ("weight_out", s["weight"]), ("freed", s["slot_idx"])):
            s[name] = torch.zeros_like(like)
        s["len_out"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
    elif op == "summary":
        n = -(-stride // case["block"])
        s["from_len"] = (s["prefix_len"] - case["fresh"]).clamp_(min=0) if case["fresh"] else None
        s["summary"] = torch.zeros(batch, n, D_QK, dtype=torch.bfloat16, device="cuda")
        s["scale"] = torch.zeros(batch, n, device="cuda")
    elif op == "select":
        n = -(-stride // case["block"])
        mean = torch.randn(batch, n, D_QK, device="cuda", generator=gen) / math.sqrt(case["block"])
        s["scale"] = mean.abs().amax(-1) / 127
        s["summary"] = torch.round(mean / s["scale"][..., None]).clamp_(-127, 127).to(torch.bfloat16)
    elif op == "blocks":
        s["parent"] = _tree(batch, nodes, host).cuda()
        # nodes of one tree want mostly the same blocks: a score shared by the request plus the node's own
        block, topk = case["block"], case["topk"]
        n = -(-stride // block)
        score = torch.randn(batch, 1, n, device="cuda", generator=gen) + 0.5 * torch.randn(
            batch, nodes, n, device="cuda", generator=gen)
        there = -(-s["prefix_len"] // block)
        at = torch.arange(n, device="cuda")
        score.masked_fill_(at[None, None, :] >= there[:, None, None], -math.inf)
        score.masked_fill_(at[None, None, :] == there[:, None, None] - 1, math.inf)
        top = torch.full((batch, nodes, topk), -1, device="cuda", dtype=torch.long)
        got = score.topk(min(topk, n), -1)
        top[..., :min(topk, n)] = torch.where(got.values > -math.inf, got.indices, -1)
        big = torch.where(top < 0, n + 1, top).sort(-1).values
        s["block_idx"] = torch.where(big > n, -1, big).to(torch.int32).contiguous()
    if own:
        s["handle"] = _handle(case, s)
    return s


def _handle(case, s):
    """The object that a user's program keeps for one set of sizes."""
    from speculative_decoding_tree_05_gb300 import ddtree
    op, batch, stride = case["op"], case["batch"], case["max_len"]
    if op == "weight":
        return ddtree.KeyWeights(batch, case["nodes"], case["heads"], case["pool"], stride)
    if op == "select":
        return ddtree.BlockSelector(batch, case["nodes"], case["heads"], stride, case["block"], case["topk"],
                                    first=case["first"], last=case["last"])
    if op == "blocks":
        return ddtree.BlockVerifier(batch, case["nodes"], case["heads"], case["pool"], stride, case["block"],
                                    case["topk"])
    return torch.empty(1 << 20, dtype=torch.uint8, device="cuda")


# ----------------------------------------------------------------------------- one pass

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _own_weight(s):
    return s["handle"](s["q"], s["kv"], s["slot_idx"], s["prefix_len"], s["lse"], SM_SCALE, weight=s["old"],
                       decay=s["case"]["decay"], node_idx=s["chosen"], out=s["out"])


def _own_evict(s):
    from speculative_decoding_tree_05_gb300 import ddtree
    c = s["case"]
    slots, weight, length, freed = ddtree.kv_evict(
        s["weight"], s["slot_idx"], s["prefix_len"], s["keep"], sink=c["sink"], recent=c["recent"],
        slot_idx_out=s["slots_out"], weight_out=s["weight_out"], prefix_len_out=s["len_out"], freed=s["freed"],
        workspace=s["handle"])
    return dict(slot_idx=slots, weight=weight, prefix_len=length, freed=freed)


def _own_summary(s):
    from speculative_decoding_tree_05_gb300 import ddtree
    summary, scale = ddtree.block_summary(s["kv"], s["slot_idx"], s["prefix_len"], s["case"]["block"],
                                          from_len=s["from_len"], summary=s["summary"], scale=s["scale"],
                                          workspace=s["handle"])
    return dict(summary=summary, scale=scale)


def _own_select(s):
    return s["handle"](s["q"], s["summary"], s["scale"], s["prefix_len"])


def _own_blocks(s):
    out, lse = s["handle"](s["q"], s["kv"], s["slot_idx"], s["prefix_len"], s["parent"], s["tree_slots"],
                           s["block_idx"], SM_SCALE)
    return dict(out=out, lse=lse)


def _live(s, width):
    return torch.arange(width, device="cuda")[None, :] < s["prefix_len"][:, None]


def _plain_weight(s):
    c, b = s["case"], s["case"]["batch"]
    k = s["kv"][s["slot_idx"].long()].float()
    q, lse = s["q"], s["lse"]
    if s["chosen"] is not None:
        rows = torch.arange(b, device="cuda")[:, None]
        q, lse = q[rows, s["chosen"].long()], lse[rows, s["chosen"].long()]
    sc = torch.baddbmm(-lse.reshape(b, -1, 1), q.float().reshape(b, -1, D_QK), k.transpose(1, 2), alpha=SM_SCALE)
    add = sc.exp_().sum(1)
    if c["decay"]:
        add = add + c["decay"] * s["old"]
    return torch.where(_live(s, c["max_len"]), add, s["out"])


def _ranked(score, there, first, last, keep):
    """Mask of the `keep` best of the first `there` entries of each row: entries before `first` and from
    there - last on before all others, then the larger score, then the lower index; NaN ranks lowest."""
    n = score.shape[-1]
    at = torch.arange(n, device="cuda")
    there = there[..., None].expand(score.shape[:-1] + (1,))
    key = torch.nan_to_num(score.double(), nan=-1e300, posinf=1e300, neginf=-1e300)
    key = torch.where((at < first) | (at >= there - last), math.inf, key)
    key = torch.where(at < there, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order).contiguous())
    return (rank < keep[..., None]) & (at < there)


def _plain_evict(s):
    c, n = s["case"], s["case"]["max_len"]
    live = _live(s, n)
    keep = _ranked(s["weight"], s["prefix_len"], c["sink"], c["recent"], s["keep"])
    gone = live & ~keep

    def pack(mask, values, into):
        to = torch.where(mask, mask.cumsum(1) - 1, n)
        wide = torch.cat([into, into[:, :1]], 1)
        return wide.scatter(1, to, torch.where(mask, values, wide[:, n:]))[:, :n].contiguous()
    return dict(slot_idx=pack(keep, s["slot_idx"], s["slots_out"]), weight=pack(keep, s["weight"], s["weight_out"]),
                prefix_len=keep.sum(1).to(torch.int32), freed=pack(gone, s["slot_idx"], s["freed"]))


def _plain_summary(s):
    c, block, b = s["case"], s["case"]["block"], s["case"]["batch"]
    n = s["scale"].shape[1]
    wide = n if s["from_len"] is None else min(n, (c["fresh"] + block - 1) // block + 1)
    start = torch.zeros_like(s["prefix_len"]) if s["from_len"] is None else s["from_len"] // block
    blk = start.long()[:, None] + torch.arange(wide, device="cuda")
    pos = blk[..., None] * block + torch.arange(block, device="cuda")
    live = pos < s["prefix_len"][:, None, None]
    slot = s["slot_idx"].long().gather(1, pos.clamp(max=c["max_len"] - 1).reshape(b, -1)).reshape(pos.shape)
    rows = s["kv"][slot].double() * live[..., None]
    count = live.sum(-1)
    mean = (rows.sum(2) / count.clamp(min=1)[..., None]).float()
    scale = mean.abs().amax(-1) / 127
    whole = torch.round(mean / scale[..., None]).nan_to_num_(0.0).clamp_(-127, 127).to(torch.bfloat16)
    here = count > 0
    at = torch.where(here, blk, n)
    summary = torch.cat([s["summary"], s["summary"][:, :1]], 1)
    scales = torch.cat([s["scale"], s["scale"][:, :1]], 1)
    summary = summary.scatter(1, at[..., None].expand(-1, -1, D_QK), torch.where(here[..., None], whole, 0))
    scales = scales.scatter(1, at, torch.where(here, scale, 0))
    return dict(summary=summary[:, :n].contiguous(), scale=scales[:, :n].contiguous())


def _plain_select(s):
    c, b = s["case"], s["case"]["batch"]
    q = s["q"].float().reshape(b, -1, D_QK)
    q_scale = q.abs().amax(-1, keepdim=True) / 127
    whole = torch.round(q / q_scale).nan_to_num_(0.0).clamp_(-127, 127)
    dots = torch.bmm(whole, s["summary"].float().transpose(1, 2))  # integers below 2^24: exact in 32 bits
    score = (dots * q_scale).reshape(b, c["nodes"], c["heads"], -1).amax(2) * s["scale"][:, None, :]
    there = (-(-s["prefix_len"] // c["block"]))[:, None].expand(-1, c["nodes"])
    keep = torch.full_like(there, c["topk"])
    picked = _ranked(score, there, c["first"], c["last"], keep)
    n = picked.shape[-1]
    at = torch.where(picked, torch.arange(n, device="cuda"), n).sort(-1).values
    at = torch.cat([at, torch.full((b, c["nodes"], c["topk"]), n, device="cuda")], -1)[..., :c["topk"]]
    return torch.where(at < n, at, -1).to(torch.int32)


def _plain_blocks(s):
    c = s["case"]
    b, nodes, heads, block = c["batch"], c["nodes"], c["heads"], c["block"]
    idx = s["block_idx"].long()
    pos = (idx[..., None] * block + torch.arange(block, device="cuda")).reshape(b, nodes, -1)
    seen = (pos >= 0) & (pos < s["prefix_len"][:, None, None])
    slot = s["slot_idx"].long().gather(1, pos.clamp(0, c["max_len"] - 1).reshape(b, -1)).reshape(pos.shape)
    k = s["kv"][slot].float()
    tree = s["kv"][s["tree_slots"].long()].float()
    link = (s["parent"].long()[..., None] == torch.arange(nodes, device="cuda")).double()
    path = torch.matrix_power(link + torch.eye(nodes, device="cuda", dtype=torch.float64), nodes) > 0
    q = s["q"].float() * SM_SCALE
    sc = torch.cat([(q @ k.transpose(2, 3)).masked_fill_(~seen[:, :, None], -math.inf),
                    (q @ tree[:, None].transpose(2, 3)).masked_fill_(~path[:, :, None], -math.inf)], -1)
    top = sc.amax(-1, keepdim=True)
    p = (sc - top).exp_()
    total = p.sum(-1, keepdim=True)
    n = pos.shape[-1]
    out = (p[..., :n] @ k[..., :D_V] + p[..., n:] @ tree[:, None, :, :D_V]) / total
    return dict(out=out.to(torch.bfloat16), lse=(top + total.log())[..., 0])


_OWN = dict(weight=_own_weight, evict=_own_evict, summary=_own_summary, select=_own_select, blocks=_own_blocks)
_PLAIN = dict(weight=_plain_weight, evict=_plain_evict, summary=_plain_summary, select=_plain_select,
              blocks=_plain_blocks)


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op, b = case, case["op"], case["batch"]
    # mixed lengths are uniform between min_len and max_len, the first one max_len
    keys = c["max_len"] + (b - 1) * (c["min_len"] + c["max_len"]) / 2
    if op == "weight":
        rows = (c["chosen"] or c["nodes"]) * c["heads"]
        return dict(bytes=keys * (D_QK * 2 + 4 + 4 + (4 if c["decay"] else 0)) + b * rows * (D_QK * 2 + 4),
                    flops=keys * rows * (2 * D_QK + 4))
    if op == "evict":
        return dict(bytes=keys * 8 + keys * min(1.0, c["keep"]) * 8 + keys * max(0.0, 1 - c["keep"]) * 4,
                    flops=keys * 2)
    if op == "summary":
        rows = min(keys, b * (c["fresh"] + c["block"] / 2)) if c["fresh"] else keys
        return dict(bytes=rows * (D_QK * 2 + 4) + rows / c["block"] * (D_QK * 2 + 4), flops=rows * D_QK)
    n = keys / c["block"]
    if op == "select":
        rows = c["nodes"] * c["heads"]
        return dict(bytes=n * (D_QK * 2 + 4) + b * rows * D_QK * 2 + b * c["nodes"] * c["topk"] * 4,
                    flops=n * rows * 2 * D_QK)
    # rows of the union of a request's lists are read once at least; half of the blocks are taken to be shared
    picked = min(keys, b * c["topk"] * c["block"])
    pairs = picked * c["nodes"] * c["heads"]
    rows = b * c["nodes"] * c["heads"]
    return dict(bytes=picked * (D_QK * 2 + 4) + rows * (D_QK * 2 + D_V * 2 + 4), flops=pairs * 2 * (D_QK + D_V))


# ----------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, op, b = case, case["op"], case["batch"]
    lens = s["prefix_len"].tolist()
    if op == "weight":
        w = s["out"].double()
        for i in range(b):
            n = lens[i]
            picks = range(c["nodes"]) if s["chosen"] is None else s["chosen"][i].tolist()
            k = s["kv"][s["slot_idx"][i, :n].long()].double()
            total = c["decay"] * s["old"][i, :n].double() if c["decay"] else torch.zeros(n, device="cuda").double()
            for t in picks:
                total = total + torch.exp(SM_SCALE * (k @ s["q"][i, t].double().T) - s["lse"][i, t].double()).sum(1)
            w[i, :n] = total
        return w
    if op == "evict":
        return dict(slot_idx=None, weight=_exact_evict(s, c, lens), prefix_len=None, freed=None)
    if op == "summary":
        return dict(summary=None, scale=_exact_scale(s, c, lens))
    if op == "select":
        return None
    out = torch.empty(b, c["nodes"], c["heads"], D_V, dtype=torch.float64, device="cuda")
    lse = torch.empty(b, c["nodes"], c["heads"], dtype=torch.float64, device="cuda")
    for i in range(b):
        parent, table = s["parent"][i].tolist(), s["slot_idx"][i].long()
        for t in range(c["nodes"]):
            pos = [p for blk in s["block_idx"][i, t].tolist() if blk >= 0
                   for p in range(blk * c["block"], min(lens[i], (blk + 1) * c["block"]))]
            up, u = [], t
            while u >= 0:
                up.append(u)
                u = parent[u]
            slots = torch.cat([table[torch.tensor(pos, dtype=torch.long, device="cuda")],
                               s["tree_slots"][i][torch.tensor(up, device="cuda")].long()])
            k = s["kv"][slots].double()
            sc = SM_SCALE * (s["q"][i, t].double() @ k.T)
            lse[i, t] = torch.logsumexp(sc, -1)
            out[i, t] = torch.softmax(sc, -1) @ k[:, :D_V]
    return dict(out=out, lse=lse)


def _exact_evict(s, c, lens):
    kept = s["weight_out"].double()
    for i, n in enumerate(lens):
        w = s["weight"][i, :n].tolist()
        held = set(range(min(n, c["sink"]))) | set(range(max(0, n - c["recent"]), n))
        best = sorted(range(n), key=lambda j: (j not in held, -w[j] if j not in held else 0.0, j))
        stay = sorted(best[:int(s["keep"][i])])
        kept[i, :len(stay)] = torch.tensor([w[j] for j in stay], dtype=torch.float64)
    return kept


def _exact_scale(s, c, lens):
    scale = s["scale"].double()
    for i, n in enumerate(lens):
        first = 0 if s["from_len"] is None else int(s["from_len"][i]) // c["block"]
        for j in range(first, -(-n // c["block"])):
            rows = s["kv"][s["slot_idx"][i, j * c["block"]:min(n, (j + 1) * c["block"])].long()].double()
            scale[i, j] = rows.mean(0).abs().max() / 127
    return scale
