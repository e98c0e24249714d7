"""Cases, plain forms and 64-bit values of the 8-bit latent cache and of draft-tree verification.

Four operators are measured. Three keep the page_size=1 latent cache in 8 bits: a slot holds 512 latent values in
e4m3 and 64 rope values in bf16, both divided by a power of two of the slot (640 bytes and an fp32 scale).

  store     rows are normalised, rotated to their positions, quantised and scattered to their slots, and read back
  load      rows of listed slots, read back as bf16
  attend    tree verify attention over the 8-bit cache: prefix, ancestors and the node itself
  accept    the drafted tokens of a tree against the target's probabilities, from given random numbers: the accepted
            path and the next token

`run` computes an operator in elementary torch operations where `own` is false, and calls the framework
where it is true.
"""
import math

import torch

own = False

D_QK, D_V, D_ROPE, ROW = 576, 512, 64, 640
SM_SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # the rows of one verify step: 16 requests with chains of 9 drafted tokens
        dict(name="store_step", op="store", rows=144, pool=1 << 18, norm=True, rotate="halves", slots="perm"),
        # a prompt's rows, an odd number of them
        dict(name="store_prompt", op="store", rows=60001, pool=1 << 18, norm=True, rotate="pairs", slots="runs"),
        # a short prefix that another layer needs in bf16
        dict(name="load_short", op="load", rows=4097, pool=1 << 18, slots="runs"),
        # one long conversation, scattered over the pool
        dict(name="load_185k", op="load", rows=185000, pool=1 << 20, slots="perm"),
        # the smallest call: one short request, a chain of 9 nodes
        dict(name="attend_short", op="attend", batch=1, min_len=256, max_len=256, nodes=9, heads=16, pool=4096,
             slots="perm", tree="chain", ragged=False),
        # plain decoding, one token a request
        dict(name="attend_decode", op="attend", batch=16, min_len=1024, max_len=32768, nodes=1, heads=16,
             pool=1 << 20, slots="perm", tree="random", ragged=False),
        # one long conversation
        dict(name="attend_185k", op="attend", batch=1, min_len=185000, max_len=185000, nodes=9, heads=16,
             pool=1 << 20, slots="perm", tree="chain", ragged=False),
        # a serving batch of mixed lengths, trees of 1 to 33 nodes
        dict(name="attend_batch", op="attend", batch=8, min_len=4096, max_len=131072, nodes=33, heads=16,
             pool=1 << 20, slots="runs", tree="random", ragged=True),
        # a wide tree with 128 heads: the most arithmetic
        dict(name="attend_heads128", op="attend", batch=1, min_len=65536, max_len=65536, nodes=65, heads=128,
             pool=1 << 18, slots="perm", tree="random", ragged=False),
        # one request, a chain of 9, the drafter's best tokens
        dict(name="accept_chain", op="accept", batch=1, nodes=9, vocab=32768, type="bf16", drafted="best",
             tree="chain", temperature=1.0),
        # 8 requests with wide trees over a large vocabulary
        dict(name="accept_batch", op="accept", batch=8, nodes=65, vocab=131072, type="bf16", drafted="best",
             tree="random", temperature=0.7),
        # drafted tokens that were drawn from the drafter's own distribution; an odd vocabulary
        dict(name="accept_drawn", op="accept", batch=16, nodes=9, vocab=128001, type="fp32", drafted="drawn",
             tree="random", temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "load", "attend", "attend", "accept"])
    slots, tree = rng.choice(["perm", "runs"]), rng.choice(["chain", "random"])
    if op in ("store", "load"):
        rows = _log_int(rng, 1, 60001 if op == "store" else 185000)
        case = dict(op=op, rows=rows, pool=rows + _log_int(rng, 2, 1 << 18), slots=slots)
        if op == "store":
            case.update(norm=rng.random() < 0.7, rotate=rng.choice(["halves", "pairs", "none"]))
        return case
    if op == "attend":
        heads = rng.choice([1, 8, 16, 24, 64, 128])
        while True:
            batch, hi, nodes = rng.randint(1, 32), _log_int(rng, 1, 185000), rng.randint(1, 65)
            if batch * hi <= 600000 and batch * hi * nodes * heads <= 65536 * 65 * 128 // 2:
                break
        return dict(op=op, batch=batch, min_len=hi // rng.randint(1, 16), max_len=hi, nodes=nodes, heads=heads,
                    pool=batch * hi + batch * nodes + 4096, slots=slots, tree=tree, ragged=rng.random() < 0.4)
    while True:
        batch, nodes, vocab = rng.randint(1, 32), rng.randint(1, 65), _log_int(rng, 100, 200000)
        if batch * nodes * vocab <= 30000000:
            break
    return dict(op=op, batch=batch, nodes=nodes, vocab=vocab, type=rng.choice(["bf16", "fp32"]),
                drafted=rng.choice(["best", "drawn"]), tree=tree, temperature=rng.choice([0.0, 0.5, 1.0, 1.3]))


# ----------------------------------------------------------------------------- inputs

def _lengths(case, gen):
    lens = torch.randint(case["min_len"], case["max_len"] + 1, (case["batch"],), generator=gen)
    lens[0] = case["max_len"]
    return lens.to(torch.int32)


def _slot_order(pool, kind, gen):
    """An order of the pool's slots 1.. : scattered ("perm"), or runs of about 64 consecutive slots ("runs")."""
    if kind == "perm":
        return torch.randperm(pool - 1, generator=gen, device="cuda") + 1
    run = (torch.rand(pool - 1, generator=gen, device="cuda") < 1.0 / 64).cumsum(0)
    key = torch.rand(pool, generator=gen, device="cuda")[run]
    return torch.argsort(key, stable=True) + 1


def _tree(batch, nodes, kind, host):
    """Parents in topological order: a chain, or random ones with at most four children each."""
    if kind == "chain":
        return torch.arange(-1, nodes - 1, dtype=torch.int32).expand(batch, nodes).contiguous()
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


def _cache(pool, gen):
    """A cache that has been written: normalised latent rows with a few large channels, rotated rope values."""
    gain = torch.exp(0.5 * torch.randn(D_V, device="cuda", generator=gen))
    store = torch.empty(pool, ROW, dtype=torch.uint8, device="cuda")
    scale = torch.empty(pool, device="cuda")
    for at in range(0, pool, 1 << 17):
        n = min(1 << 17, pool - at)
        row = torch.randn(n, D_QK, device="cuda", generator=gen)
        row[:, :D_V] *= gain
        s = torch.exp2(torch.ceil(torch.log2(row[:, :D_V].abs().amax(-1) / 448)))
        row /= s[:, None]
        store[at:at + n, :D_V] = row[:, :D_V].clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        store[at:at + n, D_V:] = row[:, D_V:].to(torch.bfloat16).view(torch.uint8).reshape(n, -1)
        scale[at:at + n] = s
    return store, scale


def _prepare_attend(case, gen, host):
    batch, stride, nodes, pool = case["batch"], case["max_len"], case["nodes"], case["pool"]
    lens = _lengths(case, host)
    order = _slot_order(pool, case["slots"], gen).to(torch.int32)
    start = torch.cumsum(lens, 0) - lens
    pos = torch.arange(stride)
    slot_idx = order[(start[:, None] + pos[None, :]).clamp_(max=pool - 2).cuda()]
    slot_idx[(pos[None, :] >= lens[:, None]).cuda()] = 0
    used = int(lens.sum())
    s = dict(case=case, prefix_len=lens.cuda(), slot_idx=slot_idx.contiguous(), tree_len=None)
    s["tree_slots"] = order[used:used + batch * nodes].reshape(batch, nodes).contiguous()
    s["parent"] = _tree(batch, nodes, case["tree"], host).cuda()
    if case["ragged"]:
        s["tree_len"] = torch.randint(1, nodes + 1, (batch,), generator=host).to(torch.int32).cuda()
    s["store"], s["scale"] = _cache(pool, gen)
    s["q"] = torch.randn(batch, nodes, case["heads"], D_QK, device="cuda", generator=gen).to(torch.bfloat16)
    if own:
        from speculative_decoding_tree_05_gb300 import ddtree
        s["handle"] = ddtree.Kv8Verifier(batch, nodes, case["heads"], pool, stride, prefix_len_sum=used)
    return s


def _prepare_accept(case, gen, host):
    b, t, v = case["batch"], case["nodes"], case["vocab"]
    logits = 2.5 * torch.randn(b, t, v, device="cuda", generator=gen)
    # a few tokens of each row are likely
    likely = torch.randint(0, v, (b, t, 6), device="cuda", generator=gen)
    logits.scatter_(2, likely, 9 + 4 * torch.rand(b, t, 6, device="cuda", generator=gen) + math.log(v) / 2)
    logits = logits.to(torch.bfloat16 if case["type"] == "bf16" else torch.float32)
    parent = _tree(b, t, case["tree"], host)
    up = parent.long().clamp(min=0).cuda()
    rows = torch.arange(b, device="cuda")[:, None]
    s = dict(case=case, logits=logits, parent=parent.cuda(), draft=None)
    if case["drafted"] == "best":
        # a node's children are the drafter's best tokens for it, the first child the best
        sib = torch.tensor([[int((parent[i, :j] == parent[i, j]).sum()) for j in range(t)] for i in range(b)])
        noisy = logits.gather(2, likely).float() + torch.randn(b, t, 6, device="cuda", generator=gen)
        best = likely.gather(2, noisy.argsort(-1, descending=True))
        s["tokens"] = best[rows, up, sib.cuda()].to(torch.int32)
    else:
        draft = torch.empty(b, t, v, device="cuda")
        for i in range(b):
            noise = 0.7 * torch.randn(t, v, device="cuda", generator=gen)
            draft[i] = torch.softmax(logits[i].float() + noise, -1)
        s["draft"] = draft
        u = torch.rand(b, t, device="cuda", generator=gen, dtype=torch.float64)
        token = torch.empty(b, t, dtype=torch.int32, device="cuda")
        for i in range(b):
            total = draft[i].double().cumsum(-1)[up[i]]
            token[i] = torch.searchsorted(total, (u[i] * total[:, -1])[:, None])[:, 0].clamp_(max=v - 1)
        s["tokens"] = token
    s["uniform"] = torch.rand(b, t, device="cuda", generator=gen)
    s["temperature"] = torch.full((b,), float(case["temperature"]), device="cuda")
    if own:
        from speculative_decoding_tree_05_gb300 import ddtree
        s["handle"] = ddtree.TreeAcceptor(b, t, v)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed + 1)
    if case["op"] == "attend":
        return _prepare_attend(case, gen, host)
    if case["op"] == "accept":
        return _prepare_accept(case, gen, host)
    n, pool = case["rows"], case["pool"]
    s = dict(case=case, slots=_slot_order(pool, case["slots"], gen)[:n].to(torch.int32).contiguous())
    if case["op"] == "load":
        s["store"], s["scale"] = _cache(pool, gen)
    else:
        s["rows"] = torch.randn(n, D_QK, device="cuda", generator=gen).mul_(3).to(torch.bfloat16)
        s["weight"] = s["table"] = s["position"] = None
        if case["norm"]:
            s["weight"] = torch.exp(0.5 * torch.randn(D_V, device="cuda", generator=gen)).to(torch.bfloat16)
        if case["rotate"] != "none":
            turn = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32).double() / 32)
            s["table"] = torch.cat([turn.cos(), turn.sin()], 1).float().cuda()
            s["position"] = torch.randperm(n, generator=host).to(torch.int32).cuda()
        s["store"] = torch.zeros(pool, ROW, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.ones(pool, device="cuda")
    s["back"] = torch.empty(n, D_QK, dtype=torch.bfloat16, device="cuda")
    return s


# ----------------------------------------------------------------------------- one pass

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _own_store(s):
    from speculative_decoding_tree_05_gb300 import ddtree
    ddtree.kv8_write(s["rows"], s["slots"], s["store"], s["scale"], norm_weight=s["weight"], eps=EPS,
                     rotation=s["table"], position=s["position"], interleaved=s["case"]["rotate"] == "pairs")
    return ddtree.kv8_read(s["store"], s["scale"], s["slots"], out=s["back"])


def _own_load(s):
    from speculative_decoding_tree_05_gb300 import ddtree
    return ddtree.kv8_read(s["store"], s["scale"], s["slots"], out=s["back"])


def _own_attend(s):
    out, lse = s["handle"](s["q"], s["store"], s["scale"], s["slot_idx"], s["prefix_len"], s["parent"],
                           s["tree_slots"], SM_SCALE, tree_len=s["tree_len"])
    return dict(out=out, lse=lse)


def _own_accept(s):
    path, length, token = s["handle"](s["logits"], s["tokens"], s["parent"], s["uniform"], s["temperature"],
                                      draft_prob=s["draft"])
    return dict(path=path, length=length, token=token)


def _read(s, slots):
    """The values that listed slots stand for, in 32 bits."""
    rows, scale = s["store"][slots], s["scale"][slots][..., None]
    latent = rows[..., :D_V].view(torch.float8_e4m3fn).float()
    return torch.cat([latent, rows[..., D_V:].view(torch.bfloat16).float()], -1) * scale


def _plain_load(s):
    return _read(s, s["slots"].long()).to(torch.bfloat16)


def _plain_store(s):
    c = s["case"]
    latent, rope = s["rows"][:, :D_V].double(), s["rows"][:, D_V:].double()
    if c["norm"]:
        latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
    if c["rotate"] != "none":
        turn = s["table"][s["position"].long()].double()
        cos, sin = turn[:, :32], turn[:, 32:]
        if c["rotate"] == "pairs":
            x, y = rope[:, 0::2], rope[:, 1::2]
            rope = torch.stack([x * cos - y * sin, y * cos + x * sin], -1).flatten(1)
        else:
            x, y = rope[:, :32], rope[:, 32:]
            rope = torch.cat([x * cos - y * sin, y * cos + x * sin], -1)
    # the smallest power of two by which the row's largest latent value stays within 448
    frac, power = torch.frexp(latent.abs().amax(-1))
    scale = torch.exp2((power - 9 + (frac > 0.875)).float())[:, None]
    slots = s["slots"].long()
    low = (latent / scale).float().to(torch.float8_e4m3fn).view(torch.uint8)
    high = (rope / scale).float().to(torch.bfloat16).view(torch.uint8)
    s["store"].index_copy_(0, slots, torch.cat([low, high], 1))
    s["scale"].index_copy_(0, slots, scale[:, 0])
    return _plain_load(s)


def _paths(parent):
    """[B, T, T] truth values: the second node is an ancestor of the first, or the first itself."""
    nodes = parent.shape[1]
    at = torch.arange(nodes, device="cuda")
    link = (parent.long()[..., None] == at).double() + torch.eye(nodes, device="cuda", dtype=torch.float64)
    return torch.matrix_power(link, nodes) > 0


def _plain_attend(s):
    c = s["case"]
    b, nodes, heads, n = c["batch"], c["nodes"], c["heads"], c["max_len"]
    k = _read(s, s["slot_idx"].long())
    tree = _read(s, s["tree_slots"].long())
    q = (s["q"].float() * SM_SCALE).reshape(b, nodes * heads, D_QK)
    seen = torch.arange(n, device="cuda")[None, :] < s["prefix_len"][:, None]
    path = _paths(s["parent"]).repeat_interleave(heads, 1)
    sc = torch.cat([(q @ k.transpose(1, 2)).masked_fill_(~seen[:, None], -math.inf),
                    (q @ tree.transpose(1, 2)).masked_fill_(~path, -math.inf)], -1)
    top = sc.amax(-1, keepdim=True)
    p = (sc - top).exp_()
    total = p.sum(-1, keepdim=True)
    out = ((p[..., :n] @ k[..., :D_V] + p[..., n:] @ tree[..., :D_V]) / total).reshape(b, nodes, heads, D_V)
    lse = (top + total.log()).reshape(b, nodes, heads)
    if s["tree_len"] is not None:
        gone = torch.arange(nodes, device="cuda")[None, :] >= s["tree_len"][:, None]
        out = out.masked_fill(gone[..., None, None], 0)
        lse = lse.masked_fill(gone[..., None], -math.inf)
    return dict(out=out.to(torch.bfloat16), lse=lse)


def _plain_accept(s):
    c = s["case"]
    b, t, v = c["batch"], c["nodes"], c["vocab"]
    rows = torch.arange(b, device="cuda")[:, None]
    at = torch.arange(t, device="cuda")
    if c["temperature"] > 0:
        w = s["logits"].double() / s["temperature"].double()[:, None, None]
        w = (w - w.amax(-1, keepdim=True)).exp_()
        w /= w.sum(-1, keepdim=True)
    else:
        best = s["logits"].float().eq(s["logits"].float().amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)
        w = torch.zeros(b, t, v, dtype=torch.float64, device="cuda").scatter_(2, best, 1.0)
    up, token, u = s["parent"].long().clamp(min=0), s["tokens"].long(), s["uniform"].double()
    child = (s["parent"][:, None, :] == at[:, None]) & (at > 0)          # [b, node, child]
    before = (s["parent"][:, :, None] == s["parent"][:, None, :]) & (at[None, :] < at[:, None]) & (at > 0)
    rank, kids = before.sum(-1), child.sum(-1)
    taken = torch.zeros(b, t, dtype=torch.bool, device="cuda")
    total = w.sum(-1)
    for r in range(int(kids.max())):   # siblings are tried one after the other
        here = (rank == r) & (at > 0)
        weight, left = w[rows, up, token], total.gather(1, up)
        if s["draft"] is None:
            taken |= here & (u * left < weight)
            hit = torch.where(here, token, v)
            wide = torch.cat([w, w[..., :1]], -1)
            wide[rows, up, hit] = 0
            w = wide[..., :v]
        else:
            taken |= here & (u * left * s["draft"][rows, up, token].double() < weight)
            less = (w - total[..., None] * s["draft"].double()).clamp_(min=0)
            some = (kids > r) & (less.sum(-1) > 0)
            w = torch.where(some[..., None], less, w)
        total = w.sum(-1)
    first = taken & ~(before & taken[:, None, :]).any(-1)
    on = (~_paths(s["parent"]) | (first | (at == 0))[:, None, :]).all(-1)
    last = torch.where(on, at, -1).amax(-1)
    path = torch.where(on, at, t).sort(-1).values
    w = w[rows[:, 0], last]
    sums = w.cumsum(-1)
    next_token = (sums <= u[:, :1] * sums[:, -1:]).sum(-1)
    return dict(path=torch.where(path < t, path, -1).to(torch.int32), length=on.sum(-1).to(torch.int32),
                token=next_token.to(torch.int32))


_OWN = dict(store=_own_store, load=_own_load, attend=_own_attend, accept=_own_accept)
_PLAIN = dict(store=_plain_store, load=_plain_load, attend=_plain_attend, accept=_plain_accept)


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "load":
        return dict(bytes=c["rows"] * (ROW + 4 + 4 + D_QK * 2), flops=c["rows"] * D_QK)
    if op == "store":  # and the reading back
        turn = 64 * 4 + 4 if c["rotate"] != "none" else 0
        return dict(bytes=c["rows"] * (2 * D_QK * 2 + 2 * (ROW + 4 + 4) + turn), flops=c["rows"] * D_QK * 6)
    if op == "attend":
        # mixed lengths are uniform between min_len and max_len, the first one max_len; trees too, if ragged
        b = c["batch"]
        keys = c["max_len"] + (b - 1) * (c["min_len"] + c["max_len"]) / 2
        nodes = (c["nodes"] + 1) / 2 if c["ragged"] else c["nodes"]
        rows = nodes * c["heads"]
        return dict(bytes=keys * (ROW + 4 + 4) + b * rows * (D_QK * 2 + 4 + D_V * 2) + b * nodes * (ROW + 12),
                    flops=keys * rows * 2 * (D_QK + D_V))
    # the rows of a path are wanted, and which they are turns out on the way: about half of a chain's, a tenth of a tree's
    nodes = 1 + (c["nodes"] - 1) * (0.5 if c["tree"] == "chain" else 0.1)
    size = (2 if c["type"] == "bf16" else 4) + (4 if c["drafted"] == "drawn" else 0)
    return dict(bytes=c["batch"] * nodes * c["vocab"] * size, flops=c["batch"] * nodes * c["vocab"] * 4)


# ----------------------------------------------------------------------------- the definitions in 64 bits

def _rounded(x, bits, lowest):
    """x to `bits` significant bits, halves to even, in steps of at least 2^lowest."""
    power = torch.frexp(x).exponent.double()
    step = torch.exp2(torch.clamp(power - bits, min=lowest))
    return torch.round(x / step) * step


def _values(s, slots):
    raw = s["store"][slots]
    byte = raw[..., :D_V].int()
    power, frac = (byte >> 3) & 15, (byte & 7).double()
    size = torch.where(power > 0, (1 + frac / 8) * torch.exp2((power - 7).double()), frac * 2.0 ** -9)
    latent = torch.where(byte >= 128, -size, size)
    pair = raw[..., D_V:].int().reshape(raw.shape[:-1] + (D_ROPE, 2))
    rope = ((pair[..., 0] << 16) | (pair[..., 1] << 24)).view(torch.float32).double()
    return torch.cat([latent, rope], -1) * s["scale"][slots].double()[..., None]


def exact(case, seed):
    if case["op"] == "accept":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "load":
        return _values(s, s["slots"].long())
    if case["op"] == "store":
        return _exact_store(s)
    b, nodes, heads = case["batch"], case["nodes"], case["heads"]
    if case["max_len"] * b * nodes * heads > 2e8:
        return None
    out = torch.zeros(b, nodes, heads, D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((b, nodes, heads), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["prefix_len"].tolist()
    for i in range(b):
        parent = s["parent"][i].tolist()
        k = _values(s, torch.cat([s["slot_idx"][i, :lens[i]], s["tree_slots"][i]]).long())
        for t in range(nodes if s["tree_len"] is None else int(s["tree_len"][i])):
            up, u = [], t
            while u >= 0:
                up.append(lens[i] + u)
                u = parent[u]
            keys = torch.cat([k[:lens[i]], k[torch.tensor(up, device="cuda")]])
            sc = SM_SCALE * (s["q"][i, t].double() @ keys.T)
            lse[i, t] = torch.logsumexp(sc, -1)
            out[i, t] = torch.softmax(sc, -1) @ keys[:, :D_V]
    return dict(out=out, lse=lse)


def _exact_store(s):
    c, x = s["case"], s["rows"].double()
    latent, rope = x[:, :D_V], x[:, D_V:].clone()
    if c["norm"]:
        latent = latent / torch.sqrt((latent * latent).sum(-1, keepdim=True) / D_V + EPS) * s["weight"].double()
    if c["rotate"] != "none":
        turn = s["table"][s["position"].long()].double()
        a = torch.arange(32, device="cuda")
        i, j = (2 * a, 2 * a + 1) if c["rotate"] == "pairs" else (a, a + 32)
        spin = torch.complex(rope[:, i], rope[:, j]) * torch.complex(turn[:, :32], turn[:, 32:])
        rope[:, i], rope[:, j] = spin.real, spin.imag
    scale = torch.exp2(torch.ceil(torch.log2(latent.abs().amax(-1, keepdim=True) / 448)))
    return torch.cat([_rounded(latent / scale, 4, -9), _rounded(rope / scale, 8, -133)], -1) * scale
