"""The drafted-token operators of the recurrent-state library, in their plain form and as calls of the library.

A serving program that drafts tokens keeps its sequences as slots of an fp32 state handle.  For each
sequence it has a tree of nodes: node 0 is the last token, whose state is not in the slot yet, the
others are drafted continuations; node j continues node parents[j] < j (-1: the slot's state).

  tree      the recurrence along every path of the trees: o_j = S_j q_j with S_j the state of node
            j's path, the slots left as they are;
  verify    the drafted nodes tested against the target model's probabilities from given uniform
            numbers (rejection by the ratio, then the residual for the next sibling), and one more
            token drawn where the walk ends;
  accept    the nodes of each accepted path written into the slot's state.

Per value head, S [dv, dk] fp32, q and k shared by heads/qk_heads value heads:
  S_j = alpha_j S_p + beta_j (v_j - delta alpha_j S_p k_j) k_j^T,   p the parent,   o_j = S_j q_j.
Verification at a node with target row p and draft row q, its children x_1, x_2, ... in order:
  P_1 = p, T_1 = Q_1 = 1, c_1 = 0;  x_i is taken if u T_i q(x_i) < P_i(x_i) Q_i, else
  c_i+1 = c_i + T_i / Q_i, P_i+1 = max(p - c_i+1 q, 0), T_i+1 its sum, and Q_i+1 = 1, or without
  replacement 1 - q(x_1) - ... - q(x_i).  Where no child is taken the next token is the first y
  whose cumulative sum of the last P exceeds u_next times the sum.  Drafts that come without
  probabilities are one-hot rows: x_i is taken if u T_i < P_i(x_i), else P_i+1 is P_i without
  x_i, and T_i+1 = T_i - P_i(x_i).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one user, three drafted tokens in a row: the launch counts
        dict(name="tree-one", op="tree", dtype="bf16", seqs=1, nodes=4, fewest=4, spread=0, heads=16,
             qk_heads=16, dk=128, dv=128, slots=8, delta=0, diag=0, recipe="gdn", fresh="none"),
        # a decode batch of a gated delta-rule layer with trees of up to 16 nodes
        dict(name="tree-batch-bf16", op="tree", dtype="bf16", seqs=64, nodes=16, fewest=6, spread=3,
             heads=32, qk_heads=16, dk=128, dv=128, slots=96, delta=1, diag=0, recipe="gdn", fresh="none"),
        # wide trees over many value heads for each key head
        dict(name="tree-wide-bf16", op="tree", dtype="bf16", seqs=32, nodes=64, fewest=40, spread=9,
             heads=64, qk_heads=8, dk=128, dv=64, slots=40, delta=0, diag=0, recipe="mamba2", fresh="none"),
        # fp32 activations and a decay for each key channel
        dict(name="tree-diag-f32", op="tree", dtype="f32", seqs=24, nodes=25, fewest=9, spread=4, heads=16,
             qk_heads=16, dk=128, dv=128, slots=24, delta=0, diag=1, recipe="gla", fresh="none"),
        # ragged trees of a small model, some sequences at their first token
        dict(name="tree-odd-f16", op="tree", dtype="f16", seqs=9, nodes=37, fewest=1, spread=5, heads=16,
             qk_heads=16, dk=64, dv=80, slots=32, delta=1, diag=0, recipe="la", fresh="some"),
        # the largest decode batch, a chain of eight tokens each
        dict(name="tree-large-bf16", op="tree", dtype="bf16", seqs=256, nodes=8, fewest=8, spread=0,
             heads=32, qk_heads=16, dk=128, dv=128, slots=256, delta=1, diag=0, recipe="gdn", fresh="none"),
        # one user's accepted tokens
        dict(name="accept-one", op="accept", dtype="bf16", seqs=1, nodes=4, fewest=4, depth=3, heads=16,
             qk_heads=16, dk=128, dv=128, slots=8, delta=0, diag=0, recipe="gdn", fresh="none"),
        # a decode batch of a gated delta-rule layer, one to five tokens accepted
        dict(name="accept-batch-bf16", op="accept", dtype="bf16", seqs=64, nodes=16, fewest=6, depth=5,
             heads=32, qk_heads=16, dk=128, dv=128, slots=96, delta=1, diag=0, recipe="gdn", fresh="some"),
        # the largest batch, fp32 activations and a decay for each key channel
        dict(name="accept-large-f32", op="accept", dtype="f32", seqs=256, nodes=8, fewest=8, depth=8,
             heads=32, qk_heads=32, dk=128, dv=128, slots=256, delta=0, diag=1, recipe="gla", fresh="none"),
        # one user: a chain of four drafted tokens behind the last one
        dict(name="verify-one", op="verify", seqs=1, nodes=5, fewest=5, spread=0, vocab=65536,
             drawn="with", depth=5),
        # a decode batch with trees, siblings drawn without replacement
        dict(name="verify-batch", op="verify", seqs=64, nodes=16, fewest=6, spread=3, vocab=131072,
             drawn="without", depth=8),
        # drafts that come without probabilities, an odd vocabulary
        dict(name="verify-given", op="verify", seqs=24, nodes=31, fewest=1, spread=4, vocab=50021,
             drawn="given", depth=31),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "accept", "verify"))
    nodes = rng.choice((_log(rng, 1, 64), rng.randint(1, 16)))
    fewest = rng.choice((nodes, max(1, nodes // 3), 1))
    spread = rng.choice((0, 2, 5, 9))
    if op == "verify":
        vocab = rng.choice((32000, 65536, 131072, rng.randint(1000, 131072)))
        # at most the bytes of the largest listed batch's rows
        seqs = _log(rng, 1, max(1, min(128, 64 * 16 * 131072 // (nodes * vocab))))
        return dict(op=op, seqs=seqs, nodes=nodes, fewest=fewest, spread=spread, vocab=vocab,
                    drawn=rng.choice(("with", "without", "given")), depth=rng.randint(1, nodes))
    dk = rng.choice((64, 128, 128))
    dv = rng.choice((64, 128, 128, rng.randint(16, 256)))
    heads = _log(rng, 1, 64)
    seqs = _log(rng, 1, max(1, min(256, 128 * 32 * 128 * 128 // (heads * dk * dv))))
    if op == "tree":                    # at most the work of the wide trees
        nodes = max(1, min(nodes, 32 * 64 * 64 * 64 * 128 // (seqs * heads * dv * dk)))
        fewest = min(fewest, nodes)
    diag = rng.choice((0, 0, 1))
    case = dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16", "f32")), seqs=seqs, nodes=nodes,
                fewest=fewest, heads=heads, qk_heads=max(d for d in (1, rng.randint(1, heads), heads) if heads % d == 0),
                dk=dk, dv=dv, slots=seqs + rng.randint(0, 40), delta=rng.choice((0, 1)), diag=diag,
                recipe="gla" if diag else rng.choice(("la", "gdn", "mamba2")), fresh=rng.choice(("none", "some")))
    if op == "tree":
        case["spread"] = spread
    else:
        case["depth"] = rng.randint(1, min(nodes, 16))
    return case


def _counts(case):
    """The trees' nodes: the largest first, the others spread evenly down to the smallest."""
    lo, hi = case["fewest"], case["nodes"]
    return [hi] + [lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, case["seqs"])]


def _accepted(case):
    """The accepted paths' lengths."""
    d = case["depth"]
    return [min(c, 1 + int(d * ((0.9 + i * 0.6180339887498949) % 1.0))) for i, c in enumerate(_counts(case))]


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _inputs(case, n, g):
    """q, k, v, alpha, beta of n nodes, distributed as the recurrent layers of each family make them."""
    d, f = "cuda", torch.float32
    h, hk, dk, dv, kind = case["heads"], case["qk_heads"], case["dk"], case["dv"], case["recipe"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=d, dtype=f)

    if kind == "mamba2":
        alpha = torch.exp(-0.1 * torch.nn.functional.softplus(normal(n, h) - 2.0))
        beta = torch.nn.functional.softplus(normal(n, h))
        # a delta rule wants beta |k|^2 below 2
        size = 4.0 * dk ** 0.5 if case["delta"] else dk ** 0.5
        q, k = normal(n, hk, dk) / dk ** 0.5, normal(n, hk, dk) / size
    else:
        q, k = _unit(normal(n, hk, dk)), _unit(normal(n, hk, dk))
        if kind == "gla":
            alpha = torch.sigmoid(3.0 + normal(n, h, dk))
        else:
            alpha = torch.sigmoid((4.0 if kind == "gdn" else 3.0) + 0.5 ** 0.5 * normal(n, h))
        beta = torch.sigmoid(normal(n, h))
    t = DTYPES[case["dtype"]]
    return q.to(t), k.to(t), normal(n, h, dv).to(t), alpha, beta


def _parents(case, r):
    """Node j continues one of the spread + 1 nodes before it."""
    out = []
    for n in _counts(case):
        out += [-1] + [max(0, j - 1 - r.randint(0, case["spread"])) for j in range(1, n)]
    return out


def _drafts(case, parents, counts, g, st):
    """Target rows, draft rows and drafted tokens.  A node's row is the distribution of its children;
    the draft model's logits are the target's with an error."""
    n, vocab = sum(counts), case["vocab"]
    logits = 2.5 * torch.randn((n, vocab), generator=g, device="cuda")
    st["target"] = logits.softmax(-1)
    logits += 0.6 * torch.randn((n, vocab), generator=g, device="cuda")
    # the r-th largest of logits and Gumbel noise is the r-th draw without replacement
    row, rank, start, most = [0] * n, [0] * n, 0, 1
    for c in counts:
        seen = {}
        for j in range(1, c):
            p = parents[start + j]
            row[start + j], rank[start + j] = start + p, seen.get(p, 0)
            seen[p] = seen.get(p, 0) + 1
            most = max(most, seen[p])
        start += c
    row = torch.tensor(row, device="cuda")
    rank = torch.tensor(rank, device="cuda")
    if case["drawn"] == "given":
        ids = logits.topk(most, -1).indices[row, rank]
    else:
        st["draft"] = logits.softmax(-1)
        u = torch.rand((n, vocab), generator=g, device="cuda").clamp_(min=1e-30)
        u.log_().neg_().log_().neg_()
        if case["drawn"] == "without":
            ids = u.add_(logits).topk(most, -1).indices[row, rank]
        else:
            ids = u.add_(logits[row]).argmax(-1)
        del u
    st["ids"] = ids.to(torch.int32)
    st["uniform"] = torch.rand(n, generator=g, device="cuda")
    st["uniform_next"] = torch.rand(case["seqs"], generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = random.Random(int(seed))
    st = {"case": case}
    m, counts = case["seqs"], _counts(case)
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] != "accept":
        parents = _parents(case, r)
        st["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    if case["op"] == "verify":
        st["draft"] = None
        _drafts(case, parents, counts, g, st)
        return st
    st["q"], st["k"], st["v"], st["alpha"], st["beta"] = _inputs(case, cu[-1], g)
    st["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:m].to(torch.int32)
    st["fresh"] = None if case["fresh"] == "none" else torch.rand(m, generator=g, device="cuda") < 0.4
    if case["op"] == "accept":
        path = torch.full((m, case["depth"]), -1, dtype=torch.int32)
        for i, (c, n) in enumerate(zip(counts, _accepted(case))):
            path[i, :n] = torch.tensor([0] + sorted(r.sample(range(1, c), n - 1)), dtype=torch.int32)
        st["path"] = path.cuda()
        st["lengths"] = torch.tensor(_accepted(case), dtype=torch.int32, device="cuda")
    # fp32 states as a running recurrence leaves them: rows and heads of different sizes
    pool = torch.randn((case["slots"] * case["heads"], case["dv"], case["dk"]), generator=g, device="cuda")
    pool *= torch.exp(torch.randn((case["slots"] * case["heads"], case["dv"], 1), generator=g, device="cuda") - 1.5)
    if own:                             # the handle that a serving program keeps, over the same values
        import quantized_recurrent_state_amd as lsq

        st["state"] = lsq.LsqState(lsq.LsqConfig(
            batch=case["slots"], heads=case["heads"], dk=case["dk"], dv=case["dv"], bits=32, group=1,
            policy=lsq.POLICY_NONE, delta=case["delta"], decay=case["diag"]))
        st["state"].f32.copy_(pool)
    else:
        st["pool"] = pool
    return st


def run(st):
    case = st["case"]
    if own:
        if case["op"] == "verify":
            import quantized_recurrent_state_amd as lsq

            path, lengths, token = lsq.verify_tree(
                st["target"], st["ids"], st["parents"], st["cu"], st["uniform"], st["uniform_next"],
                draft=st["draft"], replacement=case["drawn"] == "with", depth=case["depth"])
            return {"path": path, "lengths": lengths, "next": token}
        s = st["state"]
        if case["op"] == "tree":
            o = s.step_tree(st["q"], st["k"], st["v"], st["alpha"], st["beta"], st["cu"], st["parents"],
                            slots=st["slots"], fresh=st["fresh"], max_nodes=case["nodes"])
            return {"o": o}
        s.accept_path(st["k"], st["v"], st["alpha"], st["beta"], st["cu"], st["path"], st["lengths"],
                      slots=st["slots"], fresh=st["fresh"])
        return {"state": s.f32}
    if case["op"] == "verify":
        return _verify(st)
    if case["op"] == "tree":
        return {"o": _tree(st)}
    _accept(st)
    return {"state": st["pool"]}


# ---- the plain forms ---------------------------------------------------------------------------

def _initial(st, view):
    s = view[st["slots"].long()]
    return s if st["fresh"] is None else s * (~st["fresh"]).float()[:, None, None, None]


def _padded(st):
    """Row of node j of tree i, clamped, and whether there is one: [m, nodes]."""
    cu = st["cu"].long()
    pos = torch.arange(st["case"]["nodes"], device="cuda")
    live = pos[None] < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + pos[None]).clamp(max=st["parents"].shape[0] - 1), live


def _tree(st):
    c = st["case"]
    h, dk, dv, m, n = c["heads"], c["dk"], c["dv"], c["seqs"], c["nodes"]
    share = h // c["qk_heads"]
    at, live = _padded(st)
    parent = torch.where(live, st["parents"].long()[at], -1)
    # onto[b, j, i]: node i lies on the path to node j, both ends counted
    onto = torch.zeros((m, n + 1, n), dtype=torch.bool, device="cuda")       # row 0: before every tree
    each = torch.arange(m, device="cuda")
    for j in range(n):
        onto[:, j + 1] = onto[each, parent[:, j] + 1]
        onto[:, j + 1, j] = True
    onto = onto[:, 1:]

    def rows(x):                        # [tokens, heads, d] -> [m, h, nodes, d], zeros behind each tree
        x = x[at].float() * live[:, :, None, None]
        if x.shape[2] != h:
            x = x.repeat_interleave(share, dim=2)
        return x.transpose(1, 2).contiguous()

    q, k, v = rows(st["q"]), rows(st["k"]), rows(st["v"])
    beta = rows(st["beta"][:, :, None])
    alpha = st["alpha"] if c["diag"] else st["alpha"][:, :, None]
    la = torch.where(live[:, :, None, None], alpha[at].double().log(), 0.0).transpose(1, 2).contiguous()
    # sums of logarithms along the paths, in 64 bits: they are subtracted
    cum = torch.matmul(onto.double()[:, None], la)                           # [m, h, nodes, 1 or dk]
    g = cum.exp().float()
    view = st["pool"].view(c["slots"], h, dv, dk)
    s = _initial(st, view).transpose(-1, -2).contiguous()                    # [m, h, dk, dv]
    seen = torch.matmul(g * q, s)                                            # [m, h, nodes, dv]
    if c["diag"]:
        qk = torch.zeros((m, h, n, n), device="cuda")
        kk = torch.zeros((m, h, n, n), device="cuda") if c["delta"] else None
        for j in range(n):
            d = (cum[:, :, j:j + 1] - cum).masked_fill(~onto[:, j][:, None, :, None], float("-inf")).exp().float()
            d = d * k
            qk[:, :, j] = torch.matmul(d, q[:, :, j, :, None])[..., 0]
            if c["delta"]:
                kk[:, :, j] = torch.matmul(d, k[:, :, j, :, None])[..., 0]
    else:
        d = (cum - cum.transpose(-1, -2)).masked_fill(~onto[:, None], float("-inf")).exp().float()
        kt = k.transpose(-1, -2).contiguous()
        qk = torch.matmul(q, kt) * d
        kk = torch.matmul(k, kt) * d if c["delta"] else None
    w = v
    if c["delta"]:
        w = v - torch.matmul(g * k, s)
        for j in range(n):              # the writes of a node's ancestors come before its own
            if j:
                w[:, :, j] -= torch.matmul(kk[:, :, j, None, :j], w[:, :, :j])[:, :, 0]
            w[:, :, j] *= beta[:, :, j]
    else:
        w = v * beta
    o = seen + torch.matmul(qk, w)
    return o.transpose(1, 2)[live].to(st["q"].dtype)


def _accept(st):
    c = st["case"]
    share = c["heads"] // c["qk_heads"]
    pool = st["pool"].view(c["slots"], c["heads"], c["dv"], c["dk"])
    s = _initial(st, pool)
    start = st["cu"].long()[:-1]
    for t in range(c["depth"]):
        live = (st["lengths"] > t)[:, None, None, None]
        at = start + st["path"][:, t].long().clamp(min=0)
        k = st["k"][at].float().repeat_interleave(share, dim=1)[:, :, None]
        v = st["v"][at].float()
        alpha = st["alpha"][at]
        now = s * (alpha[:, :, None] if c["diag"] else alpha[:, :, None, None])
        if c["delta"]:
            v = v - (now * k).sum(-1)
        now = now + (st["beta"][at][:, :, None] * v)[..., None] * k
        s = torch.where(live, now, s)
    pool[st["slots"].long()] = s


def _verify(st):
    c = st["case"]
    m, n, depth, drawn = c["seqs"], c["nodes"], c["depth"], c["drawn"]
    at, live = _padded(st)
    start = st["cu"].long()[:-1]
    each = torch.arange(m, device="cuda")
    ids, parents = st["ids"].long()[at], st["parents"].long()[at]
    u = st["uniform"].double()[at]
    one, zero = torch.ones(m, device="cuda", dtype=torch.float64), torch.zeros(m, device="cuda", dtype=torch.float64)
    cur = torch.zeros(m, dtype=torch.long, device="cuda")
    path = torch.full((m, depth), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    length = torch.ones(m, dtype=torch.long, device="cuda")
    cut, total, rest = zero, one, one
    column = torch.arange(depth, device="cuda")
    left = torch.ones((m, c["vocab"]), dtype=torch.bool, device="cuda") if drawn == "given" else None
    for j in range(1, n):               # children come behind their parents: one look at each node
        here = live[:, j] & (parents[:, j] == cur) & (length < depth)
        x, row = ids[:, j], start + cur
        px = st["target"][row, x].double()
        if drawn == "given":
            px = px * left[each, x]
            take = here & (u[:, j] * total < px)
        else:
            qx = st["draft"][row, x].double()
            take = here & (u[:, j] * total * qx < (px - cut * qx).clamp(min=0) * rest)
        miss = here & ~take
        if drawn == "given":
            total = torch.where(miss, (total - px).clamp(min=0), total)
            left[each, x] &= ~miss
            left |= take[:, None]
        else:
            cut = torch.where(miss, cut + total / rest, cut)
            left_over = (st["target"][row].double() - cut[:, None] * st["draft"][row].double()).clamp_(min=0).sum(-1)
            total = torch.where(miss, left_over, total)
            if drawn == "without":
                rest = torch.where(miss, rest - qx, rest)
        path = torch.where(take[:, None] & (column[None] == length[:, None]), j, path)
        length = length + take
        cur = torch.where(take, j, cur)
        cut, total, rest = torch.where(take, zero, cut), torch.where(take, one, total), torch.where(take, one, rest)
    p = st["target"][start + cur].double()
    if drawn == "given":
        p = p * left
    else:
        p = (p - cut[:, None] * st["draft"][start + cur].double()).clamp_(min=0)
    cum = p.cumsum(-1)
    threshold = st["uniform_next"].double() * cum[:, -1]
    last = (p > 0).double().mul_(torch.arange(c["vocab"], device="cuda")).amax(-1).long()
    token = torch.minimum((cum <= threshold[:, None]).sum(-1), last)
    return {"path": path.to(torch.int32), "lengths": length.to(torch.int32), "next": token.to(torch.int32)}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    m = case["seqs"]
    if case["op"] == "verify":          # the rows of the node where the walk ends
        rows = 1 if case["drawn"] == "given" else 2
        return {"bytes": m * case["vocab"] * 4 * rows + 16 * sum(_counts(case)) + 4 * m * (case["depth"] + 2),
                "flops": m * case["vocab"] * (2 * rows - 1)}
    h, dk, dv = case["heads"], case["dk"], case["dv"]
    state, e = h * dv * dk, DTYPES[case["dtype"]].itemsize
    gates = 4 * h * (dk if case["diag"] else 1) + 4 * h
    read = 0.6 if case["fresh"] == "some" else 1.0
    if case["op"] == "tree":
        n = sum(_counts(case))
        return {"bytes": n * (2 * case["qk_heads"] * dk * e + 2 * h * dv * e + gates) + m * state * 4 * read,
                "flops": n * state * (4 if case["delta"] else 2)}
    n = sum(_accepted(case))
    return {"bytes": n * (case["qk_heads"] * dk * e + h * dv * e + gates) + m * state * 4 * (1 + read),
            "flops": n * state * (5 if case["delta"] else 3)}


# ---- the definition, in 64 bits ----------------------------------------------------------------

def _exact_token(st, at, s, head, case):
    """The state after one node of each listed row, from the states before it."""
    kt = st["k"][at].double()[:, head]
    a = st["alpha"][at].double()
    s = s * (a[:, :, None, :] if a.dim() == 3 else a[:, :, None, None])
    gap = st["v"][at].double()
    if case["delta"]:
        gap = gap - torch.matmul(s, kt[..., None])[..., 0]
    return s.add_((st["beta"][at].double()[..., None] * gap)[..., None] * kt[:, :, None, :])


def _exact_verify(case, st):
    """Sequence by sequence, the residual distributions normalised as they are defined."""
    paths, lengths, tokens = [], [], []
    ids, parents, u = st["ids"].tolist(), st["parents"].tolist(), st["uniform"].tolist()
    nexts, start = st["uniform_next"].tolist(), 0
    for i, count in enumerate(_counts(case)):
        path = [0]
        while True:
            row = start + path[-1]
            p = st["target"][row].double()
            q = st["draft"][row].double() if st["draft"] is not None else None
            taken, gone = None, 0.0
            for j in range(path[-1] + 1, count) if len(path) < case["depth"] else ():
                if parents[start + j] != path[-1]:
                    continue
                x = ids[start + j]
                px = float(p[x])
                if q is None:
                    if u[start + j] < px:
                        taken = j
                        break
                    p = p.clone()       # the token left out, the others scaled up
                    p[x] = 0.0
                    p = p / (1.0 - px) if px < 1.0 else p
                    continue
                now = q / (1.0 - gone) if case["drawn"] == "without" else q
                if u[start + j] * float(now[x]) < px:
                    taken = j
                    break
                # tokens drawn before have no residual left: their share of q needs no care
                p = torch.relu(p - now)
                p = p / p.sum()
                gone += float(q[x])
            if taken is None:
                break
            path.append(taken)
        sums = torch.cumsum(p.cpu(), 0)
        y = int(torch.searchsorted(sums, nexts[i] * float(sums[-1]), right=True))
        positive = torch.nonzero(p.cpu() > 0)
        tokens.append(min(y, int(positive[-1]) if len(positive) else 0))
        paths.append(path + [-1] * (case["depth"] - len(path)))
        lengths.append(len(path))
        start += count
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"path": torch.tensor(paths, **i32), "lengths": torch.tensor(lengths, **i32),
            "next": torch.tensor(tokens, **i32)}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "verify":
        return _exact_verify(case, st)
    h, m = case["heads"], case["seqs"]
    pool = st["pool"].double().view(case["slots"], h, case["dv"], case["dk"])
    slot = st["slots"].long()
    first = pool[slot].clone()
    if st["fresh"] is not None:
        first[st["fresh"]] = 0.0
    head = torch.arange(h, device="cuda") // (h // case["qk_heads"])
    counts = _counts(case)
    start = [sum(counts[:i]) for i in range(m)]
    if case["op"] == "accept":
        path, lengths = st["path"].tolist(), st["lengths"].tolist()
        for t in range(max(lengths)):
            alive = [i for i in range(m) if lengths[i] > t]
            at = torch.tensor([start[i] + path[i][t] for i in alive], device="cuda")
            who = torch.tensor(alive, device="cuda")
            first[who] = _exact_token(st, at, first[who], head, case)
        pool[slot] = first
        return {"state": pool.view(st["pool"].shape)}
    # every node's state from its parent's, a group of sequences at a time
    parents = st["parents"].tolist()
    o = torch.empty(sum(counts), h, case["dv"], dtype=torch.float64, device="cuda")
    group = max(1, int(2 ** 31 // (case["nodes"] * h * case["dv"] * case["dk"])))
    for i0 in range(0, m, group):
        ids = range(i0, min(m, i0 + group))
        states = torch.empty((len(ids), case["nodes"]) + tuple(first.shape[1:]), dtype=torch.float64, device="cuda")
        for j in range(max(counts[i] for i in ids)):
            alive = [i for i in ids if counts[i] > j]
            who = torch.tensor([i - i0 for i in alive], device="cuda")
            at = torch.tensor([start[i] + j for i in alive], device="cuda")
            before = [parents[start[i] + j] for i in alive]
            old = first[torch.tensor(alive, device="cuda")] if j == 0 else \
                states[who, torch.tensor(before, device="cuda")]
            new = _exact_token(st, at, old, head, case)
            states[who, j] = new
            o[at] = torch.matmul(new, st["q"][at].double()[:, head][..., None])[..., 0]
    return {"o": o}
