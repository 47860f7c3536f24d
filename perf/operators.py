"""The operators that verify a tree of drafted tokens, as measured workloads.

A speculative step drafts a tree: node i of sequence b follows node parent[b][i] (-1: the last committed token;
-2: no node), so node i sits at position pos[b] + depth(i) and sees the committed cache and its own ancestors.  One
step of a layer is: norm_rope (queries, latent keys and index queries normalised and rotated), compress_tree
(projections of the drafted tokens and the compressed rows that they complete, each along its own path),
index_scores_tree (every node against the index keys that it sees), attend_tree (selection, attention, inverse
rotation) and, once a leaf is accepted, commit_tree (its path enters the cache).  Each is timed on its own here.

Shapes are the Flash layer's (64 heads over a 512-dim latent, 64 index heads of 128, 128-token window, 512 selected
rows, ratio 4 or 128) and, for other types and sizes, the small fp32 layer of the tests.
"""
import math

import numpy as np
import torch

own = False

FLASH = dict(H=64, D=512, R=64, W=128, Hi=64, Di=128, topk=512, X=4096, dtype="bf16", base=160000.0)
SMALL = dict(H=8, D=64, R=16, W=32, Hi=4, Di=32, topk=16, X=128, dtype="f32", base=10000.0)
EPS = 1e-6


def listed():
    return [
        # one token of one sequence: the least a decode step does, all latency
        dict(name="norm_rope_decode_b1", op="norm_rope", layer="flash", B=1, T=1, ctx=8192, tree=False),
        # fp32 rows of odd counts, a ragged tree
        dict(name="norm_rope_tree_f32", op="norm_rope", layer="small", B=5, T=7, ctx=1000, tree=True),
        # a prefill chunk's queries and keys
        dict(name="norm_rope_prefill_t4096", op="norm_rope", layer="flash", B=1, T=4096, ctx=65536, tree=False),
        # a single user's draft of 8 nodes
        dict(name="compress_tree_b1_t8", op="compress_tree", layer="flash", ratio=4, B=1, T=8, ctx=8192),
        # a serving batch, 16 nodes a sequence
        dict(name="compress_tree_b32_t16", op="compress_tree", layer="flash", ratio=4, B=32, T=16, ctx=32768),
        # odd node count over a short odd cache
        dict(name="index_scores_tree_b1_t13", op="index_scores_tree", layer="flash", ratio=4, B=1, T=13, ctx=5003),
        dict(name="index_scores_tree_b32_t16", op="index_scores_tree", layer="flash", ratio=4, B=32, T=16, ctx=32768),
        dict(name="attend_tree_b1_t8", op="attend_tree", layer="flash", ratio=4, B=1, T=8, ctx=8192),
        dict(name="attend_tree_b32_t16", op="attend_tree", layer="flash", ratio=4, B=32, T=16, ctx=32768),
        # a layer without an indexer: every node sees every row of a 256K context at ratio 128
        dict(name="attend_tree_r128_b16_t8", op="attend_tree", layer="flash", ratio=128, B=16, T=8, ctx=262144),
        dict(name="commit_tree_b1_t5", op="commit_tree", layer="flash", ratio=4, B=1, T=5, ctx=4096),
        dict(name="commit_tree_b32_t16", op="commit_tree", layer="flash", ratio=4, B=32, T=16, ctx=4096),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm_rope", "compress_tree", "index_scores_tree", "attend_tree", "commit_tree"])
    if op == "norm_rope":
        tree = rng.random() < 0.5
        B = size(1, 32)
        T = size(1, 64) if tree else size(1, 4096 // B)
        return dict(op=op, layer=rng.choice(["flash", "flash", "small"]), B=B, T=T, ctx=size(64, 65536), tree=tree)
    B = size(1, 32)
    T = size(1, min(64, 512 // B))
    if op == "commit_tree":
        return dict(op=op, layer="flash", ratio=rng.choice([4, 128]), B=B, T=min(T, 16), ctx=size(64, 4096))
    if op == "compress_tree":
        return dict(op=op, layer="flash", ratio=rng.choice([4, 128]), B=B, T=T, ctx=size(64, 32768))
    if op == "index_scores_tree":
        return dict(op=op, layer="flash", ratio=4, B=B, T=T, ctx=size(64, 32768))
    if rng.random() < 0.5:
        return dict(op=op, layer="flash", ratio=4, B=B, T=T, ctx=size(64, 32768))
    B = min(B, 16)
    return dict(op=op, layer="flash", ratio=128, B=B, T=min(T, 128 // B), ctx=size(256, 262144))


# ---------------------------------------------------------------------------------------------------- inputs


def dims(case):
    return dict(FLASH if case["layer"] == "flash" else SMALL)


def lanes(case):
    return 2 if case["ratio"] == 4 else 1


def slots(case):
    return 8 if case["ratio"] == 4 else case["ratio"]


def capacity(case):
    return case["ctx"] // case["ratio"] + 64


def positions(case):
    """The sequences' lengths: ragged, the longest ctx."""
    return [case["ctx"] - (61 * b) % (case["ctx"] // 4 + 1) for b in range(case["B"])]


def nodes(case):
    """Nodes of each sequence's tree: some trees are smaller than the widest."""
    return [max(1, case["T"] - b % 3) for b in range(case["B"])]


def trees(case, seed):
    """parent [B, T]: a few branches off the last token, then mostly children of recent nodes."""
    r = np.random.RandomState(seed % (1 << 31))
    par = np.full((case["B"], case["T"]), -2, dtype=np.int32)
    for b, n in enumerate(nodes(case)):
        for i in range(n):
            par[b, i] = -1 if i == 0 else r.randint(max(0, i - 6), i) if r.rand() < 0.85 else r.randint(-1, i)
    return par


def prepare(case, seed):
    c = dims(case)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    g = torch.Generator("cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    B, T = case["B"], case["T"]
    s = dict(case=case, c=c, kept={})
    s["pos"] = torch.tensor(positions(case), dtype=torch.int32, device="cuda")
    half = np.arange(c["R"] // 2, dtype=np.float64)
    s["inv_freq"] = torch.from_numpy((c["base"] ** (-2.0 * half / c["R"])).astype(np.float32)).cuda()
    if case["op"] != "norm_rope" or case["tree"]:
        s["parent"] = torch.from_numpy(trees(case, seed)).cuda()
    else:
        s["parent"] = None
    if case["op"] == "norm_rope":
        s["q"] = normal(B, T, c["H"], c["D"])
        s["kv"] = normal(B, T, 1, c["D"], scale=3.0)
        s["iq"] = normal(B, T, c["Hi"], c["Di"])
        s["kv_w"] = 1.0 + 0.1 * normal(c["D"], dtype=torch.float32)
        s["outs"] = [torch.zeros_like(s[k]) for k in ("q", "kv", "iq")]
        return s
    L, r, F, cap = lanes(case), case["ratio"], slots(case), capacity(case)
    s["n_rows"] = s["pos"] // r
    if case["op"] == "compress_tree":
        s["x"] = normal(B, T, c["X"])
        for k, d in (("a", c["D"]), ("i", c["Di"]))[: 2 if r == 4 else 1]:
            s["wkv_" + k] = normal(L * d, c["X"], scale=c["X"] ** -0.5)
            s["wgate_" + k] = normal(L * d, c["X"], scale=c["X"] ** -0.5)
            s["ape_" + k] = normal(r, L * d, dtype=torch.float32)
            s["norm_" + k] = 1.0 + 0.1 * normal(d, dtype=torch.float32)
            s["frontier_" + k] = normal(B, F, 2 * L * d)
            s["proj_" + k] = torch.zeros(B, T, 2 * L * d, dtype=dt, device="cuda")
            s["rows_" + k] = torch.zeros(B, T, d, dtype=dt, device="cuda")
    elif case["op"] == "index_scores_tree":
        s["iq"] = normal(B, T, c["Hi"], c["Di"])
        s["iw"] = normal(B, T, c["Hi"])
        s["ikeys"] = normal(B, cap, c["Di"])
        s["rows_i"] = normal(B, T, c["Di"])
        s["scores"] = torch.zeros(B, T, cap + T, device="cuda")
    elif case["op"] == "attend_tree":
        s["q"] = normal(B, T, c["H"], c["D"])
        s["kv"] = normal(B, T, c["D"])
        s["sink"] = normal(c["H"], dtype=torch.float32)
        s["window"] = normal(B, c["W"], c["D"])
        s["pool"] = normal(B, cap, c["D"])
        s["rows_a"] = normal(B, T, c["D"])
        s["scores"] = normal(B, T, cap + T, dtype=torch.float32) if r == 4 else None
        s["out"] = torch.zeros(B, T, c["H"], c["D"], dtype=dt, device="cuda")
        s["sel"] = torch.full((B, T, c["topk"]), -1, dtype=torch.int32, device="cuda") if r == 4 else None
    else:
        # the accepted node: any node of the tree, or none
        rr = np.random.RandomState((seed + 1) % (1 << 31))
        leaf = [int(rr.randint(n // 2, n)) if b % 7 != 6 else -1 for b, n in enumerate(nodes(case))]
        s["leaf"] = torch.tensor(leaf, dtype=torch.int32, device="cuda")
        s["kv"] = normal(B, T, c["D"])
        s["window"] = normal(B, c["W"], c["D"])
        for k, d in (("a", c["D"]), ("i", c["Di"]))[: 2 if r == 4 else 1]:
            s["frontier_" + k] = normal(B, F, 2 * L * d)
            s["proj_" + k] = normal(B, T, 2 * L * d)
            s["rows_" + k] = normal(B, T, d)
            s["pool_" + k] = normal(B, cap, d)
        for k in ("pos_out", "n_rows_a_out", "n_rows_i_out"):
            s[k] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------- plain forms


def ancestors(parent):
    """(anc [B, T, T], depth [B, T], valid [B, T]): anc[b, i, j] says that j is i or one of its ancestors."""
    B, T = parent.shape
    i = torch.arange(T, device=parent.device)
    step = (parent[:, :, None] == i).float()
    anc = torch.linalg.matrix_power(torch.eye(T, device=parent.device) + step, 64) > 0.5
    valid = parent > -2
    return anc & valid[:, :, None], anc.sum(-1) - 1, valid


def rotate(x, p, inv_freq, R, inverse=False):
    """The last R dims of x [.., heads, dim], pairs of neighbours, turned by p * inv_freq (x's type is fp32)."""
    a = (p.float()[..., None] * inv_freq).double()  # the library's angle: one fp32 product
    cs, sn = a.cos().float()[..., None, :], a.sin().float()[..., None, :]
    sn = -sn if inverse else sn
    u, v = x[..., -R::2], x[..., -R + 1 :: 2]
    y = torch.stack((u * cs - v * sn, u * sn + v * cs), -1).flatten(-2)
    return torch.cat((x[..., :-R], y), -1)


def plain_norm_rope(s):
    c, (B, T) = s["c"], s["q"].shape[:2]
    if s["parent"] is None:
        depth = torch.arange(T, device="cuda").expand(B, T)
        valid = torch.ones(B, T, dtype=torch.bool, device="cuda")
    else:
        _, depth, valid = ancestors(s["parent"])
    p = s["pos"][:, None] + depth

    def one(x, w, norm, out):
        y = x.float()
        if norm:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
            y = y if w is None else y * w
        y = rotate(y, p, s["inv_freq"], c["R"]).to(x.dtype)
        return torch.where(valid[:, :, None, None], y, out)

    q, kv, iq = s["outs"]
    return one(s["q"], None, True, q), one(s["kv"], s["kv_w"], True, kv), one(s["iq"], None, False, iq)


def plain_compress(s, k, d, anc, depth, valid):
    case, c = s["case"], s["c"]
    r, L, F = case["ratio"], lanes(case), slots(case)
    B, T = depth.shape
    dt = s["x"].dtype
    # the projections are kept, and pooled, in the layer's type
    proj = torch.cat((s["x"].float() @ s["wkv_" + k].float().T, s["x"].float() @ s["wgate_" + k].float().T), -1).to(dt)
    p = s["pos"][:, None] + depth
    closes = valid & ((p + 1) % r == 0)
    j = (p + 1) // r - 1
    n_ent = r * L
    t = (j * r - (r if L == 2 else 0))[..., None] + torch.arange(n_ent, device="cuda")  # [B, T, n_ent]
    b = torch.arange(B, device="cuda")[:, None, None]
    past = s["frontier_" + k][b, t.clamp(min=0) % F]
    k_of = (t - s["pos"][:, None, None]).clamp(0, T - 1)
    node = (anc[:, :, None, :] & (depth[:, None, None, :] == k_of[..., None])).int().argmax(-1)
    ent = torch.where((t < s["pos"][:, None, None])[..., None], past, proj[b, node]).float()
    lane = torch.arange(n_ent, device="cuda") // r if L == 2 else torch.zeros(n_ent, dtype=torch.long, device="cuda")
    ch = lane[:, None] * d + torch.arange(d, device="cuda")  # [n_ent, d]
    kv = torch.gather(ent, -1, ch.expand(B, T, n_ent, d))
    gate = torch.gather(ent, -1, (ch + L * d).expand(B, T, n_ent, d))
    gate = gate + s["ape_" + k][(torch.arange(n_ent, device="cuda") % r)[:, None], ch]
    gate = gate.masked_fill((t < 0)[..., None], -math.inf)
    e = (gate - gate.amax(-2, keepdim=True)).exp()
    # a pool row is stored in the layer's type at each of its steps, as the committed rows are
    u = ((e * kv).sum(-2) / e.sum(-2)).to(dt).float()
    y = (u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * s["norm_" + k]).to(dt).float()
    row = rotate(y[..., None, :], j * r, s["inv_freq"], c["R"])[..., 0, :].to(dt)
    return torch.where(valid[..., None], proj, s["proj_" + k]), torch.where(closes[..., None], row, s["rows_" + k])


def plain_scores(s):
    case, c = s["case"], s["c"]
    anc, depth, valid = ancestors(s["parent"])
    B, T = depth.shape
    closes = valid & ((s["pos"][:, None] + depth + 1) % case["ratio"] == 0)
    n = s["n_rows"]
    cols = torch.arange(s["scores"].shape[-1], device="cuda")
    # column j: committed row j below n, then the nodes' rows
    node = (cols - n[:, None]).clamp(0, T - 1)
    b = torch.arange(B, device="cuda")[:, None]
    keys = torch.where((cols < n[:, None])[..., None], s["ikeys"][b, cols.clamp(max=s["ikeys"].shape[1] - 1)],
                       s["rows_i"][b, node]).float()
    dots = (s["iq"].float().flatten(1, 2) @ keys.transpose(1, 2)).clamp(min=0).view(B, T, c["Hi"], -1)
    w = s["iw"].float() * (c["Di"] * c["Hi"]) ** -0.5
    score = (w[..., None, :] @ dots)[..., 0, :]
    sees = torch.where(cols < n[:, None, None], True, torch.gather(anc & closes[:, None, :], 2, node[:, None].expand(B, T, -1)))
    score = score.masked_fill(~sees, -math.inf)
    return torch.where(valid[..., None] & (cols < n[:, None, None] + T), score, s["scores"])


def visible(s, anc, depth, valid, cols):
    case = s["case"]
    T, n = depth.shape[1], s["n_rows"]
    closes = valid & ((s["pos"][:, None] + depth + 1) % case["ratio"] == 0)
    node = (cols - n[:, None]).clamp(0, T - 1)
    on_path = torch.gather(anc & closes[:, None, :], 2, node[:, None].expand(-1, T, -1))
    return torch.where(cols < n[:, None, None], True, on_path & (cols < n[:, None, None] + T))


def plain_attend(s):
    case, c = s["case"], s["c"]
    anc, depth, valid = ancestors(s["parent"])
    B, T = depth.shape
    p, n, W, D = s["pos"][:, None] + depth, s["n_rows"], c["W"], c["D"]
    cap = s["pool"].shape[1]
    cols = torch.arange(cap + T, device="cuda")
    sees = visible(s, anc, depth, valid, cols)
    if s["scores"] is not None:
        # the topk largest, ties to the lower column, in ascending order; every visible one where they are fewer
        order = s["scores"].masked_fill(~sees, -math.inf).sort(stable=True, dim=-1, descending=True).indices
        rank = torch.empty_like(order).scatter_(-1, order, cols.expand_as(order))
        keep = sees & ((rank < c["topk"]) | (sees.sum(-1, keepdim=True) <= c["topk"]))
        width = min(c["topk"], cap + T)
        at = torch.where(keep, cols, cap + T).sort(-1).values[..., :width]
    else:
        at = torch.where(sees, cols, cap + T).sort(-1).values
    live = at < cap + T
    b = torch.arange(B, device="cuda")[:, None, None]
    at_n = at - n[:, None, None]
    rows = torch.where((at_n < 0)[..., None], s["pool"][b, at.clamp(max=cap - 1)], s["rows_a"][b, at_n.clamp(0, T - 1)])
    # window tokens t in (p - W, p]: the ring before pos, the nodes of the path from there
    t = p[..., None] - torch.arange(W - 1, -1, -1, device="cuda")
    k_of = t - s["pos"][:, None, None]
    node = (anc[:, :, None, :] & (depth[:, None, None, :] == k_of.clamp(0, T - 1)[..., None])).int().argmax(-1)
    win = torch.where((k_of < 0)[..., None], s["window"][b, t.clamp(min=0) % W], s["kv"][b, node])
    keys = torch.cat((rows, win), 2).float()
    live = torch.cat((live, t >= 0), 2)
    logit = (s["q"].float() @ keys.transpose(-1, -2)) * D**-0.5
    logit = logit.masked_fill(~live[:, :, None], -math.inf)
    m = torch.maximum(logit.amax(-1, keepdim=True), s["sink"][:, None])
    e = (logit - m).exp()
    o = (e @ keys) / (e.sum(-1, keepdim=True) + (s["sink"][:, None] - m).exp())
    o = rotate(o, p, s["inv_freq"], c["R"], inverse=True).to(s["out"].dtype)
    o = torch.where(valid[..., None, None], o, s["out"])
    if s["scores"] is None:
        return o
    sel = torch.nn.functional.pad(torch.where(at < cap + T, at, -1), (0, c["topk"] - at.shape[-1]), value=-1)
    return o, torch.where(valid[..., None], sel.int(), s["sel"])


def plain_commit(s):
    case, c = s["case"], s["c"]
    r, F, W = case["ratio"], slots(case), c["W"]
    anc, depth, _ = ancestors(s["parent"])
    B, T = depth.shape
    leaf = s["leaf"].long()
    took = leaf >= 0
    path = torch.gather(anc, 1, leaf.clamp(min=0)[:, None, None].expand(B, 1, T))[:, 0] & took[:, None]
    pos = s["pos"].long()
    end = pos + path.sum(-1)
    b = torch.arange(B, device="cuda")[:, None]

    def node_at(k):  # the path's node of depth k [B, n]
        return (path[:, None, :] & (depth[:, None, :] == k[..., None])).int().argmax(-1)

    def ring(buf, src):
        n = buf.shape[1]
        t = end[:, None] - 1 - (end[:, None] - 1 - torch.arange(n, device="cuda")) % n  # the token that a slot ends with
        k = t - pos[:, None]
        return torch.where((k >= 0)[..., None], src[b, node_at(k)], buf)

    def pool(buf, src):
        j = (pos // r)[:, None] + torch.arange((T + r - 1) // r, device="cuda")
        new = j < (end // r)[:, None]
        buf[b, j] = torch.where(new[..., None], src[b, node_at((j + 1) * r - 1 - pos[:, None])], buf[b, j])
        return buf

    out = [ring(s["window"], s["kv"]), ring(s["frontier_a"], s["proj_a"]), pool(s["pool_a"], s["rows_a"])]
    if r == 4:
        out += [ring(s["frontier_i"], s["proj_i"]), pool(s["pool_i"], s["rows_i"])]
    return out + [end.int(), (end // r).int()]


# ---------------------------------------------------------------------------------------------------- one pass


def run(s):
    if own:
        return run_own(s)
    op, c = s["case"]["op"], s["c"]
    if op == "norm_rope":
        return plain_norm_rope(s)
    if op == "compress_tree":
        tree = ancestors(s["parent"])
        out = plain_compress(s, "a", c["D"], *tree)
        return out + plain_compress(s, "i", c["Di"], *tree) if s["case"]["ratio"] == 4 else out
    if op == "index_scores_tree":
        return plain_scores(s)
    if op == "attend_tree":
        return plain_attend(s)
    return plain_commit(s)


def layer_of(s, csa):
    c, case = s["c"], s["case"]
    return csa.Layer(dtype=torch.bfloat16 if c["dtype"] == "bf16" else torch.float32, H=c["H"], D=c["D"], R=c["R"],
                     W=c["W"], ratio=case.get("ratio", 4), Hi=c["Hi"], Di=c["Di"], topk=c["topk"], X=c["X"], rms_eps=EPS)


def run_own(s):
    import deepseek_v4_compressed_csa_gb300 as csa

    case, c, kept = s["case"], s["c"], s["kept"]
    op = case["op"]
    B, T = case["B"], case["T"]
    if not kept:  # what a program keeps beside its cache: the layer's description, the error word, the workspace
        kept["layer"] = layer_of(s, csa)
        kept["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        of = {"compress_tree": csa.OP_COMPRESS_TREE, "attend_tree": csa.OP_ATTEND_TREE}
        if op in of:
            n = csa.workspace_size(kept["layer"], of[op], B, T, s["pool"].shape[1] if op == "attend_tree" else 1)
            kept["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        if op == "compress_tree":
            for k, d in (("a", c["D"]), ("i", c["Di"]))[: 2 if case["ratio"] == 4 else 1]:
                kept["comp_" + k] = csa.Compressor(s["wkv_" + k], s["wgate_" + k], s["ape_" + k], s["norm_" + k], d)
    layer, err = kept["layer"], kept["err"]
    if op == "norm_rope":
        return csa.norm_rope(layer, [s["q"], s["kv"], s["iq"]], s["pos"], s["inv_freq"], parent=s["parent"],
                             weights=[None, s["kv_w"], None], norm=[True, True, False], outs=s["outs"], err=err)
    if op == "compress_tree":
        index = dict(comp_i=kept["comp_i"], frontier_i=s["frontier_i"], proj_i=s["proj_i"], rows_i=s["rows_i"]) if case["ratio"] == 4 else {}
        csa.compress_tree(layer, kept["comp_a"], s["x"], s["parent"], s["pos"], s["frontier_a"], s["proj_a"],
                          s["rows_a"], s["inv_freq"], **index, ws=kept["ws"], err=err)
        return [s[k] for k in ("proj_a", "rows_a", "proj_i", "rows_i") if k in s]
    if op == "index_scores_tree":
        csa.index_scores_tree(layer, s["iq"], s["iw"], s["ikeys"], s["rows_i"], s["parent"], s["n_rows"], s["pos"],
                              s["scores"], err=err)
        return s["scores"]
    if op == "attend_tree":
        csa.attend_tree(layer, s["q"], s["kv"], s["sink"], s["window"], s["pool"], s["rows_a"], s["scores"],
                        s["parent"], s["n_rows"], s["pos"], s["inv_freq"], s["out"], sel_out=s["sel"], ws=kept["ws"],
                        err=err)
        return s["out"] if s["sel"] is None else (s["out"], s["sel"])
    index = {k: s[k] for k in ("frontier_i", "proj_i", "rows_i", "pool_i")} if case["ratio"] == 4 else {}
    if case["ratio"] == 4:
        index |= dict(n_rows_i=s["n_rows"], n_rows_i_out=s["n_rows_i_out"])
    csa.commit_tree(layer, s["parent"], s["leaf"], s["pos"], s["n_rows"], s["kv"], s["window"], s["proj_a"],
                    s["frontier_a"], s["rows_a"], s["pool_a"], **index, pos_out=s["pos_out"],
                    n_rows_a_out=s["n_rows_a_out"], err=err)
    return [s[k] for k in ("window", "frontier_a", "pool_a", "frontier_i", "pool_i", "pos_out", "n_rows_a_out") if k in s]


# ---------------------------------------------------------------------------------------------------- what a pass needs


def work(case):
    c = dims(case)
    es = 2 if c["dtype"] == "bf16" else 4
    B, T = case["B"], case["T"]
    N = B * T if not case.get("tree", True) else sum(nodes(case))
    if case["op"] == "norm_rope":
        vals = c["H"] * c["D"] + c["D"] + c["Hi"] * c["Di"]
        return dict(bytes=2 * N * vals * es + 4 * c["D"] + 8 * B, flops=N * 5 * vals)
    r, L, F = case["ratio"], lanes(case), slots(case)
    ds = [c["D"], c["Di"]] if r == 4 else [c["D"]]
    n_rows = [p // r for p in positions(case)]
    if case["op"] == "compress_tree":
        wide = sum(2 * L * d for d in ds)
        closing = N / r
        return dict(bytes=es * (c["X"] * (N + wide) + N * wide + closing * sum(ds) + B * (r * L - 1) * wide / L),
                    flops=2.0 * N * c["X"] * wide)
    if case["op"] == "index_scores_tree":
        cells = sum(m * (n + T) for m, n in zip(nodes(case), n_rows))
        return dict(bytes=es * (N * (c["Hi"] * c["Di"] + c["Hi"]) + (sum(n_rows) + N / r) * c["Di"]) + 4 * cells,
                    flops=2.0 * cells * c["Hi"] * (c["Di"] + 1))
    if case["op"] == "attend_tree":
        took = [min(n, c["topk"]) if r == 4 else n for n in n_rows]
        # the rows of a cache that m independent selections of k out of n touch
        touched = sum(n * (1 - (1 - k / max(1, n)) ** m) if r == 4 else n for n, k, m in zip(n_rows, took, nodes(case)))
        wins = [min(c["W"], p + 1) for p in positions(case)]
        cells = sum(m * (k + w) for m, k, w in zip(nodes(case), took, wins))
        scores = sum(m * (n + T) for m, n in zip(nodes(case), n_rows)) if r == 4 else 0
        return dict(bytes=es * (2 * N * c["H"] * c["D"] + c["D"] * (touched + sum(wins) + N)) + 4 * scores,
                    flops=4.0 * cells * c["H"] * c["D"])
    # a path of such a tree is about 1 + T/3 nodes long
    moved = sum(1 + m / 3 for m in nodes(case))
    return dict(bytes=2 * es * moved * (c["D"] + sum(2 * L * d + d / r for d in ds)) + 24 * B, flops=0)


# ---------------------------------------------------------------------------------------------------- in 64 bits


def _paths(parent):
    """For every (b, i): the node's path from its root, by walking the parents; None where there is no node."""
    par = parent.cpu().tolist()
    found = []
    for row in par:
        paths = []
        for i, a in enumerate(row):
            paths.append(None if a < -1 else [i] if a < 0 else paths[a] + [i])
        found.append(paths)
    return found


def _turn(x, p, inv_freq, R, sign):
    """x [heads, dim] (64 bits) turned as complex numbers by the angles that the layer defines (fp32 products)."""
    th = (torch.tensor(float(p), dtype=torch.float32, device=x.device) * inv_freq).double()
    z = torch.view_as_complex(x[:, -R:].reshape(x.shape[0], R // 2, 2).contiguous())
    z = z * torch.polar(torch.ones_like(th), sign * th)
    return torch.cat((x[:, :-R], torch.view_as_real(z).reshape(x.shape[0], R)), 1)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["c"], case["op"]
    B, T, pos = case["B"], case["T"], positions(case)
    d64 = torch.float64
    if op == "norm_rope":
        paths = _paths(s["parent"]) if s["parent"] is not None else [[range(i + 1) for i in range(T)] for _ in range(B)]
        outs = []
        for x, w, norm, old in ((s["q"], None, True, s["outs"][0]), (s["kv"], s["kv_w"], True, s["outs"][1]), (s["iq"], None, False, s["outs"][2])):
            y = old.to(d64)
            for b in range(B):
                for i in range(T):
                    if paths[b][i] is None:
                        continue
                    v = x[b, i].to(d64)
                    if norm:
                        v = v / (v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt()
                        v = v if w is None else v * w.to(d64)
                    y[b, i] = _turn(v, pos[b] + len(paths[b][i]) - 1, s["inv_freq"], c["R"], 1.0)
            outs.append(y)
        return tuple(outs)
    paths, r, L, F = _paths(s["parent"]), case["ratio"], lanes(case), slots(case)
    n_rows = [p // r for p in pos]
    if op == "compress_tree":
        outs = []
        for k, d in (("a", c["D"]), ("i", c["Di"]))[: 2 if r == 4 else 1]:
            w = torch.cat((s["wkv_" + k], s["wgate_" + k])).to(d64)
            proj, rows = s["proj_" + k].to(d64), s["rows_" + k].to(d64)
            full = s["x"].to(d64).reshape(B * T, -1) @ w.T
            for b in range(B):
                for i in range(T):
                    if paths[b][i] is None:
                        continue
                    proj[b, i] = full[b * T + i]
                    p = pos[b] + len(paths[b][i]) - 1
                    if (p + 1) % r:
                        continue
                    first = p + 1 - r * L
                    ts = [t for t in range(first, p + 1) if t >= 0]
                    ent = torch.stack([s["frontier_" + k][b, t % F].to(d64) if t < pos[b] else full[b * T + paths[b][i][t - pos[b]]] for t in ts])
                    lane = [1 if L == 2 and t > p - r else 0 for t in ts]
                    kv = torch.stack([e[l * d : l * d + d] for e, l in zip(ent, lane)])
                    gt = torch.stack([e[(L + l) * d : (L + l) * d + d] + s["ape_" + k][t % r, l * d : l * d + d] for e, l, t in zip(ent, lane, ts)])
                    u = (torch.softmax(gt, 0) * kv).sum(0)
                    u = u / (u.pow(2).mean() + EPS).sqrt() * s["norm_" + k]
                    rows[b, i] = _turn(u[None], p + 1 - r, s["inv_freq"], c["R"], 1.0)[0]
            outs += [proj, rows]
        return tuple(outs)
    if op == "index_scores_tree":
        out = s["scores"].to(d64)
        for b in range(B):
            n = n_rows[b]
            keys = torch.cat((s["ikeys"][b, :n], s["rows_i"][b])).to(d64).T
            for i in range(T):
                if paths[b][i] is None:
                    continue
                w = s["iw"][b, i].to(d64) / math.sqrt(c["Di"] * c["Hi"])
                row = w @ (s["iq"][b, i].to(d64) @ keys).relu()
                seen = {a for k, a in enumerate(paths[b][i]) if (pos[b] + k + 1) % r == 0}
                row[[n + a for a in range(T) if a not in seen]] = -math.inf
                out[b, i, : n + T] = row
        return out
    if op == "attend_tree":
        out = s["out"].to(d64)
        for b in range(B):
            n = n_rows[b]
            for i in range(T):
                path = paths[b][i]
                if path is None:
                    continue
                p = pos[b] + len(path) - 1
                col = list(range(n)) + [n + a for k, a in enumerate(path) if (pos[b] + k + 1) % r == 0]
                col = torch.tensor(col, dtype=torch.long, device="cuda")
                if s["scores"] is not None and len(col) > c["topk"]:
                    v = s["scores"][b, i, col]
                    col = col[v.argsort(descending=True, stable=True)[: c["topk"]]]
                rows = torch.cat((s["pool"][b, :n], s["rows_a"][b]))[col]
                first = max(0, p - c["W"] + 1)
                old = torch.arange(first, pos[b], device="cuda") % c["W"]
                new = s["kv"][b][torch.tensor([path[t - pos[b]] for t in range(max(first, pos[b]), p + 1)], dtype=torch.long, device="cuda")]
                keys = torch.cat((rows, s["window"][b][old], new)).to(d64)
                lg = torch.cat((s["q"][b, i].to(d64) @ keys.T / math.sqrt(c["D"]), s["sink"].to(d64)[:, None]), 1)
                out[b, i] = _turn(torch.softmax(lg, 1)[:, :-1] @ keys, p, s["inv_freq"], c["R"], -1.0)
        return out if s["scores"] is None else (out, None)
    return None  # commit_tree moves values and computes none
