"""The operators of a verification step over a paged K/V cache, as cases to measure.

Four operators (public entry points of ``tree_verify_b200``):

  append     rotary positions applied to the queries and keys of a packed batch of tokens, the
             rotated keys and the values written to the pages of their sequences
             (``rope_append``);
  attention  tree attention over a paged cache whose sequences share a prefix, the shared part
             computed once for the whole batch (``tree_attention_paged``); N = 1 is decoding of
             single tokens, a shared length of 0 plain paged attention;
  commit     the root and the accepted nodes' K/V appended to the pages, their hidden rows
             gathered (``commit_accepted_paged``);
  logits     LM-head logits in 8-bit floating point (e4m3) with one scale for each block of 128:
             the hidden rows are quantised in the call (1 x 128 blocks, power-of-two scales),
             the weight (128 x 128 blocks) was quantised when it was loaded (``quantize_rows``,
             ``lm_head_logits_scaled``).

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or, with
``own`` true, by the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128          # elements that share a scale
E4M3_MAX = 448.0     # largest finite e4m3 value
ROPE_BASE = 500000.0

# query heads, kv heads, head size: the head layouts of the repository's workloads
HEADS = ((32, 32, 128), (64, 8, 128), (32, 8, 128), (4, 4, 64), (8, 2, 64), (6, 3, 128))


def listed():
    return [
        # one new token of each of eight sequences deep in their contexts: the smallest call
        dict(name="append_decode", op="append", tokens=8, batch=8, start=8000, hq=32, hkv=8, d=128, dtype="bf16",
             page=16, rotary=128, interleaved=False, padding=0),
        # five prompts of unequal lengths in one packed batch, with padding rows behind them
        dict(name="append_prompts", op="append", tokens=8191, batch=5, start=0, hq=32, hkv=8, d=128, dtype="bf16",
             page=64, rotary=128, interleaved=False, padding=9),
        # the fp32 path, neighbouring pairs, half of the head rotated
        dict(name="append_f32", op="append", tokens=333, batch=3, start=37, hq=4, hkv=4, d=64, dtype="f32",
             page=16, rotary=32, interleaved=True, padding=0),
        # one sequence decoding one token at a time: latency
        dict(name="attention_token", op="attention", batch=1, nodes=1, hq=32, hkv=8, d=128, dtype="bf16", shared=0,
             own_min=4097, own_max=4097, page=16),
        # eight draft trees behind one long system prompt
        dict(name="attention_shared", op="attention", batch=8, nodes=64, hq=32, hkv=8, d=128, dtype="bf16",
             shared=8192, own_min=131, own_max=512, page=64),
        # ragged contexts without grouped heads, a short shared prefix that ends inside a page
        dict(name="attention_ragged", op="attention", batch=16, nodes=60, hq=32, hkv=32, d=128, dtype="bf16",
             shared=500, own_min=12, own_max=3596, page=128),
        # the fp32 path; one sequence has nothing of its own in the cache
        dict(name="attention_f32", op="attention", batch=3, nodes=13, hq=8, hkv=2, d=64, dtype="f32", shared=333,
             own_min=0, own_max=300, page=32),
        # the commit of one verified tree: latency
        dict(name="commit_one", op="commit", batch=1, nodes=45, hq=32, hkv=32, d=128, dtype="bf16", hidden=4096,
             length=1000, page=16),
        # a large batch of verified trees
        dict(name="commit_batch", op="commit", batch=64, nodes=60, hq=64, hkv=8, d=128, dtype="bf16", hidden=8192,
             length=700, page=64),
        # logits of a single token: the weight's bytes alone
        dict(name="logits_token", op="logits", rows=1, hidden=4096, vocab=32000),
        # logits of one draft tree
        dict(name="logits_tree", op="logits", rows=60, hidden=8192, vocab=32000),
        # logits of eight draft trees over a large vocabulary: the largest case
        dict(name="logits_batch", op="logits", rows=512, hidden=4096, vocab=128256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "commit", "logits", "logits"))
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128, 256))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "append":
        tokens = _log(rng, 1, 16000)
        return dict(op=op, tokens=tokens, batch=min(tokens, _log(rng, 1, 64)), start=rng.randrange(0, 3000), hq=hq,
                    hkv=hkv, d=d, dtype=dtype, page=page, rotary=rng.choice((d, d, d // 2)),
                    interleaved=rng.random() < 0.3, padding=rng.choice((0, 0, 3)))
    if op == "commit":
        return dict(op=op, batch=_log(rng, 1, 64), nodes=_log(rng, 1, 64), hq=hq, hkv=hkv, d=d, dtype=dtype,
                    hidden=8 * _log(rng, 8, 1024), length=rng.randrange(0, 1500), page=page)
    if op == "logits":
        rows, hidden, vocab = _log(rng, 1, 1024), 16 * _log(rng, 8, 512), _log(rng, 500, 128256)
        while rows * hidden * vocab > 512 * 4096 * 128256:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, hidden=hidden, vocab=vocab)
    batch, nodes = _log(rng, 1, 32), rng.choice((1, rng.randrange(2, 65)))
    shared = rng.choice((0, _log(rng, 1, 16000)))
    own_max = _log(rng, 1, 4000)
    # about the work of the largest bf16 case, and of a small one for fp32
    most = 3e11 if dtype == "bf16" else 1e10
    while 4.0 * batch * nodes * hq * d * (shared + own_max) > most or batch * hkv * d * own_max > 1 << 28:
        batch, shared, own_max = max(1, batch // 2), (3 * shared) // 4, max(1, (3 * own_max) // 4)
    return dict(op=op, batch=batch, nodes=nodes, hq=hq, hkv=hkv, d=d, dtype=dtype, shared=shared,
                own_min=rng.randrange(0, own_max + 1), own_max=own_max, page=page)


# ------------------------------------------------------------------------------ inputs

def _own_lens(case):
    """Own lengths spread over [own_min, own_max], the longest first."""
    b, lo, hi = case["batch"], case["own_min"], case["own_max"]
    return [hi - (hi - lo) * ((7 * i) % b) // max(1, b - 1) if b > 1 else hi for i in range(b)]


def _new_counts(case):
    """New tokens of each sequence: unequal parts of the whole."""
    t, b = case["tokens"], case["batch"]
    edges = [0] + [max(i, min(t - (b - i), (t * i * (2 * b + i)) // (3 * b * b))) for i in range(1, b)] + [t]
    return [edges[i + 1] - edges[i] for i in range(b)]


def _depths(nodes):
    """Each node's parent in the cases' trees (about three children a node), and its depth."""
    parents = [-1] + [(i - 1) // 3 for i in range(1, nodes)]
    depth = [0] * nodes
    for i in range(1, nodes):
        depth[i] = depth[parents[i]] + 1
    return parents, depth


def _tables(g, count, width):
    """Page tables over a shuffled pool: [count, width], every page used once."""
    return torch.randperm(count * width, generator=g, device="cuda").to(torch.int32).view(count, width)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    if op == "logits":
        rows, hidden, vocab = case["rows"], case["hidden"], case["vocab"]
        # features with a few large channels, as hidden states have; the weight as it was
        # quantised when it was loaded
        x = (normal(rows, hidden) * torch.exp(0.7 * normal(1, hidden))).to(torch.bfloat16)
        kb, vb = -(-hidden // BLOCK), -(-vocab // BLOCK)
        w8 = torch.empty((vocab, hidden), dtype=torch.float8_e4m3fn, device="cuda")
        ws = torch.empty((vb, kb), dtype=torch.float32, device="cuda")
        step = 128 * BLOCK
        for v0 in range(0, vocab, step):
            n = min(step, vocab - v0)
            w = normal(n, hidden) / math.sqrt(hidden)
            pad = torch.nn.functional.pad(w, (0, kb * BLOCK - hidden, 0, -n % BLOCK))
            pad = pad.view(-1, BLOCK, kb, BLOCK)
            scale = pad.abs().amax(dim=(1, 3)) / E4M3_MAX
            q = (pad / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
            w8[v0:v0 + n] = q.reshape(-1, kb * BLOCK)[:n, :hidden].to(torch.float8_e4m3fn)
            ws[v0 // BLOCK:v0 // BLOCK + scale.shape[0]] = scale
        return dict(case=case, x=x, w8=w8, ws=ws,
                    x8=torch.empty((rows, hidden), dtype=torch.float8_e4m3fn, device="cuda"),
                    xs=torch.empty((kb, -(-rows // 4) * 4), dtype=torch.float32, device="cuda"),
                    logits=torch.empty((rows, vocab), dtype=torch.float32, device="cuda"))

    hq, hkv, d, page, dt = case["hq"], case["hkv"], case["d"], case["page"], DTYPES[case["dtype"]]
    batch = case["batch"]
    if op == "append":
        new = _new_counts(case)
        first = [case["start"] + 13 * i for i in range(batch)]
        seqs = [i for i in range(batch) for _ in range(new[i])] + [-1] * case["padding"]
        pos = [first[i] + j for i in range(batch) for j in range(new[i])] + [-1] * case["padding"]
        width = max(pos) // page + 1
        rd = case["rotary"]
        freq = ROPE_BASE ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
        angle = torch.arange(width * page, dtype=torch.float64, device="cuda")[:, None] * freq
        rows = len(pos)
        qkv = normal(rows, (hq + 2 * hkv) * d, dtype=dt)  # the packed output of one projection
        table = _tables(g, batch, width)
        return dict(case=case, q=qkv[:, :hq * d].view(rows, hq, d), k=qkv[:, hq * d:(hq + hkv) * d].view(rows, hkv, d),
                    v=qkv[:, (hq + hkv) * d:].view(rows, hkv, d),
                    positions=torch.tensor(pos, dtype=torch.int32, device="cuda"),
                    seq_ids=torch.tensor(seqs, dtype=torch.int32, device="cuda"),
                    cos_sin=torch.cat([angle.cos(), angle.sin()], dim=1).float(), table=table,
                    k_pages=torch.zeros((batch * width, hkv, page, d), dtype=dt, device="cuda"),
                    v_pages=torch.zeros((batch * width, hkv, page, d), dtype=dt, device="cuda"),
                    q_out=torch.zeros((rows, hq, d), dtype=dt, device="cuda"))

    nodes = case["nodes"]
    parents, _ = _depths(nodes)
    parents = torch.tensor([parents] * batch, dtype=torch.int32, device="cuda")
    k_tree, v_tree = normal(batch, nodes, hkv, d, dtype=dt), normal(batch, nodes, hkv, d, dtype=dt)
    if op == "commit":
        width = -(-(case["length"] + 13 * batch + nodes) // page)
        # an accepted path of each sequence: from a node up to the root
        acc, alen = [], []
        tree = _depths(nodes)[0]
        ends = torch.randint(0, nodes, (batch,), generator=g, device="cuda").tolist()
        for b in range(batch):
            path, a = [], ends[b]
            while a > 0:
                path.append(a)
                a = tree[a]
            acc.append(path[::-1] + [-1] * (nodes - len(path)))
            alen.append(len(path))
        lens = [case["length"] + (13 * i) % (13 * batch) for i in range(batch)]
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(case=case, k_tree=k_tree, v_tree=v_tree, parents=parents,
                    hidden=normal(batch * nodes, case["hidden"], dtype=dt), table=_tables(g, batch, width),
                    k_pages=torch.zeros((batch * width, hkv, page, d), dtype=dt, device="cuda"),
                    v_pages=torch.zeros((batch * width, hkv, page, d), dtype=dt, device="cuda"),
                    lens=torch.tensor(lens, **i32), acc=torch.tensor(acc, **i32), alen=torch.tensor(alen, **i32),
                    new_lens=torch.zeros((batch,), **i32),
                    feat=torch.zeros((batch, nodes, case["hidden"]), dtype=dt, device="cuda"))

    shared = case["shared"]
    lens = [shared + n for n in _own_lens(case)]
    full, rest = shared // page, shared % page
    width = max(1, -(-max(lens) // page))
    table = _tables(g, batch, width)
    table[:, :full] = table[:1, :full].clone()  # the full pages of the prefix are the same pages
    k_pages, v_pages = normal(batch * width, hkv, page, d, dtype=dt), normal(batch * width, hkv, page, d, dtype=dt)
    if rest:  # the page in which the prefix ends was copied when the sequences parted
        last = table[:, full].long()
        for t in (k_pages, v_pages):
            t[last, :, :rest] = t[last[:1], :, :rest].clone()
    return dict(case=case, q=normal(batch, nodes, hq, d, dtype=dt), k_tree=k_tree, v_tree=v_tree, parents=parents,
                k_pages=k_pages, v_pages=v_pages, table=table, max_len=max(1, max(lens)),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                out=torch.empty((batch, nodes, hq, d), dtype=dt, device="cuda"))


# ------------------------------------------------------------------------------ plain form

def _rotate(x, cos, sin, rd, interleaved):
    """x [rows, heads, d] in 32 bits, its first rd columns rotated in pairs."""
    r, keep = x[..., :rd], x[..., rd:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :rd // 2], r[..., rd // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, keep], dim=-1)


def _plain_append(s):
    c = s["case"]
    rd, page = c["rotary"], c["page"]
    live = (s["positions"] >= 0).nonzero()[:, 0]
    pos, seq = s["positions"][live].long(), s["seq_ids"][live].long()
    cs = s["cos_sin"][pos][:, None, :]
    cos, sin = cs[..., :rd // 2], cs[..., rd // 2:]
    dt = s["q_out"].dtype
    s["q_out"][live] = _rotate(s["q"][live].float(), cos, sin, rd, c["interleaved"]).to(dt)
    where, slot = s["table"][seq, pos // page].long(), pos % page
    s["k_pages"][where, :, slot] = _rotate(s["k"][live].float(), cos, sin, rd, c["interleaved"]).to(dt)
    s["v_pages"][where, :, slot] = s["v"][live]
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _visible(parents):
    """[B, N, N]: whether node j is node i or one of its ancestors."""
    n = parents.shape[1]
    eye = torch.eye(n, device=parents.device)
    up = (parents[:, :, None] == torch.arange(n, device=parents.device)).float()
    return torch.linalg.matrix_power(eye + up, n) > 0


def _plain_attention(s):
    q, lens = s["q"], s["lens"].long()
    b, n, hq, d = q.shape
    hkv, page = s["k_pages"].shape[1:3]
    j = torch.arange(int(s["max_len"]), device=q.device)
    where, slot = s["table"][:, j // page].long(), (j % page)[None]
    inside = j[None] < lens[:, None]
    keys = torch.cat([s["k_pages"][where, :, slot], s["k_tree"]], dim=1).float()
    values = torch.cat([s["v_pages"][where, :, slot], s["v_tree"]], dim=1).float()
    seen = torch.cat([inside[:, None].expand(b, n, -1), _visible(s["parents"])], dim=2)
    qg = q.float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    score = torch.matmul(qg, keys.permute(0, 2, 3, 1)) / math.sqrt(d)
    score = score.view(b, hkv, hq // hkv, n, -1).masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(dim=-1, keepdim=True))
    p = p / p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), values.transpose(1, 2)).view(b, hkv, hq // hkv, n, d)
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d))
    return s["out"]


def _plain_commit(s):
    lens, alen = s["lens"].long(), s["alen"].long()
    b, n = s["acc"].shape
    page = s["k_pages"].shape[2]
    t = torch.arange(n, device=lens.device)[None]
    path = torch.cat([torch.zeros_like(s["acc"][:, :1]), s["acc"][:, :-1]], dim=1).long()
    seq, row = (t <= alen[:, None]).nonzero(as_tuple=True)
    node, pos = path[seq, row], lens[seq] + row
    where, slot = s["table"][seq, pos // page].long(), pos % page
    s["k_pages"][where, :, slot] = s["k_tree"][seq, node]
    s["v_pages"][where, :, slot] = s["v_tree"][seq, node]
    s["feat"][seq, row] = s["hidden"].view(b, n, -1)[seq, node]
    s["new_lens"].copy_(lens + alen + 1)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "feat": s["feat"], "lens": s["new_lens"]}


def _plain_logits(s):
    x, w8, ws = s["x"].float(), s["w8"], s["ws"]
    rows, hidden = x.shape
    vocab = w8.shape[0]
    kb, vb = -(-hidden // BLOCK), -(-vocab // BLOCK)
    pad = torch.nn.functional.pad(x, (0, kb * BLOCK - hidden)).view(rows, kb, BLOCK)
    # the smallest power of two that brings the block's largest magnitude within 448: the
    # quotients are exact and the only rounding is the one to 8 bits
    frac, exp = torch.frexp(pad.abs().amax(dim=-1, keepdim=True))
    scale = torch.ldexp(torch.ones_like(frac), (exp - 9 + (frac > 0.875).int()).clamp(min=-126))
    x = ((pad / scale).to(torch.float8_e4m3fn).float() * scale).view(rows, -1)[:, :hidden]
    w = w8.float() * ws.repeat_interleave(BLOCK, 0)[:vocab].repeat_interleave(BLOCK, 1)[:, :hidden]
    torch.matmul(x, w.t(), out=s["logits"])
    return s["logits"]


# ------------------------------------------------------------------------------ the framework's calls

def _own_run(s):
    from tree_verify_b200 import binding as eb
    c = s["case"]
    op = c["op"]
    if op == "logits":
        eb.quantize_rows(s["x"], s["x8"], s["xs"])
        eb.lm_head_logits_scaled(s["x8"], s["xs"], s["w8"], s["ws"], s["logits"])
        return s["logits"]
    if "shape" not in s:
        batch, width = s["table"].shape
        page = c["page"]
        longest = s["max_len"] if op == "attention" else width * page
        s["shape"] = eb.make_shape(batch, c.get("nodes", 1), c["hq"], c["hkv"], c["d"], longest,
                                   c.get("hidden", 8), 1, c["dtype"])
        s["pages"] = eb.make_pages(s["k_pages"].shape[0], page, width)
        if op == "attention":
            need = eb.paged_workspace_bytes(s["shape"], s["pages"], c["shared"])
            s["workspace"] = torch.empty((max(need, 256),), dtype=torch.uint8, device="cuda")
    if op == "append":
        eb.rope_append(s["shape"], s["pages"], s["q"], s["k"], s["v"], s["positions"], s["seq_ids"], s["cos_sin"],
                       s["k_pages"], s["v_pages"], s["table"], s["q_out"], interleaved=c["interleaved"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "commit":
        eb.commit_accepted_paged(s["shape"], s["pages"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                 s["k_tree"], s["v_tree"], s["hidden"], s["parents"], s["acc"], s["alen"],
                                 s["new_lens"], s["feat"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "feat": s["feat"], "lens": s["new_lens"]}
    eb.tree_attention_paged(s["shape"], s["pages"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                            c["shared"], s["k_tree"], s["v_tree"], s["parents"], s["out"], s["workspace"])
    return s["out"]


def run(state):
    if own:
        return _own_run(state)
    plain = {"append": _plain_append, "attention": _plain_attention, "commit": _plain_commit, "logits": _plain_logits}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ the work of a pass

def work(case):
    op = case["op"]
    if op == "logits":
        m, h, v = case["rows"], case["hidden"], case["vocab"]
        scales = 4 * (-(-h // BLOCK)) * (-(-v // BLOCK))
        return {"bytes": v * h + scales + 2 * m * h + 4 * m * v, "flops": 2 * m * h * v}
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "append":
        t = case["tokens"]
        return {"bytes": t * ((hq + 2 * hkv) * d * 2 * e + 4 * case["rotary"] + 8),
                "flops": 3 * t * (hq + hkv) * case["rotary"]}
    b, n = case["batch"], case["nodes"]
    depth = _depths(n)[1]
    if op == "commit":
        # the path to the middle node, on average
        rows = b * (1 + sum(depth) / n)
        return {"bytes": 2 * rows * (2 * hkv * d + case["hidden"]) * e + 8 * b * n, "flops": 0}
    lens = _own_lens(case)
    keys = n * sum(case["shared"] + x for x in lens) + b * sum(1 + x for x in depth)
    cached = case["shared"] + sum(lens)
    return {"bytes": e * d * (2 * hkv * (cached + b * n) + 2 * hq * b * n) + 4 * b * n, "flops": 4 * d * hq * keys}


# ------------------------------------------------------------------------------ exact values

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "logits":
        x = s["x"].double()
        rows, hidden = x.shape
        out = torch.empty(s["logits"].shape, dtype=torch.float64, device="cuda")
        xq = torch.empty_like(x)
        for k0 in range(0, hidden, BLOCK):
            part = x[:, k0:k0 + BLOCK]
            top = part.abs().max(dim=1, keepdim=True).values.clamp(min=1e-30)
            scale = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))
            xq[:, k0:k0 + BLOCK] = _to_e4m3(part / scale) * scale
        for v0 in range(0, case["vocab"], BLOCK * 64):
            w = s["w8"][v0:v0 + BLOCK * 64].double()
            for k0 in range(0, hidden, BLOCK):
                scale = s["ws"][v0 // BLOCK:v0 // BLOCK + 64, k0 // BLOCK].double()
                w[:, k0:k0 + BLOCK] *= scale.repeat_interleave(BLOCK)[:w.shape[0], None]
            out[:, v0:v0 + BLOCK * 64] = xq @ w.t()
        return out
    page = case["page"]
    if op == "append":
        rd = case["rotary"]
        q_out, k_pages, v_pages = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
        rows = s["positions"].shape[0] - case["padding"]
        pos, seq = s["positions"][:rows].long(), s["seq_ids"][:rows].long()
        c = torch.complex(s["cos_sin"][:, :rd // 2].double(), s["cos_sin"][:, rd // 2:].double())[pos]

        def turned(x):  # pairs as complex numbers, times the unit number of the angle
            x = x[:rows].double().clone()
            a = slice(0, rd, 2) if case["interleaved"] else slice(0, rd // 2)
            b = slice(1, rd, 2) if case["interleaved"] else slice(rd // 2, rd)
            z = torch.complex(x[:, :, a], x[:, :, b]) * c[:, None]
            x[:, :, a], x[:, :, b] = z.real, z.imag
            return x

        q_out[:rows] = turned(s["q"])
        page_of = torch.gather(s["table"][seq].long(), 1, (pos // page)[:, None])[:, 0]
        k_pages[page_of, :, pos % page] = turned(s["k"])
        v_pages[page_of, :, pos % page] = s["v"][:rows].double()
        return {"q": q_out, "k_pages": k_pages, "v_pages": v_pages}
    if op == "commit":
        k_pages, v_pages, feat = s["k_pages"].double(), s["v_pages"].double(), s["feat"].double()
        new = []
        for b in range(case["batch"]):
            length = int(s["lens"][b])
            nodes = [0] + s["acc"][b, :int(s["alen"][b])].tolist()
            for t, node in enumerate(nodes):
                at = int(s["table"][b, (length + t) // page])
                k_pages[at, :, (length + t) % page] = s["k_tree"][b, node].double()
                v_pages[at, :, (length + t) % page] = s["v_tree"][b, node].double()
                feat[b, t] = s["hidden"][b * case["nodes"] + node].double()
            new.append(length + len(nodes))
        return {"k_pages": k_pages, "v_pages": v_pages, "feat": feat,
                "lens": torch.tensor(new, dtype=torch.int32, device="cuda")}
    n, group = case["nodes"], case["hq"] // case["hkv"]
    parents = _depths(n)[0]
    mask = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        a = i
        while a >= 0:
            mask[i, a] = True
            a = parents[a]
    mask = mask.cuda()
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        length = int(s["lens"][b])
        pages = s["table"][b, :-(-length // page)].long()
        for h in range(case["hkv"]):
            k = torch.cat([s["k_pages"][pages, h].flatten(0, 1)[:length], s["k_tree"][b, :, h]]).double()
            v = torch.cat([s["v_pages"][pages, h].flatten(0, 1)[:length], s["v_tree"][b, :, h]]).double()
            see = torch.cat([torch.ones((n, length), dtype=torch.bool, device="cuda"), mask], dim=1)
            qh = s["q"][b, :, h * group:(h + 1) * group].double()
            score = torch.einsum("ngd,kd->ngk", qh, k) / math.sqrt(case["d"])
            score = score.masked_fill(~see[:, None], -math.inf)
            out[b, :, h * group:(h + 1) * group] = torch.einsum("ngk,kd->ngd", torch.softmax(score, dim=-1), v)
    return out


def _to_e4m3(x):
    """The nearest e4m3 value of each number (ties to even): 3 fraction bits, exponents from -6."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
