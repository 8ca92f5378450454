"""Measured cases of the operators a drafted step needs over a paged KV cache.

Three operators, each for fp16 pools and for E4M3 pools with one scale per KV
head:

  rope    rotary positions on a step's queries and keys, and the step's keys
          and values written to their slots of the rows' blocks;
  tree    attention of each row's drafted nodes over the row's cached tokens
          and the nodes their mask lets them see;
  commit  the accepted path's keys and values moved to the row's next
          positions, every layer at once, and the rows' new lengths.

``run`` computes a case in plain torch operations (32 bits, 64 where 32 lose
digits) or, where ``own`` is true, through the framework's operators.
``exact`` gives the same outputs in 64 bits from the definition.

Row lengths, node counts, trees and accepted paths follow from the case alone;
the values, the block permutation and the scales from the seed.
"""
import math
import random

import torch

own = False

D = 128
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases

def _case(name, op, rows, lo, hi, nodes_lo, nodes_hi, block, q_heads=12, kv_heads=2, fp8=False,
          spread="uniform", tall=0, shape=1, **kw):
    c = {"name": name, "op": op, "rows": rows, "lo": lo, "hi": hi, "nodes_lo": nodes_lo,
         "nodes_hi": nodes_hi, "block": block, "q_heads": q_heads, "kv_heads": kv_heads,
         "fp8": fp8, "spread": spread, "tall": tall, "shape": shape}
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a ragged batch: a new token a row, whole heads rotated
        _case("rope_step", "rope", 32, 16, 512, 1, 1, 64, tall=4096, layout="half", rot=128,
              scaling="none", far=0, fused=True),
        # a drafted tree a row, half of each head rotated, quantised as it is written
        _case("rope_tree_fp8", "rope", 32, 100, 2000, 8, 32, 16, fp8=True, shape=2,
              layout="interleaved", rot=64, scaling="ntk", far=0, fused=True),
        # prompts written whole, far along a context whose frequencies are scaled by parts
        _case("rope_prompt", "rope", 8, 0, 200, 1500, 2300, 64, shape=3, layout="half", rot=128,
              scaling="by_parts", far=98304, fused=True),
        # the smallest batch: a few short rows, small trees, 16-token blocks
        _case("tree_tiny", "tree", 4, 0, 200, 1, 8, 16, shape=4, mask=True),
        # a ragged serving batch with one long row
        _case("tree_mixed", "tree", 32, 16, 512, 8, 24, 64, tall=4096, shape=5, mask=True),
        # even lengths, quantised pools, a tree of 25 nodes
        _case("tree_even_fp8", "tree", 32, 1024, 1024, 25, 25, 64, fp8=True, shape=6, mask=True),
        # few rows over a long context
        _case("tree_long", "tree", 4, 32768, 32768, 5, 16, 64, shape=7, mask=True),
        # a chain of drafted tokens a row, lengths over three decades, quantised pools
        _case("tree_chain_fp8", "tree", 96, 16, 8192, 3, 7, 16, fp8=True, spread="log", shape=8,
              mask=False),
        # other head counts, a block size that is no power of two, odd lengths
        _case("tree_wide_heads", "tree", 16, 701, 2111, 1, 48, 48, q_heads=32, kv_heads=8, shape=9,
              mask=True),
        # the largest: many rows, long prefixes, wide trees
        _case("tree_large", "tree", 64, 4000, 4096, 64, 64, 64, shape=10, mask=True),
        # one layer's accepted tokens
        _case("commit_step", "commit", 32, 16, 512, 8, 24, 64, tall=2048, shape=11, layers=1),
        # all layers of a model at once, quantised pools, 16-token blocks
        _case("commit_layers_fp8", "commit", 64, 16, 300, 16, 48, 16, fp8=True, shape=12,
              layers=28),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "commit"])
    heads = rng.choice([(12, 2), (32, 8), (8, 1), (4, 4), (28, 4)])
    c = {"op": op, "q_heads": heads[0], "kv_heads": heads[1], "block": rng.choice([16, 32, 48, 64, 128]),
         "fp8": rng.random() < 0.4, "spread": rng.choice(["uniform", "log"]), "tall": 0,
         "shape": rng.randrange(1 << 30)}
    if op == "rope":
        c["layout"] = rng.choice(["half", "interleaved"])
        c["rot"] = rng.choice([32, 64, 96, 128])
        c["scaling"] = rng.choice(["none", "linear", "ntk", "by_parts"])
        c["far"] = rng.choice([0, 0, _logint(rng, 100, 1000000)])
        c["fused"] = rng.random() < 0.5
        c["rows"] = _logint(rng, 1, 96)
        c["lo"] = rng.randrange(0, 100)
        c["hi"] = c["lo"] + _logint(rng, 1, 2000)
        # up to about 10,000 tokens over all rows
        c["nodes_lo"] = 1
        c["nodes_hi"] = max(1, min(2048, _logint(rng, 1, 10000) // c["rows"]))
    elif op == "tree":
        c["mask"] = rng.random() < 0.75
        c["rows"] = _logint(rng, 1, 96)
        # bytes and node-tokens stay below the largest listed case's
        top = max(2, min(32768, 500000 // (c["rows"] * c["kv_heads"])))
        c["hi"] = _logint(rng, 1, top)
        c["lo"] = rng.randrange(0, c["hi"] + 1) if c["spread"] == "uniform" else max(1, c["hi"] // 50)
        most = int(12e6 * 12 / (c["rows"] * c["hi"] * c["q_heads"])) + 1
        c["nodes_hi"] = max(1, min(_logint(rng, 1, 128), most))
        c["nodes_lo"] = rng.randrange(0, c["nodes_hi"] + 1)
        if c["rows"] > 2 and rng.random() < 0.3:
            c["tall"] = min(top, 4 * c["hi"] + 1)
            c["hi"] = max(1, c["hi"] // 2)
            c["lo"] = min(c["lo"], c["hi"])
    else:
        c["rows"] = _logint(rng, 1, 96)
        c["layers"] = rng.choice([1, 4, 28]) if c["rows"] * c["kv_heads"] < 100 else 1
        c["lo"] = rng.randrange(0, 100)
        c["hi"] = c["lo"] + _logint(rng, 1, 300)
        c["nodes_hi"] = _logint(rng, 2, 64)
        c["nodes_lo"] = rng.randrange(1, c["nodes_hi"] + 1)
    return c


# ---------------------------------------------------------------------------
# shapes: all that follows from the case alone

def _shape(case):
    rng = random.Random(case["shape"])
    rows = case["rows"]
    prefix, nodes = [], []
    for _ in range(rows):
        if case["spread"] == "log":
            prefix.append(int(math.exp(rng.uniform(math.log(max(1, case["lo"])),
                                                   math.log(max(1, case["hi"]))))))
        else:
            prefix.append(rng.randint(case["lo"], case["hi"]))
        nodes.append(rng.randint(case["nodes_lo"], case["nodes_hi"]))
    if case["tall"]:
        prefix[rng.randrange(rows)] = case["tall"]
    if not any(nodes):
        nodes[0] = 1
    # drafted trees: node 0 is the root; the most likely continuation comes
    # first as a chain, the alternatives follow, each below an earlier node
    parents, depths = [], []
    for n in nodes:
        trunk = (n + 2) // 3
        par = []
        for i in range(n):
            if i <= trunk:
                par.append(i - 1)
            else:
                par.append(rng.randint(max(0, i - 12), i - 1))
        dep = []
        for p in par:
            dep.append(0 if p < 0 else dep[p] + 1)
        parents.append(par)
        depths.append(dep)
    return prefix, nodes, parents, depths


def _paths(case, nodes):
    """Accepted nodes of each row: the trunk for a while, then alternatives."""
    rng = random.Random(case["shape"] + 1)
    out = []
    for n in nodes:
        trunk = (n + 2) // 3
        keep = rng.randint(0, trunk)          # accepted on the trunk: nodes 0 .. keep - 1
        path = list(range(keep))
        first = trunk
        while len(path) < trunk and first < n and rng.random() < 0.8:
            first = rng.randint(first, n - 1)
            path.append(first)
            first += 1
        out.append(path)
    return out


def _frequencies(case):
    """float64 angular frequencies of the rotated pairs."""
    rot, base, s, l0 = case["rot"], 10000.0, 8.0, 16384.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * s ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "by_parts":
        ramp = ((l0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f = (1 - ramp) * f / s + ramp * f
    return f


def _mscale(case):
    return 0.1 * math.log(8.0) + 1.0 if case.get("scaling") == "by_parts" else 1.0


# ---------------------------------------------------------------------------
# inputs

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _inputs(case, seed):
    prefix, nodes, parents, depths = _shape(case)
    rows, bs, hq, hk, fp8 = case["rows"], case["block"], case["q_heads"], case["kv_heads"], case["fp8"]
    gen = torch.Generator(device=DEV).manual_seed(seed)
    lens = [p + n for p, n in zip(prefix, nodes)]
    need = [(n + bs - 1) // bs for n in lens]
    nb = max(1, sum(need))
    perm = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)
    mb = max(1, max(need))
    tables = torch.full((rows, mb), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(need):
        tables[r, :n] = perm[at:at + n]
        at += n
    starts = [0]
    for n in nodes:
        starts.append(starts[-1] + n)
    total = starts[-1]
    s = {"case": case, "lens": lens, "nodes": nodes, "starts": starts, "total": total,
         "tables": tables, "seq_lens": _i32(lens), "q_start": _i32(starts), "nb": nb,
         "max_len": max(lens), "parents": parents, "scale": float(torch.tensor(1 / math.sqrt(D)))}
    layers = case.get("layers", 1)
    for name in ("k_pool", "v_pool"):
        if fp8:
            # codes of unit normal values at a per-head scale
            sc = 0.02 + 0.02 * torch.rand(hk, generator=gen, device=DEV)
            pool = torch.empty((layers, nb, bs, hk, D), dtype=torch.uint8, device=DEV)
            for i in range(layers):
                x = _randn((nb, bs, hk, D), gen) / sc[:, None]
                pool[i] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name[0] + "_scale"] = sc
        else:
            pool = torch.empty((layers, nb, bs, hk, D), dtype=torch.float16, device=DEV)
            for i in range(layers):
                pool[i] = _randn((nb, bs, hk, D), gen).half()
            s[name[0] + "_scale"] = None
        s[name] = pool if case["op"] == "commit" else pool[0]
    if case["op"] == "rope":
        if case["fused"]:
            # views of one projection's output, a token's queries, keys and values in a row
            qkv = _randn((total, hq + 2 * hk, D), gen).half()
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            s["q"] = _randn((total, hq, D), gen).half()
            s["k"] = _randn((total, hk, D), gen).half()
            s["v"] = _randn((total, hk, D), gen).half()
        pos = [case["far"] + prefix[r] + d for r in range(rows) for d in depths[r]]
        s["rope_positions"] = _i32(pos)
        s["freqs"] = _frequencies(case).to(DEV)
        s["q_out"] = torch.empty((total, hq, D), dtype=torch.float16, device=DEV)
    elif case["op"] == "tree":
        s["q"] = _randn((total, hq, D), gen).half()
        s["out"] = torch.empty((total, hq, D), dtype=torch.float16, device=DEV)
        s["mask"] = None
        if case["mask"]:
            words = (max(nodes) + 31) // 32
            bits = [[0] * words for _ in range(total)]
            for r in range(rows):
                for i, p in enumerate(parents[r]):
                    row = bits[starts[r] + i]
                    if p >= 0:
                        row[:] = bits[starts[r] + p]
                    row[i // 32] |= 1 << (i % 32)
            signed = [[w - (1 << 32) if w >= 1 << 31 else w for w in row] for row in bits]
            s["mask"] = _i32(signed)
    else:
        paths = _paths(case, nodes)
        width = max(1, max(len(p) for p in paths))
        s["path"] = _i32([p + [-1] * (width - len(p)) for p in paths])
        s["path_lens"] = _i32([len(p) for p in paths])
        s["path_sizes"] = [len(p) for p in paths]
        s["new_lens"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from paged_kv_cache_06_gb300 import ops
        if case["op"] == "rope":
            s["rates"] = ops.rope_rates(s["freqs"])
        elif case["op"] == "tree":
            s["workspace"] = ops.alloc_tree_workspace(case["rows"], s["total"], case["q_heads"],
                                                      case["kv_heads"], D, case["block"])
    return s


# ---------------------------------------------------------------------------
# one pass

def _values(pool):
    """A pool as the values its elements stand for (a view)."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "tree": _own_tree, "commit": _own_commit}[op](state)
    return {"rope": _plain_rope, "tree": _plain_tree, "commit": _plain_commit}[op](state)


def _own_rope(s):
    from paged_kv_cache_06_gb300 import ops
    c = s["case"]
    ops.rope_append(s["k_pool"], s["v_pool"], s["tables"], s["seq_lens"], s["q_start"], s["k"],
                    s["v"], s["rates"], s["max_len"], layout=c["layout"], q=s["q"],
                    q_out=s["q_out"], rope_positions=s["rope_positions"], mscale=_mscale(c),
                    k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["q_out"], _values(s["k_pool"]), _values(s["v_pool"])


def _own_tree(s):
    from paged_kv_cache_06_gb300 import ops
    ops.tree_attention(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["seq_lens"],
                       s["q_start"], s["scale"], s["max_len"], s["workspace"], mask=s["mask"],
                       k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["out"]


def _own_commit(s):
    from paged_kv_cache_06_gb300 import ops
    ops.tree_commit(s["k_pool"], s["v_pool"], s["tables"], s["seq_lens"], s["q_start"], s["path"],
                    s["path_lens"], s["max_len"], new_seq_lens=s["new_lens"])
    return _values(s["k_pool"]), _values(s["v_pool"]), s["new_lens"]


def _token_rows(s):
    """Row of each of the step's tokens, and its index among the row's."""
    counts = (s["q_start"][1:] - s["q_start"][:-1]).long()
    row = torch.repeat_interleave(torch.arange(len(s["nodes"]), device=DEV), counts,
                                  output_size=s["total"])
    index = torch.arange(s["total"], device=DEV) - s["q_start"].long()[row]
    return row, index, counts


def _store(pool, block, slot, x, scale):
    if scale is None:
        pool[block, slot] = x.half()
    else:
        q = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        pool[block, slot] = q.view(torch.uint8)


def _plain_rope(s):
    c = s["case"]
    rot, bs = c["rot"], c["block"]
    row, index, counts = _token_rows(s)
    # angles of far positions need 64 bits
    angle = s["rope_positions"].double()[:, None] * s["freqs"][None, :]
    cos = (torch.cos(angle) * _mscale(c)).float()[:, None, :]
    sin = (torch.sin(angle) * _mscale(c)).float()[:, None, :]

    def turn(x):
        x = x.float()
        y = x.clone()
        if c["layout"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2] = a * cos - b * sin
            y[..., rot // 2:rot] = a * sin + b * cos
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2] = a * cos - b * sin
            y[..., 1:rot:2] = a * sin + b * cos
        return y

    s["q_out"].copy_(turn(s["q"]))
    pos = s["seq_lens"].long()[row] - counts[row] + index
    block = s["tables"][row, pos // bs].long()
    _store(s["k_pool"], block, pos % bs, turn(s["k"]), s["k_scale"])
    _store(s["v_pool"], block, pos % bs, s["v"].float(), s["v_scale"])
    return s["q_out"], _values(s["k_pool"]), _values(s["v_pool"])


def _plain_tree(s):
    c = s["case"]
    bs, hq, hk = c["block"], c["q_heads"], c["kv_heads"]
    g = hq // hk
    for r, n in enumerate(s["nodes"]):
        if n == 0:
            continue
        length = s["lens"][r]
        prefix = length - n
        blocks = s["tables"][r, :(length + bs - 1) // bs].long()
        k = _values(s["k_pool"][blocks]).float().reshape(-1, hk, D)[:length].transpose(0, 1)
        v = _values(s["v_pool"][blocks]).float().reshape(-1, hk, D)[:length].transpose(0, 1)
        if s["k_scale"] is not None:
            k = k * s["k_scale"][:, None, None]
            v = v * s["v_scale"][:, None, None]
        q0 = s["starts"][r]
        q = s["q"][q0:q0 + n].float().reshape(n, hk, g, D).permute(1, 0, 2, 3).reshape(hk, n * g, D)
        score = torch.matmul(q, k.transpose(1, 2)).mul_(s["scale"])
        node = torch.arange(n, device=DEV)
        if s["mask"] is None:
            seen = node[None, :] <= node[:, None]
        else:
            words = s["mask"][q0:q0 + n].long()
            seen = ((words[:, node // 32] >> (node % 32)[None, :]) & 1) != 0
        score = score.reshape(hk, n, g, length)
        score[..., prefix:].masked_fill_(~seen[None, :, None, :], float("-inf"))
        top = score.amax(-1, keepdim=True)
        top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
        weight = score.sub_(top).exp_()
        total = weight.sum(-1, keepdim=True)
        weight = torch.where(total > 0, weight / total, torch.zeros_like(weight))
        out = torch.matmul(weight.reshape(hk, n * g, length), v).reshape(hk, n, g, D)
        s["out"][q0:q0 + n] = out.permute(1, 0, 2, 3).reshape(n, hq, D).half()
    return s["out"]


def _plain_commit(s):
    bs = s["case"]["block"]
    rows, width = s["path"].shape
    prefix = (s["seq_lens"] - (s["q_start"][1:] - s["q_start"][:-1])).long()
    j = torch.arange(width, device=DEV)[None, :]
    row, step = ((j < s["path_lens"][:, None]) & (s["path"] != j)).nonzero(as_tuple=True)
    src = prefix[row] + s["path"].long()[row, step]
    dst = prefix[row] + step
    sb, db = s["tables"][row, src // bs].long(), s["tables"][row, dst // bs].long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, db, dst % bs] = pool[:, sb, src % bs]
    torch.add(prefix, s["path_lens"], out=s["new_lens"])
    return _values(s["k_pool"]), _values(s["v_pool"]), s["new_lens"]


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    prefix, nodes, parents, depths = _shape(case)
    hq, hk, bs = case["q_heads"], case["kv_heads"], case["block"]
    elt = 1 if case["fp8"] else 2
    total = sum(nodes)
    lens = [p + n for p, n in zip(prefix, nodes)]
    index = 4 * (2 * case["rows"] + 1)
    if case["op"] == "rope":
        entries = sum((n + bs - 1) // bs - p // bs for p, n in zip(prefix, lens))
        read = total * (hq + 2 * hk) * D * 2 + total * 4 + 8 * (case["rot"] // 2)
        write = total * hq * D * 2 + 2 * total * hk * D * elt
        return {"bytes": read + write + index + 4 * entries,
                "flops": 3 * total * (hq + hk) * case["rot"]}
    if case["op"] == "tree":
        entries = sum((n + bs - 1) // bs for n in lens)
        kv = 2 * sum(n for n, c in zip(lens, nodes) if c) * hk * D * elt
        mask = total * ((max(nodes) + 31) // 32) * 4 if case["mask"] else 0
        seen = 0
        for p, par, dep in zip(prefix, parents, depths):
            for i, d in enumerate(dep):
                seen += p + (d + 1 if case["mask"] else i + 1)
        return {"bytes": kv + 2 * total * hq * D * 2 + mask + index + 4 * entries,
                "flops": 4 * D * hq * seen}
    moved = sum(1 for p in _paths(case, nodes) for j, n in enumerate(p) if n != j)
    return {"bytes": moved * 2 * 2 * hk * D * elt * case["layers"] + index + 8 * case["rows"]
            + 4 * sum(len(p) for p in _paths(case, nodes)) + 8 * moved, "flops": 0}


# ---------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    if case["op"] == "commit":
        return None  # moved, not computed
    s = _inputs(case, seed)
    prefix, nodes, parents, depths = _shape(case)
    bs, hq, hk = case["block"], case["q_heads"], case["kv_heads"]
    group = hq // hk

    def widen(pool):
        return _values(pool).to(torch.float64)

    if case["op"] == "rope":
        rot, half = case["rot"], case["rot"] // 2
        at = torch.tensor([case["far"] + prefix[r] + d for r in range(case["rows"])
                           for d in depths[r]], dtype=torch.float64, device=DEV)
        turn = torch.polar(torch.full((s["total"], half), _mscale(case), dtype=torch.float64,
                                      device=DEV), torch.outer(at, _frequencies(case).to(DEV)))

        def rotate(x):
            x = x.to(torch.float64)
            head, rest = x[..., :rot], x[..., rot:]
            if case["layout"] == "half":
                z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous())
                z = z * turn[:, None, :]
                return torch.cat([z.real, z.imag, rest], dim=-1)
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous())
            z = torch.view_as_real(z * turn[:, None, :])
            return torch.cat([z.flatten(-2), rest], dim=-1)

        slots = []
        tables = s["tables"].tolist()
        for r, n in enumerate(nodes):
            for i in range(n):
                t = prefix[r] + i
                slots.append(tables[r][t // bs] * bs + t % bs)
        slots = torch.tensor(slots, device=DEV)
        outs = [rotate(s["q"])]
        for name, x in (("k", rotate(s["k"])), ("v", s["v"].to(torch.float64))):
            pool = widen(s[name + "_pool"])
            sc = s[name + "_scale"]
            if sc is not None:
                x = (x / sc.to(torch.float64)[:, None]).clamp(-448, 448)
            pool.view(-1, hk, D)[slots] = x
            outs.append(pool)
        return tuple(outs)

    out = torch.zeros((s["total"], hq, D), dtype=torch.float64, device=DEV)
    tables = s["tables"].tolist()
    for r, n in enumerate(nodes):
        if n == 0:
            continue
        length = prefix[r] + n
        slots = torch.tensor([tables[r][t // bs] * bs + t % bs for t in range(length)], device=DEV)
        keys = widen(s["k_pool"].view(-1, hk, D)[slots])
        vals = widen(s["v_pool"].view(-1, hk, D)[slots])
        if s["k_scale"] is not None:
            keys = keys * s["k_scale"].to(torch.float64)[None, :, None]
            vals = vals * s["v_scale"].to(torch.float64)[None, :, None]
        seen = torch.ones((n, length), dtype=torch.bool)
        seen[:, prefix[r]:] = False
        for i, par in enumerate(parents[r]):
            if case["mask"]:
                j = i
                while j >= 0:
                    seen[i, prefix[r] + j] = True
                    j = parents[r][j]
            else:
                seen[i, prefix[r]:prefix[r] + i + 1] = True
        bias = torch.zeros((n, length), dtype=torch.float64)
        bias[~seen] = -math.inf
        bias = bias.to(DEV)
        q0 = s["starts"][r]
        for h in range(hq):
            score = s["q"][q0:q0 + n, h].to(torch.float64) @ keys[:, h // group].T
            score = score * s["scale"] + bias
            out[q0:q0 + n, h] = torch.softmax(score, dim=-1) @ vals[:, h // group]
    return out
