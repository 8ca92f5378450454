"""Measured cases of the operators that keep a paged KV cache within a budget.

Four operators, each for fp16 pools and for E4M3 pools with one scale per KV
head:

  norm     per-head norms and rotary positions on a step's queries and keys, and
           the step's keys and values written to their slots of the rows' blocks;
  decode   attention of one new token a row, and the weight that each cached
           token got added to its running sum;
  prefill  the weights that a prompt's queries, or its last few, give to the
           row's tokens, added to the same sums;
  evict    the tokens of lowest weight dropped from each KV head's list, the
           others moved together, every layer at once.

``run`` computes a case in plain torch operations (32 bits, 64 for the angles of
far positions) or, where ``own`` is true, through the framework's operators.
``exact`` gives the same outputs in 64 bits from the definition.

Row lengths and chunk sizes follow from the case alone; the values, the block
permutation and the scales from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases

def _case(name, op, rows, lo, hi, block, q_heads=12, kv_heads=2, dim=128, fp8=False, tall=0,
          spread="uniform", shape=1, **kw):
    c = {"name": name, "op": op, "rows": rows, "lo": lo, "hi": hi, "block": block,
         "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "fp8": fp8, "tall": tall,
         "spread": spread, "shape": shape}
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a ragged batch: a new token a row, whole heads rotated
        _case("norm_step", "norm", 32, 16, 512, 64, tall=4096, nodes_lo=1, nodes_hi=1,
              layout="half", rot=128, far=0, fused=True),
        # several drafted tokens a row, half of each head rotated, quantised as it is written
        _case("norm_drafts_fp8", "norm", 32, 100, 2000, 16, fp8=True, shape=2, nodes_lo=8,
              nodes_hi=32, layout="interleaved", rot=64, far=100000, fused=True),
        # whole prompts, queries, keys and values views of one projection's output
        _case("norm_prompt", "norm", 8, 0, 200, 64, shape=3, nodes_lo=1500, nodes_hi=2300,
              layout="half", rot=128, far=0, fused=True),
        # a decode step of a ragged batch with one long row
        _case("decode_mixed", "decode", 32, 16, 512, 64, tall=4096, shape=4),
        # even lengths, quantised pools
        _case("decode_even_fp8", "decode", 32, 1024, 1024, 64, fp8=True, shape=5),
        # few rows over a long context
        _case("decode_long", "decode", 4, 32768, 32768, 64, shape=6),
        # the last 32 queries of a prompt's last chunk look back over it, quantised pools
        _case("window_fp8", "prefill", 16, 500, 4000, 16, fp8=True, shape=7, nodes_lo=100,
              nodes_hi=512, window=32),
        # every query of a 512-token chunk over what is cached, other head counts
        _case("chunk", "prefill", 8, 300, 2100, 48, q_heads=32, kv_heads=8, shape=8, nodes_lo=512,
              nodes_hi=512, window=0),
        # every query of whole prompts
        _case("prompts", "prefill", 4, 0, 0, 64, shape=9, nodes_lo=3900, nodes_hi=4096, window=0),
        # every layer of a model after one step past the budget: a token a list goes
        _case("evict_step", "evict", 32, 1025, 1025, 16, shape=10, layers=28, budget=1024, sinks=4,
              recent=64, tracked=True),
        # every layer after a ragged stretch of steps, quantised pools
        _case("evict_stretch_fp8", "evict", 16, 1900, 2304, 64, fp8=True, shape=11, layers=28,
              budget=2048, sinks=4, recent=256, tracked=True),
        # long prompts cut down to an eighth, four layers at a time
        _case("evict_prompt", "evict", 4, 30000, 32768, 64, shape=12, layers=4, budget=4096,
              sinks=4, recent=512, tracked=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "decode", "prefill", "evict"])
    heads = rng.choice([(12, 2), (32, 8), (8, 1), (4, 4), (28, 4)])
    c = {"op": op, "q_heads": heads[0], "kv_heads": heads[1], "dim": 128,
         "block": rng.choice([16, 32, 48, 64, 128]), "fp8": rng.random() < 0.4, "tall": 0,
         "spread": rng.choice(["uniform", "log"]), "shape": rng.randrange(1 << 30)}
    rows = c["rows"] = _logint(rng, 1, 96)
    if op == "norm":
        c["dim"] = rng.choice([64, 96, 128, 128, 256])
        c["layout"] = rng.choice(["half", "interleaved"])
        c["rot"] = rng.choice([32, 64, c["dim"], c["dim"]])
        c["far"] = rng.choice([0, 0, _logint(rng, 100, 1000000)])
        c["fused"] = rng.random() < 0.5
        c["lo"] = rng.randrange(0, 100)
        c["hi"] = c["lo"] + _logint(rng, 1, 2000)
        c["nodes_lo"] = 1
        c["nodes_hi"] = max(1, min(2048, _logint(rng, 1, 8000) // rows))
    elif op == "decode":
        top = max(2, min(32768, 250000 // (rows * c["kv_heads"])))
        c["hi"] = _logint(rng, 1, top)
        c["lo"] = rng.randrange(0, c["hi"] + 1) if c["spread"] == "uniform" else max(1, c["hi"] // 50)
        if rows > 2 and rng.random() < 0.3:
            c["hi"] = max(1, c["hi"] // 2)
            c["lo"] = min(c["lo"], c["hi"])
            c["tall"] = min(top, 4 * c["hi"] + 1)
    elif op == "prefill":
        c["window"] = rng.choice([0, 1, 16, 32, 64, _logint(rng, 1, 500)])
        c["nodes_hi"] = _logint(rng, 1, max(2, 16000 // rows))
        # (query, key, head) triples stay below the largest listed case's
        top = max(2, min(32768, 200000 // (rows * c["kv_heads"])))
        seen = min(c["nodes_hi"], c["window"] or c["nodes_hi"])
        top = max(2, min(top, int(4e8 / (rows * seen * c["q_heads"]))))
        c["nodes_hi"] = min(c["nodes_hi"], top)
        c["nodes_lo"] = rng.randrange(0, c["nodes_hi"] + 1)
        c["hi"] = _logint(rng, 1, max(2, top - c["nodes_hi"]))
        c["lo"] = rng.randrange(0, c["hi"] + 1)
    else:
        c["layers"] = rng.choice([1, 4, 28])
        lists = c["layers"] * rows * c["kv_heads"]
        top = max(40, min(32768, 1000000 // lists))
        c["hi"] = _logint(rng, 20, top)
        c["lo"] = rng.randrange(c["hi"] // 2, c["hi"] + 1)
        c["budget"] = rng.randrange(1, c["hi"] + 1)
        c["sinks"] = min(c["budget"], rng.choice([0, 4]))
        c["recent"] = rng.randrange(0, (c["budget"] - c["sinks"]) // 2 + 1)
        c["tracked"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# sizes: all that follows from the case alone

def _sizes(case):
    """Tokens cached before the step, and new tokens, of each row."""
    rng = random.Random(case["shape"])
    before, new = [], []
    for _ in range(case["rows"]):
        if case["spread"] == "log":
            before.append(int(math.exp(rng.uniform(math.log(max(1, case["lo"])),
                                                   math.log(max(1, case["hi"]))))))
        else:
            before.append(rng.randint(case["lo"], case["hi"]))
        if case["op"] in ("norm", "prefill"):
            new.append(rng.randint(case["nodes_lo"], case["nodes_hi"]))
        else:
            new.append(0)
    if case["tall"]:
        before[rng.randrange(case["rows"])] = case["tall"]
    if case["op"] in ("norm", "prefill") and not any(new):
        new[0] = 1
    if case["op"] == "decode" and not any(before):
        before[0] = 1
    return before, new


def _frequencies(case):
    """float64 angular frequencies of the rotated pairs."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    return 10000.0 ** (-2.0 * i / case["rot"])


# ---------------------------------------------------------------------------
# inputs

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _inputs(case, seed):
    before, new = _sizes(case)
    rows, bs, hq, hk, d = (case[k] for k in ("rows", "block", "q_heads", "kv_heads", "dim"))
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)

    lens = [b + n for b, n in zip(before, new)]
    need = [(n + bs - 1) // bs for n in lens]
    nb = max(1, sum(need))
    perm = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32).tolist()
    width = max(1, max(need))
    tables, at = [], 0
    for n in need:
        tables.append(perm[at:at + n] + [-1] * (width - n))
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    total = starts[-1]
    s = {"case": case, "lens": lens, "new": new, "starts": starts, "total": total, "nb": nb,
         "tables": _i32(tables), "seq_lens": _i32(lens), "max_len": max(lens),
         "scale": float(torch.tensor(1 / math.sqrt(d)))}
    layers = case.get("layers", 1)
    for name in ("k_pool", "v_pool"):
        s[name[0] + "_scale"] = None
        if case["fp8"]:
            # codes of unit normal values at a per-head scale
            sc = 0.02 + 0.02 * torch.rand(hk, generator=gen, device=DEV)
            s[name[0] + "_scale"] = sc
            pool = torch.empty((layers, nb, bs, hk, d), dtype=torch.uint8, device=DEV)
            for i in range(layers):
                x = (randn(nb, bs, hk, d) / sc[:, None]).clamp(-448, 448)
                pool[i] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            pool = torch.empty((layers, nb, bs, hk, d), dtype=torch.float16, device=DEV)
            for i in range(layers):
                pool[i] = randn(nb, bs, hk, d).half()
        s[name] = pool if case["op"] == "evict" else pool[0]
    stride = (max(lens) + 3) // 4 * 4
    if case["op"] == "norm":
        if case["fused"]:
            # views of one projection's output, a token's queries, keys and values in a row
            qkv = randn(total, hq + 2 * hk, d).half()
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            s["q"], s["k"], s["v"] = (randn(total, h, d).half() for h in (hq, hk, hk))
        s["q_weight"] = (1 + 0.2 * randn(d)).half()
        s["k_weight"] = (1 + 0.2 * randn(d)).half()
        s["q_start"] = _i32(starts)
        s["rope_positions"] = _i32([case["far"] + before[r] + i for r in range(rows)
                                    for i in range(new[r])])
        s["freqs"] = _frequencies(case).to(DEV)
        s["q_out"] = torch.empty((total, hq, d), dtype=torch.float16, device=DEV)
    elif case["op"] == "decode":
        s["q"] = randn(rows, hq, d).half()
        s["out"] = torch.empty((rows, hq, d), dtype=torch.float16, device=DEV)
        # what earlier steps gave: most tokens little, a few much
        s["weights"] = torch.exp(2 * randn(rows, hk, stride) - 6)
    elif case["op"] == "prefill":
        s["q"] = randn(total, hq, d).half()
        s["q_start"] = _i32(starts)
        s["weights"] = torch.exp(2 * randn(rows, hk, stride) - 6)
    else:
        w = torch.exp(2 * randn(layers, rows, hk, stride) - 3)
        # some tokens never got a weight that 32 bits hold
        dead = torch.rand(w.shape, generator=gen, device=DEV) < 0.02
        s["weights"] = w.masked_fill_(dead, 0.0)
        s["tracked"] = [min(n, case["budget"]) if case["tracked"] else 0 for n in lens]
        # a list's recorded positions: any of the tokens that the row has had, in any order
        had = [2 * t for t in s["tracked"]]
        key = torch.rand((layers, rows, hk, max(1, max(had))), generator=gen, device=DEV)
        key.masked_fill_(torch.arange(key.shape[-1], device=DEV) >= _i32(had)[None, :, None, None], 2)
        pos = key.argsort(-1)[..., :max(1, max(s["tracked"]))].to(torch.int32)
        s["token_pos"] = torch.zeros((layers, rows, hk, stride), dtype=torch.int32, device=DEV)
        n = min(stride, pos.shape[-1])
        s["token_pos"][..., :n] = pos[..., :n]
        s["next_pos"] = _i32([h + n - t for h, n, t in zip(had, lens, s["tracked"])])
        s["tracked"] = _i32(s["tracked"])
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["token_pos_out"] = torch.zeros_like(s["token_pos"])
        s["new_lens"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from paged_kv_cache_06_gb300 import ops
        c = case
        heads = (c["q_heads"], c["kv_heads"], c["dim"])
        if c["op"] == "norm":
            s["rates"] = ops.rope_rates(s["freqs"])
        elif c["op"] == "decode":
            s["workspace"] = ops.alloc_decode_weights_workspace(c["rows"], *heads, s["max_len"],
                                                                c["block"])
        elif c["op"] == "prefill":
            s["workspace"] = ops.alloc_prefill_weights_workspace(
                c["rows"], s["total"], *heads, s["max_len"], c["block"], window=c["window"] or None)
    return s


# ---------------------------------------------------------------------------
# one pass

def _values(pool):
    """A pool as the values its elements stand for (a view)."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "decode": _own_decode, "prefill": _own_prefill,
                "evict": _own_evict}[op](state)
    return {"norm": _plain_norm, "decode": _plain_decode, "prefill": _plain_prefill,
            "evict": _plain_evict}[op](state)


def _own_norm(s):
    from paged_kv_cache_06_gb300 import ops
    ops.norm_rope_append(s["k_pool"], s["v_pool"], s["tables"], s["seq_lens"], s["q_start"], s["k"],
                         s["v"], s["rates"], s["k_weight"], s["max_len"], eps=EPS,
                         layout=s["case"]["layout"], q=s["q"], q_out=s["q_out"],
                         q_weight=s["q_weight"], rope_positions=s["rope_positions"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["q_out"], _values(s["k_pool"]), _values(s["v_pool"])


def _own_decode(s):
    from paged_kv_cache_06_gb300 import ops
    ops.decode_weights(s["out"], s["weights"], s["q"], s["k_pool"], s["v_pool"], s["tables"],
                       s["seq_lens"], s["scale"], s["max_len"], s["workspace"],
                       k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["out"], s["weights"]


def _own_prefill(s):
    from paged_kv_cache_06_gb300 import ops
    ops.prefill_weights(s["weights"], s["q"], s["k_pool"], s["tables"], s["seq_lens"], s["q_start"],
                        s["scale"], s["max_len"], s["workspace"], window=s["case"]["window"] or None,
                        k_scale=s["k_scale"])
    return s["weights"]


def _own_evict(s):
    from paged_kv_cache_06_gb300 import ops
    c = s["case"]
    ops.evict(s["k_pool"], s["v_pool"], s["tables"], s["seq_lens"], s["weights"], s["token_pos"],
              c["budget"], s["max_len"], sinks=c["sinks"], recent=c["recent"], tracked=s["tracked"],
              next_pos=s["next_pos"], weights_out=s["weights_out"],
              token_pos_out=s["token_pos_out"], new_seq_lens=s["new_lens"])
    return (_values(s["k_pool"]), _values(s["v_pool"]), s["weights_out"], s["token_pos_out"],
            s["new_lens"])


def _store(pool, block, slot, x, scale):
    if scale is None:
        pool[block, slot] = x.half()
    else:
        q = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        pool[block, slot] = q.view(torch.uint8)


def _plain_norm(s):
    c = s["case"]
    rot, bs = c["rot"], c["block"]
    counts = (s["q_start"][1:] - s["q_start"][:-1]).long()
    row = torch.repeat_interleave(torch.arange(c["rows"], device=DEV), counts,
                                  output_size=s["total"])
    index = torch.arange(s["total"], device=DEV) - s["q_start"].long()[row]
    # angles of far positions need 64 bits
    angle = s["rope_positions"].double()[:, None] * s["freqs"][None, :]
    cos = torch.cos(angle).float()[:, None, :]
    sin = torch.sin(angle).float()[:, None, :]

    def turn(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
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

    s["q_out"].copy_(turn(s["q"], s["q_weight"]))
    pos = s["seq_lens"].long()[row] - counts[row] + index
    block = s["tables"][row, pos // bs].long()
    _store(s["k_pool"], block, pos % bs, turn(s["k"], s["k_weight"]), s["k_scale"])
    _store(s["v_pool"], block, pos % bs, s["v"].float(), s["v_scale"])
    return s["q_out"], _values(s["k_pool"]), _values(s["v_pool"])


def _gathered(s, pool, scale):
    """A pool's tokens of every row, padded to the longest: 32 bits [rows][heads][len][dim]."""
    x = _values(pool)[s["tables"].clamp(min=0).long()].float()
    x = x.flatten(1, 2)[:, :s["max_len"]].transpose(1, 2)
    return x if scale is None else x * scale[:, None, None]


def _plain_decode(s):
    c = s["case"]
    rows, hq, hk, d, top = c["rows"], c["q_heads"], c["kv_heads"], c["dim"], s["max_len"]
    lens = s["seq_lens"][:, None, None, None]
    q = s["q"].float().reshape(rows, hk, hq // hk, d)
    score = torch.matmul(q, _gathered(s, s["k_pool"], s["k_scale"]).transpose(2, 3)).mul_(s["scale"])
    t = torch.arange(top, device=DEV)
    score.masked_fill_(t >= lens, float("-inf"))
    high = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(high == float("-inf"), 0, high)).exp_()
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0)
    v = _gathered(s, s["v_pool"], s["v_scale"])
    # slots past a row's length may hold anything
    v = torch.where(t[:, None] < lens, v, 0)
    s["out"].copy_(torch.matmul(p, v).reshape(rows, hq, d))
    given = p.sum(2)
    w, n = s["weights"][..., :top], s["seq_lens"][:, None, None]
    # the step's own token starts from zero
    w.copy_(torch.where(t < n - 1, w + given, torch.where(t == n - 1, given, w)))
    return s["out"], s["weights"]


def _plain_prefill(s):
    c = s["case"]
    rows, hq, hk, d, top = c["rows"], c["q_heads"], c["kv_heads"], c["dim"], s["max_len"]
    counts = (s["q_start"][1:] - s["q_start"][:-1]).long()
    most = max(s["new"])
    width = min(most, c["window"] or most)
    # the last `width` queries of each row, padded at the front
    back = torch.arange(width, 0, -1, device=DEV)
    there = back <= counts[:, None]
    at = torch.where(there, s["q_start"][1:, None] - back, 0)
    pos = (s["seq_lens"].long()[:, None] - back).clamp(min=0)
    q = s["q"][at].float().reshape(rows, width, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(rows, hk, hq // hk * width, d)
    score = torch.matmul(q, _gathered(s, s["k_pool"], s["k_scale"]).transpose(2, 3)).mul_(s["scale"])
    score = score.reshape(rows, hk, hq // hk, width, top)
    t = torch.arange(top, device=DEV)
    score.masked_fill_((t > pos[..., None])[:, None, None], float("-inf"))
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    # padding gives nothing
    part = torch.where(there[:, None, None, :, None], 1 / total, 0)
    given = score.mul_(part).sum((2, 3))
    w, n = s["weights"][..., :top], s["seq_lens"][:, None, None]
    first = n - counts[:, None, None]
    # the chunk's own tokens start from zero; rows without a chunk stay as they are
    new = torch.where(t < first, w + given, torch.where(t < n, given, w))
    w.copy_(torch.where(counts[:, None, None] > 0, new, w))
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    bs, top = c["block"], s["max_len"]
    lens = s["seq_lens"].long()[None, :, None, None]
    keep = lens.clamp(max=c["budget"])
    t = torch.arange(top, device=DEV)
    end = s["next_pos"].long()[None, :, None, None]
    pos = torch.where(t < s["tracked"][None, :, None, None], s["token_pos"][..., :top], end - lens + t)
    safe = (pos < c["sinks"]) | (pos >= end - c["recent"])
    w = s["weights"][..., :top]
    key = torch.where(t < lens, torch.where(safe, float("inf"), w), float("-inf"))
    order = key.sort(dim=-1, descending=True, stable=True).indices
    stays = torch.zeros_like(safe).scatter_(-1, order, t.expand_as(order) < keep)
    hole = (~stays & (t < keep)).nonzero(as_tuple=True)
    fill = (stays & (t >= keep)).nonzero(as_tuple=True)
    layer, row, head, dst = hole
    src = fill[3]
    db, sb = s["tables"][row, dst // bs].long(), s["tables"][row, src // bs].long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[layer, db, dst % bs, head] = pool[layer, sb, src % bs, head]
    for out, x in ((s["weights_out"], w), (s["token_pos_out"], pos)):
        part = out[..., :top]
        part.copy_(torch.where(t < keep, x, part))
        part[hole] = x[fill].to(out.dtype)
    s["new_lens"].copy_(s["seq_lens"].clamp(max=c["budget"]))
    return (_values(s["k_pool"]), _values(s["v_pool"]), s["weights_out"], s["token_pos_out"],
            s["new_lens"])


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    before, new = _sizes(case)
    lens = [b + n for b, n in zip(before, new)]
    hq, hk, bs, d = case["q_heads"], case["kv_heads"], case["block"], case["dim"]
    elt = 1 if case["fp8"] else 2
    total, rows = sum(new), case["rows"]
    index = 4 * (2 * rows + 1)
    entries = sum((n + bs - 1) // bs for n in lens)
    if case["op"] == "norm":
        entries = sum((n + bs - 1) // bs - b // bs for b, n in zip(before, lens))
        read = total * (hq + 2 * hk) * d * 2 + total * 4 + 8 * (case["rot"] // 2) + 4 * d
        write = total * hq * d * 2 + 2 * total * hk * d * elt
        return {"bytes": read + write + index + 4 * entries,
                "flops": total * (hq + hk) * (4 * d + 3 * case["rot"])}
    if case["op"] == "decode":
        tokens = sum(lens)
        return {"bytes": 2 * tokens * hk * d * elt + 2 * rows * hq * d * 2 + 8 * tokens * hk
                + 4 * rows + 4 * entries, "flops": 4 * d * hq * tokens}
    if case["op"] == "prefill":
        used = [min(n, case["window"] or n) for n in new]
        tokens = sum(n for n, u in zip(lens, used) if u)
        fresh = sum(new)
        seen = sum(u * n - u * (u - 1) // 2 for n, u in zip(lens, used))
        return {"bytes": tokens * hk * d * elt + sum(used) * hq * d * 2
                + 4 * hk * (2 * tokens - fresh) + index + 4 * entries, "flops": 2 * d * hq * seen}
    lists, read, write, moved = case["layers"] * hk, 0, 0, 0
    for n in lens:
        keep, track = min(n, case["budget"]), min(n, case["budget"]) if case["tracked"] else 0
        read += 4 * n + 4 * track
        write += 8 * keep
        # tokens at and past the budget: the recent stay, of the others as many as of all
        late = n - keep
        fresh = min(case["recent"], late)
        safe = case["recent"] + case["sinks"] if not case["tracked"] else fresh
        if late:
            moved += fresh + int((late - fresh) * max(0, keep - safe) / max(1, n - safe))
    return {"bytes": lists * (read + write + moved * 4 * d * elt) + 16 * rows + 4 * entries, "flops": 0}


# ---------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    if case["op"] == "evict":
        return None  # moved, not computed
    s = _inputs(case, seed)
    before, new = _sizes(case)
    bs, hq, hk, d = case["block"], case["q_heads"], case["kv_heads"], case["dim"]
    group = hq // hk
    tables = s["tables"].tolist()

    def slots(r, a, b):
        return torch.tensor([tables[r][t // bs] * bs + t % bs for t in range(a, b)], device=DEV,
                            dtype=torch.long)

    def widen(x, sc=None):
        x = _values(x).to(torch.float64)
        return x if sc is None else x * sc.to(torch.float64)[:, None]

    if case["op"] == "norm":
        rot, half = case["rot"], case["rot"] // 2
        at = torch.tensor([case["far"] + before[r] + i for r in range(case["rows"])
                           for i in range(new[r])], dtype=torch.float64, device=DEV)
        ang = torch.outer(at, _frequencies(case).to(DEV))
        circle = torch.polar(torch.ones_like(ang), ang)

        def rotate(x, weight):
            x = x.to(torch.float64)
            x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * weight.to(torch.float64)
            head, rest = x[..., :rot], x[..., rot:]
            if case["layout"] == "half":
                z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous())
                z = z * circle[:, None, :]
                return torch.cat([z.real, z.imag, rest], dim=-1)
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous())
            return torch.cat([torch.view_as_real(z * circle[:, None, :]).flatten(-2), rest], dim=-1)

        where = torch.cat([slots(r, before[r], before[r] + n) for r, n in enumerate(new)])
        outs = [rotate(s["q"], s["q_weight"])]
        for name, x in (("k", rotate(s["k"], s["k_weight"])), ("v", s["v"].to(torch.float64))):
            pool = widen(s[name + "_pool"])
            sc = s[name + "_scale"]
            if sc is not None:
                x = (x / sc.to(torch.float64)[:, None]).clamp(-448, 448)
            pool.view(-1, hk, d)[where] = x
            outs.append(pool)
        return tuple(outs)

    weights = s["weights"].to(torch.float64)
    out = torch.zeros((case["rows"], hq, d), dtype=torch.float64, device=DEV)
    for r, n in enumerate(s["lens"]):
        queries = 1 if case["op"] == "decode" else new[r]
        if n == 0 or queries == 0:
            continue
        used = min(queries, case.get("window") or queries)
        end = r + 1 if case["op"] == "decode" else s["starts"][r + 1]
        keys = widen(s["k_pool"].view(-1, hk, d)[slots(r, 0, n)], s["k_scale"])
        bias = torch.zeros((used, n), dtype=torch.float64, device=DEV)
        for i in range(used):
            bias[i, n - used + i + 1:] = -math.inf
        given = torch.zeros((hk, n), dtype=torch.float64, device=DEV)
        for h in range(hq):
            score = widen(s["q"][end - used:end, h]) @ keys[:, h // group].T
            p = torch.softmax(score * s["scale"] + bias, dim=-1)
            given[h // group] += p.sum(0)
            if case["op"] == "decode":
                vals = widen(s["v_pool"].view(-1, hk, d)[slots(r, 0, n)], s["v_scale"])
                out[r, h] = p[0] @ vals[:, h // group]
        weights[r, :, n - queries:n] = 0
        weights[r, :, :n] += given
    return (out, weights) if case["op"] == "decode" else weights
