"""Cases, plain forms and exact results of the 4-bit cache operators and of the
row commit after a verified draft tree.

  kv_append_fp4         quantise new K/V rows into a block-scaled 4-bit paged cache
  kv_load_fp4           read rows of that cache back at 16 or 32 bits
  paged_attention_fp4   decode, causal verification and tree verification over it
  commit_rows           move the rows of the accepted path together, in every layer

The 4-bit cache.  A value is code * block scale * tensor scale: the code is E2M1
(0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign), the block scale is E4M3, one for 16
consecutive head dims of a row, and the tensor scale is one float per cache.  The
tile of one (block, KV head) holds 16 rows in 9 * D bytes, its codes first (low
nibble: even dim) and its scales after them:
  keys    codes [D / P][16 rows][P / 2] with P = min(D, 128), scales [16 rows][D / 16]
  values  codes [D / 8][16 rows][4],                          scales [D / 16][16 rows]
"""
import math

import numpy as np
import torch

own = False

ROWS = 16  # rows of a cache block
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
K_SCALE, V_SCALE = 0.0091, 0.0047  # tensor scales: about the largest magnitude / (6 * 448)


def listed():
    return [
        # The append of one decode step of a 40-head layer: latency counts.
        {"name": "append_step", "op": "append", "tokens": 32, "kv_heads": 40, "dim": 128, "type": "bf16"},
        # The prompts of several requests written at once.
        {"name": "append_prompt", "op": "append", "tokens": 8192, "kv_heads": 8, "dim": 128, "type": "bf16"},
        # A short odd piece of a cache read back at full precision, to look at or to hand on.
        {"name": "load_odd", "op": "load", "tokens": 777, "kv_heads": 3, "dim": 64, "type": "f32"},
        # A long prompt's rows read back to 16 bits, for a chunk's prefill attention.
        {"name": "load_prompt", "op": "load", "tokens": 32768, "kv_heads": 8, "dim": 128, "type": "bf16"},
        # A handful of short sequences, float32 queries: the smallest call.
        {"name": "decode_tiny", "op": "attend", "batch": 4, "heads": 6, "kv_heads": 6, "dim": 64, "queries": 1,
         "low": 17, "high": 256, "tree": False, "type": "f32"},
        # One decode step of a 40-head layer, every query head with its own keys and values.
        {"name": "decode_mha", "op": "attend", "batch": 32, "heads": 40, "kv_heads": 40, "dim": 128, "queries": 1,
         "low": 2048, "high": 2048, "tree": False, "type": "bf16"},
        # One decode step with four query heads to a KV head, many sequences of ragged lengths.
        {"name": "decode_gqa", "op": "attend", "batch": 128, "heads": 32, "kv_heads": 8, "dim": 128, "queries": 1,
         "low": 128, "high": 4096, "tree": False, "type": "bf16"},
        # Two long contexts: the work has to be split along the rows.
        {"name": "decode_long", "op": "attend", "batch": 2, "heads": 32, "kv_heads": 8, "dim": 128, "queries": 1,
         "low": 32768, "high": 65536, "tree": False, "type": "bf16"},
        # Speculative verification: the last token and four drafts of each sequence.
        {"name": "verify_drafts", "op": "attend", "batch": 16, "heads": 32, "kv_heads": 8, "dim": 128, "queries": 5,
         "low": 512, "high": 8192, "tree": False, "type": "bf16"},
        # Verification of a tree of ten candidates.
        {"name": "verify_tree", "op": "attend", "batch": 16, "heads": 32, "kv_heads": 8, "dim": 128, "queries": 10,
         "low": 512, "high": 8192, "tree": True, "type": "f16"},
        # The accepted rows of one layer's cache: latency counts.
        {"name": "commit_layer", "op": "commit", "layers": 1, "batch": 4, "kv_heads": 6, "dim": 64, "queries": 5,
         "low": 17, "high": 256, "type": "f32"},
        # The accepted rows in all 32 layers of a model, after a tree of ten candidates.
        {"name": "commit_model", "op": "commit", "layers": 32, "batch": 16, "kv_heads": 8, "dim": 128, "queries": 10,
         "low": 32, "high": 300, "type": "bf16"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "load", "attend", "attend", "attend", "commit"])
    dim, kind = rng.choice([64, 128, 128, 256]), rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("append", "load"):
        kv_heads = _spread(rng, 1, 40)
        most = (8192 * 8 * 128 if op == "append" else 32768 * 8 * 128) // (2 if kind == "f32" else 1)
        tokens = _spread(rng, 1, most // (kv_heads * dim))
        return {"op": op, "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "type": kind}
    batch, kv_heads = _spread(rng, 1, 128), _spread(rng, 1, 16)
    queries = rng.choice([1, 1, 1, 2, 3, 5, 8, 10])
    if op == "commit":
        most = 32 * 16 * 8 * 128 // (2 if kind == "f32" else 1)
        batch = min(batch, max(1, most // (kv_heads * dim)))
        layers = _spread(rng, 1, max(1, min(32, most // (batch * kv_heads * dim))))
        low = _spread(rng, 16, 64)
        return {"op": op, "layers": layers, "batch": batch, "kv_heads": kv_heads, "dim": dim, "queries": max(3, queries),
                "low": low, "high": low + _spread(rng, 1, 200), "type": kind}
    group = rng.choice([1, 2, 3, 4, 4, 7, 8])
    # cached bytes and products stay under the largest listed cases'
    most = min(32 * 2048 * 40 * 128 // (batch * kv_heads * dim),
               16 * 4352 * 32 * 10 * 128 // (batch * kv_heads * group * queries * dim), 65536)
    high = _spread(rng, 16, max(16, most))
    low = max(1, int(high * rng.choice([0.03, 0.3, 1.0])))
    return {"op": op, "batch": batch, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "queries": queries,
            "low": low, "high": high, "tree": queries > 1 and rng.random() < 0.4, "type": kind}


# ---- sizes that follow from a case alone -----------------------------------------


def _lengths(case):
    """Context lengths over [low, high], both met, in no order."""
    n, low, high = case["batch"], case["low"], case["high"]
    at = [(i * 0.6180339887498949 + 0.31) % 1.0 for i in range(n)]
    order = sorted(range(n), key=at.__getitem__)
    out = [0] * n
    for rank, i in enumerate(order):
        out[i] = high if n == 1 else low + (high - low) * rank // (n - 1)
    return out


def _parents(queries):
    """A tree in which node j hangs under node (j - 1) // 3: node 0 is the last accepted token."""
    return [-1] + [(j - 1) // 3 for j in range(1, queries)]


def _ancestors(queries):
    """Bit k of mask j: node k is node j or one of its ancestors."""
    masks = []
    for j, parent in enumerate(_parents(queries)):
        masks.append((masks[parent] if parent >= 0 else 0) | (1 << j))
    return masks


def _paths(case):
    """The accepted path of each sequence: from node 0 down to a node, another one for each."""
    masks = _ancestors(case["queries"])
    out = []
    for b in range(case["batch"]):
        leaf = (b * 7 + case["queries"] - 1) % case["queries"]
        out.append([k for k in range(case["queries"]) if masks[leaf] >> k & 1])
    return out


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}[case["type"]]
    if case["op"] in ("append", "load"):
        rows = case["tokens"] * case["kv_heads"] * 2
        code, wide = rows * case["dim"] * 9 / 16, rows * case["dim"] * size
        # append: rows in, codes and scales out, and both ways again to return the rows as they are held
        return {"bytes": (2 if case["op"] == "append" else 1) * (code + wide) + 8 * case["tokens"], "flops": 0}
    if case["op"] == "commit":
        rows = sum(sum(1 for i, k in enumerate(p) if i != k) for p in _paths(case))
        named = 4 * sum(len(p) + 3 for p in _paths(case))  # path entries, lengths and table entries
        return {"bytes": 2 * 2 * case["layers"] * rows * case["kv_heads"] * case["dim"] * size + named, "flops": 0}
    seen = sum(_lengths(case))
    held = 2 * seen * case["kv_heads"] * case["dim"] * 9 / 16
    ends = 2 * case["batch"] * case["queries"] * case["heads"] * case["dim"] * size
    return {"bytes": held + ends + 4 * seen / ROWS, "flops": 4 * seen * case["queries"] * case["heads"] * case["dim"]}


# ---- the 4-bit cache in plain form -------------------------------------------------


def _views(cache, dim, keys):
    """Codes and scales of a cache [blocks, heads, 16, 9 * dim / 16] as [blocks, heads, part, row, bytes]
    and [blocks, heads, row, dim / 16] (views)."""
    flat = cache.view(cache.shape[0], cache.shape[1], 9 * dim)
    codes, scales = flat[..., :8 * dim], flat[..., 8 * dim:]
    if keys:
        panel = min(dim, 128)
        return codes.unflatten(-1, (dim // panel, ROWS, panel // 2)), scales.unflatten(-1, (ROWS, dim // 16))
    return codes.unflatten(-1, (dim // 8, ROWS, 4)), scales.unflatten(-1, (dim // 16, ROWS)).transpose(-1, -2)


def _quantise(x, tensor_scale):
    """Rows [..., dim] -> (code bytes [..., dim / 2], scale bytes [..., dim / 16])."""
    blocks = x.float().unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1)
    scale = (amax / tensor_scale / torch.full_like(tensor_scale, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    factor = scale.float() * tensor_scale
    y = blocks / torch.where(factor > 0, factor, torch.ones_like(factor)).unsqueeze(-1)
    y = torch.where((factor > 0).unsqueeze(-1), y, torch.zeros_like(y))
    a = y.abs()
    code = torch.signbit(y).to(torch.uint8) << 3
    # round to nearest, ties to the even code
    code += ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _dequantise(codes, scales):
    """Code bytes [..., dim / 2] and scale bytes [..., dim / 16] -> code * block scale, [..., dim]."""
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([half, -half])
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([table[byte & 15], table[byte >> 4]], -1)
    values = pairs[codes.int()].flatten(-2)
    return (values.unflatten(-1, (-1, 16)) * scales.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _write(cache, dim, keys, block, row, codes, scales):
    to_codes, to_scales = _views(cache, dim, keys)
    to_codes[block, :, :, row] = codes.unflatten(-1, to_codes.shape[2:3] + to_codes.shape[4:])
    to_scales[block, :, row] = scales


def _read(cache, dim, keys, block, row):
    codes, scales = _views(cache, dim, keys)
    return codes[block, :, :, row].flatten(-2), scales[block, :, row]


# ---- inputs --------------------------------------------------------------------------


def _rows(gen, shape, kind, sharp):
    """Rows as a layer makes them: normal, a few channels several times larger in keys than in the rest."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if sharp:
        gain = torch.ones(shape[-1], device="cuda")
        gain[torch.randint(0, shape[-1], (max(1, shape[-1] // 32),), generator=gen, device="cuda")] = 4.0
        x *= gain
    return x.to(TYPES[kind])


def _held(gen, blocks, heads, dim, keys, scale, unused):
    """A cache of `blocks` blocks whose rows hold quantised values, and bytes that stand for nothing in the unused rows."""
    cache = torch.empty(blocks, heads, ROWS, 9 * dim // 16, dtype=torch.uint8, device="cuda")
    codes, scales = _views(cache, dim, keys)
    step = max(1, (1 << 26) // (heads * ROWS * dim))
    for lo in range(0, blocks, step):
        x = _rows(gen, (min(step, blocks - lo), heads, ROWS, dim), "bf16", keys)
        c, s = _quantise(x, scale)
        c = c.unflatten(-1, codes.shape[2:3] + codes.shape[4:]).transpose(2, 3)
        codes[lo:lo + step], scales[lo:lo + step] = c, s
    codes.masked_fill_(unused[:, None, None, :, None], 255)
    scales.masked_fill_(unused[:, None, :, None], 255)
    return cache


def _table(gen, lengths):
    """Block table over a shuffled pool, the pool's size, and its unused rows."""
    need = [-(-n // ROWS) for n in lengths]
    pool = sum(need) + max(1, sum(need) // 10)
    order = torch.randperm(pool, generator=gen, device="cuda").cpu().numpy()
    table = np.full((len(need), max(max(need), 1)), -1, np.int32)
    unused = np.ones((pool, ROWS), bool)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        unused[order[at:at + n]] = False
        if lengths[b] % ROWS:
            unused[order[at + n - 1], lengths[b] % ROWS:] = True
        at += n
    return torch.from_numpy(table).cuda(), pool, torch.from_numpy(unused).cuda()


def _slots(gen, tokens):
    """Slots of a padded batch of rows in shuffled blocks: every 41st is padding."""
    pool = -(-tokens // ROWS) + 2
    order = torch.randperm(pool, generator=gen, device="cuda")
    at = torch.arange(tokens, device="cuda")
    slots = order[at // ROWS] * ROWS + at % ROWS
    return torch.where(at % 41 == 40, torch.full_like(slots, -1), slots), pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dim, kind = case["dim"], case["type"]
    s = {"case": case, "k_scale": torch.tensor(K_SCALE, device="cuda"), "v_scale": torch.tensor(V_SCALE, device="cuda")}
    if case["op"] in ("append", "load"):
        s["slots"], pool = _slots(gen, case["tokens"])
        spare = torch.full((pool, ROWS), case["op"] == "append", device="cuda")
        s["k_cache"] = _held(gen, pool, case["kv_heads"], dim, True, s["k_scale"], spare)
        s["v_cache"] = _held(gen, pool, case["kv_heads"], dim, False, s["v_scale"], spare)
        if case["op"] == "append":
            s["k_new"] = _rows(gen, (case["tokens"], case["kv_heads"], dim), kind, True)
            s["v_new"] = _rows(gen, (case["tokens"], case["kv_heads"], dim), kind, False)
        return s
    lengths, queries = _lengths(case), case["queries"]
    s["table"], pool, unused = _table(gen, lengths)
    s["lens"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    s["longest"] = max(lengths)
    if case["op"] == "commit":
        shape = (case["layers"], pool, case["kv_heads"], ROWS, dim)
        s["k_all"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(TYPES[kind])
        s["v_all"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(TYPES[kind])
        s["k_caches"], s["v_caches"] = list(s["k_all"]), list(s["v_all"])
        paths = _paths(case)
        most = max(len(p) for p in paths)
        s["path"] = torch.tensor([p + [-1] * (most - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        s["path_lens"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        return s
    s["k_cache"] = _held(gen, pool, case["kv_heads"], dim, True, s["k_scale"], unused)
    s["v_cache"] = _held(gen, pool, case["kv_heads"], dim, False, s["v_scale"], unused)
    q = _rows(gen, (case["batch"], queries, case["heads"], dim), kind, False)
    s["q"] = q[:, 0].contiguous() if queries == 1 else q
    s["tree"] = torch.tensor(_ancestors(queries), dtype=torch.int64, device="cuda") if case["tree"] else None
    return s


# ---- one pass ------------------------------------------------------------------------


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "append":
        return _append_plain(state, case["dim"])
    if case["op"] == "load":
        return _load_plain(state, case["dim"], TYPES[case["type"]])
    if case["op"] == "commit":
        return _commit_plain(state, case)
    return _attend_plain(state, case)


def _run_own(s, case):
    import paged_kv_cache_18_gb300 as pkv
    if case["op"] == "commit":
        lens = pkv.commit_rows(s["k_caches"], s["v_caches"], s["table"], s["lens"], s["path"], s["path_lens"],
                               num_queries=case["queries"])
        return {"k": s["k_all"], "v": s["v_all"], "lens": lens}
    if case["op"] == "attend":
        return pkv.paged_attention_fp4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], K_SCALE, V_SCALE,
                                       max_context_len=s["longest"], tree_mask=s["tree"])
    if case["op"] == "append":
        pkv.kv_append_fp4(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["slots"], K_SCALE, V_SCALE)
    k, v = pkv.kv_load_fp4(s["k_cache"], s["v_cache"], s["slots"], K_SCALE, V_SCALE, dtype=TYPES[case["type"]])
    return {"k": k, "v": v}


def _load_plain(s, dim, kind):
    kept = (s["slots"] >= 0)[:, None, None]
    slots = s["slots"].clamp(min=0)
    out = {}
    for name, keys in (("k", True), ("v", False)):
        x = _dequantise(*_read(s[name + "_cache"], dim, keys, slots // ROWS, slots % ROWS)) * s[name + "_scale"]
        out[name] = torch.where(kept, x, torch.zeros_like(x)).to(kind)
    return out


def _append_plain(s, dim):
    at = s["slots"] >= 0  # the others are padding
    slots = s["slots"][at]
    for name, keys in (("k", True), ("v", False)):
        codes, scales = _quantise(s[name + "_new"][at], s[name + "_scale"])
        _write(s[name + "_cache"], dim, keys, slots // ROWS, slots % ROWS, codes, scales)
    return _load_plain(s, dim, s["k_new"].dtype)


def _commit_plain(s, case):
    first = (s["lens"] - case["queries"]).long()[:, None]
    i = torch.arange(s["path"].shape[1], device="cuda")[None, :]
    taken = i < s["path_lens"][:, None]
    to = first + i
    frm = torch.where(taken, first + s["path"].long(), to)
    at = lambda pos: (torch.gather(s["table"].long(), 1, pos // ROWS).flatten(), (pos % ROWS).flatten())  # noqa: E731
    (block_to, row_to), (block, row) = at(to), at(frm)
    for x in (s["k_all"], s["v_all"]):
        x[:, block_to, :, row_to] = x[:, block, :, row]
    return {"k": s["k_all"], "v": s["v_all"], "lens": (first[:, 0] + s["path_lens"]).int()}


def _attend_plain(s, case):
    batch, dim, heads, queries = case["batch"], case["dim"], case["kv_heads"], case["queries"]
    group = case["heads"] // heads
    q = s["q"].float().reshape(batch, queries, heads, group, dim)
    q = q.permute(0, 2, 1, 3, 4).reshape(batch, heads, queries * group, dim)
    table = s["table"].clamp(min=0).long()
    blocks = table.shape[1]

    def rows(name, keys):  # [batch, heads, blocks * 16, dim]
        codes, scales = _views(s[name + "_cache"], dim, keys)
        x = _dequantise(codes[table].transpose(3, 4).flatten(-2), scales[table])
        return x.transpose(1, 2).reshape(batch, heads, blocks * ROWS, dim)

    key = torch.arange(blocks * ROWS, device="cuda")
    lens = s["lens"].long()
    held = key[None, :] < lens[:, None]
    j = torch.arange(queries, device="cuda")
    if s["tree"] is None:
        seen = key[None, None, :] <= (lens[:, None] - queries + j[None, :])[:, :, None]
    else:
        node = key[None, :] - (lens[:, None] - queries)
        bits = (s["tree"][None, :, None] >> node.clamp(0, 63)[:, None, :]) & 1
        seen = (node < 0)[:, None, :] | (bits == 1)
    seen = (seen & held[:, None, :]).repeat_interleave(group, 1)[:, None]
    scores = (q @ rows("k", True).transpose(-1, -2)) * (s["k_scale"] / math.sqrt(dim))
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    v = rows("v", False)
    v = torch.where(held[:, None, :, None], v, torch.zeros_like(v))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) * s["v_scale"] / torch.where(total > 0, total, torch.ones_like(total))
    out = out.reshape(batch, heads, queries, group, dim).permute(0, 2, 1, 3, 4)
    return out.reshape(s["q"].shape).to(s["q"].dtype)


# ---- exact results, in 64 bits -------------------------------------------------------


def _value64(code):
    """E2M1 codes as numbers: a sign, two exponent bits (bias 1, 0 subnormal) and one mantissa bit."""
    code = code.to(torch.int64)
    e, m = (code >> 1) & 3, (code & 1).double()
    size = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1).clamp(min=0))
    return torch.where(code >= 8, -size, size)


def _scale64(byte):
    """E4M3 bytes as numbers (non-negative ones): bias 7, 0 subnormal, 127 no number."""
    byte = byte.to(torch.int64)
    e, m = (byte >> 3) & 15, (byte & 7).double() / 8
    size = torch.where(e == 0, m * 2.0 ** -6, (1 + m) * 2.0 ** (e - 7).double())
    return torch.where(byte & 127 == 127, torch.full_like(size, math.nan), size)


def _tile64(cache, dim, keys, block):
    """The rows of the named blocks as code * scale: [len(block), heads, 16, dim]."""
    tile = cache.reshape(cache.shape[0], cache.shape[1], 9 * dim)[block]
    n, heads = tile.shape[:2]
    d = torch.arange(dim, device=tile.device)[None, :]
    r = torch.arange(ROWS, device=tile.device)[:, None]
    if keys:
        panel = min(dim, 128)
        place = (d // panel) * (ROWS * panel // 2) + r * (panel // 2) + (d % panel) // 2
        where = 8 * dim + r * (dim // 16) + d // 16
    else:
        place = (d // 8) * (ROWS * 4) + r * 4 + (d % 8) // 2
        where = 8 * dim + (d // 16) * ROWS + r
    byte = tile[:, :, place.flatten()].reshape(n, heads, ROWS, dim).int()
    nibble = torch.where(d % 2 == 1, byte >> 4, byte & 15)
    return _value64(nibble) * _scale64(tile[:, :, where.flatten()].reshape(n, heads, ROWS, dim))


def _near64(x, grid):
    """The nearest value of an increasing grid, ties to the even place."""
    mid = (grid[1:] + grid[:-1]) / 2
    low = torch.searchsorted(mid, x, right=False)   # places under x's upper neighbour: a tie stays below
    tie = (low < len(mid)) & (mid[low.clamp(max=len(mid) - 1)] == x)
    return grid[low + (tie & (low % 2 == 1)).long()]


def _held64(x, tensor_scale):
    """What the cache holds of the rows x, as numbers."""
    scales = _scale64(torch.arange(127, device="cuda"))
    codes = _value64(torch.arange(8, device="cuda"))
    b = x.double().unflatten(-1, (-1, 16))
    scale = _near64(b.abs().amax(-1) / (6 * tensor_scale), scales) * tensor_scale
    y = b.abs() / torch.where(scale > 0, scale, torch.full_like(scale, math.inf)).unsqueeze(-1)
    return (torch.sign(b) * _near64(y, codes) * scale.unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    dim = case["dim"]
    scales = {"k": float(s["k_scale"]), "v": float(s["v_scale"])}
    if case["op"] in ("append", "load"):
        out = {}
        kept = (s["slots"] >= 0).double()[:, None, None]
        slots = s["slots"].clamp(min=0)
        for name in ("k", "v"):
            if case["op"] == "append":
                x = _held64(s[name + "_new"], scales[name])
            else:
                block, at = torch.unique(slots // ROWS, return_inverse=True)
                tiles = _tile64(s[name + "_cache"], dim, name == "k", block)
                x = tiles.transpose(1, 2)[at, slots % ROWS] * scales[name]
            out[name] = x * kept
        return out
    if case["op"] == "commit":
        lens = s["lens"].tolist()
        k, v = s["k_all"].clone(), s["v_all"].clone()
        table = s["table"].tolist()
        for b, path in enumerate(_paths(case)):
            first = lens[b] - case["queries"]
            for i, node in enumerate(path):
                to, frm = first + i, first + node
                for new, old in ((k, s["k_all"]), (v, s["v_all"])):
                    new[:, table[b][to // ROWS], :, to % ROWS] = old[:, table[b][frm // ROWS], :, frm % ROWS]
        total = k.numel()
        wide = (lambda x: x.double()) if total < 1 << 30 else (lambda x: x)
        return {"k": wide(k), "v": wide(v), "lens": None}
    out = []
    group, queries = case["heads"] // case["kv_heads"], case["queries"]
    for b, n in enumerate(s["lens"].tolist()):
        block = s["table"][b, :-(-n // ROWS)].long()
        k = _tile64(s["k_cache"], dim, True, block).transpose(0, 1).flatten(1, 2)[:, :n] * scales["k"]
        v = _tile64(s["v_cache"], dim, False, block).transpose(0, 1).flatten(1, 2)[:, :n] * scales["v"]
        q = s["q"][b].double().reshape(queries, case["kv_heads"], group, dim)
        scores = torch.einsum("jhgd,hnd->hgjn", q, k) / math.sqrt(dim)
        for j in range(queries):
            if s["tree"] is None:
                scores[:, :, j, max(0, n - queries + j + 1):] = -math.inf
            else:
                hidden = [n - queries + t for t in range(queries) if not _ancestors(queries)[j] >> t & 1]
                scores[:, :, j, [t for t in hidden if t >= 0]] = -math.inf
        p = torch.nan_to_num(torch.softmax(scores, -1)) if n else scores
        out.append(torch.einsum("hgjn,hnd->jhgd", p, v).reshape(s["q"].shape[1:]))
    return torch.stack(out)
