"""Operators of a paged serving path, as cases that can be measured: writing
rotated keys and values into a paged cache (16-bit, or 8-bit with one scale
per block and head), and attention over such caches with a sliding window and
a few first tokens that stay visible (one query per sequence, several, and
one query over the 8-bit cache).

``own`` selects what ``run`` does: the operators' plain form in elementary
torch operations, or the calls a program makes of ``paged_kv_cache_481_b200``.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 sequences with 40 heads of 128 (13B shapes):
        # the smallest call, all latency
        dict(name="rope cache, decode step", op="rope_cache", dtype="f16", heads=40, kv_heads=40,
             head_dim=128, block_size=16, seqs=32, new_min=1, new_max=1, start_max=2048,
             rotary=128, interleaved=False, padding=0),
        # prompts and chunks of a packed batch with grouped heads and padded rows at its end
        dict(name="rope cache, packed prompts", op="rope_cache", dtype="bf16", heads=32, kv_heads=8,
             head_dim=128, block_size=16, seqs=9, new_min=37, new_max=2048, start_max=8192,
             rotary=64, interleaved=True, padding=21),
        # a serving batch's decode step into the 8-bit cache: most blocks are
        # part full, so older rows of a block meet a larger scale
        dict(name="rope cache q8, decode step", op="rope_cache_q8", dtype="f16", heads=40,
             kv_heads=40, head_dim=128, block_size=16, seqs=256, new_min=1, new_max=1,
             start_max=4096, rotary=128, interleaved=False, padding=0, codes="int8"),
        # chunks that start and end inside a block
        dict(name="rope cache q8, chunks", op="rope_cache_q8", dtype="bf16", heads=32, kv_heads=8,
             head_dim=128, block_size=32, seqs=12, new_min=100, new_max=900, start_max=8192,
             rotary=128, interleaved=False, padding=5, codes="e4m3"),
        # one long stream of one user: only the window's and the first blocks are still held
        dict(name="window decode, one stream", op="decode_window", dtype="bf16", heads=32,
             kv_heads=8, head_dim=128, block_size=16, seqs=1, len_min=131071, len_max=131071,
             window=4096, sinks=4),
        # the 13B decode batch with a 1024-token window
        dict(name="window decode, 13B batch", op="decode_window", dtype="f16", heads=40,
             kv_heads=40, head_dim=128, block_size=16, seqs=32, len_min=256, len_max=2048,
             window=1024, sinks=4),
        # a large serving batch with grouped heads; many contexts pass the window
        dict(name="window decode, serving batch", op="decode_window", dtype="bf16", heads=64,
             kv_heads=8, head_dim=128, block_size=16, seqs=256, len_min=1000, len_max=32768,
             window=4096, sinks=4),
        # a few draft tokens of each sequence to be verified
        dict(name="window prefill, drafts", op="prefill_window", dtype="bf16", heads=32, kv_heads=8,
             head_dim=128, block_size=16, seqs=16, new_min=1, new_max=7, len_min=300,
             len_max=4096, window=1024, sinks=4),
        # chunks of several prompts, each continuing its cached context
        dict(name="window prefill, chunks", op="prefill_window", dtype="f16", heads=40, kv_heads=40,
             head_dim=128, block_size=16, seqs=8, new_min=100, new_max=512, len_min=600,
             len_max=2048, window=1000, sinks=0),
        # one whole long prompt
        dict(name="window prefill, long prompt", op="prefill_window", dtype="bf16", heads=32,
             kv_heads=8, head_dim=128, block_size=16, seqs=1, new_min=8192, new_max=8192,
             len_min=8192, len_max=8192, window=4096, sinks=4),
        # a small batch over the 8-bit cache, whole contexts
        dict(name="q8 decode, small batch", op="decode_q8", dtype="f16", heads=40, kv_heads=40,
             head_dim=128, block_size=16, seqs=4, len_min=17, len_max=2047, window=2047, sinks=0,
             codes="int8"),
        # a large batch over the 8-bit cache, whole contexts, grouped heads
        dict(name="q8 decode, large batch", op="decode_q8", dtype="bf16", heads=64, kv_heads=8,
             head_dim=128, block_size=32, seqs=128, len_min=1024, len_max=16384, window=16384,
             sinks=0, codes="e4m3"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_cache", "rope_cache_q8", "decode_window", "prefill_window", "decode_q8"])
    heads, kv_heads = rng.choice([(40, 40), (72, 72), (32, 8), (64, 8), (16, 2), (12, 4), (8, 1),
                                  (10, 2), (7, 1), (4, 4), (32, 2)])
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), heads=heads, kv_heads=kv_heads,
             head_dim=rng.choice([64, 128, 128]), block_size=rng.choice([8, 16, 16, 32, 64, 128]))
    if op in ("rope_cache", "rope_cache_q8"):
        most = int(min(10000, 6e7 / ((heads + 2 * kv_heads) * c["head_dim"])))
        tokens = _logint(rng, 1, most)
        c["seqs"] = _logint(rng, 1, min(tokens, 256))
        c["new_max"] = max(1, tokens // c["seqs"])
        c["new_min"] = rng.randint(1, c["new_max"])
        c["start_max"] = rng.randint(0, 16000)
        c["rotary"] = rng.choice([c["head_dim"], c["head_dim"] // 2, 16])
        c["interleaved"] = rng.random() < 0.5
        c["padding"] = rng.choice([0, 0, 1, rng.randint(1, 64)])
    elif op == "prefill_window":
        c["new_max"] = _logint(rng, 1, 2048)
        c["new_min"] = rng.randint(1, c["new_max"])
        c["len_max"] = c["new_max"] + rng.randint(0, 4096)
        c["len_min"] = rng.randint(c["new_max"], c["len_max"])
        c["window"], c["sinks"] = _logint(rng, 1, 8192), rng.choice([0, 1, 4, 4, 64, 130])
        seen = min(c["len_max"], c["window"] + c["sinks"] + c["new_max"])
        c["seqs"] = _logint(rng, 1, max(1, min(64, int(1.2e9 / (heads * c["new_max"] * seen)))))
    else:
        c["len_max"] = _logint(rng, 1, 40000)
        c["len_min"] = rng.randint(0, c["len_max"])
        c["window"], c["sinks"] = _logint(rng, 1, 8192), rng.choice([0, 1, 4, 4, 64, 130])
        if op == "decode_q8" and rng.random() < 0.7:
            c["window"], c["sinks"] = max(1, c["len_max"]), 0
        seen = min(c["len_max"], c["window"] + c["sinks"])
        c["seqs"] = _logint(rng, 1, max(1, min(300, int(8e8 / (seen * kv_heads * c["head_dim"])))))
    if op in ("rope_cache_q8", "decode_q8"):
        c["codes"] = rng.choice(["int8", "e4m3"])
    return c


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], evenly and in no order; the first is hi."""
    return [hi - int((hi - lo + 1) * ((b * 0.6180339887498949) % 1.0)) for b in range(n)]


def _first_seen(length, new, window, sinks):
    """(sinks seen, first position of the window) of a sequence's `new` last queries."""
    start = max(0, length - new - window + 1)
    return min(sinks, start), start


def work(case):
    c, d = case, case["head_dim"]
    if c["op"] in ("rope_cache", "rope_cache_q8"):
        new = sum(_spread(c["seqs"], c["new_min"], c["new_max"]))
        moved = new * d * 2 * (2 * c["heads"] + 2 * c["kv_heads"])   # q in and out, k and v in
        moved += min(new, c["start_max"] + c["new_max"]) * c["rotary"] * 4 + new * 16
        if c["op"] == "rope_cache":
            moved += new * d * 2 * 2 * c["kv_heads"]
        else:
            blocks = sum(1 + (s % c["block_size"] + n - 1) // c["block_size"]
                         for s, n in zip(_spread(c["seqs"], 0, c["start_max"]),
                                         _spread(c["seqs"], c["new_min"], c["new_max"])))
            moved += new * d * 2 * c["kv_heads"] + blocks * c["kv_heads"] * 16
        return {"bytes": moved, "flops": new * (c["heads"] + c["kv_heads"]) * c["rotary"] * 3}
    size = 1 if c["op"] == "decode_q8" else 2
    lens = _spread(c["seqs"], c["len_min"], c["len_max"])
    news = (_spread(c["seqs"], c["new_min"], c["new_max"]) if c["op"] == "prefill_window"
            else [1] * c["seqs"])
    moved = pairs = 0
    for length, n in zip(lens, news):
        s, start = _first_seen(length, n, c["window"], c["sinks"])
        moved += (length - start + s) * c["kv_heads"] * 2 * d * size
        moved += n * c["heads"] * d * 2 * 2
        if size == 1:
            moved += -(-(length - start + s) // c["block_size"]) * c["kv_heads"] * 8
        p = np.arange(max(0, length - n), length)
        low = np.maximum(0, p - c["window"] + 1)
        pairs += int((p + 1 - low + np.minimum(low, c["sinks"])).sum())
    return {"bytes": moved, "flops": pairs * c["heads"] * 4 * d}


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    c, d, bs, kvh = case, case["head_dim"], case["block_size"], case["kv_heads"]
    dev, dtype = torch.device("cuda"), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def ints(values, kind=np.int32):
        return torch.from_numpy(np.ascontiguousarray(values, dtype=kind)).to(dev)

    writes = c["op"] in ("rope_cache", "rope_cache_q8")
    news = (_spread(c["seqs"], c["new_min"], c["new_max"]) if "new_min" in c else [1] * c["seqs"])
    if writes:
        starts = _spread(c["seqs"], 0, c["start_max"])
        lens = [s + n for s, n in zip(starts, news)]
    else:
        lens = _spread(c["seqs"], c["len_min"], c["len_max"])
    # the blocks that a sequence still holds: for a write the ones from its
    # first new token on, for attention those that hold a visible position
    held = []
    for length, n in zip(lens, news):
        if writes:
            held.append(list(range((length - n) // bs, -(-length // bs))))
        else:
            s, start = _first_seen(length, n, c["window"], c["sinks"])
            held.append(sorted(set(range(-(-s // bs))) | set(range(start // bs, -(-length // bs)))))
    used = sum(len(h) for h in held)
    num_blocks = used + used // 8 + 1
    ids = rng.permutation(num_blocks).astype(np.int32)
    tables = np.full((c["seqs"], max(1, -(-max(lens) // bs))), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        tables[b, h] = ids[at:at + len(h)]
        at += len(h)
    shape = (num_blocks, kvh, bs, d)
    st = dict(case=case, block_size=bs)
    if c["op"] in ("rope_cache_q8", "decode_q8"):
        code_type, top = CODES[c["codes"]]
        for name in ("k", "v"):
            x = torch.randn(shape, generator=gen, device=dev) * (top / 3.5)
            x = x.round_() if c["codes"] == "int8" else x
            st[name + "_codes"] = x.clamp_(-top, top).to(code_type)
        st["kv_scales"] = (3.5 / top) * (0.6 + 0.6 * torch.rand(
            (num_blocks, kvh + kvh % 2, 2), generator=gen, device=dev))
    else:
        st["k_cache"], st["v_cache"] = randn(*shape), randn(*shape)
    if writes:
        n, pad = sum(news), c["padding"]
        st["q"], st["key"] = randn(n + pad, c["heads"], d), randn(n + pad, kvh, d)
        st["value"], st["q_out"] = randn(n + pad, kvh, d), randn(n + pad, c["heads"], d)
        pos = np.concatenate([np.arange(length - m, length) for length, m in zip(lens, news)])
        row = np.repeat(np.arange(c["seqs"]), news)
        slots = tables[row, pos // bs].astype(np.int64) * bs + pos % bs
        st["positions"] = ints(np.concatenate([pos, np.zeros(pad)]), np.int64)
        st["slots"] = ints(np.concatenate([slots, np.full(pad, -1)]), np.int64)
        angle = (torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(0, c["rotary"], 2, device=dev,
                                             dtype=torch.float64) / c["rotary"]))
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        return st
    st["tables"], st["lens"] = ints(tables), ints(lens)
    st["max_len"], st["scale"] = max(lens), d ** -0.5
    st["q"] = randn(sum(news), c["heads"], d)
    if c["op"] == "prefill_window":
        st["starts"], st["max_new"] = ints(np.concatenate([[0], np.cumsum(news)])), max(news)
    elif own:
        from paged_kv_cache_481_b200 import binding
        # the split-context scratch that a serving loop allocates once
        st["workspace"] = binding.new_window_workspace(c["seqs"], c["heads"], kvh, d)
    return st


# ----------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if op == "rope_cache":
        return _rope_cache(state)
    if op == "rope_cache_q8":
        return _rope_cache_q8(state)
    if op == "prefill_window":
        return _prefill_window(state)
    if op == "decode_q8":
        return _decode_q8(state)
    return _decode_window(state)


def _rope_cache(st):
    if own:
        from paged_kv_cache_481_b200 import binding
        binding.pa_rope_and_cache(st["q_out"], st["q"], st["key"], st["value"], st["k_cache"],
                                  st["v_cache"], st["cos_sin"], st["positions"], st["slots"],
                                  interleaved=st["case"]["interleaved"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    q, k, v, slot, row = _rotated(st)
    bs = st["block_size"]
    st["q_out"][row] = q.to(st["q_out"].dtype)
    st["k_cache"][slot // bs, :, slot % bs] = k.to(st["k_cache"].dtype)
    st["v_cache"][slot // bs, :, slot % bs] = v.to(st["v_cache"].dtype)
    return st["q_out"], st["k_cache"], st["v_cache"]


def _values(codes, scales, dtype):
    """What the 8-bit codes stand for."""
    out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    return torch.mul(codes.to(dtype), scales[:, :, None, None], out=out)


def _rope_cache_q8(st):
    dtype, kvh = st["q"].dtype, st["key"].shape[1]
    if own:
        from paged_kv_cache_481_b200 import binding
        binding.pa_rope_and_cache_q8(st["q_out"], st["q"], st["key"], st["value"], st["k_codes"],
                                     st["v_codes"], st["kv_scales"], st["cos_sin"],
                                     st["positions"], st["slots"],
                                     interleaved=st["case"]["interleaved"])
    else:
        q, k, v, slot, row = _rotated(st)
        st["q_out"][row] = q.to(dtype)
        _quantized_write(st, 0, st["k_codes"], k, slot)
        _quantized_write(st, 1, st["v_codes"], v, slot)
    return (st["q_out"], _values(st["k_codes"], st["kv_scales"][:, :kvh, 0], dtype),
            _values(st["v_codes"], st["kv_scales"][:, :kvh, 1], dtype), st["kv_scales"])


def _rotated(st):
    """q, k (rotated) and v in 32 bits, with their slots and rows; the rows of
    padding tokens (slot < 0) stand for the first token that is none."""
    valid = st["slots"] >= 0
    row = torch.where(valid, torch.arange(valid.numel(), device=valid.device),
                      valid.to(torch.int8).argmax())
    rot = st["cos_sin"].shape[1]
    cos, sin = st["cos_sin"][st["positions"][row]][:, None].split(rot // 2, dim=-1)

    def turn(x):
        x = x[row].float()
        a = x[..., 0:rot:2] if st["case"]["interleaved"] else x[..., :rot // 2]
        b = x[..., 1:rot:2] if st["case"]["interleaved"] else x[..., rot // 2:rot]
        y = [a * cos - b * sin, b * cos + a * sin]
        y = torch.stack(y, -1).flatten(-2) if st["case"]["interleaved"] else torch.cat(y, -1)
        return torch.cat([y, x[..., rot:]], -1)

    return turn(st["q"]), turn(st["key"]), st["value"][row].float(), st["slots"][row], row


def _quantized_write(st, which, codes, x, slot):
    """Rows x [N, heads, D] into the 8-bit blocks.  A block's scale is the
    largest magnitude it has held over the codes' top; where it grows, the
    rows that the block holds already are rounded again."""
    nb, kvh, bs, _ = codes.shape
    code_type, top = CODES[st["case"]["codes"]]
    block, offset = slot // bs, slot % bs

    def rounded(y):
        return (y.round() if code_type == torch.int8 else y).clamp(-top, top).to(code_type)

    def over(a, b):
        return torch.where(b > 0, a / b, torch.zeros_like(a))

    new = torch.zeros((nb, kvh), device=x.device).scatter_reduce_(
        0, block[:, None].expand(-1, kvh), x.abs().amax(-1), "amax") / top
    first = torch.full((nb,), bs, device=x.device).scatter_reduce_(0, block, offset, "amin")
    old = st["kv_scales"][:, :kvh, which]
    scale = torch.where((first > 0)[:, None], torch.maximum(old, new), new)
    ratio = over(old, scale)
    older = torch.arange(bs, device=x.device)[None] < first[:, None]
    kept = torch.where((older & (first < bs)[:, None])[:, None, :, None],
                       rounded(codes.float() * ratio[:, :, None, None]).float(), codes.float())
    codes.copy_(kept.to(code_type))
    codes.view(torch.uint8)[block, :, offset] = rounded(
        over(x, scale[block][:, :, None].expand_as(x))).view(torch.uint8)
    st["kv_scales"][:, :kvh, which] = scale


def _decode_window(st):
    if own:
        from paged_kv_cache_481_b200 import binding
        out = torch.empty_like(st["q"])
        binding.pa_decode_window(out, st["q"], st["k_cache"], st["v_cache"], st["tables"],
                                 st["lens"], st["max_len"], st["case"]["window"],
                                 st["case"]["sinks"], st["scale"], st["workspace"])
        return out
    new = torch.ones_like(st["lens"])
    return _attend(st, st["q"][:, None], new, st["k_cache"], st["v_cache"])[:, 0].to(st["q"].dtype)


def _decode_q8(st):
    if own:
        from paged_kv_cache_481_b200 import binding
        out = torch.empty_like(st["q"])
        binding.pa_decode_q8(out, st["q"], st["k_codes"], st["v_codes"], st["kv_scales"],
                             st["tables"], st["lens"], st["max_len"], st["case"]["window"],
                             st["case"]["sinks"], st["scale"], st["workspace"])
        return out
    new, kvh = torch.ones_like(st["lens"]), st["case"]["kv_heads"]
    return _attend(st, st["q"][:, None], new, st["k_codes"], st["v_codes"],
                   st["kv_scales"][:, :kvh])[:, 0].to(st["q"].dtype)


def _prefill_window(st):
    if own:
        from paged_kv_cache_481_b200 import binding
        out = torch.empty_like(st["q"])
        binding.pa_prefill_window(out, st["q"], st["k_cache"], st["v_cache"], st["tables"],
                                  st["lens"], st["max_len"], st["starts"], st["max_new"],
                                  st["case"]["window"], st["case"]["sinks"], st["scale"])
        return out
    new = st["starts"].diff()
    rows = st["starts"][:-1, None] + torch.arange(st["max_new"], device=new.device)
    out = _attend(st, st["q"][rows.clamp(max=st["q"].shape[0] - 1)], new, st["k_cache"],
                  st["v_cache"])
    seq = torch.searchsorted(st["starts"][1:], torch.arange(
        st["q"].shape[0], device=new.device, dtype=torch.int32), right=True)
    at = torch.arange(st["q"].shape[0], device=new.device) - st["starts"][seq]
    return out[seq, at].to(st["q"].dtype)


def _attend(st, q, new, k_cache, v_cache, scales=None):
    """q [B, n, H, D] of each sequence's last `new` positions over its paged
    context, in 32 bits; only positions that some query may see are gathered."""
    c, bs, lens = st["case"], st["block_size"], st["lens"].long()[:, None]
    window, sinks, kvh = c["window"], c["sinks"], c["kv_heads"]
    b, n, heads, d = q.shape
    start = (lens - new[:, None] - window + 1).clamp(min=0)
    most = min(st["max_len"], sinks + window + n - 1)
    i = torch.arange(max(most, 1), device=q.device)[None]
    pos = torch.where(i < sinks, i, i - sinks + start.clamp(min=sinks))
    at = torch.minimum(pos, (lens - 1).clamp(min=0))
    block = st["tables"].gather(1, at // bs).long().clamp(min=0)
    k, v = (x[block, :, at % bs].float() for x in (k_cache, v_cache))      # [B, M, KVH, D]
    if scales is not None:
        s = scales[block]                                                  # [B, M, KVH, 2]
        k, v = k * s[..., 0, None], v * s[..., 1, None]
    mine = lens - new[:, None] + torch.arange(n, device=q.device)[None]    # [B, n]
    seen = ((pos[:, None] <= mine[..., None]) & (pos < lens)[:, None]
            & ((pos[:, None] > mine[..., None] - window) | (pos < sinks)[:, None]))
    seen = seen[:, None, None]                                             # [B, 1, 1, n, M]
    q = q.float().view(b, n, kvh, heads // kvh, d).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)[:, :, None]) * st["scale"]
    s = s.masked_fill_(~seen, -math.inf)
    w = torch.exp(s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)))
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w, v.permute(0, 2, 1, 3)[:, :, None])
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.permute(0, 3, 1, 2, 4).reshape(b, n, heads, d)


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope_cache":
        return _exact_rope_cache(st)
    if case["op"] == "rope_cache_q8":
        return _exact_rope_cache_q8(st)
    return _exact_attention(st)


def _exact_turn(st, x):
    """Each pair of components as a complex number, turned by its position's angle."""
    rot = st["cos_sin"].shape[1]
    table = st["cos_sin"].double()[st["positions"]]
    turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]
    x = x.double()
    y = x.clone()
    if st["case"]["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], -1, 2).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).reshape(*x.shape[:2], rot)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_rope_cache(st):
    live = torch.nonzero(st["slots"] >= 0)[:, 0]
    q, k, v = (t.double() for t in (st["q_out"], st["k_cache"], st["v_cache"]))
    q[live] = _exact_turn(st, st["q"])[live]
    block, offset = st["slots"][live] // st["block_size"], st["slots"][live] % st["block_size"]
    k[block, :, offset] = _exact_turn(st, st["key"])[live]
    v[block, :, offset] = st["value"].double()[live]
    return q, k, v


def _exact_rope_cache_q8(st):
    live = torch.nonzero(st["slots"] >= 0)[:, 0]
    bs, kvh = st["block_size"], st["case"]["kv_heads"]
    code_type, top = CODES[st["case"]["codes"]]
    q = st["q_out"].double()
    q[live] = _exact_turn(st, st["q"])[live]
    slots = st["slots"][live].cpu().numpy()
    scales, values = st["kv_scales"].double(), []
    for which, codes, rows in ((0, st["k_codes"], _exact_turn(st, st["key"])),
                               (1, st["v_codes"], st["value"].double())):
        rows, held = rows[live], codes.double()
        for block in sorted(set((slots // bs).tolist())):
            mine = np.nonzero(slots // bs == block)[0]
            first = int((slots[mine] % bs).min())
            x, offset = rows[mine], torch.from_numpy(slots[mine] % bs).to(rows.device)
            scale = x.abs().amax(dim=(0, 2)) / top
            older = held[block, :, :first] * scales[block, :kvh, which, None, None]
            if first:
                scale = torch.maximum(scale, scales[block, :kvh, which])
            scales[block, :kvh, which] = scale
            for at, y in ((slice(0, first), older), (offset, x.transpose(0, 1))):
                y = y / scale[:, None, None]
                held[block, :, at] = (y.round() if code_type == torch.int8
                                      else y.float().to(code_type).double())
        values.append(held * scales[:, :kvh, which, None, None])
    return q, values[0], values[1], scales


def _exact_attention(st):
    c, bs, d = st["case"], st["block_size"], st["case"]["head_dim"]
    kvh, group = c["kv_heads"], c["heads"] // c["kv_heads"]
    lens = st["lens"].tolist()
    starts = st["starts"].tolist() if "starts" in st else list(range(len(lens) + 1))
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    for b, length in enumerate(lens):
        n = starts[b + 1] - starts[b]
        if not length or not n:
            continue
        t = torch.arange(length, device=out.device)
        p = torch.arange(length - n, length, device=out.device)[:, None]
        seen = (t <= p) & ((p - t < c["window"]) | (t < c["sinks"]))
        t, seen = t[seen.any(0)], seen[:, seen.any(0)]
        block, row = st["tables"][b].long()[t // bs], t % bs
        for h in range(kvh):
            if c["op"] == "decode_q8":
                scale = st["kv_scales"][block, h].double()
                k = st["k_codes"][block, h, row].double() * scale[:, :1]
                v = st["v_codes"][block, h, row].double() * scale[:, 1:]
            else:
                k, v = st["k_cache"][block, h, row].double(), st["v_cache"][block, h, row].double()
            x = st["q"][starts[b]:starts[b + 1], h * group:(h + 1) * group].double()
            s = (x.reshape(n * group, d) @ k.T) * st["scale"]
            s = s.view(n, group, -1).masked_fill(~seen[:, None], -math.inf)
            w = torch.softmax(s, -1).view(n * group, -1)
            out[starts[b]:starts[b + 1], h * group:(h + 1) * group] = (w @ v).view(n, group, d)
    return out
