"""Cases, plain forms and measured work of the operators around the decode step.

Four operators: ``mla_page_map`` (page tables, slot and index maps of a step,
from request lengths), ``mla_kv_append`` (norm of the latent, rotation of the
key and of the queries, quantisation and scatter into the cache in one pass),
``mla_prefill_fwd`` (attention of prompts, expanded form) and
``mla_attn_merge`` (joins pieces of attention over disjoint keys).

With ``own`` false ``run`` computes them with elementary torch operations; with
``own`` true it calls the framework.
"""
import math

import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
QK = NOPE + ROPE
KV_DIM = LATENT + ROPE
EPS = 1e-6
MAX_POS = 32768


def listed():
    return [
        # One decode step of four short requests: the latency of building its tables.
        {"name": "map_decode_4", "op": "map", "batch": 4, "max_len": 1024, "max_new": 1, "page": 64},
        # A mixed step: ragged cached lengths, chunks of prompts, small pages, an odd batch.
        {"name": "map_mixed_33", "op": "map", "batch": 33, "max_len": 3001, "max_new": 700, "page": 16},
        # A full decode batch at long contexts: two million tokens of indices.
        {"name": "map_decode_256", "op": "map", "batch": 256, "max_len": 8192, "max_new": 1, "page": 64, "uniform": True},
        # A decode step's new tokens into an e4m3 cache, few rows and many.
        {"name": "append_decode_4", "op": "append", "tokens": 4, "heads": 16, "cache": "e4m3", "interleaved": True, "dense": False},
        {"name": "append_decode_256", "op": "append", "tokens": 256, "heads": 16, "cache": "e4m3", "interleaved": True, "dense": False},
        # A prompt's tokens into a bf16 cache, with the dense copy that its expansion reads.
        {"name": "append_prompt_8192", "op": "append", "tokens": 8192, "heads": 16, "cache": "bf16", "interleaved": False, "dense": True},
        # A short prompt alone: latency.
        {"name": "prefill_100", "op": "prefill", "batch": 1, "max_q": 100, "max_prefix": 0, "heads": 16, "causal": True},
        # A chunk of a prompt (or a draft) over a long prefix: few queries, many keys.
        {"name": "prefill_chunk_64", "op": "prefill", "batch": 1, "max_q": 64, "max_prefix": 8192, "heads": 16, "causal": True},
        # A ragged batch of prompts.
        {"name": "prefill_ragged_12", "op": "prefill", "batch": 12, "max_q": 2047, "max_prefix": 0, "heads": 16, "causal": True},
        # One long prompt.
        {"name": "prefill_16384", "op": "prefill", "batch": 1, "max_q": 16384, "max_prefix": 0, "heads": 16, "causal": True},
        # Joining a chunk with its prefix, and four pieces of a long prompt.
        {"name": "merge_2x64", "op": "merge", "pieces": 2, "tokens": 64, "heads": 16},
        {"name": "merge_4x16384", "op": "merge", "pieces": 4, "tokens": 16384, "heads": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["map", "append", "prefill", "prefill", "merge"])
    if op == "map":
        new = rng.choice([1, 1, _log(rng, 2, 1000)])
        batch = _log(rng, 1, 256)
        return {"op": op, "batch": batch, "max_len": _log(rng, 16, 8192), "max_new": new,
                "page": rng.choice([1, 16, 48, 64, 128])}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 8192), "heads": rng.choice([4, 16, 16]),
                "cache": rng.choice(["e4m3", "bf16"]), "interleaved": rng.random() < 0.5,
                "dense": rng.random() < 0.5}
    if op == "prefill":
        batch = _log(rng, 1, 24)
        max_q = _log(rng, 1, 8192 // batch if batch > 4 else 4096)
        prefix = rng.choice([0, _log(rng, 1, 8192 // batch + 1)])
        return {"op": op, "batch": batch, "max_q": max_q, "max_prefix": prefix,
                "heads": rng.choice([5, 16, 16]), "causal": rng.random() < 0.8}
    return {"op": op, "pieces": rng.randint(1, 6), "tokens": _log(rng, 1, 8192),
            "heads": rng.choice([5, 16, 16])}


# ---------------------------------------------------------------- sizes
def _spread(n, top, phase, uniform=False):
    """n lengths in 1 .. top, spread over the range, the first of them top."""
    return [top if i == 0 or uniform else 1 + int((top - 1) * ((i * 0.6180339887 + phase) % 1.0))
            for i in range(n)]


def _map_lens(case):
    b, uniform = case["batch"], case.get("uniform", False)
    new = _spread(b, case["max_new"], 0.29)
    return [n - 1 if uniform else n for n in _spread(b, case["max_len"], 0.37, uniform)], new


def _prefill_lens(case):
    b = case["batch"]
    q = _spread(b, case["max_q"], 0.37)
    prefix = _spread(b, case["max_prefix"], 0.61) if case["max_prefix"] else [0] * b
    return q, [x + y for x, y in zip(q, prefix)]


def _indptr(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def work(case):
    op = case["op"]
    if op == "map":
        before, new = _map_lens(case)
        page = case["page"]
        total = sum(before) + sum(new)
        pages = sum(-(-(x + y) // page) for x, y in zip(before, new))
        taken = sum(-(-(x + y) // page) + (-x // page) for x, y in zip(before, new))
        return {"bytes": 4 * (4 * case["batch"] + 2 + pages + taken + total + 2 * sum(new) + 1), "flops": 0}
    if op == "append":
        t, h = case["tokens"], case["heads"]
        row = 2 * KV_DIM + (KV_DIM if case["cache"] == "e4m3" else 2 * KV_DIM)
        row += (2 * KV_DIM if case["dense"] else 0) + 2 * 2 * ROPE * h + 8 + 4 * ROPE
        return {"bytes": t * row + 2 * LATENT, "flops": t * (5 * LATENT + 3 * ROPE * (h + 1))}
    if op == "prefill":
        q, kv = _prefill_lens(case)
        h = case["heads"]
        pairs = sum(n * k - (n * (n - 1) // 2 if case["causal"] else 0) for n, k in zip(q, kv))
        data = sum(q) * h * (2 * QK + 2 * VDIM + 4) + sum(kv) * (h * 2 * (NOPE + VDIM) + 2 * ROPE)
        return {"bytes": data, "flops": 2 * (QK + VDIM) * h * pairs}
    rows = case["tokens"] * case["heads"]
    return {"bytes": (case["pieces"] + 1) * rows * (2 * VDIM + 4), "flops": 3 * case["pieces"] * rows * VDIM}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rope_table(positions):
    """cos | sin of 32 frequencies for each position, float32 [positions, 64]."""
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "map":
        before, new = _map_lens(case)
        page, batch = case["page"], case["batch"]
        pages0 = [-(-n // page) for n in before]
        pages1 = [-(-(x + y) // page) for x, y in zip(before, new)]
        need, width = sum(pages1) - sum(pages0), max(pages1)
        pool = sum(pages1) + 8
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        rows = torch.repeat_interleave(torch.arange(batch, device="cuda"), _ints(pages0).long())
        cols = torch.arange(sum(pages0), device="cuda") - _ints(_indptr(pages0)).long()[rows]
        table[rows, cols] = ids[:sum(pages0)]
        s |= {"kv_lens": _ints(before), "new_lens": _ints(new), "table": table, "num_pages": pool,
              "free": ids[sum(pages0):].contiguous(), "need": need, "total": sum(before) + sum(new),
              "num_new": sum(new)}
        s["out"] = [torch.empty(n, dtype=torch.int32, device="cuda")
                    for n in (batch + 1, batch + 1, s["total"], s["num_new"], s["num_new"], 1)]
    elif op == "append":
        t, h = case["tokens"], case["heads"]
        rows = 2 * t + 64
        # the key's latent and rope part as a slice of a wider down-projection
        s["kv"] = (_randn(g, t, KV_DIM + 1536) * 0.7).bfloat16()[:, 1536:]
        s["weight"] = (1.0 + 0.2 * _randn(g, LATENT)).bfloat16()
        s["table"] = _rope_table(MAX_POS)
        s["positions"] = torch.randint(0, MAX_POS, (t,), generator=g, device="cuda", dtype=torch.int32)
        s["slots"] = torch.randperm(rows, generator=g, device="cuda")[:t].to(torch.int32)
        # the queries' rope part as a slice of the projected queries; the rotated one lands in the decode query
        s["q_pe"] = _randn(g, t, h, QK).bfloat16()[..., NOPE:]
        s["q"] = _randn(g, t, h, KV_DIM).bfloat16()
        old = _randn(g, rows, KV_DIM)
        s["scale"] = torch.full((1,), 8.0 / 448.0, device="cuda")
        s["pool"] = (old * 40).to(torch.float8_e4m3fn).view(torch.uint8) if case["cache"] == "e4m3" else old.bfloat16()
        s["latent"] = torch.empty(t, KV_DIM, dtype=torch.bfloat16, device="cuda") if case["dense"] else None
    elif op == "prefill":
        q, kv = _prefill_lens(case)
        h = case["heads"]
        s["q_lens"], s["kv_lens"] = q, kv
        s["q"] = (2.0 * _randn(g, sum(q), h, QK)).bfloat16()
        # keys and values side by side, as one expansion product leaves them; the rope key in the latent's row
        s["expanded"] = _randn(g, sum(kv), h, NOPE + VDIM).bfloat16()
        s["latent"] = _randn(g, sum(kv), KV_DIM).bfloat16()
        s["qo_indptr"], s["kv_indptr"] = _ints(_indptr(q)), _ints(_indptr(kv))
        s["out"] = torch.empty(sum(q), h, VDIM, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(sum(q), h, device="cuda")
    else:
        n, t, h = case["pieces"], case["tokens"], case["heads"]
        s["parts"] = _randn(g, n, t, h, VDIM).bfloat16()
        lse = 6.0 + 2.0 * _randn(g, n, t, h)
        empty = torch.rand(n, t, h, generator=g, device="cuda") < 0.05  # a piece that this query does not see
        s["lses"] = lse.masked_fill(empty, -math.inf)
        s["out"] = torch.empty(t, h, VDIM, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(t, h, device="cuda")
    if own:
        from mla_decode_attention_08_gb300 import binding
        s["lib"] = binding
        if op == "prefill":
            s["plan"] = binding.mla_prefill_plan(case["batch"], sum(s["q_lens"]), max(s["kv_lens"]), case["heads"])
            s["ws"] = binding.new_workspace(s["plan"])
        else:
            s["ws"] = torch.zeros(binding.STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _own_map(s):
    qo, kv, indices, slots, positions, used = s["out"]
    s["lib"].mla_page_map(s["kv_lens"], s["new_lens"], s["table"], s["free"], qo, kv, indices, slots, positions, used,
                          page_size=s["page"], num_pages=s["num_pages"], workspace=s["ws"])
    return s["out"] + [s["table"]]


def _own_append(s):
    args = (s["kv"], s["weight"], s["table"], s["positions"], s["slots"])
    more = dict(workspace=s["ws"], eps=EPS, interleaved=s["interleaved"], q_pe=s["q_pe"], q_out=s["q"][..., LATENT:],
                latent_out=s["latent"])
    if s["cache"] == "e4m3":
        s["lib"].mla_kv_append(*args, s["pool"], s["scale"], **more)
        pool = s["pool"].view(torch.float8_e4m3fn)
    else:
        s["lib"].mla_kv_append_bf16kv(*args, s["pool"], **more)
        pool = s["pool"]
    return [pool, s["q"]] + ([s["latent"]] if s["dense"] else [])


def _own_prefill(s):
    s["lib"].mla_prefill_fwd(s["q"], s["expanded"][..., :NOPE], s["latent"][:, LATENT:], s["expanded"][..., NOPE:],
                             s["qo_indptr"], s["kv_indptr"], s["out"], plan=s["plan"], workspace=s["ws"],
                             causal=s["causal"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _own_merge(s):
    s["lib"].mla_attn_merge(s["parts"], s["lses"], s["out"], lse_out=s["lse"])
    return [s["out"], s["lse"]]


def _plain_map(s):
    page, dev = s["page"], s["kv_lens"].device
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    before, new = s["kv_lens"].long(), s["new_lens"].long()
    total = before + new
    kv = torch.cat([zero, total.cumsum(0)])
    qo = torch.cat([zero, new.cumsum(0)])
    first = (before + page - 1) // page
    need = torch.cat([zero, ((total + page - 1) // page - first).cumsum(0)])
    table = s["table"].clone()
    i = torch.arange(s["need"], device=dev)
    b = torch.searchsorted(need[1:], i, right=True)
    table[b, first[b] + i - need[b]] = s["free"][:s["need"]]
    j = torch.arange(s["total"], device=dev)
    b = torch.searchsorted(kv[1:], j, right=True)
    at = j - kv[b]
    indices = table[b, at // page] * page + (at % page).int()
    j = torch.arange(s["num_new"], device=dev)
    b = torch.searchsorted(qo[1:], j, right=True)
    at = before[b] + j - qo[b]
    slots = table[b, at // page] * page + (at % page).int()
    return [qo.int(), kv.int(), indices, slots, at.int(), need[-1:].int(), table]


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_append(s):
    x = s["kv"].float()
    c, k_pe = x[:, :LATENT], x[:, LATENT:]
    c = c * torch.rsqrt(c.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    cos, sin = s["table"][s["positions"].long()].chunk(2, dim=1)
    row = torch.cat([c, _rotate(k_pe, cos, sin, s["interleaved"])], dim=1)
    slots = s["slots"].long()
    if s["cache"] == "e4m3":
        s["pool"][slots] = (row / s["scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        pool = s["pool"].view(torch.float8_e4m3fn)
    else:
        s["pool"][slots] = row.bfloat16()
        pool = s["pool"]
    s["q"][..., LATENT:] = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None], s["interleaved"]).bfloat16()
    return [pool, s["q"]] + ([row.bfloat16()] if s["dense"] else [])


def _padded(s, name, width):
    """Rows of a ragged batch as [batch, width], and which places of it are tokens."""
    at = s[name].long()
    place = torch.arange(width, device=at.device)
    inside = place < (at[1:] - at[:-1])[:, None]
    index = torch.minimum(at[:-1, None] + place, at[-1] - 1)
    return index, inside


def _plain_prefill(s):
    qi, q_in = _padded(s, "qo_indptr", max(s["q_lens"]))
    ki, k_in = _padded(s, "kv_indptr", max(s["kv_lens"]))
    q = s["q"][qi].float().transpose(1, 2)                        # [B, H, Lq, 192]
    e = s["expanded"][ki].float().transpose(1, 2)                 # [B, H, Lk, 256]
    rope = s["latent"][ki][:, None, :, LATENT:].float()           # [B, 1, Lk, 64], shared by the heads
    scores = (q[..., :NOPE] @ e[..., :NOPE].transpose(2, 3)).add_(q[..., NOPE:] @ rope.transpose(2, 3))
    scores *= 1.0 / math.sqrt(QK)
    seen = k_in[:, None, :]
    if s["causal"]:
        n, k = q_in.sum(1), k_in.sum(1)
        last = (k - n)[:, None] + torch.arange(qi.shape[1], device=qi.device)
        seen = seen & (torch.arange(ki.shape[1], device=qi.device) <= last[:, :, None])
    scores.masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(dim=3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(dim=3, keepdim=True)
    out = torch.where(total > 0, (p @ e[..., NOPE:]) / total, 0.0)
    lse = (total.log() + top).squeeze(3)
    at = _token_places(s, qi.shape[1])
    out = out.transpose(1, 2).flatten(0, 1)[at].bfloat16()
    return [out, lse.transpose(1, 2).flatten(0, 1)[at]]


def _token_places(s, width):
    """Where each token of the batch stands in the padded rows."""
    at = s["qo_indptr"].long()
    i = torch.arange(s["q"].shape[0], device=at.device)
    b = torch.searchsorted(at[1:], i, right=True)
    return b * width + i - at[b]


def _plain_merge(s):
    lses = s["lses"]
    top = lses.amax(dim=0)
    top = torch.where(top == -math.inf, 0.0, top)
    w = (lses - top).exp()
    total = w.sum(dim=0)
    out = torch.where(total[..., None] > 0, (w[..., None] * s["parts"].float()).sum(dim=0) / total[..., None], 0.0)
    return [out.bfloat16(), total.log() + top]


_OWN = {"map": _own_map, "append": _own_append, "prefill": _own_prefill, "merge": _own_merge}
_PLAIN = {"map": _plain_map, "append": _plain_append, "prefill": _plain_prefill, "merge": _plain_merge}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "map":
        return None  # whole numbers
    if case["op"] == "append":
        row = s["kv"].to(f64)
        mean = (row[:, :LATENT] ** 2).sum(1, keepdim=True) / LATENT
        row[:, :LATENT] *= s["weight"].to(f64) / (mean + EPS) ** 0.5
        turn = torch.complex(*s["table"][s["positions"].long()].to(f64).reshape(-1, 2, ROPE // 2).unbind(1))

        def turned(x, by):
            pairs = x.unflatten(-1, (ROPE // 2, 2)) if case["interleaved"] else x.unflatten(-1, (2, ROPE // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * by)
            return (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)

        row[:, LATENT:] = turned(row[:, LATENT:].clone(), turn)
        e4m3 = case["cache"] == "e4m3"
        pool = (s["pool"].view(torch.float8_e4m3fn) if e4m3 else s["pool"]).to(f64)
        pool[s["slots"].long()] = (row / s["scale"].to(f64)).clamp(-448.0, 448.0) if e4m3 else row
        q = s["q"].to(f64)
        q[..., LATENT:] = turned(s["q_pe"].to(f64), turn[:, None])
        return [pool, q] + ([row] if case["dense"] else [])
    if case["op"] == "prefill":
        h = case["heads"]
        outs, lses = [], []
        q0 = k0 = 0
        for n, k in zip(s["q_lens"], s["kv_lens"]):
            out = torch.zeros(n, h, VDIM, dtype=f64, device="cuda")
            lse = torch.zeros(n, h, dtype=f64, device="cuda")
            e, rope = s["expanded"][k0:k0 + k], s["latent"][k0:k0 + k, LATENT:].to(f64)
            hidden = None
            if case["causal"]:
                hidden = torch.ones(n, k, dtype=torch.bool, device="cuda").triu(k - n + 1)
            for i in range(h):
                key = torch.cat([e[:, i, :NOPE].to(f64), rope], dim=1)
                z = s["q"][q0:q0 + n, i].to(f64) @ key.T / QK ** 0.5
                if hidden is not None:
                    z.masked_fill_(hidden, -math.inf)
                lse[:, i] = torch.logsumexp(z, dim=1)
                out[:, i] = torch.exp(z - lse[:, i:i + 1]) @ e[:, i, NOPE:].to(f64)
            outs.append(out)
            lses.append(lse)
            q0, k0 = q0 + n, k0 + k
        return [torch.cat(outs), torch.cat(lses)]
    lse = torch.logsumexp(s["lses"].to(f64), dim=0)
    w = torch.where(s["lses"] == -math.inf, 0.0, torch.exp(s["lses"].to(f64) - lse))
    out = torch.einsum("pth,pthd->thd", w, s["parts"].to(f64))
    return [out, lse]
