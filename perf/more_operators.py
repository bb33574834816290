"""Cases, plain forms and measured work of the operators for decode steps over long contexts.

Five operators: ``mla_shared_fwd`` (decode queries of many rows over a prefix that
the rows share), ``mla_decode_fwd`` with the log-sum-exp that joins its rows to such
a prefix, ``mla_block_means`` (a mean of each page that a step has written to),
``mla_block_scores`` (what a row's queries score against its pages' means) and
``mla_block_select`` (the pages that a row attends, as the decode step's page table).

With ``own`` false ``run`` computes them with elementary torch operations; with
``own`` true it calls the framework.
"""
import math

import torch

own = False

HEADS, LATENT, DIM = 16, 512, 576
SCALE = 1.0 / 24.0  # 1 / sqrt(576)


def listed():
    return [
        # A few decode rows over a system prompt: latency.
        {"name": "shared_8x1000", "op": "shared", "groups": 1, "max_q": 8, "max_kv": 1000, "paged": True},
        # A decode batch over a long prefix that all of its rows share.
        {"name": "shared_64x8192", "op": "shared", "groups": 1, "max_q": 64, "max_kv": 8192, "paged": True},
        # Several prefixes, rows of each side by side; odd numbers of rows and tokens.
        {"name": "shared_groups_5", "op": "shared", "groups": 5, "max_q": 101, "max_kv": 6001, "paged": False},
        # The full batch over a document.
        {"name": "shared_256x32768", "op": "shared", "groups": 1, "max_q": 256, "max_kv": 32768, "paged": True},
        # The rows' own tokens behind a prefix: few, ragged, two query tokens a row.
        {"name": "lse_12x500", "op": "lse", "batch": 12, "max_kv": 500, "tokens": 2, "paged": False},
        # Long rows of their own.
        {"name": "lse_64x8192", "op": "lse", "batch": 64, "max_kv": 8192, "tokens": 1, "paged": True},
        # One new token a row: the page that each of them stands in.
        {"name": "means_decode_64", "op": "means", "batch": 64, "max_new": 1, "max_kv": 8192, "page": 64, "cache": "e4m3"},
        # Chunks of prompts.
        {"name": "means_prompts_9", "op": "means", "batch": 9, "max_new": 8000, "max_kv": 16001, "page": 64, "cache": "e4m3"},
        # Few rows at ordinary lengths, two query tokens each.
        {"name": "scores_4x8192", "op": "scores", "batch": 4, "max_kv": 8192, "tokens": 2, "page": 64},
        # A decode batch at long contexts.
        {"name": "scores_64x131072", "op": "scores", "batch": 64, "max_kv": 131072, "tokens": 1, "page": 64},
        # The same two for the choice.
        {"name": "select_4x8192", "op": "select", "batch": 4, "max_kv": 8192, "page": 64, "blocks": 32},
        {"name": "select_64x131072", "op": "select", "batch": 64, "max_kv": 131072, "page": 64, "blocks": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "lse", "means", "scores", "select"])
    if op == "shared":
        groups = rng.choice([1, 1, 1, _log(rng, 2, 12)])
        most = 256 // groups
        return {"op": op, "groups": groups, "max_q": _log(rng, 2, most), "max_kv": _log(rng, 1, 32768 // groups),
                "paged": rng.random() < 0.6}
    if op == "lse":
        batch = _log(rng, 1, 128)
        return {"op": op, "batch": batch, "max_kv": _log(rng, 8, min(16384, 524288 // batch)),
                "tokens": rng.choice([1, 1, 2, 3, 4]), "paged": rng.random() < 0.5}
    page = rng.choice([16, 32, 48, 64, 64, 128])
    if op == "means":
        batch = _log(rng, 1, 64)
        most = 65536 // batch
        return {"op": op, "batch": batch, "max_new": rng.choice([1, 1, _log(rng, 2, most // 2)]),
                "max_kv": _log(rng, most // 2 + 1, most), "page": page, "cache": rng.choice(["e4m3", "e4m3", "bf16"])}
    batch = _log(rng, 1, 64)
    case = {"op": op, "batch": batch, "max_kv": _log(rng, 1024, 131072 * page // 64), "page": page}
    if op == "scores":
        return case | {"tokens": rng.choice([1, 1, 2, 3, 4])}
    return case | {"blocks": _log(rng, 4, 128)}


# ---------------------------------------------------------------- sizes
def _spread(n, top, phase, low=1):
    """n lengths in low .. top, spread over the range, the first of them top."""
    return [top if i == 0 else low + int((top - low) * ((i * 0.6180339887 + phase) % 1.0)) for i in range(n)]


def _indptr(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _rows(case):
    """Query tokens and keys of each row (or group of rows) of the case."""
    if case["op"] == "shared":
        return _spread(case["groups"], case["max_q"], 0.29), _spread(case["groups"], case["max_kv"], 0.37)
    n = case.get("tokens", 1)
    low = max(n, case["max_kv"] // 2) if case["op"] in ("scores", "select") else n
    return [n] * case["batch"], _spread(case["batch"], case["max_kv"], 0.37, low)


def _new_tokens(case):
    """Of each row the tokens that it has after the step, and how many of them are the step's."""
    total = _spread(case["batch"], case["max_kv"], 0.37, case["max_new"])
    return total, [min(n, t) for n, t in zip(_spread(case["batch"], case["max_new"], 0.29), total)]


def _blocks(case):
    return [-(-n // case["page"]) for n in _rows(case)[1]]


def _chosen_tokens(case):
    kv = _rows(case)[1]
    k, page = case["blocks"], case["page"]
    return [n if b <= k else (k - 1) * page + n - (b - 1) * page for n, b in zip(kv, _blocks(case))]


def work(case):
    op = case["op"]
    if op in ("shared", "lse"):
        q, kv = _rows(case)
        heads = sum(q) * HEADS
        # causal: of n query tokens, token i does not see the last n - 1 - i keys
        pairs = sum(n * k - (n * (n - 1) // 2 if op == "lse" else 0) for n, k in zip(q, kv))
        data = sum(kv) * (DIM + (4 if case["paged"] else 0)) + heads * (2 * DIM + 2 * LATENT + 4)
        return {"bytes": data, "flops": 2 * (DIM + LATENT) * HEADS * pairs}
    if op == "means":
        total, new = _new_tokens(case)
        page = case["page"]
        first = [(t - n) // page for t, n in zip(total, new)]
        pages = sum(-(-t // page) - f for t, f in zip(total, first))
        tokens = sum(t - f * page for t, f in zip(total, first))
        elem = 1 if case["cache"] == "e4m3" else 2
        return {"bytes": tokens * DIM * elem + pages * DIM * 2 + 4 * sum(new), "flops": tokens * DIM}
    if op == "scores":
        q, blocks = _rows(case)[0], sum(_blocks(case))
        pairs = sum(n * b for n, b in zip(q, _blocks(case)))
        return {"bytes": blocks * (2 * DIM + 4 + 4) + sum(q) * HEADS * 2 * DIM, "flops": 2 * DIM * HEADS * pairs}
    taken = sum(min(b, case["blocks"]) for b in _blocks(case))
    return {"bytes": 4 * (sum(_blocks(case)) + 2 * taken + sum(_chosen_tokens(case)) + 2 * case["batch"]), "flops": 0}


# ---------------------------------------------------------------- inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _e4m3(g, rows):
    """A latent cache: codes whose values, times the scale, are about normal."""
    x = torch.randn(rows, DIM, generator=g, device="cuda")
    return x.mul_(60.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _pages(g, case, lens, spare=8):
    """Block table of rows of these lengths over a pool of shuffled pages, and the pool's size."""
    need = [-(-n // case["page"]) for n in lens]
    pool = sum(need) + spare
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    place = torch.arange(max(need), device="cuda")
    at = _ints(_indptr(need)).long()
    inside = place < (at[1:] - at[:-1])[:, None]
    table = torch.where(inside, ids[(at[:-1, None] + place).clamp_(max=sum(need) - 1)], -1)
    return table.contiguous(), pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("shared", "lse"):
        q, kv = _rows(case)
        rows = sum(kv) + (300 if case["paged"] else 0)
        s["cache"], s["scale"] = _e4m3(g, rows), torch.full((1,), 1.0 / 60.0, device="cuda")
        s["q"] = (1.5 * torch.randn(sum(q), HEADS, DIM, generator=g, device="cuda")).bfloat16()
        s["indices"] = None
        if case["paged"]:
            s["indices"] = torch.randperm(rows, generator=g, device="cuda")[:sum(kv)].to(torch.int32)
        s["qo_indptr"], s["kv_indptr"] = _ints(_indptr(q)), _ints(_indptr(kv))
        s["q_lens"], s["kv_lens"] = q, kv
        s["out"] = torch.empty(sum(q), HEADS, LATENT, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(sum(q), HEADS, device="cuda")
    elif op == "means":
        total, new = _new_tokens(case)
        table, pool = _pages(g, case, total)
        page = case["page"]
        s["num_pages"] = sum(-(-t // page) - (t - n) // page for t, n in zip(total, new))
        at = _ints(_indptr(new)).long()
        i = torch.arange(sum(new), device="cuda")
        row = torch.searchsorted(at[1:], i, right=True)
        pos = (_ints(total) - _ints(new))[row] + i - at[row]
        s["slots"] = (table[row, pos // page] * page + pos % page).int()
        if case["cache"] == "e4m3":
            s["pool"], s["scale"] = _e4m3(g, pool * page), torch.full((1,), 1.0 / 60.0, device="cuda")
        else:
            s["pool"] = torch.randn(pool * page, DIM, generator=g, device="cuda").bfloat16()
        s["means"] = torch.randn(pool, DIM, generator=g, device="cuda").bfloat16()
    else:
        q, kv = _rows(case)
        s["table"], pool = _pages(g, case, kv)
        s["kv_indptr"], s["num_blocks"] = _ints(_indptr(kv)), _blocks(case)
        if op == "scores":
            s["means"] = (0.25 * torch.randn(pool, DIM, generator=g, device="cuda")).bfloat16()
            s["q"] = torch.randn(sum(q), HEADS, DIM, generator=g, device="cuda").bfloat16()
            s["qo_indptr"] = _ints(_indptr(q))
            s["scores"] = torch.empty(s["table"].shape, device="cuda")
        else:
            # kept to few bits, so that some are alike
            s["scores"] = torch.randn(s["table"].shape, generator=g, device="cuda").bfloat16().float()
            s["total"], s["num_pages"] = sum(_chosen_tokens(case)), pool
            s["out"] = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (case["batch"] + 1, s["total"])]
            s["chosen"] = torch.empty(case["batch"], case["blocks"], dtype=torch.int32, device="cuda")
    if own:
        from mla_decode_attention_08_gb300 import binding
        s["lib"] = binding
        if op == "shared":
            s["plan"] = binding.mla_shared_plan(case["groups"], sum(q), max(kv))
            s["ws"] = binding.new_workspace(s["plan"])
        elif op == "lse":
            s["plan"] = binding.mla_decode_plan(case["batch"], max(kv), qo_len=case["tokens"])
            s["ws"] = binding.new_workspace(s["plan"])
        else:
            s["ws"] = torch.zeros(binding.STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _own_attention(s):
    call = s["lib"].mla_shared_fwd if s["op"] == "shared" else s["lib"].mla_decode_fwd
    call(s["q"], s["cache"], s["scale"], s["qo_indptr"], s["kv_indptr"], s["out"], plan=s["plan"], workspace=s["ws"],
         kv_indices=s["indices"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _own_means(s):
    more = dict(page_size=s["page"], workspace=s["ws"])
    if s["cache"] == "e4m3":
        s["lib"].mla_block_means(s["pool"], s["scale"], s["slots"], s["means"], **more)
    else:
        s["lib"].mla_block_means_bf16kv(s["pool"], s["slots"], s["means"], **more)
    return [s["means"]]


def _own_scores(s):
    s["lib"].mla_block_scores(s["q"], s["means"], s["table"], s["qo_indptr"], s["kv_indptr"], s["scores"],
                              page_size=s["page"], workspace=s["ws"])
    return [s["scores"]]


def _own_select(s):
    indptr, indices = s["out"]
    s["lib"].mla_block_select(s["scores"], s["table"], s["kv_indptr"], indptr, indices, page_size=s["page"],
                              num_pages=s["num_pages"], blocks=s["blocks"], sink=1, recent=2, chosen=s["chosen"],
                              workspace=s["ws"])
    return [indptr, indices, s["chosen"]]


def _plain_attention(s):
    """Rows as [rows, width], behind their ends the last token's place, which is masked."""
    qo, kv = s["qo_indptr"].long(), s["kv_indptr"].long()
    dev = qo.device
    i, j = torch.arange(max(s["q_lens"]), device=dev), torch.arange(max(s["kv_lens"]), device=dev)
    n, length = qo[1:] - qo[:-1], kv[1:] - kv[:-1]
    qi = torch.minimum(qo[:-1, None] + i, qo[-1] - 1)
    ki = torch.minimum(kv[:-1, None] + j, kv[-1] - 1)
    if s["indices"] is not None:
        ki = s["indices"].long()[ki]
    keys = s["cache"].view(torch.float8_e4m3fn)[ki].float() * s["scale"]              # [B, Lk, 576]
    q = s["q"][qi].float().flatten(1, 2)                                              # [B, Lq * 16, 576]
    scores = (q @ keys.transpose(1, 2)).mul_(SCALE).unflatten(1, (-1, HEADS))         # [B, Lq, 16, Lk]
    last = length[:, None] + 0 * i if s["op"] == "shared" else (length - n + 1)[:, None] + i
    scores.masked_fill_((j >= last[:, :, None])[:, :, None], -math.inf)
    top = scores.amax(dim=3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(dim=3, keepdim=True)
    out = (p.flatten(1, 2) @ keys[..., :LATENT]).unflatten(1, (-1, HEADS))
    out = torch.where(total > 0, out / total, 0.0)
    lse = (total.log() + top).squeeze(3)
    t = torch.arange(s["q"].shape[0], device=dev)
    row = torch.searchsorted(qo[1:], t, right=True)
    return [out[row, t - qo[row]].bfloat16(), lse[row, t - qo[row]]]


def _plain_means(s):
    page, slots = s["page"], s["slots"].long()
    # tokens that end their page, or with which their row ends
    goes_on = torch.cat([slots[1:] == slots[:-1] + 1, slots.new_zeros(1, dtype=torch.bool)])
    ends = (slots % page == page - 1) | ~goes_on
    ends = slots[torch.sort(ends.int(), descending=True, stable=True).indices[:s["num_pages"]]]
    pages, count = ends // page, (ends % page + 1)[:, None]
    x = s["pool"].view(torch.float8_e4m3fn) if s["cache"] == "e4m3" else s["pool"]
    x = x.unflatten(0, (-1, page))[pages].float()
    inside = torch.arange(page, device=slots.device) < count
    mean = torch.where(inside[..., None], x, 0.0).sum(dim=1) / count
    s["means"][pages] = (mean * s["scale"] if s["cache"] == "e4m3" else mean).bfloat16()
    return [s["means"]]


def _plain_scores(s):
    n = s["tokens"]
    kv = s["kv_indptr"].long()
    blocks = (kv[1:] - kv[:-1] + s["page"] - 1) // s["page"]
    means = s["means"][s["table"].long().clamp(min=0)].float()                          # [B, blocks, 576]
    q = s["q"].unflatten(0, (-1, n)).flatten(1, 2).float()                              # [B, n * 16, 576]
    scores = (q @ means.transpose(1, 2)).amax(dim=1) * SCALE
    j = torch.arange(scores.shape[1], device=kv.device)
    return [scores.masked_fill_(j >= blocks[:, None], -math.inf)]


def _plain_select(s):
    page, k = s["page"], s["blocks"]
    kv = s["kv_indptr"].long()
    length = (kv[1:] - kv[:-1])[:, None]
    count = (length + page - 1) // page
    j = torch.arange(s["scores"].shape[1], device=kv.device)
    always = (j < 1) | (j >= count - 2)
    score = s["scores"].masked_fill(always, math.inf).masked_fill(j >= count, -math.inf)
    order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k]
    order = torch.where(order < count, order, 1 << 30).sort(dim=1).values
    taken = order < count
    chosen = torch.full((len(order), k), -1, dtype=torch.int32, device=kv.device)
    chosen[:, :order.shape[1]] = torch.where(taken, order, -1).int()
    tokens = torch.where(taken, (length - order * page).clamp(max=page), 0)
    indptr = torch.cat([kv.new_zeros(1), tokens.sum(dim=1).cumsum(0)])
    page_at = s["table"].gather(1, torch.where(taken, order, 0)).flatten()
    ends = tokens.flatten().cumsum(0)
    i = torch.arange(s["total"], device=kv.device)
    piece = torch.searchsorted(ends, i, right=True)
    indices = page_at[piece] * page + i - (ends - tokens.flatten())[piece]
    return [indptr.int(), indices.int(), chosen]


_OWN = {"shared": _own_attention, "lse": _own_attention, "means": _own_means, "scores": _own_scores, "select": _own_select}
_PLAIN = {"shared": _plain_attention, "lse": _plain_attention, "means": _plain_means, "scores": _plain_scores,
          "select": _plain_select}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64, op = torch.float64, case["op"]
    if op in ("shared", "lse"):
        if work(case)["flops"] > 1e12:
            return None  # half a minute
        out = torch.zeros(*s["out"].shape, dtype=f64, device="cuda")
        lse = torch.zeros(*s["lse"].shape, dtype=f64, device="cuda")
        values = s["cache"].view(torch.float8_e4m3fn)
        q0 = k0 = 0
        for n, k in zip(s["q_lens"], s["kv_lens"]):
            rows = slice(k0, k0 + k) if s["indices"] is None else s["indices"][k0:k0 + k].long()
            key = values[rows].to(f64) * s["scale"].to(f64)
            for i in range(0, n, 64 if op == "shared" else 1):
                at = slice(q0 + i, q0 + min(n, i + 64 if op == "shared" else i + 1))
                seen = key if op == "shared" else key[:k - n + 1 + i]
                z = torch.einsum("thd,kd->thk", s["q"][at].to(f64), seen) / math.sqrt(DIM)
                lse[at] = torch.logsumexp(z, dim=2)
                out[at] = torch.einsum("thk,kd->thd", torch.exp(z - lse[at][..., None]), seen[:, :LATENT])
            q0, k0 = q0 + n, k0 + k
        return [out, lse]
    if op == "means":
        page = case["page"]
        means = s["means"].to(f64)
        x = (s["pool"].view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else s["pool"])
        scale = s["scale"].to(f64) if case["cache"] == "e4m3" else 1.0
        total, new = _new_tokens(case)
        slots = s["slots"].tolist()
        end = 0
        for t, n in zip(total, new):
            end += n
            for block in range((t - n) // page, -(-t // page)):
                last = min(t, (block + 1) * page) - 1
                slot = slots[end - t + last]
                row = slot - last % page
                means[row // page] = x[row:slot + 1].to(f64).mean(dim=0) * scale
        return [means]
    if op == "scores":
        scores = torch.full(s["scores"].shape, -math.inf, dtype=f64, device="cuda")
        n = case["tokens"]
        for b, blocks in enumerate(s["num_blocks"]):
            m = s["means"][s["table"][b, :blocks].long()].to(f64)
            z = torch.einsum("thd,kd->kth", s["q"][b * n:(b + 1) * n].to(f64), m) / math.sqrt(DIM)
            scores[b, :blocks] = z.flatten(1).max(dim=1).values
        return [scores]
    return None  # whole numbers
