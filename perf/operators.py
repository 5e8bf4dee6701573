"""The operators of dense MLA serving over the paged latent cache, as they are measured.

Two operators, each over a bf16 cache and over an E4M3 cache with one fp32 scale:

* append: a step's new latent rows, RMS-normalised, with the position rotation applied to
  their last 64 channels (none where rope is 0), written to their pages; and the rotation of
  the step's query heads on the way.
* attention: MLA of a batch whose requests share a prefix, over the prefix's pages and each
  request's own, causal by the query's position.

With `own` false, run() computes them in their plain form: elementary torch operations in
fp32, rounded once at the end. With `own` true it calls the library.
"""
import math

import torch

own = False

LORA = 512                # latent width: key and value
DEV = "cuda"


def listed():
    def attn(name, **kw):
        case = dict(name=name, op="attention", requests=1, per_request=1, heads=64, prefix=0, longest=512, page=64, rope=0, fp8=False)
        case.update(kw)
        return case

    def append(name, **kw):
        case = dict(name=name, op="append", requests=1, tokens=1, heads=64, context=512, page=64, rope=64, interleaved=True, fp8=False)
        case.update(kw)
        return case

    return [
        # the smallest step: one request of 512 tokens on a rank that holds 16 heads
        attn("attend 1x512", heads=16, page=16),
        # one user's long conversation, decoded alone; an odd length, rotated keys, all heads on one GPU
        attn("attend 1x65537 rope", heads=128, longest=65537, rope=64),
        # a batch behind one system prompt; NoPE latents
        attn("attend 16 behind 6144", requests=16, prefix=6144, longest=2048),
        # many short questions about one long document, 16 heads a rank, two draft tokens each, small pages
        attn("attend 64x2 behind 16389 rope", requests=64, per_request=2, heads=16, prefix=16389, longest=700, page=16, rope=64),
        # four unshared long contexts: the cache is read once from HBM
        attn("attend 4x131072", requests=4, longest=131072),
        # a full batch of all 128 heads behind a long prompt: the largest product
        attn("attend 64 behind 16384 rope", requests=64, heads=128, prefix=16384, longest=1000, rope=64),
        # a ragged batch with nothing shared, fp8 cache
        attn("attend 64 ragged fp8", requests=64, longest=32768, fp8=True),
        # a batch behind one prompt, fp8 cache with rotated keys, 32 heads a rank, pages that are no power of two
        attn("attend 33 behind 4100 fp8 rope", requests=33, heads=32, prefix=4100, longest=1500, page=24, rope=64, fp8=True),
        # one new token of one request
        append("append 1", heads=16),
        # a decode step of a full batch
        append("append 64 heads 128", requests=64, tokens=1, heads=128, context=1024),
        # a chunk of a prompt into an fp8 cache, halves rotated
        append("append 2048 fp8", tokens=2048, context=4096, interleaved=False, fp8=True),
        # several prompts at once; NoPE, so no query heads pass through; small pages
        append("append 16x1021 nope", requests=16, tokens=1021, rope=0, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    rope = rng.choice((0, 64))
    page = rng.choice((16, 24, 32, 64, 128))
    fp8 = rng.random() < 0.4
    if rng.random() < 0.4:
        requests = _log(rng, 1, 64)
        return dict(op="append", requests=requests, tokens=max(1, _log(rng, 1, 8192) // requests), heads=rng.choice((16, 32, 64, 128)), context=_log(rng, 1, 4096), page=page, rope=rope, interleaved=rng.random() < 0.5, fp8=fp8)
    case = dict(op="attention", requests=_log(rng, 1, 128), per_request=rng.choice((1, 1, 1, 2, 3)), heads=rng.choice((16, 32, 48, 64, 96, 128)), prefix=rng.choice((0, _log(rng, 16, 32768))), longest=_log(rng, 1, 32768), page=page, rope=rope, fp8=fp8)
    top = next(c for c in listed() if c["name"] == "attend 64 behind 16384 rope")
    while case["requests"] > 1 and (work(case)["flops"] > work(top)["flops"] or case["requests"] * case["longest"] > 1 << 21):
        case["requests"] = case["requests"] * 3 // 4
    return case


def _own_lengths(case):
    """Tokens of each request behind the prefix: all the longest for up to four requests, else
    spread from 1 (a 32nd of the longest where nothing is shared) up to the longest."""
    n, top = case["requests"], case["longest"]
    if n <= 4:
        return [top] * n
    low = 1 if case["prefix"] else max(1, top // 32)
    return [low + int((top - low) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(n - 1)] + [top]


def work(case):
    width = LORA + case["rope"]
    size = 1 if case["fp8"] else 2
    if case["op"] == "append":
        n = case["requests"] * case["tokens"]
        rotated = n * case["heads"] * case["rope"] * 2 * 2
        return {"bytes": n * (width * (2 + size) + 4 * case["rope"] + 8) + rotated, "flops": n * (5 * LORA + 3 * case["rope"] * (1 + case["heads"]))}
    lengths, per = _own_lengths(case), case["per_request"]
    rows = case["requests"] * per * case["heads"]
    seen = sum(case["prefix"] + n - (per - 1 - j) for n in lengths for j in range(per) if case["prefix"] + n - (per - 1 - j) > 0)
    held = case["prefix"] + sum(lengths)
    return {"bytes": held * width * size + rows * (2 * width + 2 * LORA + 4), "flops": 2 * seen * case["heads"] * (width + LORA)}


def _table(counts, page, gen):
    """Pages of several sequences, scattered over one pool: ([n, most] page numbers, pages in the pool)."""
    need = [-(-c // page) for c in counts]
    total, most = sum(need) + 3, max(1, max(need))
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(counts), most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table, total


def _cache(rows, width, fp8, gen):
    x = torch.empty(rows, width, dtype=torch.bfloat16, device=DEV)
    step = 1 << 18
    for i in range(0, rows, step):
        x[i:i + step] = torch.randn(min(step, rows - i), width, generator=gen, device=DEV)
    return x.to(torch.float8_e4m3fn) if fp8 else x


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return _prepare_append(case, gen) if case["op"] == "append" else _prepare_attention(case, gen)


def _prepare_append(case, gen):
    B, each, page, rope, heads = case["requests"], case["tokens"], case["page"], case["rope"], case["heads"]
    n, width = B * each, LORA + rope
    first = [max(0, case["context"] - 7 * i) for i in range(B)]          # position of each request's first new token
    table, pages = _table([f + each for f in first], page, gen)
    s = dict(case=case, n=n, width=width, table=table, rows=pages * page, scale=0.125)
    s["cache"] = _cache(pages * page, width, case["fp8"], gen)
    # the rows come out of a projection whose other columns (the query's latents) lie beside them
    s["joint"] = (torch.randn(n, 64 + width, generator=gen, device=DEV) * 2).to(torch.bfloat16)
    s["new"] = s["joint"][:, 64:]
    s["norm"] = (1 + 0.1 * torch.randn(LORA, generator=gen, device=DEV)).to(torch.bfloat16)
    s["req"] = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(each)
    s["pos"] = (torch.tensor(first, device=DEV)[:, None] + torch.arange(each, device=DEV)).reshape(-1).to(torch.int32)
    s["max_pos"] = case["context"] + each
    s["cos_sin"] = s["q"] = s["q_new"] = s["q_rot"] = None
    if rope:
        freq = 10000.0 ** (-torch.arange(rope // 2, device=DEV, dtype=torch.float64) * 2 / rope)
        angle = torch.arange(s["max_pos"], device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        # query heads of 128 unrotated and 64 rotated channels; the first 512 columns of q are already in the latent space
        s["q_new"] = torch.randn(n, heads, 128 + rope, generator=gen, device=DEV).to(torch.bfloat16)
        s["q_rot"] = s["q_new"][..., 128:]
        s["q"] = torch.randn(n, heads, width, generator=gen, device=DEV).to(torch.bfloat16)
    return s


def _prepare_attention(case, gen):
    B, per, page, width, heads = case["requests"], case["per_request"], case["page"], LORA + case["rope"], case["heads"]
    P, lengths = case["prefix"], _own_lengths(case)
    whole = P // page * page                             # the requests' own pages begin with the page that the prefix ends in
    both, pages = _table([P] + [P - whole + n for n in lengths], page, gen)
    s = dict(case=case, width=width, scale=0.125, rows=pages * page, sm_scale=1.0 / math.sqrt(width))
    s["prefix_table"] = both[0, :max(1, -(-P // page))].contiguous()
    s["table"] = torch.cat([torch.full((B, whole // page), -1, dtype=torch.int32, device=DEV), both[1:]], 1).contiguous()
    s["prefix_len"] = torch.tensor([P], dtype=torch.int32, device=DEV)
    s["seq_len"] = torch.tensor([P + n for n in lengths], dtype=torch.int32, device=DEV)
    s["q_req"] = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(per)
    back = torch.arange(per, device=DEV, dtype=torch.int32) - per       # the request's last tokens
    s["q_pos"] = (s["seq_len"][:, None] + back).reshape(-1).contiguous()
    s["cache"] = _cache(pages * page, width, case["fp8"], gen)
    s["q"] = torch.randn(B * per, heads, width, generator=gen, device=DEV).to(torch.bfloat16)
    s["out"] = torch.empty(B * per, heads, LORA, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(B * per, heads, dtype=torch.float32, device=DEV)
    s["ws"] = None                                       # the library's scratch, kept from the first call on
    return s


def run(s):
    if own:
        return _own_append(s) if s["case"]["op"] == "append" else _own_attention(s)
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attention(s)


def _own_append(s):
    from sparse_attention_indexer_head_b200 import binding as lib
    c = s["case"]
    shape = (s["joint"].stride(0), s["norm"], 1e-6, s["cos_sin"], s["max_pos"], int(c["interleaved"]), s["req"], s["pos"], s["n"], LORA, c["rope"], s["table"], c["requests"], s["table"].shape[1], c["page"])
    queries = (s["q_rot"], s["q_new"].stride(0), s["q_new"].stride(1), c["heads"], s["q"]) if c["rope"] else (None, 0, 0, 0, None)
    if c["fp8"]:
        lib.dsa_latent_append_paged_fp8(s["new"], *shape, s["cache"], s["scale"], s["rows"], *queries)
    else:
        lib.dsa_latent_append_paged(s["new"], *shape, s["cache"], s["rows"], *queries)
    return (s["cache"], s["q"]) if c["rope"] else s["cache"]


def _own_attention(s):
    from sparse_attention_indexer_head_b200 import binding as lib
    c = s["case"]
    Q = s["q"].shape[0]
    if s["ws"] is None:
        s["ws"] = torch.empty(lib.dsa_prefix_mla_workspace_size(Q, c["heads"]), dtype=torch.uint8, device=DEV)
    where = (s["prefix_table"], s["prefix_table"].numel(), s["prefix_len"], s["table"], s["table"].shape[1], c["page"], s["seq_len"], s["q_req"], s["q_pos"], Q, c["requests"], c["heads"], LORA, c["rope"], s["sm_scale"], s["out"], s["lse"], s["ws"], s["ws"].numel())
    if c["fp8"]:
        lib.dsa_prefix_mla_decode_paged_fp8(s["q"], s["cache"], s["scale"], s["rows"], *where)
    else:
        lib.dsa_prefix_mla_decode_paged(s["q"], s["cache"], s["rows"], *where)
    return s["out"], s["lse"]


def _rotate(x, cos, sin, interleaved):
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def _plain_append(s):
    c, page, rope = s["case"], s["case"]["page"], s["case"]["rope"]
    pos = s["pos"].long()
    row = s["table"][s["req"].long(), pos // page].long() * page + pos % page
    x = s["new"].float()
    lat = x[:, :LORA]
    y = lat * torch.rsqrt((lat * lat).mean(1, keepdim=True) + 1e-6) * s["norm"].float()
    if rope:
        cos, sin = s["cos_sin"][pos].split(rope // 2, 1)
        y = torch.cat([y, _rotate(x[:, LORA:], cos, sin, c["interleaved"])], 1)
        s["q"][..., LORA:] = _rotate(s["q_rot"].float(), cos[:, None], sin[:, None], c["interleaved"]).to(torch.bfloat16)
    if c["fp8"]:
        s["cache"].view(torch.uint8)[row] = (y / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["cache"][row] = y.to(torch.bfloat16)
    return (s["cache"], s["q"]) if rope else s["cache"]


def _gather(s, table, at):
    """Rows of the cache that hold the tokens `at` of the sequences of `table`, in fp32."""
    page = s["case"]["page"]
    row = torch.gather(table.long(), 1, at // page).clamp_min(0) * page + at % page
    if s["case"]["fp8"]:
        return s["cache"].view(torch.uint8)[row].view(torch.float8_e4m3fn).float() * s["scale"]
    return s["cache"][row].float()


def _plain_attention(s):
    c = s["case"]
    B, P, heads, width = c["requests"], c["prefix"], c["heads"], s["width"]
    q = s["q"].float().view(B, -1, width)                            # [requests, queries x heads, width]
    at = torch.arange(P, P + c["longest"], device=DEV)
    shared = _gather(s, s["prefix_table"][None], torch.arange(P, device=DEV)[None])[0]
    mine = _gather(s, s["table"], at.clamp_max(s["table"].shape[1] * c["page"] - 1).expand(B, -1))
    z = torch.cat([q @ shared.t(), q @ mine.transpose(1, 2)], 2) * s["sm_scale"]
    token = torch.cat([torch.arange(P, device=DEV), at])
    last = torch.minimum(s["q_pos"], s["seq_len"][s["q_req"].long()] - 1).view(B, -1).repeat_interleave(heads, 1)
    z = z.masked_fill(token > last[..., None], -math.inf)
    top = z.amax(2, keepdim=True).clamp_min(-3e38)
    p = torch.exp(z - top)
    total = p.sum(2, keepdim=True)
    o = (p[..., :P] @ shared[:, :LORA] + p[..., P:] @ mine[..., :LORA]) / total.clamp_min(1e-38)
    lse = torch.log(total) + torch.where(total > 0, top, 0.0)
    return o.view(-1, heads, LORA).to(torch.bfloat16), lse.view(-1, heads)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    """Row by row formula in complex arithmetic: a rotated pair is (a + ib) (cos + i sin)."""
    c, page, rope, heads = s["case"], s["case"]["page"], s["case"]["rope"], s["case"]["heads"]
    cache = s["cache"].double()
    pages = s["table"].double()[s["req"].long(), torch.div(s["pos"].long(), page, rounding_mode="floor")]
    row = (pages * page + torch.remainder(s["pos"], page)).long()
    x = s["joint"].double()
    lat = x[:, 64:64 + LORA]
    norm = (lat.square().sum(1) / LORA + 1e-6).sqrt()
    unit = 1.0 / s["scale"] if c["fp8"] else 1.0
    most = 448.0 if c["fp8"] else math.inf               # E4M3 saturates
    cache[row, :LORA] = (lat / norm[:, None] * s["norm"].double() * unit).clamp(-most, most)
    if not rope:
        return cache
    turn = torch.complex(s["cos_sin"].double()[s["pos"].long(), :rope // 2], s["cos_sin"].double()[s["pos"].long(), rope // 2:])

    def turned(v, by):
        pair = v.unflatten(-1, (rope // 2, 2)) if c["interleaved"] else v.unflatten(-1, (2, rope // 2)).transpose(-1, -2)
        w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * by)
        return (w if c["interleaved"] else w.transpose(-1, -2)).flatten(-2)

    cache[row, LORA:] = (turned(x[:, 64 + LORA:], turn) * unit).clamp(-most, most)
    q = s["q"].double()
    for h in range(heads):
        q[:, h, LORA:] = turned(s["q_new"][:, h, 128:].double(), turn)
    return cache, q


def _exact_attention(s):
    """One query after another, its tokens in order, in blocks of heads."""
    c, page, P = s["case"], s["case"]["page"], s["case"]["prefix"]
    unit = s["scale"] if c["fp8"] else 1.0
    raw = s["cache"].view(torch.uint8) if c["fp8"] else s["cache"]
    value = (lambda rows: raw[rows].view(torch.float8_e4m3fn).double() * unit) if c["fp8"] else (lambda rows: raw[rows].double())
    prefix = s["prefix_table"].long()
    out, lse = [], []
    held, kv = None, None
    for i, (b, pos) in enumerate(zip(s["q_req"].tolist(), s["q_pos"].tolist())):
        n = min(pos + 1, int(s["seq_len"][b]))
        if held != b:
            t = torch.arange(max(0, int(s["seq_len"][b])), device=DEV)
            row = torch.where(t < P, prefix[(t // page).clamp_max(prefix.numel() - 1)], s["table"].long()[b][t // page]) * page + t % page
            held, kv = b, value(row)
        if n <= 0:
            out.append(torch.zeros(c["heads"], LORA, dtype=torch.float64, device=DEV))
            lse.append(torch.full((c["heads"],), -math.inf, dtype=torch.float64, device=DEV))
            continue
        z = torch.einsum("hd,td->ht", s["q"][i].double(), kv[:n]) * s["sm_scale"]
        lse.append(torch.logsumexp(z, 1))
        out.append(torch.einsum("ht,td->hd", torch.softmax(z, 1), kv[:n, :LORA]))
    return torch.stack(out), torch.stack(lse)
