"""The paged K/V cache operators: what is measured, their plain forms and their exact values.

A pool holds pages of cache rows; a row is one position of a sequence, all kv
heads: ``Hkv * 128`` values and 16 bytes.  bf16 rows end in 8 zeros; E4M3 rows
hold codes, then one E8M0 scale byte (2^(byte - 127)) per kv head, then zeros.
``block_table[b, j // page_size]`` is the page of position j of sequence b.
Queries of all sequences are packed: sequence b owns tokens ``q_start[b] ..
q_start[b + 1]``, the last ones of its ``kv_len[b]`` positions.

Four operators: ``write`` stores the new tokens' K and V into their pages,
``gather`` reads selected rows back as compact bf16 rows, ``attn`` attends with
a chunk of new tokens (one token is the smallest chunk) over every cached
position up to its own, ``sparse`` attends with one token per sequence over
selected rows.
"""
import torch

own = False

D = 128
PAD = 16   # bytes at the end of a row


# ------------------------------------------------------------------ cases
def _case(name, op, kv_type, hq, hkv, page, q="", kv="", k=0, counts=""):
    return {"name": name, "op": op, "type": kv_type, "hq": hq, "hkv": hkv, "page": page, "q": q, "kv": kv, "k": k,
            "counts": counts}


def _text(v):
    return ",".join(str(x) for x in v)


def listed():
    return [
        # one decode step of 8 short conversations: the smallest call, latency
        _case("write_decode_8", "write", "e4m3", 32, 8, 64, _text([1] * 8), "2049,130,64,1,777,1500,2048,65"),
        # a prefill batch appended behind cached prefixes, ragged, odd lengths
        _case("write_prefill_32k", "write", "e4m3", 32, 8, 64, "16384,9001,4096,3286,1", "16384,12001,4097,3286,700"),
        # the selected rows of one decode step of the 8 x 32K workload, read back once for a group of layers
        _case("gather_8x2048", "gather", "e4m3", 32, 8, 64, "", _text([32769] * 8), 2048, _text([2048] * 8)),
        # rows of a gist route with few chunks, ragged counts, one sequence with none
        _case("gather_ragged", "gather", "bf16", 16, 4, 16, "", "9000,1088,40,5", 1088, "1088,1071,17,0"),
        # the 8 x 32K decode step itself, straight from the pages
        _case("sparse_8x32k", "sparse", "e4m3", 32, 8, 64, "", _text([32769] * 8), 2048, _text([2048] * 8)),
        # one sequence of a million tokens
        _case("sparse_1m", "sparse", "bf16", 32, 8, 64, "", "1048577", 2048, "2048"),
        # a dense layer's decode step of one short conversation: the smallest attention call
        _case("decode_1x2k", "attn", "bf16", 32, 8, 16, "1", "2049"),
        # a dense layer's decode step of the 8 x 32K workload
        _case("decode_8x32k", "attn", "e4m3", 32, 8, 64, _text([1] * 8), _text([32769] * 8)),
        # four drafted tokens and the last accepted one checked for 16 sequences
        _case("draft_16x5", "attn", "e4m3", 16, 2, 16, _text([5] * 16), _text([8197 - 509 * i for i in range(16)])),
        # a whole prompt of 2K tokens
        _case("prompt_2k", "attn", "bf16", 32, 8, 64, "2048", "2048"),
        # a mixed batch: one chunk of a prompt among sequences that decode
        _case("mixed_1536", "attn", "bf16", 32, 8, 32, "1,1536,1,1,7,1", "8193,5633,77,12001,4103,1"),
        # the last 8K chunk of a 64K prompt: the largest call
        _case("chunk_8k_of_64k", "attn", "e4m3", 32, 8, 64, "8192", "65536"),
    ]


def _unnamed(*args):
    case = _case("", *args)
    del case["name"]
    return case


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["write", "gather", "sparse", "attn", "attn", "attn"])
    kv_type = rng.choice(["e4m3", "bf16"])
    hkv = rng.choice([1, 2, 3, 4, 6, 8, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    B = _log_int(rng, 1, 32)
    if op in ("gather", "sparse"):
        kv = [_log_int(rng, 1, 524288 // B) for _ in range(B)]
        k = _log_int(rng, 1, 4096)
        counts = [0 if rng.random() < 0.05 else min(k, n) for n in kv]
        return _unnamed(op, kv_type, hq, hkv, page, "", _text(kv), k, _text(counts))
    most = 65536 if op == "attn" else 8192
    kv = [_log_int(rng, 1, min(most, 524288 // B)) for _ in range(B)]
    longest = rng.choice([1, 8, 512, 8192])   # decode, drafts, chunks, whole prompts
    q = [min(n, _log_int(rng, 1, longest)) for n in kv]
    budget = 8192 * 57344 * 32                # pairs x heads of the largest listed call
    for i in range(B):
        q[i] = max(1, min(q[i], budget // (B * hq * kv[i])))
    return _unnamed(op, kv_type, hq, hkv, page, _text(q), _text(kv))


# ----------------------------------------------------------------- inputs
def _ints(text):
    return [int(x) for x in text.split(",") if x]


def _exponents(amax):
    """The least e within [-118, 119] with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 0.875, ex - 9, ex - 8).clamp(-118, 119)
    return torch.where(amax == 0, torch.full_like(e, -118), e)


def _rows_of(x, kv_type):
    """Cache rows [n, row] of new K or V values x [n, Hkv, 128]."""
    n, hkv = x.shape[:2]
    if kv_type == "bf16":
        return torch.nn.functional.pad(x.reshape(n, hkv * D), (0, PAD // 2))
    v = x.float()
    e = _exponents(v.abs().amax(-1))
    codes = torch.ldexp(v, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    tail = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, PAD - hkv))
    return torch.cat([codes.reshape(n, hkv * D), tail], 1)


def _values_of(rows, kv_type):
    """fp32 values [..., Hkv, 128] of cache rows [..., row]."""
    if kv_type == "bf16":
        return rows[..., :-PAD // 2].float().unflatten(-1, (-1, D))
    hkv = (rows.shape[-1] - PAD) // D
    v = rows[..., :hkv * D].view(torch.float8_e4m3fn).float().unflatten(-1, (hkv, D))
    return torch.ldexp(v, rows[..., hkv * D:hkv * D + hkv].int()[..., None] - 127)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    hq, hkv, page, kv_type, op = case["hq"], case["hkv"], case["page"], case["type"], case["op"]
    q_len, kv_len = _ints(case["q"]), _ints(case["kv"])
    B = len(kv_len)
    need = [(n + page - 1) // page for n in kv_len]
    num_pages = sum(need) + 3
    perm = torch.randperm(num_pages, generator=host)
    table = torch.zeros(B, max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].int()
        at += n
    # keys have a few channels much larger than the others, values a mean: what quantisation and softmax meet
    gain = torch.ones(hkv, D, device=dev)
    gain[:, ::29] = 5.0
    mean = torch.randn(hkv, D, device=dev, generator=g) * 0.5
    slots = num_pages * page

    def pool(scale, shift):
        parts = []
        for s in range(0, slots, 1 << 16):
            x = torch.randn(min(1 << 16, slots - s), hkv, D, device=dev, generator=g) * scale + shift
            parts.append(_rows_of(x.bfloat16(), kv_type))
        return torch.cat(parts).view(num_pages, page, -1)

    s = {"case": case, "q_len": q_len, "kv": kv_len, "k_pages": pool(gain, 0.0), "v_pages": pool(1.0, mean),
         "table": table.to(dev), "kv_len": torch.tensor(kv_len, dtype=torch.int32, device=dev)}
    if op in ("write", "attn"):
        N = sum(q_len)
        s["max_q"] = max(q_len)
        s["q_start"] = torch.tensor([sum(q_len[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
        # what a fused projection gives: q, k and v of a token side by side
        qkv = torch.randn(N, hq + 2 * hkv, D, device=dev, generator=g)
        qkv[:, hq:hq + hkv] *= gain
        qkv[:, hq + hkv:] += mean
        qkv = qkv.bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        k, counts = case["k"], _ints(case["counts"])
        idx = torch.full((B, k), -1, dtype=torch.int32, device=dev)
        for b, c in enumerate(counts):   # ascending distinct positions, as the top-k gives them
            idx[b, :c] = torch.randperm(kv_len[b], device=dev, generator=g)[:c].sort().values.int()
        s["idx"], s["count"] = idx, torch.tensor(counts, dtype=torch.int32, device=dev)
        s["q"] = torch.randn(B, hq, D, device=dev, generator=g).bfloat16()
    if op == "write":   # the updated pools, codes as the values they stand for beside their scale bytes
        w = hkv * D
        if kv_type == "bf16":
            s["pools"] = (s["k_pages"], s["v_pages"])
        else:
            s["pools"] = tuple(x for p in (s["k_pages"], s["v_pages"])
                               for x in (p[..., :w].view(torch.float8_e4m3fn), p[..., w:]))
    return s


# ------------------------------------------------------------ plain forms
def _plain_write(s):
    case = s["case"]
    page, N = case["page"], s["k"].shape[0]
    i = torch.arange(N, device=s["k"].device)
    b = torch.searchsorted(s["q_start"][1:].long(), i, right=True)
    pos = s["kv_len"][b] - s["q_start"][b + 1] + i
    slot = s["table"][b, pos // page].long() * page + pos % page
    for new, pages in ((s["k"], s["k_pages"]), (s["v"], s["v_pages"])):
        pages.view(-1, pages.shape[-1])[slot] = _rows_of(new, case["type"])
    return s["pools"]


def _selected(s):
    """The selected rows [B, k, row] of both pools; rows past the count are any rows."""
    page = s["case"]["page"]
    j = s["idx"].clamp(min=0).long()
    slot = torch.gather(s["table"].long(), 1, j // page) * page + j % page
    return [p.view(-1, p.shape[-1])[slot] for p in (s["k_pages"], s["v_pages"])]


def _plain_gather(s):
    used = torch.arange(s["idx"].shape[1], device=s["idx"].device) < s["count"][:, None]
    out = []
    for rows in _selected(s):
        v = torch.where(used[..., None, None], _values_of(rows, s["case"]["type"]), 0.0)
        out.append(torch.nn.functional.pad(v.flatten(-2).bfloat16(), (0, PAD // 2)))
    return tuple(out)


def _attend(q, k, v, seen):
    """q [h, g, n, D], k and v [h, S, D], all fp32; seen [n, S] or [S].  out [h, g, n, D], lse [h, g, n]."""
    h, g, n, _ = q.shape
    z = torch.matmul(q.flatten(1, 2) * D ** -0.5, k.transpose(1, 2)).view(h, g, n, -1)
    z.masked_fill_(~seen, float("-inf"))
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)   # a row that sees nothing stays finite
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(1, 2), v).view(h, g, n, D) / total.clamp(min=1e-30)
    return o, (m + torch.log(total)).squeeze(-1)


def _plain_sparse(s):
    B, k = s["idx"].shape
    hkv = s["case"]["hkv"]
    kr, vr = (_values_of(r, s["case"]["type"]).transpose(1, 2).reshape(B * hkv, k, D) for r in _selected(s))
    q = s["q"].float().view(B * hkv, -1, 1, D)
    seen = torch.arange(k, device=q.device) < s["count"].repeat_interleave(hkv)[:, None]
    o, lse = _attend(q, kr, vr, seen[:, None, None, :])
    return o.reshape(B, -1, D).bfloat16(), lse.reshape(B, -1)


def _plain_attn(s):
    case = s["case"]
    hkv, hq, page = case["hkv"], case["hq"], case["page"]
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=s["q"].device)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
    at = 0
    for b, (T, S) in enumerate(zip(s["q_len"], s["kv"])):
        pages = s["table"][b, :(S + page - 1) // page].long()
        k, v = (_values_of(p[pages].flatten(0, 1)[:S], case["type"]).transpose(0, 1) for p in (s["k_pages"], s["v_pages"]))
        j = torch.arange(S, device=k.device)
        step = max(1, (1 << 30) // (hq * S))     # 4 GiB of scores at a time
        for t in range(0, T, step):
            n = min(step, T - t)
            q = s["q"][at + t:at + t + n].float().view(n, hkv, hq // hkv, D).permute(1, 2, 0, 3)
            o, l = _attend(q, k, v, j <= (S - T + t + torch.arange(n, device=k.device))[:, None])
            out[at + t:at + t + n] = o.permute(2, 0, 1, 3).reshape(n, hq, D).bfloat16()
            lse[at + t:at + t + n] = l.permute(2, 0, 1).reshape(n, hq)
        at += T
    return out, lse


def run(s):
    op = s["case"]["op"]
    if own:
        import shared_top_routing_b200 as sa
        if op == "write":
            sa.sa_paged_kv_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["q_start"], s["kv_len"])
            return s["pools"]
        if op == "gather":
            return sa.sa_paged_kv_gather(s["k_pages"], s["v_pages"], s["table"], s["idx"], s["count"])
        if op == "sparse":
            return sa.sa_paged_sparse_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["idx"], s["count"],
                                                  with_lse=True)
        return sa.sa_paged_attn(s["q"], s["k_pages"], s["v_pages"], s["table"], s["q_start"], s["kv_len"], s["max_q"],
                                with_lse=True)
    return {"write": _plain_write, "gather": _plain_gather, "sparse": _plain_sparse, "attn": _plain_attn}[op](s)


def work(case):
    hq, hkv = case["hq"], case["hkv"]
    q, kv = _ints(case["q"]), _ints(case["kv"])
    row = hkv * (2 * D if case["type"] == "bf16" else D + 1)   # values and scales of one position, K or V
    if case["op"] == "write":
        return {"bytes": 2 * sum(q) * (hkv * 2 * D + row), "flops": 0}
    if case["op"] == "gather":
        counts = _ints(case["counts"])
        return {"bytes": 2 * (sum(counts) * row + len(kv) * case["k"] * (hkv * 2 * D + PAD)) + 4 * sum(counts), "flops": 0}
    if case["op"] == "sparse":
        counts = _ints(case["counts"])
        return {"bytes": sum(counts) * (2 * row + 4) + len(kv) * hq * (4 * D + 4), "flops": 4 * D * hq * sum(counts)}
    pairs = sum(t * n - t * (t - 1) // 2 for t, n in zip(q, kv))
    return {"bytes": 2 * sum(kv) * row + sum(q) * hq * (4 * D + 4), "flops": 4 * D * hq * pairs}


# ------------------------------------------------------- exact, in 64 bits
def _exact_pool(pages, kv_type):
    """float64 values [slots, Hkv, 128] of a pool, the codes taken apart by hand."""
    rows = pages.flatten(0, 1)
    if kv_type == "bf16":
        return rows[:, :rows.shape[1] - 8].double().unflatten(1, (-1, D))
    hkv = rows.shape[1] // D
    c = rows[:, :hkv * D].int().unflatten(1, (hkv, D))
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(2.0, (e - 10).double()))
    return mag * (1 - 2 * (c >> 7)) * torch.pow(2.0, rows[:, hkv * D:hkv * D + hkv].double() - 127)[..., None]


def _exact_rows(keys, values, queries, G, visible):
    """One kv head: keys and values [S, D], queries [n, G, D], visible [n, S]; float64."""
    w = torch.einsum("ngd,sd->ngs", queries, keys) / D ** 0.5
    w = torch.where(visible[:, None, :], w, torch.full((), float("-inf"), dtype=w.dtype, device=w.device))
    lse = torch.logsumexp(w, 2)
    w = torch.exp(w - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return torch.einsum("ngs,sd->ngd", w, values), lse


def exact(case, seed):
    s = prepare(case, seed)
    kind, hkv, hq, page = case["type"], case["hkv"], case["hq"], case["page"]
    G, dev = hq // hkv, s["q"].device
    slot_of = lambda b, j: s["table"][b].long()[torch.div(j, page, rounding_mode="floor")] * page + j % page  # noqa: E731
    if case["op"] == "write":
        # the pools after the call: the new values where they go (over their scale in E4M3 pools, before the
        # rounding to a code), what was there elsewhere; scale bytes are whole numbers
        w, res = hkv * D, []
        for pages, new in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])):
            after = pages[..., :w] if kind == "bf16" else pages[..., :w].view(torch.float8_e4m3fn)
            after = torch.nn.functional.pad(after.double(), (0, 8 if kind == "bf16" else 0))
            x = new.double()
            if kind != "bf16":
                peak = x.abs().amax(2, keepdim=True)
                power = torch.floor(torch.log2(peak / 448)) - 1       # log2 may be a bit off at powers of two
                for _ in range(3):
                    power = power + (448 * torch.pow(2.0, power) < peak)
                power = power.clamp(-118, 119)
                x = torch.where(peak > 0, x / torch.pow(2.0, power), x)   # a row of zeros is zeros at any scale
            at = 0
            for b, (T, S) in enumerate(zip(s["q_len"], s["kv"])):
                after.view(-1, after.shape[2])[slot_of(b, torch.arange(S - T, S, device=dev)), :w] = x[at:at + T].flatten(1)
                at += T
            res += [after] if kind == "bf16" else [after, None]
        return tuple(res)
    if case["op"] == "gather":
        out = []
        for pages in (s["k_pages"], s["v_pages"]):
            full = torch.zeros(len(s["kv"]), case["k"], hkv * D + 8, dtype=torch.float64, device=dev)
            vals = _exact_pool(pages, kind)
            for b, c in enumerate(_ints(case["counts"])):
                full[b, :c, :hkv * D] = vals[slot_of(b, s["idx"][b, :c].long())].flatten(1)
            out.append(full)
        return tuple(out)
    n_out = s["q"].shape[0]
    out = torch.zeros(n_out, hkv, G, D, dtype=torch.float64, device=dev)
    lse = torch.full((n_out, hkv, G), float("-inf"), dtype=torch.float64, device=dev)
    q = s["q"].double().unflatten(1, (hkv, G))
    at = 0
    for b, S in enumerate(s["kv"]):
        T = s["q_len"][b] if case["op"] == "attn" else 1
        if case["op"] == "attn":
            pos = torch.arange(S, device=dev)
        else:
            pos = s["idx"][b, :_ints(case["counts"])[b]].long()
        where = slot_of(b, pos)
        if pos.numel():
            lanes = [_exact_pool(p.flatten(0, 1)[where][None], kind) for p in (s["k_pages"], s["v_pages"])]
            step = max(1, (1 << 29) // (G * pos.numel()))
            for h in range(hkv):
                for t in range(0, T, step):
                    u = torch.arange(t, min(T, t + step), device=dev)
                    seen = pos[None] <= (S - T + u)[:, None] if case["op"] == "attn" else pos[None] >= 0
                    o, l = _exact_rows(lanes[0][:, h], lanes[1][:, h], q[at + u, h], G, seen)
                    out[at + u, h], lse[at + u, h] = o, l
        at += T
    return out.flatten(1, 2), lse.flatten(1, 2)
