"""What the ragged and paged attention operators are measured on: the cases, their plain forms and their exact values.

Four operators, one `op` each in a case:
  prompt  attention over packed sequences of different lengths, grouped heads, forward (output and log-sum-exp)
  train   the same with its gradients: forward, then backward
  paged   attention of the newest tokens of every sequence (one, or a chunk) over a cache kept in pages
  append  writing new keys and values into the pages of that cache
A case names its sequence lengths as text ("8192,77,1"); `new` gives the number of new tokens of each sequence.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _ints(text):
    return [int(x) for x in text.split(",")]


# 64 decoding sequences of one server: lengths spread from a few tokens to 8 K, none a round number
_DECODE_LENS = ",".join(str(1 + (i * i * 2027 + 977 * i + 11) % 8191) for i in range(64))
_ONES = ",".join(["1"] * 64)


def listed():
    return [
        # a batch of prompts of a grouped-head language model, one long, one a single token
        dict(name="prompt_dense_d128", op="prompt", dtype="bf16", kind="dense", mode="merged", l=1, c=1, H=32, Hkv=8, d=128, lens="8192,4096,2047,1531,130,1"),
        # the text-like workload of this repository (fixed pattern, merged heads, l = 128, c = 8), packed without padding
        dict(name="prompt_fixed_merged", op="prompt", dtype="bf16", kind="fixed", mode="merged", l=128, c=8, H=8, Hkv=8, d=64, lens="12288,9001,2999"),
        # a few short prompts: latency
        dict(name="prompt_strided_short", op="prompt", dtype="f16", kind="strided", mode="split", l=16, c=1, H=8, Hkv=2, d=64, lens="37,256,5,1"),
        # one training step's attention of a grouped-head model on packed documents
        dict(name="train_dense_d128", op="train", dtype="bf16", kind="dense", mode="merged", l=1, c=1, H=32, Hkv=8, d=128, lens="4096,2531,1024,541"),
        # the image-like stride (one row of 64 x 3 values), both index sets in every head, packed rasters
        dict(name="train_strided_merged", op="train", dtype="bf16", kind="strided", mode="merged", l=192, c=1, H=8, Hkv=4, d=64, lens="12288,6211"),
        # the small float32 workload of this repository
        dict(name="train_f32_small", op="train", dtype="f32", kind="strided", mode="split", l=16, c=1, H=2, Hkv=2, d=32, lens="256"),
        # a server's decoding step: 64 sequences, one new token each
        dict(name="decode_dense_64", op="paged", dtype="bf16", kind="dense", mode="merged", l=1, c=1, H=32, Hkv=8, d=128, lens=_DECODE_LENS, new=_ONES, page=16),
        # one token of one long audio-like sequence (T = 65536, l = 256): latency
        dict(name="decode_strided_one", op="paged", dtype="bf16", kind="strided", mode="merged", l=256, c=1, H=8, Hkv=8, d=64, lens="65536", new="1", page=64),
        # chunked prefill: chunks of new tokens, and one decoding sequence, behind long contexts
        dict(name="chunk_dense_d128", op="paged", dtype="bf16", kind="dense", mode="merged", l=1, c=1, H=32, Hkv=8, d=128, lens="32768,8192,4097,20000", new="512,512,333,1", page=64),
        # chunks of the text-like pattern over a cache
        dict(name="chunk_fixed_merged", op="paged", dtype="f16", kind="fixed", mode="merged", l=128, c=8, H=8, Hkv=8, d=64, lens="12288,9000", new="1024,700", page=48),
        # the cache write of a decoding step: latency
        dict(name="append_decode_64", op="append", dtype="bf16", kind="dense", mode="merged", l=1, c=1, H=32, Hkv=8, d=128, lens=_DECODE_LENS, new=_ONES, page=16),
        # the cache write of a prefill chunk
        dict(name="append_chunk", op="append", dtype="bf16", kind="dense", mode="merged", l=1, c=1, H=32, Hkv=8, d=128, lens="32768,8192,16391,20000", new="8192,8192,16391,4096", page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "train", "paged", "append"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"] if op != "append" else ["bf16", "f16"])
    kind = rng.choice(["dense", "strided", "fixed"])
    mode = rng.choice(["split", "merged"])
    l = 1 if kind == "dense" else _log_int(rng, 4, 512)
    c = rng.randint(1, max(1, min(l // 2, 32))) if kind == "fixed" else 1
    d = rng.choice([32, 64]) if dtype == "f32" else rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    case = dict(op=op, dtype=dtype, kind=kind, mode=mode, l=l, c=c, H=Hkv * G, Hkv=Hkv, d=d)
    if op in ("prompt", "train"):
        lens = [_log_int(rng, 1, 1024 if dtype == "f32" else 8192) for _ in range(rng.randint(1, 8))]
        limit = (1 << 25) if dtype == "f32" else (1 << 30) if op == "prompt" else (1 << 29)  # squares times heads
        while sum(n * n for n in lens) * Hkv * G > limit:
            k = lens.index(max(lens))
            lens[k] = lens[k] * 2 // 3
        return dict(case, lens=",".join(map(str, lens)))
    S = _log_int(rng, 1, 64)
    lens = [_log_int(rng, 1, 2048 if dtype == "f32" else 32768) for _ in range(S)]
    chunk = rng.random() < 0.5
    new = [min(n, _log_int(rng, 1, 64 if dtype == "f32" else 1024)) if chunk else 1 for n in lens]
    while max(lens) * S * Hkv * d > (1 << 28) or max(lens) * max(new) * S * Hkv * G > ((1 << 25) if dtype == "f32" else (1 << 31)):
        lens = [max(1, n * 2 // 3) for n in lens]
        new = [min(n, max(1, m * 4 // 5)) for n, m in zip(lens, new)]
    return dict(case, lens=",".join(map(str, lens)), new=",".join(map(str, new)), page=rng.choice([1, 16, 16, 20, 64, 128]))


# ---- what a user's program has in hand ------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    lens = _ints(case["lens"])

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = dict(case=case, lens=lens, scale=d ** -0.5)
    if case["op"] in ("prompt", "train"):
        total = sum(lens)
        s.update(q=randn(total, H, d), k=randn(total, Hkv, d), v=randn(total, Hkv, d), max_len=max(lens))
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        if case["op"] == "train":
            s["dout"] = randn(total, H, d)
    else:
        new, page = _ints(case["new"]), case["page"]
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = order[at:at + m]
            at += m
        s.update(k_cache=randn(pages, page, Hkv, d), v_cache=randn(pages, page, Hkv, d), table=table,
                 max_q=max(new), max_kv=max(lens), new=new)
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if case["op"] == "paged":
            s["q"] = randn(sum(new), H, d)
        else:
            s.update(k=randn(sum(new), Hkv, d), v=randn(sum(new), Hkv, d))
    if own:
        import factorized_sparse_self_b200 as st
        s["pattern"] = st.st_pattern(case["kind"], case["mode"], case["l"], case["c"])
    return s


# ---- one pass ---------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        import factorized_sparse_self_b200 as st
        if op == "prompt":
            return st.st_packed_attn_fwd(s["pattern"], s["q"], s["k"], s["v"], s["cu"], s["max_len"])
        if op == "train":
            o, lse = st.st_packed_attn_fwd(s["pattern"], s["q"], s["k"], s["v"], s["cu"], s["max_len"])
            dq, dk, dv = st.st_packed_attn_bwd(s["pattern"], s["q"], s["k"], s["v"], o, lse, s["dout"], s["cu"],
                                               s["max_len"])
            return o, dq, dk, dv
        if op == "paged":
            return st.st_paged_attn(s["pattern"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"],
                                    s["max_q"], s["max_kv"])
        st.st_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"])
        return s["k_cache"], s["v_cache"]
    if op == "prompt":
        return _plain_prompt(s)
    if op == "train":
        return _plain_train(s)
    if op == "paged":
        return _plain_paged(s)
    return _plain_append(s)


def _keeps(case, i, j):
    """Which keys (positions j) each query (position i) may attend, for even and for odd heads: [..., 2]."""
    l, c = case["l"], case["c"]
    causal = j <= i
    if case["kind"] == "dense":
        return torch.stack([causal, causal], -1)
    if case["kind"] == "strided":
        first, second = causal & (i - j <= l), causal & ((i - j) % l == 0)
    else:
        first, second = causal & (i // l == j // l), causal & (j % l >= l - c)
    if case["mode"] == "merged":
        first = second = first | second
    return torch.stack([first, second], -1)


def _softmax(scores, keeps):
    """Weights, and log of their sum: rows that keep nothing have weights of zero and a log of -inf."""
    scores = scores.masked_fill(~keeps, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(scores - top)
    total = w.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    return w / torch.where(total == 0, torch.ones_like(total), total), lse


def _plain_one(s, a, b):
    """One packed sequence, all heads at once: queries, keys, values in 32 bits, weights [Hkv, G, n, n] and their lse."""
    case = s["case"]
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    q = s["q"][a:b].float().view(b - a, Hkv, H // Hkv, d).permute(1, 2, 0, 3)
    k, v = (s[x][a:b].float().permute(1, 0, 2).unsqueeze(1) for x in ("k", "v"))
    p = torch.arange(b - a, device=q.device)
    keeps = _keeps(case, p[:, None], p[None, :])
    keeps = keeps[..., torch.arange(H, device=q.device) % 2].permute(2, 0, 1).view(Hkv, H // Hkv, b - a, b - a) \
        if case["mode"] == "split" and case["kind"] != "dense" else keeps[..., 0]
    w, lse = _softmax((q @ k.transpose(-1, -2)) * s["scale"], keeps)
    return q, k, v, w, lse


def _rows(x):
    """[Hkv, G, n, d] as [n, H, d]."""
    return x.permute(2, 0, 1, 3).reshape(x.shape[2], -1, x.shape[3])


def _plain_prompt(s):
    o, lse, a = [], [], 0
    for n in s["lens"]:
        q, k, v, w, m = _plain_one(s, a, a + n)
        o.append(_rows(w @ v).to(s["q"].dtype))
        lse.append(m.permute(2, 0, 1).reshape(n, -1))
        del q, k, v, w, m
        a += n
    return torch.cat(o), torch.cat(lse)


def _plain_train(s):
    got, a, dt = [], 0, s["q"].dtype
    for n in s["lens"]:
        q, k, v, w, _ = _plain_one(s, a, a + n)
        o = w @ v
        do = s["dout"][a:a + n].float().view(n, k.shape[0], -1, q.shape[-1]).permute(1, 2, 0, 3)
        dv = (w.transpose(-1, -2) @ do).sum(1)
        ds = w * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) * s["scale"]
        dk = (ds.transpose(-1, -2) @ q).sum(1)
        got.append((_rows(o).to(dt), _rows(ds @ k).to(dt), dk.permute(1, 0, 2).to(dt), dv.permute(1, 0, 2).to(dt)))
        del q, k, v, w, o, do, ds
        a += n
    return tuple(torch.cat(x) for x in zip(*got))


def _plain_paged(s):
    case = s["case"]
    H, Hkv, d, page = case["H"], case["Hkv"], case["d"], case["page"]
    S, G = len(s["lens"]), case["H"] // case["Hkv"]
    dev, max_q, max_kv = s["q"].device, s["max_q"], s["max_kv"]
    table = s["table"].clamp(min=0).long()
    j = torch.arange(max_kv, device=dev)
    page_of, slot = table[:, j // page], (j % page).expand(S, -1)
    k = s["k_cache"][page_of, slot].float().permute(0, 2, 1, 3).unsqueeze(2)  # [S, Hkv, 1, max_kv, d]
    v = s["v_cache"][page_of, slot].float().permute(0, 2, 1, 3).unsqueeze(2)
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    t = torch.arange(max_q, device=dev)
    new = cu[1:] - cu[:-1]
    real = t[None, :] < new[:, None]  # [S, max_q]
    row = torch.where(real, cu[:-1, None] + t[None, :], torch.zeros_like(t)[None, :])
    pos = kv[:, None] - new[:, None] + t[None, :]
    q = s["q"][row].float().view(S, max_q, Hkv, G, d).permute(0, 2, 3, 1, 4)  # [S, Hkv, G, max_q, d]
    keeps = _keeps(case, pos[:, :, None], j[None, None, :])  # [S, max_q, max_kv, 2]
    if case["mode"] == "split" and case["kind"] != "dense":
        keeps = keeps[..., torch.arange(H, device=dev) % 2].permute(0, 3, 1, 2).reshape(S, Hkv, G, max_q, max_kv)
    else:
        keeps = keeps[..., 0][:, None, None]
    w, lse = _softmax((q @ k.transpose(-1, -2)) * s["scale"], keeps)
    o = (w @ v).permute(0, 3, 1, 2, 4).reshape(S, max_q, H, d)[real]
    return o.to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(S, max_q, H)[real]


def _plain_append(s):
    page, cu = s["case"]["page"], s["cu"].long()
    row = torch.arange(s["k"].shape[0], device=s["k"].device)
    seq = torch.searchsorted(cu[1:], row, right=True)
    pos = s["kv_lens"].long()[seq] - cu[1:][seq] + row
    at = (s["table"][seq, pos // page].long(), pos % page)
    s["k_cache"][at] = s["k"]
    s["v_cache"][at] = s["v"]
    return s["k_cache"], s["v_cache"]


# ---- what a pass cannot do without ---------------------------------------------------


def _live(case, pos, cls):
    """Keys that a query at each of the positions `pos` attends, for heads of the class cls (0 even, 1 odd)."""
    l, c, kind = case["l"], case["c"], case["kind"]
    if kind == "dense":
        return pos + 1
    if kind == "strided":
        near, far = np.minimum(pos, l) + 1, pos // l + 1
        both = near + np.maximum(0, pos // l - 1)
    else:
        inside = np.maximum(0, pos % l + 1 - (l - c))
        near, far = pos % l + 1, pos // l * c + inside
        both = near + pos // l * c
    return both if case["mode"] == "merged" else far if cls else near


def _touched(case, first, end, cls):
    """How many keys any query at the positions first..end-1 attends."""
    l, c, kind = case["l"], case["c"], case["kind"]
    j = np.arange(end)
    if kind == "dense":
        return end
    if kind == "strided":
        near = j >= first - l
        seen = np.zeros(l, bool)
        seen[np.arange(first, min(end, first + l)) % l] = True
        far = seen[j % l]
    else:
        near, far = j >= first // l * l, j % l >= l - c
    if case["mode"] == "merged":
        return int((near | far).sum())
    return int(((near | far) if cls == 2 else far if cls else near).sum())


def work(case):
    H, Hkv, d, op = case["H"], case["Hkv"], case["d"], case["op"]
    es = 4 if case["dtype"] == "f32" else 2
    lens = _ints(case["lens"])
    new = _ints(case["new"]) if op in ("paged", "append") else lens
    if op == "append":
        return {"bytes": 4.0 * sum(new) * Hkv * d * es, "flops": 0.0}
    heads = [(H + 1) // 2, H // 2]
    pairs = sum(heads[x] * int(_live(case, np.arange(n - m, n, dtype=np.int64), x).sum()) for n, m in zip(lens, new) for x in (0, 1))
    rows = sum(new)
    q_bytes, lse_bytes = rows * H * d * es, rows * H * 4
    if op == "paged":
        G = H // Hkv
        keys = sum(_touched(case, n - m, n, 2 if G > 1 else h % 2) for n, m in zip(lens, new) for h in range(Hkv))
        return {"bytes": float(2 * q_bytes + lse_bytes + 2 * keys * d * es), "flops": 4.0 * d * pairs}
    kv_bytes = rows * Hkv * d * es
    fwd = 2 * q_bytes + 2 * kv_bytes + lse_bytes
    if op == "prompt":
        return {"bytes": float(fwd), "flops": 4.0 * d * pairs}
    # the backward pass reads q, k, v, o, dout, lse and writes dq, dk, dv; it forms the scores once more
    return {"bytes": float(fwd + 4 * q_bytes + 4 * kv_bytes + lse_bytes), "flops": 14.0 * d * pairs}


# ---- the definition in 64 bits ---------------------------------------------------------


def _sets(case, i0, n, parity):
    """Index sets as a table of truth values [n - i0, n]: queries i0..n-1, keys 0..n-1, built from bands, blocks and residues."""
    l, c, kind = case["l"], case["c"], case["kind"]
    ones = torch.ones(n - i0, n, dtype=torch.bool, device="cuda")
    past = torch.tril(ones, i0)
    if kind == "dense":
        return past
    key = torch.arange(n, device="cuda")
    query = key[i0:]
    if kind == "strided":
        sets = [torch.triu(past, i0 - l), past & torch.eq((query % l)[:, None], (key % l)[None])]
    else:
        block = torch.div(key, l, rounding_mode="floor")
        inside = key - block * l
        sets = [past & torch.eq(block[i0:, None], block[None]), past & (inside > l - c - 1)[None]]
    return sets[0] | sets[1] if case["mode"] == "merged" else sets[parity]


def _exact_head(case, q, k, v, i0, parity):
    """One head in float64: o, lse of queries i0.. (rows of q) over all keys."""
    s = torch.einsum("id,jd->ij", q, k) / float(case["d"]) ** 0.5
    s = s.masked_fill(~_sets(case, i0, k.shape[0], parity), float("-inf"))
    lse = torch.logsumexp(s, 1)
    none = torch.isneginf(lse)
    p = torch.exp(s - lse.masked_fill(none, 0.0)[:, None])
    return p @ v, lse


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, H, Hkv, d = case["op"], case["H"], case["Hkv"], case["d"]
    G = H // Hkv
    lens = s["lens"]
    if op == "append":
        k, v = s["k_cache"].double().cpu().numpy(), s["v_cache"].double().cpu().numpy()
        table, kn, vn = s["table"].cpu().numpy(), s["k"].double().cpu().numpy(), s["v"].double().cpu().numpy()
        r = 0
        for i, (n, m) in enumerate(zip(lens, s["new"])):
            for p in range(n - m, n):
                k[table[i, p // case["page"]], p % case["page"]] = kn[r]
                v[table[i, p // case["page"]], p % case["page"]] = vn[r]
                r += 1
        return torch.from_numpy(k), torch.from_numpy(v)
    if op == "paged":
        o, lse = torch.zeros(sum(s["new"]), H, d, dtype=torch.float64, device="cuda"), torch.zeros(sum(s["new"]), H, dtype=torch.float64, device="cuda")
        a = 0
        for i, (n, m) in enumerate(zip(lens, s["new"])):
            use = s["table"][i, :-(-n // case["page"])].long()
            k, v = (s[x][use].reshape(-1, Hkv, d)[:n].double() for x in ("k_cache", "v_cache"))
            for h in range(H):
                o[a:a + m, h], lse[a:a + m, h] = _exact_head(case, s["q"][a:a + m, h].double(), k[:, h // G], v[:, h // G], n - m, h % 2)
            a += m
        return o, lse
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    a = 0
    for n in lens:
        for h in range(H):
            x = [t[a:a + n, u].detach().requires_grad_(op == "train") for t, u in ((q, h), (k, h // G), (v, h // G))]
            y, m = _exact_head(case, *x, 0, h % 2)
            o[a:a + n, h], lse[a:a + n, h] = y.detach(), m.detach()
            if op == "train":  # the gradients come from differentiating the definition
                gq, gk, gv = torch.autograd.grad(y, x, s["dout"][a:a + n, h].double())
                dq[a:a + n, h] = gq
                dk[a:a + n, h // G] += gk
                dv[a:a + n, h // G] += gv
        a += n
    return (o, dq, dk, dv) if op == "train" else (o, lse)
