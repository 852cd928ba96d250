"""What is measured of the prompt, draft-tree, append and sampling operators.

Four operators around the decode step (include/oda_serve.h), each as a user's program calls it:

  prompt   causal attention over packed prompts, S^F or S^L        oda_attend_full_prompt / _local_prompt
  tree     a tree of drafted tokens over the paged cache           oda_attend_full_tree
  append   rows of K and V into the pages of every layer           oda_append / oda_append_fp8
  sample   a token per row of logits from given uniform numbers    oda_sample

With `own` false, run() computes the plain forms from elementary torch operations; with `own`
true it makes the library's calls.  Head counts and contexts are those of the Qwen3-shaped
workloads (16 or 32 query heads, 8 KV heads of 128; 4 sinks, a window of 2048; pages of 16).
"""
import math

import numpy as np
import torch

own = False

PAGE, D = 16, 128
SINKS, WINDOW = 4, 2048
SCALE = 1.0 / math.sqrt(D)
BLOCK8 = 4224          # bytes of one fp8 page block (one page, one KV head)
INF = float("inf")


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of chat turns admitted together: latency, ragged lengths, rows behind the last
        {"name": "prompt_chat_b8", "op": "prompt", "set": "full", "n": 8, "lo": 5, "hi": 400,
         "hq": 16, "hkv": 8, "behind": 3},
        # documents of different lengths packed into one call
        {"name": "prompt_ragged_b5", "op": "prompt", "set": "full", "n": 5, "lo": 700, "hi": 3900,
         "hq": 16, "hkv": 8, "behind": 0},
        # one long document, 8B-shaped heads
        {"name": "prompt_8k", "op": "prompt", "set": "full", "n": 1, "lo": 8192, "hi": 8192,
         "hq": 32, "hkv": 8, "behind": 0},
        # the same document read through the local set (the method's local pass over a prompt)
        {"name": "prompt_8k_local", "op": "prompt", "set": "local", "n": 1, "lo": 8191, "hi": 8191,
         "hq": 32, "hkv": 8, "behind": 1},
        # one request verifying a drafted chain of 5 over a short context: the smallest call
        {"name": "tree_b1_4k", "op": "tree", "b": 1, "lo": 4096, "hi": 4096, "nodes": 5, "chain": True,
         "hq": 16, "hkv": 8},
        # a divergent batch on shuffled pages with trees of up to 16 nodes
        {"name": "tree_b32_divergent", "op": "tree", "b": 32, "lo": 2000, "hi": 32768, "nodes": 16,
         "chain": False, "hq": 16, "hkv": 8},
        # long contexts with full 64-node trees: 256 query rows per KV head
        {"name": "tree_b4_128k", "op": "tree", "b": 4, "lo": 131072, "hi": 131072, "nodes": 64,
         "chain": False, "hq": 32, "hkv": 8},
        # a prompt's keys and values into the bf16 pages of 28 layers
        {"name": "append_prompt_bf16", "op": "append", "fmt": "bf16", "b": 2, "lo": 900, "hi": 2100,
         "ctx": 40, "layers": 28, "hkv": 8, "pick": False},
        # the accepted paths of a batch of draft trees into fp8 pages
        {"name": "append_accepted_fp8", "op": "append", "fmt": "fp8", "b": 32, "lo": 0, "hi": 6,
         "ctx": 3000, "layers": 36, "hkv": 8, "pick": True},
        # one request's next token
        {"name": "sample_b1", "op": "sample", "rows": 1, "vocab": 151936, "mix": "nucleus"},
        # a served batch, every row with its own settings
        {"name": "sample_b32", "op": "sample", "rows": 32, "vocab": 151936, "mix": "each"},
        # a token at every node of a batch's draft trees
        {"name": "sample_nodes_256", "op": "sample", "rows": 256, "vocab": 151936, "mix": "each"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "tree", "append", "sample"])
    hq = rng.choice([8, 16, 24, 32])
    if op == "prompt":
        n = rng.choice([1, 1, 2, 3, 5, 8])
        top = int(8192 * math.sqrt(16 / max(16, hq)) / n)
        hi = _log_int(rng, 40, top)
        return {"op": op, "set": rng.choice(["full", "local"]), "n": n, "lo": max(1, hi // rng.choice([1, 3, 20])),
                "hi": hi, "hq": hq, "hkv": 8, "behind": rng.choice([0, 1, 17])}
    if op == "tree":
        b = rng.choice([1, 2, 3, 4, 7, 8])
        hi = _log_int(rng, 30, 131072 // max(1, b // 4))
        return {"op": op, "b": b, "lo": max(0, hi // rng.choice([1, 2, 9]) - 3), "hi": hi,
                "nodes": _log_int(rng, 1, 64), "chain": rng.random() < 0.3, "hq": hq, "hkv": 8}
    if op == "append":
        b = rng.choice([1, 2, 5, 8])
        hi = _log_int(rng, 1, 4200 // b)
        return {"op": op, "fmt": rng.choice(["bf16", "fp8"]), "b": b, "lo": hi // 3, "hi": hi,
                "ctx": rng.randrange(0, 3000), "layers": rng.choice([1, 6, 28]), "hkv": rng.choice([4, 8]),
                "pick": rng.random() < 0.5}
    return {"op": op, "rows": _log_int(rng, 1, 256), "vocab": rng.choice([151936, 32000, 50257, 1000, 128256]) - rng.randrange(0, 9),
            "mix": rng.choice(["plain", "nucleus", "topk", "each"])}


# ------------------------------------------------------------------------------- inputs
def _lengths(case, gen, n):
    lo, hi = case["lo"], case["hi"]
    r = torch.rand(n, generator=gen)
    out = [lo + int(float(x) * (hi - lo + 1)) for x in r]
    out = [min(x, hi) for x in out]
    out[0] = hi
    return out


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _shape(case):
    """Lengths and cumulative rows of a case.  They are fixed by the case (so that work() can
    count them); the seed changes the values."""
    gen = torch.Generator().manual_seed(1234 + 7 * case["hi"] + case["lo"])
    n = case.get("n", case.get("b"))
    lens = _lengths(case, gen, n)
    return lens, _cu(lens)


def _trees(case, nb, gen):
    """Parents of the nodes of one sequence: a chain, or each node below a random earlier one."""
    if case["chain"]:
        return [i - 1 for i in range(nb)]
    r = torch.rand(max(nb, 1), generator=gen)
    return [-1 if i == 0 else int(float(r[i]) * (i + 1)) - 1 for i in range(nb)]


def _node_counts(case):
    gen = torch.Generator().manual_seed(4321 + case["nodes"])
    r = torch.rand(case["b"], generator=gen)
    n = [max(1, case["nodes"] - int(float(x) * case["nodes"] / 3)) for x in r]
    n[0] = case["nodes"]
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gh = torch.Generator().manual_seed(seed + 99)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["op"] == "prompt":
        _, cu = _shape(case)
        T, hq, hkv = cu[-1] + case["behind"], case["hq"], case["hkv"]
        # queries a little wider than unit variance: attention that is peaked here and flat there
        s.update(n=cu[-1], T=T, q=normal(T, hq, D) * 1.5, k=normal(T, hkv, D), v=normal(T, hkv, D),
                 cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                 out=torch.zeros(T, hq, D, dtype=torch.bfloat16, device="cuda"))
        s["ctx"] = _context(case["n"], hq, hkv, 1)
    elif case["op"] == "tree":
        lens, _ = _shape(case)
        b, hq, hkv = case["b"], case["hq"], case["hkv"]
        nodes = _node_counts(case)
        cu = _cu(nodes)
        pages = [(n + PAGE - 1) // PAGE for n in lens]
        mp, total = max(max(pages), 1), max(sum(pages), 1)
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        pt = torch.zeros(b, mp, dtype=torch.int32, device="cuda")
        at = 0
        for i, p in enumerate(pages):
            pt[i, :p] = perm[at:at + p]
            at += p
        N = cu[-1]
        s.update(L=max(lens), mp=mp, page_table=pt, k_pool=normal(total, hkv, PAGE, D), v_pool=normal(total, hkv, PAGE, D),
                 pos=torch.tensor([n + 1 for n in lens], dtype=torch.int32, device="cuda"), nodes=max(nodes), N=N,
                 cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                 parent=torch.tensor([p for n in nodes for p in _trees(case, n, gh)], dtype=torch.int32, device="cuda"),
                 q=normal(N, hq, D) * 1.5, k_new=normal(N, hkv, D), v_new=normal(N, hkv, D),
                 out=torch.zeros(N, hq, D, dtype=torch.bfloat16, device="cuda"))
        s["ctx"] = _context(b, hq, hkv, mp)
        s["layer"] = _layer(s["k_pool"], s["v_pool"])
    elif case["op"] == "append":
        lens, cu = _shape(case)
        b, hkv, L, ctx = case["b"], case["hkv"], case["layers"], case["ctx"]
        cap = [(ctx + n + PAGE - 1) // PAGE for n in lens]
        mp, total = max(max(cap), 1), max(sum(cap), 1)
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        pt = torch.zeros(b, mp, dtype=torch.int32, device="cuda")
        at = 0
        for i, p in enumerate(cap):
            pt[i, :p] = perm[at:at + p]
            at += p
        n_rows = cu[-1]
        n_stage = max(1, 2 * n_rows if case["pick"] else n_rows)
        s.update(n=n_rows, n_stage=n_stage, page_table=pt, mp=mp,
                 cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                 rows=torch.randint(0, n_stage, (n_rows,), generator=g, device="cuda", dtype=torch.int32) if case["pick"] else None,
                 pos=torch.full((b,), ctx + 1, dtype=torch.int32, device="cuda"),
                 pos_next=torch.zeros(b, dtype=torch.int32, device="cuda"),
                 k=normal(L, n_stage, hkv, D), v=normal(L, n_stage, hkv, D))
        s["ctx"] = _context(b, 2 * hkv, hkv, mp)
        if case["fmt"] == "bf16":
            s["k_pool"] = torch.zeros(L, total, hkv, PAGE, D, dtype=torch.bfloat16, device="cuda")
            s["v_pool"] = torch.zeros_like(s["k_pool"])
            s["layers"] = [_layer(s["k_pool"][i], s["v_pool"][i]) for i in range(L)]
        else:
            s["pool"] = torch.zeros(L, total, hkv, BLOCK8, dtype=torch.uint8, device="cuda")
            s["layers"] = [_layer8(s["pool"][i]) for i in range(L)]
    else:
        rows, vocab = case["rows"], case["vocab"]
        # an output distribution's look: a wide body and a handful of tokens well above it
        x = normal(rows, vocab, dtype=torch.float32) * 2.5
        up = torch.rand(rows, vocab, generator=g, device="cuda")
        x += torch.where(up < 40.0 / vocab, up * (14.0 * vocab / 40.0), 0.0)
        t = torch.ones(rows, device="cuda")
        kk = torch.zeros(rows, dtype=torch.int32, device="cuda")
        pp = torch.ones(rows, device="cuda")
        mm = torch.zeros(rows, device="cuda")
        r = torch.arange(rows, device="cuda")
        u01 = torch.rand(4, rows, generator=g, device="cuda")
        if case["mix"] in ("nucleus", "each"):
            t = 0.6 + 0.6 * u01[0]
            pp = 0.8 + 0.19 * u01[1]
        if case["mix"] == "topk":
            kk = (1 + u01[2] * 200).to(torch.int32)
        if case["mix"] == "each":
            kk = torch.where(r % 3 == 0, (1 + u01[2] * 100).to(torch.int32), kk)
            mm = torch.where(r % 4 == 1, 0.02 + 0.1 * u01[3], mm)
            pp = torch.where(r % 5 == 4, torch.ones_like(pp), pp)
            t = torch.where(r % 16 == 7, torch.zeros_like(t), t)     # greedy rows
        s.update(logits=x, temperature=t, top_k=kk, top_p=pp, min_p=mm,
                 u=torch.rand(rows, generator=g, device="cuda"),
                 token=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                 prob=torch.zeros(rows, device="cuda"))
        s["ctx"] = _context(1, 16, 8, 1)
    return s


def _context(b, hq, hkv, max_pages):
    """The handle a program keeps; the plain forms need none."""
    if not own:
        return None
    from conditional_sparse_attention_b200 import oda
    return oda.oda_create(oda.make_config(b, hq, hkv, max_pages, 512, SINKS, WINDOW))


def _layer(k, v):
    if not own:
        return None
    from conditional_sparse_attention_b200 import oda
    return oda.kv_layer(k, v)


def _layer8(kv):
    if not own:
        return None
    from conditional_sparse_attention_b200 import oda
    return oda.kv8_layer(kv)


# ---------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"prompt": _plain_prompt, "tree": _plain_tree, "append": _plain_append,
            "sample": _plain_sample}[s["case"]["op"]](s)


def _run_own(s):
    from conditional_sparse_attention_b200 import oda
    c = s["case"]
    if c["op"] == "prompt":
        call = oda.oda_attend_full_prompt if c["set"] == "full" else oda.oda_attend_local_prompt
        call(s["ctx"], s["cu"], s["q"], s["k"], s["v"], s["out"])
        return s["out"]
    if c["op"] == "tree":
        oda.oda_attend_full_tree(s["ctx"], s["layer"], s["page_table"], s["pos"], None, s["cu"], s["parent"], s["q"],
                                 s["k_new"], s["v_new"], s["out"])
        return s["out"]
    if c["op"] == "append":
        call = oda.oda_append if c["fmt"] == "bf16" else oda.oda_append_fp8
        call(s["ctx"], s["layers"], s["page_table"], s["pos"], s["cu"], s["rows"], s["k"], s["v"], pos_next=s["pos_next"])
        return _append_outputs(s)
    oda.oda_sample(s["ctx"], s["logits"], s["u"], s["token"], temperature=s["temperature"], top_k=s["top_k"],
                   top_p=s["top_p"], min_p=s["min_p"], prob=s["prob"])
    return {"token": s["token"], "prob": s["prob"]}


def _append_outputs(s):
    if s["case"]["fmt"] == "bf16":
        return {"k": s["k_pool"], "v": s["v_pool"], "pos": s["pos_next"]}
    return {"codes": s["pool"][..., :4096].view(torch.float8_e4m3fn), "scales": s["pool"][..., 4096:].view(torch.float32),
            "pos": s["pos_next"]}


# ------------------------------------------------------------------------- plain forms
def _plain_prompt(s):
    c, n = s["case"], s["n"]
    hq, hkv = c["hq"], c["hkv"]
    g = hq // hkv
    q = s["q"][:n].float().view(n, hkv, g, D).permute(1, 2, 0, 3).reshape(hkv, g * n, D)
    k = s["k"][:n].float().permute(1, 2, 0)
    v = s["v"][:n].float().permute(1, 0, 2)
    at = torch.arange(n, device=q.device)
    seq = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    place = at - s["cu"].long()[seq]
    seen = (seq[:, None] == seq[None, :]) & (place[None, :] <= place[:, None])
    if c["set"] == "local":
        seen &= (place[None, :] < SINKS) | (place[None, :] > place[:, None] - WINDOW)
    x = torch.matmul(q * SCALE, k).view(hkv, g, n, n)
    x.masked_fill_(~seen, -INF)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1)
    o = torch.matmul(x.view(hkv, g * n, n), v).view(hkv, g, n, D) / total[..., None]
    s["out"][:n] = o.permute(2, 0, 1, 3).reshape(n, hq, D).to(torch.bfloat16)
    return s["out"]


def _plain_tree(s):
    c = s["case"]
    b, hq, hkv, M = c["b"], c["hq"], c["hkv"], s["nodes"]
    g = hq // hkv
    dev = s["q"].device
    cu = s["cu"].long()
    at = torch.arange(M, device=dev)
    there = at[None] < (cu[1:] - cu[:-1])[:, None]                       # [b, M]
    row = torch.where(there, cu[:-1, None] + at[None], 0)
    P = (s["L"] + PAGE - 1) // PAGE
    idx = s["page_table"][:, :P].long()
    kc = s["k_pool"][idx].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, P * PAGE, D)
    vc = s["v_pool"][idx].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, P * PAGE, D)
    q = (s["q"][row].float() * SCALE).view(b, M, hkv, g, D).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * M, D)
    kn = s["k_new"][row].float().permute(0, 2, 3, 1)
    vn = s["v_new"][row].float().permute(0, 2, 1, 3)
    par = s["parent"].long()[row]
    up = (par[:, :, None] == at[None, None, :]) & there[:, :, None]
    eye = torch.eye(M, device=dev)
    seen = (torch.matrix_power(eye + up.float(), 64) > 0) & there[:, None, :]   # ancestors and itself
    xc = torch.matmul(q, kc.transpose(2, 3)).view(b, hkv, g, M, P * PAGE)
    cached = torch.arange(P * PAGE, device=dev)[None] < (s["pos"].long() - 1)[:, None]
    xc.masked_fill_(~cached[:, None, None, None, :], -INF)
    xn = torch.matmul(q, kn).view(b, hkv, g, M, M).masked_fill(~seen[:, None, None], -INF)
    x = torch.cat([xc, xn], -1)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hkv, g * M, -1), torch.cat([vc, vn], 2)).view(b, hkv, g, M, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(b, M, hq, D).to(torch.bfloat16)
    s["out"][row[there]] = o[there]
    return s["out"]


def _append_places(s):
    """Staging row, page and slot of every appended row."""
    n = s["n"]
    at = torch.arange(n, device=s["pos"].device)
    seq = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    place = s["pos"].long()[seq] - 1 + at - s["cu"].long()[seq]
    row = s["rows"].long() if s["rows"] is not None else at
    return row, s["page_table"].long()[seq, place // PAGE], place % PAGE


def _plain_append(s):
    row, page, slot = _append_places(s)
    cu = s["cu"]
    if s["case"]["fmt"] == "bf16":
        s["k_pool"][:, page, :, slot] = s["k"][:, row].transpose(0, 1)
        s["v_pool"][:, page, :, slot] = s["v"][:, row].transpose(0, 1)
    else:
        dev = row.device
        d = torch.arange(D, device=dev)
        head = torch.arange(s["case"]["hkv"], device=dev)
        # K: 16-value chunk k of token j at chunk place k ^ (j & 7); V: transposed, token j at slot
        k_at = slot[:, None] * 128 + ((d // 16)[None] ^ (slot & 7)[:, None]) * 16 + (d % 16)[None]
        v_slot = 4 * ((slot & 7) // 2) + 2 * (slot // 8) + slot % 2
        v_at = 2048 + 16 * d[None] + v_slot[:, None]
        pool = s["pool"]
        scales = pool[..., 4096:].view(torch.float32)
        codes, sc = _plain_codes(s["k"][:, row])
        pool[:, page[:, None, None], head[None, :, None], k_at[:, None, :]] = codes
        scales[:, page[:, None], head[None], slot[:, None]] = sc
        codes, sc = _plain_codes(s["v"][:, row])
        pool[:, page[:, None, None], head[None, :, None], v_at[:, None, :]] = codes
        scales[:, page[:, None], head[None], 16 + slot[:, None]] = sc
    torch.add(s["pos"], cu[1:] - cu[:-1], out=s["pos_next"])
    return _append_outputs(s)


def _plain_codes(x):
    x = x.float()
    top = x.abs().amax(-1)
    sc = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return (x / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), sc


def _plain_sample(s):
    l = s["logits"].double()
    rows, vocab = l.shape
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    z = (l - l.amax(-1, keepdim=True)) / torch.where(greedy, 1.0, t)
    w, order = torch.sort(z, dim=-1, descending=True, stable=True)
    w = w.exp()
    rank = torch.arange(vocab, device=l.device)[None]
    k = s["top_k"].long()[:, None]
    k = torch.where((k <= 0) | (k > vocab), vocab, k)
    k = torch.where(greedy, 1, k)
    w = torch.where(rank < k, w, 0.0)
    p = s["top_p"].double()[:, None]
    before = w.cumsum(-1) - w
    keep = (rank < k) & ((before < p * w.sum(-1, keepdim=True)) | (p >= 1) | (rank == 0))
    keep &= w >= s["min_p"].double()[:, None]
    mass = torch.zeros_like(l).scatter_(1, order, torch.where(keep, w, 0.0))
    sums = mass.cumsum(-1)
    token = (sums <= s["u"].double()[:, None] * sums[:, -1:]).sum(-1)
    s["token"].copy_(token)
    s["prob"].copy_((mass.gather(1, token[:, None]) / sums[:, -1:])[:, 0])
    return {"token": s["token"], "prob": s["prob"]}


# --------------------------------------------------------------------------------- work
def _attended(n, kind):
    """Pairs (row, place) that a causal sequence of n rows reads."""
    if kind == "full" or n <= WINDOW:
        return n * (n + 1) // 2
    m = n - WINDOW                                        # rows whose window has left place 0
    return WINDOW * (WINDOW + 1) // 2 + m * WINDOW + sum(min(SINKS, i) for i in range(1, min(m, SINKS) + 1)) + max(0, m - SINKS) * SINKS


def work(case):
    if case["op"] == "prompt":
        lens, cu = _shape(case)
        pairs = sum(_attended(n, case["set"]) for n in lens)
        return {"bytes": cu[-1] * D * 2 * 2 * (case["hq"] + case["hkv"]), "flops": 4 * D * case["hq"] * pairs}
    if case["op"] == "tree":
        lens, _ = _shape(case)
        nodes = _node_counts(case)
        kv = sum(n + m for n, m in zip(lens, nodes)) * case["hkv"] * D * 2 * 2
        rows = sum(nodes) * case["hq"] * D * 2 * 2
        return {"bytes": kv + rows, "flops": 4 * D * case["hq"] * sum((n + 1) * m for n, m in zip(lens, nodes))}
    if case["op"] == "append":
        _, cu = _shape(case)
        vals = 2 * case["layers"] * cu[-1] * case["hkv"]      # rows of 128 values, K and V
        return {"bytes": vals * (256 + (256 if case["fmt"] == "bf16" else 132)) + 16 * case["b"], "flops": 0}
    return {"bytes": 4 * case["rows"] * case["vocab"], "flops": 10 * case["rows"] * case["vocab"]}


# -------------------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "tree": _exact_tree, "append": _exact_append, "sample": _exact_sample}[case["op"]](s)


def _softmax_rows(q, k, v, ok):
    x = torch.where(ok, (q @ k.T) / math.sqrt(D), -INF)
    x = torch.exp(x - x.max(-1, keepdim=True).values)
    return (x @ v) / x.sum(-1, keepdim=True)


def _exact_prompt(s):
    c = s["case"]
    cu = s["cu"].tolist()
    out = s["out"].double()
    for i in range(len(cu) - 1):
        a, e = cu[i], cu[i + 1]
        for lo in range(a, e, 2048):                          # rows lo..hi-1 of sequence i
            hi = min(lo + 2048, e)
            t = torch.arange(lo - a, hi - a, device="cuda")[:, None]
            j = torch.arange(hi - a, device="cuda")[None]
            ok = j <= t
            if c["set"] == "local":
                ok = ok & ((j < SINKS) | (t - j < WINDOW))
            for h in range(c["hq"]):
                kv = h // (c["hq"] // c["hkv"])
                out[lo:hi, h] = _softmax_rows(s["q"][lo:hi, h].double(), s["k"][a:hi, kv].double(), s["v"][a:hi, kv].double(), ok)
    return out


def _exact_tree(s):
    c = s["case"]
    cu, parent, pos, pt = s["cu"].tolist(), s["parent"].tolist(), s["pos"].tolist(), s["page_table"].long()
    g = c["hq"] // c["hkv"]
    out = s["out"].double()
    for b in range(c["b"]):
        a, e, n = cu[b], cu[b + 1], pos[b] - 1
        ok = torch.zeros(e - a, n + e - a, dtype=torch.bool)
        ok[:, :n] = True
        for i in range(e - a):
            j = i
            while j >= 0:
                ok[i, n + j] = True
                j = parent[a + j]
        ok = ok.cuda()
        pages = pt[b, :(n + PAGE - 1) // PAGE]
        for kv in range(c["hkv"]):
            k = torch.cat([s["k_pool"][pages, kv].reshape(-1, D)[:n], s["k_new"][a:e, kv]]).double()
            v = torch.cat([s["v_pool"][pages, kv].reshape(-1, D)[:n], s["v_new"][a:e, kv]]).double()
            for h in range(kv * g, kv * g + g):
                out[a:e, h] = _softmax_rows(s["q"][a:e, h].double(), k, v, ok)
    return out


def _exact_append(s):
    c = s["case"]
    cu, pos, pt = s["cu"].tolist(), s["pos"].tolist(), s["page_table"].tolist()
    rows = s["rows"].tolist() if s["rows"] is not None else list(range(s["n"]))
    src, page, slot = [], [], []
    for b in range(c["b"]):
        for i in range(cu[b], cu[b + 1]):
            p = pos[b] - 1 + i - cu[b]
            src.append(rows[i])
            page.append(pt[b][p // PAGE])
            slot.append(p % PAGE)
    nxt = torch.tensor([pos[b] + cu[b + 1] - cu[b] for b in range(c["b"])], dtype=torch.int32)
    if c["fmt"] == "bf16":
        k, v = s["k_pool"], s["v_pool"]
        for layer in range(c["layers"]):
            k[layer][page, :, slot] = s["k"][layer][src]
            v[layer][page, :, slot] = s["v"][layer][src]
        return {"k": k, "v": v, "pos": nxt}
    L, total, hkv = s["pool"].shape[:3]
    codes = np.zeros((L, total, hkv, 4096))
    scales = np.zeros((L, total, hkv, 32))
    page, slot = np.array(page, np.int64), np.array(slot, np.int64)
    for which, x in ((0, s["k"]), (1, s["v"])):
        x = x[:, src].double().cpu().numpy()
        top = np.abs(x).max(-1)
        sc = np.where(top > 0, top / 448.0, 1.0)
        y = _e4m3(x / sc[..., None])
        for d in range(D):
            if which == 0:
                at = 128 * slot + 16 * ((d // 16) ^ (slot % 8)) + d % 16
            else:
                at = 2048 + 16 * d + np.array([[0, 1, 4, 5, 8, 9, 12, 13, 2, 3, 6, 7, 10, 11, 14, 15][j] for j in slot], np.int64)
            for h in range(hkv):
                codes[:, page, h, at] = y[:, :, h, d]
        for h in range(hkv):
            scales[:, page, h, 16 * which + slot] = sc[:, :, h]
    return {"codes": codes, "scales": scales, "pos": nxt}


def _e4m3(x):
    """Nearest value with 3 bits of fraction, exponents down to 2^-6 (then steps of 2^-9)."""
    a = np.abs(x)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 1e-30))), -6) - 3)
    return np.sign(x) * np.minimum(np.round(a / step) * step, 448.0)


def _exact_sample(s):
    l = s["logits"].cpu().numpy().astype(np.float64)
    get = {n: s[n].cpu().numpy().astype(np.float64) for n in ("temperature", "top_k", "top_p", "min_p", "u")}
    token, prob = [], []
    for r in range(l.shape[0]):
        t, k, p = get["temperature"][r], int(get["top_k"][r]), get["top_p"][r]
        if t <= 0:
            token.append(int(np.argmax(l[r])))
            prob.append(1.0)
            continue
        w = np.exp((l[r] - l[r].max()) / t)
        order = np.argsort(-l[r], kind="stable")
        if 0 < k < len(order):
            order = order[:k]
        if p < 1:
            sums = np.cumsum(w[order])
            order = order[:int(np.searchsorted(sums, p * sums[-1])) + 1]
        order = np.sort(order[w[order] >= get["min_p"][r]])
        sums = np.cumsum(w[order])
        i = int(np.searchsorted(sums, get["u"][r] * sums[-1], side="right"))
        token.append(int(order[i]))
        prob.append(w[order[i]] / sums[-1])
    return {"token": np.array(token, np.int32), "prob": np.array(prob)}
