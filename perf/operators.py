"""Performance cases of the paged-cache (serving) operators.

Three operators of ``block_sparse_attention_scores_gb300`` over one paged cache
(pages of 128 tokens, one page per KV block):

* ``append``: new tokens' K, V and index keys into their pages, position
  rotation on the way, queries rotated beside them;
* ``sparse``: the MSA layer for new tokens, the index branch's selection over
  the cached index keys and the exact attention over the selected pages;
* ``dense``: full attention for new tokens, a batch whose sequences share
  their first pages.

``run`` computes them in elementary torch operations, or through the library
where ``own`` is set.
"""
import math

import torch

own = False

BLOCK = 128  # tokens per page
D = 128      # head dim
E = 64       # index dim


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one user, one new token (the latency floor of a decode step)
        dict(name="append_1", op="append", S=1, rows=1, ragged=False, Hq=32, G=8, length=8192, prefix=0, rot=128,
             rot_idx=64, interleaved=False, fused=False, index=True),
        # a decode step of a full batch behind one 120K-token system prompt, inputs sliced from a fused projection
        dict(name="append_b64_far", op="append", S=64, rows=1, ragged=False, Hq=32, G=8, length=131000, prefix=960,
             rot=128, rot_idx=64, interleaved=False, fused=True, index=True),
        # several drafted tokens a sequence, ragged, a layer without an index branch, partial interleaved rotation
        dict(name="append_draft_ragged", op="append", S=37, rows=7, ragged=True, Hq=64, G=8, length=5003, prefix=0,
             rot=64, rot_idx=0, interleaved=True, fused=True, index=False),
        # prompts of up to 8191 tokens written at once (prefill)
        dict(name="append_prefill", op="append", S=4, rows=8191, ragged=False, Hq=32, G=8, length=8191, prefix=0,
             rot=128, rot_idx=64, interleaved=False, fused=False, index=True),
        # one user decoding at 128K tokens
        dict(name="sparse_1_t128k", op="sparse", S=1, rows=1, ragged=False, Hq=32, G=8, length=131072, k=16,
             shared=False),
        # a serving batch of ragged contexts up to 32K tokens
        dict(name="sparse_b64_t32k", op="sparse", S=64, rows=1, ragged=True, Hq=32, G=8, length=32768, k=16,
             shared=False),
        # two users at a million tokens: the index keys are most of what is read
        dict(name="sparse_b2_t1m", op="sparse", S=2, rows=1, ragged=False, Hq=16, G=4, length=1048575, k=16,
             shared=False),
        # a layer that reuses an earlier layer's selection (IndexShare), drafted tokens, short ragged contexts
        dict(name="sparse_shared_draft", op="sparse", S=19, rows=4, ragged=True, Hq=16, G=2, length=6007, k=9,
             shared=True),
        # a handful of short chats behind a 1K-token prompt
        dict(name="dense_b4_p1k", op="dense", S=4, rows=1, ragged=True, Hq=8, G=2, prefix=8, suffix=301),
        # a serving batch behind a 32K-token document
        dict(name="dense_b64_p32k", op="dense", S=64, rows=1, ragged=True, Hq=32, G=8, prefix=256, suffix=2048),
        # drafted tokens, eight heads a group, odd suffixes
        dict(name="dense_draft_p8k", op="dense", S=23, rows=5, ragged=True, Hq=64, G=8, prefix=64, suffix=1117),
        # many samples (two drafted tokens each) of one 128K-token prompt: tensor cores
        dict(name="dense_b128_p128k", op="dense", S=128, rows=2, ragged=False, Hq=32, G=8, prefix=1024, suffix=1000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        op = rng.choice(["append", "sparse", "dense"])
        G = rng.choice([1, 2, 4, 8])
        c = dict(op=op, S=_log_int(rng, 1, 128), rows=1, ragged=rng.random() < 0.6, Hq=G * rng.choice([1, 2, 4, 8]), G=G)
        if op == "append":
            c["rows"] = 1 if rng.random() < 0.4 else _log_int(rng, 2, 8191)
            c["prefix"] = 0 if rng.random() < 0.5 else _log_int(rng, 1, 960)
            c["length"] = c["prefix"] * BLOCK + c["rows"] + _log_int(rng, 1, 8000) - 1
            c.update(rot=rng.choice([32, 64, 128]), rot_idx=rng.choice([0, 32, 64]), interleaved=rng.random() < 0.5,
                     fused=rng.random() < 0.5, index=rng.random() < 0.8)
        elif op == "sparse":
            c["rows"] = 1 if rng.random() < 0.6 else rng.randint(2, 6)
            c.update(length=_log_int(rng, 8, 1048576), k=_log_int(rng, 1, 33), shared=rng.random() < 0.3)
            if c["S"] * c["length"] * G > (64 << 20) // 4:  # keep a state within a few GB
                continue
        else:
            c["rows"] = 1 if rng.random() < 0.5 else rng.randint(2, 8)
            c.update(prefix=0 if rng.random() < 0.15 else _log_int(rng, 1, 1024), suffix=_log_int(rng, 8, 4096))
            if c["S"] * c["rows"] * c["suffix"] * G > (1 << 20):
                continue
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def _batch(case):
    """Rows and lengths (new rows included) of every sequence: whole numbers, from the case alone."""
    S, rows = case["S"], case["rows"]
    fixed = case["prefix"] * BLOCK if "prefix" in case else 0
    longest = case["length"] if "length" in case else fixed + case["suffix"]
    count, lens = [], []
    for i in range(S):
        n = rows - (i * 5 % rows) if case["ragged"] else rows
        if case["ragged"] and S > 4 and i % 11 == 7:
            n = 0  # an idle slot of the batch
        own_part = longest - fixed
        cut = ((i * 2654435761) % (1 << 32)) * (own_part // 2) >> 32 if case["ragged"] else 0
        count.append(n)
        lens.append(max(longest - cut, fixed + rows))
    pad = 2 if case["ragged"] else 0  # rows behind the last sequence, as a padded batch has
    return count, lens, pad


def work(case):
    count, lens, pad = _batch(case)
    Hq, G = case["Hq"], case["G"]
    n = sum(count)
    if case["op"] == "append":
        row = 2 * (Hq + 2 * G) * D * 2 + (2 * (G + 1) * E * 2 if case["index"] else 0)
        return {"bytes": n * row + 8 * case["S"] + 4 * n,
                "flops": n * 3 * ((Hq + G) * case["rot"] + ((G + 1) * case["rot_idx"] if case["index"] else 0))}
    nbytes = 2 * n * Hq * D * 2 + 4 * n * Hq
    flops = 0
    if case["op"] == "sparse":
        k = case["k"]
        nbytes += 4 * n * G * k + (0 if case["shared"] else n * G * E * 2)
        for c, L in zip(count, lens):
            if not c:
                continue
            per_row = [(t // BLOCK, t + 1) for t in range(L - c, L)]
            if not case["shared"]:
                nbytes += per_row[-1][0] * BLOCK * E * 2
                flops += sum(2 * E * G * own_ * BLOCK for own_, _ in per_row)
            tokens = [min(k - 1, own_) * BLOCK + see - own_ * BLOCK for own_, see in per_row]
            nbytes += min(sum(tokens), L) * G * D * 4
            flops += sum(4 * D * Hq * x for x in tokens)
        return {"bytes": nbytes, "flops": flops}
    fixed = case["prefix"] * BLOCK
    nbytes += fixed * G * D * 4
    for c, L in zip(count, lens):
        if c:
            nbytes += (L - fixed) * G * D * 4
            flops += sum(4 * D * Hq * (t + 1) for t in range(L - c, L))
    return {"bytes": nbytes, "flops": flops}


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    count, lens, pad = _batch(case)
    S, Hq, G, op = case["S"], case["Hq"], case["G"], case["op"]
    prefix = case.get("prefix", 0)
    starts = [0]
    for c in count:
        starts.append(starts[-1] + c)
    N = starts[-1] + pad
    blocks = [-(-L // BLOCK) for L in lens]
    max_blocks = max(blocks)
    num_pages = prefix + sum(b - prefix for b in blocks) + 3
    order = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((S, max_blocks), -1, dtype=torch.int32, device="cuda")
    at = prefix
    for i, b in enumerate(blocks):
        table[i, :prefix] = order[:prefix]
        table[i, prefix:b] = order[at:at + b - prefix]
        at += b - prefix
    K, V = normal(num_pages, G, BLOCK, D), normal(num_pages, G, BLOCK, D)
    index = case["index"] if op == "append" else op == "sparse" and not case["shared"]
    k_idx = None
    if index:
        k_idx = (normal(num_pages, BLOCK, E).float() + 0.5 * normal(num_pages, 1, E).float()).to(torch.bfloat16)
    st = dict(case=case, S=S, N=N, Hq=Hq, G=G, num_pages=num_pages, max_blocks=max_blocks, prefix=prefix, K=K, V=V,
              k_idx=k_idx, table=table, row_start=torch.tensor(starts, dtype=torch.int32, device="cuda"),
              seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    # the rows' sequences and positions, as a serving program's batch builder knows them
    st["row_seq"] = torch.tensor([i for i, c in enumerate(count) for _ in range(c)], dtype=torch.long, device="cuda")
    st["row_pos"] = torch.tensor([L - c + j for c, L in zip(count, lens) for j in range(c)], dtype=torch.long,
                                 device="cuda")
    if op == "append":
        widths = [Hq * D, G * D, G * D] + ([G * E, E] if index else [])
        if case["fused"]:
            parts = list(normal(N, sum(widths)).split(widths, dim=1))
        else:
            parts = [normal(N, w) for w in widths]
        shapes = [(Hq, D), (G, D), (G, D), (G, E), (E,)]
        parts = [p.unflatten(1, s) for p, s in zip(parts, shapes)] + [None, None]
        st["new"] = dict(zip(("Q", "K", "V", "q_idx", "k_idx"), parts))

        def freq(dim):
            return 1.0 / 500000.0 ** (torch.arange(0, dim, 2, device="cuda", dtype=torch.float32) / max(dim, 1))

        st["freq"], st["freq_idx"] = freq(case["rot"]), freq(case["rot_idx"] if index else 0)
        st["Q_out"] = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda")
        st["q_idx_out"] = torch.zeros(N, G, E, dtype=torch.bfloat16, device="cuda") if index else None
    else:
        st["Q"] = normal(N, Hq, D)
        st["O"] = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda")
        st["LSE"] = torch.zeros(N, Hq, dtype=torch.float32, device="cuda")
    if op == "sparse":
        k = case["k"]
        st["block_idx"] = torch.full((N, G, k), -1, dtype=torch.int32, device="cuda")
        st["q_idx"] = None
        if case["shared"]:  # an earlier layer's selection: the own block and k - 1 earlier ones
            own_block = (st["row_pos"] // BLOCK)[:, None, None]
            noise = torch.rand(starts[-1], G, max_blocks, generator=gen, device="cuda")
            ids = torch.arange(max_blocks, device="cuda")
            noise = torch.where(ids < own_block, noise, torch.where(ids == own_block, 2.0, -1.0))
            val, pick = noise.topk(min(k, max_blocks), dim=2)
            pick = torch.where(val >= 0, pick, max_blocks).sort(dim=2).values
            st["block_idx"][:starts[-1], :, :pick.shape[2]] = torch.where(pick < max_blocks, pick, -1).to(torch.int32)
        else:
            st["q_idx"] = normal(N, G, E)
    if own:
        import block_sparse_attention_scores_gb300 as msa

        which = {"append": msa.MSA_WS_PAGED_APPEND, "sparse": msa.MSA_WS_PAGED_SPARSE,
                 "dense": msa.MSA_WS_PAGED_DENSE}[op]
        st["shape"] = msa.PagedShape(S=S, N=N, Hq=Hq, G=G, num_pages=num_pages, max_blocks=max_blocks,
                                     k=case.get("k", 1), prefix_blocks=prefix if op == "dense" else 0)
        st["cache"] = msa.PagedCache(K, V, k_idx, table, st["row_start"], st["seq_len"])
        st["ws"] = msa.alloc_paged_workspace(st["shape"], which)
        if op == "append":
            st["rope"] = msa.Rope(st["freq"], st["freq_idx"] if index else None, interleaved=case["interleaved"])
    return st


# ----------------------------------------------------------------- the operators
def run(st):
    op = st["case"]["op"]
    if own:
        import block_sparse_attention_scores_gb300 as msa

        if op == "append":
            x = st["new"]
            msa.msa_paged_append(st["shape"], st["cache"], st["rope"], x["K"], x["V"], x["k_idx"], x["Q"], x["q_idx"],
                                 st["Q_out"], st["q_idx_out"], st["ws"])
        elif op == "sparse":
            msa.msa_paged_sparse_attn(st["shape"], st["cache"], st["Q"], st["q_idx"], st["block_idx"], st["O"],
                                      st["LSE"], st["ws"])
        else:
            msa.msa_paged_dense_attn(st["shape"], st["cache"], st["Q"], st["O"], st["LSE"], st["ws"])
    elif op == "append":
        _append(st)
    elif op == "sparse":
        _sparse(st)
    else:
        _dense(st)
    if op == "append":
        out = {"Q": st["Q_out"], "K": st["K"], "V": st["V"]}
        if st["k_idx"] is not None:
            out.update(q_idx=st["q_idx_out"], k_idx=st["k_idx"])
        return out
    out = {"O": st["O"], "LSE": st["LSE"]}
    if op == "sparse" and not st["case"]["shared"]:
        out["block_idx"] = st["block_idx"]
    return out


def _rotated(x, pos, freq, interleaved):
    """x [n, ..., dim] with the first 2 len(freq) dims rotated by pos * freq; angles in 64 bits, the rest in 32."""
    rot = 2 * freq.numel()
    x = x.float()
    if rot == 0:
        return x
    ang = pos.double()[:, None] * freq.double()
    ang = ang.reshape([ang.shape[0]] + [1] * (x.dim() - 2) + [rot // 2])
    c, s = ang.cos().float(), ang.sin().float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _append(st):
    n, pos, how = st["row_pos"].numel(), st["row_pos"], st["case"]["interleaved"]
    new, f, fi = st["new"], st["freq"], st["freq_idx"]
    page = st["table"][st["row_seq"], pos // BLOCK].long()
    slot = pos % BLOCK
    st["K"][page, :, slot] = _rotated(new["K"][:n], pos, f, how).to(torch.bfloat16)
    st["V"][page, :, slot] = new["V"][:n]
    st["Q_out"][:n] = _rotated(new["Q"][:n], pos, f, how).to(torch.bfloat16)
    if st["k_idx"] is not None:
        st["k_idx"][page, slot] = _rotated(new["k_idx"][:n], pos, fi, how).to(torch.bfloat16)
        st["q_idx_out"][:n] = _rotated(new["q_idx"][:n], pos, fi, how).to(torch.bfloat16)


def _sparse(st):
    n, pos, G, k = st["row_pos"].numel(), st["row_pos"], st["G"], st["case"]["k"]
    hg = st["Hq"] // G
    own_block = pos // BLOCK
    table = st["table"].clamp(min=0).long()
    if not st["case"]["shared"]:
        # scores in 64 bits: a border between two blocks may be narrower than the rounding of 32
        keys = st["k_idx"][table].flatten(1, 2).double()[st["row_seq"]]             # [n, tokens, E]
        score = st["q_idx"][:n].double() @ keys.transpose(1, 2)                     # [n, G, tokens]
        pooled = score.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf).unflatten(2, (-1, BLOCK)).amax(3)
        ids = torch.arange(pooled.shape[2], device=pooled.device)
        pooled = torch.where(ids < own_block[:, None, None], pooled, -math.inf)
        pooled = torch.where(ids == own_block[:, None, None], math.inf, pooled)
        best = pooled.sort(dim=2, descending=True, stable=True).indices[:, :, :k]   # equal scores: the lower id first
        best = torch.where(best <= own_block[:, None, None], best, st["max_blocks"]).sort(dim=2).values
        st["block_idx"][:n, :, :best.shape[2]] = torch.where(best < st["max_blocks"], best, -1).to(torch.int32)
    pick = st["block_idx"][:n].long()                                               # [n, G, k]
    page = table[st["row_seq"][:, None, None], pick.clamp(min=0)]
    group = torch.arange(G, device=pick.device)[None, :, None]
    K = st["K"][page, group].float().flatten(2, 3)                                  # [n, G, k * 128, D]
    V = st["V"][page, group].float().flatten(2, 3)
    token = (pick[..., None] * BLOCK + torch.arange(BLOCK, device=pick.device)).flatten(2)
    seen = (pick >= 0).repeat_interleave(BLOCK, dim=2) & (token <= pos[:, None, None])
    s = st["Q"][:n].float().unflatten(1, (G, hg)) @ K.transpose(2, 3) / math.sqrt(D)
    s = s.masked_fill(~seen[:, :, None, :], -math.inf)
    top = s.amax(3, keepdim=True)
    p = (s - top).exp()
    total = p.sum(3, keepdim=True)
    st["O"][:n] = ((p @ V) / total).flatten(1, 2).to(torch.bfloat16)
    st["LSE"][:n] = (top + total.log()).flatten(1)


def _dense(st):
    n, pos, G, P = st["row_pos"].numel(), st["row_pos"], st["G"], st["prefix"]
    hg = st["Hq"] // G
    q = st["Q"][:n].float().unflatten(1, (G, hg)) / math.sqrt(D)                    # [n, G, hg, D]
    table = st["table"].clamp(min=0).long()
    own_pages = table[st["row_seq"], P:]                                            # [n, pages]
    K = st["K"][own_pages].float().transpose(1, 2).flatten(2, 3)                    # [n, G, tokens, D]
    V = st["V"][own_pages].float().transpose(1, 2).flatten(2, 3)
    token = torch.arange(K.shape[2], device=q.device) + P * BLOCK
    s = (q @ K.transpose(2, 3)).masked_fill((token > pos[:, None])[:, None, None, :], -math.inf)
    # the shared pages, once for every row
    Kp = st["K"][table[0, :P]].float().transpose(0, 1).flatten(1, 2)                # [G, tokens, D]
    Vp = st["V"][table[0, :P]].float().transpose(0, 1).flatten(1, 2)
    sp = q.transpose(0, 1).flatten(1, 2) @ Kp.transpose(1, 2)                       # [G, n * hg, tokens]
    sp = sp.unflatten(1, (n, hg)).transpose(0, 1)
    top = s.amax(3, keepdim=True)
    top = torch.maximum(top, sp.amax(3, keepdim=True)) if P else top
    p, pp = (s - top).exp(), (sp - top).exp()
    total = p.sum(3, keepdim=True) + pp.sum(3, keepdim=True)
    o = p @ V + (pp.transpose(0, 1).flatten(1, 2) @ Vp).unflatten(1, (n, hg)).transpose(0, 1)
    st["O"][:n] = (o / total).flatten(1, 2).to(torch.bfloat16)
    st["LSE"][:n] = (top + total.log()).flatten(1)


# ----------------------------------------------------------------- in 64 bits, row by row
def exact(case, seed):
    st = prepare(case, seed)
    table, pos, seq = st["table"].tolist(), st["row_pos"].tolist(), st["row_seq"].tolist()
    if case["op"] == "append":
        return _exact_append(st, case)
    G, hg, n = st["G"], st["Hq"] // st["G"], len(pos)
    O = torch.zeros(st["N"], st["Hq"], D, dtype=torch.float64, device="cuda")
    LSE = torch.zeros(st["N"], st["Hq"], dtype=torch.float64, device="cuda")
    chosen = st["block_idx"].clone() if case["op"] == "sparse" else None
    for r in range(n):
        t, pages = pos[r], table[seq[r]]
        last = t // BLOCK
        if case["op"] == "dense":
            at = torch.tensor(pages[:last + 1], device="cuda")
            for g0 in range(G):
                q = st["Q"][r, g0 * hg:(g0 + 1) * hg].double()
                k, v = st["K"][at, g0].reshape(-1, D)[:t + 1].double(), st["V"][at, g0].reshape(-1, D)[:t + 1].double()
                x = torch.einsum("hd,jd->hj", q, k) * D ** -0.5
                LSE[r, g0 * hg:(g0 + 1) * hg] = torch.logsumexp(x, 1)
                O[r, g0 * hg:(g0 + 1) * hg] = torch.einsum("hj,jd->hd", torch.softmax(x, 1), v)
            continue
        if not case["shared"]:
            keys = st["k_idx"][torch.tensor(pages[:last] or [0], device="cuda")].double()
            best = torch.einsum("ge,cje->gcj", st["q_idx"][r].double(), keys).amax(2)
            for g0, line in enumerate(best.tolist()):
                line = line[:last]
                by = sorted(range(last), key=lambda c: (-line[c], c))[:case["k"] - 1]
                got = sorted(by + [last])
                chosen[r, g0] = torch.tensor(got + [-1] * (case["k"] - len(got)), dtype=torch.int32, device="cuda")
        for g0, ids in enumerate(chosen[r].tolist()):
            ids = [c for c in ids if c >= 0]
            at = torch.tensor([pages[c] for c in ids], device="cuda")
            token = (torch.tensor(ids, device="cuda")[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(-1)
            k, v = st["K"][at, g0].reshape(-1, D)[token <= t].double(), st["V"][at, g0].reshape(-1, D)[token <= t].double()
            x = torch.einsum("hd,jd->hj", st["Q"][r, g0 * hg:(g0 + 1) * hg].double(), k) * D ** -0.5
            LSE[r, g0 * hg:(g0 + 1) * hg] = torch.logsumexp(x, 1)
            O[r, g0 * hg:(g0 + 1) * hg] = torch.einsum("hj,jd->hd", torch.softmax(x, 1), v)
    out = {"O": O, "LSE": LSE}
    if case["op"] == "sparse" and not case["shared"]:
        out["block_idx"] = chosen
    return out


def _exact_append(st, case):
    """Each pair as a complex number times exp(i * position * frequency)."""
    n, pos = st["row_pos"].numel(), st["row_pos"].double()

    def turned(x, freq):
        x = x[:n].double()
        m = freq.numel()
        if m == 0:
            return x
        i = torch.arange(m, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + m)
        z = torch.complex(x[..., first], x[..., second])
        phase = torch.outer(pos, freq.double())
        z = z * torch.polar(torch.ones_like(phase), phase).view([n] + [1] * (x.dim() - 2) + [m])
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    new = st["new"]
    where = st["table"][st["row_seq"], torch.div(st["row_pos"], BLOCK, rounding_mode="floor")].long() * BLOCK
    where += st["row_pos"] % BLOCK  # slot of the pool, all pages in a line

    def pool(p, rows):
        line = p.double().movedim(-2, 1).flatten(0, 1)  # [pages * 128, (G,) dim]
        line[where] = rows
        return line.unflatten(0, (-1, BLOCK)).movedim(1, -2).contiguous()

    out = {"Q": torch.zeros(st["N"], st["Hq"], D, dtype=torch.float64, device="cuda")}
    out["Q"][:n] = turned(new["Q"], st["freq"])
    out["K"] = pool(st["K"], turned(new["K"], st["freq"]))
    out["V"] = pool(st["V"], new["V"][:n].double())
    if st["k_idx"] is not None:
        out["q_idx"] = torch.zeros(st["N"], st["G"], E, dtype=torch.float64, device="cuda")
        out["q_idx"][:n] = turned(new["q_idx"], st["freq_idx"])
        out["k_idx"] = pool(st["k_idx"], turned(new["k_idx"], st["freq_idx"]))
    return out
