"""Performance cases of the operators over a paged cache in 8 bits, and of positions with several axes.

The cache's pools hold E4M3 codes with one power of two (an E8M0 byte) for each token and group:

* ``append``: new tokens into their pages, rotated by their positions and quantised (``bits`` 8), or into a bf16 cache
  (``bits`` 16) with positions of several axes (time, height, width);
* ``read``: tokens of the cache back as bf16 rows;
* ``sparse``: the MSA layer for new tokens over such a cache, selection and attention;
* ``dense``: full attention for new tokens over it, a batch whose sequences may share their first pages.

``run`` computes them in elementary torch operations, or through the library where ``own`` is set.
"""
import math

import torch

own = False

BLOCK = 128  # tokens per page
D = 128      # head dim
E = 64       # index dim
AXES = 3     # time, height, width


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one user, one new token (the latency floor of a decode step)
        dict(name="append8_1", op="append", bits=8, axes=0, S=1, rows=1, ragged=False, Hq=32, G=8, length=8192, prefix=0,
             rot=128, rot_idx=64, interleaved=False, fused=False, index=True),
        # a decode step of a full batch behind one 120K-token system prompt, positions of three axes, fused projection
        dict(name="append8_b64_axes", op="append", bits=8, axes=AXES, S=64, rows=1, ragged=False, Hq=32, G=8,
             length=131000, prefix=960, rot=128, rot_idx=64, interleaved=False, fused=True, index=True),
        # prompts of up to 8191 tokens written at once (prefill)
        dict(name="append8_prefill", op="append", bits=8, axes=0, S=4, rows=8191, ragged=False, Hq=32, G=8, length=8191,
             prefix=0, rot=128, rot_idx=64, interleaved=False, fused=False, index=True),
        # drafted tokens behind images, a layer without an index branch, partial interleaved rotation, a bf16 cache
        dict(name="append_axes_draft", op="append", bits=16, axes=AXES, S=37, rows=7, ragged=True, Hq=64, G=8,
             length=5003, prefix=0, rot=64, rot_idx=0, interleaved=True, fused=True, index=False),
        # the prompts of two videos into a bf16 cache
        dict(name="append_axes_video", op="append", bits=16, axes=AXES, S=2, rows=6001, ragged=False, Hq=32, G=8,
             length=6001, prefix=0, rot=128, rot_idx=64, interleaved=False, fused=False, index=True),
        # a short chat's tokens for the training calls, which take bf16 rows
        dict(name="read8_short", op="read", S=1, ragged=False, G=8, length=701, index=True),
        # a batch's cache for another step of the pipeline
        dict(name="read8_b8_t16k", op="read", S=8, ragged=True, G=8, length=16384, index=True),
        # one user decoding at 128K tokens
        dict(name="sparse8_1_t128k", op="sparse", S=1, rows=1, ragged=False, Hq=32, G=8, length=131072, k=16,
             shared=False),
        # a serving batch of ragged contexts up to 32K tokens
        dict(name="sparse8_b64_t32k", op="sparse", S=64, rows=1, ragged=True, Hq=32, G=8, length=32768, k=16,
             shared=False),
        # a handful of chats of their own
        dict(name="dense8_b16_t4k", op="dense", S=16, rows=1, ragged=True, Hq=32, G=8, prefix=0, suffix=4099),
        # a serving batch behind a 32K-token document
        dict(name="dense8_b64_p32k", op="dense", S=64, rows=1, ragged=True, Hq=32, G=8, prefix=256, suffix=2048),
        # drafted tokens, eight heads a group, odd suffixes
        dict(name="dense8_draft_p8k", op="dense", S=23, rows=5, ragged=True, Hq=64, G=8, prefix=64, suffix=1117),
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
        op = rng.choice(["append", "append", "read", "sparse", "dense", "dense"])
        G = rng.choice([1, 2, 4, 8])
        c = dict(op=op, S=_log_int(rng, 1, 128), ragged=rng.random() < 0.6, G=G)
        if op == "read":
            c.update(length=_log_int(rng, 1, 131072), index=rng.random() < 0.8)
        else:
            c.update(rows=1, Hq=G * rng.choice([1, 2, 4, 8]))
        if op == "append":
            c["rows"] = 1 if rng.random() < 0.4 else _log_int(rng, 2, 8191)
            c["prefix"] = 0 if rng.random() < 0.5 else _log_int(rng, 1, 960)
            c["length"] = c["prefix"] * BLOCK + c["rows"] + _log_int(rng, 1, 8000) - 1
            c["bits"] = rng.choice([8, 8, 16])
            c["axes"] = AXES if c["bits"] == 16 or rng.random() < 0.3 else 0
            c.update(rot=rng.choice([32, 64, 128]), rot_idx=rng.choice([0, 32, 64]), interleaved=rng.random() < 0.5,
                     fused=rng.random() < 0.5, index=rng.random() < 0.8)
        elif op == "sparse":
            c["rows"] = 1 if rng.random() < 0.6 else rng.randint(2, 6)
            c.update(length=_log_int(rng, 8, 524288), k=_log_int(rng, 1, 33), shared=rng.random() < 0.3)
            if c["S"] * c["length"] * G > (64 << 20) // 4:  # keep a state within a few GB
                continue
        elif op == "dense":
            c["rows"] = 1 if rng.random() < 0.6 else rng.randint(2, 8)
            c.update(prefix=0 if rng.random() < 0.5 else _log_int(rng, 1, 256), suffix=_log_int(rng, 8, 16384))
            if c["S"] * c["rows"] * c["suffix"] * G > (1 << 20):
                continue
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def _batch(case):
    """Rows and lengths (new rows included) of every sequence: whole numbers, from the case alone."""
    S, rows = case["S"], case.get("rows", 0)
    fixed = case.get("prefix", 0) * BLOCK
    longest = case["length"] if "length" in case else fixed + case["suffix"]
    count, lens = [], []
    for i in range(S):
        n = rows - (i * 5 % rows) if case["ragged"] and rows else rows
        if case["ragged"] and S > 4 and i % 11 == 7:
            n = 0  # an idle slot of the batch
        own_part = longest - fixed
        cut = ((i * 2654435761) % (1 << 32)) * (own_part // 2) >> 32 if case["ragged"] else 0
        count.append(n)
        lens.append(max(longest - cut, fixed + rows))
    pad = 2 if case["ragged"] else 0  # rows behind the last sequence, as a padded batch has
    return count, lens, pad


def work(case):
    count, lens, _ = _batch(case)
    G = case["G"]
    if case["op"] == "read":
        n = sum(lens)
        return {"bytes": n * (2 * G * (D + 1 + 2 * D) + ((E + 1 + 2 * E) if case["index"] else 0)) + 8 * case["S"],
                "flops": n * (2 * G * D + (E if case["index"] else 0))}
    Hq, n = case["Hq"], sum(count)
    if case["op"] == "append":
        token = 2 * G * (D + 1) if case["bits"] == 8 else 2 * G * D * 2  # a token's part of the cache
        row = 2 * Hq * D * 2 + 2 * G * D * 2 + token
        if case["index"]:
            row += (2 * G + 1) * E * 2 + ((E + 1) if case["bits"] == 8 else 2 * E)
        return {"bytes": n * (row + 4 + 4 * case["axes"]) + 8 * case["S"],
                "flops": n * (3 * ((Hq + G) * case["rot"] + ((G + 1) * case["rot_idx"] if case["index"] else 0))
                              + 2 * G * D)}
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
                nbytes += per_row[-1][0] * BLOCK * (E + 1)
                flops += sum(2 * E * G * own_ * BLOCK for own_, _ in per_row)
            tokens = [min(k - 1, own_) * BLOCK + see - own_ * BLOCK for own_, see in per_row]
            nbytes += min(sum(tokens), L) * G * 2 * (D + 1)
            flops += sum(4 * D * Hq * x for x in tokens)
        return {"bytes": nbytes, "flops": flops}
    fixed = case["prefix"] * BLOCK
    nbytes += fixed * G * 2 * (D + 1)
    for c, L in zip(count, lens):
        if c:
            nbytes += (L - fixed) * G * 2 * (D + 1)
            flops += sum(4 * D * Hq * (t + 1) for t in range(L - c, L))
    return {"bytes": nbytes, "flops": flops}


# ----------------------------------------------------------------- 8 bits
def _quantised(x):
    """E4M3 codes of x [..., dim] (fp32) and the E8M0 byte of each vector: the smallest power of two 2^e with
    max |x| <= 448 * 2^e, e in [-117, 120]. What is not finite becomes NaN and counts for nothing in the scale."""
    fine = x.isfinite()
    m, up = torch.frexp(torch.where(fine, x, 0.0).abs().amax(-1))  # the maximum is m * 2^up, m in [0.5, 1)
    e = torch.where(m > 0, up - 9 + (m > 0.875).int(), -117).clamp(-117, 120)
    code = torch.where(fine, torch.ldexp(x, -e[..., None]), math.nan).to(torch.float8_e4m3fn)
    return code, (e + 127).to(torch.uint8)


def _values(code, byte):
    """What codes [..., dim] and their bytes stand for, in fp32."""
    return torch.ldexp(code.float(), (byte.int() - 127)[..., None])


def _take(pool, *at):
    """Elements of an 8-bit pool."""
    return pool.view(torch.uint8)[at].view(pool.dtype)


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    count, lens, pad = _batch(case)
    S, G, op = case["S"], case["G"], case["op"]
    Hq, prefix, bits = case.get("Hq", G), case.get("prefix", 0), case.get("bits", 8)
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

    def pool(*shape, mean=False):
        """Random values in the cache's type, a few pages at a time; the bytes are None in 16 bits."""
        kind = torch.float8_e4m3fn if bits == 8 else torch.bfloat16
        data = torch.empty(num_pages, *shape, dtype=kind, device="cuda")
        byte = torch.empty(num_pages, *shape[:-1], dtype=torch.uint8, device="cuda") if bits == 8 else None
        for p in range(0, num_pages, 512):
            q = min(num_pages, p + 512)
            x = normal(q - p, *shape).float()
            if mean:
                x = x + 0.5 * normal(q - p, 1, shape[-1]).float()
            if bits == 8:
                data[p:q], byte[p:q] = _quantised(x)
            else:
                data[p:q] = x.to(kind)
        return data, byte

    K, K_exp = pool(G, BLOCK, D)
    V, V_exp = pool(G, BLOCK, D)
    index = case["index"] if "index" in case else op == "sparse" and not case["shared"]
    k_idx, k_idx_exp = pool(BLOCK, E, mean=True) if index else (None, None)
    st = dict(case=case, S=S, N=N, Hq=Hq, G=G, num_pages=num_pages, max_blocks=max_blocks, prefix=prefix, bits=bits, K=K,
              V=V, K_exp=K_exp, V_exp=V_exp, k_idx=k_idx, k_idx_exp=k_idx_exp, table=table,
              row_start=torch.tensor(starts, dtype=torch.int32, device="cuda"),
              seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    # the rows' sequences and positions, as a serving program's batch builder knows them
    if op == "read":
        out_start = [0]
        for L in lens:
            out_start.append(out_start[-1] + L)
        st["M"] = out_start[-1]
        st["out_start"] = torch.tensor(out_start, dtype=torch.int32, device="cuda")
        n = torch.tensor(lens, device="cuda")
        st["row_seq"] = torch.repeat_interleave(torch.arange(S, device="cuda"), n)
        st["row_pos"] = torch.arange(st["M"], device="cuda") - st["out_start"][:-1].long()[st["row_seq"]]
    else:
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
        st["positions"] = st["axis"] = st["axis_idx"] = None
        if case["axes"]:
            # images of 24 x 18 patches: a time for each, and the patch's line and column
            t = torch.zeros(N, dtype=torch.int64, device="cuda")
            t[:starts[-1]] = st["row_pos"]
            frame, patch = t // 432, t % 432
            st["positions"] = torch.stack([frame, frame + patch // 24, frame + patch % 24], dim=1).to(torch.int32)
            # pairs take turns between height and width, the slowest quarter is the time's
            def axis(m):
                i = torch.arange(m, device="cuda")
                return torch.where(i >= m - m // 4, 0, 1 + i % 2).to(torch.int32)

            st["axis"], st["axis_idx"] = axis(case["rot"] // 2), axis(case["rot_idx"] // 2 if index else 0)
        st["Q_out"] = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda")
        st["q_idx_out"] = torch.zeros(N, G, E, dtype=torch.bfloat16, device="cuda") if index else None
    elif op == "read":
        st["K_out"], st["V_out"] = (torch.zeros(st["M"], G, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        st["k_idx_out"] = torch.zeros(st["M"], E, dtype=torch.bfloat16, device="cuda") if index else None
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

        st["shape"] = msa.PagedShape(S=S, N=max(N, 1), Hq=Hq, G=G, num_pages=num_pages, max_blocks=max_blocks,
                                     k=case.get("k", 1), prefix_blocks=prefix if op == "dense" else 0)
        which = {"append": msa.MSA_WS_PAGED_APPEND, "read": msa.MSA_WS_PAGED_APPEND,
                 "sparse": msa.MSA_WS_PAGED_SPARSE_FP8, "dense": msa.MSA_WS_PAGED_DENSE_FP8}[op]
        if bits == 8:
            st["cache"] = msa.PagedCacheFp8(K, V, K_exp, V_exp, k_idx, k_idx_exp, table, st["row_start"], st["seq_len"])
        else:
            st["cache"] = msa.PagedCache(K, V, k_idx, table, st["row_start"], st["seq_len"])
        st["ws"] = msa.alloc_paged_workspace(st["shape"], which)
        if op == "append":
            st["rope"] = msa.Rope(st["freq"], st["freq_idx"] if index else None, interleaved=case["interleaved"],
                                  axis=st["axis"], axis_idx=st["axis_idx"] if index else None)
    return st


# ----------------------------------------------------------------- the operators
def run(st):
    op = st["case"]["op"]
    if own:
        import block_sparse_attention_scores_gb300 as msa

        if op == "append":
            x = st["new"]
            call = msa.msa_paged_append_fp8 if st["bits"] == 8 else msa.msa_paged_append
            call(st["shape"], st["cache"], st["rope"], x["K"], x["V"], x["k_idx"], x["Q"], x["q_idx"], st["Q_out"],
                 st["q_idx_out"], st["ws"], positions=st["positions"])
        elif op == "read":
            msa.msa_paged_read_fp8(st["shape"], st["cache"], None, st["out_start"], st["K_out"], st["V_out"],
                                   st["k_idx_out"], st["ws"])
        elif op == "sparse":
            msa.msa_paged_sparse_attn_fp8(st["shape"], st["cache"], st["Q"], st["q_idx"], st["block_idx"], st["O"],
                                          st["LSE"], st["ws"])
        else:
            msa.msa_paged_dense_attn_fp8(st["shape"], st["cache"], st["Q"], st["O"], st["LSE"], st["ws"])
    elif op == "append":
        _append(st)
    elif op == "read":
        _read(st)
    elif op == "sparse":
        _sparse(st)
    else:
        _dense(st)
    if op == "read":
        return {"K": st["K_out"], "V": st["V_out"], "k_idx": st["k_idx_out"]}
    if op == "append":
        out = {"Q": st["Q_out"], "K": st["K"], "V": st["V"]}
        if st["k_idx"] is not None:
            out.update(q_idx=st["q_idx_out"], k_idx=st["k_idx"])
        if st["bits"] == 8:  # the codes' powers of two
            for n in ("K_exp", "V_exp", "k_idx_exp"):
                if st[n] is not None:
                    out[n] = st[n].view(torch.float8_e8m0fnu)
        return out
    out = {"O": st["O"], "LSE": st["LSE"]}
    if op == "sparse" and not st["case"]["shared"]:
        out["block_idx"] = st["block_idx"]
    return out


def _rotated(x, where, freq, interleaved):
    """x [n, ..., dim] in fp32 with the first 2 len(freq) dims rotated by where [n, len(freq)] * freq; angles in 64 bits,
    the rest in 32."""
    rot = 2 * freq.numel()
    x = x.float()
    if rot == 0:
        return x
    ang = where.double() * freq.double()
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
    if st["positions"] is None:
        where, where_idx = pos[:, None], pos[:, None]
    else:
        where, where_idx = (st["positions"][:n][:, st[a].long()] for a in ("axis", "axis_idx"))
    page = st["table"][st["row_seq"], pos // BLOCK].long()
    slot = pos % BLOCK

    def put(name, at, x):
        if st["bits"] == 8:
            code, byte = _quantised(x)
            st[name].view(torch.uint8)[at] = code.view(torch.uint8)
            st[name + "_exp"][at] = byte
        else:
            st[name][at] = x.to(torch.bfloat16)

    put("K", (page, slice(None), slot), _rotated(new["K"][:n], where, f, how))
    put("V", (page, slice(None), slot), new["V"][:n].float())
    st["Q_out"][:n] = _rotated(new["Q"][:n], where, f, how).to(torch.bfloat16)
    if st["k_idx"] is not None:
        put("k_idx", (page, slot), _rotated(new["k_idx"][:n], where_idx, fi, how))
        st["q_idx_out"][:n] = _rotated(new["q_idx"][:n], where_idx, fi, how).to(torch.bfloat16)


def _read(st):
    page = st["table"][st["row_seq"], st["row_pos"] // BLOCK].long()
    slot = st["row_pos"] % BLOCK
    for name, at in (("K", (page, slice(None), slot)), ("V", (page, slice(None), slot)), ("k_idx", (page, slot))):
        if st[name] is not None:
            st[name + "_out"][:] = _values(_take(st[name], *at), st[name + "_exp"][at]).to(torch.bfloat16)


def _sparse(st):
    n, pos, G, k = st["row_pos"].numel(), st["row_pos"], st["G"], st["case"]["k"]
    hg = st["Hq"] // G
    own_block = pos // BLOCK
    table = st["table"].clamp(min=0).long()
    if not st["case"]["shared"]:
        # scores in 64 bits: a border between two blocks may be narrower than the rounding of 32
        keys = _values(_take(st["k_idx"], table), st["k_idx_exp"][table]).flatten(1, 2).double()[st["row_seq"]]
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
    K = _values(_take(st["K"], page, group), st["K_exp"][page, group]).flatten(2, 3)  # [n, G, k * 128, D]
    V = _values(_take(st["V"], page, group), st["V_exp"][page, group]).flatten(2, 3)
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
    own_pages = table[:, P:]                                                        # [S, pages]
    seq = st["row_seq"]
    K, V = (_values(_take(st[x], own_pages), st[x + "_exp"][own_pages]).transpose(1, 2).flatten(2, 3)[seq]
            for x in ("K", "V"))                                                    # [n, G, tokens, D]
    token = torch.arange(K.shape[2], device=q.device) + P * BLOCK
    s = (q @ K.transpose(2, 3)).masked_fill((token > pos[:, None])[:, None, None, :], -math.inf)
    # the shared pages, once for every row
    Kp, Vp = (_values(_take(st[x], table[0, :P]), st[x + "_exp"][table[0, :P]]).transpose(0, 1).flatten(1, 2)
              for x in ("K", "V"))                                                  # [G, tokens, D]
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
def _decoded(code, byte):
    """Values of E4M3 codes from their bits: (-1)^s 2^(x - 7) (1 + m / 8), 2^-6 m / 8 below, and the byte's power of two."""
    b = code.view(torch.uint8).long()
    x, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(x > 0, torch.exp2((x - 7).double()) * (1 + m / 8), m / 512)
    v = torch.where((b & 127) == 127, math.nan, torch.where(b >= 128, -v, v))
    return v * torch.exp2(byte.double() - 127).unsqueeze(-1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st, case)
    table, pos, seq = st["table"].tolist(), st["row_pos"].tolist(), st["row_seq"].tolist()
    G, n = st["G"], len(pos)
    if case["op"] == "read":
        line = torch.cat([st["table"][s, :-(-L // BLOCK)].long().repeat_interleave(BLOCK)[:L] * BLOCK
                          + torch.arange(L, device="cuda") % BLOCK for s, L in enumerate(_batch(case)[1])])
        out = {}
        for x in ("K", "V"):
            rows = [_decoded(st[x][:, g].reshape(-1, D)[line], st[x + "_exp"][:, g].reshape(-1)[line]) for g in range(G)]
            out[x] = torch.stack(rows, dim=1)
        out["k_idx"] = _decoded(st["k_idx"].reshape(-1, E)[line], st["k_idx_exp"].reshape(-1)[line]) if case["index"] else None
        return out
    hg = st["Hq"] // G
    O = torch.zeros(st["N"], st["Hq"], D, dtype=torch.float64, device="cuda")
    LSE = torch.zeros(st["N"], st["Hq"], dtype=torch.float64, device="cuda")
    chosen = st["block_idx"].clone() if case["op"] == "sparse" else None
    for r in range(n):
        t, pages = pos[r], table[seq[r]]
        last = t // BLOCK
        if case["op"] == "sparse" and not case["shared"]:
            at = torch.tensor(pages[:last] or [0], device="cuda")
            best = torch.einsum("ge,cje->gcj", st["q_idx"][r].double(), _decoded(_take(st["k_idx"], at), st["k_idx_exp"][at]))
            for g, line in enumerate(best.amax(2).tolist()):
                by = sorted(range(last), key=lambda c: (-line[c], c))[:case["k"] - 1]
                got = sorted(by + [last])
                chosen[r, g] = torch.tensor(got + [-1] * (case["k"] - len(got)), dtype=torch.int32, device="cuda")
        lists = chosen[r].tolist() if chosen is not None else [list(range(last + 1))] * G
        for g, ids in enumerate(lists):
            ids = [c for c in ids if c >= 0]
            at = torch.tensor([pages[c] for c in ids], device="cuda")
            token = (torch.tensor(ids, device="cuda")[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(-1)
            k, v = (_decoded(_take(st[x], at, g), st[x + "_exp"][at, g]).reshape(-1, D)[token <= t] for x in ("K", "V"))
            x = torch.einsum("hd,jd->hj", st["Q"][r, g * hg:(g + 1) * hg].double(), k) * D ** -0.5
            LSE[r, g * hg:(g + 1) * hg] = torch.logsumexp(x, 1)
            O[r, g * hg:(g + 1) * hg] = torch.einsum("hj,jd->hd", torch.softmax(x, 1), v)
    out = {"O": O, "LSE": LSE}
    if case["op"] == "sparse" and not case["shared"]:
        out["block_idx"] = chosen
    return out


def _exact_append(st, case):
    """Each pair as a complex number times exp(i * position * frequency); codes before their rounding."""
    n = st["row_pos"].numel()

    def turned(x, freq, axis):
        x = x[:n].double()
        m = freq.numel()
        if m == 0:
            return x
        i = torch.arange(m, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + m)
        z = torch.complex(x[..., first], x[..., second])
        if axis is None:
            phase = torch.outer(st["row_pos"].double(), freq.double())
        else:
            phase = st["positions"][:n].double().index_select(1, axis.long()) * freq.double()
        z = z * torch.polar(torch.ones_like(phase), phase).view([n] + [1] * (x.dim() - 2) + [m])
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    new = st["new"]
    where = st["table"][st["row_seq"], torch.div(st["row_pos"], BLOCK, rounding_mode="floor")].long() * BLOCK
    where += st["row_pos"] % BLOCK  # slot of the pool, all pages in a line

    def pool(p, rows, vectors):
        """The pool `p` with `rows` at its slots, in 64 bits; vectors: its last dim is a vector's."""
        p = p if vectors else p.unsqueeze(-1)
        line = p.double().movedim(-2, 1).flatten(0, 1)  # [pages * 128, (G,) dim]
        line[where] = rows if vectors else rows.unsqueeze(-1)
        line = line.unflatten(0, (-1, BLOCK)).movedim(1, -2)
        return (line if vectors else line.squeeze(-1)).contiguous()

    out = {"Q": torch.zeros(st["N"], st["Hq"], D, dtype=torch.float64, device="cuda")}
    out["Q"][:n] = turned(new["Q"], st["freq"], st["axis"])
    if st["k_idx"] is not None:
        out["q_idx"] = torch.zeros(st["N"], st["G"], E, dtype=torch.float64, device="cuda")
        out["q_idx"][:n] = turned(new["q_idx"], st["freq_idx"], st["axis_idx"])
    rows = {"K": turned(new["K"], st["freq"], st["axis"]), "V": new["V"][:n].double()}
    if st["k_idx"] is not None:
        rows["k_idx"] = turned(new["k_idx"], st["freq_idx"], st["axis_idx"])
    for name, x in rows.items():
        if case["bits"] == 8:
            up = torch.log2(x.abs().amax(-1) / 448).ceil().clamp(-117, 120)
            out[name] = pool(st[name], x * torch.exp2(-up)[..., None], True)
            out[name + "_exp"] = pool(torch.exp2(st[name + "_exp"].double() - 127), torch.exp2(up), False)
        else:
            out[name] = pool(st[name], x, True)
    return out
