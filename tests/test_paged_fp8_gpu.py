"""The operators over a paged cache in 8 bits, and positions with several axes, on the GPU against their 64-bit forms
(tests/paged_ref.py and tests/paged_fp8_ref.py, bounds derived there)."""
import numpy as np
import pytest

import paged_fp8_ref as ref8
import paged_ref as ref

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__

    __graft_entry__.build_library()
    import block_sparse_attention_scores_gb300 as m

    return m


def _freq(rot, base=500000.0):
    import torch

    return 1.0 / base ** (torch.arange(0, rot, 2, dtype=torch.float32) / max(rot, 1))


def _check_padding(b, O, LSE, bi=None):
    assert bool((O[b.n:] == 5.0).all()) and bool((LSE[b.n:] == 5.0).all())
    assert bi is None or (bi[b.n:] == -7).all()


# ----------------------------------------------------------------- append
APPEND = {
    "one": dict(counts=[1], lens=[1], Hq=8, G=2, rot=128, rot_idx=64),
    "page_ends": dict(counts=[1, 1, 1, 2, 128, 129, 3], lens=[127, 128, 129, 129, 256, 300, 3], Hq=4, G=4, rot=64, rot_idx=32),
    "idle_and_padding": dict(counts=[0, 5, 0, 0, 1, 0], lens=[7, 133, 0, 128, 500, 64], pad=3, Hq=16, G=2, rot=128, rot_idx=64),
    "interleaved": dict(counts=[3, 130], lens=[1000, 130], Hq=8, G=1, rot=128, rot_idx=64, interleaved=True),
    "partial_interleaved": dict(counts=[9], lens=[200], Hq=6, G=3, rot=48, rot_idx=16, interleaved=True),
    "partial_strided": dict(counts=[9, 4], lens=[200, 77], Hq=6, G=3, rot=96, rot_idx=48, fused=True),
    "no_rotation": dict(counts=[6], lens=[6], Hq=2, G=2, rot=0, rot_idx=0, fused=True),
    "no_index": dict(counts=[2, 2], lens=[140, 129], Hq=64, G=8, rot=128, rot_idx=0, index=False),
    "no_index_one_group": dict(counts=[2, 2], lens=[140, 129], Hq=1, G=1, rot=128, rot_idx=0, index=False),
    "many_sequences": dict(counts=[1] * 70, lens=list(range(1, 141, 2)), Hq=2, G=1, rot=32, rot_idx=64),
    "blocks_of_rows": dict(counts=[2433, 0, 37], lens=[2600, 5, 37], pad=2, Hq=2, G=1, rot=128, rot_idx=64, fused=True),
    "blocks_of_rows_g3": dict(counts=[1500], lens=[1500], Hq=3, G=3, rot=64, rot_idx=16, interleaved=True),
}


def _new_rows(b, seed=5, fused=False):
    """Rows to append, with vectors that are hard to quantise among them."""
    import torch

    gen = torch.Generator().manual_seed(seed)
    index = b.k_idx is not None
    widths = [b.Hq * 128, b.G * 128, b.G * 128] + ([b.G * 64, 64] if index else [])
    lines = torch.randn(b.N, sum(widths) + 8, generator=gen).to(torch.bfloat16).cuda()[:, :sum(widths)]
    parts = list(lines.split(widths, dim=1)) if fused else [x.contiguous() for x in lines.split(widths, dim=1)]
    x = dict(zip(("Q", "K", "V", "q_idx", "k_idx"),
                 [p.unflatten(1, s) for p, s in zip(parts, [(b.Hq, 128), (b.G, 128), (b.G, 128), (b.G, 64), (64,)])]))
    hard = [0.0, 1e30, 1e-30, 1e38, 1e-38, 1e-39]
    for r in range(min(b.n, len(hard))):
        for n in ("K", "V", "k_idx"):
            if n in x:
                x[n][r] = (x[n][r].float() * hard[r]).clamp(-1.5e38, 1.5e38).to(torch.bfloat16)
    return x


def _turned(x, r, where, freq, how):
    """Row r of x in 64 bits, pair i turned by where[i] * freq[i]; and |a| + |b| of each value's pair."""
    import torch

    return ref.rotated(x[r].double(), torch.as_tensor(where, dtype=torch.float64), freq, how)


def _check_vector(code, byte, y, mag, exactly, what):
    """Codes and byte of one vector against its values in 64 bits, which the kernel has within 2^-20 mag: the byte is that
    of its largest magnitude (either of two where that is so near to the border between them), and a value is off by half of
    its code's step at most: 2^-4 of it, or 2^-10 of the power of two."""
    if exactly:
        want, want_byte = ref8.encode(y.numpy())
        assert byte == want_byte and np.array_equal(code.numpy(), want), what
        return
    most, slack = float(y.abs().max()), 2.0 ** -20 * float(mag.max())
    assert byte - 127 in {ref8.exponent(max(0.0, most - slack)), ref8.exponent(most + slack)}, what
    import torch

    got = ref8.decode(code, torch.tensor(byte))
    bound = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10 * 2.0 ** (byte - 127), dtype=torch.float64))
    # (a value past 448 2^e by the kernel's rounding is that much further off)
    assert bool(((got - y).abs() <= bound * (1 + 2.0 ** -20) + 2.0 ** -19 * mag).all()), what


@pytest.mark.parametrize("axes", [0, 1, 3, 8])
@pytest.mark.parametrize("name", APPEND)
def test_append(msa, name, axes):
    import torch

    kw = dict(APPEND[name])
    rot, rot_idx, how, fused = kw.pop("rot"), kw.pop("rot_idx"), kw.pop("interleaved", False), kw.pop("fused", False)
    if axes in (1, 8) and name not in ("page_ends", "idle_and_padding", "partial_interleaved"):
        pytest.skip("three batches are enough for these")
    b = ref8.Batch(**kw)
    shape, cache, t = b.gpu()
    index = b.k_idx is not None
    x = _new_rows(b, fused=fused)
    src = {n: v.cpu() for n, v in x.items()}
    f, fi = _freq(rot), _freq(rot_idx)
    gen = torch.Generator().manual_seed(9)
    axis = torch.randint(0, max(1, axes), (rot // 2,), generator=gen, dtype=torch.int32)
    axis_idx = torch.randint(0, max(1, axes), (rot_idx // 2,), generator=gen, dtype=torch.int32)
    positions = torch.randint(-70000, 1 << 20, (b.N, max(1, axes)), generator=gen, dtype=torch.int32)
    named = dict(axis=axis.cuda(), axis_idx=axis_idx.cuda() if index else None) if axes > 1 else {}
    rope = msa.Rope(f.cuda(), fi.cuda() if index else None, interleaved=how, **named)
    out = torch.full((b.N, b.Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    qi_out = torch.full((b.N, b.G, 64), 3.0, dtype=torch.bfloat16, device="cuda") if index else None
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
    msa.msa_paged_append_fp8(shape, cache, rope, x["K"], x["V"], x.get("k_idx"), x["Q"], x.get("q_idx"), out, qi_out, ws,
                             positions=positions.cuda() if axes else None)
    msa.msa_check_device_status(ws)

    names = [n for n in ("K", "V", "k_idx") if getattr(b, n) is not None]
    want = {n: (getattr(b, n + "8").view(torch.uint8).clone(), getattr(b, n + "_exp").clone()) for n in names}
    got = {n: (t[n + "8"].cpu().view(torch.uint8), t[n + "_exp"].cpu()) for n in names}
    for r in range(b.n):
        page, slot = int(b.table[b.row_seq[r], b.row_pos[r] // 128]), b.row_pos[r] % 128
        for n in names:
            here = (page, slice(None), slot) if n != "k_idx" else (page, slot)
            ax, fr = (axis_idx, fi) if n == "k_idx" else (axis, f)
            where = positions[r][ax.long()] if axes else b.row_pos[r]
            y, mag = _turned(src[n], r, where, fr, how)
            if n == "V":
                y, mag = src[n][r].double(), 0.0 * mag
            code, byte = (v[here] for v in got[n])
            if r < 8 or r % 7 == 0:
                for c, e, yy, mm in zip(code.view(-1, code.shape[-1]), byte.view(-1), y.view(-1, y.shape[-1]),
                                        mag.view(-1, y.shape[-1])):
                    _check_vector(c, int(e), yy, mm, n == "V" or fr.numel() == 0, (n, r))
            for v, w in zip(got[n], want[n]):
                v[here] = w[here]
        if r < 8 or r % 7 == 0:
            y, mag = _turned(src["Q"], r, positions[r][axis.long()] if axes else b.row_pos[r], f, how)
            assert bool(((out[r].cpu().double() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -20 * mag).all()), ("Q", r)
    for n in names:  # nothing else of the pools was touched
        for v, w in zip(got[n], want[n]):
            assert torch.equal(v, w), n
    assert bool((out[b.n:] == 3.0).all())


def test_append_of_every_magnitude(msa):
    """V, which is not rotated, has exactly the codes of the definition: every bf16 exponent, ties, and what is not finite."""
    import torch

    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # every bf16
    rows = bits.view(512, 1, 128).clone()  # 128 neighbouring values at a time ...
    mixed = torch.stack([bits[torch.randperm(1 << 16, generator=torch.Generator().manual_seed(i))][:128] for i in range(128)])
    rows = torch.cat([rows, mixed.view(128, 1, 128)])  # ... and of any magnitudes
    # (a vector of a magnitude m has codes that are ties where its other values end in ...1000)
    n = rows.shape[0]
    b = ref8.Batch(counts=[n], lens=[n], Hq=1, G=1)
    shape, cache, t = b.gpu()
    new = rows.cuda()
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
    ki = rows[:, 0, 64:].contiguous().cuda()
    msa.paged_append_fp8(shape, cache, msa.Rope(), new, new, ki, workspace=ws)
    msa.msa_check_device_status(ws)
    for r in range(n):
        page, slot = int(b.table[0, r // 128]), r % 128
        want, byte = ref8.encode(rows[r, 0].double().numpy())
        for name in ("K", "V"):
            got = t[name + "8"][page, 0, slot].cpu().view(torch.uint8).numpy()
            assert int(t[name + "_exp"][page, 0, slot]) == byte, r
            assert np.array_equal(np.where(rows[r, 0].isfinite().numpy(), got, 0x7f), want), r
            assert ((got & 0x7f) == 0x7f).sum() == (want == 0x7f).sum()
        want, byte = ref8.encode(rows[r, 0, 64:].double().numpy())
        got = t["k_idx8"][page, slot].cpu().view(torch.uint8).numpy()
        assert int(t["k_idx_exp"][page, slot]) == byte and np.array_equal(got & 0x7f, want & 0x7f), r


# ----------------------------------------------------------------- positions with several axes, in bf16
@pytest.mark.parametrize("name", ["page_ends", "idle_and_padding", "interleaved", "partial_interleaved", "partial_strided",
                                  "no_rotation", "no_index", "blocks_of_rows"])
@pytest.mark.parametrize("axes", [1, 2, 3, 8])
def test_append_axes(msa, name, axes):
    import torch

    kw = dict(APPEND[name])
    rot, rot_idx, how, fused = kw.pop("rot"), kw.pop("rot_idx"), kw.pop("interleaved", False), kw.pop("fused", False)
    b = ref.Batch(stale=7.0, **kw)
    shape, cache, t = b.gpu()
    index = b.k_idx is not None
    x = _new_rows(b, fused=fused)
    f, fi = _freq(rot), _freq(rot_idx)
    gen = torch.Generator().manual_seed(9)
    axis, axis_idx = (torch.randint(0, axes, (m // 2,), generator=gen, dtype=torch.int32) for m in (rot, rot_idx))
    positions = torch.randint(-(2 ** 31), 2 ** 31 - 1, (b.N, axes), generator=gen).to(torch.int32)
    positions[::2] = positions[::2] >> 12
    positions[0] = -2 ** 31
    rope = msa.Rope(f.cuda(), fi.cuda() if index else None, interleaved=how, axis=axis.cuda() if axes > 1 else None,
                    axis_idx=axis_idx.cuda() if index and axes > 1 else None)
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
    Q, qi = msa.paged_append(shape, cache, rope, x["K"], x["V"], x.get("k_idx"), x["Q"], x.get("q_idx"), workspace=ws,
                             positions=positions.cuda())
    msa.msa_check_device_status(ws)
    src = {n: v.cpu() for n, v in x.items()}
    got = {n: t[n].cpu() for n in ("K", "V", "k_idx") if t[n] is not None}
    for r in range(0, b.n, 1 if b.n < 300 else 7):
        page, slot = int(b.table[b.row_seq[r], b.row_pos[r] // 128]), b.row_pos[r] % 128
        where, where_idx = positions[r][axis.long()], positions[r][axis_idx.long()]
        # the bounds of the append with one axis: the phase is kept to 2^-32 turns, sin and cos to fp32
        for n, g, p, fr in (("K", got["K"][page, :, slot], where, f), ("Q", Q[r].cpu(), where, f),
                            *((("k_idx", got["k_idx"][page, slot], where_idx, fi), ("q_idx", qi[r].cpu(), where_idx, fi))
                              if index else ())):
            y, mag = _turned(src[n], r, p, fr, how)
            # (positions to 2^31 in 64 bits: the reference's own product is off by 2^-53 of up to 2^31 radians). Below the
            # smallest normal number, 2^-126, bf16's steps are 2^-133, so that a rounding is off by 2^-134 there.
            bound = 2.0 ** -8 * y.abs() + 2.0 ** -20 * mag + 2.0 ** -134
            assert bool(((g.double() - y).abs() <= bound).all()), (n, r)
        assert torch.equal(got["V"][page, :, slot], src["V"][r])


def test_append_axes_of_own_positions_is_the_append(msa):
    import torch

    b = ref.Batch(counts=[3, 0, 130, 1], lens=[1000, 4, 131, 77], Hq=8, G=2, stale=7.0, pad=2)
    x = _new_rows(b)
    f, fi = _freq(128).cuda(), _freq(64).cuda()
    positions = torch.zeros(b.N, 3, dtype=torch.int32)
    positions[:b.n] = torch.tensor(b.row_pos)[:, None]
    axis, axis_idx = torch.arange(64, dtype=torch.int32).cuda() % 3, torch.arange(32, dtype=torch.int32).cuda() % 3
    got = []
    for rope, p in ((msa.Rope(f, fi), None), (msa.Rope(f, fi, axis=axis, axis_idx=axis_idx), positions.cuda()),
                    (msa.Rope(f, fi), positions[:, :1].contiguous().cuda())):
        shape, cache, t = b.gpu()
        Q, qi = msa.paged_append(shape, cache, rope, x["K"], x["V"], x["k_idx"], x["Q"], x["q_idx"], positions=p)
        got.append([v.cpu() for v in (Q[:b.n], qi[:b.n], t["K"], t["V"], t["k_idx"])])
    for other in got[1:]:
        assert all(torch.equal(u, v) for u, v in zip(got[0], other))


@pytest.mark.parametrize("rows", [5, 1100])  # the call's checks in a block of their own, and in each
@pytest.mark.parametrize("bad", [-1, 3, 2 ** 31 - 1, -2 ** 31])
def test_append_axes_outside_are_reported(msa, rows, bad):
    import torch

    for index in (False, True):
        b = ref8.Batch(counts=[rows], lens=[rows], Hq=2, G=1)
        shape, cache, t = b.gpu()
        x = _new_rows(b)
        axis, axis_idx = torch.zeros(64, dtype=torch.int32), torch.zeros(32, dtype=torch.int32)
        (axis_idx if index else axis)[17] = bad
        rope = msa.Rope(_freq(128).cuda(), _freq(64).cuda(), axis=axis.cuda(), axis_idx=axis_idx.cuda())
        ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
        msa.paged_append_fp8(shape, cache, rope, x["K"], x["V"], x["k_idx"], x["Q"], x["q_idx"], workspace=ws,
                             positions=torch.zeros(rows, 3, dtype=torch.int32, device="cuda"))
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE
        for v, (code, byte) in (("V", (t["V8"], t["V_exp"])),):  # what has no axis is as it should be
            want = [ref8.encode(x[v][r, 0].cpu().double().numpy()) for r in range(5)]
            page = int(b.table[0, 0])
            assert all(np.array_equal(code[page, 0, r].cpu().view(torch.uint8).numpy(), w[0]) for r, w in enumerate(want))


# ----------------------------------------------------------------- reading back
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("lens,first,count", [([1], None, [1]), ([127, 129, 0, 700], None, [127, 129, 0, 700]),
                                              ([300, 1000, 50], [100, 999, 0], [200, 1, 0]),
                                              ([5000] + [0] * 40 + [130], [1, *[0] * 40, 2], [4099, *[0] * 40, 128])], ids=str)
def test_read(msa, G, lens, first, count):
    import torch

    for index in (True, False):
        b = ref8.Batch(counts=[0] * len(lens), lens=lens, Hq=G, G=G, seed=2, index=index)
        shape, cache, t = b.gpu()
        starts = np.concatenate([[0], np.cumsum(count)])
        n = int(starts[-1])
        M = n + 3
        K, V = (torch.full((M, G, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ki = torch.full((M, 64), 5.0, dtype=torch.bfloat16, device="cuda") if index else None
        ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
        ws.fill_(255)
        at = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
        msa.msa_paged_read_fp8(shape, cache, at, torch.tensor(starts, dtype=torch.int32, device="cuda"), K, V, ki, ws)
        msa.msa_check_device_status(ws)
        seq = np.repeat(np.arange(len(lens)), count)
        token = np.concatenate([np.arange(c) + (first[s] if first else 0) for s, c in enumerate(count)])
        page, slot = b.table[torch.tensor(seq), torch.tensor(token // 128)].long(), torch.tensor(token % 128)
        assert torch.equal(K[:n].cpu(), b.K[page, :, slot]) and torch.equal(V[:n].cpu(), b.V[page, :, slot])
        for x in (K, V, ki):
            assert x is None or bool((x[n:] == 5.0).all())
        if index:
            assert torch.equal(ki[:n].cpu(), b.k_idx[page, slot])


def test_read_bad_tokens_are_reported(msa):
    import torch

    def run(change, first, starts):
        b = ref8.Batch(counts=[0, 0], lens=[300, 500], Hq=2, G=2, seed=2)
        change(b)
        shape, cache, t = b.gpu()
        ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
        K, V = (torch.full((900, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        i32 = dict(dtype=torch.int32, device="cuda")
        msa.msa_paged_read_fp8(shape, cache, torch.tensor(first, **i32), torch.tensor(starts, **i32), K, V, None, ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE
        msa.msa_check_device_status(ws)
        return b, K.cpu(), V.cpu()

    nothing = lambda b: None  # noqa: E731
    b, K, V = run(nothing, [0, 0], [0, 301, 400])  # one token too many: the others are there
    assert torch.equal(K[:128], b.K[int(b.table[0, 0])].transpose(0, 1)) and bool((K[300] == 5.0).all())
    assert torch.equal(V[301:400], b.V[int(b.table[1, 0]), :, :99].transpose(0, 1))
    run(nothing, [-1, 0], [0, 10, 20])
    run(nothing, [0, 2 ** 31 - 1], [0, 10, 20])
    run(nothing, [-2 ** 31, 0], [0, 10, 20])
    for v in (-1, 1 << 20, 2 ** 31 - 1, -2 ** 31):
        def change(b):
            b.table[1, 2] = v

        b, K, V = run(change, [0, 0], [0, 300, 800])
        assert torch.equal(K[300:428], b.K[int(b.table[1, 0])].transpose(0, 1)) and bool((K[300 + 256:300 + 384] == 5.0).all())
    for v in (1 << 30, -1):  # lengths that the table cannot hold, or none
        def change(b):
            b.lens[0] = v

        run(change, [0, 0], [0, 300 if v < 0 else 700, 800])


# ----------------------------------------------------------------- sparse
SPARSE = {
    "first_token": dict(counts=[1], lens=[1], Hq=8, G=2, k=4),
    "page_ends": dict(counts=[1, 1, 1, 1, 1, 1], lens=[2, 127, 128, 129, 256, 257], Hq=8, G=2, k=2),
    "k1": dict(counts=[1, 2], lens=[700, 1300], Hq=4, G=2, k=1),
    "hg1_g3": dict(counts=[2, 1], lens=[1500, 2000], Hq=3, G=3, k=5),
    "hg2_idle_padding": dict(counts=[0, 3, 0, 1], lens=[50, 1027, 0, 4000], Hq=4, G=2, k=7, pad=2),
    "hg8_rows": dict(counts=[5, 1, 9], lens=[5000, 640, 900], Hq=16, G=2, k=16),
    "g8": dict(counts=[1, 1, 2], lens=[3000, 2999, 5111], Hq=32, G=8, k=16),
    "all_blocks_kept": dict(counts=[1, 4], lens=[1000, 260], Hq=8, G=1, k=40),
    "k33": dict(counts=[1, 1], lens=[9000, 8193], Hq=4, G=1, k=33),
    "k128": dict(counts=[2], lens=[128 * 140 + 5], Hq=2, G=1, k=128),
    "many_rows": dict(counts=[40, 1, 30], lens=[2040, 1, 1037], Hq=8, G=2, k=4),
}


def _sparse(msa, b, k, **kw):
    import torch

    shape, cache, t = b.gpu(k)
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE_FP8)
    ws.fill_(255)  # no result may depend on what a workspace held
    bi = torch.full((b.N, b.G, k), -7, dtype=torch.int32, device="cuda")
    O = torch.full((b.N, b.Hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((b.N, b.Hq), 5.0, device="cuda")
    msa.msa_paged_sparse_attn_fp8(shape, cache, t["Q"], t["q_idx"], bi, O, LSE, ws, **kw)
    msa.msa_check_device_status(ws)
    return O.cpu(), LSE.cpu(), bi.cpu().numpy()


def _check_sparse(b, k, O, LSE, bi, rows=None):
    for r in range(b.n):
        np.testing.assert_array_equal(bi[r], ref.select(b, r, k), err_msg=f"row {r}")
    rows = rows or (range(b.n) if b.n < 20 else range(0, b.n, 5))
    ref8.check_attention(b, rows, range(b.Hq), O, LSE, lambda r, g: bi[r, g].tolist())
    _check_padding(b, O, LSE, bi)


@pytest.mark.parametrize("stale", ["nan", "huge"])
@pytest.mark.parametrize("name", SPARSE)
def test_sparse(msa, name, stale):
    kw = dict(SPARSE[name])
    k = kw.pop("k")
    b = ref8.Batch(stale=stale, seed=3, **kw)
    _check_sparse(b, k, *_sparse(msa, b, k))


def test_sparse_long(msa):
    """A quarter of a million tokens, two rows: more blocks than a pass of the selection's threads."""
    b = ref8.Batch(counts=[2], lens=[1 << 18], Hq=2, G=1, seed=8)
    _check_sparse(b, 16, *_sparse(msa, b, 16))


@pytest.mark.parametrize("what", ["ties", "zero queries", "zero keys", "equal keys", "huge", "tiny", "very huge", "spread",
                                  "nan keys", "nan and infinite queries", "all nan", "one large query value"])
def test_selection_at_narrow_borders(msa, what):
    """Blocks that fp32 sums cannot tell apart, scores out of fp32's comfortable range, and ones that are not finite: the
    selection is that of the exact scores of the codes' values, ties to the lower id, NaN as -infinity."""
    import torch

    gen = torch.Generator().manual_seed(2)

    def change(b):
        for s in range(2):
            pages = b.table[s, :24].long()
            first = b.k_idx[pages[0]].clone()
            for c, page in enumerate(pages.tolist()):
                if what == "ties":  # the same page again, its keys in another order, or one key larger by one code
                    b.k_idx[page] = first if c % 3 else first[torch.randperm(128, generator=gen)]
                    if c % 5 == 1:
                        b.k_idx[page, c] *= 1.125
                elif what == "zero keys" and c % 4:
                    b.k_idx[page] = 0.0
                elif what == "equal keys":
                    b.k_idx[page] = first[c % 2]
                elif what == "huge":
                    b.k_idx[page] *= 2.0 ** 60
                elif what == "very huge":
                    b.k_idx[page] *= 2.0 ** 118
                elif what == "tiny":
                    b.k_idx[page] *= 2.0 ** -100
                elif what == "spread":
                    b.k_idx[page] = (b.k_idx[page].float() * torch.exp2(torch.randint(-60, 60, (128, 1), generator=gen).float())
                                     ).to(torch.bfloat16)
                elif what == "nan keys":
                    b.k_idx[page, 5:9, 3] = NAN
                    b.k_idx[page, 7] = INF
                elif what == "all nan" and c % 2:
                    b.k_idx[page, :, 1] = NAN

    b = ref8.Batch(counts=[1, 3], lens=[128 * 24 + 40, 128 * 24 + 3], Hq=2, G=2, seed=11, change=change)
    if what == "zero queries" or what == "all nan":
        b.q_idx[1] = 0.0
        b.q_idx[0, 1] = 0.0
    if what == "huge":
        b.q_idx[1] *= 2.0 ** 50
    if what == "very huge":
        b.q_idx *= 2.0 ** -60
        b.q_idx[2] *= 2.0 ** -40
    if what == "tiny":
        b.q_idx[1] *= 2.0 ** 100
        b.q_idx[2] *= 2.0 ** -20
    if what == "nan and infinite queries":
        b.q_idx[0, 0, 5] = INF
        b.q_idx[1, 0, 5] = NAN
        b.q_idx[2, 1] = -INF
    if what == "one large query value":
        b.q_idx[:, :, 7] = 2.0 ** 40
        b.q_idx[1, 0, 9] = -2.0 ** 20
    for k in (2, 4, 9):
        _, _, bi = _sparse(msa, b, k)
        for r in range(b.n):
            np.testing.assert_array_equal(bi[r], ref.select(b, r, k), err_msg=f"row {r}, k {k}")


def test_sparse_with_a_given_selection(msa):
    """IndexShare: block_idx is read; no index keys are needed; an empty list gives O = 0 and LSE = -infinity."""
    import torch

    b = ref8.Batch(counts=[1, 3, 0, 2], lens=[1000, 2000, 9, 130], Hq=8, G=2, seed=4, index=False, pad=1)
    k = 6
    rng = np.random.default_rng(0)
    bi = np.full((b.N, b.G, k), -1, np.int32)
    for r in range(b.n):
        for g in range(b.G):
            last = b.row_pos[r] // 128
            ids = sorted(rng.choice(last, min(last, k - 1), replace=False).tolist() + [last]) if last else [0]
            bi[r, g, :len(ids)] = ids
    bi[1, 0] = -1                     # nothing selected
    bi[2, 1] = [0, 3, -1, -1, -1, -1]  # without the own block
    shape, cache, t = b.gpu(k)
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE_FP8)
    O, LSE, _ = msa.paged_sparse_attn_fp8(shape, cache, t["Q"], block_idx=torch.from_numpy(bi).cuda(), workspace=ws)
    msa.msa_check_device_status(ws)
    ref8.check_attention(b, range(b.n), range(b.Hq), O.cpu(), LSE.cpu(), lambda r, g: bi[r, g].tolist())
    assert float(LSE[1, 0]) == -INF and bool((O[1, :4] == 0).all())
    for ids in ([0, 6, -1], [3, 1, 5], [2, 2, 5], [0, -1, 5], [-5, 1, 2], [2 ** 31 - 1, -1, -1]):
        b = ref8.Batch(counts=[1, 1], lens=[128 * 5 + 3, 128 * 5 + 3], Hq=8, G=2, seed=1)
        bi = torch.tensor([[[0, 2, 5]] * 2] * 2, dtype=torch.int32)
        bi[0, 1] = torch.tensor(ids, dtype=torch.int32)
        shape, cache, t = b.gpu(3)
        ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE_FP8)
        O, LSE, _ = msa.paged_sparse_attn_fp8(shape, cache, t["Q"], block_idx=bi.cuda(), workspace=ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE, ids
        ref8.check_attention(b, [1], range(8), O.cpu(), LSE.cpu(), lambda r, g: [0, 2, 5])


# ----------------------------------------------------------------- dense
DENSE = {
    "first_token": dict(counts=[1], lens=[1], Hq=8, G=2),
    "page_ends": dict(counts=[1, 1, 1, 1, 1], lens=[127, 128, 129, 256, 257], Hq=8, G=2),
    "rows_hg1": dict(counts=[20, 3, 17], lens=[20, 131, 400], Hq=3, G=3),
    "rows_hg2_idle": dict(counts=[0, 7, 0, 1], lens=[0, 300, 77, 900], Hq=4, G=2, pad=2),
    "rows_hg4": dict(counts=[9, 1, 5], lens=[1000, 2, 133], Hq=8, G=2),
    "rows_hg8": dict(counts=[3, 4], lens=[1500, 260], Hq=16, G=2),
    "g8_long": dict(counts=[1, 2], lens=[7000, 6001], Hq=32, G=8),
    "long_one": dict(counts=[1], lens=[60001], Hq=4, G=1),
    "prefix1": dict(counts=[1, 1], lens=[129, 200], Hq=8, G=2, prefix=1),
    "prefix_hg1": dict(counts=[1, 3, 0, 2], lens=[128 * 5 + 1, 128 * 5 + 300, 9, 128 * 5 + 2], Hq=3, G=3, prefix=5, pad=1),
    "prefix_hg2": dict(counts=[2, 1], lens=[128 * 9 + 2, 128 * 9 + 128], Hq=2, G=1, prefix=9),
    "prefix_idle_first": dict(counts=[0, 1, 2], lens=[0, 128 * 3 + 5, 128 * 3 + 9], Hq=4, G=1, prefix=3),
    # longer shared prefixes
    "shared_hg1": dict(counts=[1, 3, 0, 2] * 5, lens=[128 * 40 + 3 + 9 * i for i in range(20)], Hq=2, G=2, prefix=40, pad=1),
    "shared_hg2": dict(counts=[2, 1, 1] * 10, lens=[128 * 26 + 2 + 41 * i for i in range(30)], Hq=4, G=2, prefix=26),
    "shared_hg4": dict(counts=[0] + [1, 2] * 12 + [1], lens=[7] + [128 * 60 + 2 + 17 * i for i in range(25)], Hq=4, G=1, prefix=60),
    "shared_hg8": dict(counts=[1] * 16, lens=[128 * 100 + 1 + 64 * i for i in range(16)], Hq=8, G=1, prefix=100, pad=2),
    "shared_three_pairs": dict(counts=[1] * 70, lens=[128 * 12 + 1 + i for i in range(70)], Hq=16, G=2, prefix=12),
    # several rows a sequence
    "runs_hg8": dict(counts=[5, 3, 8], lens=[700, 130, 1000], Hq=16, G=2),
    "runs_one_group": dict(counts=[4, 9], lens=[513, 900], Hq=8, G=1),
    "runs_two_tiles": dict(counts=[20, 33, 1], lens=[600, 400, 300], Hq=16, G=2, pad=3),
    "runs_two_tiles_one_group": dict(counts=[17, 40], lens=[17, 390], Hq=8, G=1),
    "runs_hg1": dict(counts=[300, 10, 0, 129], lens=[1000, 300, 50, 129], Hq=2, G=2),
    "runs_hg2_three_groups": dict(counts=[6, 70], lens=[256, 500], Hq=6, G=3),
    "runs_hg4_ends": dict(counts=[4, 4, 4, 4, 4], lens=[127, 128, 130, 256, 259], Hq=8, G=2),
    "runs_long": dict(counts=[4], lens=[128 * 70 + 2], Hq=16, G=2),
    "runs_long_across_pages": dict(counts=[16], lens=[128 * 30 + 7], Hq=8, G=1),
    "runs_prefix": dict(counts=[3, 18, 0, 5], lens=[128 * 6 + 3, 128 * 6 + 400, 4, 128 * 7 + 5], Hq=16, G=2, prefix=6),
    "runs_prefix_three_pairs": dict(counts=[7] * 13, lens=[128 * 3 + 7 + 11 * i for i in range(13)], Hq=24, G=3, prefix=3),
    "runs_prefix_hg1": dict(counts=[12, 140], lens=[128 * 2 + 12, 128 * 2 + 300], Hq=1, G=1, prefix=2, pad=2),
}
# shared prefixes of so many pages, counted for every eight columns that read them, that they are read once for the batch
SHARED = {
    "hg1": dict(counts=[1, 3, 0, 2] * 10, lens=[128 * 40 + 3 + 9 * i for i in range(40)], Hq=2, G=2, prefix=40, pad=1),
    "hg2": dict(counts=[2, 1, 1] * 10, lens=[128 * 50 + 2 + 41 * i for i in range(30)], Hq=4, G=2, prefix=50),
    "hg4": dict(counts=[0] + [1, 2] * 12 + [1], lens=[7] + [128 * 120 + 2 + 17 * i for i in range(25)], Hq=4, G=1, prefix=120),
    "hg8": dict(counts=[1] * 16, lens=[128 * 180 + 1 + 64 * i for i in range(16)], Hq=8, G=1, prefix=180, pad=2),
    "three_pairs": dict(counts=[1] * 70, lens=[128 * 21 + 1 + i for i in range(70)], Hq=16, G=2, prefix=21),
    "page_of_rows": dict(counts=[127], lens=[128 * 60 + 127], Hq=16, G=2, prefix=60),
}
# several rows a sequence, and enough pages to read for them that 128-row tiles do it
TILES = {
    "hg8": dict(counts=[70, 33, 40], lens=[128 * 12 - 5, 900, 1400], Hq=16, G=2, pad=3),
    "hg8_one_tile": dict(counts=[12, 16, 3, 0, 9] * 4, lens=[900 + 17 * i for i in range(20)], Hq=16, G=2),
    "hg8_one_tile_three_groups": dict(counts=[12, 16, 3, 0, 9] * 3, lens=[900 + 17 * i for i in range(15)], Hq=24, G=3),
    "hg8_one_group": dict(counts=[300, 290, 17], lens=[700, 650, 17], Hq=8, G=1),
    "hg4_page_ends": dict(counts=[128, 129, 127, 64, 65], lens=[1024, 1025, 1023, 900, 128 * 7 + 1], Hq=8, G=2),
    "hg2_three_groups": dict(counts=[250, 300], lens=[1100, 999], Hq=6, G=3, pad=1),
    "hg1": dict(counts=[500, 400, 0, 300], lens=[1000, 470, 50, 300], Hq=3, G=3),
    "long": dict(counts=[17], lens=[128 * 90 + 2], Hq=16, G=2),
    "prefix": dict(counts=[12] * 16, lens=[128 * 14 - 90 + 5 * i for i in range(16)], Hq=16, G=2, prefix=6),
    "prefix_two_tiles": dict(counts=[40, 3, 25, 61], lens=[128 * 20 + 3, 128 * 9 + 4, 128 * 19 + 60, 2500], Hq=16, G=2, prefix=9, pad=2),
    # behind a prefix that is read by tiles, few own pages, too: drafts, three groups, idle sequences, two rows, one sequence
    "drafts": dict(counts=[5] * 9, lens=[128 * 40 + 5 + 13 * i for i in range(9)], Hq=16, G=2, prefix=40, pad=1),
    "drafts_three_groups": dict(counts=[0, 4, 7, 1, 6, 0] * 3, lens=[128 * 30 + 7 + 31 * i for i in range(18)], Hq=24, G=3, prefix=30),
    "drafts_one_group": dict(counts=[9, 3, 17] * 5, lens=[128 * 75 + 20 + 100 * i for i in range(15)], Hq=4, G=1, prefix=75, pad=3),
    "two_rows": dict(counts=[2] * 30, lens=[128 * 26 + 2 + 9 * i for i in range(30)], Hq=16, G=2, prefix=26),
    "many_teams": dict(counts=[6] * 8, lens=[128 * 300 + 6 + 150 * i for i in range(8)], Hq=16, G=2, prefix=300),
}


def _dense(msa, b, **kw):
    import torch

    shape, cache, t = b.gpu()
    ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE_FP8)
    ws.fill_(255)
    O = torch.full((b.N, b.Hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((b.N, b.Hq), 5.0, device="cuda")
    msa.msa_paged_dense_attn_fp8(shape, cache, t["Q"], O, LSE, ws, **kw)
    msa.msa_check_device_status(ws)
    return O.cpu(), LSE.cpu()


def _all(b):
    return lambda r, g: list(range(b.row_pos[r] // 128 + 1))


def _check_dense(b, O, LSE):
    rows = range(b.n) if b.n < 30 else range(0, b.n, 7)
    heads = range(b.Hq) if b.Hq <= 8 else range(0, b.Hq, 5)
    ref8.check_attention(b, rows, heads, O, LSE, _all(b), bf16_p=ref8.tiles(b))
    _check_padding(b, O, LSE)


@pytest.mark.parametrize("stale", ["nan", "huge"])
@pytest.mark.parametrize("name", DENSE)
def test_dense(msa, name, stale):
    b = ref8.Batch(stale=stale, seed=6, **DENSE[name])
    _check_dense(b, *_dense(msa, b))


@pytest.mark.parametrize("stale", ["nan", "huge"])
@pytest.mark.parametrize("name", TILES)
def test_dense_tiles(msa, name, stale):
    b = ref8.Batch(stale=stale, seed=6, **TILES[name])
    before = msa.msa_kernel_launches()
    O, LSE = _dense(msa, b)
    assert msa.msa_kernel_launches() - before == 3  # rows, tiles, merge
    _check_dense(b, O, LSE)


@pytest.mark.parametrize("stale", ["nan", "huge"])
@pytest.mark.parametrize("name", SHARED)
def test_dense_shared(msa, name, stale):
    b = ref8.Batch(stale=stale, seed=6, **SHARED[name])
    before = msa.msa_kernel_launches()
    O, LSE = _dense(msa, b)
    # rows, the prefix by tiles, own pages beside it (of 127 rows by tiles, too), merge
    assert msa.msa_kernel_launches() - before == (3 if name == "page_of_rows" else 4)
    _check_dense(b, O, LSE)


@pytest.mark.parametrize("name", ["rows_hg4", "g8_long", "prefix1", "runs_hg1", "shared_hg1"])
def test_dense_few_pages(msa, name):
    """Eight columns at a time, a small shared prefix as own pages: two launches."""
    b = ref8.Batch(seed=6, **DENSE[name])
    before = msa.msa_kernel_launches()
    _dense(msa, b)
    assert msa.msa_kernel_launches() - before == 2


SCALES = {"tokens": dict(counts=[1, 2], lens=[1000, 700], Hq=8, G=2),
          "shared": dict(counts=[1, 2] * 10, lens=[128 * 60 + 2 + 17 * i for i in range(20)], Hq=8, G=2, prefix=60),
          "prefix": dict(counts=[1, 2] * 13, lens=[128 * 60 + 2 + 17 * i for i in range(26)], Hq=8, G=2, prefix=60),
          "runs": dict(counts=[20, 9], lens=[600, 390], Hq=16, G=2),
          "tiles": dict(counts=[20] * 8 + [9, 31], lens=[1100 - 30 * i for i in range(8)] + [390, 1024], Hq=16, G=2)}


@pytest.mark.parametrize("what", ["v outlier", "v tiny", "v huge", "v spread", "v zero", "k spread", "k huge, q tiny",
                                  "k tiny, q huge", "rising", "q outlier"])
@pytest.mark.parametrize("name", SCALES)
def test_dense_scales(msa, name, what):
    """Powers of two that differ from token to token, and far from 1: a token counts by what it adds to the result."""
    import torch

    gen = torch.Generator().manual_seed(3)
    kw = SCALES[name]
    prefix = kw.get("prefix", 0)

    def change(b):
        some = lambda lo, hi, x: torch.exp2(torch.randint(lo, hi, x.shape[:-1] + (1,), generator=gen).float())  # noqa: E731
        if what == "v outlier":  # a token that nobody attends to, with values of 2^100
            for s in range(b.S):
                at = (int(b.table[s, prefix if s else 0]), slice(None), 1)
                b.K[at] = -b.Q[0, 0] * 0.0
                b.V[at] = b.V[at] * 2.0 ** 100
                b.K[at] = 0.0
            # (a row's scores are made so that the token's probability is below 2^-130)
            b.Q[:b.n] = b.Q[:b.n].abs() * 2
            for s in range(b.S):
                for c in range(-(-b.lens[s] // 128)):
                    b.K[int(b.table[s, c])] = b.K[int(b.table[s, c])].abs() + 1.0
            for s in range(b.S):
                b.K[int(b.table[s, prefix if s else 0]), :, 1] = -3.0
        elif what == "v tiny":
            b.V *= 2.0 ** -115
        elif what == "v huge":
            b.V *= 2.0 ** 110
        elif what == "v spread":
            b.V = (b.V.float() * some(-30, 30, b.V)).to(torch.bfloat16)
        elif what == "v zero":
            b.V[:, :, 3::5] = torch.where(b.V[:, :, 3::5].isnan(), b.V[:, :, 3::5], 0.0)
        elif what == "k spread":
            b.K = (b.K.float() * some(-20, 3, b.K)).to(torch.bfloat16)
        elif what == "k huge, q tiny":
            b.K *= 2.0 ** 80
            b.Q *= 2.0 ** -80
        elif what == "k tiny, q huge":
            b.K *= 2.0 ** -90
            b.Q *= 2.0 ** 90
        elif what == "rising":
            for s in range(b.S):
                for c in range(-(-b.lens[s] // 128)):
                    b.K[int(b.table[s, c])] *= float(1 + (c * 5) % 7) if c >= prefix or s == 0 else 1.0
            b.Q *= 3
        elif what == "q outlier":
            b.Q[:, :, 5] = 2.0 ** 12
            b.K[:, :, :, 5] *= 2.0 ** -12

    b = ref8.Batch(seed=7, change=change, **kw)
    O, LSE = _dense(msa, b)
    _check_dense(b, O, LSE)


@pytest.mark.parametrize("name", SCALES)
def test_values_that_are_not_finite(msa, name):
    """NaN codes of V reach the rows that see them, in their dims alone; NaN of K every dim of those rows; the rows before
    them have the same bits as without."""
    import torch

    b = ref8.Batch(seed=10, **SCALES[name])
    clean = _dense(msa, b)

    def put(pool, d):  # a NaN code into the vectors of the sequences' last tokens
        for s in range(b.S):
            if b.counts[s]:
                t = b.lens[s] - 1
                pool.view(torch.uint8)[int(b.table[s, t // 128]), :, t % 128, d] = 0x7f

    put(b.V8, 3)
    O, LSE = _dense(msa, b)
    assert bool((LSE[:b.n] == clean[1][:b.n]).all())
    for r in range(b.n):
        want = clean[0][r].clone()
        if b.row_pos[r] == b.lens[b.row_seq[r]] - 1:
            want[:, 3] = NAN
        assert bool(((O[r] == want) | (O[r].isnan() & want.isnan())).all()), r
    put(b.K8, 77)
    O, LSE = _dense(msa, b)
    for r in range(b.n):
        if b.row_pos[r] == b.lens[b.row_seq[r]] - 1:
            assert bool(O[r].isnan().all()) and bool(LSE[r].isnan().all()), r
        else:
            assert bool((O[r] == clean[0][r]).all()) and bool((LSE[r] == clean[1][r]).all()), r


@pytest.mark.parametrize("name", ["hg8", "hg8_one_tile", "hg4_page_ends", "hg1", "prefix"])
def test_later_rows_do_not_reach_earlier_ones_of_a_tile(msa, name):
    """NaN codes of V in the last tokens of every sequence: the rows that see them have NaN in their dims, and nothing else
    of any row changes; of K: the rows before have the same bits."""
    import torch

    b = ref8.Batch(seed=10, **TILES[name])
    clean = _dense(msa, b)

    def put(pool, back, d):
        for s in range(b.S):
            t = b.lens[s] - 1 - back
            if b.counts[s] > back:
                pool.view(torch.uint8)[int(b.table[s, t // 128]), :, t % 128, d] = 0x7f if d % 2 else 0xff

    for back, d in ((0, 3), (1, 40), (2, 77)):
        put(b.V8, back, d)
    O, LSE = _dense(msa, b)
    assert bool((LSE[:b.n] == clean[1][:b.n]).all())
    for r in range(b.n):
        want = clean[0][r].clone()
        behind = b.lens[b.row_seq[r]] - 1 - b.row_pos[r]
        for back, d in ((0, 3), (1, 40), (2, 77)):
            if behind <= back < b.counts[b.row_seq[r]]:
                want[:, d] = NAN
        same = (O[r] == want) | (O[r].isnan() & want.isnan())
        assert bool(same.all()), (r, behind, torch.nonzero(~same)[:4].tolist())
    put(b.K8, 1, 5)
    O, LSE = _dense(msa, b)
    for r in range(b.n):
        behind = b.lens[b.row_seq[r]] - 1 - b.row_pos[r]
        if behind > 2:
            assert bool((O[r] == clean[0][r]).all()) and bool((LSE[r] == clean[1][r]).all()), r
        elif behind <= 1 < b.counts[b.row_seq[r]]:
            assert bool(O[r].isnan().all()) and bool(LSE[r].isnan().all()), r


def test_pools_past_32_bit_offsets(msa):
    """Pages whose codes lie more than 2^32 bytes into the pools (and whose bytes past 2^25 vectors)."""
    import torch

    G, pages = 8, 34000
    f8 = torch.float8_e4m3fn
    K, V = (torch.zeros(pages, G, 128, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    Ke, Ve = (torch.full((pages, G, 128), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    ki, kie = torch.zeros(pages, 128, 64, dtype=torch.uint8, device="cuda"), torch.full((pages, 128), 127, dtype=torch.uint8, device="cuda")
    b = ref8.Batch(counts=[1], lens=[128 * 9 + 30], Hq=8, G=G, seed=13, spare=0)
    far = torch.tensor([pages - 1 - 3 * i for i in range(b.num_pages)], device="cuda")
    assert int(far.min()) * G * 128 * 128 > 2 ** 32
    for big, small in ((K, b.K8), (V, b.V8), (ki, b.k_idx8), (Ke, b.K_exp), (Ve, b.V_exp), (kie, b.k_idx_exp)):
        big[far] = small.view(torch.uint8).cuda()
    table = far.cpu()[b.table.long()].to(torch.int32).cuda()
    one, ln = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor(b.lens, dtype=torch.int32, device="cuda")
    cache = msa.PagedCacheFp8(K.view(f8), V.view(f8), Ke, Ve, ki.view(f8), kie, table, one, ln)
    shape = msa.PagedShape(S=1, N=1, Hq=8, G=G, num_pages=pages, max_blocks=b.max_blocks, k=5)
    O, LSE, bi = msa.paged_sparse_attn_fp8(shape, cache, b.Q.cuda(), b.q_idx.cuda())
    np.testing.assert_array_equal(bi[0].cpu().numpy(), ref.select(b, 0, 5))
    ref8.check_attention(b, [0], range(8), O.cpu(), LSE.cpu(), lambda r, g: bi[r, g].tolist())
    O, LSE = msa.paged_dense_attn_fp8(shape, cache, b.Q.cuda())
    ref8.check_attention(b, [0], range(8), O.cpu(), LSE.cpu(), _all(b))
    n = b.lens[0]
    k, v, i = msa.paged_read_fp8(shape, cache, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    token = torch.arange(n)
    page = b.table[0, token // 128].long()
    assert torch.equal(k.cpu(), b.K[page, :, token % 128]) and torch.equal(v.cpu(), b.V[page, :, token % 128])
    assert torch.equal(i.cpu(), b.k_idx[page, token % 128])
    new = torch.randn(1, G, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    msa.paged_append_fp8(shape, cache, msa.Rope(), new.cuda(), new.cuda())
    want = ref8.quantised(new[0])
    at = (int(far[b.table[0, 9].long()]), slice(None), 29)
    assert torch.equal(K[at].cpu(), want[0].view(torch.uint8)) and torch.equal(Ve[at].cpu(), want[1])
    del K, V, Ke, Ve


def test_bad_pages_and_positions_are_reported(msa):
    def run(change, which="sparse", prefix=0, good=None):
        b = ref8.Batch(counts=[1, 2], lens=[128 * 5 + 3, 128 * 6 + 9], Hq=8, G=2, prefix=prefix, seed=1)
        change(b)
        shape, cache, t = b.gpu(4)
        if which == "append":
            ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_APPEND)
            x = _new_rows(b)
            msa.paged_append_fp8(shape, cache, msa.Rope(), x["K"], x["V"], x["k_idx"], workspace=ws)
        elif which == "sparse":
            ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_SPARSE_FP8)
            O, LSE, bi = msa.paged_sparse_attn_fp8(shape, cache, t["Q"], t["q_idx"], workspace=ws)
        else:
            ws = msa.alloc_paged_workspace(shape, msa.MSA_WS_PAGED_DENSE_FP8)
            O, LSE = msa.paged_dense_attn_fp8(shape, cache, t["Q"], workspace=ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_check_device_status(ws)
        assert e.value.status == msa.MSA_ERR_DEVICE
        msa.msa_check_device_status(ws)  # the word was cleared
        if good is not None:  # the rows that were in order
            blocks = (lambda r, g: bi[r, g].tolist()) if which == "sparse" else _all(b)
            ref8.check_attention(b, good, range(8), O.cpu(), LSE.cpu(), blocks, bf16_p=prefix > 0)

    def page(s, c, v):
        def change(b):
            b.table[s, c] = v
        return change

    def length(s, v):
        def change(b):
            b.lens[s] = v
        return change

    for v in (-1, 1 << 20, 2 ** 31 - 1, -2 ** 31):
        run(page(0, 2, v), "sparse", good=[1, 2])
        run(page(1, 6, v), "sparse", good=[0])
        run(page(0, 5, v), "dense", good=[1, 2])
        run(page(0, 5, v), "append")
        run(page(0, 1, v), "dense", prefix=3)
    for v in (0, -5, 128 * 7 + 1, 2 ** 31 - 1, -2 ** 31):
        run(length(0, v), "sparse", good=[1, 2])
        run(length(0, v), "dense", good=[1, 2])
        run(length(0, v), "append")
    run(length(1, 128 * 3 + 1), "dense", prefix=3, good=[0])  # a row inside the prefix
    run(page(1, 2, 0), "dense", prefix=3)                      # a prefix that is not shared


def test_binding_refuses_what_does_not_fit(msa):
    import torch

    b = ref8.Batch(counts=[1, 2], lens=[300, 200], Hq=4, G=2, seed=1)
    shape, cache, t = b.gpu(4)
    x = _new_rows(b)
    f, fi = _freq(128).cuda(), _freq(64).cuda()
    axis = torch.zeros(64, dtype=torch.int32, device="cuda")
    at = torch.zeros(3, 2, dtype=torch.int32, device="cuda")

    def append(rope, positions):
        msa.paged_append_fp8(shape, cache, rope, x["K"], x["V"], x["k_idx"], x["Q"], x["q_idx"], positions=positions)

    for rope, positions, what in ((msa.Rope(f, fi, axis=axis), None, "positions"), (msa.Rope(f, fi), at.long(), "int32"),
                                  (msa.Rope(f, fi), at[:2], "shape"), (msa.Rope(f, fi), at[0], "shape"),
                                  (msa.Rope(f, fi), at.cpu(), "GPU"), (msa.Rope(f, fi), at.t().contiguous().t(), "contiguous")):
        with pytest.raises(ValueError, match=what):
            append(rope, positions)
    with pytest.raises(msa.MsaError, match="axes"):
        append(msa.Rope(f, fi), torch.zeros(3, 9, dtype=torch.int32, device="cuda"))
    for bad in (axis[:32], axis.long()):
        with pytest.raises(ValueError, match="axis"):
            msa.Rope(f, fi, axis=bad)
    pools = [cache.K, cache.V, cache.K_exp, cache.V_exp, cache.k_idx, cache.k_idx_exp]
    rest = [cache.page_table, cache.row_start, cache.seq_len]
    for i, bad in ((0, cache.K.view(torch.uint8)), (1, cache.V[:, :1].contiguous()), (2, cache.K_exp.float()), (3, cache.V_exp[:-1]),
                   (4, cache.k_idx[:, ::2]), (5, cache.k_idx_exp.cpu()), (5, None)):
        with pytest.raises(ValueError):
            msa.PagedCacheFp8(*[bad if j == i else p for j, p in enumerate(pools)], *rest)
    with pytest.raises(TypeError, match="PagedCacheFp8"):
        msa.paged_dense_attn_fp8(shape, msa.PagedCache(*[p.float().to(torch.bfloat16) for p in (cache.K, cache.V)], None, *rest), t["Q"])
    start = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
    for args, what in (((start.long(), 20), "int32"), ((start[:2], 20), "shape"), ((start, 20, start[:1]), "shape")):
        with pytest.raises(ValueError, match=what):
            msa.paged_read_fp8(shape, cache, *args)
    none = msa.PagedCacheFp8(*pools[:4], None, None, *rest)
    with pytest.raises(ValueError, match="k_idx"):
        msa.paged_sparse_attn_fp8(shape, none, t["Q"], t["q_idx"])
    with pytest.raises(ValueError, match="k_idx"):
        msa.paged_append_fp8(shape, none, msa.Rope(f, fi), x["K"], x["V"], x["k_idx"])


def test_copied_cache_has_its_own_tensors(msa):
    """A deep copy is another cache: appending to it leaves the first one alone."""
    import copy

    import torch

    b = ref8.Batch(counts=[2], lens=[130], Hq=2, G=1, seed=1)
    shape, cache, t = b.gpu(4)
    x = _new_rows(b)
    same, other = copy.copy(cache), copy.deepcopy(cache)
    was = [p.clone() for p in (cache.K.view(torch.uint8), cache.V_exp)]
    msa.paged_append_fp8(shape, other, msa.Rope(), x["K"], x["V"], x["k_idx"])
    assert torch.equal(cache.K.view(torch.uint8), was[0]) and torch.equal(cache.V_exp, was[1])
    msa.paged_append_fp8(shape, same, msa.Rope(), x["K"], x["V"], x["k_idx"])
    for n in ("K", "V", "k_idx"):
        assert torch.equal(getattr(cache, n).view(torch.uint8), getattr(other, n).view(torch.uint8)), n
        assert torch.equal(getattr(cache, n + "_exp"), getattr(other, n + "_exp")), n


# ----------------------------------------------------------------- streams, graphs, together
BITS = {"sparse": (dict(counts=[1, 2, 0, 1], lens=[40000, 700, 3, 129], Hq=16, G=2), "sparse"),
        "tokens": (dict(counts=[1] * 6, lens=[30000 + 999 * i for i in range(6)], Hq=8, G=2), "dense"),
        "shared": (SCALES["shared"], "dense"),
        "prefix": (SCALES["prefix"], "dense"),
        "runs": (dict(counts=[5, 33, 9], lens=[3000, 700, 1290], Hq=16, G=2), "dense"),
        "tiles": (dict(counts=[40, 33, 19], lens=[3000, 700, 1290], Hq=16, G=2), "dense"),
        "many_pages": (dict(counts=[1] * 8, lens=[30000 + 999 * i for i in range(8)], Hq=32, G=8, index=False), "dense")}


@pytest.mark.parametrize("name", BITS)
def test_same_bits_on_other_streams_and_at_once(msa, name):
    """Two calls at once with workspaces of their own, reruns and a captured call: the same bits every time."""
    import torch

    kw, which = BITS[name]
    b = ref8.Batch(seed=17, **kw)
    shape, cache, t = b.gpu(4)
    kind = msa.MSA_WS_PAGED_SPARSE_FP8 if which == "sparse" else msa.MSA_WS_PAGED_DENSE_FP8
    ws = [msa.alloc_paged_workspace(shape, kind) for _ in range(2)]
    out = [(torch.zeros_like(t["Q"]), torch.zeros(b.N, b.Hq, device="cuda"),
            torch.zeros(b.N, b.G, 4, dtype=torch.int32, device="cuda")) for _ in range(2)]

    def call(i, stream=None):
        O, LSE, bi = out[i]
        if which == "sparse":
            msa.msa_paged_sparse_attn_fp8(shape, cache, t["Q"], t["q_idx"], bi, O, LSE, ws[i], stream)
        else:
            msa.msa_paged_dense_attn_fp8(shape, cache, t["Q"], O, LSE, ws[i], stream)

    call(0)
    torch.cuda.synchronize()
    want = [x.clone() for x in out[0]]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in (0, 1, 0):
            call(i)
    for again in range(3):
        for i in range(2):
            msa.msa_check_device_status(ws[i])
            assert all(torch.equal(x, y) for x, y in zip(out[i], want)), again
            for x in out[i]:
                x.zero_()
        g.replay()
        torch.cuda.synchronize()


def test_helpers_on_a_stream(msa):
    """The allocating helpers given a stream run on it, and their workspaces belong to it."""
    import torch

    b = ref8.Batch(counts=[1, 2], lens=[3000, 700], Hq=8, G=2, seed=3)
    shape, cache, t = b.gpu(4)
    x = _new_rows(b)
    start = torch.tensor([0, 3000, 3700], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    rope = msa.Rope(_freq(128).cuda(), _freq(64).cuda())
    calls = (lambda **kw: msa.paged_append_fp8(shape, cache, rope, x["K"], x["V"], x["k_idx"], x["Q"], x["q_idx"], **kw),
             lambda **kw: msa.paged_sparse_attn_fp8(shape, cache, t["Q"], t["q_idx"], **kw),
             lambda **kw: msa.paged_dense_attn_fp8(shape, cache, t["Q"], **kw),
             lambda **kw: msa.paged_read_fp8(shape, cache, start, 3700, **kw))
    want = [f() for f in calls]
    side.wait_stream(torch.cuda.current_stream())
    got = [f(stream=side) for f in calls]
    held = [torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(8)]
    torch.cuda.current_stream().wait_stream(side)
    for g, w in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(g, w))
    del held


def test_captured_step_replays_on_another_batch(msa):
    """One decode step (append, selection and attention, full attention, reading back) captured once, replayed with other
    lengths, pages and rows of the same shape."""
    import torch

    b = ref8.Batch(counts=[1, 2, 1], lens=[900, 700, 129], Hq=8, G=2, pad=2, seed=20, max_blocks=12, spare=8)
    shape, cache, t = b.gpu(4)
    N, M = b.N, 2000
    new = {n: torch.zeros(N, *s, dtype=torch.bfloat16, device="cuda")
           for n, s in (("K", (2, 128)), ("V", (2, 128)), ("k_idx", (64,)), ("Q", (8, 128)), ("q_idx", (2, 64)))}
    axis, axis_idx = torch.arange(64, dtype=torch.int32).cuda() % 2, torch.arange(32, dtype=torch.int32).cuda() % 2
    rope = msa.Rope(_freq(128).cuda(), _freq(64).cuda(), axis=axis, axis_idx=axis_idx)
    positions = torch.zeros(N, 2, dtype=torch.int32, device="cuda")
    kinds = (msa.MSA_WS_PAGED_APPEND, msa.MSA_WS_PAGED_SPARSE_FP8, msa.MSA_WS_PAGED_DENSE_FP8, msa.MSA_WS_PAGED_APPEND)
    wsa, wss, wsd, wsr = (msa.alloc_paged_workspace(shape, w) for w in kinds)
    Qr, qir = torch.zeros_like(new["Q"]), torch.zeros_like(new["q_idx"])
    O, Od = torch.zeros_like(Qr), torch.zeros_like(Qr)
    LSE, LSEd = (torch.zeros(N, 8, device="cuda") for _ in range(2))
    bi = torch.zeros(N, 2, 4, dtype=torch.int32, device="cuda")
    start = torch.zeros(4, dtype=torch.int32, device="cuda")
    Ko, Vo = (torch.zeros(M, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kio = torch.zeros(M, 64, dtype=torch.bfloat16, device="cuda")

    def step():
        msa.msa_paged_append_fp8(shape, cache, rope, new["K"], new["V"], new["k_idx"], new["Q"], new["q_idx"], Qr, qir, wsa,
                                 positions=positions)
        msa.msa_paged_sparse_attn_fp8(shape, cache, Qr, qir, bi, O, LSE, wss)
        msa.msa_paged_dense_attn_fp8(shape, cache, Qr, Od, LSEd, wsd)
        msa.msa_paged_read_fp8(shape, cache, None, start, Ko, Vo, kio, wsr)

    step()  # once before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed, counts, lens in ((1, [1, 2, 1], [900, 700, 129]), (2, [0, 1, 4], [0, 1300, 500]), (3, [6, 0, 0], [6, 0, 0])):
        c = ref8.Batch(counts=counts, lens=lens, Hq=8, G=2, pad=N - sum(counts), seed=seed, max_blocks=12, spare=0)
        gen = torch.Generator().manual_seed(seed)
        t["table"].copy_(c.table)
        t["row_start"].copy_(torch.tensor(c.starts, dtype=torch.int32))
        t["seq_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        start.copy_(torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))
        for n in ("K", "V", "k_idx"):
            t[n + "8"].view(torch.uint8).zero_()
            t[n + "8"].view(torch.uint8)[:c.num_pages].copy_(getattr(c, n + "8").view(torch.uint8))
            t[n + "_exp"][:c.num_pages].copy_(getattr(c, n + "_exp"))
        for v in new.values():
            v.copy_(torch.randn(v.shape, generator=gen))
        positions.copy_(torch.randint(0, 5000, (N, 2), generator=gen))
        g.replay()
        for ws in (wsa, wss, wsd, wsr):
            msa.msa_check_device_status(ws)
        for n in ("K", "V", "k_idx"):
            setattr(c, n + "_exp", t[n + "_exp"].cpu()[:c.num_pages])
            setattr(c, n, ref8.decode(t[n + "8"].cpu()[:c.num_pages], getattr(c, n + "_exp")).to(torch.bfloat16))
        c.Q, c.q_idx = Qr.cpu(), qir.cpu()
        got = bi.cpu().numpy()
        for r in range(c.n):
            np.testing.assert_array_equal(got[r], ref.select(c, r, 4))
        ref8.check_attention(c, range(c.n), range(8), O.cpu(), LSE.cpu(), lambda r, g_: got[r, g_].tolist())
        ref8.check_attention(c, range(c.n), range(8), Od.cpu(), LSEd.cpu(), _all(c))
        at = 0
        for s, n in enumerate(lens):
            token = torch.arange(n)
            page = c.table[s, token // 128].long()
            assert torch.equal(Ko[at:at + n].cpu(), c.K[page, :, token % 128])
            assert torch.equal(kio[at:at + n].cpu(), c.k_idx[page, token % 128])
            at += n


def test_served_rows_are_those_of_the_training_calls(msa):
    """A sequence written into the cache in pieces (a prompt, drafts, single tokens) and attended to from there gives
    what msa_index_topk + msa_sparse_fwd and msa_dense_fwd give for the sequence as it is read back."""
    import torch

    T, Hq, G, k = 1536, 8, 2, 5
    gen = torch.Generator().manual_seed(30)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16).cuda()

    Q, K, V, qi, ki = normal(T, Hq, 128), normal(T, G, 128), normal(T, G, 128), normal(T, G, 64), normal(T, 64)
    f, fi = _freq(128).cuda(), _freq(64).cuda()
    axis, axis_idx = torch.arange(64, dtype=torch.int32).cuda() % 3, torch.arange(32, dtype=torch.int32).cuda() % 3
    rope = msa.Rope(f, fi, axis=axis, axis_idx=axis_idx)
    at3 = torch.stack([torch.arange(T) // 64, torch.arange(T) % 64 // 8, torch.arange(T) % 8], dim=1).to(torch.int32).cuda()
    pages = 20
    order = torch.randperm(pages, generator=gen)[:12].to(torch.int32)
    pools = [torch.full((pages, *s), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for s in ((G, 128, 128), (G, 128, 128), (128, 64))]
    exps = [torch.full((pages, *s), 255, dtype=torch.uint8, device="cuda") for s in ((G, 128), (G, 128), (128,))]
    table = order.view(1, 12).cuda()
    got = {n: [] for n in ("Q", "qi", "O", "LSE", "bi", "Od", "LSEd")}
    at = 0
    for n in (700, 1, 1, 5, 128, 61, 512, 1, 127):
        cache = msa.PagedCacheFp8(pools[0], pools[1], exps[0], exps[1], pools[2], exps[2], table,
                                  torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                  torch.tensor([at + n], dtype=torch.int32, device="cuda"))
        shape = msa.PagedShape(S=1, N=n, Hq=Hq, G=G, num_pages=pages, max_blocks=12, k=k, prefix_blocks=at // 128)
        s = slice(at, at + n)
        Qr, qir = msa.paged_append_fp8(shape, cache, rope, K[s], V[s], ki[s], Q[s], qi[s], positions=at3[s])
        O, LSE, bi = msa.paged_sparse_attn_fp8(shape, cache, Qr, qir)
        Od, LSEd = msa.paged_dense_attn_fp8(shape, cache, Qr)  # the sequence's own full blocks as the shared prefix
        for name, v in zip(got, (Qr, qir, O, LSE, bi, Od, LSEd)):
            got[name].append(v)
        at += n
    assert at == T
    got = {n: torch.cat(v) for n, v in got.items()}
    Kr, Vr, kir = msa.paged_read_fp8(shape, cache, torch.tensor([0, T], dtype=torch.int32, device="cuda"), T)
    # what was read back is what was written, by half a code's step: 2^-4 of a value, or 2^-10 of 2^e <= max|v| / 224
    most = V.float().abs().amax(2, keepdim=True)
    assert bool(((Vr.float() - V.float()).abs() <= torch.maximum(2.0 ** -4 * V.float().abs(), 2.0 ** -10 / 224 * most)).all())
    s = msa.Shape(B=1, T=T, Hq=Hq, G=G, k=k)
    bi = msa.index_topk(s, got["qi"][None].contiguous(), kir[None])
    same = (bi[0].transpose(0, 1) == got["bi"]).all(dim=2)
    assert float(same.float().mean()) > 0.999  # the training call decides near-ties in fp32
    O, LSE = msa.sparse_fwd(s, got["Q"][None].contiguous(), Kr[None], Vr[None], bi)
    Od, LSEd = msa.dense_fwd(s, got["Q"][None].contiguous(), Kr[None], Vr[None])
    same = same.repeat_interleave(Hq // G, dim=1)
    # both round P to bf16 at most, O to bf16, from scores within 1e-4: 2^-8 of |O| twice and of sum p |v| (< 4.5) once
    for a, c, m in ((got["O"], O[0], same), (got["Od"], Od[0], torch.ones_like(same))):
        err = (a.float() - c.float()).abs()
        assert float((err * m[..., None]).max()) <= 2.0 ** -8 * (4.5 + 2 * float(c.float().abs().max()))
        assert float((err * m[..., None]).mean()) <= 2.0 ** -8
    assert float(((got["LSE"] - LSE[0]).abs() * same).max()) <= 1e-3
    assert float((got["LSEd"] - LSEd[0]).abs().max()) <= 1e-3
