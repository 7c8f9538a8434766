"""Plain 64-bit forms for the paged cache in 8 bits (test infrastructure): its format from the definition, and batches whose
pools hold it. A batch's K, V and k_idx are the values that its codes stand for, so paged_ref's forms apply to it as they are."""
import math

import numpy as np

import paged_ref as ref

# E4M3's non-negative finite values by code: 2^-6 m / 8, then 2^(x - 7) (1 + m / 8)
VALUES = np.array([m / 512 for m in range(8)] + [2.0 ** (x - 7) * (1 + m / 8) for x in range(1, 16) for m in range(8)][:-1])


def exponent(most):
    """The smallest e in [-117, 120] with most <= 448 * 2^e."""
    e = -117
    while most > 448 * 2.0 ** e and e < 120:
        e += 1
    return e


def encode(x):
    """Codes (uint8) and byte of one vector of float64 (exactly representable in fp32)."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    e = exponent(np.abs(x[fine]).max() if fine.any() else 0.0)
    y = np.abs(np.where(fine, x, 0)) * 2.0 ** -e
    up = np.clip(np.searchsorted(VALUES, y), 1, len(VALUES) - 1)
    lo, hi = VALUES[up - 1], VALUES[up]
    code = np.where((y - lo < hi - y) | ((y - lo == hi - y) & ((up - 1) % 2 == 0)), up - 1, up)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(fine, code, 0x7f).astype(np.uint8), e + 127


def decode(codes, byte):
    """float64 values of codes [..., dim] and bytes [...] (torch, CPU)."""
    import torch

    table = torch.tensor(np.concatenate([VALUES, [np.nan], -VALUES, [np.nan]]))
    return table[codes.view(torch.uint8).long()] * torch.exp2(byte.double() - 127)[..., None]


def quantised(x):
    """Codes and bytes of x [..., dim] (torch, bf16 or fp32, CPU), by way of the table; quick enough for pools."""
    import torch

    y = x.double()
    fine = y.isfinite()
    most = torch.where(fine, y, 0.0).abs().amax(-1)
    m, up = torch.frexp(most)
    e = torch.where(most > 0, up - 9 + (m > 0.875).int(), -117).clamp(-117, 120)
    table = torch.tensor(VALUES)
    a = torch.where(fine, y, 0.0).abs() * torch.exp2(-e.double())[..., None]
    hi = torch.searchsorted(table, a).clamp(1, len(VALUES) - 1)
    dl, dh = a - table[hi - 1], table[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & ((hi - 1) % 2 == 0)), hi - 1, hi)
    code = torch.where(torch.signbit(y), code | 128, code)
    return torch.where(fine, code, 0x7f).to(torch.uint8).view(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


class Batch(ref.Batch):
    """A paged_ref.Batch whose pools are in 8 bits. Stale slots hold NaN codes and byte 255, or with stale "huge" the
    largest code and byte 247. `change`: called with the batch before its pools are quantised."""

    def __init__(self, *args, stale="nan", change=None, **kw):
        super().__init__(*args, stale=float("nan"), **kw)
        self.stale = stale
        if change:
            change(self)
        self.quantise()

    def quantise(self):
        """Codes and bytes of K, V and k_idx as they are now; the three become the codes' values."""
        import torch

        for n in ("K", "V", "k_idx"):
            x = getattr(self, n)
            if x is None:
                setattr(self, n + "8", None)
                setattr(self, n + "_exp", None)
                continue
            gone = x.isnan().all(-1)  # stale vectors
            code, byte = quantised(x)
            code, byte = code.view(torch.uint8).clone(), byte.clone()
            code[gone], byte[gone] = (0x7f, 255) if self.stale == "nan" else (0x7e, 247)
            setattr(self, n + "8", code.view(torch.float8_e4m3fn))
            setattr(self, n + "_exp", byte)
            value = decode(code, byte)
            assert torch.equal(value[~gone].to(torch.bfloat16).double().nan_to_num(nan=3.0), value[~gone].nan_to_num(nan=3.0))
            setattr(self, n, value.to(torch.bfloat16))

    def gpu(self, k=16):
        import torch

        import block_sparse_attention_scores_gb300 as msa

        t = {n: getattr(self, n) for n in ("K8", "V8", "K_exp", "V_exp", "k_idx8", "k_idx_exp", "Q", "q_idx", "table")}
        t = {n: None if x is None else x.cuda() for n, x in t.items()}
        t["row_start"] = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        t["seq_len"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        shape = msa.PagedShape(S=self.S, N=self.N, Hq=self.Hq, G=self.G, num_pages=self.num_pages,
                               max_blocks=self.max_blocks, k=k, prefix_blocks=self.prefix)
        cache = msa.PagedCacheFp8(t["K8"], t["V8"], t["K_exp"], t["V_exp"], t["k_idx8"], t["k_idx_exp"], t["table"],
                                  t["row_start"], t["seq_len"])
        return shape, cache, t


def tiles(b):
    """Whether the full attention may take 128-row tiles, where P is one bf16 (half a step of it: 2^-8): a shared prefix, or
    more than nine columns (rows x heads) a sequence."""
    return b.prefix > 0 or b.N * b.hg > 9 * b.S


def check_attention(b, rows, heads, O, LSE, blocks_of, bf16_p=False):
    """paged_ref.check_attention with the bounds of the calls over 8 bits: a score's and the sums' as there; P is held in
    fp16 as 2^15 p 2^f / max(p 2^f), f its token's exponent of V, that is with 2^-11 of itself, and 2^-25 (half of fp16's
    last step) at least: 2^-40 of max(p 2^f) times a code (448 at most) for each token. Where 128-row tiles may be taken
    (`bf16_p`), P is one bf16: 2^-8."""
    import torch

    for r in rows:
        for h in heads:
            g = h // b.hg
            blocks = [c for c in blocks_of(r, g) if c >= 0]
            o, lse, tol, tol_lse = ref.attend(b, r, h, blocks, bf16_p)
            if blocks:
                at = b.table[b.row_seq[r], blocks].long()
                token = (torch.tensor(blocks)[:, None] * 128 + torch.arange(128)).reshape(-1) <= b.row_pos[r]
                k, v = (x[at, g].reshape(-1, 128)[token].double() for x in (b.K, b.V))
                f = b.V_exp[at, g].reshape(-1)[token].double() - 127
                p = (k @ b.Q[r, h].double() / math.sqrt(128) - lse).exp()
                tol = tol + 2.0 ** -11 * (p @ v.abs()) + len(p) * 2.0 ** -40 * 448 * float((p * torch.exp2(f)).max())
            err = (O[r, h].double() - o).abs()
            assert bool((err <= tol + 1e-30).all()), (
                f"row {r} (position {b.row_pos[r]}) head {h}: O off by {float((err / (tol + 1e-30)).max()):.2f} of what "
                f"it may be")
            got = float(LSE[r, h])
            assert got == lse or abs(got - lse) <= tol_lse, f"row {r} head {h}: LSE {got} against {lse}, {tol_lse:.2e}"
