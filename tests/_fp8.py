"""Plain 64-bit definitions of the 8-bit cache and of what is computed over it, for the tests."""

import numpy as np
import torch

from workloads import EPS, PAGE_SIZE, ROPE

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def e4m3_table():
    """Value of each of the 256 e4m3 codes (0x7f and 0xff: NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where(c & 128, -v, v)
    v[(c & 127) == 127] = np.nan
    return torch.from_numpy(v)


def quantise(y):
    """(codes uint8 [..., D], scale bytes uint8 [...]) of float64 rows y [..., D], by the definition."""
    y = np.asarray(y, dtype=np.float64)
    amax = np.abs(y).max(-1)
    bad = ~np.isfinite(y).all(-1)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    k = np.ceil(np.log2(safe / 448.0)).astype(np.int64)
    k = np.where(safe > 448.0 * 2.0 ** k, k + 1, k)          # log2 may round across a border
    k = np.where(safe <= 448.0 * 2.0 ** (k - 1), k - 1, k)
    k = np.clip(np.where(amax == 0, -126, k), -126, 127)
    z = np.where(bad[..., None], 0.0, y) / 2.0 ** k[..., None]
    a = np.abs(z)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    q = np.rint(a / step) * step                             # nearest even; may reach the next power of two
    e = np.floor(np.log2(np.maximum(q, 2.0 ** -6)))
    m = np.rint(q / 2.0 ** (e - 3)).astype(np.int64)         # 8..15 normal, 0..7 below 2^-6
    code = np.where(m >= 8, ((e + 7).astype(np.int64) << 3) | (m - 8), m)
    code = np.where(np.signbit(z), code | 128, code)
    code = np.where(bad[..., None], 127, code)
    return code.astype(np.uint8), np.where(bad, 255, k + 127).astype(np.uint8)


def dequantise(codes, scales):
    """float64 pools [P, 16, Hkv, D] from codes (any 8-bit view) and scales [P, Hkv, 16]."""
    c = codes.view(torch.uint8)
    s = scales.view(torch.uint8).transpose(1, 2).to(torch.float64)
    f = torch.where(s == 255, torch.full_like(s, float("nan")), torch.pow(2.0, s - 127))
    f = torch.where(s == 0, torch.zeros_like(s), f)
    return e4m3_table().to(c.device)[c.long()] * f[..., None]


class Fp8Case:
    """A decode case whose pools are quantised: what the query may not read stays NaN (code 0x7f, scale 255)."""

    def __init__(self, case):
        self.base = case
        arrays = []
        for pool in (case.k_pool, case.v_pool):
            codes, scales = quantise(pool.double().cpu().numpy())
            arrays.append((torch.from_numpy(codes), torch.from_numpy(np.ascontiguousarray(scales.transpose(0, 2, 1)))))
        (self.k, self.ks), (self.v, self.vs) = arrays
        self.q, self.block_table, self.seq_lens = case.q, case.block_table, case.seq_lens

    def on(self, dev):
        c = self.base.to(dev)
        return (c.q, self.k.view(F8).to(dev), self.v.view(F8).to(dev), self.ks.view(E8).to(dev),
                self.vs.view(E8).to(dev), c.block_table, c.seq_lens)


def attention_rows(q, k_pool, v_pool, block_table, seq_lens, window, prefix=None, v_scale=None):
    """o [B, Hq, D] in 64 bits over float64 pools, and what a tolerance needs: A = sum w |v| / sum w of every element
    and the largest sum |q_i k_i| of every row.  prefix: (table, length) seen by every sequence before its own.

    With the 8-bit cache's value scales (v_scale [P, Hkv, 16]) also the floors of its f16 operands (decode_bound): Q, the
    largest max|q| sum |k_i| of every row, and F = max_l(w_l s_l) * sum_l |v_l| / s_l / sum w of every element."""
    q = q.double().cpu()
    k_pool, v_pool = k_pool.cpu(), v_pool.cpu()
    B, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    G = Hq // Hkv
    o, A, S = torch.zeros_like(q), torch.zeros_like(q), torch.zeros((B, Hq, 1), dtype=torch.float64)
    Q, F = torch.zeros_like(S), torch.zeros_like(q)
    for b in range(B):
        L = int(seq_lens[b])
        lo = max(0, L - window) if window > 0 else 0
        pos = torch.arange(lo, L)
        page, row = block_table[b].cpu()[pos // PAGE_SIZE].long(), pos % PAGE_SIZE
        if prefix is not None and prefix[1] > 0:
            pp = torch.arange(prefix[1])
            page = torch.cat([prefix[0].cpu()[pp // PAGE_SIZE].long(), page])
            row = torch.cat([pp % PAGE_SIZE, row])
        if page.numel() == 0:
            continue
        for c in range(Hkv):
            k, v = k_pool[page, row, c].double(), v_pool[page, row, c].double()
            qh = q[b, c * G:(c + 1) * G]
            w = torch.softmax(qh @ k.t(), -1)
            o[b, c * G:(c + 1) * G] = w @ v
            A[b, c * G:(c + 1) * G] = w @ v.abs()
            S[b, c * G:(c + 1) * G, 0] = (qh.abs() @ k.abs().t()).max(-1).values
            if v_scale is not None:
                byte = v_scale.view(torch.uint8).cpu()[page, c, row].double()
                scale = torch.pow(2.0, byte - 127)
                Q[b, c * G:(c + 1) * G, 0] = qh.abs().max(-1).values * k.abs().sum(-1).max()
                F[b, c * G:(c + 1) * G] = (w * scale).max(-1, keepdim=True).values * (v.abs() / scale[:, None]).sum(0)
    return (o, A, S) if v_scale is None else (o, A, S, Q, F)


def decode_bound(o, A, S, D, out_dtype, weight_eps, Q=0, F=0):
    """|got - o| allowed, element by element.

    Logits: D / 16 products accumulated in one chain, and at most 8 more
    roundings (chains joined, scales, log2 e), each off by at most 2^-23 of the
    largest partial sum, <= S: delta = (D/16 + 8) 2^-23 S; a weight is then off
    by a factor exp(delta) up and its sum by as much down.  Weights are rounded
    to their type (weight_eps) and their 2^x is off by at most 2^-21.  Sums are
    fp32 (2^-18 for their chains).  The output is rounded once.

    Over an 8-bit cache (Q, F): q and the weights w_l s_l (s_l the value row's scale) are f16 numbers whose largest is
    above 2^14, so half the smallest step, 2^-25, is 2^-39 of the largest: a logit moves by 2^-39 Q more, and against
    the values v_l / s_l the weights lose 2^-39 F.
    """
    delta = (D / 16 + 8) * 2.0 ** -23 * S + 2.0 ** -39 * Q
    rel = torch.expm1(2 * delta) + weight_eps + 2.0 ** -20 + 2.0 ** -18
    out = torch.finfo(out_dtype).eps / 2
    return (rel * A + 2.0 ** -39 * F) * (1 + out) + out * o.abs() + 1e-30


def append_rows(kind, qkv, w_q, w_k, positions, Hq, Hkv, D):
    """(q, k, v) rows [T, H, D] in 64 bits for tokens at `positions`."""
    theta, pairs = ROPE[kind]["theta"], ROPE[kind]["pairs"]
    x = qkv.double().cpu().numpy()
    T = x.shape[0]
    pos = np.asarray(positions, dtype=np.float64)

    def norm(y):
        return y / np.sqrt((y * y).mean(-1, keepdims=True) + EPS)

    def rope(y):
        i = np.arange(pairs)
        ang = pos[:, None, None] * theta ** (-2.0 * i / D)
        a, b = y[..., :pairs].copy(), y[..., D // 2:D // 2 + pairs].copy()
        y = y.copy()
        y[..., :pairs] = a * np.cos(ang) - b * np.sin(ang)
        y[..., D // 2:D // 2 + pairs] = b * np.cos(ang) + a * np.sin(ang)
        return y

    wq, wk = w_q.double().cpu().numpy(), w_k.double().cpu().numpy()
    q = rope(norm(x[:, :Hq * D].reshape(T, Hq, D)) * wq)
    xk = x[:, Hq * D:(Hq + Hkv) * D].reshape(T, Hkv, D)
    xv = x[:, -Hkv * D:].reshape(T, Hkv, D)
    return q, rope(norm(xk) * wk), norm(xv)


# fp32 error of an appended element against its row's largest: two turns' sin and cos (2^-21.4 each) and angle (2^-22),
# the norm's sum, root and products (32 steps of 2^-24): 2^-18.3 together, doubled
ROW_EPS = 2.0 ** -17.3
