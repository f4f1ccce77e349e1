"""Plain attention in 64 bits, with bounds on what the kernels may be off by.

The reference forms every row explicitly in float64.  The bounds follow from the
roundings of include/lard_attn.h, element by element.  Let u be half a step of the
type (bf16 2^-8, fp32 2^-24) and a(t) = t 2^-23 the relative error of a sum of t terms
in fp32 (one ulp an addition: the tensor cores may truncate).

* logits: Z = tau sum_c q_c k_c in fp32 is off by at most e_z = (a(d + 8)) tau sum |q_c k_c|
  + 2^-22 |Z|; an exponential of it adds 2^-20 (ex2.approx and the reduction of its
  argument by a row maximum of the same size as the logits).
* LSE: e_lse = max_j e_z + a(keys) + 2^-20 + 2^-22 |LSE|.
* P entering a product is rounded to the type: each P_j is off by (u + E) P_j with
  E = 2 max_j e_z + a(keys) + 2^-19; so O is off by (u + E) sum_j P_j |v_j| + u |O|.
* dV: the same with P's columns, E also holding the LSE's own error; and a(rows).
* dZ = P (dP - delta): dP in fp32 is off by a(d) sum |dO v|; delta by sum_c |dO_c| e_O,c
  (it is formed from the rounded O) + a(d) sum |dO O|; dZ is rounded to the type.
  With the rest of out's rounding beside it (off by u^2 |O| at most), the u |O| of e_O goes.
* dQ, dK: tau sum |e_dZ| |k| (|q|), + a(terms) tau sum |dZ k|, + u |dQ|.
A normal result cannot be below the type's smallest normal, so 1e-30 is added to every
bound.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def a(t):
    return t * 2.0 ** -23


class Row:
    """One (sequence, query head): float64 q [n, d], the keys it may see, seen [n, keys]."""

    def __init__(self, q, k, v, seen, tau, dtype):
        self.u, self.tau, self.k, self.v, self.q = U[dtype], tau, k, v, q
        n, keys, d = q.shape[0], k.shape[0], q.shape[1]
        z = (tau * (q @ k.T)).masked_fill(~seen, -math.inf) if keys else torch.zeros((n, 0), dtype=torch.float64)
        self.any = seen.any(-1) if keys else torch.zeros(n, dtype=torch.bool)
        lse = torch.logsumexp(z, -1) if keys else torch.full((n,), -math.inf, dtype=torch.float64)
        self.lse = torch.where(self.any, lse, torch.full_like(lse, -math.inf))
        base = torch.where(self.any, lse, torch.zeros_like(lse))
        self.p = torch.exp(z - base[:, None])
        self.out = self.p @ v
        ez = a(d + 8) * tau * (q.abs() @ k.abs().T) + 2.0 ** -22 * torch.where(seen, z, torch.zeros_like(z)).abs()
        top = torch.where(seen, ez, torch.zeros_like(ez)).amax(-1) if keys else torch.zeros(n, dtype=torch.float64)
        lse0 = torch.where(self.any, self.lse, torch.zeros_like(lse)).abs()
        self.e_lse = top + a(keys) + 2.0 ** -20 + 2.0 ** -22 * lse0
        self.E = 2 * top + a(keys) + 2.0 ** -19
        in_sum = (self.u + self.E)[:, None] * (self.p @ v.abs())
        self.e_out = in_sum + self.u * self.out.abs() + 1e-30
        self.e_with_rest = in_sum + self.u ** 2 * self.out.abs() + 2.0 ** -23 * self.out.abs() + 1e-30

    def backward(self, do, rest=False):
        """dq, and this head's part of dk, dv, with bounds."""
        d, n, keys, u, tau = self.q.shape[1], self.q.shape[0], self.k.shape[0], self.u, self.tau
        E = (self.E + 2 * self.e_lse)[:, None]
        dp = do @ self.v.T
        delta = (do * self.out).sum(-1, keepdim=True)
        dz = self.p * (dp - delta)
        e_dp = a(d) * (do.abs() @ self.v.abs().T)
        e_delta = ((do.abs() * (self.e_with_rest if rest else self.e_out)).sum(-1) + a(d) * (do * self.out).abs().sum(-1))[:, None]
        e_dz = (1 + u) * self.p * (1 + E) * (e_dp + e_delta) + (u + E) * dz.abs() + a(2) * self.p * (dp.abs() + delta.abs())
        dq = tau * (dz @ self.k)
        e_dq = tau * (e_dz @ self.k.abs()) + a(keys) * tau * (dz.abs() @ self.k.abs())
        dk = tau * (dz.T @ self.q)
        e_dk = tau * (e_dz.T @ self.q.abs()) + a(n) * tau * (dz.abs().T @ self.q.abs())
        dv = self.p.T @ do
        e_dv = (self.p * (u + E)).T @ do.abs() + a(n) * (self.p.T @ do.abs())
        return (dq, e_dq + u * dq.abs() + 1e-30), (dk, e_dk), (dv, e_dv)


def f64(t):
    return t.detach().cpu().double()


def clamp_len(x, cap):
    return max(0, min(cap, int(x)))


def cross(q, k, v, tau, k_len=None, dout=None, rest=False):
    """Reference of cross attention: {name: (value, bound)} in float64 on the CPU; with rest,
    "sum" is what out + rest has to be and delta is formed from that."""
    (B, Hq, n, d), (Hkv, m), dt = q.shape, k.shape[1:3], q.dtype
    q, k, v = f64(q), f64(k), f64(v)
    got = {"out": torch.zeros((2, B, Hq, n, d), dtype=torch.float64), "lse": torch.zeros((2, B, Hq, n), dtype=torch.float64)}
    if dout is not None:
        dout = f64(dout)
        got["dq"] = torch.zeros((2, B, Hq, n, d), dtype=torch.float64)
        got["dk"], got["dv"] = (torch.zeros((2, B, Hkv, m, d), dtype=torch.float64) for _ in range(2))
    if rest:
        got["sum"] = torch.zeros((2, B, Hq, n, d), dtype=torch.float64)
    for b in range(B):
        size = m if k_len is None else clamp_len(k_len[b], m)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            r = Row(q[b, h], k[b, g, :size], v[b, g, :size], torch.ones((n, size), dtype=torch.bool), tau, dt)
            got["out"][0, b, h], got["out"][1, b, h] = r.out, r.e_out
            got["lse"][0, b, h], got["lse"][1, b, h] = r.lse, r.e_lse
            if rest:
                got["sum"][0, b, h], got["sum"][1, b, h] = r.out, r.e_with_rest
            if dout is not None:
                dq, dk, dv = r.backward(dout[b, h], rest)
                got["dq"][0, b, h], got["dq"][1, b, h] = dq
                for name, x in (("dk", dk), ("dv", dv)):
                    got[name][0, b, g, :size] += x[0]
                    got[name][1, b, g, :size] += x[1]
    for name in ("dk", "dv"):
        if name in got:  # the sum over the heads of a group, rounded once
            got[name][1] += (U[dt] + a(8)) * got[name][0].abs() + 1e-30
    return {k: (x[0], x[1]) for k, x in got.items()}


def prefix(q, kp, vp, ks, vs, s_len, tau):
    """Reference of prefix attention: {name: (value, bound)}."""
    (B, Hq, n, d), dt = q.shape, q.dtype
    Hkv = ks.shape[1] if ks is not None else kp.shape[0]
    q = f64(q)
    none = torch.zeros((0, d), dtype=torch.float64)
    out, lse = torch.zeros((2, B, Hq, n, d), dtype=torch.float64), torch.zeros((2, B, Hq, n), dtype=torch.float64)
    P = 0 if kp is None else kp.shape[1]
    for b in range(B):
        size = 0 if ks is None else (ks.shape[2] if s_len is None else clamp_len(s_len[b], ks.shape[2]))
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k = torch.cat((none if kp is None else f64(kp[g]), none if ks is None else f64(ks[b, g, :size])))
            v = torch.cat((none if kp is None else f64(vp[g]), none if ks is None else f64(vs[b, g, :size])))
            j, i = torch.arange(P + size)[None, :], torch.arange(n)[:, None]
            r = Row(q[b, h], k, v, (j < P) | (j - P <= size - n + i), tau, dt)
            out[0, b, h], out[1, b, h] = r.out, r.e_out
            lse[0, b, h], lse[1, b, h] = r.lse, r.e_lse
    return {"out": (out[0], out[1]), "lse": (lse[0], lse[1])}


def check(got, want, what=""):
    """Every element within its bound of the reference; infinities equal."""
    for name, (ref, bound) in want.items():
        x = f64(got[name])
        assert x.shape == ref.shape, f"{what} {name}: shape {tuple(x.shape)}, expected {tuple(ref.shape)}"
        inf = torch.isinf(ref)
        assert bool((x[inf] == ref[inf]).all()), f"{what} {name}: infinities differ"
        err, fine = (x - ref).abs(), ~inf
        bad = fine & ~(err <= bound)
        if bool(bad.any()):
            at = tuple(int(i) for i in bad.nonzero()[0])
            raise AssertionError(f"{what} {name}: {int(bad.sum())} of {ref.numel()} outside, first at {at}: "
                                 f"{x[at].item():.6g}, expected {ref[at].item():.6g} +- {bound[at].item():.2g}")


def randn(shape, dtype, seed, layout="bhnd", scale=1.0, device="cuda"):
    """Normal values [B, H, rows, d]; "bnhd" lays rows before heads in memory; "wide" makes a
    slice of a tensor with room on every side."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(shape, generator=gen) * scale).to(dtype)
    if layout == "bnhd":
        return x.transpose(1, 2).contiguous().to(device).transpose(1, 2)
    if layout == "wide":
        B, H, n, d = shape
        big = torch.full((B + 1, H + 2, n + 3, d + 16), float("nan"), dtype=dtype)
        big[:B, 1:H + 1, 2:n + 2, 8:d + 8] = x
        return big.to(device)[:B, 1:H + 1, 2:n + 2, 8:d + 8]
    return x.to(device)
