"""fp64 reference of the windowed attention, the 8-bit cache and the attention over it, with a
bound on how far a kernel may be off at every output element.

The bounds add up what the kernels' documented arithmetic may lose, element by element:
  - a score is an fp32 dot product of d terms: (d + 8) 2^-24 sum |q||k| scale, and an fp32
    exponential of it, 2^-21 (1 + |z|); so a probability is off by a factor of at most 1 + EP;
  - bf16 calls round each probability (and dz) to bf16, half a step, u = 2^-8 relative, the
    cache's attention to fp16 (2^-11; fp32 calls keep 2^-21);
  - sums of m terms in fp32: m 2^-24 of the sum of magnitudes;
  - the result is rounded once to its type: u |x|.
"""
import math

import torch

F8 = torch.float8_e4m3fn
E_MIN = -100
F32U = 2.0 ** -24


def half_step(dtype):
    """Largest relative error of rounding to this type."""
    return torch.finfo(dtype).eps / 2


def visible(pos, keys, window, sinks):
    """[rows, keys] truth values for query positions (negative: no such row)."""
    t = torch.arange(keys, device=pos.device)[None, :]
    i = pos[:, None]
    return (t <= i) & ((i - t < window) | (t < sinks)) & (i >= 0)


def attend(q, k, v, see, scale, round_p):
    """One head: q [r, d], k and v [m, d] fp64. Returns o, lse, p, z and the bounds (eo, else).
    round_p: relative error of the rounded probabilities."""
    d, m = q.shape[1], k.shape[0]
    z = (q @ k.T) * scale
    zm = torch.where(see, z, -math.inf)
    lse = torch.logsumexp(zm, 1)
    p = torch.where(see, torch.exp(z - torch.where(lse.isfinite(), lse, 0.0)[:, None]), 0.0)
    ep = 2 * ((d + 8) * F32U * scale * (q.abs() @ k.abs().T) + 2.0 ** -21 * (1 + z.abs()))
    ep = torch.where(see, ep, 0.0)
    o = p @ v
    worst = ep.amax(1, keepdim=True) if m else torch.zeros(q.shape[0], 1, dtype=q.dtype, device=q.device)
    # numerator and denominator are both off by at most the row's worst factor
    eo = (p * (ep + worst + round_p + 2 * m * F32U)) @ v.abs()
    el = worst[:, 0] + m * F32U + 4 * F32U * (1 + torch.where(lse.isfinite(), lse, 0.0).abs())
    return o, lse, p, z, ep, eo, el


def window_forward(q, k, v, window, sinks, lens, scale, dtype):
    """q [B, n, hq, d], k/v [B, n, hkv, d] (any float type). Returns o, lse, eo, else in fp64."""
    B, n, hq, d = q.shape
    G = hq // k.shape[2]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    eo = torch.zeros_like(o)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
    el = torch.zeros_like(lse)
    up = half_step(torch.bfloat16) if dtype == torch.bfloat16 else 0.0
    for b in range(B):
        m = n if lens is None else int(lens[b])
        if m == 0:
            continue
        see = visible(torch.arange(m, device=q.device), m, window, sinks)
        for h in range(hq):
            a = [x[b, :m, y].double() for x, y in ((q, h), (k, h // G), (v, h // G))]
            ob, lb, _, _, _, e1, e2 = attend(*a, see, scale, up)
            o[b, :m, h], lse[b, :m, h], el[b, :m, h] = ob, lb, e2
            eo[b, :m, h] = e1 + half_step(dtype) * (ob.abs() + e1) + 1e-30
    return o, lse, eo, el


def window_backward(q, k, v, dout, window, sinks, lens, scale, dtype):
    """Gradients of sum(o * dout) and their bounds: (dq, dk, dv), (eq, ek, ev)."""
    B, n, hq, d = q.shape
    G = hq // k.shape[2]
    grads = [torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v)]
    errs = [torch.zeros_like(x) for x in grads]
    u = half_step(torch.bfloat16) if dtype == torch.bfloat16 else 0.0
    ut = half_step(dtype)
    for b in range(B):
        m = n if lens is None else int(lens[b])
        if m == 0:
            continue
        see = visible(torch.arange(m, device=q.device), m, window, sinks)
        for h in range(hq):
            qh, kh, vh = (x[b, :m, y].double() for x, y in ((q, h), (k, h // G), (v, h // G)))
            do = dout[b, :m, h].double()
            o, lse, p, z, ep, eo, el = attend(qh, kh, vh, see, scale, u)
            dp = do @ vh.T
            delta = (do * o).sum(1, keepdim=True)
            ds = p * (dp - delta)
            # the kernel's delta comes from the forward's rounded o
            edelta = (do.abs() * (eo + ut * o.abs())).sum(1, keepdim=True) + (d + 8) * F32U * (do * o).abs().sum(1, keepdim=True)
            epp = p * (ep + el[:, None])  # exp(z - lse) with both off
            eds = epp * (dp - delta).abs() + p * ((d + 8) * F32U * (do.abs() @ vh.abs().T) + edelta)
            eds = eds + u * (ds.abs() + eds) + 2.0 ** -22 * ds.abs()
            epp = epp + u * (p + epp)
            sums = 2 * m * G * F32U
            grads[0][b, :m, h] = scale * (ds @ kh)
            errs[0][b, :m, h] = scale * ((eds + sums * ds.abs()) @ kh.abs())
            grads[1][b, :m, h // G] += scale * (ds.T @ qh)
            errs[1][b, :m, h // G] += scale * ((eds + sums * ds.abs()).T @ qh.abs())
            grads[2][b, :m, h // G] += p.T @ do
            errs[2][b, :m, h // G] += (epp + sums * p).T @ do.abs()
    errs = [e + ut * (g.abs() + e) + 1e-30 for g, e in zip(grads, errs)]
    return grads, errs


# ---- the cache --------------------------------------------------------------------------------------


def block_scale(amax):
    """2^e, the smallest e >= E_MIN with amax <= 448 * 2^e; NaN for what is not finite."""
    if not math.isfinite(amax):
        return math.nan
    e = E_MIN
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def nearest_e4m3(x):
    """fp64 values of magnitude at most 448 rounded to e4m3, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    return torch.round(x * torch.exp2(3 - e)) * torch.exp2(e - 3)


def append(k, v, cache, new_lens=None):
    """cache: dict kq, vq (float8, CPU), ks, vs, table, lens (before). Writes it like the call."""
    B, t, hkv, d = k.shape
    page = cache["kq"].shape[2]
    for x, pool, scales in ((k, cache["kq"], cache["ks"]), (v, cache["vq"], cache["vs"])):
        for b in range(B):
            have = int(cache["lens"][b])
            n = t if new_lens is None else int(new_lens[b])
            at = have
            while at < have + n:
                stop = min(have + n, (at // page + 1) * page)
                blk, off = int(cache["table"][b, at // page]), at % page
                for h in range(hkv):
                    val = x[b, at - have: stop - have, h].double()
                    s = block_scale(float(val.abs().max()))
                    old = float(scales[blk, h])
                    if off and not math.isnan(s):
                        s = old if math.isnan(old) else max(s, old)
                    if not math.isnan(s):
                        if off and s != old:
                            pool[blk, h, :off] = nearest_e4m3(pool[blk, h, :off].double() * (old / s)).to(F8)
                        pool[blk, h, off: off + stop - at] = nearest_e4m3(val / s).to(F8)
                    scales[blk, h] = s
                at = stop


def cached(cache, name, b, h, length):
    """Keys or values [length, d] of one head as fp64."""
    page = cache["kq"].shape[2]
    blocks = cache["table"][b, : -(-length // page)].long()
    x = cache[name + "q"].view(torch.uint8)[blocks, h].view(F8).double()
    return (x * cache[name + "s"][blocks, h].double()[:, None, None]).flatten(0, 1)[:length]


def cache_attention(q, cache, window, sinks, q_lens, scale, dtype, edges=None):
    """gm_kv8_attention_forward, or gm_kv8_sea_forward with edges (idx, w): o, lse, eo, else."""
    B, t, hq, d = q.shape
    hkv = cache["kq"].shape[1]
    G = hq // hkv
    o = torch.zeros(q.shape, dtype=torch.float64)
    eo = torch.zeros_like(o)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64)
    el = torch.zeros_like(lse)
    rp = 2.0 ** -21 if dtype == torch.float32 else half_step(torch.float16)
    for b in range(B):
        length = int(cache["lens"][b])
        n = t if q_lens is None else int(q_lens[b])
        pos = length - n + torch.arange(n)
        if n == 0 or length == 0:
            continue
        for h in range(hq):
            kh, vh = (cached(cache, x, b, h // G, length) for x in ("k", "v"))
            qh = q[b, :n, h].double()
            if edges is None:
                see = visible(pos, length, window, sinks)
                ob, lb, _, _, _, e1, e2 = attend(qh, kh, vh, see, scale, rp)
                # fp32 queries keep 22 bits of the row's largest element
                if dtype == torch.float32:
                    extra = 2 * scale * 2.0 ** -21 * qh.abs().amax() * kh.abs().sum(1).amax()
                    e1, e2 = e1 + extra * (ob.abs() + vh.abs().amax()), e2 + extra
                # probabilities below fp16's subnormals
                e1 = e1 + length * 2.0 ** -38 * vh.abs().amax()
            else:
                idx, w = edges[0][b, :n, h // G].long(), edges[1][b, :n, h // G].double()
                ob, lb, e1, e2 = (torch.zeros(n, *s, dtype=torch.float64) for s in ((d,), (), (d,), ()))
                for x in range(n):
                    on = w[x] > 0
                    if int(pos[x]) < 0 or not bool(on.any()):
                        lb[x] = -math.inf
                        continue
                    kk, vv, ww = kh[idx[x][on]], vh[idx[x][on]], w[x][on]
                    z = (kk @ qh[x]) * scale + ww.log()
                    lb[x] = torch.logsumexp(z, 0)
                    p = torch.exp(z - lb[x])
                    ob[x] = p @ vv
                    worst = 2 * ((d + 8) * F32U * scale * (kk.abs() @ qh[x].abs()) + 2.0 ** -20 * (1 + z.abs())).max()
                    e1[x] = (p * (2 * worst + 64 * F32U)) @ vv.abs()
                    e2[x] = worst + 40 * F32U * (1 + lb[x].abs())
            o[b, :n, h], lse[b, :n, h], el[b, :n, h] = ob, lb, e2
            eo[b, :n, h] = e1 + half_step(dtype) * (ob.abs() + e1) + 1e-30
    return o, lse, eo, el


def check(got, want, bound, what):
    """Every element within its bound; infinities and NaN equal."""
    got, want, bound = got.double().cpu(), want.cpu(), bound.cpu()
    assert got.shape == want.shape, what
    fine = want.isfinite()
    assert torch.equal(fine, got.isfinite()), f"{what}: finite elsewhere"
    assert torch.equal(want[~fine & ~want.isnan()], got[~fine & ~got.isnan()]), f"{what}: infinities differ"
    off = (got - want).abs()
    over = torch.where(off == 0, 0.0, off / bound)[fine]  # exact values (empty rows) have bound 0
    if over.numel():
        assert float(over.max()) <= 1.0, f"{what}: {float(over.max()):.3g} times the bound"
