"""Inputs of the operators around the FFN whose results are exact, so that a single bit lost
on the way shows, and the same arithmetic on the CPU with a chosen number of bf16 planes.

A float of 24 significant bits is the sum of three bf16 planes of 8 bits each: the float
rounded, the remainder rounded, and what is left. Taking the first two planes of a value away
again from the value leaves the third, which any arithmetic in fewer than 24 bits has lost."""
import torch


def planes(v, count=3):
    """fp32 -> its bf16 planes, as fp32."""
    out, rest = [], v.float()
    for _ in range(count):
        out.append(rest.bfloat16().float())
        rest = rest - out[-1]
    return out


def cut(v, count):
    """fp32 to its first `count` planes."""
    return sum(planes(v, count))


def full_floats(g, *shape):
    """Random fp32 values in +-[1, 2), each with three planes other than zero."""
    bits = torch.randint(0, 1 << 23, shape, generator=g)
    v = (1 + bits.double() / (1 << 23)).float()
    v = torch.where(planes(v)[2] == 0, torch.tensor(1 + 2.0 ** -10 + 2.0 ** -20), v)
    assert bool((sum(planes(v)) == v).all() and (planes(v)[2] != 0).all())
    return v * (1 - 2 * torch.randint(0, 2, shape, generator=g)).float()


def lora_exact(g, S, n, r, K, N, x_dtype, whole):
    """x, a, b, scale, ids (int64 [S]), the exact adapter term d [S, N] (y = 0) and how far a
    result may be off it.

    Ranks 2i and 2i+1 form a pair: rank 2i of z is a value v of 24 bits, rank 2i+1 the
    negative of v's first two planes, both times a power of two of the adapter. Column c of b
    adds up pair c % (r / 2), or, `whole`, takes its v alone, times a power of two and a sign
    of its own. bf16 rows of x hold the planes of v in three places, fp32 rows v and its
    first two planes in two; where a pair's places lie in K is random."""
    pairs, each = r // 2, 3 if x_dtype == torch.bfloat16 else 2
    assert K >= pairs * each
    place = torch.randperm(K, generator=g)[:pairs * each].view(pairs, each)
    v = full_floats(g, S, pairs)
    p = planes(v)
    x, a = torch.zeros(S, K), torch.zeros(n, r, K)
    e = torch.exp2((torch.arange(n) % 5 - 2).float()).view(n, 1)
    i = torch.arange(pairs)
    if each == 3:
        for q in range(3):
            x[:, place[:, q]] = p[q]
            a[:, 2 * i, place[:, q]] = e
        for q in range(2):
            a[:, 2 * i + 1, place[:, q]] = -e
    else:
        x[:, place[:, 0]] = v
        x[:, place[:, 1]] = p[0] + p[1]
        a[:, 2 * i, place[:, 0]] = e
        a[:, 2 * i + 1, place[:, 1]] = -e
    c = torch.arange(N)
    factor = torch.exp2((c % 7 - 3).float()) * (1 - 2 * (c // 5 % 2)).float()
    b = torch.zeros(n, N, r)
    b[:, c, c % pairs * 2] = factor
    if not whole:
        b[:, c, c % pairs * 2 + 1] = factor
    scale = torch.exp2((torch.arange(n) % 3 - 1).float())
    ids = torch.randint(-1, n, (S,), generator=g)
    ids[0] = 0
    at = ids.clamp(min=0)
    d = (v if whole else p[2]).double()[:, c % pairs] * factor.double()
    d = d * (e[at] * scale[at].view(S, 1)).double()
    # Exact, but where the first plane of v is a power of two above v (2 for 1.998): a sum of
    # 24 bits with the term 2 in it ends at 2^-22 and v at 2^-23. Half a step there, 2^-23, for
    # each of the two sums, of a x and of b z.
    off = (p[0].abs() == 2).double()[:, c % pairs] * 2.0 ** -22
    off = off * factor.double().abs() * (e[at] * scale[at].view(S, 1)).double()
    d[ids < 0] = off[ids < 0] = 0
    return dict(x=x.to(x_dtype), a=a.bfloat16(), b=b.bfloat16(), scale=scale, ids=ids, d=d,
                off=off)


def exactly(got, ref, off):
    """got is ref rounded to its type, or within off of ref and that rounding."""
    tol = torch.where(off > 0, off + torch.finfo(got.dtype).eps / 2 * (ref.abs() + off), 0.0)
    want = torch.where(off > 0, ref, ref.float().to(got.dtype).double())
    return bool(((got.double() - want).abs() <= tol).all())


def lora_emulated(t, y_dtype, x_planes=3, z_planes=3):
    """The adapter term with x and z cut to so many planes, rounded to y_dtype."""
    out = torch.zeros(t["ids"].numel(), t["b"].shape[1], dtype=torch.float64)
    for s, g in enumerate(t["ids"].tolist()):
        if g >= 0:
            z = t["a"][g].double() @ cut(t["x"][s].float(), x_planes).double()
            z = cut(z.float(), z_planes)
            out[s] = (t["b"][g].double() @ z.double()) * t["scale"][g].double()
    return out.float().to(y_dtype)


def router_exact(g, T, E, H, x_dtype, kind):
    """x, w (fp32), the exact logits and how far a result may be off them. `w`: one-hot rows of
    x pick 24-bit values of w; `x`: the other way round (fp32 x); `rest`: rows of x take the
    first two planes of a value of w away from it."""
    x, w = torch.zeros(T, H), torch.zeros(E, H)
    if kind == "w":
        w = full_floats(g, E, H)
        at = torch.randint(0, H, (T,), generator=g)
        f = torch.exp2((torch.arange(T) % 9 - 4).float()) * (1 - 2 * (torch.arange(T) % 2)).float()
        x[torch.arange(T), at] = f
        ref = w.t()[at].double() * f.double().view(T, 1)
    elif kind == "x":
        x = full_floats(g, T, H)
        at = torch.randint(0, H, (E,), generator=g)
        f = torch.exp2((torch.arange(E) % 9 - 4).float())
        w[torch.arange(E), at] = f
        ref = x[:, at].double() * f.double()
    else:
        half = H // 2
        where = torch.randperm(H, generator=g)[:2 * half].view(2, half)
        v = full_floats(g, E, half)
        w[:, where[0]] = v
        w[:, where[1]] = cut(v, 2)
        i = torch.randint(0, half, (T,), generator=g)
        x[torch.arange(T), where[0][i]] = 1
        x[torch.arange(T), where[1][i]] = -1
        ref = planes(v)[2].t()[i].double()
    # (as for the adapters, with one sum)
    off = torch.zeros_like(ref)
    if kind == "rest":
        off = (planes(v)[0].abs() == 2).t()[i].double() * 2.0 ** -23
    return dict(x=x.to(x_dtype), w=w, ref=ref, off=off)


def router_emulated(t, x_planes=3, w_planes=3):
    """Logits with x and w cut to so many planes."""
    return (cut(t["x"].float(), x_planes).double() @ cut(t["w"], w_planes).double().t()).float()


# The largest rms error allowed of random fp32 operands, in units of u = 2^-24 times the size
# sqrt(sum of the squares of the products) that a sum of independent terms has. m roundings of
# a growing partial sum add up to sqrt(m / 6) of it: a wave adds 6 products of planes for each
# 32 k, K / 8 k to a wave at least, so 2 at K = 1024 and 4 at 4096; the adapters' second product
# adds less than that again. A product whose third plane is missing is off by some 2^-18.6 of
# itself: 40.
RMS_LIMIT = 16


def router_sizes(x, w):
    return ((x * x) @ (w * w).t()).sqrt()


def lora_sizes(x, a, b):
    """For one adapter: a [r, K], b [N, r]."""
    return (((x * x) @ (a * a).t()) @ (b * b).t()).sqrt()


def rms_error(got, ref, sizes):
    """Root mean square of the error in units of u and of each result's size."""
    return float((((got.double() - ref) / sizes) ** 2).mean().sqrt() * 2.0 ** 24)
