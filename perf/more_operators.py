"""Operators around the Muon step: what is measured, their plain forms and their values in 64 bits.

Operators (include/ob_adam.h documents the calls):
  clip    ob_tensor_norms and ob_clip_grads: the norm of every tensor of a list and of all together, and the gradients times
          the factor that clips them (all by the global norm, or each by its own), written out in another or the same type.
  matmul  ob_matmul: D = alpha A B + beta C in 16-bit operands with fp32 sums; batches, four layouts, symmetric results.
  muon    ob_muon_step: momentum, five iterations towards the nearest orthogonal matrix, decay and update, over a list of
          matrices; with `clip` after the global gradient norm.

Layout: tensors are views into flat buffers and start at multiples of 256 elements; the gaps hold zeros, which every
operator maps to zeros.  Where a case says `packed`, gradients follow each other without gaps, as in one communication bucket.
Matrices of one shape lie behind each other, so that the plain form takes them as one batch.
"""
import math
import random

import torch

own = False

LR, WD, MU, EPS, MAX_NORM = 2e-4, 0.1, 0.95, 1e-7, 1.0
ALPHA, BETA = 0.75, 0.9
COEFFS = (3.4445, -4.7750, 2.0315)
ITERATIONS = 5
BLOCK = 256
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    def clip(name, n, tensors, g="f32", out="f32", max_norm=1.0, kind="2", per_tensor=False, packed=False, loss_scale=1.0):
        return dict(name=name, op="clip", n=n, tensors=tensors, g=g, out=out, max_norm=max_norm, kind=kind,
                    per_tensor=per_tensor, packed=packed, loss_scale=loss_scale)

    def matmul(name, m, n, k, batch=1, a="bf16", out="bf16", layout="nn", residual=False, symmetric=False):
        return dict(name=name, op="matmul", batch=batch, m=m, n=n, k=k, a=a, out=out, layout=layout, residual=residual,
                    symmetric=symmetric)

    def muon(name, shapes, p="f32", g="f32", master=False, clip=False, nesterov=True):
        return dict(name=name, op="muon", shapes=shapes, p=p, g=g, master=master, clip=clip, nesterov=nesterov)

    return [
        # the gradients of one layer's adapters: a few tiny tensors, where latency is everything
        clip("clip-small", 20_011, 12, max_norm=0.05),
        # a 110M-parameter encoder under a loss scale: fp16 gradients in one bucket, unscaled into fp32, each tensor clipped alone
        clip("clip-110M-each", 108_891_648, 197, g="f16", max_norm=0.5, per_tensor=True, packed=True, loss_scale=1024.0),
        # a billion bf16 gradients, clipped by the global norm before two optimizers step them
        clip("clip-1B", 1_000_000_007, 290, g="bf16", out="bf16"),
        # one small product, where the launch is everything
        matmul("matmul-small", 96, 200, 136, a="f16", out="f32", residual=True),
        # odd sizes: no row starts at a multiple of 16 bytes
        matmul("matmul-odd", 1531, 1003, 777, out="f32", residual=True, layout="nt"),
        # the largest: an ordinary product, second operand as it lies, residual of the same type
        matmul("matmul-8192", 8192, 8192, 8192, residual=True),
        # statistics of one gradient: its rows' products, added to what was there; a long sum
        matmul("gram-4096", 4096, 4096, 11008, out="f32", layout="nt", residual=True, symmetric=True),
        # adapters: small odd matrices
        muon("muon-small", "4*64x64,3*100x37,1*5x129", clip=True),
        # the attention projections of a 12-layer encoder, fp32, clipped
        muon("muon-encoder", "48*768x768", clip=True),
        # experts: two tensors of 32 matrices each, bf16 without a master copy, one of them tall
        muon("muon-experts", "1*32x512x1408,1*32x1408x512", p="bf16", g="bf16"),
        # one layer of a 7B-parameter decoder, mixed precision with fp32 masters
        muon("muon-7B-layer", "4*4096x4096,2*11008x4096,1*4096x11008", p="bf16", g="bf16", master=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["clip", "matmul", "matmul", "muon"])
    if op == "clip":
        n = _log(rng, 1e4, 6e8) | 1
        return dict(op=op, n=n, tensors=max(1, min(n // 600, _log(rng, 1, 300))), g=rng.choice(list(DT)), out=rng.choice(list(DT)),
                    max_norm=10.0 ** rng.uniform(-2, 1), kind=rng.choice(["2", "2", "max"]), per_tensor=rng.random() < 0.4,
                    packed=n < 1.2e8 and rng.random() < 0.4, loss_scale=rng.choice([1.0, 256.0]))
    if op == "matmul":
        m, n, k = (_log(rng, 16, 8192) for _ in range(3))
        if rng.random() < 0.6:  # the sizes of real layers: multiples of 64
            m, n, k = (max(64, x // 64 * 64) for x in (m, n, k))
        symmetric = rng.random() < 0.3
        n = m if symmetric else n
        batch = rng.choice([1, 1, 1, 4, 16])
        if m * n * k * batch > 4e10:
            batch = 1
        return dict(op=op, batch=batch, m=m, n=n, k=k, a=rng.choice(["bf16", "f16"]), out=rng.choice(["bf16", "f16", "f32"]),
                    layout=rng.choice(["nt", "tn"]) if symmetric else rng.choice(["nn", "nt", "tn", "tt"]),
                    residual=rng.random() < 0.6, symmetric=symmetric)
    p = rng.choice(["f32", "bf16"])
    shapes, spent = [], 0.0
    for _ in range(rng.choice([1, 2, 3])):
        count, r, c, e = rng.choice([1, 2, 6]), _log(rng, 16, 4096), _log(rng, 16, 4096), rng.choice([1, 1, 8])
        if rng.random() < 0.6:
            r, c = max(32, r // 32 * 32), max(32, c // 32 * 32)
        cost = count * e * 2.0 * min(r, c) ** 2 * max(r, c)
        if shapes and spent + cost > 2e12:
            continue
        if cost > 2e12:
            count = e = 1
        spent += cost
        shapes.append("%d*%s%dx%d" % (count, "%dx" % e if e > 1 else "", r, c))
    return dict(op=op, shapes=",".join(shapes), p=p, g=rng.choice([p, "f32"]), master=p != "f32" and rng.random() < 0.6,
                clip=rng.random() < 0.5, nesterov=rng.random() < 0.8)


# ---------------------------------------------------------------------------------------------------
# the lists: sizes and offsets (the same for every seed)
# ---------------------------------------------------------------------------------------------------

def _sizes(case):
    n, T = case["n"], case["tensors"]
    r = random.Random("%d/%d" % (n, T))
    w = [(1e-4 if j % 3 == 1 else 1.0) * 8.0 ** r.random() for j in range(T)]  # matrices, with a small vector between
    sizes = [max(1, int(n * x / sum(w))) for x in w]
    sizes[0] += max(0, n - sum(sizes))
    return sizes


def _up(n):
    return -(-n // BLOCK) * BLOCK


def _offsets(sizes):
    off = [0]
    for s in sizes:
        off.append(off[-1] + _up(s))
    return off


def _shapes(case):
    """(count, shape) of each kind of matrix; a shape has two dimensions, or three for a batch in one tensor."""
    kinds = []
    for kind in case["shapes"].split(","):
        count, shape = kind.split("*")
        kinds.append((int(count), tuple(int(x) for x in shape.split("x"))))
    return kinds


def work(case):
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": float(n) * (BYTES[case["g"]] + BYTES[case["out"]]), "flops": 3.0 * n}
    if case["op"] == "matmul":
        b, m, n, k = (case[x] for x in ("batch", "m", "n", "k"))
        a, o = BYTES[case["a"]], BYTES[case["out"]]
        by = a * m * k + (0 if case["symmetric"] else a * k * n) + o * m * n * (2 if case["residual"] else 1)
        return {"bytes": float(b * by), "flops": float(b * k * (m * (m + 1) if case["symmetric"] else 2 * m * n))}
    by = fl = 0.0
    per = BYTES[case["g"]] + 8 + (8 + BYTES[case["p"]] if case["master"] else 2 * BYTES[case["p"]])
    for count, shape in _shapes(case):
        c = count * math.prod(shape[:-2])
        r, k = sorted(shape[-2:])
        by += c * r * k * per
        fl += c * float(ITERATIONS) * (r * (r + 1) * k + r * r * (r + 1) + 2 * r * r * k)  # two of three products are symmetric
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------

def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def prepare(case, seed):
    gen = torch.Generator(device=_dev()).manual_seed(seed)
    return {"clip": _prepare_clip, "matmul": _prepare_matmul, "muon": _prepare_muon}[case["op"]](case, gen)


def _prepare_clip(case, gen):
    dev = gen.device
    sizes = _sizes(case)
    off = _offsets(sizes)
    T, nb = len(sizes), off[-1] // BLOCK
    st = {"case": dict(case), "sizes": sizes, "off": off}
    blocks = torch.tensor([o // BLOCK for o in off], dtype=torch.int64, device=dev)
    tensor_of = torch.repeat_interleave(torch.arange(T, device=dev), blocks[1:] - blocks[:-1])
    left = torch.tensor(sizes, device=dev)[tensor_of] - (torch.arange(nb, device=dev) - blocks[:-1][tensor_of]) * BLOCK
    valid = torch.arange(BLOCK, device=dev)[None, :] < left[:, None]
    # per 256 elements a magnitude of its own, two decades wide; a few rows without any gradient
    sigma = 1e-4 * torch.exp(1.5 * torch.randn(nb, 1, generator=gen, device=dev))
    sigma[torch.rand(nb, 1, generator=gen, device=dev) < 0.01] = 0
    g = torch.randn(nb, BLOCK, generator=gen, device=dev).mul_(sigma * case["loss_scale"]).mul_(valid).to(DT[case["g"]])
    if case["packed"]:
        st["g"] = torch.cat([g[valid], g.new_zeros(1)])
        # places of the rows' elements in the bucket; the gaps go to the zero behind it
        st["at"] = torch.where(valid.view(-1), valid.view(-1).cumsum(0) - 1, st["g"].numel() - 1)
        starts = [0]
        for s in sizes:
            starts.append(starts[-1] + s)
        st["grads"] = [st["g"][a:a + s] for a, s in zip(starts, sizes)]
    else:
        st["g"] = g
        st["grads"] = [g.view(-1)[o:o + s] for o, s in zip(off, sizes)]
    st["tensor_of"] = tensor_of
    st["out"] = torch.zeros(nb, BLOCK, dtype=DT[case["out"]], device=dev)
    st["outs"] = [st["out"].view(-1)[o:o + s] for o, s in zip(off, sizes)]
    st["norms"] = torch.zeros(T + 1, device=dev)
    if own:  # the list's handle and workspace, made once by a program
        import adam_ob_compress_amd as ob

        st["list"] = ob.ob_tensors_create(sizes, DT[case["g"]], DT[case["out"]])
        st["work"] = torch.empty(ob.ob_tensor_norms_workspace(st["list"]), dtype=torch.uint8, device=dev)
    return st


def _matrix(gen, batch, rows, cols, transposed, dtype, scale=1.0):
    """A batch of matrices, [rows, cols] as the product sees them; transposed: they lie by columns."""
    shape = (batch, cols, rows) if transposed else (batch, rows, cols)
    x = torch.randn(shape, generator=gen, device=gen.device).mul_(scale).to(dtype)
    return x.transpose(1, 2) if transposed else x


def _prepare_matmul(case, gen):
    b, m, n, k = (case[x] for x in ("batch", "m", "n", "k"))
    dt = DT[case["a"]]
    # rows whose products with each other are of the order of one, as gradients' and weights' are
    a = _matrix(gen, b, m, k, case["layout"][0] == "t", dt, k ** -0.25)
    bb = a.transpose(1, 2) if case["symmetric"] else _matrix(gen, b, k, n, case["layout"][1] == "t", dt, k ** -0.25)
    c = None
    if case["residual"]:
        c = torch.randn(b, m, n, generator=gen, device=gen.device)
        c = ((c + c.transpose(1, 2)) * 0.5 if case["symmetric"] else c).to(DT[case["out"]]).contiguous()
    out = torch.zeros(b, m, n, dtype=DT[case["out"]], device=gen.device)
    if b == 1:
        a, bb, out, c = a[0], bb[0], out[0], None if c is None else c[0]
    return {"case": dict(case), "a": a, "b": bb, "c": c, "out": out}


def _gradients(gen, count, shape):
    """Matrices with a few strong directions over noise whose rows and columns differ in magnitude."""
    r, c = shape[-2:]
    n = count * math.prod(shape[:-2])
    rand = lambda *s: torch.randn(n, *s, generator=gen, device=gen.device)  # noqa: E731
    x = rand(r, c) * torch.exp(0.5 * rand(r, 1)) * torch.exp(0.5 * rand(1, c))
    rank = max(1, min(r, c) // 32)
    x += (rand(r, rank) * torch.arange(1, rank + 1, device=gen.device) ** -0.5) @ rand(rank, c)
    return x.mul_(1e-3)


def _prepare_muon(case, gen):
    dev = gen.device
    kinds = _shapes(case)
    st = {"case": dict(case), "kinds": kinds}
    sizes, starts = [], []
    for count, shape in kinds:
        starts.append(sum(_up(s) for s in sizes))
        sizes += [math.prod(shape)] * count
    N = sum(_up(s) for s in sizes)

    def buffer(dtype):
        """A flat buffer, its views by kind and by tensor."""
        flat = torch.zeros(N, dtype=dtype, device=dev)
        by_kind = [flat.as_strided((count, *shape), (_up(math.prod(shape)), *[math.prod(shape[j + 1:]) for j in range(len(shape))]), at)
                   for (count, shape), at in zip(kinds, starts)]
        return flat, by_kind, [x for stack in by_kind for x in stack]

    st["g"], g_kinds, st["grads"] = buffer(DT[case["g"]])
    st["p"], p_kinds, st["params"] = buffer(DT[case["p"]])
    st["m"], m_kinds, _ = buffer(torch.float32)
    st["master"], w_kinds, _ = buffer(torch.float32) if case["master"] else (None, p_kinds, None)
    for (count, shape), g, m, p, w in zip(kinds, g_kinds, m_kinds, p_kinds, w_kinds):
        fresh = _gradients(gen, count, shape).view(count, *shape)
        g.copy_(fresh)
        m.copy_(fresh.mul_(0.2)).add_(_gradients(gen, count, shape).view(count, *shape), alpha=0.2)  # what earlier steps left
        w.copy_(torch.randn(count, *shape, generator=gen, device=dev).mul_(0.02))
        p.copy_(w)
    st["stacks"] = list(zip(kinds, g_kinds, m_kinds, p_kinds, w_kinds))
    if own:  # handles and workspace, made once by a program
        import adam_ob_compress_amd as ob

        st["list"] = ob.ob_tensors_create(sizes, DT[case["g"]], DT[case["p"]])
        st["plan"] = ob.ob_muon_create(st["list"], [tuple(x.shape) for x in st["params"]])
        st["work"] = torch.empty(st["plan"].workspace_bytes, dtype=torch.uint8, device=dev)
        st["hp"] = ob.muon_hparams(lr=LR, momentum=MU, weight_decay=WD, eps=EPS, nesterov=case["nesterov"],
                                   iterations=ITERATIONS, scale=ob.OB_MUON_MATCH_RMS)
        st["ctl"] = ob.control_create(dev) if case["clip"] else None
    return st


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"clip": _own_clip, "matmul": _own_matmul, "muon": _own_muon}[op](state)
    return {"clip": _plain_clip, "matmul": _plain_matmul, "muon": _plain_muon}[op](state)


def _own_clip(st):
    import adam_ob_compress_amd as ob

    c = st["case"]
    ob.ob_tensor_norms(st["list"], st["grads"], st["norms"], g_mult=1.0 / c["loss_scale"],
                       kind=ob.OB_NORM_MAX if c["kind"] == "max" else ob.OB_NORM_2, workspace=st["work"])
    ob.ob_clip_grads(st["list"], st["grads"], st["norms"], c["max_norm"], g_mult=1.0 / c["loss_scale"], out=st["outs"],
                     per_tensor=c["per_tensor"])
    return {"norms": st["norms"], "out": st["out"]}


def _own_matmul(st):
    import adam_ob_compress_amd as ob

    c = st["case"]
    ob.ob_matmul(st["a"], st["b"], st["out"], alpha=ALPHA, beta=BETA if c["residual"] else 0.0, c=st["c"], symmetric=c["symmetric"])
    return {"out": st["out"]}


def _own_muon(st):
    import adam_ob_compress_amd as ob

    ob.ob_muon_step(st["plan"], st["grads"], st["params"], st["m"], st["hp"], st["work"], master=st["master"], control=st["ctl"],
                    norm=(1.0, MAX_NORM) if st["case"]["clip"] else None)
    out = {"norm": st["ctl"].view(torch.float32)[0]} if st["case"]["clip"] else {}
    return out | _muon_result(st)


def _muon_result(st):
    return {"p": st["p"], "m": st["m"]} | ({} if st["master"] is None else {"master": st["master"]})


def _plain_clip(st):
    c, mult = st["case"], 1.0 / st["case"]["loss_scale"]
    g = (st["g"][st["at"]].view(-1, BLOCK) if c["packed"] else st["g"]).float()
    T = len(st["sizes"])
    if c["kind"] == "max":
        rows = g.abs().amax(1).double()
        each = torch.zeros(T, dtype=torch.float64, device=g.device).index_reduce_(0, st["tensor_of"], rows, "amax")
        norms = torch.cat([each, each.amax().view(1)]) * mult
    else:
        rows = g.square().sum(1, dtype=torch.float64)
        each = torch.zeros(T, dtype=torch.float64, device=g.device).index_add_(0, st["tensor_of"], rows)
        norms = torch.cat([each, each.sum().view(1)]).sqrt() * mult
    st["norms"].copy_(norms)
    factor = (mult * torch.clamp(c["max_norm"] / (norms + 1e-6), max=1.0)).float()
    st["out"].copy_(g * (factor[st["tensor_of"]][:, None] if c["per_tensor"] else factor[T]))
    return {"norms": st["norms"], "out": st["out"]}


def _plain_matmul(st):
    d = (st["a"].float() @ st["b"].float()).mul_(ALPHA)
    if st["c"] is not None:
        d.add_(st["c"].float(), alpha=BETA)
    st["out"].copy_(d)
    return {"out": st["out"]}


def _plain_muon(st):
    case, out, factor = st["case"], {}, 1.0
    if case["clip"]:
        norm = st["g"].float().square().sum(dtype=torch.float64).sqrt()
        out["norm"] = norm.float()
        factor = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0).float()
    for (_, shape), g, m, p, w in st["stacks"]:
        g = g.float() * factor
        m.mul_(MU).add_(g * (1.0 - MU))
        u = g * (1.0 - MU) + m * MU if case["nesterov"] else m
        r, k = shape[-2:]
        x = u / (u.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
        x = x.transpose(-2, -1) if r > k else x
        for _ in range(ITERATIONS):
            gram = x @ x.transpose(-2, -1)
            x = COEFFS[0] * x + (COEFFS[1] * gram + COEFFS[2] * (gram @ gram)) @ x
        x = x.transpose(-2, -1) if r > k else x
        w32 = w.float() * (1.0 - LR * WD) - (LR * 0.2 * math.sqrt(max(r, k))) * x
        w.copy_(w32)
        if p is not w:
            p.copy_(w32)
    return out | _muon_result(st)


# ---------------------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"clip": _exact_clip, "matmul": _exact_matmul, "muon": _exact_muon}[case["op"]](case, st)


def _exact_clip(case, st):
    grads = [g.double() / case["loss_scale"] for g in st["grads"]]
    if case["kind"] == "max":
        each = torch.stack([g.abs().max() for g in grads])
        total = each.max()
    else:
        each = torch.stack([torch.linalg.vector_norm(g) for g in grads])
        total = torch.linalg.vector_norm(each)
    out = torch.zeros(st["out"].numel(), dtype=torch.float64, device=total.device)
    for j, (g, o) in enumerate(zip(grads, st["off"])):
        norm = float(each[j] if case["per_tensor"] else total)
        out[o:o + g.numel()] = g * min(1.0, case["max_norm"] / (norm + 1e-6))
    return {"norms": torch.cat([each, total.view(1)]), "out": out.view(st["out"].shape)}


def _exact_matmul(case, st):
    d = torch.zeros(st["out"].shape, dtype=torch.float64, device=st["out"].device)
    step = 2048  # the sum in parts, so that the operands are widened piece by piece
    for k in range(0, case["k"], step):
        d += torch.matmul(st["a"][..., k:k + step].double(), st["b"][..., k:k + step, :].double())
    d *= ALPHA
    if st["c"] is not None:
        d += BETA * st["c"].double()
    return {"out": d}


def _exact_muon(case, st):
    out, factor = {}, 1.0
    if case["clip"]:
        norm = math.sqrt(sum(float(g.double().pow(2).sum()) for g in st["grads"]))
        out["norm"] = torch.tensor(norm, dtype=torch.float64)
        factor = min(1.0, MAX_NORM / (norm + 1e-6))
    m_all, p_all = st["m"].double(), (st["p"] if st["master"] is None else st["master"]).double()
    at = 0
    for g in st["grads"]:
        size, shape = g.numel(), g.shape
        m = MU * m_all[at:at + size].view(shape) + (1.0 - MU) * factor * g.double()
        m_all[at:at + size] = m.reshape(-1)
        u = MU * m + (1.0 - MU) * factor * g.double() if case["nesterov"] else m
        tall = shape[-2] > shape[-1]
        x = u / (torch.linalg.matrix_norm(u, keepdim=True) + EPS)
        for _ in range(ITERATIONS):  # x (a + b x'x + c (x'x)^2) from the smaller side
            gram = x.mT @ x if tall else x @ x.mT
            odd = torch.eye(gram.shape[-1], dtype=x.dtype, device=x.device) * COEFFS[0] + COEFFS[1] * gram + COEFFS[2] * gram @ gram
            x = x @ odd if tall else odd @ x
        p = p_all[at:at + size].view(shape)
        p_all[at:at + size] = (p - LR * WD * p - LR * 0.2 * math.sqrt(max(shape[-2:])) * x).reshape(-1)
        at += _up(size)
    out |= {"p": p_all, "m": m_all}
    return out | ({} if st["master"] is None else {"master": p_all})
