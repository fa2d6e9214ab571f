"""Cases of the two ends of a tensor-parallel training step over p virtual ranks.

Two operators, each in every direction a training step takes:

  dropout   y_r = residual_r + D(x_0 + ... + x_{p-1}), the output of a
            row-parallel layer (all-reduce, dropout, residual addition), its
            reduce-scatter form for sequence-sharded activations, and their
            gradients: D on every rank's own buffer, and D on the way through
            an all-gather.  D keeps element i when word i mod 4 of
            Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random
            numbers: as easy as 1, 2, 3", SC 2011) with key = seed and counter
            = (floor(i / 4), offset) is at least floor(drop * 2^32), and then
            scales it by 1 / (1 - drop); the mask is never stored.
  loss      softmax cross entropy of hidden states against a vocabulary cut
            into p shards (rank r holds rows floor(r V / p) up to
            floor((r + 1) V / p) of the output weight), alone ("loss") and with the gradients of
            the hidden states and of every shard ("step"); the [tokens, V]
            logits are never kept.

``own`` selects between plain torch operations and the framework's calls.
"""

import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
DEVICE = "cuda"
MASKED = -100  # a target outside the vocabulary: no loss, no gradient


def _dropout(name, form, p, n, dtype, drop, residual="none"):
    return {"name": name, "kind": "dropout", "form": form, "p": p, "n": n, "dtype": dtype, "drop": drop,
            "residual": residual}


def _loss(name, form, p, tokens, dim, vocab, dtype, masked=0.0):
    return {"name": name, "kind": "loss", "form": form, "p": p, "tokens": tokens, "dim": dim, "vocab": vocab,
            "dtype": dtype, "masked": masked}


def listed():
    return [
        # one decoding-size activation per rank: the latency of a call
        _dropout("drop_ar_small_bf16_p4", "all_reduce", 4, 4096, "bfloat16", 0.1, "each"),
        # the row-parallel output [8, 2048, 4096] of eight ranks, every rank with its own residual stream
        _dropout("drop_ar_tp_bf16_p8", "all_reduce", 8, 8 * 2048 * 4096, "bfloat16", 0.1, "each"),
        # an odd length in full precision over an odd number of ranks, one residual for all of them
        _dropout("drop_ar_odd_fp32_p5", "all_reduce", 5, 4000037, "float32", 0.25, "shared"),
        # the same layer with the sequence [2048, 4096] sharded over the ranks
        _dropout("drop_rs_seq_fp16_p8", "reduce_scatter", 8, 2048 * 4096, "float16", 0.1, "each"),
        # the gradient of the sequence-sharded form of a batch of four sequences
        _dropout("drop_ag_grad_bf16_p8", "all_gather", 8, 4 * 2048 * 4096, "bfloat16", 0.1),
        # the gradient of the replicated form: every rank masks its own copy
        _dropout("drop_ranks_grad_bf16_p4", "ranks", 4, 2 * 2048 * 4096, "bfloat16", 0.1),
        # one token scored against a GPT-2-size vocabulary at d = 768: one pass over the weights
        _loss("loss_one_token_bf16_p2", "loss", 2, 1, 768, 50257, "bfloat16"),
        # scoring one sequence of 2048 tokens at d = 4096
        _loss("loss_seq_bf16_p8", "loss", 8, 2048, 4096, 50257, "bfloat16"),
        # a fine-tuning step on a short batch whose prompt tokens carry no loss
        _loss("step_short_fp16_p4", "step", 4, 96, 768, 50257, "float16", 0.5),
        # odd sizes everywhere, in full precision
        _loss("step_odd_fp32_p3", "step", 3, 333, 770, 10007, "float32", 0.1),
        # a training step on one sequence at d = 4096
        _loss("step_seq_bf16_p8", "step", 8, 2048, 4096, 32000, "bfloat16"),
        # a training step on four sequences, some positions padded
        _loss("step_batch_bf16_p8", "step", 8, 4 * 2048, 4096, 50257, "bfloat16", 0.1),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        form = rng.choice(["all_reduce", "all_reduce", "reduce_scatter", "all_gather", "ranks"])
        p = rng.randint(1, 8)
        dtype = rng.choice(["float32", "bfloat16", "bfloat16", "float16"])
        top = 8 * 2048 * 4096 // (2 if dtype == "float32" else 1)
        n = _spread(rng, 4096, top)
        if form in ("reduce_scatter", "all_gather"):
            n = max(1, n // p) * p
        residual = rng.choice(["none", "shared", "each"]) if form in ("all_reduce", "ranks") else "none"
        if form == "reduce_scatter":
            residual = rng.choice(["none", "each"])
        return {"kind": "dropout", "form": form, "p": p, "n": n, "dtype": dtype,
                "drop": rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]), "residual": residual}
    form = rng.choice(["loss", "step"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    limit = 8192 * 4096 * 50257 // (8 if dtype == "float32" else 1)
    tokens = _spread(rng, 1, 8192)
    dim = _spread(rng, 64, 4096)
    if rng.random() < 0.6:
        dim = max(64, dim // 64 * 64)
    vocab = _spread(rng, 1000, 131072)
    while tokens * dim * vocab > limit:
        tokens = max(1, tokens // 2)
    return {"kind": "loss", "form": form, "p": rng.randint(1, 8), "tokens": tokens, "dim": dim, "vocab": vocab,
            "dtype": dtype, "masked": rng.choice([0.0, 0.1, 0.5])}


def _shard_bounds(p, vocab):
    return [r * vocab // p for r in range(p + 1)]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        # in pieces, so that making a 16-bit tensor needs no float32 copy of all of it
        out = torch.empty(shape, dtype=dt, device=DEVICE)
        flat = out.view(-1)
        for lo in range(0, flat.numel(), 1 << 26):
            part = flat[lo:lo + (1 << 26)]
            part.copy_(torch.randn(part.numel(), generator=gen, device=DEVICE) * std)
        return out

    p = case["p"]
    state = {"case": case}
    if case["kind"] == "dropout":
        n = case["n"]
        form = case["form"]
        shard = n // p
        length = {"all_reduce": (n, n), "reduce_scatter": (n, shard), "all_gather": (shard, n), "ranks": (n, n)}[form]
        # partial outputs of a row-parallel product: each rank's share of a unit variance
        state["x"] = normal(p, length[0], std=1.0 / math.sqrt(p))
        if case["residual"] == "each":
            state["residual"] = normal(p, length[1])
        elif case["residual"] == "shared":
            state["residual"] = normal(length[1])
        # the seed of the run and the position of this layer and step in it
        state["seed"] = seed * 1000003 + 12345
        state["offset"] = seed * 7919 + 3
        if own:
            state["out"] = torch.empty(p, length[1], dtype=dt, device=DEVICE)
        return state
    tokens, dim, vocab = case["tokens"], case["dim"], case["vocab"]
    bounds = _shard_bounds(p, vocab)
    weight = normal(vocab, dim, std=2.0 / math.sqrt(dim))
    targets = torch.randint(0, vocab, (tokens,), generator=gen, device=DEVICE)
    hidden = normal(tokens, dim)
    # every other token points towards its target, as in a model that has learnt something
    hidden[::2] += (3.0 * weight[targets[::2]].float()).to(dt)
    if case["masked"] > 0:
        targets[torch.rand(tokens, generator=gen, device=DEVICE) < case["masked"]] = MASKED
    state["hidden"] = hidden
    state["weights"] = [weight[bounds[r]:bounds[r + 1]].clone() for r in range(p)]
    state["targets"] = targets
    if case["form"] == "step":
        # the mean over the tokens, with a weight for each as sequence packing gives them
        w = torch.rand(tokens, generator=gen, device=DEVICE) * 0.5 + 0.75
        state["grad_loss"] = (w / tokens).float()
        if case["dtype"] == "float16":
            # float16 gradients are taken of a scaled loss
            state["grad_loss"] *= 1024.0
    if own:
        import collective_communication_reduction_way_amd as rr

        # a training loop keeps its outputs and its workspace
        state["loss"] = torch.empty(tokens, dtype=torch.float32, device=DEVICE)
        state["lse"] = torch.empty(tokens, dtype=torch.float32, device=DEVICE)
        step = case["form"] == "step"
        if step:
            state["dhidden"] = torch.empty_like(hidden)
            state["dweights"] = [torch.empty_like(w) for w in state["weights"]]
        need = rr.vocab_cross_entropy_workspace_size(p, tokens, dim, vocab, dt, grad=step)
        state["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEVICE)
    return state


# ---------------------------------------------------------------------------
# Plain forms.

def _philox_words(blocks, seed, offset):
    """The four 32-bit output words of Philox4x32-10 for an int64 tensor of
    block numbers, each word in an int64 tensor."""
    low = 0xFFFFFFFF
    c0, c1 = blocks & low, (blocks >> 32) & low
    c2 = torch.full_like(blocks, offset & low)
    c3 = torch.full_like(blocks, (offset >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        # 64-bit products wrap, and their bits are those of the unsigned product
        a = c0 * 0xD2511F53
        b = c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _keep(n, seed, offset, drop):
    """Which of the elements 0..n-1 stay."""
    threshold = int(drop * 2 ** 32)
    parts = []
    for lo in range(0, (n + 3) // 4, 1 << 24):
        hi = min(lo + (1 << 24), (n + 3) // 4)
        words = _philox_words(torch.arange(lo, hi, device=DEVICE), seed, offset)
        parts.append(torch.stack([w >= threshold for w in words], dim=1).reshape(-1))
    return torch.cat(parts)[:n]


def _plain_dropout(s):
    case = s["case"]
    x, p, n = s["x"], case["p"], case["n"]
    scale = 1.0 / (1.0 - case["drop"])
    keep = _keep(n, s["seed"], s["offset"], case["drop"])
    res = s.get("residual")
    dt = x.dtype

    def apply(v):
        return torch.where(keep, v * scale, torch.zeros((), device=DEVICE))

    if case["form"] == "ranks":
        out = torch.empty(p, n, dtype=dt, device=DEVICE)
        for r in range(p):
            y = apply(x[r].float())
            if res is not None:
                y = y + (res if res.dim() == 1 else res[r]).float()
            out[r] = y.to(dt)
        return out
    if case["form"] == "all_gather":
        y = apply(x.reshape(-1).float()).to(dt)
        return y.unsqueeze(0).repeat(p, 1)
    total = x[0].float()
    for r in range(1, p):
        total = total + x[r].float()
    y = apply(total)
    if case["form"] == "reduce_scatter":
        y = y.reshape(p, n // p)
        if res is not None:
            y = y + res.float()
        return y.to(dt)
    out = torch.empty(p, n, dtype=dt, device=DEVICE)
    for r in range(p):
        out[r] = (y if res is None else y + (res if res.dim() == 1 else res[r]).float()).to(dt)
    return out


def _plain_loss(s):
    """One shard of the vocabulary at a time, with the running maximum and sum
    of the softmax over the shards."""
    case = s["case"]
    x = s["hidden"].float()
    targets = s["targets"]
    tokens, vocab = case["tokens"], case["vocab"]
    valid = (targets >= 0) & (targets < vocab)
    rows = torch.arange(tokens, device=DEVICE)
    top = torch.full((tokens,), -math.inf, device=DEVICE)
    total = torch.zeros(tokens, device=DEVICE)
    hit = torch.zeros(tokens, device=DEVICE)
    base = 0
    for w in s["weights"]:
        z = x @ w.float().t()
        new = torch.maximum(top, z.amax(dim=1))
        total = total * torch.exp(top - new) + torch.exp(z - new[:, None]).sum(dim=1)
        top = new
        here = valid & (targets >= base) & (targets < base + w.shape[0])
        col = torch.where(here, targets - base, torch.zeros_like(targets))
        hit = torch.where(here, z[rows, col], hit)
        base += w.shape[0]
    lse = top + torch.log(total)
    loss = torch.where(valid, lse - hit, torch.zeros_like(lse))
    if case["form"] == "loss":
        return [loss, lse]
    scale = torch.where(valid, s["grad_loss"], torch.zeros_like(lse))
    dx = torch.zeros_like(x)
    dws = []
    base = 0
    for w in s["weights"]:
        wf = w.float()
        g = torch.exp(x @ wf.t() - lse[:, None])
        here = valid & (targets >= base) & (targets < base + w.shape[0])
        col = torch.where(here, targets - base, torch.zeros_like(targets))
        g[rows, col] -= here.float()
        g *= scale[:, None]
        dx += g @ wf
        dws.append((g.t() @ x).to(w.dtype))
        base += w.shape[0]
    return [loss, lse, dx.to(s["hidden"].dtype)] + dws


# ---------------------------------------------------------------------------
# The framework's calls.

def _own_dropout(s):
    import collective_communication_reduction_way_amd as rr

    case = s["case"]
    x, out = s["x"], s["out"]
    args = dict(drop=case["drop"], seed=s["seed"], offset=s["offset"])
    res = s.get("residual")
    if res is not None and res.dim() == 1:
        res = [res] * case["p"]
    if case["form"] == "all_reduce":
        rr.all_reduce_dropout(x, out, residuals=res, **args)
    elif case["form"] == "reduce_scatter":
        rr.reduce_scatter_dropout(x, out, residuals=res, **args)
    elif case["form"] == "all_gather":
        rr.all_gather_dropout(x, out, **args)
    else:
        rr.dropout(x, out, residuals=res, **args)
    return out


def _own_loss(s):
    import collective_communication_reduction_way_amd as rr

    rr.vocab_cross_entropy(s["hidden"], s["weights"], s["targets"], s["loss"], s["lse"], workspace=s["workspace"])
    if s["case"]["form"] == "loss":
        return [s["loss"], s["lse"]]
    rr.vocab_cross_entropy_grad(s["hidden"], s["weights"], s["targets"], s["lse"], s["grad_loss"], s["dhidden"],
                                s["dweights"], workspace=s["workspace"])
    return [s["loss"], s["lse"], s["dhidden"]] + s["dweights"]


def run(state):
    if state["case"]["kind"] == "dropout":
        return _own_dropout(state) if own else _plain_dropout(state)
    return _own_loss(state) if own else _plain_loss(state)


# ---------------------------------------------------------------------------

def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    p = case["p"]
    if case["kind"] == "dropout":
        n = case["n"]
        reads, writes = {"all_reduce": (p * n, p * n), "reduce_scatter": (p * n, n), "all_gather": (n, p * n),
                         "ranks": (p * n, p * n)}[case["form"]]
        if case["residual"] == "each":
            reads += writes
        elif case["residual"] == "shared":
            reads += n
        # a multiplication for each kept element, and the additions of the sum and the residual
        return {"bytes": (reads + writes) * size, "flops": reads}
    t, d, v = case["tokens"], case["dim"], case["vocab"]
    inputs = (t * d + v * d) * size + 8 * t
    if case["form"] == "loss":
        return {"bytes": inputs + 8 * t, "flops": 2 * t * d * v}
    # the logits, and the two products of their gradient
    return {"bytes": inputs + 4 * t + (t * d + v * d) * size + 8 * t, "flops": 6 * t * d * v}


# ---------------------------------------------------------------------------
# The definition in 64 bits.

def _exact_mask(n, seed, offset, drop):
    """The kept elements, with the generator's products formed from 16-bit
    halves, so that no intermediate leaves 63 bits."""
    threshold = math.floor(drop * 4294967296.0)
    blocks = torch.arange((n + 3) // 4, device=DEVICE, dtype=torch.int64)
    state = [blocks % 2 ** 32, blocks // 2 ** 32, torch.zeros_like(blocks) + offset % 2 ** 32,
             torch.zeros_like(blocks) + (offset // 2 ** 32) % 2 ** 32]
    key = [seed % 2 ** 32, (seed // 2 ** 32) % 2 ** 32]

    def product(word, constant):
        low = word * (constant % 65536)
        mid = word * (constant // 65536) + low // 65536
        return mid // 65536, (mid % 65536) * 65536 + low % 65536

    for r in range(10):
        hi0, lo0 = product(state[0], 3528531795)
        hi1, lo1 = product(state[2], 3449720151)
        state = [hi1 ^ state[1] ^ ((key[0] + r * 2654435769) % 2 ** 32), lo1,
                 hi0 ^ state[3] ^ ((key[1] + r * 3144134277) % 2 ** 32), lo0]
    word = torch.stack(state, dim=1).reshape(-1)[:n]
    return ~(word < threshold)


def _exact_dropout(s):
    case = s["case"]
    p, n = case["p"], case["n"]
    factor = _exact_mask(n, s["seed"], s["offset"], case["drop"]).double() / (1.0 - float(case["drop"]))
    res = s.get("residual")
    out_len = n // p if case["form"] == "reduce_scatter" else n
    add = None
    if res is not None:
        add = res if res.dim() == 2 else res.unsqueeze(0).expand(p, out_len)
    if case["form"] == "ranks":
        y = s["x"].double() * factor
    elif case["form"] == "all_gather":
        y = (s["x"].double().reshape(1, n) * factor).expand(p, n)
    elif case["form"] == "reduce_scatter":
        y = (s["x"].double().sum(dim=0) * factor).reshape(p, out_len)
    else:
        y = (s["x"].double().sum(dim=0) * factor).unsqueeze(0).expand(p, n)
    return y.clone() if add is None else y + add.double()


def _exact_loss(s):
    """The softmax of whole rows, a block of tokens at a time."""
    case = s["case"]
    tokens, vocab = case["tokens"], case["vocab"]
    weight = torch.cat(s["weights"]).double()
    hidden = s["hidden"].double()
    step = case["form"] == "step"
    block = max(1, (1 << 27) // vocab)
    losses, sums, dx = [], [], []
    dw = torch.zeros_like(weight) if step else None
    for lo in range(0, tokens, block):
        x = hidden[lo:lo + block]
        t = s["targets"][lo:lo + block]
        counted = (t >= 0) & (t < vocab)
        onehot = torch.zeros(x.shape[0], vocab, dtype=torch.float64, device=DEVICE)
        onehot.scatter_(1, t.clamp(0, vocab - 1)[:, None], counted.double()[:, None])
        logits = torch.mm(x, weight.t())
        lse = torch.logsumexp(logits, dim=1)
        sums.append(lse)
        losses.append((lse - (logits * onehot).sum(dim=1)) * counted.double())
        if step:
            g = (torch.exp(logits - lse[:, None]) - onehot) * (s["grad_loss"][lo:lo + block].double()
                                                              * counted.double())[:, None]
            dx.append(torch.mm(g, weight))
            dw += torch.mm(g.t(), x)
    out = [torch.cat(losses), torch.cat(sums)]
    if step:
        bounds = _shard_bounds(case["p"], vocab)
        out.append(torch.cat(dx))
        out += [dw[bounds[r]:bounds[r + 1]] for r in range(case["p"])]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_dropout(s) if case["kind"] == "dropout" else _exact_loss(s)
