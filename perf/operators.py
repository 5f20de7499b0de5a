"""What the attention operators with learned score terms cost, and what they answer.

Two operators over a causal CSR block schedule (row i lists the key blocks that query block i
visits; a query sees the listed blocks' keys up to its own token):

* biased attention: softmax(scale q.k + bias[head, bucket(q - k)]) V, the distances q - k sorted
  into buckets by their ascending starts (single distances up to half of them, then borders in
  geometric steps up to a largest distance);
* differential attention: (softmax(scale q1.k1) - lambda softmax(scale q2.k2)) V, where q1 | q2 and
  k1 | k2 are the halves of the head dimension and
  lambda = exp(lq1.lk1) - exp(lq2.lk2) + lambda_init, learned per head or shared by the heads.

Each in three forms: "fwd" (the output), "train" (the output and the gradients of every input for
an upstream gradient) and "decode" (one new token per sequence against a key/value cache; row b of
the schedule lists the cache blocks that sequence b's token visits, its own token is the last of
its `length`).
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    fwd = {"form": "fwd", "block": 64, "schedule": "topology", "sink": 1, "radius": 1, "topk": 2}
    bias = {"op": "biased", "buckets": 32, "max_distance": 128}
    diff = {"op": "differential", "lambda_heads": "each"}
    return [
        # one short sequence of one head: latency counts
        {"name": "biased fwd s1024", **fwd, **bias, "B": 1, "H": 1, "S": 1024, "D": 64, "dtype": "f16"},
        # a batch of prompts through a sparse schedule
        {"name": "biased fwd b4h16s8192", **fwd, **bias, "B": 4, "H": 16, "S": 8192, "D": 64, "dtype": "f16",
         "radius": 2, "topk": 4},
        # a ragged prompt through the dense causal schedule, buckets that reach far
        {"name": "biased fwd dense s1999", **fwd, **bias, "B": 1, "H": 8, "S": 1999, "D": 128, "dtype": "bf16",
         "schedule": "dense", "buckets": 64, "max_distance": 1024},
        # a training step on short ragged sequences
        {"name": "biased train s1000", **fwd, **bias, "form": "train", "B": 2, "H": 8, "S": 1000, "D": 64,
         "dtype": "f16", "schedule": "dense"},
        # a training step on a long sequence
        {"name": "biased train h32s32768", **fwd, **bias, "form": "train", "B": 1, "H": 32, "S": 32768, "D": 128,
         "dtype": "bf16", "sink": 2, "radius": 4, "topk": 8},
        # the next token of one sequence, and of a full batch
        {"name": "biased decode b1s1000", **fwd, **bias, "form": "decode", "B": 1, "H": 16, "S": 1000, "D": 64,
         "dtype": "f16", "schedule": "dense"},
        {"name": "biased decode b16s8192", **fwd, **bias, "form": "decode", "B": 16, "H": 32, "S": 8192, "D": 128,
         "dtype": "bf16", "schedule": "dense"},
        {"name": "diff fwd s1024", **fwd, **diff, "B": 1, "H": 1, "S": 1024, "D": 64, "dtype": "f16"},
        {"name": "diff fwd b4h16s8192", **fwd, **diff, "B": 4, "H": 16, "S": 8192, "D": 64, "dtype": "f16",
         "radius": 2, "topk": 4, "lambda_heads": "shared"},
        {"name": "diff train s1000", **fwd, **diff, "form": "train", "B": 2, "H": 8, "S": 1000, "D": 128,
         "dtype": "bf16", "schedule": "dense"},
        {"name": "diff train h32s32768", **fwd, **diff, "form": "train", "B": 1, "H": 32, "S": 32768, "D": 128,
         "dtype": "bf16", "sink": 2, "radius": 4, "topk": 8},
        {"name": "diff decode b16s8192", **fwd, **diff, "form": "decode", "B": 16, "H": 32, "S": 8192, "D": 128,
         "dtype": "bf16", "schedule": "topology", "sink": 2, "radius": 8, "topk": 32, "lambda_heads": "shared"},
    ]


def _visited(case):
    """An upper bound of the (lane, query block, key block) visits, in blocks of 64 tokens."""
    nb = -(-case["S"] // 64)
    per = case["sink"] + case["radius"] + 1 + case["topk"]
    if case["schedule"] == "topology":
        per *= max(1, case["block"] // 64)
    else:
        per = nb
    rows = 1 if case["form"] == "decode" else nb
    return case["B"] * case["H"] * rows * min(per, nb)


def draw(rng):
    most = _visited(listed()[4])
    while True:
        form = rng.choice(["fwd", "train", "decode"])
        case = {"op": rng.choice(["biased", "differential"]), "form": form,
                "B": rng.randint(1, 16 if form == "decode" else 4), "H": rng.choice([1, 2, 3, 5, 8, 12, 16, 32]),
                "S": int(round(2 ** rng.uniform(4 if form == "train" else 0, 13 if form == "decode" else 15))), "D": rng.choice([64, 128]),
                "dtype": rng.choice(["f16", "bf16"]), "block": rng.choice([64, 128] if form == "train" else [32, 64, 128]),
                "schedule": rng.choice(["topology", "dense", "random"]), "sink": rng.randint(0, 2),
                "radius": rng.randint(0, 4), "topk": rng.randint(0, 8)}
        if case["op"] == "biased":
            case["buckets"] = rng.choice([2, 16, 32, 64, 128])
            case["max_distance"] = case["buckets"] * rng.choice([2, 4, 16])
        else:
            case["lambda_heads"] = rng.choice(["each", "shared"])
        lanes, nb = case["B"] * case["H"], -(-case["S"] // 64)
        if form == "decode":
            if lanes * case["S"] <= 16 * 32 * 8192:
                return case
        elif _visited(case) <= most and lanes * nb * 64 * case["D"] <= 32 * 32768 * 128:
            if case["schedule"] == "topology" or lanes * nb * nb <= 1 << 16:
                return case


def _bucket_starts(n, most):
    """Starts of n buckets of distances: 0, 1, .., n/2 - 1, then the smallest integers d with
    d / h >= (most / h) ** (i / m), h = n/2, m = n - h, i = 0 .. m - 1 (integer arithmetic)."""
    h = n // 2
    m = n - h
    starts, d = list(range(h)), h
    for i in range(m):
        while d ** m * h ** i < most ** i * h ** m:
            d += 1
        starts.append(d)
    return starts


def _rows(case, rng):
    """The key blocks of each row of the schedule: sink blocks, a local window and the topk blocks of
    largest salience (drawn here), every block, or a random choice that leaves some rows empty. For
    "decode" a row per sequence, made of the blocks below its length; also the lengths."""
    block, S = case["block"], case["S"]
    nb = -(-S // block)
    lengths = None
    if case["form"] == "decode":  # ragged lengths up to the capacity, the first one full
        lengths = [S if b == 0 else rng.randint(S // 2, S) for b in range(case["B"])]
        if case["schedule"] == "random" and case["B"] > 1:
            lengths[-1] = 0
        last = [-(-n // block) - 1 for n in lengths]
    else:
        last = list(range(nb))
    salience = [rng.random() for _ in range(nb)]
    order = sorted(range(nb), key=lambda j: -salience[j])
    rows = []
    for i in last:
        if case["schedule"] == "dense":
            row = range(i + 1)
        elif case["schedule"] == "random":
            row = [] if rng.random() < 0.1 else [j for j in range(i + 1) if rng.random() < 0.4]
        else:
            row = set(range(min(case["sink"], i + 1))) | set(range(max(0, i - case["radius"]), i + 1))
            n = 0
            for j in order:
                if n == case["topk"]:
                    break
                if j <= i:
                    row.add(j)
                    n += 1
            row = sorted(row)
        rows.append(list(row))
    return rows, lengths


def prepare(case, seed):
    rng = random.Random(seed)
    rows, lengths = _rows(case, rng)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, H, S, D = case["B"], case["H"], case["S"], case["D"]

    def normal(*shape, std=1.0, grad=False):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt).requires_grad_(grad)

    train, decode = case["form"] == "train", case["form"] == "decode"
    ptr = [0]
    for r in rows:
        ptr.append(ptr[-1] + len(r))
    s = {"op": case["op"], "form": case["form"], "block": case["block"], "most": max(1, max(map(len, rows))),
         "row_ptr": torch.tensor(ptr, dtype=torch.int32, device="cuda"),
         "col_idx": torch.tensor([j for r in rows for j in r] or [0], dtype=torch.int32, device="cuda"),
         "Q": normal(*((B, H, D) if decode else (B, H, S, D)), grad=train),
         "K": normal(B, H, S, D, grad=train), "V": normal(B, H, S, D, grad=train)}
    if train:
        s["dO"] = normal(B, H, S, D)
    if decode:
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if case["op"] == "biased":
        s["bias"] = normal(H, case["buckets"], grad=train)
        s["starts"] = _bucket_starts(case["buckets"], case["max_distance"])
        s["starts_on_gpu"] = torch.tensor(s["starts"], dtype=torch.int64, device="cuda")
    else:
        n = H if case["lambda_heads"] == "each" else 1
        s["lambdas"] = [normal(n, D // 2, std=0.1, grad=train) for _ in range(4)]
        s["lambda_init"] = 0.8 - 0.6 * math.exp(-0.3 * 3)  # of a layer in the middle
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import topology_scheduled_gb300 as tsa
    from topology_scheduled_gb300 import autograd
    lam = s.get("lambdas")
    if s["form"] == "decode":
        if lam is None:
            return tsa.tsa_biased_attention_decode(s["Q"], s["K"], s["V"], s["lengths"], s["row_ptr"], s["col_idx"],
                                                   s["bias"], s["starts"], block=s["block"])
        return tsa.tsa_differential_attention_decode(s["Q"], s["K"], s["V"], s["lengths"], s["row_ptr"], s["col_idx"],
                                                     *lam, s["lambda_init"], block=s["block"])
    if s["form"] == "fwd":
        if lam is None:
            return tsa.tsa_biased_attention(s["Q"], s["K"], s["V"], s["row_ptr"], s["col_idx"], s["bias"], s["starts"],
                                            block=s["block"])
        return tsa.tsa_differential_attention(s["Q"], s["K"], s["V"], s["row_ptr"], s["col_idx"], *lam,
                                              s["lambda_init"], block=s["block"])
    if lam is None:
        O = autograd.biased_attention(s["Q"], s["K"], s["V"], s["row_ptr"], s["col_idx"], s["bias"], s["starts"],
                                      block=s["block"])
        leaves = [s["Q"], s["K"], s["V"], s["bias"]]
    else:
        O = autograd.differential_attention(s["Q"], s["K"], s["V"], s["row_ptr"], s["col_idx"], *lam,
                                            s["lambda_init"], block=s["block"])
        leaves = [s["Q"], s["K"], s["V"], *lam]
    return [O.detach(), *torch.autograd.grad(O, leaves, s["dO"])]


def _gathered(s):
    """The schedule as a table: [rows, most] key blocks, and which entries exist."""
    start, end = s["row_ptr"][:-1].long(), s["row_ptr"][1:].long()
    at = start[:, None] + torch.arange(s["most"], device="cuda")
    there = at < end[:, None]
    cols = s["col_idx"].long()[at.clamp(max=s["col_idx"].numel() - 1)]
    return torch.where(there, cols, 0), there


def _softmax(z, seen):
    """Rows that see no key have no weights."""
    m = z.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(z - torch.where(m == -math.inf, 0.0, m)), 0.0)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _lambda(s):
    a, b, c, d = (x.detach().float() for x in s["lambdas"])
    e1, e2 = torch.exp((a * b).sum(-1)), torch.exp((c * d).sum(-1))
    return e1 - e2 + s["lambda_init"], (a, b, c, d), (e1, e2)


def _plain(s):
    with torch.no_grad():
        return _plain_decode(s) if s["form"] == "decode" else _plain_blocks(s)


def _plain_decode(s):
    Q, dt = s["Q"].float(), s["Q"].dtype
    B, H, D = Q.shape
    S, block = s["K"].shape[2], s["block"]
    cols, there = _gathered(s)
    keys = (cols[:, :, None] * block + torch.arange(block, device="cuda")).reshape(B, -1)
    n = s["lengths"].long()[:, None]
    seen = (there[:, :, None].expand(-1, -1, block).reshape(B, -1) & (keys < n))[:, None]
    at = keys.clamp(max=S - 1)
    which = torch.arange(B, device="cuda")[:, None]
    Kg, Vg = (s[x][which, :, at].float() for x in "KV")  # [B, keys, H, D]
    if s["op"] == "biased":
        far = torch.searchsorted(s["starts_on_gpu"], (n - 1 - at).clamp(min=0).contiguous(), right=True) - 1
        z = torch.einsum("bhd,bkhd->bhk", Q, Kg) * D ** -0.5 + s["bias"].float()[:, far].transpose(0, 1)
        P = _softmax(z, seen)
    else:
        h = D // 2
        lam = _lambda(s)[0].expand(H)[None, :, None]
        P1, P2 = (_softmax(torch.einsum("bhd,bkhd->bhk", Q[..., x], Kg[..., x]) * h ** -0.5, seen)
                  for x in (slice(0, h), slice(h, D)))
        P = P1 - lam * P2
    return torch.einsum("bhk,bkhd->bhd", P, Vg).to(dt)


def _plain_blocks(s):
    dt, block = s["Q"].dtype, s["block"]
    B, H, S, D = s["Q"].shape
    L, nb = B * H, s["row_ptr"].numel() - 1
    cols, there = _gathered(s)
    R = s["most"] * block

    def blocks(x):  # [L, nb, block, D], rows past S zero
        x = x.detach().reshape(L, S, D).float()
        return torch.nn.functional.pad(x, (0, 0, 0, nb * block - S)).reshape(L, nb, block, D)

    def back(x):
        return x.reshape(L, nb * block, D)[:, :S].reshape(B, H, S, D).to(dt)

    Q, K, V = blocks(s["Q"]), blocks(s["K"]), blocks(s["V"])
    Kg, Vg = (x[:, cols].reshape(L, nb, R, D) for x in (K, V))
    q = torch.arange(nb * block, device="cuda").reshape(nb, block, 1)
    k = (cols[:, :, None] * block + torch.arange(block, device="cuda")).reshape(nb, 1, R)
    seen = there[:, :, None].expand(-1, -1, block).reshape(nb, 1, R) & (k <= q) & (q < S)  # [nb, block, R]
    head = torch.arange(L, device="cuda") % H
    biased = s["op"] == "biased"
    if biased:
        scale = D ** -0.5
        far = torch.searchsorted(s["starts_on_gpu"], (q - k).clamp(min=0), right=True) - 1
        z = Q @ Kg.transpose(-1, -2) * scale
        z += s["bias"].detach().float()[head][:, far]
        P = _softmax(z, seen)
        del z
        O = P @ Vg
    else:
        h = D // 2
        scale = h ** -0.5
        lam, vectors, e = _lambda(s)
        lam = lam.expand(H)[head].reshape(L, 1, 1, 1)
        P1 = _softmax(Q[..., :h] @ Kg[..., :h].transpose(-1, -2) * scale, seen)
        P2 = _softmax(Q[..., h:] @ Kg[..., h:].transpose(-1, -2) * scale, seen)
        O = (P1 - lam * P2) @ Vg
    if s["form"] == "fwd":
        return back(O)
    dO = blocks(s["dO"])
    dP = dO @ Vg.transpose(-1, -2)

    def scattered(x):  # gradients of gathered key blocks, summed at the blocks
        x = x.reshape(L, -1, block, D)
        return torch.zeros((L, nb, block, D), device="cuda").index_add_(1, cols.reshape(-1), x)

    def through(P, dP):  # the softmax's gradient
        return P * (dP - (P * dP).sum(-1, keepdim=True))

    if biased:
        dS = through(P, dP)
        n = s["bias"].shape[1]
        at = far.reshape(1, -1) + n * head[:, None]
        dbias = torch.zeros(H * n, device="cuda", dtype=torch.float64)
        dbias.index_add_(0, at.reshape(-1), dS.double().reshape(-1))
        return [back(O), back(dS @ Kg * scale), back(scattered(dS.transpose(-1, -2) @ Q) * scale),
                back(scattered(P.transpose(-1, -2) @ dO)), dbias.reshape(H, n).to(dt)]
    dV = back(scattered((P1 - lam * P2).transpose(-1, -2) @ dO))
    # one head's lambda multiplies that head's second map everywhere
    dlam = -(P2 * dP).sum((1, 2, 3), dtype=torch.float64).reshape(B, H).sum(0)
    dlam = dlam.reshape(vectors[0].shape[0], -1).sum(1).float()[:, None]
    dS1, dS2 = through(P1, dP), through(P2, -lam * dP)
    dQ = torch.cat([dS1 @ Kg[..., :h], dS2 @ Kg[..., h:]], -1)
    dK = torch.cat([dS1.transpose(-1, -2) @ Q[..., :h], dS2.transpose(-1, -2) @ Q[..., h:]], -1)
    a, b, c, d = vectors
    e1, e2 = e[0][:, None], e[1][:, None]
    return [back(O), back(dQ * scale), back(scattered(dK) * scale), dV,
            *((dlam * x).to(dt) for x in (e1 * b, e1 * a, -e2 * d, -e2 * c))]


def work(case):
    B, H, S, D = case["B"], case["H"], case["S"], case["D"]
    rows, lengths = _rows(case, random.Random(0))
    block = case["block"]
    tensor = 2 * B * H * S * D
    learned = 2 * (H * case["buckets"] if case["op"] == "biased" else
                   4 * (H if case["lambda_heads"] == "each" else 1) * D // 2)
    # query-key pairs that are seen, of one head
    if case["form"] == "decode":
        pairs = sum(min(block, max(0, n - j * block)) for r, n in zip(rows, lengths) for j in r)
        bytes_ = 2 * pairs * H * 2 * D + 4 * B * H * D + learned
    else:
        pairs = 0
        for i, r in enumerate(rows):
            n = min(block, S - i * block)
            pairs += sum(n * (n + 1) // 2 if j == i else n * block for j in r)
        pairs *= B
        bytes_ = (4 if case["form"] == "fwd" else 8) * tensor + learned * (1 if case["form"] == "fwd" else 2)
    # products of scores and of values: the scores' take D in all, a second map's values are another product
    maps = 1 if case["op"] == "biased" else 2
    flops = pairs * H * (2 * D + 2 * D * (1 if case["form"] == "decode" else maps))
    if case["form"] == "train":
        # dP once; dQ and dK (D in all each); dV of each map
        flops += pairs * H * (2 * D + 4 * D + 2 * D * maps)
    return {"bytes": bytes_, "flops": flops}


def exact(case, seed):
    """In 64 bits from the definition, one row of the schedule at a time."""
    s = prepare(case, seed)
    with torch.no_grad():
        return _exact(case, s)


def _exact(case, s):
    B, H, S, D = case["B"], case["H"], case["S"], case["D"]
    block, decode, train = case["block"], case["form"] == "decode", case["form"] == "train"
    ptr, idx = s["row_ptr"].tolist(), s["col_idx"].tolist()
    Q, K, V = (s[x].detach().double() for x in "QKV")
    maps = 1 if case["op"] == "biased" else 2
    w = D // maps
    scale = 1 / math.sqrt(w)
    sign = [torch.ones(H, 1, 1, device="cuda", dtype=torch.float64)]
    if maps == 2:
        lq1, lk1, lq2, lk2 = (x.detach().double() for x in s["lambdas"])
        up, down = (lq1 * lk1).sum(1).exp(), (lq2 * lk2).sum(1).exp()
        sign.append(-(up - down + s["lambda_init"]).expand(H).reshape(H, 1, 1))
    else:
        bias = s["bias"].detach().double()
        bucket_of = torch.zeros(S, dtype=torch.int64, device="cuda")
        for b, first in enumerate(s["starts"]):
            bucket_of[first:] = b
    O = torch.zeros_like(Q)
    if train:
        dO = s["dO"].double()
        dQ, dK, dV = (torch.zeros_like(x) for x in (Q, K, V))
        dmap = torch.zeros(H, device="cuda", dtype=torch.float64)
        dbias = torch.zeros(s["bias"].shape, device="cuda", dtype=torch.float64) if maps == 1 else None
    for i in range(len(ptr) - 1):
        cols = idx[ptr[i]:ptr[i + 1]]
        if decode:
            n = int(s["lengths"][i])
            q, which = torch.tensor([n - 1], device="cuda"), slice(i, i + 1)
            limit = n
        else:
            q, which = torch.arange(i * block, min(S, i * block + block), device="cuda"), slice(0, B)
            limit = S
        k = [t for j in cols for t in range(j * block, min(limit, j * block + block))]
        if not k:
            continue
        k = torch.tensor(k, device="cuda")
        hidden = k[None] > q[:, None]
        Qi = Q[which][:, :, None] if decode else Q[:, :, q]
        Ki, Vi = K[which][:, :, k], V[which][:, :, k]
        P = []
        for m in range(maps):
            z = Qi[..., m * w:m * w + w] @ Ki[..., m * w:m * w + w].transpose(2, 3) * scale
            if maps == 1:
                distance = (q[:, None] - k[None]).clamp(min=0)
                z = z + bias[:, bucket_of[distance]]
            z = z.masked_fill(hidden, -math.inf)
            top = z.max(-1, keepdim=True).values
            p = (z - top.masked_fill(top == -math.inf, 0)).exp()
            total = p.sum(-1, keepdim=True)
            P.append(p / total.masked_fill(total == 0, 1))
        weights = sum(f * p for f, p in zip(sign, P))
        if decode:
            O[i] = (weights @ Vi)[0, :, 0]
            continue
        O[:, :, q] = weights @ Vi
        if not train:
            continue
        G = dO[:, :, q]
        dV[:, :, k] += weights.transpose(2, 3) @ G
        dW = G @ Vi.transpose(2, 3)
        for m in range(maps):
            dP = sign[m] * dW
            dS = P[m] * (dP - (P[m] * dP).sum(-1, keepdim=True))
            part = slice(m * w, m * w + w)
            dQ[:, :, q, part] = dS @ Ki[..., part] * scale
            dK[:, :, k, part] += dS.transpose(2, 3) @ Qi[..., part] * scale
            if maps == 1:
                dbias.index_add_(1, bucket_of[distance].reshape(-1), dS.sum(0).reshape(H, -1))
        if maps == 2:
            dmap -= (P[1] * dW).sum((0, 2, 3))
    if not train:
        return O
    if maps == 1:
        return [O, dQ, dK, dV, dbias]
    d = dmap.reshape(lq1.shape[0], -1).sum(1)
    u, v = (d * up)[:, None], (-d * down)[:, None]
    return [O, dQ, dK, dV, u * lk1, u * lq1, v * lk2, v * lq2]
