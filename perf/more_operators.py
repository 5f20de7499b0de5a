"""What rotary positions, the paged key/value cache and its attention cost, and what they answer.

Three operators:

* rotary: the pairs of the first R dimensions of every row of Q and K are rotated by the row's position
  times the pair's frequency, forwards ("fwd") and with the gradients ("train");
* append: new tokens' keys (rotated) and values are written to the pages of a paged cache, and their
  queries rotated. Sequence b holds `seq_lens[b]` tokens with the new ones, whose last it is, and its
  token p lies in slot p % page of page `page_table[b, p // page]`;
* decode: one new token per sequence against such a cache, softmax(scale q.k) V over its keys or over
  those of the key blocks that row b of a schedule lists. Query heads share keys in equal groups.
"""
import array
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
SCALINGS = {"none": None, "linear": "linear", "base": "base", "ramp": "ramp"}


def listed():
    rot = {"op": "rotary", "layout": "tokens"}
    app = {"op": "append", "layout": "tokens", "pairs": "half", "scaling": "none", "padding": "none"}
    dec = {"op": "decode", "schedule": "all", "block": 64, "idle": False, "ragged": False}
    return [
        # the next token of one sequence, far into it: latency counts
        {"name": "rotary fwd b1s1", **rot, "form": "fwd", "B": 1, "S": 1, "H": 16, "HK": 16, "D": 64, "R": 64,
         "pairs": "half", "scaling": "none", "positions": "each", "dtype": "f16"},
        # long prompts, from the projections' layout to the attention's
        {"name": "rotary fwd b2h32s32768", **rot, "form": "fwd", "B": 2, "S": 32768, "H": 32, "HK": 32, "D": 128,
         "R": 128, "pairs": "half", "scaling": "ramp", "positions": "none", "dtype": "bf16"},
        # a training step on a batch of documents
        {"name": "rotary train b4h16s8192", **rot, "form": "train", "B": 4, "S": 8192, "H": 16, "HK": 16, "D": 64,
         "R": 64, "pairs": "interleaved", "scaling": "base", "positions": "shared", "dtype": "f16"},
        # a training step on packed ragged documents, part of the head rotated, shared keys
        {"name": "rotary train s1999 part", **rot, "form": "train", "B": 3, "S": 1999, "H": 12, "HK": 4, "D": 128,
         "R": 32, "pairs": "half", "scaling": "linear", "positions": "each", "dtype": "bf16"},
        # the next token of one sequence
        {"name": "append b1t1", **app, "B": 1, "T": 1, "H": 16, "HK": 16, "D": 64, "R": 64, "page": 16,
         "held": 999, "dtype": "f16"},
        # the next token of a full batch
        {"name": "append b64t1", **app, "B": 64, "T": 1, "H": 32, "HK": 8, "D": 128, "R": 128, "page": 64,
         "held": 4095, "scaling": "ramp", "dtype": "bf16"},
        # a batch of ragged prompts, padded behind
        {"name": "append b4t8192", **app, "B": 4, "T": 8192, "H": 32, "HK": 8, "D": 128, "R": 64, "page": 64,
         "held": 0, "pairs": "interleaved", "padding": "right", "dtype": "bf16"},
        # the next token of one short sequence
        {"name": "decode b1s1000", **dec, "B": 1, "H": 16, "HK": 16, "S": 1000, "D": 64, "page": 16, "dtype": "f16"},
        # the next token of one very long sequence: few rows, the cache's length has to fill the GPU
        {"name": "decode b1s131072", **dec, "B": 1, "H": 32, "HK": 8, "S": 131072, "D": 128, "page": 64,
         "dtype": "bf16"},
        # a full batch of ragged lengths, many queries to a key, small pages, some slots idle
        {"name": "decode b64s8192 ragged", **dec, "B": 64, "H": 32, "HK": 4, "S": 8192, "D": 128, "page": 16,
         "idle": True, "ragged": True, "dtype": "bf16"},
        # a batch through a sparse schedule's rows
        {"name": "decode b16s8192 topology", **dec, "B": 16, "H": 32, "HK": 8, "S": 8192, "D": 64, "page": 128,
         "schedule": "topology", "ragged": True, "dtype": "f16"},
        # a batch whose every head has keys of its own
        {"name": "decode b16h32s8192", **dec, "B": 16, "H": 32, "HK": 32, "S": 8192, "D": 128, "page": 64,
         "dtype": "bf16"},
    ]


def _spread(rng, low, high):
    return int(round(2 ** rng.uniform(math.log2(low), math.log2(high))))


def draw(rng):
    while True:
        hk = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
        case = {"op": rng.choice(["rotary", "append", "decode"]), "H": hk * rng.choice([1, 1, 2, 3, 4, 7, 8, 16]), "HK": hk,
                "D": rng.choice([64, 128]), "dtype": rng.choice(["f16", "bf16"])}
        if case["H"] > 64:
            continue
        if case["op"] == "decode":
            case |= {"B": _spread(rng, 1, 64), "S": _spread(rng, 1, 131072), "page": rng.choice([16, 32, 64, 128, 256]),
                     "schedule": rng.choice(["all", "topology", "random"]), "block": rng.choice([32, 64, 128]),
                     "idle": rng.random() < 0.3, "ragged": rng.random() < 0.7}
            if case["B"] * case["S"] * hk * case["D"] <= 16 * 8192 * 32 * 128 and \
                    case["B"] * case["S"] * case["H"] <= 64 * 8192 * 32:
                return case
            continue
        case |= {"R": rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= case["D"]]),
                 "pairs": rng.choice(["half", "interleaved"]), "scaling": rng.choice(list(SCALINGS)),
                 "layout": rng.choice(["tokens", "heads"])}
        if case["op"] == "rotary":
            case |= {"form": rng.choice(["fwd", "train"]), "B": _spread(rng, 1, 16), "S": _spread(rng, 1, 32768),
                     "positions": rng.choice(["none", "shared", "each"])}
            if case["B"] * case["S"] * (case["H"] + hk) * case["D"] <= 2 * 32768 * 64 * 128 // (2 if case["form"] == "train" else 1):
                return case
        else:
            case |= {"B": _spread(rng, 1, 64), "T": _spread(rng, 1, 8192), "page": rng.choice([16, 32, 64, 128, 256]),
                     "held": rng.choice([0, _spread(rng, 1, 8192)]), "padding": rng.choice(["none", "left", "right"])}
            if case["padding"] == "left":
                case["held"] = 0
            if case["B"] * case["T"] * (case["H"] + 2 * hk) * case["D"] <= 4 * 8192 * 48 * 128 and \
                    case["B"] * (case["T"] + case["held"]) * hk * case["D"] <= 1 << 28:
                return case


def _frequencies(R, scaling):
    """Frequency of each pair, and the rotated rows' magnitude: base ** (-2 i / R), as it is; for contexts 4 times
    as long as the 8192 tokens trained on, divided by 4, of a larger base, or divided where a pair turns less than
    once in those tokens and as it is from 32 turns on."""
    base, factor, length = 10000.0, 4.0, 8192
    if scaling == "base" and R > 2:
        base *= factor ** (R / (R - 2))
    f = [base ** (-2 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "ramp":
        keep = [min(max((length * x / (2 * math.pi) - 1) / 31, 0.0), 1.0) for x in f]
        f = [x * (k + (1 - k) / factor) for x, k in zip(f, keep)]
    return f, 0.1 * math.log(factor) + 1 if scaling == "ramp" else 1.0


def _lengths(case, rng):
    """Tokens each sequence holds, and (append) how many of them are new."""
    B = case["B"]
    if case["op"] == "decode":
        S = case["S"]
        lengths = [S if b == 0 or not case["ragged"] else rng.randint(max(1, S // 2), S) for b in range(B)]
        if case["idle"] and B > 1:
            for b in range(3, B, 8):
                lengths[b] = 0
            lengths[-1] = 0
        return lengths, None
    T, held = case["T"], case["held"]
    before = [rng.randint(held // 2, held) for _ in range(B)]
    if case["padding"] == "none":
        return [n + T for n in before], [T] * B
    fresh = [T if b == 0 else rng.randint(0, T) for b in range(B)]
    return [n + t for n, t in zip(before, fresh)], fresh


def _schedule(case, lengths, rng):
    """The key blocks that each sequence's token visits: sinks, a window and some of large salience, or a random
    choice that leaves some rows empty; None for all keys."""
    if case["schedule"] == "all":
        return None
    rows = []
    for n in lengths:
        nb = -(-n // case["block"])
        if case["schedule"] == "topology":
            rows.append(sorted({*range(min(2, nb)), *range(max(0, nb - 9), nb), *(rng.randrange(nb) for _ in range(32 if nb else 0))}))
        else:
            rows.append([] if rng.random() < 0.1 else [j for j in range(nb) if rng.random() < 0.4])
    return rows


def prepare(case, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, H, HK, D = case["B"], case["H"], case["HK"], case["D"]
    s = {"op": case["op"]}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    def rows(heads, n):  # [B, heads, n, D], as a projection leaves it or as an attention does
        return normal(B, n, heads, D).transpose(1, 2) if case["layout"] == "tokens" else normal(B, heads, n, D)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    if case["op"] != "decode":
        f, s["magnitude"] = _frequencies(case["R"], case["scaling"])
        s["frequencies"] = array.array("d", f)
        s["interleaved"] = case["pairs"] == "interleaved"
    if case["op"] == "rotary":
        S, train = case["S"], case["form"] == "train"
        s |= {"form": case["form"], "Q": rows(H, S).requires_grad_(train), "K": rows(HK, S).requires_grad_(train),
              "positions": None}
        if case["positions"] == "shared":  # a chunk from somewhere on
            first = rng.randrange(1 << 20)
            s["positions"] = ints(list(range(first, first + S)))
        if case["positions"] == "each":  # documents of their own, each from 0 or from where it was cut
            p = torch.arange(S)[None] + torch.tensor([[rng.randrange(100000)] for _ in range(B)])
            s["positions"] = torch.where(torch.arange(S) >= S - S // 3, torch.arange(S) - (S - S // 3), p).int().cuda()
        if train:
            s["dQ"], s["dK"] = normal(B, H, S, D), normal(B, HK, S, D)
        return s
    lengths, fresh = _lengths(case, rng)
    page = case["page"]
    most = -(-(case["S"] if case["op"] == "decode" else case["held"] + case["T"]) // page)
    # pages in the order that they came free; the last one is nobody's
    pages = torch.randperm(B * most, generator=g, device="cuda").reshape(B, most)
    used = ints([-(-n // page) for n in lengths])
    there = torch.arange(most, device="cuda") < used[:, None]
    s |= {"K_cache": normal(B * most + 1, HK, page, D), "V_cache": normal(B * most + 1, HK, page, D),
          "page_table": torch.where(there, pages, -1).int(), "seq_lens": ints(lengths)}
    if case["op"] == "append":
        T = case["T"]
        s |= {"Q": rows(H, T), "K": rows(HK, T), "V": rows(HK, T),
              "counts": ints(fresh) if case["padding"] == "right" else None}
        return s
    s |= {"Q": normal(B, H, D), "block": case["block"], "row_ptr": None, "col_idx": None}
    rows_ = _schedule(case, lengths, rng)
    if rows_ is not None:
        ptr = [0]
        for r in rows_:
            ptr.append(ptr[-1] + len(r))
        s |= {"row_ptr": ints(ptr), "col_idx": ints([j for r in rows_ for j in r] or [0])}
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import topology_scheduled_gb300 as tsa
    from topology_scheduled_gb300 import autograd
    if s["op"] == "decode":
        return tsa.tsa_paged_attention_decode(s["Q"], s["K_cache"], s["V_cache"], s["page_table"], s["seq_lens"],
                                              s["row_ptr"], s["col_idx"], block=s["block"])
    if s["op"] == "append":
        Q = tsa.tsa_paged_append(s["Q"], s["K"], s["V"], s["K_cache"], s["V_cache"], s["page_table"], s["seq_lens"],
                                 s["counts"], s["frequencies"], interleaved=s["interleaved"], magnitude=s["magnitude"])
        return [Q, s["K_cache"], s["V_cache"]]
    if s["form"] == "fwd":
        return list(tsa.tsa_rotary(s["Q"], s["K"], s["frequencies"], s["positions"], interleaved=s["interleaved"],
                                   magnitude=s["magnitude"]))
    Q, K = autograd.rotary(s["Q"], s["K"], s["frequencies"], s["positions"], interleaved=s["interleaved"],
                           magnitude=s["magnitude"])
    return [Q.detach(), K.detach(), *torch.autograd.grad([Q, K], [s["Q"], s["K"]], [s["dQ"], s["dK"]])]


def _plain(s):
    with torch.no_grad():
        return {"rotary": _plain_rotary, "append": _plain_append, "decode": _plain_decode}[s["op"]](s)


def _turns(s, positions):
    """Cosine and sine of each position's angles (64 bits: positions may be far), times the magnitude."""
    f = torch.tensor(s["frequencies"], dtype=torch.float64, device="cuda")
    angle = positions.double()[..., None] * f
    return (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()


def _rotated(s, x, cos, sin):
    n = cos.shape[-1]
    x = x.float()
    if s["interleaved"]:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., 2 * n:]], -1)


def _plain_rotary(s):
    Q, K = s["Q"].detach(), s["K"].detach()
    p = s["positions"]
    if p is None:
        p = torch.arange(Q.shape[2], device="cuda")
    cos, sin = _turns(s, p if p.dim() == 1 else p[:, None])
    out = [_rotated(s, x, cos, sin).to(x.dtype) for x in (Q, K)]
    if s["form"] == "train":
        out += [_rotated(s, x, cos, -sin).to(x.dtype) for x in (s["dQ"], s["dK"])]
    return out


def _plain_append(s):
    Q, K, V, Kc, Vc = (s[x] for x in ("Q", "K", "V", "K_cache", "V_cache"))
    B, HK, T, D = K.shape
    page = Kc.shape[2]
    n = s["seq_lens"].long()[:, None]
    new = T if s["counts"] is None else s["counts"].long()[:, None]
    t = torch.arange(T, device="cuda")
    p = n - new + t
    there = (t < new) & (p >= 0)
    at = torch.where(there, p, 0)
    cos, sin = _turns(s, at[:, None])
    # a token that is not there writes what nobody's page holds already
    which = torch.where(there, s["page_table"].long().gather(1, at // page), Kc.shape[0] - 1)[:, :, None]
    slot, head = (at % page)[:, :, None], torch.arange(HK, device="cuda")
    there = there[:, :, None, None]
    for cache, new in ((Kc, _rotated(s, K, cos, sin).to(K.dtype)), (Vc, V)):
        cache[which, head, slot] = torch.where(there, new.transpose(1, 2), cache[which, head, slot])
    return [torch.where(there.transpose(1, 2), _rotated(s, Q, cos, sin), 0.0).to(Q.dtype), Kc, Vc]


def _plain_decode(s):
    Q, dt, block = s["Q"].float(), s["Q"].dtype, s["block"]
    B, H, D = Q.shape
    HK, page = s["K_cache"].shape[1:3]
    k = torch.arange(s["page_table"].shape[1] * page, device="cuda")
    seen = k < s["seq_lens"][:, None]
    if s["row_ptr"] is not None:
        entry = torch.arange(s["col_idx"].numel(), device="cuda", dtype=torch.int32)
        row = torch.searchsorted(s["row_ptr"][1:].contiguous(), entry, right=True)
        listed_ = torch.zeros((B + 1, -(-k.numel() // block)), dtype=torch.bool, device="cuda")
        listed_[row, s["col_idx"].long()] = True  # (an entry past the last row is nobody's)
        seen = seen & listed_[:B][:, k // block]
    table = s["page_table"].long().clamp(min=0)
    K, V = (s[x][table].transpose(1, 2).reshape(B, HK, -1, D).float() for x in ("K_cache", "V_cache"))
    seen = seen[:, None, None]
    z = (Q.reshape(B, HK, H // HK, D) @ K.transpose(2, 3)) * D ** -0.5
    m = z.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(z - torch.where(m == -math.inf, 0.0, m)), 0.0)
    total = e.sum(-1, keepdim=True)
    return ((e @ V) / torch.where(total > 0, total, 1.0)).reshape(B, H, D).to(dt)


def work(case):
    H, HK, D = case["H"], case["HK"], case["D"]
    if case["op"] == "rotary":
        n = case["B"] * case["S"] * (H + HK)
        times = 2 if case["form"] == "train" else 1
        return {"bytes": 4 * n * D * times, "flops": 3 * n * case["R"] * times}
    rng = random.Random(0)
    lengths, fresh = _lengths(case, rng)
    if case["op"] == "append":
        n = sum(fresh)
        return {"bytes": 4 * n * (H + 2 * HK) * D, "flops": 3 * n * (H + HK) * case["R"]}
    rows = _schedule(case, lengths, rng)
    if rows is None:
        keys = sum(lengths)
    else:
        keys = sum(min(case["block"], n - j * case["block"]) for n, r in zip(lengths, rows) for j in r)
    return {"bytes": 4 * keys * HK * D + 4 * case["B"] * H * D, "flops": 4 * keys * H * D}


def exact(case, seed):
    """In 64 bits from the definitions: pairs as complex numbers, sequences one at a time."""
    s = prepare(case, seed)
    with torch.no_grad():
        return _exact(case, s)


def _turned(case, s, x, positions, back=False):
    """Rows x [.., n, D] at positions [n]: each pair times magnitude * exp(i * position * frequency)."""
    R = case["R"]
    x = x.double()
    f = torch.tensor(list(s["frequencies"]), dtype=torch.float64, device="cuda")
    angle = torch.outer(positions.double(), -f if back else f)
    turn = torch.polar(torch.full_like(angle, s["magnitude"]), angle)
    y = x.clone()
    re, im = (slice(0, R, 2), slice(1, R, 2)) if case["pairs"] == "interleaved" else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact(case, s):
    B, H, HK, D = case["B"], case["H"], case["HK"], case["D"]
    if case["op"] == "rotary":
        p = s["positions"]
        if p is None:
            p = torch.arange(case["S"], device="cuda")
        p = p.expand(B, case["S"])
        names = [("Q", False), ("K", False)] + ([("dQ", True), ("dK", True)] if case["form"] == "train" else [])
        return [torch.stack([_turned(case, s, s[x].detach()[b], p[b], back) for b in range(B)]) for x, back in names]
    table, lengths, page = s["page_table"].tolist(), s["seq_lens"].tolist(), case["page"]
    if case["op"] == "append":
        fresh = [case["T"]] * B if s["counts"] is None else s["counts"].tolist()
        out = [torch.zeros((B, H, case["T"], D), dtype=torch.float64, device="cuda"), s["K_cache"].double(), s["V_cache"].double()]
        for b in range(B):
            begin = lengths[b] - fresh[b]
            skip = max(0, -begin)
            if fresh[b] <= skip:
                continue
            p = torch.arange(begin + skip, lengths[b], device="cuda")
            new = slice(skip, fresh[b])
            out[0][b, :, new] = _turned(case, s, s["Q"][b, :, new], p)
            at = torch.tensor(table[b], device="cuda")[p // page]
            out[1][at, :, p % page] = _turned(case, s, s["K"][b, :, new], p).transpose(0, 1)
            out[2][at, :, p % page] = s["V"][b, :, new].double().transpose(0, 1)
        return out
    O = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    ptr = None if s["row_ptr"] is None else s["row_ptr"].tolist()
    for b in range(B):
        k = torch.arange(lengths[b], device="cuda")
        if ptr is not None:
            k = k[torch.isin(k // case["block"], s["col_idx"][ptr[b]:ptr[b + 1]].long())]
        if k.numel() == 0:
            continue
        at = torch.tensor(table[b], device="cuda")[k // page]
        for h in range(HK):
            group = slice(h * (H // HK), (h + 1) * (H // HK))
            K, V = (s[x][at, h, k % page].double() for x in ("K_cache", "V_cache"))
            O[b, group] = torch.softmax(s["Q"][b, group].double() @ K.T / math.sqrt(D), -1) @ V
    return O
