"""Cases of the row operators: rows of a matrix moved and summed by their token's key.

Two families, both resting on a stable sort of small integer keys:

* tokens sorted by expert and back: ``sort`` groups the (token, slot) choices of a
  router by expert and copies each token's row to its place in expert order,
  ``back`` sums a token's rows again with the router's weights, ``grads`` is the
  backward pass of both;
* embedding lookup with scaling (``embed``) and its gradient by sorted tokens
  (``embed_grad``).

``own`` chooses what ``run`` computes with: False, elementary torch operations in 32
bits, rounded once at the end; True, the operators of
``sorting_lsd_radix_sort_amd``.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "i32": 4, "i64": 8}


def listed():
    return [
        # Serving, one step of a batch of four sequences: latency counts.
        {"name": "sort_decode", "kind": "sort", "tokens": 4, "slots": 8, "experts": 128, "first": 0, "local": 128,
         "cols": 4096, "dtype": "bf16", "ids": "i64"},
        # One rank of an expert-parallel group of eight: only its experts' rows, odd sizes.
        {"name": "sort_shard", "kind": "sort", "tokens": 2047, "slots": 6, "experts": 160, "first": 40, "local": 20,
         "cols": 1537, "dtype": "f16", "ids": "i32"},
        # Training or a long prompt: a whole micro-batch of 16K tokens on all experts.
        {"name": "sort_prompt", "kind": "sort", "tokens": 16384, "slots": 8, "experts": 256, "first": 0, "local": 256,
         "cols": 4096, "dtype": "bf16", "ids": "i64"},
        # The way back of a decode step for 32 sequences.
        {"name": "back_decode", "kind": "back", "tokens": 32, "slots": 8, "experts": 128, "first": 0, "local": 128,
         "cols": 4096, "dtype": "bf16", "ids": "i64"},
        # The way back of a long prompt in float32, a few choices lost to other ranks.
        {"name": "back_prompt", "kind": "back", "tokens": 8192, "slots": 4, "experts": 64, "first": 0, "local": 60,
         "cols": 2048, "dtype": "f32", "ids": "i64"},
        # Backward pass of a small mixture with odd sizes (a test model, a last partial batch).
        {"name": "grads_odd", "kind": "grads", "tokens": 301, "slots": 2, "experts": 8, "first": 0, "local": 8,
         "cols": 1000, "dtype": "f32", "ids": "i64"},
        # Backward pass of a training micro-batch of 16K tokens.
        {"name": "grads_train", "kind": "grads", "tokens": 16384, "slots": 8, "experts": 256, "first": 0, "local": 256,
         "cols": 4096, "dtype": "bf16", "ids": "i64"},
        # Lookup for a decode step of 64 sequences.
        {"name": "embed_decode", "kind": "embed", "tokens": 64, "first": 0, "vocab": 65536, "cols": 4096,
         "dtype": "bf16", "ids": "i64"},
        # Lookup for 32K prompt tokens in one of two vocabulary shards: half the rows are zero.
        {"name": "embed_prompt", "kind": "embed", "tokens": 32768, "first": 65536, "vocab": 65536, "cols": 5120,
         "dtype": "bf16", "ids": "i64"},
        # Gradient of a short batch with odd sizes.
        {"name": "embed_grad_short", "kind": "embed_grad", "tokens": 777, "first": 0, "vocab": 5003, "cols": 515,
         "dtype": "f16", "grad": "f16", "add": False, "ids": "i32"},
        # Gradient of a training batch: 64K tokens of Zipf's law, the whole table written.
        {"name": "embed_grad_train", "kind": "embed_grad", "tokens": 65536, "first": 0, "vocab": 131072, "cols": 4096,
         "dtype": "bf16", "grad": "bf16", "add": False, "ids": "i64"},
        # Gradient added to the float32 one that micro-batches share.
        {"name": "embed_grad_add", "kind": "embed_grad", "tokens": 16384, "first": 0, "vocab": 65536, "cols": 2048,
         "dtype": "bf16", "grad": "f32", "add": True, "ids": "i64"},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["sort", "back", "grads", "embed", "embed_grad"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    ids = rng.choice(["i32", "i64"])
    # a third of the rows has a length that is no multiple of eight
    cols = _log_int(rng, 64, 8192)
    if rng.random() < 0.67:
        cols = max(64, cols // 64 * 64)
    if kind in ("sort", "back", "grads"):
        slots = rng.randint(1, 8)
        experts = _log_int(rng, max(8, slots), 256)
        local, first = experts, 0
        if rng.random() < 0.33:  # one rank of several
            local = max(1, experts // rng.choice([2, 4, 8]))
            first = rng.randint(0, experts - local)
        most = 16384 * 8 * 4096 * 2 // (slots * cols * BYTES[dtype])
        tokens = _log_int(rng, 1, min(16384, most))
        return {"kind": kind, "tokens": tokens, "slots": slots, "experts": experts, "first": first, "local": local,
                "cols": cols, "dtype": dtype, "ids": ids}
    vocab = min(_log_int(rng, 256, 131072), 131072 * 4096 * 2 // (cols * 4))
    first = rng.choice([0, 0, vocab])
    tokens = min(_log_int(rng, 1, 65536), 65536 * 4096 * 2 // (cols * BYTES[dtype]))
    case = {"kind": kind, "tokens": tokens, "first": first, "vocab": vocab, "cols": cols, "dtype": dtype, "ids": ids}
    if kind == "embed_grad":
        case["grad"] = rng.choice([dtype, "f32"])
        case["add"] = rng.random() < 0.33
    return case


# ------------------------------------------------------------------- inputs


def _randn(g, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)
    return x if scale == 1.0 else x.mul_(scale)


def _routed(case, g):
    """A router's choices: the `slots` largest of each token's scores, with some experts liked better, and
    their softmax."""
    t, e, k = case["tokens"], case["experts"], case["slots"]
    scores = _randn(g, (t, e), torch.float32) + _randn(g, (1, e), torch.float32, 0.5)
    best, ids = torch.topk(scores, k, dim=1)
    ids = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
    return ids, torch.softmax(best, dim=1)


def _zipf_share(size):
    """Probability of each rank 1..size under Zipf's law as `_zipf` draws it."""
    edges = np.log(np.arange(1, size + 2, dtype=np.float64))
    return np.diff(edges) / edges[-1]


def _zipf(case, g):
    """Token ids by Zipf's law, spread over the table; all shards' ids where this is one of two."""
    size = case["vocab"] * (2 if case["first"] else 1)
    u = torch.rand(case["tokens"], generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(size + 1)).to(torch.int64) - 1).clamp_(0, size - 1)
    step = int(size * 0.618) | 1
    while math.gcd(step, size) != 1:
        step += 2
    return (rank * step % size).to(torch.int32 if case["ids"] == "i32" else torch.int64)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = dict(case)
    if case["kind"] in ("sort", "back", "grads"):
        ids, weights = _routed(case, g)
        n, h = ids.numel(), case["cols"]
        if case["kind"] == "sort":
            s["ids"], s["x"] = ids, _randn(g, (case["tokens"], h), dtype)
            s["rows"] = torch.zeros(n, h, device="cuda", dtype=dtype)  # the experts' input buffer
            return s
        s["weights"] = weights
        s["order"], s["position"], _ = _plain_group(ids, case["local"], case["first"])
        s["rows"] = _randn(g, (n, h), dtype)  # what the experts answered, in their order
        if case["kind"] == "grads":
            s["grad_y"] = _randn(g, (case["tokens"], h), dtype)
            s["grad_x_rows"] = _randn(g, (n, h), dtype)  # the gradient that came back through the experts
            s["grad_rows"] = torch.zeros(n, h, device="cuda", dtype=dtype)
        return s
    s["ids"] = _zipf(case, g)
    s["scale"] = math.sqrt(case["cols"])
    if case["kind"] == "embed":
        s["table"] = _randn(g, (case["vocab"], case["cols"]), dtype, 0.02)
        return s
    s["grad_y"] = _randn(g, (case["tokens"], case["cols"]), dtype)
    s["grad_dtype"] = DTYPES[case["grad"]]
    s["total"] = _randn(g, (case["vocab"], case["cols"]), s["grad_dtype"]) if case["add"] else None
    return s


# --------------------------------------------------------------- plain forms


def _plain_group(ids, groups, first):
    """order: the slots by group, stable, those of no group last; position: each slot's place, -1 for none;
    offsets: where each group begins, and the number of slots kept."""
    key = ids.reshape(-1).to(torch.int64) - first
    key = torch.where((key < 0) | (key >= groups), groups, key)
    by_key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by_key, torch.arange(groups + 1, device=key.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    place = torch.where(key < groups, place, -1)
    return order.to(torch.int32), place.to(torch.int32).reshape(ids.shape), offsets.to(torch.int32)


def _plain_sort(s):
    order, position, offsets = _plain_group(s["ids"], s["local"], s["first"])
    rows = s["x"][order.to(torch.int64) // s["slots"]]
    if s["local"] < s["experts"]:
        kept = torch.arange(rows.shape[0], device=rows.device) < offsets[-1]
        rows = torch.where(kept[:, None], rows, s["rows"])
    return {"order": order, "position": position, "offsets": offsets, "rows": rows}


def _plain_sum(rows, position, weights):
    taken = rows[position.clamp(min=0).to(torch.int64)].float()
    if weights is not None:
        taken = taken * weights.float()[:, :, None]
    return torch.where((position >= 0)[:, :, None], taken, 0.0).sum(1).to(rows.dtype)


def _plain_grads(s):
    position, order = s["position"], s["order"].to(torch.int64)
    there = position >= 0
    taken = s["rows"][position.clamp(min=0).to(torch.int64)].float()
    dots = (taken * s["grad_y"].float()[:, None, :]).sum(2)
    grad_weights = torch.where(there, dots, 0.0)
    weight = s["weights"].reshape(-1)[order]
    grad_rows = (s["grad_y"][order // s["slots"]].float() * weight[:, None]).to(s["rows"].dtype)
    if s["local"] < s["experts"]:
        grad_rows = torch.where(there.reshape(-1)[order][:, None], grad_rows, s["grad_rows"])
    return {"grad_rows": grad_rows, "grad_weights": grad_weights,
            "grad_x": _plain_sum(s["grad_x_rows"], position, None)}


def _plain_embed(s):
    row = s["ids"].to(torch.int64) - s["first"]
    there = (row >= 0) & (row < s["vocab"])
    taken = s["table"][torch.where(there, row, 0)].float() * s["scale"]
    return torch.where(there[:, None], taken, 0.0).to(s["table"].dtype)


def _plain_embed_grad(s):
    row = s["ids"].to(torch.int64) - s["first"]
    there = (row >= 0) & (row < s["vocab"])
    each = torch.where(there[:, None], s["grad_y"].float(), 0.0)
    total = torch.zeros(s["vocab"], s["cols"], device=each.device, dtype=torch.float32)
    total.index_add_(0, torch.where(there, row, 0), each)
    total = total * s["scale"]
    if s["add"]:
        return s["total"].copy_(s["total"].float() + total)
    return total.to(s["grad_dtype"])


def _own_run(s):
    import sorting_lsd_radix_sort_amd as lrs

    if s["kind"] == "sort":
        order, position, offsets = lrs.group_tokens(s["ids"], s["local"], first_id=s["first"])
        rows = lrs.dispatch_rows(s["x"], position, out=s["rows"])
        return {"order": order, "position": position, "offsets": offsets, "rows": rows}
    if s["kind"] == "back":
        return {"y": lrs.combine_rows(s["rows"], s["position"], s["weights"])}
    if s["kind"] == "grads":
        grad_rows, grad_weights = lrs.combine_rows_grad(s["grad_y"], s["rows"], s["position"], s["weights"],
                                                        grad_rows=s["grad_rows"])
        return {"grad_rows": grad_rows, "grad_weights": grad_weights,
                "grad_x": lrs.combine_rows(s["grad_x_rows"], s["position"])}
    if s["kind"] == "embed":
        return {"y": lrs.embedding(s["table"], s["ids"], scale=s["scale"], first_id=s["first"])}
    return {"grad": lrs.embedding_grad(s["grad_y"], s["ids"], s["vocab"], scale=s["scale"], first_id=s["first"],
                                       dtype=s["grad_dtype"], grad=s["total"], accumulate=s["add"])}


def run(state):
    if own:
        return _own_run(state)
    kind = state["kind"]
    if kind == "sort":
        return _plain_sort(state)
    if kind == "back":
        return {"y": _plain_sum(state["rows"], state["position"], state["weights"])}
    if kind == "grads":
        return _plain_grads(state)
    if kind == "embed":
        return {"y": _plain_embed(state)}
    return {"grad": _plain_embed_grad(state)}


# --------------------------------------------------------------------- work


def work(case):
    b, h, t = BYTES[case["dtype"]], case["cols"], case["tokens"]
    if case["kind"] in ("sort", "back", "grads"):
        n = t * case["slots"]
        kept = n * case["local"] // case["experts"]
        if case["kind"] == "sort":
            touched = t * (1 - (1 - case["local"] / case["experts"]) ** case["slots"])
            return {"bytes": n * (BYTES[case["ids"]] + 8) + 4 * (case["local"] + 1) + (touched + kept) * h * b,
                    "flops": 0}
        if case["kind"] == "back":
            return {"bytes": n * 8 + (kept + t) * h * b, "flops": 2 * kept * h}
        # rows read and their gradient written, the rows that came back read; grad_y read, grad_x written
        return {"bytes": n * 12 + (3 * kept + 2 * t) * h * b, "flops": 4 * kept * h}
    share = _zipf_share(case["vocab"] * (2 if case["first"] else 1))
    there = t / 2 if case["first"] else t
    distinct = float(np.sum(-np.expm1(t * np.log1p(-share))))
    distinct = max(1.0, distinct / 2 if case["first"] else distinct)
    if case["kind"] == "embed":
        return {"bytes": t * BYTES[case["ids"]] + (distinct + t) * h * b, "flops": there * h}
    g = BYTES[case["grad"]]
    written = 2 * distinct * h * g if case["add"] else case["vocab"] * h * g
    return {"bytes": t * BYTES[case["ids"]] + there * h * b + written, "flops": there * h}


# -------------------------------------------------------------------- exact


def _exact_group(ids, groups, first):
    """The same by numpy: a slot's place is the number of kept slots of earlier groups, and of earlier ones of its own."""
    key = ids.cpu().numpy().reshape(-1).astype(np.int64) - first
    key[(key < 0) | (key >= groups)] = groups
    order = np.lexsort((np.arange(key.size), key))
    counts = np.bincount(key, minlength=groups + 1)
    offsets = np.concatenate([[0], np.cumsum(counts[:groups])])
    place = np.empty(key.size, dtype=np.int64)
    place[order] = np.arange(key.size)
    place[key == groups] = -1
    return order, place, offsets


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "sort":
        order, place, offsets = _exact_group(s["ids"], case["local"], case["first"])
        rows = torch.zeros(order.size, case["cols"], device="cuda", dtype=torch.float64)
        kept = int(offsets[-1])
        rows[:kept] = s["x"].double()[torch.from_numpy(order[:kept] // case["slots"]).cuda()]
        as_ints = lambda a, shape: torch.from_numpy(a.astype(np.int32)).reshape(shape)  # noqa: E731
        return {"order": as_ints(order, (-1,)), "position": as_ints(place, s["ids"].shape),
                "offsets": as_ints(offsets, (-1,)), "rows": rows}
    if kind in ("back", "grads"):
        place, t, h = s["position"].to(torch.int64), case["tokens"], case["cols"]
        y = torch.zeros(t, h, device="cuda", dtype=torch.float64)
        if kind == "back":
            for k in range(case["slots"]):
                on = (place[:, k] >= 0).nonzero()[:, 0]
                y[on] += s["weights"][on, k].double()[:, None] * s["rows"][place[on, k]].double()
            return {"y": y}
        grad_y = s["grad_y"].double()
        grad_rows = torch.zeros(s["rows"].shape, device="cuda", dtype=torch.float64)
        grad_weights = torch.zeros(t, case["slots"], device="cuda", dtype=torch.float64)
        for k in range(case["slots"]):
            on = (place[:, k] >= 0).nonzero()[:, 0]
            at = place[on, k]
            y[on] += s["grad_x_rows"][at].double()
            grad_rows[at] = s["weights"][on, k].double()[:, None] * grad_y[on]
            grad_weights[on, k] = (grad_y[on] * s["rows"][at].double()).sum(1)
        return {"grad_rows": grad_rows, "grad_weights": grad_weights, "grad_x": y}
    row = s["ids"].to(torch.int64) - case["first"]
    on = ((row >= 0) & (row < case["vocab"])).nonzero()[:, 0]
    if kind == "embed":
        y = torch.zeros(case["tokens"], case["cols"], device="cuda", dtype=torch.float64)
        y[on] = s["table"][row[on]].double() * s["scale"]
        return {"y": y}
    grad = torch.zeros(case["vocab"], case["cols"], device="cuda", dtype=torch.float64)
    grad.index_add_(0, row[on], s["grad_y"][on].double())
    grad *= s["scale"]
    if case["add"]:
        grad += s["total"].double()
    return {"grad": grad}
