"""Cases of the operators that choose: the best of a row, and what moves by the choice.

Two families, both a selection (the first few places of a sort) whose answer is a
small integer key by which rows are moved:

* a router's choice of experts (``route``): scores of a token's logits, a bias for
  balance, groups of experts, the best few with their weights, and the gradient of
  those weights with respect to the logits (``route_grad``);
* beam search: the best continuations over all beams and the whole vocabulary
  (``beam``), and the beams' states put in the order of the chosen parents
  (``reorder``).

``own`` chooses what ``run`` computes with: False, elementary torch operations; True,
the operators of ``sorting_lsd_radix_sort_amd``.  Choices are compared in 64 bits, so
that they are those of the definition also where two scores agree to seven digits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "i32": 4, "i64": 8}


def listed():
    return [
        # Serving, one step of a batch of four sequences: latency counts.
        {"name": "route_decode", "kind": "route", "tokens": 4, "experts": 128, "slots": 8, "scores": "softmax",
         "bias": False, "groups": 1, "kept": 1, "group_score": "max", "normalize": True, "scale": 1.0,
         "dtype": "bf16", "ids": "i32"},
        # A prompt's odd rest; the experts of three of eight nodes, raw probabilities scaled up.
        {"name": "route_nodes", "kind": "route", "tokens": 2047, "experts": 160, "slots": 6, "scores": "softmax",
         "bias": False, "groups": 8, "kept": 3, "group_score": "max", "normalize": False, "scale": 16.0,
         "dtype": "f16", "ids": "i32"},
        # Training or a long prompt: 16K tokens, balanced by a bias, two experts speaking for a group.
        {"name": "route_prompt", "kind": "route", "tokens": 16384, "experts": 256, "slots": 8, "scores": "sigmoid",
         "bias": True, "groups": 8, "kept": 4, "group_score": "top2", "normalize": True, "scale": 2.5,
         "dtype": "f32", "ids": "i64"},
        # Backward pass of a small mixture with odd sizes (a test model, a last partial batch).
        {"name": "route_grad_odd", "kind": "route_grad", "tokens": 301, "experts": 8, "slots": 2,
         "scores": "softmax", "normalize": True, "scale": 1.0, "dtype": "bf16", "ids": "i64"},
        # Backward pass of a training micro-batch of 16K tokens, every logit having its share.
        {"name": "route_grad_train", "kind": "route_grad", "tokens": 16384, "experts": 256, "slots": 8,
         "scores": "softmax", "normalize": False, "scale": 1.0, "dtype": "f32", "ids": "i64"},
        # One sequence in four beams, twice as many continuations kept as beams: latency counts.
        {"name": "beam_one", "kind": "beam", "batch": 1, "beams": 4, "vocab": 32000, "count": 8, "normalize": True,
         "finished": False, "dtype": "f16", "ids": "i32"},
        # Odd sizes, some beams finished already, log probabilities that were worked on before.
        {"name": "beam_odd", "kind": "beam", "batch": 7, "beams": 5, "vocab": 5003, "count": 10, "normalize": False,
         "finished": True, "dtype": "f32", "ids": "i64"},
        # A served batch with a large vocabulary.
        {"name": "beam_serve", "kind": "beam", "batch": 16, "beams": 4, "vocab": 131072, "count": 8,
         "normalize": True, "finished": True, "dtype": "bf16", "ids": "i32"},
        # Many wide searches at once.
        {"name": "beam_wide", "kind": "beam", "batch": 64, "beams": 8, "vocab": 131072, "count": 16,
         "normalize": True, "finished": False, "dtype": "bf16", "ids": "i64"},
        # The cache of one search, 257 of 512 positions filled, reordered where it is.
        {"name": "reorder_one", "kind": "reorder", "batch": 1, "beams": 4, "count": 4, "layers": 8, "heads": 8,
         "length": 257, "room": 512, "dim": 128, "in_place": True, "dtype": "f16"},
        # Odd sizes, more beams afterwards than before, into another buffer.
        {"name": "reorder_odd", "kind": "reorder", "batch": 7, "beams": 5, "count": 9, "layers": 1, "heads": 3,
         "length": 129, "room": 131, "dim": 65, "in_place": False, "dtype": "f32"},
        # The caches of a served batch at a thousand positions, where they are.
        {"name": "reorder_serve", "kind": "reorder", "batch": 16, "beams": 8, "count": 8, "layers": 2, "heads": 8,
         "length": 1023, "room": 1024, "dim": 128, "in_place": True, "dtype": "bf16"},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["route", "route", "route_grad", "beam", "beam", "reorder"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if kind in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * max(1, _log_int(rng, 8, 512) // groups)
        if rng.random() < 0.5:  # whole sixteens, as most mixtures have them
            experts = max(16, experts // 16 * 16)
        tokens = _log_int(rng, 1, min(32768, 16384 * 256 // experts))
        case = {"kind": kind, "tokens": tokens, "experts": experts, "slots": rng.randint(1, min(8, experts)),
                "scores": rng.choice(["softmax", "sigmoid"]), "normalize": rng.random() < 0.6,
                "scale": rng.choice([1.0, 1.0, 2.5]), "dtype": dtype, "ids": rng.choice(["i32", "i64"])}
        if kind == "route":
            kept = rng.randint(1, groups)
            while kept * (experts // groups) < case["slots"]:
                kept += 1
            case.update(bias=rng.random() < 0.5, groups=groups, kept=kept, group_score=rng.choice(["max", "top2"]))
        return case
    if kind == "beam":
        beams = rng.randint(1, 10)
        vocab = _log_int(rng, 1000, 200000)
        if rng.random() < 0.5:
            vocab = vocab // 64 * 64
        batch = _log_int(rng, 1, max(1, min(64, 64 * 8 * 131072 * 2 // (beams * vocab * BYTES[dtype]))))
        return {"kind": kind, "batch": batch, "beams": beams, "vocab": vocab,
                "count": beams * rng.choice([1, 2]), "normalize": rng.random() < 0.7,
                "finished": rng.random() < 0.5, "dtype": dtype, "ids": rng.choice(["i32", "i64"])}
    beams = rng.randint(1, 10)
    in_place = rng.random() < 0.6
    room, heads, layers = _log_int(rng, 16, 4096), rng.randint(1, 16), rng.randint(1, 4)
    dim = rng.choice([64, 128, 128, rng.randint(16, 256)])
    most = 16 * 8 * 2 * 8 * 1024 * 128 * 2 // (beams * layers * heads * room * dim * BYTES[dtype])
    return {"kind": kind, "batch": _log_int(rng, 1, max(1, min(64, most // 2))), "beams": beams,
            "count": beams if in_place else rng.randint(1, 10), "layers": layers, "heads": heads,
            "length": rng.randint(1, room), "room": room, "dim": dim, "in_place": in_place, "dtype": dtype}


# ------------------------------------------------------------------- inputs


def _randn(g, shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return x if scale == 1.0 else x.mul_(scale)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    dtype = DTYPES[case["dtype"]]
    if case["kind"] in ("route", "route_grad"):
        t, e = case["tokens"], case["experts"]
        # some experts are liked better than others
        s["logits"] = (_randn(g, (t, e)) + _randn(g, (1, e), scale=0.5)).to(dtype)
        if case["kind"] == "route":
            # a bias that was stepped up and down by a thousandth
            steps = torch.randint(-100, 101, (e,), generator=g, device="cuda")
            s["bias_values"] = steps.float() * 1e-3 if case["bias"] else None
            return s
        s["chosen"], _ = _best(s["logits"].double(), case["slots"])
        s["chosen"] = s["chosen"].to(DTYPES[case["ids"]])
        s["grad_weights"] = _randn(g, (t, case["slots"]))
        return s
    if case["kind"] == "beam":
        b, k = case["batch"], case["beams"]
        logits = _randn(g, (b, k, case["vocab"]), scale=2.0)
        if not case["normalize"]:
            logits = torch.log_softmax(logits, -1)
        s["logits"] = logits.to(dtype)
        s["beam_scores"] = -torch.rand(b, k, generator=g, device="cuda").mul_(4.0).cumsum(1)
        s["done"] = torch.rand(b, k, generator=g, device="cuda") < 0.25 if case["finished"] else None
        s["end_id"] = 2
        return s
    b, k, n = case["batch"], case["beams"], case["count"]
    shape = (case["layers"], b, k, case["heads"], case["room"], case["dim"])
    s["cache"] = _randn(g, shape, dtype)
    s["parents"] = torch.randint(0, k, (b, n), generator=g, device="cuda", dtype=torch.int32)
    return s


# --------------------------------------------------------------- plain forms


def _best(values, count):
    """Places and values of the `count` largest of each row (float64), the largest first and of equal ones the
    lowest; the number of columns and -inf where none is left."""
    n = values.shape[1]
    values = values.clone()
    place = torch.arange(n, device=values.device, dtype=torch.int32)
    places, best = [], []
    for _ in range(count):
        top = values.amax(1, keepdim=True)
        at = torch.where(values == top, place, n).amin(1, keepdim=True).to(torch.int64)
        values.scatter_(1, at, -math.inf)
        places.append(torch.where(top == -math.inf, n, at))
        best.append(top)
    return torch.cat(places, 1), torch.cat(best, 1)


def _plain_scores(logits, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    t, e, groups = s["tokens"], s["experts"], s["groups"]
    choice = _plain_scores(s["logits"].double(), s["scores"])
    if s["bias_values"] is not None:
        choice = choice + s["bias_values"].double()
    if s["kept"] < groups:
        each = choice.reshape(t * groups, e // groups)
        spoken = _best(each, 1 if s["group_score"] == "max" else min(2, e // groups))[1].sum(1).reshape(t, groups)
        kept = torch.zeros(t, groups, device=choice.device, dtype=torch.bool)
        kept.scatter_(1, _best(spoken, s["kept"])[0], True)
        choice = torch.where(kept.repeat_interleave(e // groups, 1), choice, -math.inf)
    at = _best(choice, s["slots"])[0]
    weights = _plain_scores(s["logits"].float(), s["scores"]).gather(1, at)
    if s["normalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    return {"ids": at.to(DTYPES[s["ids"]]), "weights": weights * s["scale"]}


def _plain_route_grad(s):
    at = s["chosen"].to(torch.int64)
    scores = _plain_scores(s["logits"].float(), s["scores"])
    grad = s["grad_weights"].float() * s["scale"]
    if s["normalize"]:
        taken = scores.gather(1, at)
        total = taken.sum(1, keepdim=True)
        grad = (grad - (grad * taken).sum(1, keepdim=True) / total) / total
    grad_scores = torch.zeros_like(scores).scatter_add_(1, at, grad)
    if s["scores"] == "sigmoid":
        out = grad_scores * scores * (1.0 - scores)
    else:
        out = scores * (grad_scores - (grad_scores * scores).sum(1, keepdim=True))
    return {"grad_logits": out.to(s["logits"].dtype)}


def _plain_beam(s):
    b, k, v = s["logits"].shape
    total = s["logits"].double()
    if s["normalize"]:
        top = total.amax(2, keepdim=True)
        total = total - (top + torch.log(torch.exp(total - top).sum(2, keepdim=True)))
    total = total + s["beam_scores"].double()[:, :, None]
    if s["done"] is not None:
        only = torch.full((v,), -math.inf, device=total.device, dtype=torch.float64)
        only[s["end_id"]] = 0.0
        total = torch.where(s["done"][:, :, None], s["beam_scores"].double()[:, :, None] + only, total)
    at, best = _best(total.reshape(b, k * v), s["count"])
    none = at == k * v
    return {"scores": best.float(), "parents": torch.where(none, -1, at // v).to(torch.int32),
            "tokens": torch.where(none, -1, at % v).to(DTYPES[s["ids"]])}


def _filled(s):
    return s["cache"][:, :, :, :, :s["length"]]


def _plain_reorder(s):
    b = torch.arange(s["batch"], device="cuda")[:, None]
    moved = _filled(s)[:, b, s["parents"].to(torch.int64)]
    if not s["in_place"]:
        return {"cache": moved.contiguous()}
    _filled(s).copy_(moved)
    return {"cache": s["cache"]}


def _own_run(s):
    import sorting_lsd_radix_sort_amd as lrs

    if s["kind"] == "route":
        ids, weights = lrs.route_tokens(s["logits"], s["slots"], scores=s["scores"], bias=s["bias_values"],
                                        num_groups=s["groups"], kept_groups=s["kept"], group_score=s["group_score"],
                                        normalize=s["normalize"], scale=s["scale"], dtype=DTYPES[s["ids"]])
        return {"ids": ids, "weights": weights}
    if s["kind"] == "route_grad":
        return {"grad_logits": lrs.route_tokens_grad(s["grad_weights"], s["logits"], s["chosen"], scores=s["scores"],
                                                     normalize=s["normalize"], scale=s["scale"])}
    if s["kind"] == "beam":
        scores, parents, tokens = lrs.beam_select(s["logits"], s["beam_scores"], s["count"],
                                                  normalize=s["normalize"], finished=s["done"], end_id=s["end_id"],
                                                  dtype=DTYPES[s["ids"]])
        return {"scores": scores, "parents": parents, "tokens": tokens}
    if not s["in_place"]:
        return {"cache": lrs.beam_reorder(_filled(s), s["parents"], dim=1)}
    lrs.beam_reorder(_filled(s), s["parents"], dim=1, out=_filled(s))
    return {"cache": s["cache"]}


def run(state):
    if own:
        return _own_run(state)
    plain = {"route": _plain_route, "route_grad": _plain_route_grad, "beam": _plain_beam, "reorder": _plain_reorder}
    return plain[state["kind"]](state)


# --------------------------------------------------------------------- work


def work(case):
    b = BYTES[case["dtype"]]
    if case["kind"] in ("route", "route_grad"):
        n, picks = case["tokens"] * case["experts"], case["tokens"] * case["slots"]
        moved = picks * (BYTES[case["ids"]] + 4)
        if case["kind"] == "route":
            return {"bytes": n * b + moved + 4 * case["experts"] * case["bias"], "flops": 4 * n}
        if case["scores"] == "softmax" and not case["normalize"]:
            return {"bytes": 2 * n * b + moved, "flops": 6 * n}
        return {"bytes": n * b + picks * b + moved, "flops": 12 * picks}
    if case["kind"] == "beam":
        rows = case["batch"] * case["beams"]
        read = rows * case["vocab"] * (0.75 if case["finished"] else 1.0)
        return {"bytes": int(read * b) + 4 * rows + case["batch"] * case["count"] * (8 + BYTES[case["ids"]]),
                "flops": int(read) * (4 if case["normalize"] else 1)}
    k, n = case["beams"], case["count"]
    if case["in_place"]:  # a beam that stays is neither read nor written for itself
        blocks = k * (1.0 - (1.0 - 1.0 / k) ** (k - 1)) + k - 1
    else:
        blocks = k * (1.0 - (1.0 - 1.0 / k) ** n) + n
    block = case["layers"] * case["heads"] * case["length"] * case["dim"] * b
    return {"bytes": int(case["batch"] * blocks * block) + 4 * case["batch"] * n, "flops": 0}


# -------------------------------------------------------------------- exact


def _exact_route(s):
    logits = s["logits"].double().cpu().numpy()
    t, e = logits.shape
    if s["scores"] == "sigmoid":
        scores = 1.0 / (1.0 + np.exp(-logits))
    else:
        scores = np.exp(logits - logits.max(1, keepdims=True))
        scores /= scores.sum(1, keepdims=True)
    choice = scores if s["bias_values"] is None else scores + s["bias_values"].double().cpu().numpy()
    groups, size = s["groups"], e // s["groups"]
    if s["kept"] < groups:
        by_group = np.sort(choice.reshape(t, groups, size), 2)
        spoken = by_group[:, :, -1:] if s["group_score"] == "max" else by_group[:, :, -2:]
        order = np.argsort(-spoken.sum(2), 1, kind="stable")
        out = np.ones((t, groups), bool)
        np.put_along_axis(out, order[:, :s["kept"]], False, 1)
        choice = np.where(np.repeat(out, size, 1), -np.inf, choice)
    ids = np.argsort(-choice, 1, kind="stable")[:, :s["slots"]]
    weights = np.take_along_axis(scores, ids, 1)
    if s["normalize"]:
        weights = weights / weights.sum(1, keepdims=True)
    return {"ids": torch.from_numpy(ids).to(DTYPES[s["ids"]]), "weights": torch.from_numpy(weights * s["scale"])}


def _exact_route_grad(s):
    """By the Jacobian of the weights' logarithms: d log w[j] / d logit[e] of the score, less its mean over the
    chosen where they are normalised."""
    logits, ids = s["logits"].double().cpu().numpy(), s["chosen"].to(torch.int64).cpu().numpy()
    grad = s["grad_weights"].double().cpu().numpy() * s["scale"]
    t, e = logits.shape
    if s["scores"] == "sigmoid":
        scores = 1.0 / (1.0 + np.exp(-logits))
    else:
        scores = np.exp(logits - logits.max(1, keepdims=True))
        scores /= scores.sum(1, keepdims=True)
    rows = np.arange(t)
    taken = scores[rows[:, None], ids]
    weights = taken / taken.sum(1, keepdims=True) if s["normalize"] else taken
    by_log = grad * weights  # with respect to log w
    if s["normalize"]:
        by_log = by_log - weights * by_log.sum(1, keepdims=True)
    out = np.zeros((t, e))
    if s["scores"] == "sigmoid":
        for k in range(ids.shape[1]):
            out[rows, ids[:, k]] += by_log[:, k] * (1.0 - taken[:, k])
    else:
        out -= scores * by_log.sum(1, keepdims=True)
        for k in range(ids.shape[1]):
            out[rows, ids[:, k]] += by_log[:, k]
    return {"grad_logits": torch.from_numpy(out)}


def _exact_beam(s):
    b, k, v = s["logits"].shape
    scores, parents, tokens = [], [], []
    for i in range(b):
        rows = s["logits"][i].double()
        if s["normalize"]:
            rows = rows - torch.logsumexp(rows, 1, keepdim=True)
        rows = rows + s["beam_scores"][i].double()[:, None]
        if s["done"] is not None:
            for j in s["done"][i].nonzero()[:, 0].tolist():
                rows[j] = -math.inf
                rows[j, s["end_id"]] = s["beam_scores"][i, j].double()
        best, at = torch.sort(rows.reshape(-1), descending=True, stable=True)
        best, at = best[:s["count"]], at[:s["count"]]
        none = best == -math.inf
        scores.append(best)
        parents.append(torch.where(none, -1, at // v).to(torch.int32))
        tokens.append(torch.where(none, -1, at % v).to(DTYPES[s["ids"]]))
    return {"scores": torch.stack(scores), "parents": torch.stack(parents), "tokens": torch.stack(tokens)}


def _exact_reorder(s):
    n, parents = s["count"], s["parents"].cpu().tolist()
    old = _filled(s)
    if s["in_place"]:
        whole = s["cache"].double()
        new = whole[:, :, :, :, :s["length"]]
    else:
        whole = new = torch.empty(old.shape[0], s["batch"], n, *old.shape[3:], device="cuda", dtype=torch.float64)
    for i in range(s["batch"]):
        for j in range(n):
            new[:, i, j] = old[:, i, parents[i][j]].double()
    return {"cache": whole}


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_grad": _exact_route_grad, "beam": _exact_beam,
            "reorder": _exact_reorder}[case["kind"]](s)
