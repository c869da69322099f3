"""Timed cases of the operators that follow a verification step: log
probabilities of the emitted tokens (token_logprobs), distillation of the
draft model from the target's top alternatives (distill_topk and
distill_topk_backward), and the cache slots of the next step
(advance_blocks).

run() computes a case in plain torch operations in 32 bits, or, where `own`
is true, through the library's calls.  exact() gives the same results from
the definitions in 64 bits.
"""

import math

import torch

own = False

DEVICE = "cuda"
NEG_INF = float("-inf")


# ------------------------------------------------------------------ cases --


def _logprobs(name, rows, V, dtype, top_k, T=1.0, skip=0.0, masked=0.0, pad=0):
    """skip: share of rows without a token; masked: share of rows where all
    but a few tokens are ruled out; pad: unused columns at each row's end."""
    return dict(name=name, op="logprobs", rows=rows, V=V, dtype=dtype, top_k=top_k, T=T, skip=skip, masked=masked,
                pad=pad)


def _distill(name, rows, V, dtype, top_k, tail, form, T=1.0, skip=0.0, ragged=0.0):
    """form: "grad" (loss and gradient in one call), "loss" (loss alone),
    "two" (loss, then the gradient for per-row upstream gradients); skip:
    share of rows of weight zero; ragged: share of rows with fewer than
    top_k teacher tokens."""
    return dict(name=name, op="distill", rows=rows, V=V, dtype=dtype, top_k=top_k, tail=tail, form=form, T=T,
                skip=skip, ragged=ragged)


def _blocks(name, B, page, max_blocks, tokens, chunk, prefills):
    """tokens: new tokens of a decoding request; prefills: how many requests
    bring up to `chunk` prompt tokens instead."""
    return dict(name=name, op="blocks", B=B, page=page, max_blocks=max_blocks, tokens=tokens, chunk=chunk,
                prefills=prefills)


def listed():
    return [
        # one request with 4 drafted tokens, five alternatives each: the latency of a single answer
        _logprobs("logprobs-1req", 5, 128256, "bf16", 5),
        # 64 requests of 4 drafts with 20 alternatives; rejected positions have no token
        _logprobs("logprobs-b64", 320, 128256, "bf16", 20, skip=0.4),
        # fp32 rows of an odd vocabulary, many alternatives, half of the rows under a grammar's mask
        _logprobs("logprobs-odd-f32", 777, 50021, "f32", 64, T=0.7, masked=0.5),
        # 1024 requests of 3 drafts at the largest vocabulary of the bench
        _logprobs("logprobs-b1024", 4096, 129280, "bf16", 8, skip=0.25),
        # scoring a prompt: no alternatives, rows padded to a wider buffer
        _logprobs("logprobs-score", 2048, 128256, "bf16", 0, pad=256),
        # a small online update of the draft
        _distill("distill-small", 32, 32000, "bf16", 16, "bucket", "grad"),
        # every position of the bench batch (256 requests, 8 drafts) in one training call
        _distill("distill-b256", 2304, 128256, "bf16", 64, "bucket", "grad", T=2.0, skip=0.1),
        # fp32 logits of an odd vocabulary, teachers of differing width
        _distill("distill-odd-f32", 301, 50021, "f32", 33, "renorm", "grad", ragged=0.5),
        # validation loss, no gradient, the widest teacher
        _distill("distill-eval", 1024, 129280, "bf16", 128, "renorm", "loss"),
        # the loss and, once the upstream gradients are known, its backward pass
        _distill("distill-two-step", 1024, 128256, "bf16", 20, "bucket", "two"),
        # the decoding step of 64 requests: last token and 4 drafts each
        _blocks("blocks-decode", 64, 16, 512, 5, 0, 0),
        # 1024 requests, an eighth of them in chunked prefill
        _blocks("blocks-mixed", 1024, 64, 1024, 9, 4096, 128),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_BYTES = 4096 * 129280 * 2  # the largest listed call's logits


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "distill", "distill", "blocks"])
    if op == "blocks":
        c = _blocks("", _log_uniform(rng, 1, 1024), rng.choice([8, 16, 32, 48, 64, 128]), _log_uniform(rng, 80, 1024),
                    rng.randint(1, 16), _log_uniform(rng, 64, 4096), 0)
        c["prefills"] = rng.randint(0, c["B"] // 8)
        c["chunk"] = min(c["chunk"], c["page"] * c["max_blocks"] // 4)
    else:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        V = _log_uniform(rng, 32, 262144)
        if rng.random() < 0.5:
            V = max(32, V // 64 * 64)
        most = MOST_BYTES // (V * (2 if dtype == "bf16" else 4) * (2 if op == "distill" else 1))
        rows = _log_uniform(rng, 1, max(1, min(4096, most)))
        T = rng.choice([0.5, 0.7, 1.0, 1.3, 2.0])
        if op == "logprobs":
            c = _logprobs("", rows, V, dtype, min(V, rng.choice([0, 1, 5, 20, 64, 128])), T,
                          rng.choice([0.0, 0.25, 0.5]), rng.choice([0.0, 0.3]), rng.choice([0, 0, 3, 64]))
        else:
            c = _distill("", rows, V, dtype, min(V, _log_uniform(rng, 1, 128)), rng.choice(["bucket", "renorm"]),
                         rng.choice(["grad", "grad", "loss", "two"]), T, rng.choice([0.0, 0.1]),
                         rng.choice([0.0, 0.5]))
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _rows_fp32(rows, V, g):
    """N(0, 1) logits with a Zipf-shaped bias of up to +8 on random tokens."""
    x = torch.randn(rows, V, generator=g, device=DEVICE)
    n = min(V, 1024)
    bias = (8.0 * torch.arange(1, n + 1, device=DEVICE, dtype=torch.float32).pow(-1.1)).expand(rows, n)
    at = torch.randint(0, V, (rows, n), generator=g, device=DEVICE)
    return x.add_(torch.zeros_like(x).scatter_reduce_(1, at, bias, "amax"))


def _some(rows, share, g):
    """floor(rows * share) random rows, as a mask."""
    return torch.rand(rows, generator=g, device=DEVICE).argsort() < int(rows * share)


def _prepare_logprobs(c, g):
    R, V, K = c["rows"], c["V"], c["top_k"]
    full = torch.empty(R, V + c["pad"], dtype=_DTYPE[c["dtype"]], device=DEVICE)
    logits = full[:, :V]
    tokens = torch.empty(R, dtype=torch.int32, device=DEVICE)
    masked = _some(R, c["masked"], g)
    if c["pad"]:
        full[:, V:] = 30.0  # not part of the row
    for r0 in range(0, R, 512):
        x = _rows_fp32(min(512, R - r0), V, g)
        rule = masked[r0:r0 + 512, None] & (torch.rand(x.shape, generator=g, device=DEVICE) > 40.0 / V)
        rule[:, V // 2] = False
        x.masked_fill_(rule, NEG_INF)
        logits[r0:r0 + 512] = x.to(logits.dtype)
        noise = torch.rand(x.shape, generator=g, device=DEVICE).clamp_(1e-20).log_().neg_().log_()
        tokens[r0:r0 + 512] = (x / c["T"] - noise).argmax(1).to(torch.int32)  # a sampled token
    tokens[_some(R, c["skip"], g)] = -1
    out = dict(logprob=torch.empty(R, device=DEVICE), rank=torch.empty(R, dtype=torch.int32, device=DEVICE),
               entropy=torch.empty(R, device=DEVICE), top_ids=torch.empty(R, K, dtype=torch.int32, device=DEVICE),
               top_logprobs=torch.empty(R, K, device=DEVICE), dev_error=torch.empty(1, dtype=torch.int32, device=DEVICE))
    return dict(case=c, logits=logits, tokens=tokens, out=out)


def _prepare_distill(c, g):
    R, V, K = c["rows"], c["V"], c["top_k"]
    student = torch.empty(R, V, dtype=_DTYPE[c["dtype"]], device=DEVICE)
    ids = torch.empty(R, K, dtype=torch.int32, device=DEVICE)
    logprobs = torch.empty(R, K, device=DEVICE)
    for r0 in range(0, R, 512):
        x = _rows_fp32(min(512, R - r0), V, g)
        top, at = (x - x.logsumexp(1, keepdim=True)).topk(K, dim=1)
        ids[r0:r0 + 512], logprobs[r0:r0 + 512] = at.to(torch.int32), top
        student[r0:r0 + 512] = x.add_(torch.randn(x.shape, generator=g, device=DEVICE), alpha=0.7).to(student.dtype)
    width = torch.randint(0, K + 1, (R,), generator=g, device=DEVICE)
    absent = _some(R, c["ragged"], g)[:, None] & (torch.arange(K, device=DEVICE) >= width[:, None])
    ids[absent] = -1
    weights = torch.rand(R, generator=g, device=DEVICE) + 0.5
    weights[_some(R, c["skip"], g)] = 0.0
    out = dict(loss=torch.empty(R, device=DEVICE), row_stats=torch.empty(R, 8, device=DEVICE),
               dev_error=torch.empty(1, dtype=torch.int32, device=DEVICE))
    if c["form"] != "loss":
        out["grad"] = torch.empty_like(student)
    return dict(case=c, student=student, ids=ids, logprobs=logprobs, weights=weights, out=out)


def _prepare_blocks(c, g):
    B, P, M = c["B"], c["page"], c["max_blocks"]
    ints = dict(generator=g, device=DEVICE)
    new = torch.full((B,), c["tokens"], dtype=torch.int32, device=DEVICE)
    if c["prefills"]:
        at = torch.rand(B, **ints).argsort()[:c["prefills"]]
        new[at] = torch.randint(1, c["chunk"] + 1, (c["prefills"],), **ints).to(torch.int32)
    new[torch.rand(B, **ints) < 0.05] = 0  # requests that sit the step out
    most = P * M - 2 * max(c["tokens"], c["chunk"]) - 16
    lens = torch.randint(0, most, (B,), **ints).to(torch.int32)
    accepted = torch.randint(0, c["tokens"], (B,), **ints).to(torch.int32)
    held = (lens + c["tokens"] + P - 1) // P  # the last step's tokens have their blocks
    pool = B * M
    blocks = torch.randperm(pool, **ints).to(torch.int32)
    start = torch.cumsum(held, 0) - held
    column = torch.arange(M, device=DEVICE)
    table = torch.where(column < held[:, None], blocks[(start[:, None] + column).clamp_(max=pool - 1)], -1)
    used = int(held.sum())
    free = blocks[used:].contiguous()
    max_tokens = c["B"] * c["tokens"] + c["prefills"] * c["chunk"]
    i32 = dict(dtype=torch.int32, device=DEVICE)
    out = dict(seq_lens=torch.empty(B, **i32), held=torch.empty(B, **i32), free_count=torch.empty(1, **i32),
               cu_tokens=torch.empty(B + 1, **i32), slots=torch.empty(max_tokens, dtype=torch.int64, device=DEVICE),
               positions=torch.empty(max_tokens, **i32), dev_error=torch.empty(1, **i32))
    return dict(case=c, seq_lens=lens, accepted=accepted, new=new, held=held.to(torch.int32), table=table.to(torch.int32),
                free=free, free_count=torch.full((1,), free.numel(), **i32), max_tokens=max_tokens, out=out)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, g)
    if case["op"] == "distill":
        return _prepare_distill(case, g)
    return _prepare_blocks(case, g)


# ------------------------------------------------------------ plain forms --


def _plain_logprobs(s):
    c, tokens = s["case"], s["tokens"]
    R, V, K = c["rows"], c["V"], c["top_k"]
    raw = s["logits"].float()
    x = raw / c["T"]
    m = x.amax(1, keepdim=True)
    d = x - m
    e = d.exp()
    z = e.sum(1, keepdim=True)
    log_z = z.log()
    # (x - m) e is 0 where x is -inf
    entropy = (log_z - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / z)[:, 0]
    has = tokens >= 0
    at = tokens.clamp(min=0).long()[:, None]
    logprob = (d.gather(1, at) - log_z)[:, 0]
    column = torch.arange(V, device=raw.device)
    raw_t = raw.gather(1, at)
    rank = 1 + ((raw > raw_t) | ((raw == raw_t) & (column < at))).sum(1)
    # one integer key per element, larger = earlier: the value's order, then the lower index
    bits = (raw + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (order << 32) | (V - 1 - column)
    top = V - 1 - (key.topk(K, dim=1).values & 0xFFFFFFFF) if K else key[:, :0]
    top_logprobs = d.gather(1, top) - log_z
    return dict(logprob=torch.where(has, logprob, 0.0), rank=torch.where(has, rank, -1).to(torch.int32),
                entropy=torch.where(has, entropy, 0.0),
                top_ids=torch.where(has[:, None], top, -1).to(torch.int32),
                top_logprobs=torch.where(has[:, None], top_logprobs, NEG_INF))


def _plain_distill(s):
    c = s["case"]
    R, V = c["rows"], c["V"]
    x = s["student"].float() / c["T"]
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    z = e.sum(1, keepdim=True)
    valid = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    log_q = x.gather(1, at) - m - z.log()
    log_t = torch.where(valid, s["logprobs"], NEG_INF)
    if c["tail"] == "renorm":
        most = log_t.amax(1, keepdim=True).clamp(min=-1e30)
        log_t = log_t - (most + (log_t - most).exp().sum(1, keepdim=True).log()).clamp(min=-1e30)
    t = log_t.exp()
    in_top = torch.zeros(R, V + 1, dtype=torch.bool, device=x.device)
    in_top = in_top.scatter_(1, torch.where(valid, s["ids"], V).long(), True)[:, :V]
    q_tail = torch.where(in_top, 0.0, e).sum(1, keepdim=True) / z
    loss = torch.where(t > 0, t * (log_t - log_q), 0.0).sum(1, keepdim=True)
    if c["tail"] == "bucket":
        t_tail = (1.0 - t.sum(1, keepdim=True)).clamp(min=0.0)
        # with no tail in the student, the teacher's is rounding
        t_tail = torch.where((q_tail > 0) | (t_tail > 2.0**-16), t_tail, 0.0)
        loss = loss + torch.where(t_tail > 0, t_tail * (t_tail.log() - q_tail.log()), 0.0)
    else:
        t_tail = torch.zeros_like(q_tail)
    w = s["weights"][:, None]
    result = dict(loss=torch.where(w != 0, loss, 0.0)[:, 0])
    if c["form"] != "loss":
        mass = t.sum(1, keepdim=True) + t_tail
        share = torch.where(q_tail > 0, t_tail / q_tail, 0.0)
        grad = e / z * torch.where(in_top, mass, mass - share)
        grad = grad.scatter_add_(1, at, -t) / c["T"]
        result["grad"] = torch.where(w != 0, grad * w, 0.0).to(s["student"].dtype)
    return result


def _plain_blocks(s):
    c = s["case"]
    P, M, B = c["page"], c["max_blocks"], c["B"]
    new, held, free = s["new"], s["held"], s["free"]
    lens = s["seq_lens"] + s["accepted"] + 1
    need = torch.maximum(held, torch.div(lens + new + P - 1, P, rounding_mode="floor"))
    want = need - held
    end = torch.cumsum(want, 0)
    served = (end <= s["free_count"]) | (want == 0)
    need = torch.where(served, need, held)
    first = end - want
    column = torch.arange(M, device=lens.device)
    added = (column >= held[:, None]) & (column < need[:, None])
    # blocks leave the free list from its end, in request order
    place = s["free_count"] - 1 - (first[:, None] + column - held[:, None])
    table = torch.where(added, free[place.clamp(0, max(0, free.numel() - 1)).long()], s["table"])
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=lens.device), torch.cumsum(new, 0)])
    i = torch.arange(s["max_tokens"], device=lens.device)
    b = torch.searchsorted(cu, i, right=True) - 1
    live = i < cu[-1]
    b = b.clamp(max=B - 1)
    position = torch.where(live, lens[b] + i - cu[b], 0)
    block = table[b, torch.div(position, P, rounding_mode="floor").clamp(max=M - 1)].long()
    slots = torch.where(live & served[b], block * P + position % P, -1)
    taken = torch.where(served, want, 0).sum()
    return dict(seq_lens=lens.to(torch.int32), held=need.to(torch.int32), table=table,
                free_count=(s["free_count"] - taken).to(torch.int32), cu_tokens=cu.to(torch.int32), slots=slots,
                positions=position.to(torch.int32))


# ------------------------------------------------------------ library calls --


def _own_logprobs(s):
    import speculative_decoding_verification_60_gb300 as sv

    c = s["case"]
    out = sv.token_logprobs(s["logits"], s["tokens"], c["T"], c["top_k"], out=s["out"])
    return {key: out[key] for key in ("logprob", "rank", "entropy", "top_ids", "top_logprobs")}


def _own_distill(s):
    import speculative_decoding_verification_60_gb300 as sv

    c = s["case"]
    tail = sv.TAIL_BUCKET if c["tail"] == "bucket" else sv.TAIL_RENORM
    out = sv.distill_topk(s["student"], s["ids"], s["logprobs"], weights=s["weights"], temperature=c["T"], tail=tail,
                          with_grad=c["form"] == "grad", out=s["out"])
    if c["form"] == "loss":
        return dict(loss=out["loss"])
    if c["form"] == "two":
        sv.distill_topk_backward(s["student"], s["ids"], s["logprobs"], out["row_stats"], s["weights"],
                                 temperature=c["T"], out=out)
    return dict(loss=out["loss"], grad=out["grad"])


def _own_blocks(s):
    import speculative_decoding_verification_60_gb300 as sv

    out = sv.advance_blocks(s["seq_lens"], s["new"], s["table"], s["held"], s["free"], s["free_count"],
                            s["case"]["page"], s["max_tokens"], accepted_len=s["accepted"], out=s["out"])
    return dict(seq_lens=out["seq_lens"], held=out["held"], table=s["table"], free_count=out["free_count"],
                cu_tokens=out["cu_tokens"], slots=out["slots"], positions=out["positions"])


def run(state):
    op = state["case"]["op"]
    if op == "logprobs":
        return _own_logprobs(state) if own else _plain_logprobs(state)
    if op == "distill":
        return _own_distill(state) if own else _plain_distill(state)
    return _own_blocks(state) if own else _plain_blocks(state)


# ------------------------------------------------------------------- costs --


def work(case):
    if case["op"] == "blocks":
        B, P = case["B"], case["page"]
        tokens = B * case["tokens"] + case["prefills"] * case["chunk"] // 2
        blocks = tokens // P + B
        return dict(bytes=16 * B + 12 * B + 12 * tokens + 12 * blocks, flops=4 * tokens)
    size = 2 if case["dtype"] == "bf16" else 4
    rows = case["rows"] - int(case["rows"] * case["skip"])
    elements = rows * case["V"]
    if case["op"] == "logprobs":
        return dict(bytes=elements * size + case["rows"] * (16 + 8 * case["top_k"]), flops=8 * elements)
    small = case["rows"] * (8 + 8 * case["top_k"])
    zeros = (case["rows"] - rows) * case["V"] * size  # a skipped row's gradient is written
    if case["form"] == "loss":
        return dict(bytes=elements * size + small, flops=6 * elements)
    # the two calls of "two" read the logits once each: nothing can be kept between them
    reads = 2 if case["form"] == "two" else 1
    return dict(bytes=elements * size * (reads + 1) + zeros + small * reads, flops=10 * elements)


# ------------------------------------------------------------------- exact --


def _exact_logprobs(s):
    c = s["case"]
    lists = dict(logprob=[], entropy=[], top_logprobs=[])
    for r0 in range(0, c["rows"], 256):
        raw = s["logits"][r0:r0 + 256].double()
        tokens = s["tokens"][r0:r0 + 256].long()
        log_p = raw / c["T"]
        log_p = log_p - torch.logsumexp(log_p, 1, keepdim=True)
        p = log_p.exp()
        h = -(p * log_p.clamp(min=-1e6)).sum(1)
        lists["entropy"].append(torch.where(tokens >= 0, h, 0.0))
        lists["logprob"].append(torch.where(tokens >= 0, log_p.gather(1, tokens.clamp(min=0)[:, None])[:, 0], 0.0))
        top = log_p.topk(c["top_k"], dim=1).values if c["top_k"] else log_p[:, :0]  # ties share a value
        lists["top_logprobs"].append(torch.where(tokens[:, None] >= 0, top, NEG_INF))
    got = {key: torch.cat(v) for key, v in lists.items()}
    return dict(logprob=got["logprob"], rank=None, entropy=got["entropy"], top_ids=None,
                top_logprobs=got["top_logprobs"])


def _exact_distill(s):
    c = s["case"]
    losses, grads = [], []
    for r0 in range(0, c["rows"], 256):
        x = s["student"][r0:r0 + 256].double() / c["T"]
        ids = s["ids"][r0:r0 + 256].long()
        w = s["weights"][r0:r0 + 256].double()[:, None]
        n, V = x.shape
        t = torch.where(ids >= 0, s["logprobs"][r0:r0 + 256].double().exp(), 0.0)
        if c["tail"] == "renorm":
            t = t / t.sum(1, keepdim=True).clamp(min=1e-300)
        # the teacher over the whole vocabulary, one column more for absent entries
        column = torch.where(ids >= 0, ids, V)
        teacher = torch.zeros(n, V + 1, dtype=torch.float64, device=x.device).scatter_(1, column, t)[:, :V]
        named = torch.zeros(n, V + 1, dtype=torch.bool, device=x.device).scatter_(1, column, True)[:, :V]
        log_q = x - torch.logsumexp(x, 1, keepdim=True)
        loss = (torch.special.xlogy(teacher, teacher) - teacher * log_q.clamp(min=-1e300)).sum(1, keepdim=True)
        mass = t.sum(1, keepdim=True)
        target = teacher
        if c["tail"] == "bucket":
            rest = (1.0 - mass).clamp(min=0.0)
            log_rest = torch.logsumexp(log_q.masked_fill(named, NEG_INF), 1, keepdim=True)
            rest = torch.where((log_rest > NEG_INF) | (rest > 2.0**-16), rest, 0.0)
            loss = loss + torch.where(rest > 0, torch.special.xlogy(rest, rest) - rest * log_rest, 0.0)
            # the bucket's mass, spread as the student spreads it, makes the same gradient
            spread = rest * (log_q - log_rest).exp()
            target = torch.where(named, teacher, torch.where(log_rest > NEG_INF, spread, 0.0))
            mass = mass + rest
        losses.append(torch.where(w != 0, loss, 0.0)[:, 0])
        if c["form"] != "loss":
            grads.append(torch.where(w != 0, w * (mass * log_q.exp() - target) / c["T"], 0.0))
    got = dict(loss=torch.cat(losses))
    if grads:
        got["grad"] = torch.cat(grads)
    return got


def exact(case, seed):
    if case["op"] == "blocks":
        return None  # whole numbers
    state = prepare(case, seed)
    return _exact_logprobs(state) if case["op"] == "logprobs" else _exact_distill(state)
