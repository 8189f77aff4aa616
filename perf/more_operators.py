"""Cases of the operators of a batch of many requests around the dense FP8
product: low-rank adapters beside a shared projection, the plan that groups a
batch's tokens by adapter, and the log probabilities of given tokens with the
entropy and the top alternatives of each row of logits.

Formats (all row-major, the last index contiguous):
  ids      int32 [T]: each token's adapter; outside [0, L) it has none
  adapters a bf16 [L][r][K], b bf16 [L][N][r], a factor of each: fp32 [L]
  base     the shared projection's result, bf16 or fp32 [T][N]
  logits   bf16 or fp32 [T][V]

`run` with `own` false computes an operator with elementary torch operations
in 32 bits; with `own` true it calls the package.
"""

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of one request beside a projection
        dict(name="adapters decode", op="lora", T=1, K=4096, N=4096, r=16, L=16, ids="random", none=0.0, out="bf16"),
        # a decode batch: 64 requests, most with an adapter of their own
        dict(name="adapters batch", op="lora", T=64, K=4096, N=4096, r=16, L=64, ids="random", none=0.1, out="bf16"),
        # a large decode batch with adapters of a higher rank, several tokens to each
        dict(name="adapters crowd", op="lora", T=512, K=4096, N=2048, r=64, L=64, ids="random", none=0.1, out="bf16"),
        # a prefill chunk: the tokens of eight requests one after another
        dict(name="adapters prefill", op="lora", T=2048, K=4096, N=4096, r=32, L=16, ids="requests", requests=8, none=0.1, out="bf16"),
        # odd sizes, a projection kept in fp32
        dict(name="adapters odd", op="lora", T=333, K=1056, N=1111, r=24, L=5, ids="requests", requests=7, none=0.3, out="fp32"),
        # grouping a decode batch, and the largest prefill batch
        dict(name="plan batch", op="plan", T=64, L=64, ids="random", none=0.1),
        dict(name="plan chunk", op="plan", T=8192, L=256, ids="random", none=0.1),
        # one token sampled from a large vocabulary, with five alternatives
        dict(name="scores decode", op="scores", T=1, V=128256, type="bf16", given=1, top=5, entropy=True, mask=0.0),
        # the five positions of a speculative verify step: the drafted tokens only
        dict(name="scores verify", op="scores", T=5, V=128256, type="fp32", given=1, top=0, entropy=False, mask=0.0),
        # a decode batch whose grammar leaves a part of an odd vocabulary, twenty alternatives, four candidates each
        dict(name="scores batch", op="scores", T=77, V=50001, type="bf16", given=4, top=20, entropy=True, mask=0.7),
        # scoring a prompt's chunk
        dict(name="scores prompt", op="scores", T=2048, V=128256, type="bf16", given=1, top=5, entropy=True, mask=0.0),
        # the same of a small vocabulary in fp32
        dict(name="scores small", op="scores", T=2048, V=4096, type="fp32", given=1, top=1, entropy=True, mask=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("lora", "lora", "scores", "scores", "plan"))
    ids = dict(ids=rng.choice(("random", "requests")), requests=_log(rng, 1, 32), none=rng.choice((0.0, 0.1, 0.5)))
    if op == "lora":
        return dict(op=op, T=_log(rng, 1, 2048), K=32 * _log(rng, 2, 128), N=_log(rng, 33, 4096), r=8 * _log(rng, 1, 16),
                    L=_log(rng, 1, 64), out=rng.choice(("bf16", "bf16", "fp32")), **ids)
    if op == "plan":
        return dict(op=op, T=_log(rng, 1, 65536), L=_log(rng, 1, 1024), **ids)
    V = _log(rng, 100, 131072)
    return dict(op=op, T=_log(rng, 1, 1024), V=V, type=rng.choice(("bf16", "bf16", "fp32")), given=rng.choice((0, 1, 1, 4)),
                top=rng.choice((0, 1, 5, 20, 50)), entropy=True, mask=rng.choice((0.0, 0.0, 0.7)))


# ------------------------------------------------------------------ the inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _ids(g, c):
    """The batch's adapters: of every token by itself, or of requests whose tokens follow one another."""
    T, L = c["T"], c["L"]
    n = T if c["ids"] == "random" else min(T, c["requests"])
    who = torch.randint(0, L, (n,), generator=g, device=DEV)
    if c["none"]:
        who[torch.rand(n, generator=g, device=DEV) < c["none"]] = -1
    if n < T:
        cut = torch.rand(n - 1, generator=g, device=DEV).mul(T).long().sort().values
        who = who[torch.searchsorted(cut, torch.arange(T, device=DEV), right=True)]
    return who.to(torch.int32)


def _blocks(ids, L):
    """Tokens with an adapter in blocks of at most 64 tokens of one (the plain form's batched product), which the host knows."""
    order = torch.sort(ids, stable=True).indices
    order = order[int((ids < 0).sum()):]
    e = ids[order].long()
    counts = torch.bincount(e, minlength=L)
    size = max(1, min(64, int(counts.max())))
    blocks = (counts + size - 1) // size
    at = torch.arange(order.numel(), device=DEV) - (counts.cumsum(0) - counts)[e]
    return dict(rows=order, block=(blocks.cumsum(0) - blocks)[e] + at // size, at=at % size, size=size,
                e_block=torch.repeat_interleave(torch.arange(L, device=DEV), blocks))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=c, op=c["op"])
    if c["op"] == "scores":
        T, V = c["T"], c["V"]
        logits = torch.empty((T, V), device=DEV).normal_(0, 2.5, generator=g)
        likely = torch.randint(0, V, (T, 8), generator=g, device=DEV)
        logits.scatter_(1, likely, 8 + 6 * torch.rand((T, 8), generator=g, device=DEV))
        if c["mask"]:
            hidden = torch.rand(V, generator=g, device=DEV) < c["mask"]
            hidden[int(V * 0.1)] = False
            logits.masked_fill_(hidden, -math.inf)
            logits.scatter_(1, likely, 8 + 6 * torch.rand((T, 8), generator=g, device=DEV))
        s["logits"] = logits.to(_TYPES[c["type"]])
        # drafted and sampled tokens: the likely ones for the most part
        given = torch.where(torch.rand((T, 8), generator=g, device=DEV) < 0.9, likely,
                            torch.randint(0, V, (T, 8), generator=g, device=DEV))
        s["tokens"] = given[:, :c["given"]].to(torch.int32).contiguous() if c["given"] else None
        return s
    s["ids"] = _ids(g, c)
    if c["op"] == "plan":
        return s
    T, K, N, r, L = (c[n] for n in ("T", "K", "N", "r", "L"))
    # normal activations with a few large channels
    x = torch.randn((T, K), generator=g, device=DEV) * (1 + 9 * (torch.rand(K, generator=g, device=DEV) < 0.01))
    s["x"] = x.to(torch.bfloat16)
    s["base"] = torch.randn((T, N), generator=g, device=DEV).to(_TYPES[c["out"]])
    s["a"] = (torch.randn((L, r, K), generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16)
    s["b"] = (0.2 * torch.randn((L, N, r), generator=g, device=DEV)).to(torch.bfloat16)
    s["scales"] = torch.exp2(2 * torch.rand(L, generator=g, device=DEV) - 1)
    s["blocks"] = _blocks(s["ids"], L)
    if own:
        import quantized_routed_moe_amd as qm
        s["plan"] = qm.lora_plan(s["ids"], L)      # made once for a batch, for all its projections
    return s


# ------------------------------------------------------------------ plain forms

def _plain_plan(s):
    L = s["case"]["L"]
    ids = s["ids"].long()
    group = torch.where((ids >= 0) & (ids < L), ids, L)
    counts = torch.bincount(group, minlength=L + 1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return {"perm": torch.sort(group, stable=True).indices.to(torch.int32), "offsets": offsets.to(torch.int32)}


def _plain_lora(s):
    k = s["blocks"]
    x = s["x"].new_zeros((k["e_block"].numel(), k["size"], s["x"].shape[1]), dtype=torch.float32)
    x[k["block"], k["at"]] = s["x"][k["rows"]].float()
    v = torch.bmm(x, s["a"][k["e_block"]].float().transpose(1, 2).contiguous())
    d = torch.bmm(v, s["b"][k["e_block"]].float().transpose(1, 2).contiguous()) * s["scales"][k["e_block"]][:, None, None]
    out = s["base"].float()
    if out is s["base"]:
        out = out.clone()
    out[k["rows"]] += d[k["block"], k["at"]]
    return out.to(s["base"].dtype)


def _plain_scores(s):
    c, l = s["case"], s["logits"].float()
    m = l.amax(1, keepdim=True)
    d = l - m
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    out = {}
    if c["given"]:
        out["logprobs"] = d.gather(1, s["tokens"].long()) - log_total
    if c["entropy"]:
        out["entropy"] = (log_total - torch.where(e > 0, e * d, 0).sum(1, keepdim=True) / total)[:, 0]
    if c["top"]:
        # one key of value and place, so that of equal logits the lowest place comes first
        bits = (l + 0.0).view(torch.int32).long()
        V = c["V"]
        key = (torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) << 32) | (V - 1 - torch.arange(V, device=DEV))
        ids = V - 1 - (torch.topk(key, c["top"], dim=1).values & 0xFFFFFFFF)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = d.gather(1, ids) - log_total
    return out


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"lora": _plain_lora, "plan": _plain_plan, "scores": _plain_scores}[s["op"]](s)
    import quantized_routed_moe_amd as qm
    if s["op"] == "lora":
        return qm.lora_add(s["base"], s["x"], s["a"], s["b"], s["plan"], scales=s["scales"])
    if s["op"] == "plan":
        plan = qm.lora_plan(s["ids"], c["L"])
        return {"perm": plan.perm, "offsets": plan.offsets}
    logprobs, entropy, top_ids, top_logprobs = qm.token_logprobs(s["logits"], s["tokens"], top=c["top"], entropy=c["entropy"])
    out = {"logprobs": logprobs, "entropy": entropy, "top_ids": top_ids, "top_logprobs": top_logprobs}
    return {n: t for n, t in out.items() if t is not None}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in float64, adapter by adapter and a few rows at a time; the last rounding of an output is left out."""
    s, c = prepare(case, seed), case
    if c["op"] == "plan":
        return None
    if c["op"] == "lora":
        out = s["base"].double()
        for e in sorted(set(s["ids"].tolist())):
            if 0 <= e < c["L"]:
                t = torch.nonzero(s["ids"] == e)[:, 0]
                v = torch.mm(s["x"][t].double(), s["a"][e].double().t().contiguous())
                out[t] += float(s["scales"][e]) * torch.mm(v, s["b"][e].double().t().contiguous())
        return out
    parts = []
    for t in range(0, c["T"], 128):
        lp = torch.log_softmax(s["logits"][t:t + 128].double(), dim=1)
        o = {}
        if c["given"]:
            o["logprobs"] = lp.gather(1, s["tokens"][t:t + 128].long())
        if c["entropy"]:
            o["entropy"] = -torch.xlogy(lp.exp(), lp.exp()).sum(1)
        if c["top"]:
            o["top_logprobs"] = torch.sort(lp, dim=1, descending=True).values[:, :c["top"]]
        parts.append(o)
    out = {n: torch.cat([p[n] for p in parts]) for n in parts[0]}
    return {n: out.get(n) for n in ("logprobs", "entropy", "top_ids", "top_logprobs") if n in out or (n == "top_ids" and c["top"])}


# ------------------------------------------------------------------ the work of one pass

def _active(c):
    """Adapters that the batch is expected to use."""
    n = c["T"] if c["ids"] == "random" else min(c["T"], c["requests"])
    return c["L"] * (1 - (1 - (1 - c["none"]) / c["L"]) ** n)


def work(case):
    c = case
    size = {"bf16": 2, "fp32": 4}
    if c["op"] == "plan":
        return dict(bytes=8 * c["T"] + 4 * (c["L"] + 2), flops=c["T"])
    if c["op"] == "lora":
        T, K, N, r = c["T"], c["K"], c["N"], c["r"]
        live = T * (1 - c["none"])
        return dict(bytes=2 * live * K + 2 * T * N * size[c["out"]] + _active(c) * (2 * r * (K + N) + 4), flops=2 * live * r * (K + N))
    n = c["T"] * c["V"]
    outputs = 2 * c["given"] + (1 if c["entropy"] else 0) + 2 * c["top"]
    return dict(bytes=n * size[c["type"]] + 4 * c["T"] * outputs, flops=4 * n)
