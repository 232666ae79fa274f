"""Cases of the vocabulary-wide operators around the draft and verify step: shaping of logits (penalties for repeated
tokens, biases, grammar masks, temperature), the top logits of a teacher's rows, and the distillation loss against them
with its gradient.  Each has a plain form in elementary torch operations and a definition in 64 bits (exact)."""
import torch

own = False

V_FULL = 129280  # the vocabulary of the repository's workloads


# ------------------------------------------------------------------ cases
def _shape(name, R, P, V, dtype, out, hist, bias, masked):
    return {"name": name, "op": "shape", "R": R, "P": P, "V": V, "dtype": dtype, "out": out, "hist": hist, "bias": bias, "masked": masked}


def _top(name, n, V, dtype, k, tau, holes):
    return {"name": name, "op": "top", "n": n, "V": V, "dtype": dtype, "k": k, "tau": tau, "holes": holes}


def _distill(name, how, n, V, dtype, k, tau, tail):
    return {"name": name, "op": "distill", "how": how, "n": n, "V": V, "dtype": dtype, "k": k, "tau": tau, "tail": tail}


def listed():
    return [
        # one sequence decoding one token: latency, a chat-length history, short bias list
        _shape("shape-decode-1", 1, 1, V_FULL, "bf16", "f32", 700, 20, False),
        # 64 requests verifying five drafted tokens each, float32 rows, half of them under a grammar
        _shape("shape-verify-64-f32", 64, 6, V_FULL, "f32", "f32", 4096, 300, True),
        # few requests with long contexts: the history is as much work as the rows
        _shape("shape-long-16", 16, 6, V_FULL, "bf16", "bf16", 32768, 8, True),
        # the largest verification batch of the workloads
        _shape("shape-verify-1024", 1024, 6, V_FULL, "bf16", "bf16", 2048, 16, True),
        # the five rows of one block, few entries
        _top("top-block-5", 5, V_FULL, "bf16", 32, 1.0, False),
        # a training batch's teacher rows
        _top("top-1280-bf16", 1280, V_FULL, "bf16", 256, 2.0, False),
        # float32 teacher rows with masked vocabulary entries, the widest list
        _top("top-320-f32", 320, V_FULL, "f32", 1024, 1.0, True),
        # one small sequence, a vocabulary that is no multiple of a vector
        _distill("step-40-small", "step", 40, 20003, "bf16", 64, 1.0, True),
        # a batch through autograd: loss forward, gradient backward
        _distill("autograd-1280", "autograd", 1280, V_FULL, "bf16", 256, 2.0, True),
        # float32 student logits, teacher renormalised over its list
        _distill("step-640-f32", "step", 640, V_FULL, "f32", 1024, 1.0, False),
        # the largest training batch: 1,024 blocks of five positions
        _distill("step-5120", "step", 5120, V_FULL, "bf16", 128, 1.0, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["shape", "top", "distill"])
    V = rng.choice([V_FULL, _log_int(rng, 1000, 131072), _log_int(rng, 1000, 262144)])
    f32 = rng.random() < 0.4
    dt = "f32" if f32 else "bf16"
    cap = max(1, (5120 * V_FULL) // (V * (4 if f32 else 1)))
    if op == "shape":
        P = rng.choice([1, 5, 6])
        R = min(_log_int(rng, 1, 1024), max(1, cap // P))
        hist = min(_log_int(rng, 16, 32768), max(16, (1024 * 2048) // R))
        out = "f32" if f32 else rng.choice(["bf16", "f32"])
        case = _shape("", R, P, V, dt, out, hist, rng.choice([0, _log_int(rng, 1, 1000)]), rng.random() < 0.6)
    elif op == "top":
        n = min(_log_int(rng, 1, 5120), cap // 2 + 1)
        case = _top("", n, V, dt, min(V, _log_int(rng, 1, 1024)), rng.choice([1.0, 0.7, 2.0]), rng.random() < 0.4)
    else:
        n = min(_log_int(rng, 1, 5120), cap)
        case = _distill("", rng.choice(["step", "autograd"]), n, V, dt, min(V // 2, _log_int(rng, 1, 1024)), rng.choice([1.0, 1.5, 4.0]), rng.random() < 0.6)
    del case["name"]
    return case


def work(case):
    V = case["V"]
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "shape":
        n = case["R"] * case["P"]
        eo = 4 if case["out"] == "f32" else 2
        masks = (n + 1) // 2 if case["masked"] else 0
        # histories are 3/4 full on average; an entry of the bias list is an id and a value
        small = case["R"] * (4 * case["hist"] * 0.75 + 8 * case["bias"] + 4 * case["P"] + 24)
        return {"bytes": n * V * (es + eo) + masks * (V / 8) + small, "flops": 2.0 * n * V}
    n, k = case["n"], case["k"]
    if case["op"] == "top":
        return {"bytes": n * (V * es + 8 * k + 12), "flops": 4.0 * n * V}
    return {"bytes": n * (2.0 * V * es + 8 * k + 16), "flops": 8.0 * n * V}


# ----------------------------------------------------------------- inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(n, V, dtype, g, scale):
    """Rows [n, V] ~ N(0, scale) whose stride is a whole number of 16-byte vectors."""
    x = torch.empty(n, -(-V // 8) * 8, dtype=_DT[dtype], device="cuda")
    at = max(1, (1 << 28) // x.shape[1])
    for i in range(0, n, at):
        part = x[i:i + at]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(scale))
    return x[:, :V]


def _rand_int(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda")


def _uniform(g, shape):
    return torch.rand(shape, generator=g, device="cuda")


def _prepare_shape(c, g):
    R, P, V, H = c["R"], c["P"], c["V"], c["hist"]
    s = {"x": _rows(R * P, V, c["dtype"], g, 3.0), "out_dtype": _DT[c["out"]]}
    # tokens repeat as text does: a few ids often, the rest seldom
    s["history"] = (V * _uniform(g, (R, H)).pow(4)).to(torch.int32).clamp_(max=V - 1)
    s["history_len"] = _rand_int(g, H // 2, H + 1, (R,)).to(torch.int32)
    s["prompt_len"] = (s["history_len"] * _uniform(g, (R,))).to(torch.int32)
    s["draft"] = _rand_int(g, 0, V, (R, P - 1)).to(torch.int32) if P > 1 else None
    s["repetition"] = 1.0 + 0.3 * _uniform(g, (R,))
    s["frequency"] = 0.5 * _uniform(g, (R,))
    s["presence"] = 0.5 * _uniform(g, (R,))
    s["temperature"] = 0.5 + _uniform(g, (R,))
    s["bias"] = None
    if c["bias"]:
        n = min(c["bias"], V)
        ids = torch.sort(torch.rand((R, V), generator=g, device="cuda").topk(n, 1).indices, 1).values
        val = 4.0 * torch.randn((R, n), generator=g, device="cuda")
        val[_uniform(g, (R, n)) < 0.1] = -float("inf")  # banned tokens
        off = torch.arange(R + 1, dtype=torch.int64, device="cuda") * n
        s["bias"] = (off, ids.to(torch.int32).reshape(-1).contiguous(), val.reshape(-1).contiguous())
    s["mask"] = s["mask_row"] = None
    if c["masked"]:  # every second request follows a grammar, each of its rows in a state of its own
        M, W = ((R + 1) // 2) * P, (V + 31) // 32
        words = _rand_int(g, -2**31, 2**31, (M, W)).to(torch.int32)
        for _ in range(3):  # 1/16 of the vocabulary
            words &= _rand_int(g, -2**31, 2**31, (M, W)).to(torch.int32)
        words[1::3] = -1  # inside a free string: everything
        s["mask"] = words
        r = torch.arange(R * P, device="cuda")
        s["mask_row"] = torch.where((r // P) % 2 == 0, (r // P // 2) * P + r % P, -1).to(torch.int32)
    s["P"] = P
    return s


def _prepare_top(c, g):
    x = _rows(c["n"], c["V"], c["dtype"], g, 3.0)
    if c["holes"]:
        x[_uniform(g, x.shape) < 0.1] = -float("inf")
    return {"x": x, "k": c["k"], "tau": c["tau"]}


def _prepare_distill(c, g):
    n, V, k, tau = c["n"], c["V"], c["k"], c["tau"]
    x = _rows(n, V, c["dtype"], g, 2.0)
    ids = torch.empty(n, k, dtype=torch.int32, device="cuda")
    logits = torch.empty(n, k, device="cuda")
    lse = torch.empty(n, device="cuda")
    length = torch.full((n,), k, dtype=torch.int32, device="cuda")
    u = _uniform(g, (n,))
    length = torch.where(u < 0.1, (k * _uniform(g, (n,))).to(torch.int32) + 1, length).clamp_(max=k)
    length = torch.where(u < 0.03, torch.zeros_like(length), length)  # padding: nothing to learn
    at = max(1, (1 << 26) // V)
    for i in range(0, n, at):
        z = torch.randn((min(at, n - i), V), generator=g, device="cuda").mul_(1.2).add_(x[i:i + at].float(), alpha=0.8)
        lse[i:i + at] = torch.logsumexp(z.double() / tau, 1).float()
        top, at_ids = z.topk(k, 1)
        at_ids = torch.where(torch.arange(k, device="cuda") < length[i:i + at, None], at_ids, V + torch.arange(k, device="cuda"))
        at_ids, order = torch.sort(at_ids, 1)
        real = at_ids < V
        ids[i:i + at] = torch.where(real, at_ids, 0)
        logits[i:i + at] = torch.where(real, top.gather(1, order), 0.0)
    teacher = {"ids": ids, "logits": logits, "len": length, "lse": lse if c["tail"] else None}
    return {"x": x, "teacher": teacher, "tau": tau, "how": c["how"], "scale": _uniform(g, (n,)) / n}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"shape": _prepare_shape, "top": _prepare_top, "distill": _prepare_distill}[case["op"]](case, g)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------ plain forms
def _mask_bits(mask, V):
    bytes_ = mask.contiguous().view(torch.uint8)
    bits = (bytes_[:, :, None] >> torch.arange(8, dtype=torch.uint8, device="cuda")) & 1
    return bits.reshape(mask.shape[0], -1)[:, :V].bool()


def _plain_shape(s):
    n, V = s["x"].shape
    P = s["P"]
    R = n // P
    x = s["x"].float().view(R, P, V)
    at = torch.arange(s["history"].shape[1], device="cuda")
    live = at < s["history_len"][:, None]
    hist = s["history"].long()
    made = torch.zeros(R, V, device="cuda").scatter_add_(1, hist, (live & (at >= s["prompt_len"][:, None])).float())
    any_ = torch.zeros(R, V, device="cuda").scatter_add_(1, hist, live.float())
    count, seen = made[:, None], any_[:, None]
    if s["draft"] is not None:
        before = (torch.arange(P, device="cuda")[:, None] > torch.arange(P - 1, device="cuda")).float()
        d = torch.zeros(R, P, V, device="cuda").scatter_add_(2, s["draft"].long()[:, None].expand(R, P, P - 1), before.expand(R, P, P - 1))
        count, seen = count + d, seen + d
    rep, freq, pres, temp = (s[k][:, None, None] for k in ("repetition", "frequency", "presence", "temperature"))
    z = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    z = z - freq * count - pres * (count > 0)
    if s["bias"] is not None:
        off, ids, val = s["bias"]
        row = torch.arange(R, device="cuda").repeat_interleave(off[1:] - off[:-1], output_size=ids.numel())
        b = torch.zeros(R * V, device="cuda")
        b[row * V + ids] = val
        z = z + b.view(R, 1, V)
    z = (z / temp).view(n, V)
    if s["mask"] is not None:
        allowed = _mask_bits(s["mask"], V)[s["mask_row"].clamp(min=0).long()] | (s["mask_row"] < 0)[:, None]
        z = torch.where(allowed, z, -float("inf"))
    return {"logits": z.to(s["out_dtype"]), "status": torch.zeros(n, dtype=torch.int32, device="cuda")}


def _logsumexp(u):
    m = u.amax(1, keepdim=True)
    return (u - m).exp().sum(1, keepdim=True).log() + m


def _plain_top(s):
    n, V = s["x"].shape
    k = s["k"]
    x = s["x"].float()
    val, ids = torch.sort(x, dim=1, descending=True, stable=True)  # equal values stay in order of their ids
    val, ids = val[:, :k], ids[:, :k]
    real = val > -float("inf")
    ids, order = torch.sort(torch.where(real, ids, V + torch.arange(k, device="cuda")), 1)
    real, val = real.gather(1, order), val.gather(1, order)
    return {"ids": torch.where(real, ids, 0).to(torch.int32), "logits": torch.where(real, val, 0.0), "len": real.sum(1).to(torch.int32),
            "lse": _logsumexp(x / s["tau"])[:, 0], "status": torch.zeros(n, dtype=torch.int32, device="cuda")}


def _plain_distill(s):
    t, tau = s["teacher"], s["tau"]
    n, V = s["x"].shape
    k = t["ids"].shape[1]
    u = s["x"].float() / tau
    m = u.amax(1, keepdim=True)
    e = (u - m).exp()
    real = torch.arange(k, device="cuda") < t["len"][:, None]
    ids = t["ids"].long()
    zt = torch.where(real, t["logits"].double() / tau, -float("inf"))  # few values: 64 bits keep what 1 - sum p loses
    lse_t = _logsumexp(torch.where(t["len"][:, None] > 0, zt, 0.0)) if t["lse"] is None else t["lse"].double()[:, None]
    logp = torch.where(real, zt - lse_t, 0.0)
    p = torch.where(real, logp.exp(), 0.0)
    on = torch.zeros(n, V, device="cuda").scatter_add_(1, ids, real.float()) > 0
    off_sum = torch.where(on, 0.0, e).sum(1, keepdim=True).double()
    total = off_sum + torch.where(on, e, 0.0).sum(1, keepdim=True).double()
    logq = torch.where(real, u.gather(1, ids).double() - m, 0.0) - total.log()
    loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(1, keepdim=True)
    rest = torch.ones_like(loss)
    if t["lse"] is not None:
        P, Q = (1 - p.sum(1, keepdim=True)).clamp(min=0), off_sum / total
        both = (P > 0) & (Q > 0)
        loss = loss + torch.where(both, P * (P / Q).log(), 0.0)
        rest = torch.where(both, 1 - P / Q, 1.0)
    live = t["len"][:, None] > 0
    w = s["scale"][:, None] / tau
    q = e / total.float()
    grad = torch.where(on, q, q * rest.float())
    grad = grad.scatter_add_(1, ids, -p.float())
    grad = torch.where(live, grad * w, 0.0).to(s["x"].dtype)
    loss = torch.where(live, loss, 0.0).float()[:, 0]
    return {"loss": loss, "grad": grad}


def run(s):
    if own:
        from vocab_wide_draft_amd import binding as B
        if s["op"] == "shape":
            return B.shape_logits(s["x"], s["P"], history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"], draft=s["draft"],
                                  repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], temperature=s["temperature"],
                                  bias=s["bias"], mask=s["mask"], mask_row=s["mask_row"], out_dtype=s["out_dtype"])
        if s["op"] == "top":
            r = B.top_logits(s["x"], s["k"], temperature=s["tau"])
            return {name: r[name] for name in ("ids", "logits", "len", "lse", "status")}
        if s["how"] == "autograd":
            x = s["x"].detach().requires_grad_()
            loss = B.distill_loss(x, s["teacher"], temperature=s["tau"])
            return {"loss": loss, "grad": torch.autograd.grad(loss, x, s["scale"])[0]}
        r = B.distill_step(s["x"], s["teacher"], s["scale"], temperature=s["tau"])
        return {"loss": r["loss"], "grad": r["grad"]}
    return {"shape": _plain_shape, "top": _plain_top, "distill": _plain_distill}[s["op"]](s)


# ----------------------------------------------------- definitions, 64 bits
def _exact_shape(s):
    n, V = s["x"].shape
    P = s["P"]
    got = torch.empty(n, V, dtype=torch.float64, device="cuda")
    for r in range(n // P):
        L, L0 = int(s["history_len"][r]), int(s["prompt_len"][r])
        h = s["history"][r, :L].long()
        prompt = torch.bincount(h[:L0], minlength=V)
        made = torch.bincount(h[L0:], minlength=V)
        rep, freq, pres, temp = (float(s[k][r]) for k in ("repetition", "frequency", "presence", "temperature"))
        for i in range(P):
            z = s["x"][r * P + i].double()
            c = made if i == 0 else made + torch.bincount(s["draft"][r, :i].long(), minlength=V)
            seen = (c + prompt) > 0
            z = torch.where(seen & (z > 0), z / rep, torch.where(seen, z * rep, z))
            z = z - (freq * c + pres * (c > 0))
            if s["bias"] is not None:
                off, ids, val = s["bias"]
                a, b = int(off[r]), int(off[r + 1])
                z[ids[a:b].long()] += val[a:b].double()
            z = z / temp
            if s["mask"] is not None and int(s["mask_row"][r * P + i]) >= 0:
                w = s["mask"][int(s["mask_row"][r * P + i])]
                v = torch.arange(V, device="cuda")
                z[((w[v >> 5] >> (v & 31).to(torch.int32)) & 1) == 0] = -float("inf")
            got[r * P + i] = z
    return {"logits": got, "status": None}


def _exact_top(s):
    x, k = s["x"], s["k"]
    V = x.shape[1]
    logits, lse = [], []
    for part in x.split(max(1, (1 << 27) // V)):
        b = (part.float() + 0.0).view(torch.int32).long()
        key = torch.where(b < 0, -(b & 0x7FFFFFFF), b) * (1 << 21) + (V - 1 - torch.arange(V, device="cuda"))  # larger value, then lower id
        at = torch.sort(key.topk(k, 1).indices, 1).values
        val = part.gather(1, at).double()
        order = torch.sort((val == -float("inf")).int(), dim=1, stable=True).indices  # what is not listed goes last
        val = val.gather(1, order)
        logits.append(torch.where(val == -float("inf"), 0.0, val))
        lse.append(torch.logsumexp(part.double() / s["tau"], 1))
    return {"ids": None, "logits": torch.cat(logits), "len": None, "lse": torch.cat(lse), "status": None}


def _exact_distill(s):
    t, tau = s["teacher"], s["tau"]
    n, V = s["x"].shape
    loss = torch.zeros(n, dtype=torch.float64, device="cuda")
    grad = torch.zeros(n, V, dtype=torch.float64, device="cuda")
    for r in range(n):
        m = int(t["len"][r])
        if m == 0:
            continue
        j = t["ids"][r, :m].long()
        logq = torch.log_softmax(s["x"][r].double() / tau, 0)
        z = t["logits"][r, :m].double() / tau
        logp = z - (torch.logsumexp(z, 0) if t["lse"] is None else t["lse"][r].double())
        p = logp.exp()
        g = logq.exp()
        l = (p * (logp - logq[j])).sum()
        if t["lse"] is not None:
            off = torch.ones(V, dtype=torch.bool, device="cuda")
            off[j] = False
            P = (1 - p.sum()).clamp(min=0)
            logQ = torch.logsumexp(torch.where(off, logq, -float("inf")), 0)
            use = (P > 0) & (logQ > -float("inf"))
            l = l + torch.where(use, P * (P.log() - logQ), 0.0)
            g = torch.where(off & use, g - P * (logq - logQ).exp(), g)
        g[j] -= p
        loss[r], grad[r] = l, g * (s["scale"][r].double() / tau)
    return {"loss": loss, "grad": grad}


def exact(case, seed):
    s = prepare(case, seed)
    return {"shape": _exact_shape, "top": _exact_top, "distill": _exact_distill}[case["op"]](s)
