"""Measured cases of distillation from a teacher's top logits.

Operators, each a function of the package:

* ``lx_top_logits``: the K largest logits of every row with their ids (what a
  teacher leaves behind for a token), the row's log-sum-exp and that of the
  logits outside the K.
* ``lx_ce_kd_forward``, ``lx_ce_kd_backward``, ``lx_ce_kd_forward_backward``:
  cross entropy and the Kullback-Leibler divergence from the teacher's top
  logits (what lies outside them counts as one more token) over student logits,
  and their gradient.
* ``lx_ce_kd_linear_forward_backward``: the same loss from hidden states and
  the lm_head's weight in pieces of the vocabulary, with both gradients.

``run`` computes them from elementary torch operations while ``own`` is false
and through the package where it is true.  ``exact`` follows the definitions
in float64, some rows at a time.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORE = -100
MASKED = -1e30  # a logit below it has no mass


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the likeliest tokens beside one answered token
        top("top_one_row", BT=1, V=151936, K=20, dtype="bf16"),
        # odd vocabulary, softened teacher, rows padded to a wider array, some rows masked altogether
        top("top_odd_masked", BT=259, V=50001, K=100, dtype="f16", T=2.0, pad=3, empty=0.05),
        # a teacher's logits of a training batch, kept as 64 a token
        top("top_teacher_batch", BT=8192, V=151936, K=64, dtype="bf16"),
        # the smallest training step: latency
        kd("kd_step_tiny", "step", BT=8, V=1024, K=8, dtype="f32", ignored=0.125),
        # evaluation of long rows of fp32 logits at a temperature, part of a padded vocabulary masked
        kd("kd_forward_long_rows", "forward", BT=64, V=262144, K=32, dtype="f32", T=2.0, masked=136),
        # an unreduced loss: a factor for each row, 5% of the rows ignored
        kd("kd_backward_rows", "backward", BT=1024, V=151936, K=64, dtype="bf16", ignored=0.05, factors=True),
        # odd vocabulary in binary16, the teacher known by its top alone (renormalised), a temperature
        kd("kd_step_odd_temperature", "step", BT=2048, V=50257, K=50, dtype="f16", T=2.0, rest=False),
        # the training batch
        kd("kd_step_batch", "step", BT=8192, V=151936, K=64, dtype="bf16"),
        # scoring a few tokens from hidden states: the loss alone, no teacher
        linear("linear_score", BT=64, H=4096, V=151936, K=0, grads=False),
        # a small step with sizes off every tile, at a temperature
        linear("linear_small_odd", BT=75, H=1160, V=5001, K=16, T=2.0, ignored=0.1),
        # a middling batch
        linear("linear_middle", BT=2048, H=2048, V=50257, K=50, rest=False),
        # the training batch from hidden states
        linear("linear_batch", BT=8192, H=4096, V=151936, K=64),
    ]


def top(name, BT, V, K, dtype, T=1.0, pad=0, empty=0.0):
    return {"name": name, "op": "top", "BT": BT, "V": V, "K": K, "dtype": dtype, "T": T, "pad": pad, "empty": empty}


def kd(name, way, BT, V, K, dtype, T=1.0, pad=0, rest=True, ignored=0.0, masked=0, factors=False):
    # masked: so many of the last columns are masked; factors: upstream gradients for each row
    return {"name": name, "op": "kd_" + way, "BT": BT, "V": V, "K": K, "dtype": dtype, "T": T, "pad": pad, "rest": rest,
            "ignored": ignored, "masked": masked, "factors": factors}


def linear(name, BT, H, V, K, T=1.0, rest=True, ignored=0.0, grads=True):
    return {"name": name, "op": "linear", "BT": BT, "H": H, "V": V, "K": K, "T": T, "rest": rest, "ignored": ignored,
            "grads": grads}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["top", "top", "forward", "backward", "step", "step", "linear", "linear"])
    T = rng.choice([1.0, 1.0, 2.0, 0.7, 4.0])
    if op == "linear":
        H = 8 * _log_int(rng, 8, 512)
        V = _log_int(rng, 500, 151936)
        most = max(1, min(8192, 8192 * 4096 * 151936 // (4 * H * V)))
        grads = rng.random() < 0.75
        case = linear("", BT=_log_int(rng, 1, most), H=H, V=V, K=rng.choice([0, 1, 8, 20, 50, 64, 128]), T=T,
                      rest=rng.random() < 0.7, ignored=rng.choice([0.0, 0.0, 0.1]), grads=grads)
    else:
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        V = _log_int(rng, 300, 262144)
        most = max(1, min(8192, 8192 * 151936 // (2 * V)))
        BT = _log_int(rng, 1, most)
        K = _log_int(rng, 1, 256)
        pad = rng.choice([0, 0, 1, 8, 64])
        if op == "top":
            case = top("", BT=BT, V=V, K=K, dtype=dtype, T=T, pad=pad, empty=rng.choice([0.0, 0.0, 0.05]))
        else:
            case = kd("", op, BT=BT, V=V, K=min(K, 128), dtype=dtype, T=T, pad=pad, rest=rng.random() < 0.7,
                      ignored=rng.choice([0.0, 0.05]), masked=rng.choice([0, 0, 37]), factors=rng.random() < 0.3)
    del case["name"]
    return case


def _rng(case, what):
    return random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))


def _chosen(case, share, what):
    """The rows that are ignored or empty: fixed by the case, never all of them."""
    rng = _rng(case, what)
    rows = [r for r in range(case["BT"]) if rng.random() < case[share]]
    return rows[:max(0, case["BT"] - 1)]


def work(case):
    BT, V, K = case["BT"], case["V"], case["K"]
    if case["op"] == "top":
        es = 4 if case["dtype"] == "f32" else 2
        return {"bytes": BT * V * es + BT * K * 8 + BT * 8, "flops": 4 * BT * V}
    valid = BT - len(_chosen(case, "ignored", "ignored"))
    if case["op"] == "linear":
        H = case["H"]
        products = 3 if case["grads"] else 1
        return {"bytes": 2 * (BT + V) * H * (2 if case["grads"] else 1) + BT * (8 * K + 40),
                "flops": 2 * valid * V * H * products}
    es = 4 if case["dtype"] == "f32" else 2
    reads = valid * V * es
    writes = 0 if case["op"] == "kd_forward" else BT * V * es
    return {"bytes": reads + writes + BT * (8 * K + 48), "flops": 4 * valid * V}


# ---------------------------------------------------------------- inputs

def _logits(g, BT, V, dev):
    """Logits of a language model: a broad floor and a few dozen likely tokens."""
    z = torch.empty(BT, V, dtype=torch.float32, device=dev).normal_(0.0, 1.5, generator=g)
    few = min(32, V)
    where = torch.randint(V, (BT, few), device=dev, generator=g)
    return z.scatter_(1, where, torch.empty(BT, few, device=dev).normal_(8.0, 2.0, generator=g))


def _log_sum_exp(x):
    m = x.amax(1, keepdim=True)
    m = torch.where(m > MASKED, m, 0.0)
    return (torch.log(torch.exp(x - m).sum(1, keepdim=True)) + m).squeeze(1)


def _teacher(z, K, T, noise, g):
    """(ids, top logits, log-sum-exp of the others) of a teacher whose logits are z and an error of its own."""
    u = torch.empty_like(z).normal_(0.0, noise, generator=g).add_(z)
    values, ids = torch.topk(u, K, 1)
    u.scatter_(1, ids, -math.inf)
    return ids.to(torch.int32), values, _log_sum_exp(u.div_(T))


def _targets(case, ids, V, g, dev):
    BT = case["BT"]
    t = torch.randint(V, (BT,), device=dev, generator=g)
    if ids is not None:  # the text agrees with the teacher's first token most of the time
        t = torch.where(torch.rand(BT, device=dev, generator=g) < 0.6, ids[:, 0].long(), t)
    rows = _chosen(case, "ignored", "ignored")
    if rows:
        t[torch.tensor(rows, device=dev)] = IGNORE
    return t


def _loss_outputs(BT, dev, teacher=True):
    f = lambda *s: torch.empty(*s, dtype=torch.float32, device=dev)  # noqa: E731
    out = {"ce": f(BT), "lse": f(BT)}
    if teacher:
        out.update(kd=f(BT), state=f(BT, 4))
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"top": _prepare_top, "linear": _prepare_linear}.get(case["op"], _prepare_kd)(case, g)


def _prepare_top(case, g):
    dev, BT, V, K = "cuda", case["BT"], case["V"], case["K"]
    wide = torch.zeros(BT, V + case["pad"], dtype=DTYPES[case["dtype"]], device=dev)
    for r in range(0, BT, 1024):
        n = min(1024, BT - r)
        wide[r:r + n, :V] = _logits(g, n, V, dev)
    rows = _chosen(case, "empty", "empty")
    if rows:
        wide[torch.tensor(rows, device=dev)] = -math.inf
    out = {"top": torch.empty(BT, K, dtype=torch.float32, device=dev),
           "ids": torch.empty(BT, K, dtype=torch.int32, device=dev),
           "lse": torch.empty(BT, dtype=torch.float32, device=dev),
           "lse_rest": torch.empty(BT, dtype=torch.float32, device=dev)}
    return {"op": "top", "logits": wide[:, :V], "T": case["T"], "out": out}


def _prepare_kd(case, g):
    dev, BT, V, K, T = "cuda", case["BT"], case["V"], case["K"], case["T"]
    use = V - case["masked"]
    K = min(K, use)
    wide = torch.zeros(BT, V + case["pad"], dtype=DTYPES[case["dtype"]], device=dev)
    ids = torch.empty(BT, K, dtype=torch.int32, device=dev)
    tops = torch.empty(BT, K, dtype=torch.float32, device=dev)
    lse_rest = torch.empty(BT, dtype=torch.float32, device=dev)
    for r in range(0, BT, 1024):
        n = min(1024, BT - r)
        z = _logits(g, n, use, dev)
        wide[r:r + n, :use] = z
        ids[r:r + n], tops[r:r + n], lse_rest[r:r + n] = _teacher(z, K, T, 0.7, g)
    if case["masked"]:
        wide[:, use:V] = -math.inf
    s = {"op": case["op"], "student": wide[:, :V], "T": T, "ids": ids, "top": tops,
         "lse_rest": lse_rest if case["rest"] else None, "target": _targets(case, ids, use, g, dev),
         "out": _loss_outputs(BT, dev), "g_ce": 0.5, "g_kd": 0.5 * T * T, "ce_rows": None, "kd_rows": None,
         "scale": None}
    if case["factors"]:
        s["ce_rows"] = torch.empty(BT, device=dev).uniform_(0.5, 1.5, generator=g)
        s["kd_rows"] = torch.empty(BT, device=dev).uniform_(0.5, 1.5, generator=g)
    elif case["dtype"] != "f16":  # a mean over the valid rows (binary16 trains on a scaled loss)
        s["scale"] = torch.full((1,), 1.0 / (BT - len(_chosen(case, "ignored", "ignored"))), device=dev)
    if case["op"] != "kd_forward":
        s["grad"] = torch.empty(BT, V, dtype=DTYPES[case["dtype"]], device=dev)
    if case["op"] == "kd_backward":  # what the forward pass left behind
        o = s["out"]
        o["ce"], o["kd"], o["lse"], o["state"] = _plain_forward(s)
    return s


def _prepare_linear(case, g):
    dev, BT, V, H, K, T = "cuda", case["BT"], case["V"], case["H"], case["K"], case["T"]
    x = torch.empty(BT, H, device=dev).normal_(generator=g).to(torch.bfloat16)
    # rows of the weight that many hidden states agree with: a few likely tokens
    w = torch.empty(V, H, device=dev).normal_(0.0, 1.5 * H ** -0.5, generator=g)
    likely = (torch.rand(V, 1, device=dev, generator=g) < min(0.5, 16 * BT / V)) * (8.0 / H)
    w += likely * x[torch.randint(BT, (V,), device=dev, generator=g)].float()
    w = w.to(torch.bfloat16)
    s = {"op": "linear", "x": x, "w": w, "T": T, "ids": None, "top": None, "lse_rest": None, "g_ce": 1.0, "g_kd": 0.0,
         "ce_rows": None, "kd_rows": None,
         "scale": torch.full((1,), 1.0 / (BT - len(_chosen(case, "ignored", "ignored"))), device=dev)}
    if K:
        ids = torch.empty(BT, K, dtype=torch.int32, device=dev)
        tops = torch.empty(BT, K, dtype=torch.float32, device=dev)
        lse_rest = torch.empty(BT, dtype=torch.float32, device=dev)
        for r in range(0, BT, 1024):
            n = min(1024, BT - r)
            ids[r:r + n], tops[r:r + n], lse_rest[r:r + n] = _teacher((x[r:r + n] @ w.t()).float(), K, T, 1.5, g)
        s.update(ids=ids, top=tops, lse_rest=lse_rest if case["rest"] else None, g_ce=0.5, g_kd=0.5 * T * T)
    s["target"] = _targets(case, s["ids"], V, g, dev)
    s["out"] = _loss_outputs(BT, dev, teacher=K > 0)
    s["grad_x"] = torch.empty(BT, H, dtype=torch.bfloat16, device=dev) if case["grads"] else None
    s["grad_w"] = torch.empty(V, H, dtype=torch.bfloat16, device=dev) if case["grads"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import cross_entropy_tv_amd as lx
    o = s["out"]
    if s["op"] == "top":
        lx.lx_top_logits(s["logits"], s["T"], o["top"], o["ids"], o["lse"], o["lse_rest"])
        return o
    if s["op"] == "linear":
        lx.lx_ce_kd_linear_forward_backward(s["x"], s["w"], s["target"], IGNORE, s["ids"], s["top"], s["lse_rest"],
                                            s["T"], o["ce"], o.get("kd"), o["lse"], o.get("state"), s["grad_x"],
                                            s["grad_w"], s["g_ce"], s["g_kd"], g_scale=s["scale"])
        return dict(o, grad_x=s["grad_x"], grad_w=s["grad_w"])
    teacher = (s["ids"], s["top"], s["lse_rest"], s["T"])
    if s["op"] == "kd_forward":
        lx.lx_ce_kd_forward(s["student"], s["target"], IGNORE, *teacher, o["ce"], o["kd"], o["lse"], o["state"])
        return o
    if s["op"] == "kd_backward":
        lx.lx_ce_kd_backward(s["grad"], s["student"], s["target"], IGNORE, s["ids"], s["top"], s["T"], o["lse"],
                             o["state"], s["g_ce"], s["g_kd"], s["ce_rows"], s["kd_rows"], s["scale"])
        return s["grad"]
    lx.lx_ce_kd_forward_backward(s["student"], s["target"], IGNORE, *teacher, o["ce"], o["kd"], o["lse"], o["state"],
                                 s["grad"], s["g_ce"], s["g_kd"], s["ce_rows"], s["kd_rows"], s["scale"])
    return dict(o, grad=s["grad"])


def _run_plain(s):
    if s["op"] == "top":
        return _plain_top(s)
    if s["op"] == "linear":
        return _plain_linear(s)
    if s["op"] == "kd_backward":
        return _plain_backward(s, s["student"].float(), s["out"]["lse"], s["out"]["state"]).to(s["student"].dtype)
    ce, kd_, lse, state = _plain_forward(s)
    out = {"ce": ce, "kd": kd_, "lse": lse, "state": state}
    if s["op"] == "kd_step":
        out["grad"] = _plain_backward(s, s["student"].float(), lse, state).to(s["student"].dtype)
    return out


def _plain_top(s):
    u, K, T = s["logits"].float(), s["out"]["top"].shape[1], s["T"]
    BT, V = u.shape
    k = min(K, V)
    # whole numbers in the order of (logit, lowest id first): no two are equal
    bits = (u + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
    order = order * (1 << 32) + torch.arange(V - 1, -1, -1, device=u.device)
    ids = V - 1 - (torch.topk(order, k, 1).values & 0xffffffff)
    del order, bits
    values = torch.gather(u, 1, ids)
    given = values > MASKED
    tops = torch.full((BT, K), -math.inf, device=u.device)
    places = torch.full((BT, K), -1, dtype=torch.int32, device=u.device)
    tops[:, :k] = torch.where(given, values, -math.inf)
    places[:, :k] = torch.where(given, ids, -1).to(torch.int32)
    x = torch.where(u > MASKED, u / T, -math.inf)
    lse = _log_sum_exp(x)
    return {"top": tops, "ids": places, "lse": lse, "lse_rest": _log_sum_exp(x.scatter_(1, ids, -math.inf))}


def _plain_teacher(s):
    """(q of each entry, log q, q of the rest, log q of the rest, log of the normaliser), in float64: K values a row."""
    a = s["top"].double() / s["T"]
    rest = s["lse_rest"]
    rest = torch.full_like(a[:, 0], -math.inf) if rest is None else rest.double()
    norm = _log_sum_exp(torch.cat([a, rest[:, None]], 1))
    log_q, log_qr = a - norm[:, None], rest - norm
    return torch.exp(log_q), log_q, torch.exp(log_qr), log_qr, norm


def _plain_forward(s, z=None):
    z = s["student"].float() if z is None else z
    T, target = s["T"], s["target"]
    rows = torch.arange(z.shape[0], device=z.device)
    valid = target != IGNORE
    t = torch.where(valid, target, 0)
    x = torch.where(z > MASKED, z, -math.inf)
    lse = _log_sum_exp(x)
    ce = torch.where(valid, lse - x[rows, t], 0.0)
    if s["ids"] is None:
        return ce, None, torch.where(valid, lse, 0.0), None
    x = x / T
    ids = s["ids"].long()
    here = torch.gather(x, 1, ids).double()
    lse_t = (_log_sum_exp(x) if T != 1.0 else lse).double()
    lse_rest = _log_sum_exp(x.scatter_(1, ids, -math.inf)).double()
    del x
    q, log_q, q_rest, log_q_rest, norm = _plain_teacher(s)
    # the whole row's sum from its two parts, in float64
    both = _log_sum_exp(torch.cat([here, lse_rest[:, None]], 1))
    kd_ = (q * (log_q - here + both[:, None])).sum(1)
    kd_ = kd_ + torch.where(q_rest > 0, q_rest * (log_q_rest - lse_rest + both), 0.0)
    off = torch.exp(lse_rest - both) - q_rest
    state = torch.stack([lse_t, torch.where(lse_rest > MASKED, lse_rest, 0.0), off, norm], 1).float()
    zero = torch.zeros((), device=z.device)
    return (ce, torch.where(valid, kd_.float(), zero), torch.where(valid, lse, zero),
            torch.where(valid[:, None], state, zero))


def _plain_backward(s, z, lse, state):
    """The gradient of the logits in fp32, for whoever rounds it."""
    target = s["target"]
    valid = target != IGNORE
    k = 1.0 if s["scale"] is None else s["scale"]
    a = (k * s["g_ce"] * (1.0 if s["ce_rows"] is None else s["ce_rows"])) * valid
    z = torch.where(z > MASKED, z, -math.inf)
    p = torch.exp(z - lse[:, None])
    rows = torch.arange(z.shape[0], device=z.device)
    p[rows, torch.where(valid, target, 0)] -= 1.0
    grad = p.mul_(a[:, None])
    if s["ids"] is None:
        return grad
    T, ids = s["T"], s["ids"].long()
    b = (k * s["g_kd"] / T * (1.0 if s["kd_rows"] is None else s["kd_rows"])) * valid
    x = z.div_(T)
    here = torch.exp(torch.gather(x, 1, ids) - state[:, :1]) - torch.exp(s["top"] / T - state[:, 3:])
    x.sub_(state[:, 1:2]).exp_().mul_((b * state[:, 2])[:, None])
    x.scatter_(1, ids, b[:, None] * here)
    return grad.add_(x)


def _plain_linear(s):
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    ce, kd_, lse, state = _plain_forward(s, z)
    out = {"ce": ce, "lse": lse}
    if s["ids"] is not None:
        out.update(kd=kd_, state=state)
    grad_x = grad_w = None
    if s["grad_x"] is not None:
        grad = _plain_backward(s, z, lse, state)
        grad_x, grad_w = (grad @ w).to(torch.bfloat16), (grad.t() @ x).to(torch.bfloat16)
    return dict(out, grad_x=grad_x, grad_w=grad_w)


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "top":
        return _exact_top(s)
    BT, V = case["BT"], case["V"]
    step = max(1, min(BT, (1 << 27) // V))
    parts = []
    grad_w = None
    for r in range(0, BT, step):
        at = slice(r, min(BT, r + step))
        if s["op"] == "linear":
            x, w = s["x"][at].double(), s["w"].double()
            out, grad = _exact_rows(s, x @ w.t(), at, s["grad_x"] is not None)
            if grad is not None:
                out["grad_x"] = grad @ w
                piece = grad.t() @ x
                grad_w = piece if grad_w is None else grad_w.add_(piece)
        else:
            out, grad = _exact_rows(s, s["student"][at].double(), at, s["op"] != "kd_forward")
            if grad is not None:
                out["grad"] = grad if case["BT"] * V < 1 << 29 else grad.float()
        parts.append(out)
    joined = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if s["op"] == "linear":
        joined.setdefault("grad_x", None)
        joined["grad_w"] = grad_w
        return joined
    return joined["grad"] if s["op"] == "kd_backward" else joined


def _exact_top(s):
    logits, K, T = s["logits"], s["out"]["top"].shape[1], s["T"]
    BT, V = logits.shape
    k = min(K, V)
    step = max(1, (1 << 26) // V)
    tops, places, lses, rests = [], [], [], []
    for r in range(0, BT, step):
        u = logits[r:r + step].double()
        values, ids = torch.sort(u, dim=1, descending=True, stable=True)
        masked = ~(values > MASKED)
        values[masked] = -math.inf
        ids = ids.masked_fill(masked, -1)
        tops.append(torch.nn.functional.pad(values[:, :k], (0, K - k), value=-math.inf))
        places.append(torch.nn.functional.pad(ids[:, :k], (0, K - k), value=-1))
        lses.append(torch.logsumexp(values / T, 1))
        rests.append(torch.logsumexp(values[:, k:] / T, 1) if V > k else torch.full_like(values[:, 0], -math.inf))
    return {"top": torch.cat(tops), "ids": torch.cat(places).to(torch.int32), "lse": torch.cat(lses),
            "lse_rest": torch.cat(rests)}


def _exact_rows(s, z, at, wants_grad):
    T, target = s["T"], s["target"][at]
    n, V = z.shape
    valid = target != IGNORE
    column = torch.where(valid, target, 0)[:, None]
    log_p1 = z.clone()
    log_p1[~(z > MASKED)] = -math.inf
    z = log_p1 / T
    lse = torch.logsumexp(log_p1, 1, keepdim=True)
    log_p1 = log_p1 - lse
    out = {"ce": -log_p1.gather(1, column)[:, 0], "lse": lse[:, 0]}
    grad = None
    rows = torch.ones(n, dtype=torch.float64, device=z.device) if s["scale"] is None else s["scale"].double().expand(n)
    if wants_grad:
        grad = torch.exp(log_p1)
        grad.scatter_add_(1, column, torch.full_like(column, -1, dtype=torch.float64))
        a = s["g_ce"] * rows if s["ce_rows"] is None else s["g_ce"] * rows * s["ce_rows"][at].double()
        grad = grad * torch.where(valid, a, 0.0)[:, None]
    if s["ids"] is not None:
        ids = s["ids"][at].long()
        u = s["top"][at].double() / T
        if s["lse_rest"] is not None:
            u = torch.cat([u, s["lse_rest"][at].double()[:, None]], 1)
        norm = torch.logsumexp(u, 1, keepdim=True)
        log_q = u - norm
        outside = z.scatter(1, ids, -math.inf)
        rest = torch.logsumexp(outside, 1, keepdim=True)
        lse_t = torch.logsumexp(z, 1, keepdim=True)
        log_p = z.gather(1, ids) - lse_t
        q_rest = torch.zeros_like(rest)
        if s["lse_rest"] is not None:
            log_p = torch.cat([log_p, rest - lse_t], 1)
            q_rest = torch.exp(log_q[:, -1:])
        terms = torch.exp(log_q) * (log_q - log_p)
        out["kd"] = torch.where(torch.exp(log_q) > 0, terms, 0.0).sum(1)
        p_rest = torch.exp(rest - lse_t)
        out["state"] = torch.cat([lse_t, torch.where(torch.isinf(rest), 0.0, rest), p_rest - q_rest, norm], 1)
        if wants_grad:
            b = s["g_kd"] * rows if s["kd_rows"] is None else s["g_kd"] * rows * s["kd_rows"][at].double()
            b = torch.where(valid, b, 0.0)[:, None] / T
            p = torch.exp(z - lse_t)
            d = torch.where(torch.isinf(outside), 0.0, p - q_rest * torch.exp(outside - rest))
            d.scatter_(1, ids, p.gather(1, ids) - torch.exp(log_q[:, :ids.shape[1]]))
            grad = grad + b * d
    out = {k: torch.where(valid if v.dim() == 1 else valid[:, None], v, 0.0) for k, v in out.items()}
    return out, grad
