"""The operators of a language model's head that are measured: what each is, on which inputs, and its plain form.

All of them work on hidden states e [N, D] (bf16) and a classifier of V rows, c [V, D], with logits
z = e c^T + bias and y = z / temperature:

* ``score``  log-probabilities of K given tokens a row, y_t - lse, and the entropy of the row, without gradients:
             a reference policy, a teacher, or the ranking of candidates.
* ``train``  the same with the gradients of both outputs for e, c and the bias: a policy-gradient step with an
             entropy bonus (K = 1), or distillation on a teacher's top alternatives (K > 1).
* ``top``    the k most probable tokens of each row with their log-probabilities, highest first, the lowest id first
             among equal ones: what a server returns beside each token, and what a teacher hands on. The classifier
             is bf16, or 8-bit integers with a scale for each row (then the hidden states are rounded to 8-bit
             integers with a scale for each row within the call).
* ``int8``   the product e c^T + bias itself with such a classifier, in bf16.

A token equal to IGNORE asks for nothing: its log-probability and gradient are 0, and a row of which every token is
IGNORE has entropy 0 and gradient 0.
"""
import math

import torch

own = False

IGNORE = -100


def listed():
    return [
        # a small head: every launch counts
        dict(name="score small head", op="score", n=256, d=128, v=4096, k=1, bias=False, temperature=1.0),
        # the reference policy's log-probabilities of a batch of completions on a 1B model's head
        dict(name="score llama3.2-1b", op="score", n=2048, d=2048, v=128256, k=1, bias=False, temperature=1.0),
        # 20 candidates a position, an odd vocabulary with a bias, a sampling temperature
        dict(name="score 20 candidates", op="score", n=777, d=1288, v=50257, k=20, bias=True, temperature=0.7),
        # a policy-gradient step with an entropy bonus on a small head
        dict(name="train small head", op="train", n=256, d=128, v=4096, k=1, bias=False, temperature=1.0),
        # the same with a wide vocabulary, on a micro-batch of an odd number of tokens
        dict(name="train gemma2-2b", op="train", n=1001, d=2304, v=256000, k=1, bias=False, temperature=1.0),
        # the largest: a micro-batch of 4096 tokens on an 8B model's head
        dict(name="train llama3.1-8b", op="train", n=4096, d=4096, v=128256, k=1, bias=False, temperature=1.0),
        # distillation on a teacher's 8 best alternatives, a biased head of odd sizes
        dict(name="train 8 alternatives", op="train", n=513, d=1032, v=32003, k=8, bias=True, temperature=2.0),
        # one decoded token's 20 alternatives
        dict(name="top decode 1", op="top", n=1, d=4096, v=128256, k=20, bias=False, temperature=1.0, int8=False),
        # a batch of 33 decoded tokens on an 8-bit head
        dict(name="top decode 33 int8", op="top", n=33, d=4096, v=128256, k=5, bias=False, temperature=0.7, int8=True),
        # the alternatives of every token of a batch of prompts: a teacher's pass
        dict(name="top prompt", op="top", n=2048, d=2048, v=128256, k=20, bias=False, temperature=1.0, int8=False),
        # the logits of 16 decoded tokens, for a sampler
        dict(name="int8 decode", op="int8", n=16, d=4096, v=128256, bias=False),
        # the logits of a prompt
        dict(name="int8 prompt", op="int8", n=2048, d=2048, v=128256, bias=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """Rows from one token to 4096, widths of 64 to 4096, vocabularies of 1000 to 256000, of any parity."""
    op = rng.choice(["score", "train", "top", "top", "int8"])
    n, v = _spread(rng, 1, 4096), _spread(rng, 1000, 256000)
    d = 16 * _spread(rng, 4, 256)
    while n * v > 4096 * 128256 // 2:
        n = (n + 1) // 2
    case = dict(op=op, n=n, d=d, v=v, bias=rng.random() < 0.5)
    if op != "int8":
        case["temperature"] = rng.choice([1.0, 0.7, round(rng.uniform(0.5, 2.0), 3)])
        case["k"] = rng.choice([1, 1, rng.randint(2, 24)]) if op != "top" else rng.randint(1, 24)
    if op == "top":
        case["int8"] = rng.random() < 0.5
    return case


def prepare(case, seed):
    """Hidden states that point at a token's row of the classifier, as a trained model's do (the probability of that
    token is then about a third); tokens and gradients as a batch of padded sequences has them."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    n, d, v, op = case["n"], case["d"], case["v"], case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    c = normal(v, d).mul_(d ** -0.5)
    best = torch.randint(0, v, (n,), generator=g, device=dev)
    t = case.get("temperature", 1.0)  # the other logits are about normal: their exp(z / t) add up to v exp(1 / 2 t^2)
    e = (normal(n, d) + t * (math.log(v / 2) + 0.5 / t ** 2) * c[best]).to(torch.bfloat16)
    s = dict(case=case, e=e)
    if op == "int8" or case.get("int8"):
        s["scale"] = c.abs().amax(1).div_(127.0)
        s["c"] = c.div_(s["scale"][:, None]).round_().to(torch.int8)
    else:
        s["c"] = c.to(torch.bfloat16)
    del c
    s["bias"] = normal(v).mul_(0.5).to(torch.bfloat16) if case["bias"] else None
    if op in ("score", "train"):
        k = case["k"]
        tokens = torch.randint(0, v, (n, k), generator=g, device=dev)
        tokens[:, 0] = best
        if n > 1:  # padding behind the sequences, and rows with fewer candidates
            tokens[torch.rand(n, generator=g, device=dev) < 0.05] = IGNORE
            if k > 1:
                tokens[:, 1:][torch.rand(n, k - 1, generator=g, device=dev) < 0.1] = IGNORE
        s["tokens"] = tokens if k > 1 else tokens[:, 0]
    if op == "train":
        s["g_logprobs"] = normal(*s["tokens"].shape) / n
        s["g_entropy"] = normal(n).mul_(0.1 / n)
        s["leaves"] = [t.requires_grad_(True) for t in (s["e"], s["c"], s["bias"]) if t is not None]
    return s


def _eight_bits(x):
    """Rows of 8-bit integers and their scales: scale = max |x| / 127 rounded to 32 bits, value = x / scale to the
    nearest integer, halves to the even one (quotients in 64 bits: those near a border are not lost)."""
    scale = (x.double().abs().amax(1) / 127.0).float()
    q = (x.double() / scale.double()[:, None]).round()
    return torch.where(scale[:, None] > 0, q, torch.zeros_like(q)), scale


def _given(y, s):
    """(log-probabilities of the given tokens, entropy, the probabilities and log-probabilities of all)"""
    tokens = s["tokens"].reshape(y.shape[0], -1)
    wanted = tokens != IGNORE
    m = y.amax(1, keepdim=True)
    logp = y - m
    p = logp.exp()
    total = p.sum(1, keepdim=True)
    logp -= total.log()
    p /= total
    at = torch.where(wanted, tokens, torch.zeros_like(tokens))
    logprobs = torch.where(wanted, logp.gather(1, at), torch.zeros((), device=y.device))
    entropy = -(p * logp).sum(1) * wanted.any(1)
    return logprobs, entropy, p, logp, wanted, at


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import linear_cross_entropy_06_b200 as lce

    case, e, c, bias = s["case"], s["e"], s["c"], s["bias"]
    op = case["op"]
    if "scale" in s:
        c = lce.Int8Rows(c, s["scale"])
    if op == "int8":
        return lce.int8_linear(e, c, bias=bias)
    if op == "top":
        top = lce.linear_top_logprobs(e, c, case["k"], bias=bias, temperature=case["temperature"])
        return top.logprobs, top.ids
    out = lce.linear_logprobs(e, c, s["tokens"], bias=bias, temperature=case["temperature"], ignore_index=IGNORE)
    if op == "score":
        return out.logprobs, out.entropy
    grads = torch.autograd.grad((out.logprobs, out.entropy), s["leaves"], (s["g_logprobs"], s["g_entropy"]))
    return out.logprobs.detach(), out.entropy.detach(), *grads


@torch.no_grad()
def _plain(s):
    case, e, c, bias = s["case"], s["e"], s["c"], s["bias"]
    op = case["op"]
    if op == "int8":
        q, scale = _eight_bits(e)
        z = (q.float() @ c.float().T) * scale[:, None] * s["scale"]
        return (z if bias is None else z + bias.float()).to(torch.bfloat16)
    if op == "top":  # in 64 bits: the order of close alternatives is decided there
        if "scale" in s:
            q, scale = _eight_bits(e)
            z = (q @ c.double().T) * scale.double()[:, None] * s["scale"].double()
        else:
            z = e.double() @ c.double().T
        if bias is not None:
            z += bias.double()
        z /= case["temperature"]
        value, ids = torch.sort(z, dim=1, descending=True, stable=True)
        m = value[:, :1]
        lse = m + (value - m).exp().sum(1, keepdim=True).log()
        k = case["k"]
        return (value[:, :k] - lse).float(), ids[:, :k].clone()
    e32, c32 = e.float(), c.float()
    y = e32 @ c32.T
    if bias is not None:
        y += bias.float()
    y /= case["temperature"]
    logprobs, entropy, p, logp, wanted, at = _given(y, s)
    shape = s["tokens"].shape
    if op == "score":
        return logprobs.reshape(shape), entropy
    del y
    # d/dy of sum_k g_k logp_{t_k} + h H: sum_k g_k ([v = t_k] - p_v) - h p_v (logp_v + H)
    g = torch.where(wanted, s["g_logprobs"].reshape(at.shape), torch.zeros((), device=e.device))
    h = torch.where(wanted.any(1), s["g_entropy"], torch.zeros((), device=e.device))[:, None]
    p *= -(g.sum(1, keepdim=True) + h * (logp + entropy[:, None]))
    del logp
    p.scatter_add_(1, at, g)
    p /= case["temperature"]
    grads = [(p @ c32).to(e.dtype), (p.T @ e32).to(c.dtype)]
    if bias is not None:
        grads.append(p.sum(0).to(bias.dtype))
    return logprobs.reshape(shape), entropy, *grads


def work(case):
    """Each input once, each output once; products of 2 N V D operations: one forward, two more for the gradients."""
    n, d, v, op = case["n"], case["d"], case["v"], case["op"]
    eight = op == "int8" or case.get("int8", False)
    size = n * d * 2 + (v * (d + 4) if eight else v * d * 2) + (2 * v if case["bias"] else 0)
    flops = 2.0 * n * v * d
    if op == "int8":
        size += 2 * n * v
    elif op == "top":
        size += n * case["k"] * 12
    else:
        size += n * case["k"] * 12 + 4 * n
        if op == "train":
            size += n * case["k"] * 4 + 4 * n + n * d * 2 + v * d * 2 + (2 * v if case["bias"] else 0)
            flops *= 3
    return {"bytes": float(size), "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits, through torch's log_softmax and its gradients."""
    s = prepare(case, seed)
    op = case["op"]
    e, c = (s[name].detach().double() for name in ("e", "c"))
    bias = None if s["bias"] is None else s["bias"].detach().double()
    if "scale" in s:
        step = (s["e"].double().abs().amax(1) / 127.0).float().double()[:, None]
        e = torch.where(step > 0, torch.round(e / step), 0.0) * step
        c *= s["scale"].double()[:, None]
    leaves = [t.requires_grad_(op == "train") for t in (e, c, bias) if t is not None]
    with torch.set_grad_enabled(op == "train"):
        z = torch.nn.functional.linear(e, c, bias)
        if op == "int8":
            return z
        logp = torch.log_softmax(z / case["temperature"], 1)
        del z
        if op == "top":
            order = torch.argsort(logp, dim=1, descending=True, stable=True)[:, : case["k"]]
            return logp.gather(1, order), order
        tokens = s["tokens"].reshape(case["n"], -1)
        wanted = tokens != IGNORE
        logprobs = logp.gather(1, tokens.clamp(min=0)).where(wanted, 0.0).reshape(s["tokens"].shape)
        entropy = torch.special.entr(logp.exp()).sum(1).where(wanted.any(1), 0.0)
        if op == "score":
            return logprobs, entropy
        total = (logprobs * s["g_logprobs"].double()).sum() + (entropy * s["g_entropy"].double()).sum()
        del logp
    grads = torch.autograd.grad(total, leaves)
    return logprobs.detach(), entropy.detach(), *grads
