"""Cases for timing and checking the operators around a model's output.

What a finetuning ends in and what the merged model answers with:

  lp_fwd       log-probabilities of given tokens from logits, with the entropy
               of each row and its most likely alternatives
  lp_bwd       the gradient of the logits from those of the two
  kd_fwd       distillation from a teacher's top logits: the divergence of each row
  kd_bwd       its gradient
  int4_quant   a merged weight in 4 bits with a scale (and zero point) per group
  int4_fwd     products of few tokens with such a weight

Rows. x = z / t for logits z and a temperature t, m the row's largest z, l =
log sum exp((z - m) / t), so that log p_j = (z_j - m) / t - l. H is the
entropy. A target outside [0, V) is no token: its log-probability is 0 and has
no gradient. A forward pass keeps, per row, (m, l, H) for the backward pass.

Distillation. A row has k ids with the teacher's logits; ids outside [0, V)
are left out. q_i = exp(t_i / t - L), with L the teacher's log sum exp over its
whole vocabulary, where given, and the rest q_r = max(0, 1 - sum q) is one more
class; without L q is the softmax of the list and there is no rest. loss = sum
q_i (log q_i - log p_i) + q_r (log q_r - log p_r), p_r the student's mass off
the list. With w = sum q + q_r, d loss / d x_j = w p_j - q_j on the list and
(w - q_r / p_r) p_j off it. Kept per row: (m, l, w, w - q_r / p_r, tm, tl), tm
the list's largest logit and q_i = exp((t_i - tm) / t - tl).

4 bits. w = s (q - z), q in [0, 15], for each group of G columns of a row.
Asymmetric: lo = min(w, 0), hi = max(w, 0), s = bf16((hi - lo) / 15) and z the
nearest integer to -lo / s; symmetric: s = bf16(max|w| / 7) and z = 8. q is the
integer nearest to w / s (ties to even) plus z, cut to [0, 15]; s = 0 has q = z.
Element 2i of a row is the low half of byte i.
"""

import math

import torch

own = False


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # one decoded token of a 131072-token vocabulary, with what a server returns beside it
        dict(name="lp-fwd-1x131072-top20", op="lp_fwd", T=1, V=131072, ld=131072, f32=False, temp=1.0, top=20, pad=0),
        # a decode batch whose logits are float32, sampled at a temperature
        dict(name="lp-fwd-16x32768-top5-f32", op="lp_fwd", T=16, V=32768, ld=32768, f32=True, temp=0.7, top=5, pad=0),
        # scoring a batch of 4 x 1024 tokens; a padded vocabulary
        dict(name="lp-fwd-4096x32768", op="lp_fwd", T=4096, V=32768, ld=32768, f32=False, temp=1.0, top=0, pad=500),
        # a policy's gradient with an entropy bonus; an odd vocabulary, rows of any alignment
        dict(name="lp-bwd-1023x100003", op="lp_bwd", T=1023, V=100003, ld=100003, f32=False, temp=1.0, top=0, pad=0),
        # distillation of a batch of 4 x 1024 tokens from 64 stored logits each, with the rest's mass
        dict(name="kd-fwd-4096x32768-k64", op="kd_fwd", T=4096, V=32768, ld=32768, f32=False, temp=2.0, k=64, rest=True, pad=0),
        # a short ragged answer, float32 logits in padded rows, renormalised lists
        dict(name="kd-fwd-7x50001-k20-f32", op="kd_fwd", T=7, V=50001, ld=50048, f32=True, temp=1.0, k=20, rest=False, pad=0),
        # 2048 tokens of a large vocabulary: the largest gradient
        dict(name="kd-bwd-2048x131072-k64", op="kd_bwd", T=2048, V=131072, ld=131072, f32=False, temp=1.0, k=64, rest=True, pad=100),
        # the down projection of a merged 7B-shaped MLP
        dict(name="int4-quant-4096x11008", op="int4_quant", N=4096, K=11008, G=128, sym=False),
        # one token through an attention projection
        dict(name="int4-fwd-1x4096x4096", op="int4_fwd", M=1, N=4096, K=4096, G=128, sym=False, f32=False),
        # odd sizes, short groups, a last group that is not whole, float32 out
        dict(name="int4-fwd-5x1001x1504-f32", op="int4_fwd", M=5, N=1001, K=1504, G=64, sym=True, f32=True),
        # a decode batch through the up projection
        dict(name="int4-fwd-48x11008x4096", op="int4_fwd", M=48, N=11008, K=4096, G=32, sym=False, f32=False),
        # one token through an 8192-wide model's output layer, logits in float32
        dict(name="int4-fwd-1x32768x8192", op="int4_fwd", M=1, N=32768, K=8192, G=128, sym=False, f32=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lp_fwd", "lp_fwd", "lp_bwd", "kd_fwd", "kd_bwd", "int4_quant", "int4_fwd", "int4_fwd"])
    if op.startswith("int4"):
        G = rng.choice([32, 64, 128])
        K = 32 * _log(rng, 1, 300)
        if op == "int4_quant":
            return dict(op=op, N=_log(rng, 1, 11008), K=K, G=G, sym=rng.random() < 0.5)
        return dict(op=op, M=_log(rng, 1, 64), N=_log(rng, 1, 32768), K=K, G=G, sym=rng.random() < 0.5,
                    f32=rng.random() < 0.3)
    V = _log(rng, 200, 131072)
    f32 = rng.random() < 0.3
    T = _log(rng, 1, max(1, min(4096, 100_000_000 // V)))
    ld = V if rng.random() < 0.6 else V + rng.randint(1, 200)
    case = dict(op=op, T=T, V=V, ld=ld, f32=f32, temp=rng.choice([1.0, 1.0, 0.7, 2.0]),
                pad=rng.choice([0, 0, V // 50]))
    if op.startswith("lp"):
        return dict(case, top=rng.choice([0, 1, 5, 20, 50]) if op == "lp_fwd" and T * V <= 40_000_000 else 0)
    return dict(case, k=rng.choice([1, 10, 32, 64, 100, 128]), rest=rng.random() < 0.6)


def work(case):
    op = case["op"]
    if op == "int4_quant":  # read bf16, write codes, scales and zero points; read them, write bf16
        n = case["N"] * case["K"]
        return {"bytes": n * (2 + 0.5 + 0.5 + 2) + 2 * n / case["G"] * (2 + (not case["sym"])), "flops": 6.0 * n}
    if op == "int4_fwd":
        M, N, K = case["M"], case["N"], case["K"]
        per = 2 if case["sym"] else 3
        return {"bytes": N * K / 2 + N * K / case["G"] * per + 2 * M * K + (4 if case["f32"] else 2) * M * N,
                "flops": 2.0 * M * N * K}
    T, V, e = case["T"], case["V"], 4 if case["f32"] else 2
    if op == "lp_fwd":
        return {"bytes": T * V * e + T * (8 + 8 + 12 * case["top"]), "flops": 5.0 * T * V}
    if op == "lp_bwd":
        return {"bytes": 2 * T * V * e + T * (8 + 12 + 8), "flops": 7.0 * T * V}
    lists = T * case["k"] * 12
    if op == "kd_fwd":
        return {"bytes": T * V * e + lists + 4 * T * (2 if case["rest"] else 1), "flops": 4.0 * T * V}
    return {"bytes": 2 * T * V * e + lists + T * 28, "flops": 4.0 * T * V}


# ---------------------------------------------------------------------------
# inputs

class Draw:
    """Seeded tensors on the GPU."""

    def __init__(self, seed):
        self.dev = torch.device("cuda", torch.cuda.current_device())
        self.g = torch.Generator(device=self.dev)
        self.g.manual_seed(seed)

    def normal(self, shape, std):
        return torch.randn(shape, generator=self.g, device=self.dev) * std

    def uniform(self, shape):
        return torch.rand(shape, generator=self.g, device=self.dev)

    def integers(self, lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=self.g, device=self.dev)

    def logits(self, case):
        """Rows of N(0, 2.5) with eight tokens ahead of the rest; the last `pad` ids masked."""
        T, V, ld = case["T"], case["V"], case["ld"]
        z = self.normal((T, ld), 2.5)
        lead = self.integers(0, V, (T, 8))
        z.scatter_add_(1, lead, self.uniform((T, 8)) * 16.0)
        if case["pad"]:
            z[:, V - case["pad"]:V] = -math.inf
        return (z if case["f32"] else z.to(torch.bfloat16))[:, :V]


def prepare(case, seed):
    d = Draw(seed)
    op = case["op"]
    s = dict(case)
    if op == "int4_quant":
        s["w"] = d.normal((case["N"], case["K"]), 0.02).to(torch.bfloat16)
        return s
    if op == "int4_fwd":
        M, N, K, G = (case[n] for n in ("M", "N", "K", "G"))
        ng = -(-K // G)
        s["x"] = d.normal((M, K), 1.0).to(torch.bfloat16)
        s["codes"] = d.integers(0, 256, (N, K // 2)).to(torch.uint8)
        s["scales"] = ((0.5 + d.uniform((N, ng))) * 0.005).to(torch.bfloat16)
        s["zeros"] = None if case["sym"] else d.integers(5, 11, (N, ng)).to(torch.uint8)
        return s
    T, V = case["T"], case["V"]
    z = s["z"] = d.logits(case)
    if op.startswith("lp"):
        tgt = d.integers(0, V - case["pad"], (T,))
        s["target"] = torch.where(d.uniform((T,)) < 0.2, torch.full_like(tgt, -100), tgt) if T > 1 else tgt
        if op == "lp_bwd":
            s["g_logp"] = d.normal((T,), 1.0 / T)
            s["g_ent"] = d.normal((T,), 0.01 / T)
            s["kept"] = torch.stack(lp_rows(s)[:3], dim=1)
        return s
    # the teacher's logits lie about the student's; 64 bits only where sums need them
    t = z.float() + d.normal((T, V), 1.0)
    k = min(case["k"], V - case["pad"])
    values, ids = torch.topk(t, k, dim=1)
    # lists of different lengths: a tenth of the rows end early
    short = (torch.arange(k, device=d.dev) >= max(1, k // 2)) & (d.uniform((T, 1)) < 0.1)
    s["ids"] = torch.where(short, torch.full_like(ids, -1), ids)
    s["values"] = values
    s["lse"] = torch.logsumexp(t / case["temp"], dim=1) if case["rest"] else None
    if op == "kd_bwd":
        s["g"] = (0.5 + d.uniform((T,))) / T
        s["kept"] = torch.stack(kd_rows(s)[1:], dim=1)
    return s


# ---------------------------------------------------------------------------
# the plain form

def lp_rows(s):
    """(m, l, H, log p [T x V]) in float32."""
    z = s["z"].float()
    m = z.amax(dim=1)
    x = (z - m[:, None]) / s["temp"]
    e = torch.exp(x)
    total = e.sum(dim=1)
    l = torch.log(total)
    x -= l[:, None]
    e /= total[:, None]
    ent = -torch.where(e > 0, e * x, torch.zeros((), device=z.device)).sum(dim=1)
    return m, l, ent, x


def kd_lists(s):
    """(q [T x k] in 64 bits, q_r, tm, tl, listed ids with V for none)."""
    ids, V = s["ids"], s["V"]
    ok = (ids >= 0) & (ids < V)
    t = s["values"].double()
    tm = torch.where(ok, t, torch.full_like(t, -math.inf)).amax(dim=1, keepdim=True)
    tm = torch.where(tm == -math.inf, torch.zeros_like(tm), tm)
    rel = (t - tm) / s["temp"]
    if s["lse"] is not None:
        tl = s["lse"].double()[:, None] - tm / s["temp"]
    else:
        tl = torch.log((torch.exp(rel) * ok).sum(dim=1, keepdim=True))
    q = torch.exp(rel - tl) * ok
    qr = (1.0 - q.sum(dim=1)).clamp(min=0.0) if s["lse"] is not None else torch.zeros_like(q[:, 0])
    return q, qr, tm[:, 0], tl[:, 0], torch.where(ok, ids, torch.full_like(ids, V))


def kd_mask(at, V):
    """Which tokens are on a row's list."""
    mask = torch.zeros(at.shape[0], V + 1, dtype=torch.bool, device=at.device)
    return mask.scatter_(1, at, True)[:, :V]


def kd_rows(s):
    """(loss, m, l, w, w - q_r / p_r, tm, tl); a row's few numbers in 64 bits,
    since the loss is a difference of values near each other."""
    V, temp = s["V"], s["temp"]
    q, qr, tm, tl, at = kd_lists(s)
    z = s["z"].float()
    m = z.amax(dim=1)
    x = (z - m[:, None]) / temp
    e = torch.exp(x)
    l = torch.log(e.sum(dim=1, dtype=torch.float64))
    logp = torch.gather(x, 1, at.clamp(max=V - 1)).double() - l[:, None]
    logq = (s["values"].double() - tm[:, None]) / temp - tl[:, None]
    zero = torch.zeros((), dtype=torch.float64, device=z.device)
    loss = torch.where(q > 0, q * (logq - logp), zero).sum(dim=1)
    w = q.sum(dim=1)
    off = w
    if s["lse"] is not None:
        rest = torch.where(kd_mask(at, V), torch.zeros((), device=z.device), e).sum(dim=1, dtype=torch.float64)
        logr = torch.log(rest) - l
        there = (rest > 0) & (qr > 0)
        loss = loss + torch.where(there, qr * (torch.log(qr) - logr), zero)
        w = w + torch.where(there, qr, zero)
        off = w - torch.where(there, qr / torch.exp(logr), zero)
    return tuple(v.float() for v in (loss, m, l, w, off, tm, tl))


def nibbles(codes):
    return torch.stack([codes & 15, codes >> 4], dim=2).view(codes.shape[0], -1)


def int4_f32(q, scales, zeros, K, G):
    """s (q - z): 8 bits times 5, exact in float32."""
    z = zeros.float() if zeros is not None else torch.full_like(scales, 8.0, dtype=torch.float32)
    col = torch.arange(K, device=q.device) // G
    return scales.float()[:, col] * (q.float() - z[:, col])


def plain(s):
    op = s["op"]
    bf = torch.bfloat16
    if op == "lp_fwd":
        m, l, ent, logp = lp_rows(s)
        tgt = s["target"]
        at = torch.gather(logp, 1, tgt.clamp(min=0)[:, None])[:, 0]
        out = {"logp": torch.where(tgt >= 0, at, torch.zeros_like(at)), "entropy": ent}
        if s["top"]:  # of equal logits the lowest id first
            order = torch.sort(s["z"].float(), dim=1, descending=True, stable=True)[1][:, :s["top"]]
            out["top_ids"], out["top_logp"] = order, torch.gather(logp, 1, order)
        return out
    if op == "lp_bwd":
        m, l, ent = (c[:, None] for c in s["kept"].unbind(1))
        logp = (s["z"].float() - m) / s["temp"] - l
        p = torch.exp(logp)
        tgt = s["target"]
        g = torch.where(tgt >= 0, s["g_logp"], torch.zeros_like(s["g_logp"]))[:, None]
        dz = -g * p - s["g_ent"][:, None] * torch.where(p > 0, p * (logp + ent), torch.zeros_like(p))
        dz.scatter_add_(1, tgt.clamp(min=0)[:, None], g)
        return {"dz": (dz / s["temp"]).to(s["z"].dtype)}
    if op == "kd_fwd":
        return {"loss": kd_rows(s)[0]}
    if op == "kd_bwd":
        V = s["V"]
        m, l, w, off, tm, tl = (c[:, None] for c in s["kept"].unbind(1))
        ids = s["ids"]
        ok = (ids >= 0) & (ids < V)
        at = torch.where(ok, ids, torch.full_like(ids, V))
        q = torch.exp((s["values"] - tm) / s["temp"] - tl) * ok
        p = torch.exp((s["z"].float() - m) / s["temp"] - l)
        dz = torch.zeros(s["T"], V + 1, device=p.device)
        dz[:, :V] = p * torch.where(kd_mask(at, V), w, off)
        dz.scatter_add_(1, at, -q)
        return {"dz": (dz[:, :V] * (s["g"][:, None] / s["temp"])).to(s["z"].dtype)}
    K, G = s["K"], s["G"]
    if op == "int4_fwd":
        y = s["x"].float() @ int4_f32(nibbles(s["codes"]), s["scales"], s["zeros"], K, G).t()
        return {"y": y if s["f32"] else y.to(bf)}
    N, ng = s["N"], -(-K // G)
    # divisors as tensors: a division by a plain number is a product with its inverse
    seven, fifteen = (torch.full((), v, device=s["w"].device) for v in (7.0, 15.0))
    w = torch.zeros(N, ng * G, device=s["w"].device)  # zeros change no group's ends
    w[:, :K] = s["w"]
    w = w.view(N, ng, G)
    if s["sym"]:
        scale = (w.abs().amax(dim=2) / seven).to(bf)
        zero = torch.full_like(scale, 8.0, dtype=torch.float32)
    else:
        lo, hi = w.amin(dim=2).clamp(max=0.0), w.amax(dim=2).clamp(min=0.0)
        scale = ((hi - lo) / fifteen).to(bf)
        zero = torch.where(scale > 0, torch.round(-lo / scale.float()), torch.zeros_like(lo)).clamp(0, 15)
    sc = scale.float()[:, :, None]
    q = torch.where(sc > 0, torch.round(w / sc), torch.zeros_like(w)) + zero[:, :, None]
    q = q.clamp(0, 15).view(N, ng * G)[:, :K]
    return {"w": int4_f32(q, scale, None if s["sym"] else zero, K, G).to(bf)}


# ---------------------------------------------------------------------------
# the framework's calls

def run(s):
    if not own:
        return plain(s)
    import bit_quantized_finetuning_quantize_amd as q
    op = s["op"]
    if op == "lp_fwd":
        if "wsp" not in s:  # the workspace that a serving loop keeps
            s["wsp"] = q.logits_workspace(s["T"], s["V"], s["top"], s["z"].device)
        logp, ent, ids, top, _ = q.qlora_logprobs_fwd(s["z"], s["target"], s["temp"], n_top=s["top"], ws=s["wsp"])
        out = {"logp": logp, "entropy": ent}
        return dict(out, top_ids=ids, top_logp=top) if s["top"] else out
    if op == "lp_bwd":
        return {"dz": q.qlora_logprobs_bwd(s["z"], s["target"], s["kept"], s["g_logp"], s["g_ent"], s["temp"])}
    if op == "kd_fwd":
        if "wsp" not in s:
            s["wsp"] = q.logits_workspace(s["T"], s["V"], 0, s["z"].device)
        return {"loss": q.qlora_distill_fwd(s["z"], s["ids"], s["values"], s["lse"], s["temp"], ws=s["wsp"])[0]}
    if op == "kd_bwd":
        return {"dz": q.qlora_distill_bwd(s["z"], s["ids"], s["values"], s["kept"], s["g"], s["temp"])}
    if op == "int4_quant":
        return {"w": q.qlora_int4_dequantize(q.qlora_int4_quantize(s["w"], s["G"], s["sym"]))}
    w = q.Int4Weight(s["codes"], s["scales"], s["zeros"], (s["N"], s["K"]), s["G"])
    return {"y": q.qlora_int4_linear_fwd(s["x"], w, torch.float32 if s["f32"] else torch.bfloat16)}


# ---------------------------------------------------------------------------
# the definition in 64 bits, apart from the plain form: log-softmax over the
# whole row, gradients by the chain rule through log p, alternatives picked
# one after another, weights decoded a column at a time

PART = 1 << 26  # elements of a row block in 64 bits


def _blocks(s, f):
    """f over blocks of rows, joined."""
    rows = max(1, PART // s["V"])
    parts = [f(a, min(s["T"], a + rows)) for a in range(0, s["T"], rows)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _lp_exact(s, a, b):
    logp = torch.log_softmax(s["z"][a:b].double() / s["temp"], dim=1)
    p = logp.exp()
    plogp = torch.special.xlogy(p, p)
    ent = -plogp.sum(dim=1)
    tgt = s["target"][a:b]
    if s["op"] == "lp_bwd":
        # d/dx of sum_j c_j log p_j + H through the softmax's Jacobian
        c = torch.zeros_like(p)
        has = (tgt >= 0).nonzero()[:, 0]
        c[has, tgt[has]] = s["g_logp"][a:b].double()[has]
        dx = c - p * c.sum(dim=1, keepdim=True)
        dx -= s["g_ent"][a:b].double()[:, None] * (plogp + p * ent[:, None])
        return {"dz": dx / s["temp"]}
    row = torch.arange(b - a, device=p.device)
    out = {"logp": torch.where(tgt >= 0, logp[row, tgt.clamp(min=0)], torch.zeros_like(ent)), "entropy": ent}
    if s["top"]:
        left, V = s["z"][a:b].double(), s["V"]
        place = torch.arange(V, device=p.device)
        ids = []
        for _ in range(s["top"]):
            best = left.amax(dim=1, keepdim=True)
            ids.append(torch.where(left == best, place, V).amin(dim=1))
            left = left.scatter(1, ids[-1][:, None], -math.inf)
        out["top_ids"] = torch.stack(ids, dim=1)
        out["top_logp"] = torch.gather(logp, 1, out["top_ids"])
    return out


def _kd_exact(s, a, b):
    V, temp = s["V"], s["temp"]
    logp = torch.log_softmax(s["z"][a:b].double() / temp, dim=1)
    ids, val = s["ids"][a:b], s["values"][a:b].double() / temp
    ok = (ids >= 0) & (ids < V)
    logq = torch.where(ok, val, torch.full_like(val, -math.inf))
    rest = s["lse"] is not None
    logq = logq - (s["lse"][a:b].double()[:, None] if rest else torch.logsumexp(logq, dim=1, keepdim=True))
    q = logq.exp()
    there = torch.zeros(b - a, V, dtype=torch.float64, device=q.device)  # q spread over the vocabulary
    r, c = ok.nonzero().unbind(1)
    there[r, ids[r, c]] = q[r, c]
    on = torch.zeros_like(there)
    on[r, ids[r, c]] = 1.0
    qr = (1.0 - q.sum(dim=1)).clamp(min=0.0) * rest
    pr = (logp.exp() * (1.0 - on)).sum(dim=1)
    qr = torch.where(pr > 0, qr, torch.zeros_like(qr))
    if s["op"] == "kd_fwd":
        cross = torch.where(there > 0, there * logp, torch.zeros_like(there)).sum(dim=1)
        tail = torch.special.xlogy(qr, qr) - torch.special.xlogy(qr, pr)
        return {"loss": torch.special.xlogy(q, q).sum(dim=1) - cross + tail}
    p = logp.exp()
    # the rest's gradient goes to its tokens by their share of it
    share = torch.where(pr > 0, qr / pr, torch.zeros_like(pr))[:, None] * p * (1.0 - on)
    dx = p * (q.sum(dim=1) + qr)[:, None] - there - share
    return {"dz": dx * (s["g"][a:b].double()[:, None] / temp)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("lp"):
        return _blocks(s, lambda a, b: _lp_exact(s, a, b))
    if op.startswith("kd"):
        return _blocks(s, lambda a, b: _kd_exact(s, a, b))
    N, K, G = case["N"], case["K"], case["G"]
    if op == "int4_fwd":
        w = torch.empty(N, K, dtype=torch.float64, device=s["x"].device)
        w[:, 0::2], w[:, 1::2] = (s["codes"] % 16).double(), (s["codes"] // 16).double()
        for g in range(-(-K // G)):
            z = 8.0 if case["sym"] else s["zeros"][:, g, None].double()
            w[:, g * G:(g + 1) * G] = (w[:, g * G:(g + 1) * G] - z) * s["scales"][:, g, None].double()
        return {"y": s["x"].double() @ w.T.contiguous()}
    out = torch.empty(N, K, dtype=torch.float64, device=s["w"].device)
    for a in range(0, K, G):
        w = s["w"][:, a:a + G].double()
        # the scale is defined by float32 operations and one rounding to bf16
        if case["sym"]:
            sc = (w.abs().amax(dim=1, keepdim=True) / 7).float().to(torch.bfloat16).double()
            z = torch.full_like(sc, 8.0)
        else:
            lo, hi = w.amin(dim=1, keepdim=True).clamp(max=0), w.amax(dim=1, keepdim=True).clamp(min=0)
            sc = ((hi - lo).float().double() / 15).float().to(torch.bfloat16).double()
            z = torch.where(sc > 0, (-lo / sc).round(), torch.zeros_like(sc)).clamp(0, 15)
        q = (torch.where(sc > 0, w / sc, torch.zeros_like(w)).round() + z).clamp(0, 15)
        out[:, a:a + G] = sc * (q - z)
    return {"w": out}
