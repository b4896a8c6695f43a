"""Measured cases of the linear attention operators and of the query/key norm
with rotation: inputs, plain forms, the framework's calls and exact values.

Operators (case key ``op``):

* ``rope``      gdn_qk_norm_rope: RMS norm of every query and key head row, then
                the rotation of its first ``R`` dimensions by its token's positions.
* ``rope_bwd``  gdn_qk_norm_rope_backward: gradients of its inputs and weights.
* ``prefill``   gdn_linear_prefill: linear attention with a decay per head over
                packed sequences, states in and out.
* ``bwd``       gdn_linear_prefill_backward: its gradients.
* ``decode``    gdn_linear_decode_step: one token per sequence, in place on the
                states; ``decode_slots`` the same over a pool of state slots.

Sizes follow the head layouts this repository already works with: 16 q/k and 48
v heads of 128, layers of 4,096 tokens and up, 256 decoding sequences, and the
hybrid stack's attention heads (24 query, 4 key heads of 256, 64 rotated).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 128  # tokens per chunk of the plain chunked form


def listed():
    return [
        # one decoding step's queries and keys of an attention layer: latency
        dict(name="rope_step", op="rope", T=16, Hq=24, Hk=4, D=256, R=64, axes=1, dtype="bf16"),
        # a prompt's queries and keys of a linear layer, three position axes
        dict(name="rope_prompt", op="rope", T=16384, Hq=16, Hk=16, D=128, R=128, axes=3, dtype="bf16"),
        # training: a short odd batch in fp32, and a batch of attention heads
        dict(name="rope_bwd_small", op="rope_bwd", T=531, Hq=6, Hk=2, D=64, R=32, axes=1, dtype="fp32"),
        dict(name="rope_bwd_train", op="rope_bwd", T=16384, Hq=24, Hk=4, D=256, R=64, axes=1, dtype="bf16"),
        # a few short prompts of a small fp32 model (exact arithmetic path)
        dict(name="prefill_small", op="prefill", lens="77,0,300,1", Hqk=2, Hv=4, D=64, dtype="fp32",
             decay="slopes", state=True),
        # one layer of a 4,096-token prompt, and of a long one
        dict(name="prefill_layer4k", op="prefill", lens="4096", Hqk=16, Hv=48, D=128, dtype="bf16",
             decay="slopes", state=False),
        dict(name="prefill_long", op="prefill", lens="65536", Hqk=16, Hv=48, D=128, dtype="bf16",
             decay="slopes", state=True),
        # continued requests of mixed lengths, packed
        dict(name="prefill_ragged", op="prefill", lens="1,130,2500,64,777,4100,333,129,1500", Hqk=16, Hv=48,
             D=128, dtype="bf16", decay="none", state=True),
        # training: gradients of one 4,096-token sequence, and of a packed batch with states
        dict(name="bwd_layer4k", op="bwd", lens="4096", Hqk=16, Hv=48, D=128, dtype="bf16", decay="slopes",
             state=False),
        dict(name="bwd_ragged", op="bwd", lens="5000,1,2047,900,3333", Hqk=16, Hv=48, D=128, dtype="bf16",
             decay="slopes", state=True),
        # serving: one sequence's step (latency), and a batch of states in a slot pool
        dict(name="decode_one", op="decode", N=1, Hqk=16, Hv=48, D=128, dtype="bf16", decay="slopes"),
        dict(name="decode_slots", op="decode_slots", N=256, slots=320, Hqk=16, Hv=48, D=128, dtype="bf16",
             decay="slopes"),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "prefill", "prefill", "bwd", "bwd", "decode", "decode_slots"])
    dtype = "bf16" if rng.random() < 0.75 else "fp32"
    if op in ("rope", "rope_bwd"):
        D = rng.choice([64, 128, 256])
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 3, 6]) if Hk < 8 else rng.choice([16, 24])
        R = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= D])
        return dict(op=op, T=_spread(rng, 1, 16384), Hq=Hq, Hk=Hk, D=D, R=R, axes=rng.choice([1, 1, 2, 3]),
                    dtype=dtype)
    if op in ("decode", "decode_slots"):
        N = _spread(rng, 1, 256)
        Hqk = rng.choice([2, 4, 8, 16])
        c = dict(op=op, N=N, Hqk=Hqk, Hv=Hqk * rng.choice([1, 2, 3]), D=128 if rng.random() < 0.75 else 64,
                 dtype=dtype, decay=rng.choice(["slopes", "none", "strong"]))
        if op == "decode_slots":
            c["slots"] = N + rng.randint(0, 40)
        return c
    if dtype == "bf16":  # the tensor-core shapes
        Hqk, D, most = rng.choice([2, 4, 8, 16]), 128, 16384
    else:
        Hqk, D, most = rng.choice([1, 2, 4]), rng.choice([16, 32, 64, 128]), 1024
    total, lens = _spread(rng, 1, most), []
    left = rng.randint(1, 7)
    while left > 1 and total > 1:  # cut into pieces of any size, empty ones among them
        x = rng.choice([0, 1, rng.randint(1, total), rng.randint(1, total)])
        lens.append(min(x, total - 1))
        total -= lens[-1]
        left -= 1
    lens.append(total)
    return dict(op=op, lens=",".join(map(str, lens)), Hqk=Hqk, Hv=Hqk * rng.choice([1, 2, 3]), D=D, dtype=dtype,
                decay=rng.choice(["slopes", "none", "strong"]), state=rng.random() < 0.6)


# --------------------------------------------------------------------- inputs


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _log_decay(case, device):
    """Per-head log decays: a geometric series of slopes, none, or strong ones."""
    H = case["Hv"]
    h = torch.arange(1, H + 1, dtype=torch.float64)
    g = {"slopes": -(2.0 ** (-8.0 * h / H)), "none": 0.0 * h, "strong": -0.5 - 5.0 * h / H}[case["decay"]]
    return g.to(torch.float32).to(device)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def rand(*shape, dtype=dt, std=1.0):
        return (std * torch.randn(shape, generator=gen, device=dev)).to(dtype)

    op, s = case["op"], {"case": case}
    if op in ("rope", "rope_bwd"):
        T, Hq, Hk, D, R = case["T"], case["Hq"], case["Hk"], case["D"], case["R"]
        A = case["axes"]
        s["xq"], s["xk"] = rand(T, Hq, D), rand(T, Hk, D)
        s["wq"], s["wk"] = (1 + rand(D, dtype=torch.float32, std=0.2) for _ in range(2))
        if op == "rope_bwd":
            s["dq"], s["dk"] = rand(T, Hq, D), rand(T, Hk, D)
        # positions up to the hybrid stack's 262,144-token context
        first = torch.randint(0, 262144 - T, (1,), generator=gen, device=dev)
        p = first + torch.arange(T, device=dev)
        extra = [torch.randint(0, 1000, (T,), generator=gen, device=dev) for _ in range(A - 1)]
        s["positions"] = torch.stack([p] + extra).to(torch.int32).contiguous()
        i = torch.arange(0, R, 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = (1e7 ** (-i / R)).to(torch.float32)
        cut = [R // 2 // A] * (A - 1)  # frequencies per axis
        s["sections"] = cut + [R // 2 - sum(cut)]
        s["eps"] = 1e-6
        return s
    Hqk, Hv, D = case["Hqk"], case["Hv"], case["D"]
    s["log_decay"] = _log_decay(case, dev)
    s["scale"] = D ** -0.5
    if op in ("decode", "decode_slots"):
        N = case["N"]
        s["q"], s["k"], s["v"] = rand(N, Hqk, D), rand(N, Hqk, D), rand(N, Hv, D)
        rows = case.get("slots", N)
        s["state"] = rand(rows, Hv, D, D, dtype=torch.float32)
        if op == "decode_slots":  # slots in any order, an eighth of the requests new
            s["slot_idx"] = torch.randperm(rows, generator=gen, device=dev)[:N].to(torch.int32)
            s["reset"] = (torch.rand(N, generator=gen, device=dev) < 0.125).to(torch.int32)
        s["o"] = torch.empty(N, Hv, D, dtype=dt, device=dev)
        return s
    lens = _lens(case)
    T, N = sum(lens), len(lens)
    s["lens"] = lens
    s["q"], s["k"], s["v"] = rand(T, Hqk, D), rand(T, Hqk, D), rand(T, Hv, D)
    s["cu"] = torch.tensor([sum(lens[:n]) for n in range(N + 1)], dtype=torch.int32).to(dev)
    s["s0"] = rand(N, Hv, D, D, dtype=torch.float32) if case["state"] else None
    if op == "bwd":
        s["do"] = rand(T, Hv, D)
        s["dsT"] = rand(N, Hv, D, D, dtype=torch.float32) if case["state"] else None
    return s


# ------------------------------------------------------------------------ run


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    if op in ("rope", "rope_bwd"):
        return _plain_rope(s) if op == "rope" else _plain_rope_bwd(s)
    if op in ("decode", "decode_slots"):
        return _plain_decode(s)
    return _plain_prefill(s) if op == "prefill" else _plain_bwd(s)


def _own(op, s):
    import gated_deltanet_04_b200 as gdn

    if op == "rope":
        return gdn.gdn_qk_norm_rope(s["xq"], s["xk"], s["positions"], s["inv_freq"], wq=s["wq"], wk=s["wk"],
                                    eps=s["eps"], sections=s["sections"])
    if op == "rope_bwd":
        return gdn.gdn_qk_norm_rope_backward(s["dq"], s["dk"], s["xq"], s["xk"], s["positions"], s["inv_freq"],
                                             wq=s["wq"], wk=s["wk"], eps=s["eps"], sections=s["sections"])
    if op == "decode":
        return gdn.gdn_linear_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"],
                                          o=s["o"]), s["state"]
    if op == "decode_slots":
        return gdn.gdn_linear_decode_step_slots(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["slot_idx"],
                                                s["reset"], scale=s["scale"], o=s["o"]), s["state"]
    if op == "prefill":
        return gdn.gdn_linear_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["s0"], s["cu"], scale=s["scale"])
    dq, dk, dv, ds0 = gdn.gdn_linear_prefill_backward(
        s["do"], s["q"], s["k"], s["v"], s["log_decay"], s["s0"], s["cu"], dfinal_state=s["dsT"],
        scale=s["scale"], output_dinitial_state=s["s0"] is not None)
    return [dq, dk, dv] + ([ds0] if ds0 is not None else [])


# ---------------------------------------------------------------- plain forms


def _cos_sin(s):
    """[T, 1, R/2] each: angles in 64 bits (far positions), cosine and sine to 32."""
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=s["positions"].device),
                                   torch.tensor(s["sections"], device=s["positions"].device))
    ang = s["positions"].double()[axis].T * s["inv_freq"].double()
    return ang.cos().float()[:, None], ang.sin().float()[:, None]


def _turn(y, cos, sin):
    h = cos.shape[-1]
    a, b, rest = y[..., :h], y[..., h:2 * h], y[..., 2 * h:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1)


def _plain_rope(s):
    cos, sin = _cos_sin(s)

    def one(x, w):
        x = x.float()
        return _turn(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w, cos, sin)

    return one(s["xq"], s["wq"]).to(s["xq"].dtype), one(s["xk"], s["wk"]).to(s["xk"].dtype)


def _plain_rope_bwd(s):
    cos, sin = _cos_sin(s)

    def one(dz, x, w):
        dy, x = _turn(dz.float(), cos, -sin), x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        n = x * r
        dn = dy * w
        return r * (dn - n * (dn * n).mean(-1, keepdim=True)), (dy * n).sum((0, 1))

    (dxq, dwq), (dxk, dwk) = one(s["dq"], s["xq"], s["wq"]), one(s["dk"], s["xk"], s["wk"])
    return dxq.to(s["xq"].dtype), dxk.to(s["xk"].dtype), dwq, dwk


def _plain_decode(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    G = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    lam = s["log_decay"].exp()[None, :, None, None]
    S = s["state"]
    at = None
    if "slot_idx" in s:
        at = s["slot_idx"].long()
        S = torch.where(s["reset"].bool()[:, None, None, None], 0.0, S[at])
    S = lam * S + v[..., :, None] * k[..., None, :]
    s["o"].copy_(s["scale"] * (S * q[..., None, :]).sum(-1))
    if at is None:
        s["state"].copy_(S)
    else:
        s["state"][at] = S
    return s["o"], s["state"]


class _Padded:
    """Packed rows as [N * H, chunks, CHUNK, D], every sequence moved to the end
    of its padded row (its front filled with zeros), and back."""

    def __init__(self, s):
        lens, dev = s["lens"], s["q"].device
        self.N, self.H = len(lens), s["v"].shape[1]
        self.G = self.H // s["q"].shape[1]
        self.nc = max(1, -(-max(lens) // CHUNK))
        L = self.nc * CHUNK
        cu = s["cu"].long()
        self.len = cu[1:] - cu[:-1]
        at = cu[1:, None] - L + torch.arange(L, device=dev)
        self.valid = at >= cu[:-1, None]
        self.at = at.clamp(min=0)
        self.t = (at - cu[:-1, None]).clamp(min=0)          # token's place in its sequence
        self.left = cu[1:, None] - 1 - at                   # tokens after it
        self.g = s["log_decay"].repeat(self.N)              # [N * H]
        i = torch.arange(CHUNK, device=dev, dtype=torch.float32)
        self.i = i
        d = i[:, None] - i[None, :]
        self.D = torch.where(d >= 0, (self.g[:, None, None] * d.clamp(min=0)).exp(), 0.0)  # lam^(i-j), j <= i
        c = torch.arange(self.nc, device=dev, dtype=torch.float32)
        e = c[:, None] - c[None, :] - 1.0                   # chunks between c' < c
        self.E = torch.where(e >= 0, (self.g[:, None, None] * CHUNK * e.clamp(min=0)).exp(), 0.0)

    def pack(self, x, heads):
        x = x.float()
        if heads != self.H:
            x = x.repeat_interleave(self.H // heads, 1)
        y = torch.where(self.valid[..., None, None], x[self.at], 0.0) if x.shape[0] else \
            x.new_zeros(self.N, self.nc * CHUNK, self.H, x.shape[-1])
        return y.transpose(1, 2).reshape(self.N * self.H, self.nc, CHUNK, -1)

    def unpack(self, y):
        y = y.reshape(self.N, self.H, self.nc * CHUNK, -1).transpose(1, 2)
        return y[self.valid]

    def power(self, n):
        """lam^n for counts n [N, L] of every token: [N * H, chunks, CHUNK, 1]."""
        x = (self.g.view(self.N, self.H, 1) * n[:, None].float()).exp()
        return x.reshape(self.N * self.H, self.nc, CHUNK, 1)

    def weights(self, n):
        """lam^n for counts n [CHUNK] within a chunk: [N * H, 1, CHUNK, 1]."""
        return (self.g[:, None] * n).exp()[:, None, :, None]

    def whole(self):
        """lam^length: [N, H, 1, 1]."""
        return (self.g.view(self.N, self.H) * self.len[:, None].float()).exp()[..., None, None]

    def states(self, x, y, n, before):
        """The sum of lam^n x y^T over every chunk, n counted within it, and what
        the chunks before (or after) each one carry to it: [NH, chunks, Dx, Dy]."""
        inc = (x * self.weights(n)).transpose(-1, -2) @ y
        nh, nc, dx, dy = inc.shape
        E = self.E if before else self.E.transpose(-1, -2)
        return (E @ inc.reshape(nh, nc, dx * dy)).reshape(inc.shape), inc


def _plain_prefill(s):
    p, sc = _Padded(s), s["scale"]
    Hqk, Hv = s["q"].shape[1], s["v"].shape[1]
    q, k, v = p.pack(s["q"], Hqk), p.pack(s["k"], Hqk), p.pack(s["v"], Hv)
    S, inc = p.states(v, k, CHUNK - 1 - p.i, True)
    final = (p.g[:, None, None] * CHUNK).exp() * S[:, -1] + inc[:, -1]
    final = final.reshape(p.N, p.H, *final.shape[1:])
    o = ((q @ k.transpose(-1, -2)) * p.D[:, None]) @ v + p.weights(p.i + 1) * (q @ S.transpose(-1, -2))
    if s["s0"] is not None:
        s0 = s["s0"].reshape(-1, 1, *s["s0"].shape[2:])
        o = o + p.power(p.t + 1) * (q @ s0.transpose(-1, -2))
        final = final + p.whole() * s["s0"]
    return p.unpack(sc * o).to(s["q"].dtype), final


def _plain_bwd(s):
    p, sc = _Padded(s), s["scale"]
    Hqk, Hv = s["q"].shape[1], s["v"].shape[1]
    q, k, v = p.pack(s["q"], Hqk), p.pack(s["k"], Hqk), p.pack(s["v"], Hv)
    do = sc * p.pack(s["do"], Hv)
    P = (q @ k.transpose(-1, -2)) * p.D[:, None]
    dP = (do @ v.transpose(-1, -2)) * p.D[:, None]
    S, _ = p.states(v, k, CHUNK - 1 - p.i, True)
    G, _ = p.states(do, q, p.i + 1, False)
    up, down = p.weights(p.i + 1), p.weights(CHUNK - 1 - p.i)
    dq = dP @ k + up * (do @ S)
    dk = dP.transpose(-1, -2) @ q + down * (v @ G)
    dv = P.transpose(-1, -2) @ do + down * (k @ G.transpose(-1, -2))
    if s["s0"] is not None:
        s0 = s["s0"].reshape(-1, 1, *s["s0"].shape[2:])
        dq = dq + p.power(p.t + 1) * (do @ s0)
    ds0 = _from_start(p, do, q)
    if s["dsT"] is not None:
        dsT = s["dsT"].reshape(-1, 1, *s["dsT"].shape[2:])
        far = p.power(p.left)
        dk = dk + far * (v @ dsT)
        dv = dv + far * (k @ dsT.transpose(-1, -2))
        ds0 = ds0 + p.whole() * s["dsT"]

    def shared(x):  # sum over the v-heads that share a q/k head
        x = p.unpack(x)
        return x.reshape(x.shape[0], Hqk, Hv // Hqk, x.shape[-1]).sum(2)

    dt = s["q"].dtype
    return [shared(dq).to(dt), shared(dk).to(dt), p.unpack(dv).to(dt)] + ([ds0] if s["s0"] is not None else [])


def _from_start(p, do, q):
    """sum_t lam^(t+1) do_t q_t^T over each sequence: [N, H, Dv, Dk]."""
    w = p.power(p.t + 1)
    nh = do.shape[0]
    x = (do * w).reshape(nh, -1, do.shape[-1])
    return (x.transpose(-1, -2) @ q.reshape(nh, -1, q.shape[-1])).reshape(p.N, p.H, do.shape[-1], q.shape[-1])


# ----------------------------------------------------------------------- work


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        each = 2 if op == "rope" else 3
        return {"bytes": each * es * n + 4 * case["T"] * case["axes"] + 8 * case["D"] * (1 if op == "rope" else 2),
                "flops": (8 if op == "rope" else 16) * n}
    Hqk, Hv, D = case["Hqk"], case["Hv"], case["D"]
    if op in ("decode", "decode_slots"):
        N = case["N"]
        return {"bytes": 8 * N * Hv * D * D + es * N * (2 * Hqk + 2 * Hv) * D, "flops": 5 * N * Hv * D * D}
    lens = _lens(case)
    T, N = sum(lens), len(lens)
    st = 4 * N * Hv * D * D
    pairs = sum((n // CHUNK) * CHUNK * (CHUNK + 1) // 2 + (n % CHUNK) * (n % CHUNK + 1) // 2 for n in lens)
    if op == "prefill":
        return {"bytes": es * T * D * (2 * Hqk + 2 * Hv) + st * (2 if case["state"] else 1),
                "flops": 4 * pairs * Hv * D + 4 * T * Hv * D * D}
    return {"bytes": es * T * D * (4 * Hqk + 3 * Hv) + (3 * st if case["state"] else 0),
            "flops": 10 * pairs * Hv * D + 10 * T * Hv * D * D}


# ---------------------------------------------------------------------- exact


def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token, the rotation as
    a product of complex numbers."""
    op = case["op"]
    s = prepare(case, seed)
    if op in ("rope", "rope_bwd"):
        return _exact_rope(s, op == "rope_bwd")
    if op in ("decode", "decode_slots"):
        return _exact_decode(s)
    lens = _lens(case)
    steps = max(lens) * (1 if op == "prefill" else 2)
    if steps * (4e-5 + 6e-12 * len(lens) * case["Hv"] * case["D"] ** 2) > 18:
        return None
    return _exact_prefill(s) if op == "prefill" else _exact_bwd(s)


def _exact_rope(s, backward):
    f, pos = s["inv_freq"].double(), s["positions"].double()
    ang, at = [], 0
    for a, n in enumerate(s["sections"]):
        ang.append(pos[a][:, None] * f[at:at + n])
        at += n
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=f.device), torch.cat(ang, 1))[:, None]
    h = f.numel()

    def turn(y, u):
        z = torch.complex(y[..., :h], y[..., h:2 * h]) * u
        return torch.cat([z.real, z.imag, y[..., 2 * h:]], -1)

    out = []
    for key in "qk":
        x, w = s["x" + key].double(), s["w" + key].double()
        rms = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt()
        if not backward:
            out.append(turn(x / rms * w, unit))
            continue
        dy = turn(s["d" + key].double(), unit.conj())
        dn = dy * w
        dx = dn / rms - x * (dn * x).sum(-1, keepdim=True) / (x.shape[-1] * rms ** 3)
        out.append((dx, (dy * x / rms).sum((0, 1))))
    return (out[0], out[1]) if not backward else (out[0][0], out[1][0], out[0][1], out[1][1])


def _heads(x, H):
    return x.double().repeat_interleave(H // x.shape[1], 1)


def _exact_decode(s):
    Hv = s["v"].shape[1]
    q, k, v = _heads(s["q"], Hv), _heads(s["k"], Hv), s["v"].double()
    pool = s["state"].double()
    lam = torch.exp(s["log_decay"].double())
    o = torch.empty_like(v)
    for n in range(v.shape[0]):
        at = int(s["slot_idx"][n]) if "slot_idx" in s else n
        S = pool[at] * lam[:, None, None]
        if "reset" in s and int(s["reset"][n]):
            S = torch.zeros_like(S)
        S = S + torch.einsum("hi,hj->hij", v[n], k[n])
        pool[at] = S
        o[n] = s["scale"] * torch.einsum("hij,hj->hi", S, q[n])
    return o, pool


def _time_major(s, names):
    """The named packed tensors as [T_max, N * H, D] in 64 bits, sequences
    beginning together, and whether each token exists: [T_max, N * H, 1, 1]."""
    lens, H = s["lens"], s["v"].shape[1]
    Tm, dev = max(1, max(lens)), s["q"].device
    there = torch.arange(Tm, device=dev)[:, None] < torch.tensor(lens, device=dev)[None]
    out = []
    for name in names:
        x = _heads(s[name], H)
        y = x.new_zeros(Tm, len(lens), H, x.shape[-1])
        for n, L in enumerate(lens):
            y[:L, n] = x[sum(lens[:n]):sum(lens[:n]) + L]
        out.append(y.reshape(Tm, -1, x.shape[-1]))
    return out, there.repeat_interleave(H, 1)[..., None, None].double()


def _packed(y, s):
    N, H = len(s["lens"]), s["v"].shape[1]
    y = y.reshape(y.shape[0], N, H, -1)
    return torch.cat([y[:L, n] for n, L in enumerate(s["lens"])])


def _exact_prefill(s):
    (q, k, v), there = _time_major(s, "qkv")
    N, H, D = len(s["lens"]), v.shape[1] // len(s["lens"]), v.shape[2]
    lam = torch.exp(s["log_decay"].double()).repeat(N)[:, None, None]
    S = q.new_zeros(N * H, D, D) if s["s0"] is None else s["s0"].double().reshape(N * H, D, D).clone()
    o = torch.empty_like(v)
    decay = 1.0 + there * (lam - 1.0) if min(s["lens"]) < len(q) else None  # a finished sequence keeps its state
    for t in range(len(q)):
        S.mul_(lam if decay is None else decay[t]).baddbmm_(v[t][:, :, None], k[t][:, None, :])
        o[t] = torch.bmm(S, q[t][:, :, None])[..., 0]
    return _packed(s["scale"] * o, s), S.reshape(N, H, D, D)


def _exact_bwd(s):
    (q, k, v, do), there = _time_major(s, ["q", "k", "v", "do"])
    do = s["scale"] * do
    N, H, D = len(s["lens"]), v.shape[1] // len(s["lens"]), v.shape[2]
    lam = torch.exp(s["log_decay"].double()).repeat(N)[:, None, None]
    decay = 1.0 + there * (lam - 1.0) if min(s["lens"]) < len(q) else None
    at = (lambda t: lam) if decay is None else (lambda t: decay[t])
    S = q.new_zeros(N * H, D, D) if s["s0"] is None else s["s0"].double().reshape(N * H, D, D).clone()
    G = q.new_zeros(N * H, D, D) if s["dsT"] is None else s["dsT"].double().reshape(N * H, D, D).clone()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(len(q)):
        S.mul_(at(t)).baddbmm_(v[t][:, :, None], k[t][:, None, :])
        dq[t] = torch.bmm(do[t][:, None, :], S)[:, 0]
    for t in range(len(q) - 1, -1, -1):
        G.baddbmm_(do[t][:, :, None], q[t][:, None, :])  # dL/dS_t
        dk[t] = torch.bmm(v[t][:, None, :], G)[:, 0]
        dv[t] = torch.bmm(G, k[t][:, :, None])[..., 0]
        G.mul_(at(t))
    Hqk = s["q"].shape[1]

    def shared(x):
        x = _packed(x, s)
        return x.reshape(len(x), Hqk, H // Hqk, D).sum(2)

    out = [shared(dq), shared(dk), _packed(dv, s)]
    return out + ([G.reshape(N, H, D, D)] if s["s0"] is not None else [])
