"""Timed cases of the gated linear recurrence and the residual RMS norm.

Six kinds of pass, each as a user's program makes it:

  scan_forward   prefill: y and the last state of h_t = f_t h_{t-1} + i_t x_t
  scan_train     the recurrence's forward and its backward
  scan_step      one decoded token for every sequence of a batch, states in slots
  norm_forward   s = x + r and its RMS norm in 16 or 32 bits
  norm_e4m3      the same with the norm's output in e4m3 with scales
  norm_train     the norm's forward and its backward

Tensors follow the library's head layout [B, H, N, d]; "tokens" layouts are
views of [B, N, H, d] memory, and "packed" ones are the two halves of one
[B, N, 2, H, d] projection.  ``run`` computes the plain form in elementary torch
operations, or, with ``own`` set, calls the library.
"""

import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_E4M3_MAX = 448.0


def _scan(name, op, B, H, N, d, dtype, gate="sigmoid", coupled=True, layout="heads", ragged=False, state=True):
    return {"name": name, "op": op, "B": B, "H": H, "N": N, "d": d, "dtype": dtype, "gate": gate,
            "coupled": coupled, "layout": layout, "ragged": ragged, "state": state}


def _norm(name, op, B, H, N, d, x_dtype, r_dtype, y_dtype, group=0, residual=True):
    return {"name": name, "op": op, "B": B, "H": H, "N": N, "d": d, "x_dtype": x_dtype, "r_dtype": r_dtype,
            "y_dtype": y_dtype, "group": group, "residual": residual}


def listed():
    return [
        # Prefill of one short sequence (a 14 x 14 token grid, one head): latency.
        _scan("scan_forward_196", "scan_forward", 1, 1, 196, 32, "f32"),
        # Prefill of one long sequence (a 256 x 256 token grid, 8 heads): few columns, many tokens.
        _scan("scan_forward_65536", "scan_forward", 1, 8, 65536, 64, "bf16"),
        # A training step over a padded batch of documents of odd lengths, float32, odd width.
        _scan("scan_train_ragged", "scan_train", 5, 3, 1013, 33, "f32", gate="log", coupled=False, ragged=True),
        # A training step of a wide layer over long sequences, x and g as halves of one projection.
        _scan("scan_train_32768", "scan_train", 2, 32, 32768, 64, "bf16", layout="packed"),
        # Decoding for one request, then for a full serving batch.
        _scan("scan_step_1", "scan_step", 1, 8, 1, 64, "bf16"),
        _scan("scan_step_512", "scan_step", 512, 32, 1, 64, "bf16"),
        # After the attention of the 14 x 14 stage: its float32 [B, H, N, d] output joins a bf16 residual.
        _norm("norm_forward_heads", "norm_forward", 64, 5, 196, 64, "f32", "bf16", "bf16"),
        # Between the blocks of a model, a training-sized batch of rows.
        _norm("norm_forward_rows", "norm_forward", 8, 1, 4096, 2048, "bf16", "bf16", "bf16"),
        # Decoding in front of an 8-bit projection: a few rows, a scale a row.
        _norm("norm_e4m3_16", "norm_e4m3", 16, 1, 1, 4096, "bf16", "bf16", "e4m3"),
        # Prefill in front of an 8-bit projection, a scale every 128 columns.
        _norm("norm_e4m3_16384", "norm_e4m3", 4, 1, 4096, 4096, "bf16", "bf16", "e4m3", group=128),
        # A small training step in float32, odd width.
        _norm("norm_train_odd", "norm_train", 7, 1, 111, 1001, "f32", "f32", "f32"),
        # A training step of a wide model.
        _norm("norm_train_16384", "norm_train", 8, 1, 2048, 2560, "bf16", "bf16", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_forward", "scan_train", "scan_step", "norm_forward", "norm_e4m3", "norm_train"])
    if op.startswith("scan"):
        dtype = rng.choice(["f32", "bf16"])
        gate, coupled = rng.choice(["sigmoid", "log"]), rng.random() < 0.5
        layout = rng.choice(["heads", "tokens", "packed"])
        d = rng.choice([32, 64, 64, 128, rng.randint(1, 256)])
        H = _log_int(rng, 1, 32)
        if op == "scan_step":
            return _scan("", op, _log_int(rng, 1, 512), H, 1, min(d, 64), dtype, gate, coupled, layout)
        N = _log_int(rng, 1, 65536)
        cap = max(1, (2 * 32 * 32768 * 64) // (2 if dtype == "f32" else 1) // (H * N * d))
        if cap == 1:
            H = max(1, min(H, (2 * 32 * 32768 * 64) // (2 if dtype == "f32" else 1) // (N * d)))
        B = _log_int(rng, 1, min(64, cap))
        return _scan("", op, B, H, N, d, dtype, gate, coupled, layout, rng.random() < 0.4, rng.random() < 0.7)
    r_dtype = rng.choice(["f32", "bf16"])
    x_dtype = rng.choice([r_dtype, "f32"])
    y_dtype = "e4m3" if op == "norm_e4m3" else rng.choice(["bf16", r_dtype])
    group = 0
    if rng.random() < 0.35:  # the attention's output, heads apart
        H, d = rng.randint(1, 12), rng.choice([32, 64])
    else:
        H, d = 1, _log_int(rng, 64, 8192)
        if op == "norm_e4m3" or rng.random() < 0.5:
            d = max(128, d // 128 * 128)
            group = rng.choice([0, 128]) if op == "norm_e4m3" else 0
    rows = _log_int(rng, 1, max(2, min(32768, 2048 * 16384 // (H * d))))
    N = rng.randint(1, min(rows, 4096))
    return _norm("", op, max(1, rows // N), H, N, d, x_dtype, r_dtype, y_dtype, group, rng.random() < 0.8)


def _lengths(case):
    """Tokens of each sequence: the longest fills the batch, one is a single token, one is empty."""
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return [N] * B
    r = random.Random(B * 1000003 + N)
    n = [r.randint(0, N) for _ in range(B)]
    n[0] = N
    if B > 2:
        n[1], n[2] = 0, 1
    return n


def _layout(case, dtype, halves):
    """Empty [B, H, N, d] views in the case's layout, ``halves`` of them (packed: views of one buffer)."""
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    if case["layout"] == "heads":
        return [torch.empty(B, H, N, d, dtype=dtype, device="cuda") for _ in range(halves)]
    if case["layout"] == "tokens" or halves == 1:
        return [torch.empty(B, N, H, d, dtype=dtype, device="cuda").permute(0, 2, 1, 3) for _ in range(halves)]
    both = torch.empty(B, N, halves, H, d, dtype=dtype, device="cuda")
    return [both[:, :, i].permute(0, 2, 1, 3) for i in range(halves)]


def _scan_inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    dtype = _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x, g = _layout(case, dtype, 2)
    x.copy_(randn(B, H, N, d))
    # Gates remember from a few tokens to thousands of them, a scale for each channel.
    logits = randn(B, H, N, d).mul_(1.5).add_(torch.linspace(0.0, 7.0, H * d, device="cuda").view(H, 1, d))
    if case["gate"] == "log":
        logits.neg_().exp_().log1p_().neg_()
    g.copy_(logits)
    del logits
    st = {"case": case, "x": x, "g": g, "h0": None, "lengths": None, "dhN": None}
    if case["op"] == "scan_step":
        slots = 2 * B
        st["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
        st["h_in"] = randn(slots, H, d)
        # The states after the step have a pool of their own: the pass can be called again.
        st["h_out"] = st["h_in"].clone()
        return st
    if case["state"]:
        st["h0"] = randn(B, H, d)
    if case["ragged"]:
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if case["op"] == "scan_train":
        st["dy"], = _layout(case, dtype, 1)
        st["dy"].copy_(randn(B, H, N, d))
        if case["state"]:
            st["dhN"] = randn(B, H, d)
    return st


def _norm_inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    C = H * d
    xt, rt = _DT[case["x_dtype"]], _DT[case["r_dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    st = {"case": case, "eps": 1e-6}
    st["x"] = randn(B, H, N, d).to(xt)
    # A residual stream carries a few channels that are far larger than the rest.
    wide = torch.where(torch.rand(C, generator=gen, device="cuda") < 0.01, 20.0, 1.5)
    st["r"] = (randn(B, N, C) * wide).to(rt) if case["residual"] else None
    st["w"] = 1.0 + 0.2 * randn(C)
    if case["op"] == "norm_train":
        st["dy"] = randn(B, N, C).to(_DT[case["y_dtype"]])
        st["ds"] = randn(B, N, C).to(rt) if case["residual"] else None
    return st


def _make(case, seed):
    return (_scan_inputs if case["op"].startswith("scan") else _norm_inputs)(case, seed)


def prepare(case, seed):
    st = _make(case, seed)
    if not own:
        return st
    import laplacian_nystr_approximation_amd as L
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    st["L"] = L

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if case["op"].startswith("scan"):
        p = st["params"] = L.make_scan_params(B=B, H=H, N=N, d=d, dtype=case["dtype"], gate=case["gate"],
                                              coupled=case["coupled"])
        st["y"], = _layout(case, _DT[case["dtype"]], 1)
        if case["op"] == "scan_step":
            return st
        st["ws"] = empty(max(256, L.lapmix_scan_workspace_size(p)), dtype=torch.uint8)
        st["hN"] = empty(B, H, d)
        if case["op"] == "scan_train":
            st["states"] = empty(L.lapmix_scan_states_size(p) // 4)
            st["dx"], st["dg"] = _layout(case, _DT[case["dtype"]], 2)
            st["dh0"] = empty(B, H, d)
        return st
    C = H * d
    p = st["params"] = L.make_norm_params(B=B, H=H, N=N, d=d, x_dtype=case["x_dtype"], r_dtype=case["r_dtype"],
                                          y_dtype=case["y_dtype"], eps=st["eps"], group=case["group"])
    st["s"] = empty(B, N, C, dtype=_DT[case["r_dtype"]])
    if case["op"] == "norm_e4m3":
        st["y"] = empty(B, N, C, dtype=torch.float8_e4m3fn)
        st["scale"] = empty(B, N, C // (case["group"] or C))
    else:
        st["y"] = empty(B, N, C, dtype=_DT[case["y_dtype"]])
    if case["op"] == "norm_train":
        st["ws"] = empty(max(256, L.lapmix_norm_workspace_size(p)), dtype=torch.uint8)
        st["dr"] = empty(B, N, C, dtype=_DT[case["r_dtype"]])
        st["dx"] = empty(B, H, N, d, dtype=_DT[case["x_dtype"]])
        st["dw"] = empty(C)
    return st


def run(state):
    op = state["case"]["op"]
    if own:
        return {"scan_forward": _own_scan_forward, "scan_train": _own_scan_train, "scan_step": _own_scan_step,
                "norm_forward": _own_norm_forward, "norm_e4m3": _own_norm_e4m3,
                "norm_train": _own_norm_train}[op](state)
    return {"scan_forward": _plain_scan, "scan_train": _plain_scan, "scan_step": _plain_scan_step,
            "norm_forward": _plain_norm, "norm_e4m3": _plain_norm, "norm_train": _plain_norm}[op](state)


# ---- the library's calls

def _own_scan_forward(st):
    st["L"].lapmix_scan_forward_ws(st["x"], st["g"], st["y"], st["params"], st["ws"], h0=st["h0"], hN=st["hN"],
                                   lengths=st["lengths"])
    return [st["y"], st["hN"]]


def _own_scan_train(st):
    L = st["L"]
    L.lapmix_scan_forward_ws(st["x"], st["g"], st["y"], st["params"], st["ws"], h0=st["h0"], hN=st["hN"],
                             states=st["states"], lengths=st["lengths"])
    L.lapmix_scan_backward_ws(st["x"], st["g"], st["states"], st["dy"], st["dx"], st["dg"], st["params"], st["ws"],
                              dhN=st["dhN"], dh0=st["dh0"], lengths=st["lengths"])
    return [st["y"], st["hN"], st["dx"], st["dg"], st["dh0"]]


def _own_scan_step(st):
    st["L"].lapmix_scan_step(st["x"], st["g"], st["y"], st["h_in"], st["h_out"], st["params"], slots=st["slots"])
    return [st["y"], st["h_out"]]


def _own_norm_forward(st):
    st["L"].lapmix_norm_forward(st["x"], st["w"], st["y"], st["params"], r=st["r"], s=st["s"])
    return [st["s"], st["y"]]


def _own_norm_e4m3(st):
    st["L"].lapmix_norm_forward(st["x"], st["w"], st["y"], st["params"], r=st["r"], s=st["s"], scale=st["scale"])
    return [st["s"], st["y"], st["scale"]]


def _own_norm_train(st):
    L = st["L"]
    L.lapmix_norm_forward(st["x"], st["w"], st["y"], st["params"], r=st["r"], s=st["s"])
    L.lapmix_norm_backward_ws(st["dy"], st["s"], st["w"], st["params"], st["ws"], ds=st["ds"], dr=st["dr"],
                              dx=st["dx"], dw=st["dw"])
    return [st["s"], st["y"], st["dr"], st["dx"], st["dw"]]


# ---- the plain form: elementary operations in 32 bits, rounded once at the end

def _gate(case, g):
    """Forget gate f and 1 - f."""
    if case["gate"] == "log":
        g = torch.minimum(g, torch.zeros_like(g))
        return torch.exp(g), -torch.expm1(g)
    return 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))


def _prefix(f, u, h0):
    """h_t = f_t h_{t-1} + u_t for every t, by doubling steps along dim 2."""
    N = u.shape[2]
    A, S = f.clone(), u.clone()
    k = 1
    while k < N:
        S[:, :, k:] = S[:, :, k:] + A[:, :, k:] * S[:, :, :-k]
        A[:, :, k:] = A[:, :, k:] * A[:, :, :-k]
        k *= 2
    return S if h0 is None else S + A * h0[:, :, None]


def _plain_scan(st):
    case = st["case"]
    x, g = st["x"].float(), st["g"].float()
    B, H, N, d = x.shape
    dtype = st["x"].dtype
    f, i = _gate(case, g)
    slope = f * i if case["gate"] == "sigmoid" else torch.where(g <= 0, f, torch.zeros_like(f))
    del g
    if not case["coupled"]:
        i = torch.ones_like(f)
    live = None
    if st["lengths"] is not None:
        live = (torch.arange(N, device=x.device)[None] < st["lengths"][:, None])[:, None, :, None]
        f = torch.where(live, f, torch.ones_like(f))
        i = torch.where(live, i, torch.zeros_like(i))
        x = torch.where(live, x, torch.zeros_like(x))
    h = _prefix(f, i * x, st["h0"])
    y = h if live is None else torch.where(live, h, torch.zeros_like(h))
    out = [y.to(dtype), h[:, :, -1].clone()]
    if case["op"] == "scan_forward":
        return out
    del y
    dy = st["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, torch.zeros_like(dy))
    # dh_t = dy_t + f_{t+1} dh_{t+1}: the same recurrence from the last token back.
    after = torch.cat([f[:, :, 1:], torch.ones_like(f[:, :, :1])], dim=2)
    dh = _prefix(after.flip(2), dy.flip(2), st["dhN"]).flip(2)
    del after, dy
    first = st["h0"] if st["h0"] is not None else torch.zeros_like(h[:, :, 0])
    before = torch.cat([first[:, :, None], h[:, :, :-1]], dim=2)
    del h
    dx = dh * i
    dg = dh * (before - x if case["coupled"] else before) * slope
    if live is not None:
        dg = torch.where(live, dg, torch.zeros_like(dg))
        dx = torch.where(live, dx, torch.zeros_like(dx))
    return out + [dx.to(dtype), dg.to(dtype), f[:, :, 0] * dh[:, :, 0]]


def _plain_scan_step(st):
    case = st["case"]
    x, g = st["x"][:, :, 0].float(), st["g"][:, :, 0].float()
    f, i = _gate(case, g)
    slots = st["slots"].long()
    h = f * st["h_in"][slots] + (i * x if case["coupled"] else x)
    st["h_out"][slots] = h
    return [h[:, :, None].to(st["x"].dtype), st["h_out"]]


def _plain_norm(st):
    case = st["case"]
    B, H, N, d = st["x"].shape
    C = H * d
    rt = _DT[case["r_dtype"]]
    s = st["x"].float().permute(0, 2, 1, 3).reshape(B, N, C)
    if st["r"] is not None:
        s = s + st["r"].float()
    s = s.to(rt)
    # The norm is of the sum as the residual stream stores it.
    v = s.double() if case["op"] == "norm_e4m3" else s.float()
    rstd = 1.0 / torch.sqrt((v * v).sum(-1, keepdim=True) / C + st["eps"])
    u = v * rstd
    y = u * st["w"]
    if case["op"] == "norm_e4m3":
        # In 64 bits: values next to a border between two codes.
        parts = y.view(B, N, -1, case["group"] or C)
        scale = parts.abs().amax(-1) / _E4M3_MAX
        q = (parts / scale[..., None]).view(B, N, C).float().to(torch.float8_e4m3fn)
        return [s, q, scale.float()]
    out = [s, y.to(_DT[case["y_dtype"]])]
    if case["op"] == "norm_forward":
        return out
    dy = st["dy"].float()
    wdy = dy * st["w"]
    dr = rstd * (wdy - u * ((wdy * u).sum(-1, keepdim=True) / C))
    if st["ds"] is not None:
        dr = dr + st["ds"].float()
    dx = dr.view(B, N, H, d).permute(0, 2, 1, 3).contiguous()
    return out + [dr.to(rt), dx.to(st["x"].dtype), (dy * u).sum((0, 1))]


# ---- the definition in 64 bits, token by token

def exact(case, seed):
    st = _make(case, seed)
    if case["op"] == "scan_step":
        return _exact_step(st)
    return _exact_scan(st) if case["op"].startswith("scan") else _exact_norm(st)


def _exact_gate(case, g):
    if case["gate"] == "log":
        return torch.exp(g.clamp(max=0.0)), -torch.expm1(g.clamp(max=0.0))
    return torch.sigmoid(g), torch.sigmoid(-g)


def _exact_scan(st):
    case = st["case"]
    B, H, N, d = st["x"].shape
    lens = torch.tensor(_lengths(case), device="cuda")
    live = (torch.arange(N, device="cuda")[:, None] < lens).view(N, B, 1, 1)
    x = st["x"].double().permute(2, 0, 1, 3).contiguous().masked_fill_(~live, 0.0)
    g = st["g"].double().permute(2, 0, 1, 3).contiguous()
    f, q = _exact_gate(case, g)
    slope = f * q if case["gate"] == "sigmoid" else f.masked_fill(g > 0, 0.0)
    slope.masked_fill_(~live, 0.0)
    i = q if case["coupled"] else torch.ones_like(f)
    f.masked_fill_(~live, 1.0)
    i.masked_fill_(~live, 0.0)
    del g, q
    u = i * x
    h = torch.empty_like(u)
    zero = torch.zeros(B, H, d, dtype=torch.float64, device="cuda")
    first = st["h0"].double() if st["h0"] is not None else zero
    prev = first
    for n in range(N):
        prev = torch.addcmul(u[n], f[n], prev, out=h[n])
    del u

    def heads(t):
        return t.permute(1, 2, 0, 3).contiguous()

    out = [heads(h.masked_fill(~live, 0.0)), h[-1].clone()]
    if case["op"] == "scan_forward":
        return out
    dy = st["dy"].double().permute(2, 0, 1, 3).contiguous().masked_fill_(~live, 0.0)
    dh = torch.empty_like(dy)
    back = st["dhN"].double() if st["dhN"] is not None else zero
    for n in range(N - 1, -1, -1):
        torch.add(dy[n], back, out=dh[n])
        back = f[n] * dh[n]
    del dy
    h = torch.cat([first[None], h[:-1]])
    if case["coupled"]:
        h -= x
    return out + [heads(dh * i), heads(dh * h * slope), back]


def _exact_step(st):
    case = st["case"]
    x, g = st["x"][:, :, 0].double(), st["g"][:, :, 0].double()
    f, q = _exact_gate(case, g)
    slots = st["slots"].long()
    h = f * st["h_in"].double()[slots] + (q * x if case["coupled"] else x)
    pool = st["h_out"].double()
    pool[slots] = h
    return [h[:, :, None], pool]


def _e4m3(v):
    """The nearest e4m3 value (ties to the even code): 3 bits of fraction, exponents from -6, at most 448."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-_E4M3_MAX, _E4M3_MAX)


def _exact_norm(st):
    case = st["case"]
    B, H, N, d = st["x"].shape
    C = H * d
    s = torch.cat(list(st["x"].double().unbind(1)), dim=-1)
    if st["r"] is not None:
        s = s + st["r"].double()
    s = s.to(_DT[case["r_dtype"]]).double()
    rms = torch.sqrt(s.square().mean(-1, keepdim=True) + st["eps"])
    u = s / rms
    w = st["w"].double()
    if case["op"] == "norm_e4m3":
        G = case["group"] or C
        y = (u * w).reshape(B, N, C // G, G)
        top = y.abs().amax(-1, keepdim=True)
        return [s, _e4m3(y * (_E4M3_MAX / top)).reshape(B, N, C), (top / _E4M3_MAX).squeeze(-1)]
    out = [s, u * w]
    if case["op"] == "norm_forward":
        return out
    dy = st["dy"].double()
    du = dy * w
    dr = (du - u * (du * u).mean(-1, keepdim=True)) / rms
    if st["ds"] is not None:
        dr = dr + st["ds"].double()
    dx = torch.stack(dr.split(d, dim=-1), dim=1)
    return out + [dr, dx, (dy * u).sum((0, 1))]


def work(case):
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    size = {"f32": 4, "bf16": 2, "e4m3": 1}
    if case["op"].startswith("scan"):
        e, cols = size[case["dtype"]], B * H * d
        n = B * H * N * d
        live = sum(_lengths(case)) * H * d if case["op"] != "scan_step" else n
        state = cols * 4 * (2 if case["op"] == "scan_step" or case["state"] else 1)
        # forward: x and g in, y out; backward: x, g and dy in, dx and dg out
        nbytes, flops = (2 * live + n) * e + state, 8 * live
        if case["op"] == "scan_train":
            nbytes, flops = nbytes + (3 * live + 2 * n) * e + state, flops + 16 * live
        return {"bytes": nbytes, "flops": flops}
    n = B * N * H * d
    x, r, y = size[case["x_dtype"]], size[case["r_dtype"]], size[case["y_dtype"]]
    res = r if case["residual"] else 0
    nbytes, flops = n * (x + res + r + y) + 4 * H * d, 5 * n
    if case["op"] == "norm_e4m3":
        nbytes, flops = nbytes + 4 * n // (case["group"] or H * d), flops + 3 * n
    if case["op"] == "norm_train":
        # backward: dy, s and ds in, the stream's and the branch's gradients out, and dw
        nbytes, flops = nbytes + n * (y + r + res + r + x) + 8 * H * d, flops + 10 * n
    return {"bytes": nbytes, "flops": flops}
