"""GPU parity of the lapmix operators (through the binding) against the float64 oracle.

Tolerances: an output may lie off the oracle's value by the oracle's bound on float32
evaluation (see oracle/lapmix_oracle.py) plus half a step of the type it is rounded to,
2^-8 of the value for bf16 and 2^-24 for float32."""

import sys

import numpy as np
import pytest

from gpu_harness import gpu_available, torch_mod
from oracle import lapmix_oracle as O

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="no GPU device visible")]

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _torch_type(dtype):
    torch = torch_mod()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[dtype]


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rand(shape, seed, dtype="f32"):
    """A seeded normal tensor on the GPU and its exact float64 values."""
    torch = torch_mod()
    a = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    t = torch.from_numpy(a).to(_torch_type(dtype))
    return t.cuda(), _np(t)


def _place(t, layout, fill=None):
    """A [B, H, N, d] tensor's values in another memory layout (``fill``: values of a new one)."""
    torch = torch_mod()
    B, H, N, d = t.shape
    if layout == "heads":
        out = torch.empty(B, H, N, d, dtype=t.dtype, device="cuda")
    elif layout == "tokens":
        out = torch.empty(B, N, H, d, dtype=t.dtype, device="cuda").permute(0, 2, 1, 3)
    elif layout == "padded":  # rows of an odd pitch, not 16-byte aligned
        out = torch.empty(B, H, N, d + 3, dtype=t.dtype, device="cuda")[..., 1:d + 1]
    elif layout == "wide":  # aligned rows with a gap behind each
        out = torch.empty(B, H, N, d + 16, dtype=t.dtype, device="cuda")[..., :d]
    else:
        raise ValueError(layout)
    return out.copy_(t) if fill is None else out.fill_(fill)


def _check(name, got, want, bound, half):
    """|got - want| <= bound + half |want| element by element (with the bound's own rounding)."""
    err = np.abs(got - want)
    tol = bound * (1 + half) + half * np.abs(want) + 1e-38
    bad = ~(err <= tol)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.3g} of the tolerance at "
                           f"{np.unravel_index(np.nanargmax(err / tol), err.shape)}")
    return float(np.max(err / tol)) if err.size else 0.0


class Scan:
    """Inputs of one recurrence case, and the calls on them."""

    def __init__(self, B, H, N, d, dtype="f32", gate="sigmoid", coupled=False, layout="heads", lengths=None,
                 state=True, seed=1, bias=2.0):
        torch = torch_mod()
        import laplacian_nystr_approximation_amd as L
        self.L, self.dtype, self.shape, self.layout = L, dtype, (B, H, N, d), layout
        self.kw = dict(log_gate=gate == "log", coupled=coupled)
        self.p = L.make_scan_params(B=B, H=H, N=N, d=d, dtype=dtype, gate=gate, coupled=coupled)
        tt = _torch_type(dtype)
        x, _ = _rand((B, H, N, d), seed, dtype)
        g = np.random.default_rng(seed + 1).standard_normal((B, H, N, d)) * 1.5 + bias
        if gate == "log":
            g = -np.log1p(np.exp(-g))
            g.reshape(-1)[::17] *= -1  # some above 0, which count as 0
        g = torch.from_numpy(g.astype(np.float32)).to(tt).cuda()
        dy, _ = _rand((B, H, N, d), seed + 2, dtype)
        self.h0 = _rand((B, H, d), seed + 3)[0] if state else None
        self.dhN = _rand((B, H, d), seed + 4)[0] if state else None
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.lens = lengths
        if lengths is not None:  # nothing behind a sequence's end is read
            for b, n in enumerate(np.clip(lengths, 0, N)):
                for t, v in ((x, float("nan")), (g, float("nan")), (dy, float("inf"))):
                    t[b, :, n:] = v
        self.x, self.g, self.dy = (_place(t, layout) for t in (x, g, dy))
        # Workspaces and outputs start as garbage.
        self.ws = torch.full((max(256, L.lapmix_scan_workspace_size(self.p)),), 0xA5, dtype=torch.uint8, device="cuda")
        self.states = torch.full((L.lapmix_scan_states_size(self.p) // 4,), float("nan"), device="cuda")
        self.y, self.dx, self.dg = (_place(x, layout, float("nan")) for _ in range(3))
        self.hN, self.dh0 = (torch.full((B, H, d), float("nan"), device="cuda") for _ in range(2))

    def forward(self, **kw):
        self.L.lapmix_scan_forward_ws(self.x, self.g, self.y, self.p, self.ws, h0=self.h0, hN=self.hN,
                                      states=self.states, lengths=self.lengths, **kw)

    def backward(self, **kw):
        self.L.lapmix_scan_backward_ws(self.x, self.g, self.states, self.dy, self.dx, self.dg, self.p, self.ws,
                                       dhN=self.dhN, dh0=self.dh0, lengths=self.lengths, **kw)

    def outputs(self):
        return [self.y, self.hN, self.dx, self.dg, self.dh0]

    def want(self, heads=None):
        def np_of(t):
            return None if t is None else _np(t)
        x, g, dy = _np(self.x), _np(self.g), _np(self.dy)
        h0, dhN = np_of(self.h0), np_of(self.dhN)
        f = O.scan(x, g, h0, self.lens, **self.kw)
        f.update(O.scan_backward(x, g, dy, h0, dhN, self.lens, **self.kw))
        return f

    def check(self):
        torch_mod().cuda.synchronize()
        w, half = self.want(), HALF[self.dtype]
        worst = {}
        for name, t, h in (("y", self.y, half), ("hN", self.hN, HALF["f32"]), ("dx", self.dx, half),
                           ("dg", self.dg, half), ("dh0", self.dh0, HALF["f32"])):
            worst[name] = round(_check(name, _np(t), w[name], w["e_" + name], h), 3)
        # The kept states are the tiles' first h_{t-1}.
        B, H, N, d = self.shape
        T = self.L.LAPMIX_SCAN_TILE
        st = _np(self.states).reshape(B, H, -1, d)
        first = np.zeros((B, H, 1, d)) if self.h0 is None else _np(self.h0)[:, :, None]
        before = np.concatenate([first, w["h"][:, :, T - 1:N - 1:T]], axis=2)
        e = np.concatenate([np.zeros((B, H, 1, d)), w["e_h"][:, :, T - 1:N - 1:T]], axis=2)
        _check("states", st, before, e, HALF["f32"])
        _say(f"[scan] {self.shape} {self.dtype} {self.layout} worst/tolerance {worst}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate,coupled", [("sigmoid", False), ("sigmoid", True), ("log", False), ("log", True)])
def test_scan_gates(dtype, gate, coupled):
    c = Scan(2, 3, 300, 64, dtype, gate, coupled)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1025, 4096, 4099])
def test_scan_lengths_of_time(N, dtype):
    """Around the tile's edges, few columns (long ones are split over the chip)."""
    c = Scan(1, 2, N, 64, dtype, coupled=True, bias=4.0)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("B,H,N,d", [(1, 1, 300, 1), (3, 5, 70, 7), (2, 3, 260, 8), (1, 7, 515, 33), (2, 1, 300, 40),
                                     (1, 3, 600, 72), (5, 1, 33, 130), (1, 1, 1, 1), (40, 5, 300, 64), (2, 1, 600, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_widths(B, H, N, d, dtype):
    c = Scan(B, H, N, d, dtype, gate="log", coupled=True)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("layout", ["tokens", "padded", "wide"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_layouts(layout, dtype):
    c = Scan(2, 3, 700, 48, dtype, layout=layout, coupled=True)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d", [(600, 64), (5000, 24), (300, 5)])
def test_scan_padded_batches(dtype, N, d):
    """Lengths of zero, one, beyond N and below zero; NaN and infinities behind the ends."""
    c = Scan(6, 2, N, d, dtype, lengths=[N, 0, 1, N + 5, -3, N // 2], coupled=True)
    c.forward()
    c.backward()
    c.check()


def test_scan_all_sequences_empty():
    c = Scan(2, 1, 600, 32, "bf16", lengths=[0, 0])
    c.forward()
    c.backward()
    c.check()
    torch = torch_mod()
    assert torch.equal(c.hN, c.h0) and torch.equal(c.dh0, c.dhN)
    assert not c.y.any() and not c.dx.any() and not c.dg.any()


def test_scan_without_states_and_lengths():
    c = Scan(2, 2, 1300, 64, "bf16", state=False)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("N", [40, 6000])
def test_scan_resets_and_extreme_gates(N):
    """Gates of -inf start anew, gates of +inf keep everything, float32's extremes stay finite."""
    for gate in ("sigmoid", "log"):
        c = Scan(1, 2, N, 64, "f32", gate)
        c.g[:, :, 5::11] = -float("inf")
        c.g[:, :, 6::13] = float("inf") if gate == "sigmoid" else 0.0
        c.g[:, :, 7::17] = -1e30
        c.g[:, :, 8::19] = 1e30 if gate == "sigmoid" else -1e-30
        c.forward()
        c.backward()
        c.check()


def test_scan_remembers_over_the_whole_sequence():
    """Gates of 1: the state is a plain sum over 20000 tokens, and the gradients are sums too."""
    c = Scan(1, 1, 20000, 64, "f32", "log")
    c.g.zero_()
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("N", [5000, 70000, 700001, 8500007])
def test_scan_counts_exactly_over_long_sequences(N):
    """Gates of 1 and 0 and whole inputs: states are counts since the last reset, exact in float32, and
    so are the gradients; 700001 tokens take pairs of four levels (4096 tiles are 524288 tokens), 8500007 of five."""
    torch = torch_mod()
    d = 4
    gen = torch.Generator().manual_seed(N)
    for resets in (0, 97, 30011):
        x = torch.randint(-2, 3, (1, 1, N, d), generator=gen).float().cuda()
        dy = torch.randint(-2, 3, (1, 1, N, d), generator=gen).float().cuda()
        c = Scan(1, 1, N, d, "f32", "log", state=False)
        c.x, c.dy = x, dy
        c.g = torch.zeros_like(x)
        if resets:
            c.g[:, :, resets::resets] = -float("inf")
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        total = x.double().cumsum(2)
        back = dy.double().flip(2).cumsum(2).flip(2)
        if resets:
            n = torch.arange(N, device="cuda")
            first = n // resets * resets  # the run's first token
            before = torch.where(first > 0, first - 1, 0)
            total = total - torch.where(first[:, None] > 0, total[0, 0, before], 0.0)
            after = first + resets  # the next run's
            back = back - torch.where(after[:, None] < N, back[0, 0, after.clamp(max=N - 1)], 0.0)
        assert torch.equal(c.y.double(), total) and torch.equal(c.hN.double(), total[:, :, -1])
        assert torch.equal(c.dx.double(), back) and torch.equal(c.dh0.double()[0, 0], back[0, 0, 0])
        hp = torch.cat([torch.zeros_like(total[:, :, :1]), total[:, :, :-1]], 2)
        want = torch.where(c.g == 0, back * hp, torch.zeros_like(hp))
        assert torch.equal(c.dg, want.float())


def test_scan_nan_stays_in_its_column():
    torch = torch_mod()
    c = Scan(1, 2, 3000, 64, "f32")
    clean = Scan(1, 2, 3000, 64, "f32")
    clean.forward()
    clean.backward()
    c.x[0, 0, 100, 3] = float("nan")
    c.g[0, 1, 1500, 9] = float("nan")
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    for t, u in zip(c.outputs(), clean.outputs()):
        hit = torch.zeros_like(t, dtype=torch.bool)
        hit[0, 0, ..., 3] = True
        hit[0, 1, ..., 9] = True
        assert torch.equal(t[~hit], u[~hit])
    assert c.y[0, 0, 100:, 3].isnan().all() and not c.y[0, 0, :100, 3].isnan().any()
    assert c.y[0, 1, 1500:, 9].isnan().all() and c.hN[0, 1, 9].isnan()
    assert c.dh0[0, 1, 9].isnan() and not c.dh0[0, 0].isnan().any()


@pytest.mark.parametrize("B,H,N,d", [(1, 2, 30000, 64), (64, 8, 600, 64), (1, 1, 9000, 5)])
def test_scan_repeats_bit_for_bit(B, H, N, d):
    """The same inputs give the same bits, on a workspace that holds anything."""
    torch = torch_mod()
    c = Scan(B, H, N, d, "bf16")
    c.forward()
    c.backward()
    first = [t.clone() for t in c.outputs()]
    for fill in (0, 0xFF, 0x7F):
        c.ws.fill_(fill)
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        for t, u in zip(c.outputs(), first):
            assert torch.equal(t, u)


def test_scan_state_carries_over_in_place():
    """Two calls on the halves of a sequence, the state updated in place, are one call on it all; the
    backward the same from behind."""
    torch = torch_mod()
    c = Scan(2, 2, 5000, 64, "f32", coupled=True)
    c.forward()
    c.backward()
    cut = 2304
    h = c.h0.clone()
    parts = []
    for a, b in ((0, cut), (cut, 5000)):
        p = c.L.make_scan_params(B=2, H=2, N=b - a, d=64, coupled=True)
        ws = torch.empty(max(256, c.L.lapmix_scan_workspace_size(p)), dtype=torch.uint8, device="cuda")
        y = torch.empty(2, 2, b - a, 64, device="cuda")
        st = torch.empty(c.L.lapmix_scan_states_size(p) // 4, device="cuda")
        c.L.lapmix_scan_forward_ws(c.x[:, :, a:b], c.g[:, :, a:b], y, p, ws, h0=h, hN=h, states=st)
        parts.append((a, b, p, ws, st, y))
    w, half = c.want(), HALF["f32"]
    _check("hN", _np(h), w["hN"], w["e_hN"], half)
    r = c.dhN.clone()
    for a, b, p, ws, st, y in reversed(parts):
        _check("y", _np(y), w["y"][:, :, a:b], w["e_y"][:, :, a:b], half)
        dx, dg = c.x.new_empty(2, 2, b - a, 64), c.x.new_empty(2, 2, b - a, 64)
        xs, gs = c.x[:, :, a:b].contiguous(), c.g[:, :, a:b].contiguous()
        c.L.lapmix_scan_backward_ws(xs, gs, st, c.dy[:, :, a:b], dx, dg, p, ws, dhN=r, dh0=r)
        _check("dx", _np(dx), w["dx"][:, :, a:b], w["e_dx"][:, :, a:b], half)
        _check("dg", _np(dg), w["dg"][:, :, a:b], w["e_dg"][:, :, a:b], half)
    _check("dh0", _np(r), w["dh0"], w["e_dh0"], half)


def test_scan_packed_projection():
    """x and g, and their gradients, as the two parts of one [B, N, 2, H, d] buffer."""
    torch = torch_mod()
    B, H, N, d = 2, 3, 900, 32
    c = Scan(B, H, N, d, "bf16", coupled=True)
    both = torch.stack([c.x.permute(0, 2, 1, 3), c.g.permute(0, 2, 1, 3)], dim=2).contiguous()
    grads = torch.full_like(both, float("nan"))
    c.x, c.g = (both[:, :, i].permute(0, 2, 1, 3) for i in range(2))
    c.dx, c.dg = (grads[:, :, i].permute(0, 2, 1, 3) for i in range(2))
    c.forward()
    c.backward()
    c.check()


def test_scan_broadcast_inputs():
    """One gate for all heads (stride 0) in the forward; gradients of it are refused."""
    torch = torch_mod()
    c = Scan(2, 4, 600, 64, "bf16")
    c.g = c.g[:, :1].expand(2, 4, 600, 64)
    c.forward()
    w = c.want()
    _check("y", _np(c.y), w["y"], w["e_y"], HALF["bf16"])
    with pytest.raises(ValueError, match="dg: expected the strides"):
        c.backward()
    c.dg = c.dg[:, :1].expand(2, 4, 600, 64)
    with pytest.raises(c.L.LapnysError) as e:
        c.backward()
    assert e.value.code == -1
    torch.cuda.synchronize()


def test_scan_leaves_memory_around_its_outputs_alone():
    torch = torch_mod()
    B, H, N, d = 2, 2, 515, 24
    for dtype in ("f32", "bf16"):
        c = Scan(B, H, N, d, dtype, layout="tokens", lengths=[515, 300])
        bufs = []
        for name in ("y", "dx", "dg"):
            buf = torch.full((B, N + 9, H + 1, d + 8), 7.0, dtype=_torch_type(dtype), device="cuda")
            view = buf[:, 4:N + 4, :H, :d].permute(0, 2, 1, 3)
            if name != "y":
                src = torch.empty_like(buf)[:, 4:N + 4, :H, :d].permute(0, 2, 1, 3)
                src.copy_(getattr(c, name[1]))
                setattr(c, name[1], src)
            setattr(c, name, view)
            bufs.append(buf)
        c.dy = _place(c.dy, "tokens")
        keep, c.y = c.y, c.y
        c.forward()
        c.y = keep
        c.backward()
        c.check()
        for buf in bufs:
            inside = torch.zeros_like(buf, dtype=torch.bool)
            inside[:, 4:N + 4, :H, :d] = True
            assert (buf[~inside] == 7.0).all()


@pytest.mark.parametrize("what", ["scan", "norm"])
def test_captured_graphs_replay(what):
    """Forward and backward captured into a graph and replayed, with eager work and new inputs
    between the replays; each replay gives the eager call's bits."""
    torch = torch_mod()
    c = Scan(1, 2, 20000, 64, "bf16") if what == "scan" else Norm(70, 5, 64, "f32", "bf16", "bf16")
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward()
        c.backward()
    for seed in range(4):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        c.x.copy_(torch.randn(c.x.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in c.outputs()]
        for t in c.outputs():
            t.zero_()
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        for t, u in zip(c.outputs(), got):
            assert torch.equal(t, u)


def test_two_streams_at_once():
    """Calls on two streams, a workspace each, while the default stream is busy."""
    torch = torch_mod()
    cases = [Scan(1, 2, 20000, 64, "bf16", seed=s) for s in (1, 50)]
    want = []
    for c in cases:
        c.forward()
        c.backward()
        want.append([t.clone() for t in c.outputs()])
        for t in c.outputs():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for c, s in zip(cases, streams):
            c.forward(stream=s)
            c.backward(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        for t, u in zip(c.outputs(), w):
            assert torch.equal(t, u)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,d", [(1, 1, 1), (1, 8, 64), (5, 3, 33), (64, 5, 64), (300, 2, 20)])
def test_step(B, H, d, dtype):
    """Tokens one by one, on slots of a pool, follow the recurrence; padded places and other slots stay."""
    torch = torch_mod()
    c = Scan(B, H, 6, d, dtype, coupled=True, layout="tokens")
    w = c.want()
    n = 2 * B + 3
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32)
    slots = perm.clone()
    out = [] if B < 3 else [(1, -1), (2, n), (B - 1, 2 ** 31 - 1)][:B - 2]
    for b, v in out:
        slots[b] = v
    skip = [b for b, _ in out]
    pool = torch.full((n, H, d), 3.0, device="cuda")
    pool[perm.long().cuda()] = c.h0
    p = c.L.make_scan_params(B=B, H=H, N=1, d=d, dtype=dtype, coupled=True)
    dev = slots.cuda()
    for t in range(6):
        other = torch.full_like(pool, 5.0) if t % 2 else pool  # another pool or in place
        keep = pool.clone()
        y = torch.full((B, H, 1, d), 9.0, dtype=_torch_type(dtype), device="cuda")
        c.L.lapmix_scan_step(c.x[:, :, t:t + 1], c.g[:, :, t:t + 1], y, pool, other, p, slots=dev)
        torch.cuda.synchronize()
        live = [b for b in range(B) if b not in skip]
        rows = perm.long()[live].cuda()
        _check("y", _np(y[:, :, 0])[live], w["h"][live, :, t], w["e_h"][live, :, t], HALF[dtype])
        _check("state", _np(other[rows]), w["h"][live, :, t], w["e_h"][live, :, t], HALF["f32"])
        assert (y[skip] == 9.0).all()
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[rows] = False
        assert (other[rest] == (5.0 if t % 2 else keep[rest])).all()
        keep[rows] = other[rows]
        pool = keep


def test_step_without_slots_and_strided():
    torch = torch_mod()
    c = Scan(7, 3, 1, 48, "bf16", layout="padded")
    pool = torch.zeros(9, 3, 48, device="cuda")
    pool[:7] = c.h0
    c.L.lapmix_scan_step(c.x, c.g, c.y, pool, pool, c.p)
    torch.cuda.synchronize()
    w = c.want()
    _check("y", _np(c.y), w["y"], w["e_y"], HALF["bf16"])
    _check("state", _np(pool[:7]), w["hN"], w["e_hN"], HALF["f32"])
    assert not pool[7:].any()


def test_scan_offsets_beyond_32_bits():
    """Views whose last token lies more than 2^31 elements behind the first."""
    torch = torch_mod()
    N, pitch = 700, 3300000
    buf = torch.zeros(N * pitch, dtype=torch.bfloat16, device="cuda")
    c = Scan(1, 1, N, 64, "bf16")
    want = c.want()
    for at, name in ((0, "x"), (128, "g"), (256, "y"), (384, "dy"), (512, "dx"), (640, "dg")):
        v = buf.as_strided((1, 1, N, 64), (0, 0, pitch, 1), at)
        v.copy_(getattr(c, name))
        setattr(c, name, v)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    for name in ("y", "dx", "dg"):
        _check(name, _np(getattr(c, name)), want[name], want["e_" + name], HALF["bf16"])


# ---- norm

class Norm:
    def __init__(self, rows, H, d, x_dtype="f32", r_dtype="f32", y_dtype="f32", group=0, residual=True, B=1,
                 layout="heads", seed=5, eps=1e-5, shift=0):
        torch = torch_mod()
        import laplacian_nystr_approximation_amd as L
        assert rows % B == 0
        self.L, N, C = L, rows // B, H * d
        self.types, self.group, self.eps = (x_dtype, r_dtype, y_dtype), group, float(np.float32(eps))
        self.p = L.make_norm_params(B=B, H=H, N=N, d=d, x_dtype=x_dtype, r_dtype=r_dtype, y_dtype=y_dtype, eps=eps,
                                    group=group)
        self.x = _place(_rand((B, H, N, d), seed, x_dtype)[0], layout)

        def rows_like(dtype, values=None):  # `shift` elements off a 16-byte base
            t = torch.full((rows * C + shift,), float("nan"), device="cuda").to(_torch_type(dtype))[shift:]
            t = t.view(B, N, C)
            return t if values is None else t.copy_(values)

        wide = torch.where(torch.arange(C, device="cuda") % 37 == 5, 30.0, 1.0)
        self.r = rows_like(r_dtype, _rand((B, N, C), seed + 1)[0] * wide) if residual else None
        self.w = _rand((C,), seed + 2)[0] * 0.3 + 1.0
        self.s, self.dr = rows_like(r_dtype), rows_like(r_dtype)
        self.y = rows_like(y_dtype)
        self.scale = torch.full((B, N, C // (group or C)), float("nan"), device="cuda") if y_dtype == "e4m3" else None
        if y_dtype != "e4m3":
            self.dy = rows_like(y_dtype, _rand((B, N, C), seed + 3)[0])
            self.ds = rows_like(r_dtype, _rand((B, N, C), seed + 4)[0]) if residual else None
            self.dx = _place(self.x, layout, float("nan"))
            self.dw = torch.full((C,), float("nan"), device="cuda")
            self.ws = torch.full((L.lapmix_norm_workspace_size(self.p),), 0xFF, dtype=torch.uint8, device="cuda")

    def forward(self, **kw):
        self.L.lapmix_norm_forward(self.x, self.w, self.y, self.p, r=self.r, s=self.s, scale=self.scale, **kw)

    def backward(self, **kw):
        self.L.lapmix_norm_backward_ws(self.dy, self.s, self.w, self.p, self.ws, ds=self.ds, dr=self.dr, dx=self.dx,
                                       dw=self.dw, **kw)

    def outputs(self):
        return [self.s, self.y] + ([self.scale] if self.scale is not None else [self.dr, self.dx, self.dw])

    def flat(self, t):
        return _np(t).reshape(-1, t.shape[-1])

    def check_forward(self):
        torch = torch_mod()
        torch.cuda.synchronize()
        x_dtype, r_dtype, y_dtype = self.types
        # The stored sum is the float32 sum, rounded: the same bits.
        want = O.rows_of(_np(self.x)).astype(np.float32)
        if self.r is not None:
            want = want + self.flat(self.r).astype(np.float32)
        want = _np(torch.from_numpy(want).to(_torch_type(r_dtype)))
        s = self.flat(self.s)
        assert np.array_equal(s, want)
        w = _np(self.w)
        y, e = O.norm(s, w, self.eps)
        if y_dtype != "e4m3":
            return _check("y", self.flat(self.y), y, e, HALF[y_dtype])
        R, C = s.shape
        G = self.group or C
        top = np.maximum(np.abs(y).reshape(R, C // G, G).max(2), 2.0 ** -100)
        rel = U = 2.0 ** -24 * ((C / 64 + 16) / 2 + 12)  # y, the quotient by 448 and its rounding
        _check("scale", _np(self.scale).reshape(R, C // G), top / 448, top / 448 * rel, 0.0)
        sc = np.repeat(top / 448, G, axis=1)
        q, v = self.flat(self.y), y / sc
        # Within half a step of the code's value, where v itself is off by its float32 error.
        off = np.abs(q - v)
        assert np.all(off <= O.e4m3_half_step(np.abs(v) * (1 + 2 * U)) * (1 + 1e-9) + 2 * rel * np.abs(v))
        assert np.all(np.abs(q).reshape(R, C // G, G).max(2) <= 448)
        # In groups that are not all tiny the norm's factor cancels: the codes are those of
        # 448 s w / max|s w| in 64 bits (rounded to 32, then to e4m3), none on the other side of a border.
        z = (s * w).reshape(R, C // G, G)
        m = np.abs(z).max(2, keepdims=True)
        ok = np.broadcast_to(np.abs(y).reshape(R, C // G, G).max(2, keepdims=True) > 2.0 ** -99, z.shape)
        with np.errstate(divide="ignore", invalid="ignore"):
            want = np.where(ok, z * (448.0 / m), 0.0)
        want = _np(torch.from_numpy(want.astype(np.float32)).to(torch.float8_e4m3fn))
        assert np.array_equal(q.reshape(z.shape)[ok], want[ok])

    def check_backward(self):
        torch_mod().cuda.synchronize()
        x_dtype, r_dtype, y_dtype = self.types
        ds = None if self.ds is None else self.flat(self.ds)
        dr, dw, e, ew = O.norm_backward(self.flat(self.dy), self.flat(self.s), _np(self.w), self.eps, ds)
        _check("dr", self.flat(self.dr), dr, e, HALF[r_dtype])
        _check("dx", O.rows_of(_np(self.dx)), dr, e, HALF[x_dtype])
        _check("dw", _np(self.dw), dw, ew, HALF["f32"])


_TYPES = [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"), ("f32", "f32", "bf16"),
          ("bf16", "f32", "f32")]


@pytest.mark.parametrize("types", _TYPES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm_types(types, residual):
    c = Norm(37, 5, 64, *types, residual=residual)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("types", _TYPES[:3])
@pytest.mark.parametrize("rows,H,d", [(1, 1, 1), (3, 1, 7), (5, 1, 8), (9, 3, 5), (2, 2, 32), (4, 1, 511), (3, 1, 512),
                                      (3, 1, 520), (2, 1, 1000), (2, 1, 1024), (3, 1, 1032), (2, 1, 2047), (2, 1, 2048),
                                      (2, 1, 4100), (2, 1, 4096), (3, 2, 4096), (2, 1, 8200), (2, 1, 16383),
                                      (2, 1, 16384), (600, 1, 40), (1300, 1, 256), (5000, 1, 64)])
def test_norm_sizes(rows, H, d, types):
    c = Norm(rows, H, d, *types)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("layout", ["tokens", "padded", "wide"])
@pytest.mark.parametrize("types", _TYPES[:3])
def test_norm_layouts(layout, types):
    c = Norm(42, 3, 40, *types, layout=layout, B=3)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()


def test_norm_unaligned_rows():
    for types in _TYPES[:3]:
        c = Norm(6, 1, 256, *types, shift=1)
        c.forward()
        c.check_forward()
        c.backward()
        c.check_backward()


@pytest.mark.parametrize("r_dtype,x_dtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,H,d,group", [(1, 1, 16, 16), (5, 1, 64, 32), (7, 2, 64, 128), (3, 1, 4096, 128), (3, 1, 2048, 512),
                                            (4, 1, 1024, 256), (2, 1, 16384, 64), (5, 1, 100, 0), (3, 1, 1001, 0),
                                            (9, 1, 4096, 0), (2, 5, 64, 0), (600, 2, 32, 64), (2, 1, 5120, 512)])
def test_norm_e4m3(rows, H, d, group, r_dtype, x_dtype):
    c = Norm(rows, H, d, x_dtype, r_dtype, "e4m3", group)
    c.forward()
    c.check_forward()


@pytest.mark.parametrize("y_dtype,group", [("bf16", 0), ("e4m3", 0), ("e4m3", 16), ("e4m3", 128)])
@pytest.mark.parametrize("C", [128, 512, 4096])
def test_norm_rows_do_not_depend_on_their_neighbours(C, y_dtype, group):
    """A row gives the same bits among 600 others and alone: codes and scales of a group are decided by the
    group's values, whatever the rest of its wave holds."""
    torch = torch_mod()
    c = Norm(600, 1, C, "bf16", "bf16", y_dtype, group)
    c.forward()
    torch.cuda.synchronize()
    p = c.L.make_norm_params(B=1, H=1, N=1, d=C, x_dtype="bf16", r_dtype="bf16", y_dtype=y_dtype, eps=c.eps, group=group)
    for i in range(0, 600, 7):
        y, s = torch.empty_like(c.y[:, i]), torch.empty_like(c.s[:, i])
        scale = None if c.scale is None else torch.empty_like(c.scale[:, i])
        c.L.lapmix_norm_forward(c.x[:, :, i:i + 1], c.w, y, p, r=c.r[:, i], s=s, scale=scale)
        assert torch.equal(y.view(torch.uint8), c.y[:, i].contiguous().view(torch.uint8))
        assert scale is None or torch.equal(scale, c.scale[:, i])


def test_norm_rows_of_zeros_and_extremes():
    """A row of zeros, rows of tiny and of large values, and e4m3 of all of them."""
    torch = torch_mod()
    for y_dtype, group in (("f32", 0), ("e4m3", 0), ("e4m3", 64)):
        c = Norm(6, 2, 64, "f32", "f32", y_dtype, group, residual=False)
        c.x[0, :, 1] = 0.0
        c.x[0, :, 2] *= 1e-20
        c.x[0, :, 3] *= 1e15
        c.x[0, 0, 4] = 0.0  # a group of zeros beside one with values
        c.forward()
        c.check_forward()
        torch.cuda.synchronize()
        assert torch.isfinite(c.y.float()).all() and not c.y[0, 1].float().any()
        if y_dtype == "f32":
            c.backward()
            c.check_backward()


def test_norm_nan_and_infinity_stay_in_their_row():
    torch = torch_mod()
    for y_dtype in ("bf16", "e4m3"):
        c, clean = (Norm(6, 1, 512, "f32", "f32", y_dtype, residual=False) for _ in range(2))
        clean.forward()
        c.x[0, 0, 2, 77] = float("nan")
        c.x[0, 0, 4, 78] = float("inf")
        c.forward()
        torch.cuda.synchronize()
        for row in (0, 1, 3, 5):
            assert torch.equal(c.y[0, row].float(), clean.y[0, row].float())
        assert c.y[0, 2].float().isnan().any() and c.y[0, 4].float().isnan().any()


def test_norm_rows_beyond_a_launch():
    """More rows than one launch's 2^32 lanes take: 67117056 rows of 65 columns, one batch's x repeated
    (stride 0) 8193 times."""
    torch = torch_mod()
    import laplacian_nystr_approximation_amd as L
    B, N, C = 8193, 8192, 65
    x = torch.randn(1, 1, N, C, device="cuda").bfloat16().expand(B, 1, N, C)
    w = torch.randn(C, device="cuda")
    y = torch.zeros(B, N, C, dtype=torch.bfloat16, device="cuda")
    p = L.make_norm_params(B=B, H=1, N=N, d=C, x_dtype="bf16", r_dtype="bf16", y_dtype="bf16")
    L.lapmix_norm_forward(x, w, y, p)
    one = torch.zeros(1, N, C, dtype=torch.bfloat16, device="cuda")
    L.lapmix_norm_forward(x[:1], w, one, L.make_norm_params(B=1, H=1, N=N, d=C, x_dtype="bf16", r_dtype="bf16",
                                                            y_dtype="bf16"))
    torch.cuda.synchronize()
    assert one.any()
    for b in range(0, B, 512):
        assert (y[b:b + 512] == one).all()


def test_norm_in_place_and_optional_outputs():
    """s on top of r, dr on top of ds, and each output of the backward alone."""
    torch = torch_mod()
    for types in _TYPES[:3]:
        c = Norm(33, 2, 64, *types)
        c.forward()
        c.backward()
        want = [t.clone() for t in c.outputs()]
        r, ds = c.r.clone(), c.ds.clone()
        y2 = torch.empty_like(c.y)
        c.L.lapmix_norm_forward(c.x, c.w, y2, c.p, r=r, s=r)
        c.L.lapmix_norm_backward_ws(c.dy, c.s, c.w, c.p, c.ws, ds=ds, dr=ds)
        dx2, dw2 = torch.empty_like(c.dx), torch.empty_like(c.dw)
        c.L.lapmix_norm_backward_ws(c.dy, c.s, c.w, c.p, c.ws, ds=c.ds, dx=dx2)
        c.L.lapmix_norm_backward_ws(c.dy, c.s, c.w, c.p, c.ws, dw=dw2)
        y3 = torch.empty_like(c.y)
        c.L.lapmix_norm_forward(c.x, c.w, y3, c.p, r=c.r)
        torch.cuda.synchronize()
        for t, u in zip((r, y2, ds, dx2, dw2), want):
            assert torch.equal(t, u)
        assert torch.equal(y3, want[1])


def test_norm_repeats_bit_for_bit():
    torch = torch_mod()
    c = Norm(5000, 1, 320, "bf16", "bf16", "bf16")
    c.forward()
    c.backward()
    want = [t.clone() for t in c.outputs()]
    for _ in range(3):
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        for t, u in zip(c.outputs(), want):
            assert torch.equal(t, u)


def test_attention_norm_recurrence_run():
    """The operators as a block uses them: the attention's float32 heads join the residual and are
    normed, the normed rows drive a recurrence, whose output joins the residual, normed to e4m3."""
    torch = torch_mod()
    import laplacian_nystr_approximation_amd as L
    import oracle
    from gpu_harness import device_inputs, workload_inputs
    from lapnys_inputs import WORKLOADS
    w = WORKLOADS["stage3_14x14_bf16"].with_(B=2, name="mix_block")
    inp = workload_inputs(w)
    q, k, v = device_inputs(inp, w.dtype)
    att = torch.empty(w.B, w.H, w.N, w.d, device="cuda")
    pa = L.params_for(w)
    L.lapnys_forward_ws(q, k, v, att, pa, torch.empty(L.lapnys_workspace_size(pa), dtype=torch.uint8, device="cuda"))
    C = w.H * w.d
    rows = w.B * w.N
    n1 = Norm(rows, w.H, w.d, "f32", "bf16", "bf16", B=w.B)
    n1.x = att
    n1.forward()
    n1.check_forward()
    ref = oracle.attention_problem(inp.qf[0, 0], inp.kf[0, 0], inp.vf[0, 0], grid_h=w.grid_h, grid_w=w.grid_w,
                                   pool=w.pool, lam=float(np.float32(w.lam)), eps=float(np.float32(w.eps)),
                                   ns_iters=w.ns_iters)["O"]
    got = _np(att[0, 0])
    assert np.abs(got - ref).max() <= 1e-4 * np.abs(ref).max()
    # The normed rows, seen as heads, are the recurrence's input; its output is added to s.
    sc = Scan(w.B, w.H, w.N, w.d, "bf16", coupled=True, layout="tokens", state=False)
    sc.x = n1.y.view(w.B, w.N, w.H, w.d).permute(0, 2, 1, 3)
    sc.forward()
    sc.backward()
    sc.check()
    n2 = Norm(rows, w.H, w.d, "bf16", "bf16", "e4m3", 64, B=w.B, layout="tokens")
    n2.x, n2.r = sc.y, n1.s
    n2.forward()
    n2.check_forward()
    # Backward through the first norm: the gradient arrives in the attention's float32 heads.
    n1.dy = sc.dx.permute(0, 2, 1, 3).reshape(w.B, w.N, C).contiguous()
    n1.backward()
    n1.check_backward()
    dq, dk, dv = (torch.empty_like(att) for _ in range(3))
    L.lapnys_backward_ws(q, k, v, n1.dx, dq, dk, dv, pa,
                         torch.empty(L.lapnys_backward_workspace_size(pa), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in (dq, dk, dv))
