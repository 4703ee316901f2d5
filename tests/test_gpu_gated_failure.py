"""The gated calls' bounded waits, made to run out on the host's request (no GPU fault): a hand-off that
never comes.  The call ends by itself with OWQ_ERR_TIMEOUT, writes nothing outside its outputs and its
workspace, and the next call gives the same bits as before."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import gated_ref as ref  # noqa: E402

DEV = torch.device("cuda", 0)
WAIT_CYCLES = 2_000_000   # about 1 ms
OWQ_ERR_TIMEOUT = 8
GUARD = 4096


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).half().to(DEV)


_LAYERS = {}


def pair(owq, N, K, bits, group, kg, ku):
    key = (N, K, bits, group, kg, ku)
    if key not in _LAYERS:
        _LAYERS.clear()
        ps = [ref.draw_layer(N, K, bits, group, k, 5 + k + 9 * l, DEV) for l, k in enumerate((kg, ku))]
        _LAYERS[key] = [owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], bits, group) for p in ps]
    return _LAYERS[key]


class Calls:
    """The C calls with every output and a workspace of exactly owq_gated_workspace bytes, each followed
    by guard bytes."""

    def __init__(self, owq, layers, M):
        self.owq, self.M = owq, M
        self.g, self.u = (l.handle for l in layers)
        self.N, self.K = layers[0].N, layers[0].K
        self.x, self.dh = rand(1, M, self.K), rand(2, M, self.N, scale=0.1)
        self.dg, self.du = rand(3, M, self.N, scale=0.1), rand(4, M, self.N, scale=0.1)
        st, n = owq.owq_gated_workspace(self.g, self.u, M)
        assert st == 0
        self.n_ws = n
        self.buf = {"ws": n, "h": 2 * M * self.N, "g": 2 * M * self.N, "u": 2 * M * self.N, "dx": 2 * M * self.K}
        self.raw = {k: torch.full((v + GUARD,), 0x5A, dtype=torch.uint8, device=DEV) for k, v in self.buf.items()}

    def at(self, name):
        return self.raw[name].data_ptr()

    def run(self, call):
        o, a, M, ws = self.owq, self.at, self.M, self.at("ws")
        return {
            "gemv": lambda: o.owq_gated_gemv(self.g, self.u, 0, self.x, a("h"), M),
            "gemm": lambda: o.owq_gated_gemm(self.g, self.u, 0, self.x, a("h"), M, ws, self.n_ws),
            "grad": lambda: o.owq_gated_grad(self.g, self.u, 0, self.x, self.dh, a("g"), a("u"), M, ws, self.n_ws),
            "input_grad": lambda: o.owq_gated_input_grad(self.g, self.u, self.dg, self.du, a("dx"), M, ws, self.n_ws),
            "backward": lambda: o.owq_gated_backward(self.g, self.u, 0, self.x, self.dh, a("g"), a("u"), a("dx"), M, ws, self.n_ws),
        }[call]()

    OUTS = {"gemv": ("h",), "gemm": ("h",), "grad": ("g", "u"), "input_grad": ("dx",), "backward": ("g", "u", "dx")}

    def outputs(self, call):
        return [self.raw[k][:self.buf[k]].clone() for k in self.OUTS[call]]

    def guards_hold(self):
        torch.cuda.synchronize()
        return all(bool((self.raw[k][v:] == 0x5A).all()) for k, v in self.buf.items())


# one launch's tiles without and with a K split; long rows (a cluster's CTAs share them in the decode form);
# odd N (padded gradients); several tiles a pair with a split tail behind them
SHAPES = [((512, 512, 3, 512, 4, 4), 16), ((137, 16384, 4, 128, 100, 0), 13), ((9601, 640, 4, 128, 0, 3), 70),
          ((11008, 1024, 3, 128, 8, 8), 64), ((1001, 256, 4, 256, 5, 5), 600)]
CALLS = [(s, M, c) for s, M in SHAPES for c in Calls.OUTS if c != "gemv" or M <= 16]


@pytest.mark.parametrize("shape,M,call", CALLS, ids=lambda v: str(v))
def test_lost_hand_off_times_out_then_recovers(shape, M, call):
    import weight_only_mixed_owq_b200 as owq
    c = Calls(owq, pair(owq, *shape), M)
    assert c.run(call) == 0
    assert owq.owq_device_status() == 0 and c.guards_hold()
    want = c.outputs(call)
    assert owq.owq_debug_inject(owq.OWQ_INJECT_GATED, WAIT_CYCLES) == 0
    assert c.run(call) == 0
    assert owq.owq_device_status() == OWQ_ERR_TIMEOUT
    assert c.guards_hold()
    for _ in range(2):
        assert c.run(call) == 0
        assert owq.owq_device_status() == 0 and c.guards_hold()
        assert all(torch.equal(p, q) for p, q in zip(want, c.outputs(call)))


def test_the_workspace_is_no_larger_than_needed_and_checked():
    """One byte less than the most that a call of these needs is refused by that call; nothing runs."""
    import weight_only_mixed_owq_b200 as owq
    for shape, M in SHAPES:
        c = Calls(owq, pair(owq, *shape), M)
        full, refused = c.n_ws, 0
        c.n_ws = full - 256   # (sizes are multiples of 256)
        for call in ("grad", "gemm", "input_grad", "backward"):
            before = c.outputs(call)
            st = c.run(call)
            assert st in (0, 9)
            if st == 9:
                refused += 1
                torch.cuda.synchronize()
                assert all(torch.equal(p, q) for p, q in zip(before, c.outputs(call)))
        assert refused >= 1 and c.guards_hold()
    assert owq.owq_device_status() == 0


def test_backward_refusals():
    """owq_gated_backward's own checks, each before anything runs."""
    import weight_only_mixed_owq_b200 as owq
    layers = pair(owq, 37, 256, 4, 128, 5, 19)
    c = Calls(owq, layers, 16)
    g, u, n = c.g, c.u, c.n_ws
    good = dict(act=0, x=c.x.data_ptr(), dh=c.dh.data_ptr(), dg=c.at("g"), du=c.at("u"), dx=c.at("dx"), M=16, ws=c.at("ws"), n=n)

    def call(gate=g, up=u, **kw):
        a = {**good, **kw}
        return owq.owq_gated_backward(gate, up, a["act"], a["x"], a["dh"], a["dg"], a["du"], a["dx"], a["M"], a["ws"], a["n"])
    assert call(gate=None) == 10 and call(up=0x10000) == 10
    for act in (-1, 3):
        assert call(act=act) == 12
    for M in (0, -1, 65537):
        assert call(M=M) == 2
    for name in ("x", "dh", "dg", "du", "dx", "ws"):
        assert call(**{name: None}) == 1 and call(**{name: good[name] + 8}) == 6
    assert call(n=0) == 9 and call(n=255) == 9
    torch.cuda.synchronize()
    assert all(bool((t == 0x5A).all()) for t in c.raw.values())
    assert call() == 0 and owq.owq_device_status() == 0
