"""The layer operators called from several threads at once, each on a stream of its own, and
captured graphs of them replayed beside one another: the same bits as one call alone."""
import threading

import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import test_gpu_layers as heads  # noqa: E402
import test_gpu_linear as base  # noqa: E402


@pytest.fixture(autouse=True)
def quiet(cuda_device):
    nsg.build()
    torch.cuda.set_device(0)
    yield
    assert nsg.device_error() == 0


def program(T, K, N):
    """A layer and its way back, odd rows (copied first) or even ones, and heads cut from its result."""
    x, w, dout = base.normal(T, (T, K)), base.normal(T + 1, (N, K), 0.03), base.normal(T + 2, (T, N), 0.1)
    bias, pre, rng = base.normal(T + 3, (N,)), base.normal(T + 4, (T, K)), base.generator(T, 1)
    freq, axis = nsg.rotary_frequencies(64)
    pos = heads.positions_of(T, T, 1, gone=0.1)

    def run():
        accum = torch.zeros(N * K + N + 64, device="cuda")
        y, u = nsg.linear(x, w, bias, "gelu", dropout=0.2, rng=rng, site=3, pre=True)
        dx = nsg.linear_grad(accum, dout, x, w, (0, N, K), (N * K, 1, N), activation="silu", pre=pre)
        q = y[:, :N // 64 * 64].reshape(T, -1, 64)
        a = nsg.norm_rotary(q, None, pos, freq, axis)[0]
        b = nsg.norm_rotary_grad(a, q, positions=pos, inv_freq=freq, axis=axis, accum=accum, q_param=(N * K + N, 1, 64))[0]
        return y, u, dx, a, b, nsg.dropout(y, 0.5, rng, 4), accum

    return run


SIZES = [(3, 768, 512), (333, 1001, 576), (700, 520, 320), (2100, 264, 192)]


def test_threads():
    programs = [program(*s) for s in SIZES]
    want = [p() for p in programs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(25):
                    if not all(torch.equal(a, b) for a, b in zip(programs[i](), want[i])):
                        bad.append(i)
        except Exception as e:   # into the test's own thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(programs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_graphs_beside_one_another():
    programs = [program(*s) for s in SIZES]
    want = [p() for p in programs]
    graphs, held, streams = [], [], [torch.cuda.Stream() for _ in programs]
    for p in programs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(p())
        graphs.append(g)
    for _ in range(20):
        for out in held:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out, w in zip(held, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))
