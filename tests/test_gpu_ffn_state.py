"""FeedForward's forward() and backward() taking turns, on the GPU: what is
refused, and what comes out after a refusal or a replay. Bounds as in
test_gpu_ffn_run.py."""
import pytest

from lossless_bf16_weight_afx_amd import afx
from test_gpu_ffn_run import Block, near

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


def test_a_second_backward_is_refused_and_a_new_forward_renews_it():
    t = Block(12, 24)
    r, dro, dxo = t.values(24, 1.5), t.values(24), t.values(24)
    want = t.formula(r, dro, dxo)[2]
    for _ in range(2):
        t.ffn.forward(r)
        near("dr", t.ffn.backward(r, dro, dxo), want[0], 10)
        with pytest.raises(ValueError):
            t.ffn.backward(r, dro, dxo)
    with pytest.raises(ValueError):
        t.ffn.forward(t.ffn.r_out)


def test_captured_forward_and_eager_backward():
    """A captured forward pass, replayed before each backward()."""
    t = Block(13, 10)
    r, dro = t.values(10), t.values(10)
    t.ffn.forward(r)
    t.ffn.backward(r, dro)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.ffn.forward(r)
    for _ in range(3):
        r.copy_(t.values(10))
        dro.copy_(t.values(10))
        graph.replay()
        dr = t.ffn.backward(r, dro)
        torch.cuda.synchronize()
        near("dr", dr, t.formula(r, dro)[2][0], 10)
