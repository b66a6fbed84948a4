"""ffn.FeedForward's own part (buffers, checks, order of calls) on the CPU:
the library's calls that would run on the GPU are recorded instead."""
import pytest

from lossless_bf16_weight_afx_amd import afx, ffn

torch = pytest.importorskip("torch")


def info(rows, cols):
    i = afx.afx_info()
    i.n_elems, i.ndim = rows * cols, 2
    i.shape[0], i.shape[1] = rows, cols
    return i


def matrices(d, ff):
    blob = torch.zeros(16, dtype=torch.uint8)
    return [(info(ff, d), blob), (info(ff, d), blob), (info(d, ff), blob)]


def block(d, ff, max_tokens, training=False, **kw):
    return ffn.FeedForward(*matrices(d, ff), d, ff, torch.ones(d, dtype=torch.bfloat16), max_tokens=max_tokens,
                           training=training, **kw)


@pytest.mark.parametrize("training", [False, True])
@pytest.mark.parametrize("d,ff,max_tokens", [(768, 1024, 641), (768, 14336, 700), (1024, 1536, 321), (2048, 768, 500),
                                             (1024, 2816, 1024), (256, 512, 700), (64, 256, 3), (128, 8192, 70),
                                             (5120, 17408, 450), (320, 2560, 1300)])
def test_workspace_holds_every_token_count(d, ff, max_tokens, training):
    t = block(d, ff, max_tokens, training)
    need = 0
    for m in range(1, max_tokens + 1):
        need = max(need, afx.afx_restore_gated_workspace(ff, d, m))
        if training:
            need = max(need, afx.afx_restore_gated_workspace(ff, d, m, True),
                       afx.afx_restore_gemm_t_workspace(d, ff, m), afx.afx_block_norm_workspace(t.norm_in, m),
                       afx.afx_block_norm_workspace(t.norm_out, m))
    assert t.ws.numel() == max(need, 16)
