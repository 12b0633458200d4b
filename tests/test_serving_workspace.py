"""The attention call's default workspace: what is no tensor or number is refused as such, before one is sized."""
import pytest
import torch

import bit_weight_only_tq_amd as tq

I = torch.zeros(3, dtype=torch.int32)  # noqa: E741
H = torch.zeros((3, 1, 64), dtype=torch.float16)
C = torch.zeros((4, 1, 16, 64), dtype=torch.float16)
GOOD = dict(q=H, k_cache=C, v_cache=C, page_table=I.view(1, 3), cu_q=I[:2], kv_lens=I[:1], max_q=3, max_kv=40)
BAD = [dict(q=5), dict(q=None), dict(k_cache=None), dict(k_cache=[C]), dict(page_table=[[1, 2]]), dict(page_table=I),
       dict(page_table=torch.tensor(3, dtype=torch.int32)), dict(max_q="3"), dict(max_kv=4.5), dict(window=None), dict(sinks="x")]


def _refused(good, bad):
    with pytest.raises(TypeError):
        tq.tq_paged_attention(**dict(good, **bad))
    with pytest.raises(TypeError):
        tq.tq_paged_attention(**dict(good, workspace=None, **bad))


@pytest.mark.parametrize("bad", BAD)
def test_refused_on_the_host(bad):
    _refused(GOOD, bad)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", BAD)
def test_refused_with_device_tensors(bad):
    from gpu_common import require_gpu
    dev = require_gpu()
    _refused({k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in GOOD.items()}, bad)


@pytest.mark.gpu
def test_numbers_past_64_bits_with_device_tensors():
    from gpu_common import require_gpu
    dev = require_gpu()
    good = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in GOOD.items()}
    for name in ("max_q", "max_kv", "window", "sinks"):
        with pytest.raises(ValueError, match="64 bits"):
            tq.tq_paged_attention(**dict(good, **{name: 1 << 70}))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_default_is_the_library_s_own_size(dt):
    """The default gives the same bits as a workspace of the bytes that the library asks for, call after call, captured too."""
    from gpu_common import require_gpu
    from test_gpu_11_attention import Case
    dev = require_gpu()
    c = Case([1, 1, 30], [3000, 700, 500], 8, 2, 128, 16, dt)
    ws = tq.new_workspace(tq.tq_paged_attention_workspace_bytes(32, 8, 2, 128, 3, 30, 3000), dev)
    own, kept = c.run(), c.run(workspace=ws)
    again = c.run()
    for a, b, d in zip(own, kept, again):
        assert torch.equal(a, b) and torch.equal(a, d)
    d = [t.to(dev) for t in (c.q, c.k, c.v, c.table, c.cu, c.kv)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tq.tq_paged_attention(*d, 30, 3000)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = tq.tq_paged_attention(*d, 30, 3000, return_lse=True)
    for i in range(4):
        out.fill_(0), lse.fill_(0)
        torch.randn(1000, device=dev).sum()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, own[0]) and torch.equal(lse, own[1]), f"replay {i}"
