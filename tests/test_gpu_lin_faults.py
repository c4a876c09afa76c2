"""Tables of the decayed linear attention that do not fit their buffers: what is reported, and what is still right."""
import pytest
import torch

import kda_linear_attention_02_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,table,status", [
    ([63, 0, 40], [0, 0, 0, 0], 0),            # no sequence reaches a checkpoint
    ([63, 130, 40], [0, 0, 0, 0], -7),         # one does, and the table has no place for it
    ([63, 130, 40], [0, 0, 2, 2], -7),         # the table has places, the buffer none
    ([900, 3000], [0, 14, 60], -7)])           # cut into segments
def test_empty_checkpoints(dtype, lens, table, status):
    H, d, T = 2, 64, sum(lens)
    g = torch.Generator(DEV)
    g.manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q, k, v = (0.1 * r(T, H, d)).to(dtype), (0.1 * r(T, H, d)).to(dtype), r(T, H, d).to(dtype)
    la, cu = -0.1 * r(T, H).abs(), ints([sum(lens[:i]) for i in range(len(lens) + 1)])
    outs = []
    for kw in ({}, dict(ckpt_stride=64, checkpoints=torch.empty(0, H, d, d, device=DEV), ckpt_cu=ints(table))):
        o, fs = torch.empty_like(v), torch.empty(len(lens), H, d, d, device=DEV)
        kda.kda_lin_chunk_fwd(q, k, v, la, None, cu, o, fs, **kw)
        torch.cuda.synchronize()
        assert kda.kda_get_device_status() == (status if kw else 0)
        outs.append((o, fs))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
