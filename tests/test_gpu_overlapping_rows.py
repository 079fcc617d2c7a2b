"""Row offsets are device data and not trusted: where they go back, sequences overlap and ask for
more units than the call has. Here the overlapping sequences are the same one, so that whoever
writes a row writes the right one. Bounds as in the parity tests of the two operators."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import test_gpu_paged_append as append
import test_gpu_paged_attention as attention

pytestmark = pytest.mark.gpu


def repeated(s, times, dev):
    """The sequence of s, with rows 0 .. T - 1, `times` times over: offsets 0, T, 0, T, ..."""
    n = 2 * times - 1
    return dict(block_table=s.table.repeat(n, 1), seq_lens=s.seq_lens.repeat(n),
                cu_q=torch.tensor([0, s.T] * times, dtype=torch.int32, device=dev))


@pytest.mark.parametrize("cus", [0, 8])
@pytest.mark.parametrize("new,len,Hq,Hkv,D,P,window", [(8, 3000, 4, 2, 128, 64, 0), (1, 9000, 4, 1, 64, 16, 0), (40, 2000, 8, 2, 128, 128, 0),
                                                       (3, 5000, 16, 4, 256, 32, 900)])
def test_attention(cuda_device, new, len, Hq, Hkv, D, P, window, cus):
    s = attention.Setup(cuda_device, [new], [len], Hq, Hkv, D, P, seed=50)
    ref = s.reference(window)
    workspace = fg.make_attention_workspace()
    lse = torch.zeros(s.T, Hq, device=cuda_device)
    fg.set_num_cus(cus)
    try:
        for times in (1, 3, 40, 200):
            out = fg.paged_attention(s.q, s.cache, **repeated(s, times, cuda_device), lse=lse.fill_(float("nan")), softmax_scale=s.scale,
                                     window=window, workspace=workspace)
            torch.cuda.synchronize()
            s.check(out, lse, window, ref)
            assert int(workspace[: 64 << 10].count_nonzero()) == 0
        s.check(*s.run(window=window, workspace=workspace), window, ref)
    finally:
        fg.set_num_cus(0)


@pytest.mark.parametrize("times", [3, 200])
def test_append(cuda_device, times):
    s = append.Setup(cuda_device, [70], [70], 4, 2, 128, 32, seed=51)
    rot = append.table_of(70, 64, cuda_device)
    s.before = [t.clone() for t in s.cache]
    out = fg.rope_append_paged_kv(s.q, s.k, s.v, rot, s.cache, **repeated(s, times, cuda_device))
    torch.cuda.synchronize()
    s.check(out, rot)
