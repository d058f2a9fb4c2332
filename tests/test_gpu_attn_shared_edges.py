"""ssd_verify_attn_shared: what its workspace holds, and numbers of tokens around those of a row tile and of a pair."""
import pytest
import torch

from speculative_decoding_copy_gb300 import _binding as S
from test_gpu_attn_shared import DEV, Case

pytestmark = pytest.mark.gpu


def _size(B, NB, Dmax, Hq, Hkv, dh, dtype, S_max=8192, P_max=500):
    p = 1 << 40
    a = S.AttnSharedArgs(*[p + (i << 36) for i in range(11)], None, None, dtype, dtype, B, NB, Dmax, Hq, Hkv, dh, 0, 0, 0.0, S_max, P_max, B)
    return S.ssd_verify_attn_shared_workspace_size(a)


@pytest.mark.parametrize("B,NB,Dmax,Hq,Hkv,dh,f32", [(64, 1, 1, 32, 8, 128, False), (4096, 1, 1, 32, 8, 128, False), (512, 1, 5, 14, 2, 64, False), (32, 9, 16, 32, 8, 128, False),
                                                     (1, 1, 1, 64, 1, 128, False), (300, 1, 2, 5, 1, 64, True), (7, 1, 26, 10, 2, 64, False)])
def test_workspace_holds_the_rows_that_there_can_be(B, NB, Dmax, Hq, Hkv, dh, f32):
    sms = torch.cuda.get_device_properties(0).multi_processor_count * (4 if f32 else 1)
    G, NT = Hq // Hkv, NB * Dmax
    per = 128 // G
    rows = lambda n: n * G if n <= per else 256
    parts = lambda n: -(-n // (2 * per)) * Hkv
    most = 4 * (dh + 2) * ((parts(B * NT) + sms) * rows(B * NT) + (B * parts(NT) + sms) * rows(NT))
    most += 4 * (B * NT + 4 * (B + 1)) + 16 * 256              # lists of tokens and sequences, the plan, each at 256 bytes
    assert 0 < _size(B, NB, Dmax, Hq, Hkv, dh, S.SSD_F32 if f32 else S.SSD_BF16) <= most


@pytest.mark.parametrize("dh,paged,f32", [(128, False, False), (64, True, False), (128, False, True)])
@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("G,n", [(1, 127), (1, 128), (1, 129), (5, 24), (5, 25), (5, 26), (5, 51), (8, 16), (8, 17), (8, 33), (64, 1), (64, 2), (64, 3), (3, 42), (3, 43)])
def test_tokens_around_a_row_tile(G, n, B, dh, paged, f32):
    """One sequence's tokens fill a row tile, nearly or just not; those of all together one more tile, or not."""
    blk = [[n]] + [[max(n - 2, 0)]] * (B - 1)
    c = Case(31, S_len=400, own=([300, 17, 129] * B)[:B], NB=1, Dmax=n, G=G, Hkv=2, dh=dh, paged=paged, f32=f32, blk=blk)
    args, tables = c.device()
    size = S.ssd_verify_attn_shared_workspace_size(S.attn_shared_args(*args, c.Dmax, args[0], **tables))
    buf = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    buf[256:512] = 0                                           # the workspace's header
    c.check(c.run(ws=buf[256:256 + size]))
    assert (buf[:256] == 0xA5).all() and (buf[256 + size:] == 0xA5).all()
    assert S.ssd_read_device_error(buf[256:256 + size]) == S.SSD_OK
