"""Block scales that are none: w4a16_moe reports them on either route, so
that what a caller hears does not depend on how many tokens share the call."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests.test_gpu_moe import check, make, on_gpu

pytestmark = pytest.mark.gpu
BAD = nv.Status.ERR_NONFINITE


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


# few pairs of either row length; FP4 route with scales of a unit at once, of
# odd rows, and of a stage at a time
@pytest.mark.parametrize("M,k,H,I", [(2, 1, 512, 256), (2, 1, 272, 336), (48, 2, 512, 256), (48, 2, 272, 336),
                                     (48, 2, 4352, 64)])
def test_status(M, k, H, I):
    E = 4
    x, ids, w, w13, w2 = make(M, E, k, H, I, seed=4)
    ids[:] = torch.arange(M * k, dtype=torch.int32).view(M, k) % 3  # expert 3 is not read
    ws = torch.empty(nv.w4a16_moe_workspace_bytes(M, k, H, I), dtype=torch.uint8, device="cuda")
    e_read = int(ids[-1, -1])
    for at, e, byte, status in ((1, e_read, 0x85, BAD), (2, e_read, 0x81, BAD), (1, e_read, 0xFE, BAD),
                                (2, e_read, 0xB8, BAD), (1, e_read, 0x7F, BAD), (2, e_read, 0xFF, BAD),
                                (1, 3, 0x85, nv.Status.OK), (2, 3, 0xC0, nv.Status.OK),
                                (1, e_read, 0x80, nv.Status.OK), (2, e_read, 0x80, nv.Status.OK),
                                (1, e_read, 0x7E, nv.Status.OK), (2, e_read, 0x01, nv.Status.OK)):
        for row, block in ((3, 5 if at == 1 else 1), ((2 * I if at == 1 else H) - 1, -1), (0, 0)):
            args = [x, ids, w, list(w13), list(w2)]
            s = args[2 + at][1].clone().view(torch.uint8)
            s[e, row, block] = byte
            args[2 + at][1] = s.view(torch.float8_e4m3fn)
            out = nv.w4a16_moe(*on_gpu(*args), workspace=ws)
            assert nv.nvfp4_read_device_status(ws) == status, (at, e, hex(byte), row)
            if byte == 0x80:  # a zero
                check(out, args)
