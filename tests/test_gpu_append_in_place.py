"""msa_append_cache with q_out = q and iq_out = iq, through the C ABI (the
Python call always gives new outputs): the same bits as out of place."""
import ctypes as C

import pytest
import torch

from gpu_common import msa
from test_gpu_append import New

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dim,idim,inter", [(128, 64, False), (64, 32, False), (96, 48, True), (0, 0, False)])
@pytest.mark.parametrize("seqs,H,G", [([(5, 50), (1, 9)], 2, 3), ([(700, 700), (1500, 1700), (3, 3)], 4, 16), ([(2300, 2300)], 8, 5)])
def test_queries_rotated_in_place(seqs, H, G, dim, idim, inter, int8):
    """A few rows (one a CTA) and thousands (several a CTA, the next row's loads ahead of this one's stores)."""
    m = msa()
    x = New(seqs, H, G, int8, 64, seed=dim)
    rope = m.Rope(dim, idim, interleaved=inter) if dim else None
    q, iq = x.run(rope)
    caches = [t.clone() for t in (x.kc, x.vc, x.ikc)]
    mine, imine = x.q.contiguous(), x.iq.contiguous()
    pb = x.pb
    a = m.MsaAppend(x.k.data_ptr(), x.v.data_ptr(), x.ik.data_ptr(), mine.data_ptr(), imine.data_ptr(),
                    x.k.stride(0), x.v.stride(0), x.ik.stride(0), H * G * 128, H * 64,
                    x.kc.data_ptr(), x.vc.data_ptr(), x.ikc.data_ptr(), pb.c.k_scale, pb.c.v_scale,
                    mine.data_ptr(), imine.data_ptr())
    r = C.byref(rope._struct(None)) if rope is not None else None
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    assert m.lib().msa_append_cache(C.byref(pb.c), C.byref(a), r, C.c_void_p(ws.data_ptr()), 256,
                                    C.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert m.error_word(ws) == 0
    assert torch.equal(mine, q) and torch.equal(imine, iq)
    assert all(torch.equal(now, then) for now, then in zip((x.kc, x.vc, x.ikc), caches))
